"""Batches of sequence groups that share a prefix, and their attention in 64 bits (torch, on the GPU)."""
import numpy as np
import torch

import paged_kv_cache_75_gb300 as pk

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


class Batch:
    """groups: [(shared tokens, [(own keys, queries), ...]), ...]; own keys count the queries' own."""

    def __init__(self, groups, heads, kv_heads, dtype, bs, seed, pad_rows=0, spread=1.0, spare=3, first_id=0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.groups, self.heads, self.kv_heads, self.bs = groups, heads, kv_heads, bs
        self.dtype, self.D, self.scale = DT[dtype], 128, 128 ** -0.5
        members = [m for _, ms in groups for m in ms]
        self.lq = np.array([m[1] for m in members], np.int64)
        self.start = np.array([s for s, ms in groups for _ in ms], np.int64)
        self.lk = self.start + np.array([m[0] for m in members], np.int64)
        self.size = [len(ms) for _, ms in groups]
        self.shared = np.array([s for s, _ in groups], np.int64)
        have = -(-self.lk // bs)
        width = max(1, int(have.max()) + 1)
        total = int(sum(s // bs for s in self.shared) + (have - self.start // bs).sum())
        ids = (rng.permutation(total + spare) + first_id).astype(np.int32)
        table, at, b = np.full((len(members), width), -1, np.int32), 0, 0
        for s, ms in groups:
            pre = ids[at:at + s // bs]
            at += s // bs
            for _ in ms:
                table[b, :s // bs] = pre
                n = int(have[b]) - s // bs
                table[b, s // bs:have[b]] = ids[at:at + n]
                at += n
                b += 1
        self.table = table
        self.used = ids[:at] - first_id
        shape = (total + spare, kv_heads, bs, self.D)
        self.k = torch.randn(shape, generator=g).to(self.dtype)
        self.v = torch.randn(shape, generator=g).to(self.dtype)
        self.first_id = first_id
        # what no sequence holds may be anything: unused blocks, positions behind a sequence's last
        hidden = torch.ones(shape[0], bs, dtype=torch.bool)
        for b in range(len(members)):
            for j in range(int(have[b])):
                hidden[table[b, j] - first_id, :min(bs, int(self.lk[b]) - j * bs)] = False
        for x in (self.k, self.v):
            x.permute(0, 2, 1, 3)[hidden] = float("nan")
        self.q = (spread * torch.randn(int(self.lq.sum()) + pad_rows, heads, self.D, generator=g)).to(self.dtype)

    def device(self):
        self.kc, self.vc, self.qd = self.k.cuda(), self.v.cuda(), self.q.cuda()
        self.cache = pk.KVCache(self.kc, self.vc)
        cum = lambda a: torch.from_numpy(np.concatenate([[0], np.cumsum(a)]).astype(np.int32)).cuda()  # noqa: E731
        self.cu_q, self.cu_k, self.cu_g = cum(self.lq), cum(self.lk), cum(self.size)
        self.tab = torch.from_numpy(self.table).cuda()
        self.sh = torch.from_numpy(self.shared.astype(np.int32)).cuda()
        return self

    def bounds(self):
        return dict(max_q=int(self.lq.max(initial=0)), max_k=int(self.lk.max(initial=0)), max_group=max(self.size),
                    max_shared=int(self.shared.max()))

    def workspace(self, **more):
        b = {**self.bounds(), **more}
        n = pk.pa_varlen_cascade_workspace_size(len(self.lk), self.q.shape[0], self.heads, self.kv_heads, self.D, b["max_q"],
                                                b["max_k"], b["max_shared"], self.bs)
        # whatever it holds
        return torch.full((max(n, 16),), 0xff, dtype=torch.uint8, device="cuda")

    def call(self, out, ws, status, **more):
        b = {**self.bounds(), **more}
        pk.pa_varlen_cascade(out, self.qd, self.cache, self.tab, self.cu_q, self.cu_k, b["max_q"], b["max_k"], self.scale,
                             self.cu_g, self.sh, b["max_group"], b["max_shared"], ws, dev_status=status)

    def run(self, status=None, **more):
        out = torch.full_like(self.qd, 7.0)
        st = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
        self.call(out, self.workspace(**more), st, **more)
        torch.cuda.synchronize()
        if status is None:
            assert int(st) == 0
        return out

    def reference(self):
        """Outputs and, row by row, the weighted sum of |v| (float64)."""
        n, per = int(self.lq.sum()), self.heads // self.kv_heads
        ref = torch.zeros(n, self.heads, self.D, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(ref)
        r = 0
        for b in range(len(self.lk)):
            m, L = int(self.lq[b]), int(self.lk[b])
            if m == 0 or L == 0:
                r += m
                continue
            pos = torch.arange(L, device="cuda")
            blk = (self.tab[b].long()[pos // self.bs] - self.first_id)
            K = self.kc[blk + self.first_id if self.first_id else blk, :, pos % self.bs].double()
            V = self.vc[blk + self.first_id if self.first_id else blk, :, pos % self.bs].double()
            see = pos[None] <= L - m + torch.arange(m, device="cuda")[:, None]
            q = self.qd[r:r + m].double().unflatten(1, (self.kv_heads, per))
            s = torch.einsum("qhgd,nhd->hgqn", q, K) * self.scale
            s = s.masked_fill(~see, -float("inf"))
            w = torch.where(see.any(-1)[:, None], torch.softmax(s, -1), torch.zeros((), dtype=torch.float64, device="cuda"))
            ref[r:r + m] = torch.einsum("hgqn,nhd->qhgd", w, V).flatten(1, 2)
            mag[r:r + m] = torch.einsum("hgqn,nhd->qhgd", w, V.abs()).flatten(1, 2)
            r += m
        return ref, mag

    def check(self, out, rows=None):
        """|out - ref| within what the roundings make.

        With A = sum w |v|: the output's rounding eps/2 |ref|; a weight in 16 bits, 2^-11 A (fp16) or, in two
        truncated parts, 2^-15 A (bf16), and in fp16 2^-25 of the largest weight a key; 128 accumulations of a score
        at 2^-23 of sum |q k| scale <= 12 * spread here move a weight by 1.8e-4 spread, twice (the sum of weights
        too); N accumulations of the values at 2^-23; exponentials and their arguments 1e-5."""
        ref, mag = self.reference()
        n = ref.shape[0]
        N = int(self.lk.max())
        f16 = self.dtype == torch.float16
        lim = torch.finfo(self.dtype).eps / 2 * ref.abs() + mag * ((2.0 ** -11 if f16 else 2.0 ** -15) + 4e-4 + N * 2.0 ** -23)
        if f16:
            lim = lim + N * 2.0 ** -25 * 6 + 2.0 ** -25
        err = (out[:n].double() - ref).abs()
        ok = err <= lim
        if rows is not None:
            ok, err = ok[rows], err[rows]
        assert bool(ok.all()), "%d of %d off, worst %.3g" % (int((~ok).sum()), ok.numel(), float(err.nan_to_num(99.).max()))
        assert bool((out[n:] == 7.0).all())
