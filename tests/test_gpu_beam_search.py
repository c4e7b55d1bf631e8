"""Beam search over the paged cache: prefill of the prompts, then per step attention of all beams behind their shared
prompt (pa_varlen_cascade), selection (pa_beam_select), reordering (pa_beam_reorder) and the write of the new tokens'
keys and values, with the pool following by the same rule.  A one-layer toy model in 64 bits does the same search over
whole token sequences, without cache, blocks or sharing."""
import numpy as np
import pytest
import torch

import paged_kv_cache_75_gb300 as pk

pytestmark = pytest.mark.gpu

H, HKV, D, BS, V = 8, 2, 128, 16, 211


class Toy:
    """Embeddings to queries, keys and values in bf16; logits from the attention's output."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.q = n(V, H, D).bfloat16()
        self.k = n(V, HKV, D).bfloat16()
        self.v = n(V, HKV, D).bfloat16()
        self.out = n(H * D, V) * 0.06

    def logits64(self, tokens):
        """Of the last token of a sequence, in 64 bits."""
        t = torch.tensor(tokens)
        q = self.q[t[-1]].double().view(HKV, H // HKV, D)
        s = torch.einsum("hgd,nhd->hgn", q, self.k[t].double()) * D ** -0.5
        o = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), self.v[t].double())
        return o.reshape(-1) @ self.out.double()


def search64(toy, prompt, width, steps):
    """[(score, tokens)] best first, and how near a step's choice was."""
    beams, margin = [(0.0, list(prompt))], float("inf")
    for _ in range(steps):
        found = []
        for i, (score, tokens) in enumerate(beams):
            lp = torch.log_softmax(toy.logits64(tokens), 0) + score
            found += [(-float(x), i, t) for t, x in enumerate(lp)]
        found.sort()
        margin = min([margin] + [found[i + 1][0] - found[i][0] for i in range(width)])
        beams = [(-s, beams[i][1] + [t]) for s, i, t in found[:width]]
    return beams, margin


@pytest.mark.parametrize("width,prompts", [(4, (50, 16, 33)), (3, (32, 1)), (8, (100,)), (1, (20, 47))])
def test_beam_search(width, prompts):
    steps, R = 23, len(prompts)
    toy = Toy(width)
    rng = np.random.default_rng(width)
    text = [rng.integers(0, V, n).tolist() for n in prompts]
    dev = lambda a, t=torch.int32: torch.tensor(a, dtype=t, device="cuda")  # noqa: E731
    tq, tk, tv, w_out = toy.q.cuda(), toy.k.cuda(), toy.v.cuda(), toy.out.cuda()
    blocks = 400
    pool = pk.BlockPool(blocks, BS, free_order=rng.permutation(blocks).tolist())
    kc = torch.full((blocks, HKV, BS, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    cache, status = pk.KVCache(kc, vc), torch.zeros(1, dtype=torch.int32, device="cuda")
    layers = pk.KVLayers([cache])
    width_blocks = (max(prompts) + steps) // BS + 1

    # the prompts, all but their last token, then that one as the first "selected" token
    slots, ids = [], []
    for r, t in enumerate(text):
        pool.add_seq(r)
        s, _ = pool.append(r, len(t))
        slots += s
        ids += t
    pk.pa_kv_cache_write(cache, tk[dev(ids).long()], tv[dev(ids).long()], dev(slots, torch.int64), status)
    seqs = [[r] for r in range(R)]
    table, lens = pool.block_table(list(range(R)), width_blocks)
    table, lens = dev(table), dev(lens)
    tokens, scores, counts = dev([t[-1] for t in text]), torch.zeros(R, device="cuda"), [1] * R
    shared = [(len(t) // BS) * BS - (BS if len(t) % BS == 0 else 0) for t in text]  # whole blocks before every query
    spare = pool.reserve(R * width)
    next_id = 100
    history = [[list(t)] for t in text]
    for step in range(steps):
        n = sum(counts)
        cu = np.concatenate([[0], np.cumsum(counts)])
        q, out = tq[tokens.long()], torch.empty(n, H, D, dtype=torch.bfloat16, device="cuda")
        max_k = max(prompts) + step
        cu_k = torch.cat([dev([0]), lens.cumsum(0, dtype=torch.int32)])
        ws = torch.empty(pk.pa_varlen_cascade_workspace_size(n, n, H, HKV, D, 1, max_k, max(shared), BS) + 16, dtype=torch.uint8,
                         device="cuda")
        pk.pa_varlen_cascade(out, q, cache, table, dev(list(range(n + 1))), cu_k, 1, max_k, D ** -0.5, dev(cu.tolist()),
                             dev(shared), max(counts), max(shared), ws, status)
        logits = out.float().flatten(1) @ w_out
        best = (torch.empty(R, width, device="cuda"), torch.empty(R, width, dtype=torch.int32, device="cuda"),
                torch.empty(R, width, dtype=torch.int32, device="cuda"))
        ws = torch.empty(pk.pa_beam_select_workspace_size(n, V, width), dtype=torch.uint8, device="cuda")
        pk.pa_beam_select(*best, logits, scores, dev(cu.tolist()), workspace=ws, dev_status=status)
        scores, parents, tokens = best[0].flatten(), best[1].flatten(), best[2].flatten()
        m = R * width
        t2 = torch.empty(m, width_blocks, dtype=torch.int32, device="cuda")
        l2, used = torch.empty(m, dtype=torch.int32, device="cuda"), torch.empty(m, dtype=torch.int32, device="cuda")
        s2 = torch.empty(m, dtype=torch.int64, device="cuda")
        pk.pa_beam_reorder(layers, parents, table, lens, dev(spare), t2, l2, s2, used, status)
        pk.pa_kv_cache_write(cache, tk[tokens.long()], tv[tokens.long()], s2, status)
        table, lens = t2, l2
        # the pool follows
        par, chosen = parents.tolist(), tokens.tolist()
        old = [s for g in seqs for s in g]
        new = list(range(next_id, next_id + m))
        next_id += m
        got, took = pool.reorder(old, new, par, spare)
        assert got == s2.tolist() and took == [bool(u) for u in used.tolist()]
        assert pool.block_table(new, width_blocks) == (table.tolist(), lens.tolist())
        spare = [b for b, u in zip(spare, took) if not u] + pool.reserve(sum(took))
        seqs = [new[r * width:(r + 1) * width] for r in range(R)]
        flat = [h for g in history for h in g]
        history = [[flat[par[r * width + i]] + [chosen[r * width + i]] for i in range(width)] for r in range(R)]
        counts = [width] * R
    torch.cuda.synchronize()
    assert int(status) == 0
    for r in range(R):
        want, margin = search64(toy, text[r], width, steps)
        got = scores[r * width:(r + 1) * width].tolist()
        if margin > 0.02:  # bf16 outputs: logits off by about 0.06 * sqrt(1024) * 2^-9 * |o| a step
            assert [h for h in history[r]] == [t for _, t in want]
        # each beam's score is its own tokens', within the outputs' rounding of every step
        for h, s in zip(history[r], got):
            total = 0.0
            for i in range(len(text[r]), len(h)):
                total += float(torch.log_softmax(toy.logits64(h[:i]), 0)[h[i]])
            assert abs(total - s) < 0.02 * steps
        assert got == sorted(got, reverse=True)
    # everything goes back
    for g in seqs:
        for s in g:
            pool.free_seq(s)
    pool.unreserve(spare)
    assert pool.num_free() == blocks
