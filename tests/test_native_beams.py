"""The native marshalling of pa_varlen_cascade, pa_beam_select and pa_beam_reorder: what it refuses, and that
nothing runs before its setup.  No GPU."""
import subprocess
import sys

import pytest
import torch

import paged_kv_cache_75_gb300 as pk
from paged_kv_cache_75_gb300 import build as pkg_build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkg_build.build()


def test_refuses_before_setup():
    code = ("import importlib.util as u, sys; s = u.spec_from_file_location('_native', sys.argv[1]); m = u.module_from_spec(s); "
            "s.loader.exec_module(m)\n"
            "for f in (m.beam_select, m.beam_reorder, m.varlen_cascade):\n"
            "    try:\n        f()\n    except RuntimeError:\n        continue\n    raise SystemExit(1)\n"
            "for a in ((), (1, 2, 3), (1, 2, 0, 0, 0)):\n"
            "    try:\n        m.setup_beams(*a)\n    except (TypeError, ValueError):\n        continue\n    raise SystemExit(2)\n")
    assert subprocess.run([sys.executable, "-c", code, pkg_build.NATIVE]).returncode == 0


def test_host_tensors_and_counts():
    n = pk._binding._native()
    for f, k in ((n.beam_select, 11), (n.beam_reorder, 12), (n.varlen_cascade, 18)):
        with pytest.raises(TypeError):
            f(*[None] * (k - 1))
    x = torch.zeros(2, 8)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pk.pa_beam_select(x, i, i, x, x[0], i)
    with pytest.raises(ValueError):
        pk.pa_varlen_cascade(x, x, type("C", (), dict(k_cache=x, v_cache=x, k_scale=1.0, v_scale=1.0)), i, i, i,
                             1, 1, 1.0, i, i, 1, 0, x)
    with pytest.raises(TypeError):
        n.beam_select(x, i, i, "logits", x[0], i, None, None, 0, None, None)
    with pytest.raises(ValueError):
        n.beam_reorder(0, 1, x, *[i] * 8, None)
    with pytest.raises(TypeError):
        pk.pa_beam_reorder(None, *[i] * 8)
