"""A linear attention layer served end to end (examples/la_layer.py) against 64 bits: plans, copies of pages, norm and
rotation, prefill in chunks with kept states, a request from a kept state, single tokens from a graph, drafts and
their commit.

Tolerances, as errors over a request's largest output or a head's state's largest value.  fp32: 1e-4, the kernels' own.
bf16 activations: keys, queries and outputs are each rounded once, scores and the state read by the queries once: five
roundings of at most 2^-8 of what they meet, 2e-2.  A bf16 state is rounded once more a call, at most 2 + DECODE + 1 of them, half a
step each on average and of either sign: 3e-2."""
import importlib.util
import os

import numpy as np
import pytest

import la_ref as ref
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import f64, tile_rel_err, to_dev

pytestmark = pytest.mark.gpu

PROMPT, DECODE, DRAFTS, ACCEPT = (300, 127, 1), 4, 3, (2, 3, 0)


@pytest.fixture(scope="module")
def example():
    import torch
    bld.build()
    torch.cuda.set_device(0)
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "la_layer.py")
    spec = importlib.util.spec_from_file_location("la_layer", at)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("state,act,bound", [(wl.F32, wl.F32, 1e-4), (wl.F32, wl.BF16, 2e-2), (wl.BF16, wl.BF16, 3e-2)])
@pytest.mark.parametrize("heads,head_dim,d_state,groups", [(4, 128, 128, 4), (4, 64, 128, 1), (3, 32, 64, 3)])
def test_a_layer_served(example, state, act, bound, heads, head_dim, d_state, groups):
    shape = wl.LayerShape(heads, head_dim, d_state, groups)
    n, B = len(PROMPT), 128
    cols = max(p + DECODE + DRAFTS for p in PROMPT) // B + 1
    layer = example.LinearAttentionLayer(shape, (n + 1) * cols + n * DRAFTS, B, state, act, seed=3)
    g = wl.rng(60, 0)
    x = [wl.store(g.standard_normal((p + DECODE + DRAFTS, shape.conv_dim)), act) for p in PROMPT]
    out, shared, table = example.serve(layer, [to_dev(a, act) for a in x], PROMPT, B, DECODE, DRAFTS, ACCEPT)
    layer.check()
    pool, table = f64(layer.pool), table.cpu().numpy()
    kw, qw, freq = (f64(layer.prep[m]) for m in ("k_weight", "q_weight", "inv_freq"))
    for i, p in enumerate(PROMPT):
        T = p + DECODE + ACCEPT[i]
        v, k, q = ref.split(shape, wl.upcast(x[i][:T], act))
        k, q = (ref.norm_rotate(a, w, 1e-6, np.arange(T), freq) for a, w in ((k, kw), (q, qw)))
        S, y = ref.sequence(np.zeros((heads, head_dim, d_state)), v, k, q, f64(layer.log_decay))
        got = f64(out[i]).reshape(y.shape)
        assert tile_rel_err(got, y, 3) <= bound
        # the page that the drafts were planned to, and those of the blocks that are done
        assert tile_rel_err(pool[table[i, (p + DECODE + DRAFTS - 1) // B]], S[-1], 2) <= bound
        for j in range((p + DECODE) // B):
            assert tile_rel_err(pool[table[i, j]], S[(j + 1) * B - 1], 2) <= bound, (i, j)
        if i == 0:
            assert tile_rel_err(f64(shared).reshape(-1, heads, head_dim), y[B:p], 3) <= bound


def test_the_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["la_layer.py", "--nheads", "4", "--groups", "2"])
    example.main()
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 4 and all("rms difference" in line for line in lines)
