"""A gated delta rule layer served end to end (examples/gdn_layer.py) against 64 bits: convolution, prefill, single
tokens, drafts and their commit, and the 8-bit cache.

Tolerances, as errors over a request's largest output (one token's alone can all but cancel: where k q is near zero
the rounding of its channels is a third of what is left) or a head's state's largest value.  fp32: 1e-4, the kernels' own.  bf16 state and
activations: a state is rounded at most once a call and channels once, so at most 10 roundings of 2^-8 of the value
each: 4e-2 at the outside; half of it is asked, as roundings are 2^-9 on average and of either sign."""
import importlib.util
import os

import numpy as np
import pytest

import gdn_ref as ref
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import f64, tile_rel_err, to_dev

pytestmark = pytest.mark.gpu

PROMPT, DECODE, ACCEPT, TAIL, SPEC = (150, 64, 1), 2, (2, 3, 0), 1, 3


@pytest.fixture(scope="module")
def example():
    import torch
    bld.build()
    torch.cuda.set_device(0)
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gdn_layer.py")
    spec = importlib.util.spec_from_file_location("gdn_layer", at)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def convolved(x, w):
    """Causal convolution and SiLU of channels (T, C) from an empty window: tap W - 1 meets the newest."""
    W = w.shape[1]
    padded = np.concatenate([np.zeros((W - 1, x.shape[1])), x])
    return ref.silu(sum(padded[j:j + len(x)] * w[:, j] for j in range(W)))


@pytest.mark.parametrize("dtype,bound", [(wl.F32, 1e-4), (wl.BF16, 2e-2)])
@pytest.mark.parametrize("heads,head_dim,d_state,groups", [(4, 128, 128, 2), (4, 64, 128, 1), (3, 32, 64, 3)])
def test_a_layer_served(example, dtype, bound, heads, head_dim, d_state, groups):
    import torch
    shape = wl.LayerShape(heads, head_dim, d_state, groups, conv_kernel=4, num_spec=SPEC)
    n = len(PROMPT)
    layer = example.GatedDeltaLayer(shape, slots=n * (1 + SPEC), entries=n, state=dtype, act=dtype, seed=31)
    g, x, dt, beta = wl.rng(31, 5), [], [], []
    bias = layer.dt_bias.cpu().numpy()
    for p in PROMPT:
        T = p + DECODE + SPEC + TAIL
        x.append(wl.store(g.standard_normal((T, shape.conv_dim)), dtype))
        dt.append(wl.store(wl.step_dt(g, bias, (T,), None), wl.F32))
        beta.append(wl.store(g.standard_normal((T, heads)), wl.F32))
    dev = ([to_dev(a, dtype) for a in x], [to_dev(a, wl.F32) for a in dt], [to_dev(a, wl.F32) for a in beta])
    out = example.serve(layer, *dev, PROMPT, DECODE, ACCEPT, 0)
    layer.check()
    conv_w, A = f64(layer.conv_w), f64(layer.A)
    kept = [p + DECODE + a for p, a in zip(PROMPT, ACCEPT)]
    want = []
    for i, T in enumerate(kept):
        v, k, q = ref.split(shape, convolved(wl.upcast(x[i][:T], dtype), conv_w))
        S0 = np.zeros((heads, head_dim, d_state))
        S, y = ref.sequence(S0, v, k, q, dt[i][:T].astype(float), beta[i][:T].astype(float), A, bias.astype(float))
        want.append(S[-1])
        got = f64(out[i]).reshape(y.shape)
        assert got.shape == y.shape
        assert tile_rel_err(got, y, 3) <= bound
        assert tile_rel_err(f64(layer.ssm[i]), S[-1], 2) <= bound

    # the tail on 8 bits: from the state that the entry holds (its rounding is the store's, tested there)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    layer.to_entries(slots, slots)
    layer.from_entries(slots, slots)
    start = f64(layer.ssm)
    H, P, N = heads, head_dim, d_state
    at = (H * P * N + 255) // 256 * 256
    codes = f64(layer.store[:, :H * P * N].view(torch.int8).view(n, H, P, N))
    scales = f64(layer.store[:, at:at + 4 * H * N].view(torch.float32).view(n, H, N))
    held = codes * scales[:, :, None]
    assert np.abs(held - start[:n]).max() <= 2.0 ** -8 * np.abs(held).max()
    step = [torch.stack([t[i][kept[i]:kept[i] + 1] for i in range(n)]) for t in dev]
    y = f64(layer.step_int8(slots, *step)).reshape(n, H, P)
    layer.check()
    for i, T in enumerate(kept):
        v, k, q = ref.split(shape, convolved(wl.upcast(x[i][:T + 1], dtype), conv_w)[-1:])
        S, ye = ref.sequence(held[i], v, k, q, dt[i][T:T + 1].astype(float), beta[i][T:T + 1].astype(float), A, bias.astype(float))
        assert tile_rel_err(y[i], ye[0], 2) <= bound
    layer.from_entries(slots, slots)
    now = f64(layer.ssm[:n])
    for i, T in enumerate(kept):
        top = np.abs(now[i]).max(axis=1, keepdims=True)  # half a grid step, and the new state's own error
        v, k, q = ref.split(shape, convolved(wl.upcast(x[i][:T + 1], dtype), conv_w)[-1:])
        S, _ = ref.sequence(held[i], v, k, q, dt[i][T:T + 1].astype(float), beta[i][T:T + 1].astype(float), A, bias.astype(float))
        assert (np.abs(now[i] - S[0]) <= top * (1 / 254 + 2.0 ** -8) + bound * np.abs(S[0]).max(axis=(1, 2), keepdims=True)).all()


def test_the_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["gdn_layer.py", "--nheads", "4", "--groups", "2"])
    example.main()
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 3 and all("rms difference" in line for line in lines)
