"""Linear attention on states and channels that hold infinities and NaN: which values of a state are infinite, of which sign,
and which are NaN, is what the formula says, but for infinite keys and values in the chunked form, which count as NaN there."""
import numpy as np
import pytest

import la_ref as ref
from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import f64, to_dev, to_i32

pytestmark = pytest.mark.gpu

# e^l rounds up, down and not at all; below 2^-25, and far below what a state can notice
DECAYS = np.array([0.0, -2e-10, -1e-3, -0.01, -0.05, -0.5, -3.0, -75.0], np.float32)
H = len(DECAYS)
SHAPES = [(128, 128), (64, 128), (64, 64), (32, 64), (16, 16)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    bld.build()
    bd.lib()
    torch.cuda.set_device(0)


def spoiled(seed, slots, P, N):
    """States with one infinity of each sign and one NaN a head, none in the first or last row or column."""
    s = wl.rng(seed, 7).standard_normal((slots, H, P, N)).astype(np.float32)
    for h in range(H):
        s[:, h, 1 + h % 4, 2], s[:, h, 5, 1 + h % 7], s[:, h, 7, 11] = np.inf, -np.inf, np.nan
    return s


def same_kind(got, want, tol):
    """Infinite, NaN and finite values each where wanted, the finite ones to tol of a head's largest."""
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and not np.isinf(got[~inf]).any()
    fine = np.isfinite(want)
    assert np.abs(np.where(fine, got, 0) - np.where(fine, want, 0)).max() <= tol * np.abs(want[fine]).max()


@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("ntok", [1, 3])
def test_step_keeps_infinite_states(P, N, ntok):
    import torch
    shape = wl.LayerShape(nheads=H, head_dim=P, d_state=N, n_groups=2)
    before = spoiled(1, 2, P, N)
    xbc = wl.rng(2, 1).standard_normal((2, ntok, shape.conv_dim)).astype(np.float32)
    pool, y = to_dev(before, wl.F32), torch.zeros(2, ntok, H * P, device="cuda")
    bd.la_state_update(bd.layer_desc(shape, state=wl.F32, act=wl.F32), pool, to_i32([1, 0]), to_dev(xbc, wl.F32), to_dev(DECAYS, wl.F32), y)
    v, k, q = ref.split(shape, xbc.astype(np.float64))
    with np.errstate(all="ignore"):
        for i, s in enumerate((1, 0)):
            states, _ = ref.sequence(before[s].astype(np.float64), v[i], k[i], q[i], DECAYS)
            same_kind(f64(pool[s]), states[-1], 1e-4)


def scan(P, N, act, xbc, before):
    import torch
    T, shape = len(xbc), wl.LayerShape(nheads=H, head_dim=P, d_state=N, n_groups=2)
    desc = bd.layer_desc(shape, state=wl.F32, act=act)
    rows = to_dev(wl.store(xbc, act), act)
    v, k, q = ref.split(shape, rows)
    pool, y = to_dev(before, wl.F32), torch.zeros(T, H, P, dtype=rows.dtype, device="cuda")
    work = torch.empty(bd.la_chunk_scan_workspace_bytes(desc, T, 1), dtype=torch.uint8, device="cuda")
    bd.la_chunk_scan(desc, pool, to_i32([0, T]), to_i32([0]), v, k, q, to_dev(DECAYS, wl.F32), y, work,
                     has_initial_state=torch.ones(1, dtype=torch.uint8, device="cuda"))
    v, k, q = ref.split(shape, f64(rows))
    with np.errstate(all="ignore"):
        states, out = ref.sequence(before[0].astype(np.float64), v, k, q, DECAYS)
    return f64(pool[0]), states[-1], f64(y), out


@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("act", [wl.F32, wl.BF16])
@pytest.mark.parametrize("T", [5, 300])
def test_scan_keeps_infinite_states(P, N, act, T):
    xbc = wl.rng(3, 1).standard_normal((T, H * P + 4 * N))
    got, want, _, _ = scan(P, N, act, xbc, spoiled(4, 1, P, N))
    if act == wl.BF16 and P >= 64:  # a chunk's decay that is zero in fp32 makes NaN of an infinity
        gone = np.exp(DECAYS.astype(np.float64) * min(T, 128)) < 2.0 ** -150
        assert gone.sum() == (1 if T == 5 else 2)
        want[np.isinf(want) & gone[:, None, None]] = np.nan
    same_kind(got, want, 1e-4)


@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("act", [wl.F32, wl.BF16])
@pytest.mark.parametrize("T", [40, 300])
def test_scan_of_infinite_channels(P, N, act, T):
    """One infinite value of head 3 and one infinite key of group 1: the state's row and column of it, and no others."""
    g = wl.rng(5, 1)
    xbc = g.standard_normal((T, H * P + 4 * N))
    xbc[T // 3, 3 * P + 6] = np.inf
    xbc[T // 2, H * P + N + 9] = -np.inf
    got, want, y, out = scan(P, N, act, xbc, g.standard_normal((1, H, P, N)).astype(np.float32))
    chunked = act == wl.BF16 and P >= 64
    if not chunked:
        same_kind(got, want, 1e-4)
    # (of a head of log decay -75, 0.99 of whose memory is gone with the next token, the formula keeps an infinity as well)
    assert np.array_equal(np.isfinite(got), np.isfinite(want))
    fine = np.isfinite(want)
    assert np.abs(np.where(fine, got, 0) - np.where(fine, want, 0)).max() <= 1e-4 * np.abs(want[fine]).max()
    first = 0 if chunked else T // 3  # (a chunk's earlier outputs of that value are reached too)
    late = np.zeros(out.shape, bool)
    late[first:, 3, 6] = True
    late[T // 2:, H // 2:] = True
    assert np.isfinite(out[~late]).all() and np.isfinite(y[~late]).all()
