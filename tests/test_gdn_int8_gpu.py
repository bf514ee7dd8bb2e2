"""The gated delta rule's step on int8 entries, with numbers that its codes cannot hold and in captured graphs."""
import numpy as np
import pytest

import gdn_ref as ref
from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import f64, to_dev, to_i32
from test_gdn_gpu import FULL, SHAPES, _store_views, ids, states

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    bld.build()
    bd.lib()
    torch.cuda.set_device(0)


def _entry(shape, desc, seed):
    import torch
    store, codes, scales = _store_views(shape, desc, 1)
    sc, co = ref.int8_codes(wl.upcast(states(seed, shape, 1, wl.F32), wl.F32))
    codes.copy_(torch.from_numpy(co))
    scales.copy_(torch.from_numpy(sc))
    return store, codes, scales


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_a_state_that_codes_cannot_hold_reads_as_nan(shape, bad):
    """A value that is not finite reaches every column of its row (even a key's zero, times infinity, is NaN).  They
    read as NaN afterwards, since a symmetric grid of an infinite maximum holds nothing, and stay so; the other heads
    are what they are without it."""
    import torch
    H, P = shape.nheads, shape.head_dim
    desc = bd.layer_desc(shape)
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(60, shape))
    xbc, raw, beta = ref.inputs(60, shape, (2, 1), wl.BF16)
    x = to_dev(xbc, wl.BF16)[:, 0]
    row = min(5, P - 1)
    held = []
    for poison in (False, True):
        store, codes, scales = _entry(shape, desc, 60)
        y = torch.zeros(2, H * P, dtype=torch.bfloat16, device="cuda")
        z = x.clone()
        if poison:
            z[0, row] = bad  # a value of head 0
        states_after = []
        for t in range(2):
            bd.gdn_state_update_int8(desc, store, to_i32([0]), z[t:t + 1], to_dev(raw, wl.F32)[t], to_dev(beta, wl.F32)[t], A,
                                     y[t:t + 1], dt_bias=bias)
            states_after.append(f64(codes[0]) * f64(scales[0])[:, None])
        held.append((states_after, f64(y).reshape(2, H, P)))
    (good, good_y), (got, got_y) = held
    for t in range(2):
        np.testing.assert_array_equal(got[t][1:], good[t][1:])  # the other heads
        np.testing.assert_array_equal(got_y[t][1:], good_y[t][1:])
    assert np.isnan(got[0][0]).all()
    assert not np.isfinite(got_y[0][0][row]) and np.isfinite(np.delete(got_y[0][0], row)).all()
    assert np.isnan(got[1][0]).all() and np.isnan(got_y[1][0]).all()


def test_a_nan_gate_leaves_nothing_that_reads_as_a_number():
    import torch
    desc = bd.layer_desc(FULL)
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(61, FULL))
    xbc, raw, beta = ref.inputs(61, FULL, (1,), wl.BF16)
    store, codes, scales = _entry(FULL, desc, 61)
    r = to_dev(raw, wl.F32)
    r[0, 2] = float("nan")
    y = torch.zeros(1, 512, dtype=torch.bfloat16, device="cuda")
    bd.gdn_state_update_int8(desc, store, to_i32([0]), to_dev(xbc, wl.BF16), r, to_dev(beta, wl.F32), A, y, dt_bias=bias)
    S = f64(codes[0]) * f64(scales[0])[:, None]
    assert np.isnan(S[2]).all() and np.isfinite(S[[0, 1, 3]]).all()
