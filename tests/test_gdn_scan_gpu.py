"""The gated delta rule's scan where its number formats, plan and launches are strained, through the binding.

Tolerances are those of test_gdn_gpu.py, whose helpers compare every 64-token tile of the outputs, every final state
and every checkpoint with the 64-bit form."""
import numpy as np
import pytest

import gdn_ref as ref
from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import f64, to_dev, to_i32
from test_gdn_gpu import FULL, _vkq, _work, states

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    bld.build()
    bd.lib()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
@pytest.mark.parametrize("inner", [(2**31 - 1, -2**31, -1), (-2**31, -1, 5), (2**31 - 1, 2**31 - 1, 2**31 - 1)])
def test_boundaries_whose_differences_wrap_are_refused(st, inner):
    """Every difference of (0, 2^31 - 1, -2^31, -1, T) is non-negative in 32 bits."""
    import torch
    T = 90
    xbc, raw, beta = ref.inputs(50, FULL, (T,), wl.BF16)
    before = to_dev(states(50, FULL, 5, st), st)
    pool = before.clone()
    y = torch.full((T, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.gdn_chunk_scan(bd.layer_desc(FULL, state=st), pool, to_i32([0, *inner, T]), to_i32([0, 1, 2, 3]),
                      *[t.contiguous() for t in _vkq(FULL, to_dev(xbc, wl.BF16))], to_dev(raw, wl.F32), to_dev(beta, wl.F32),
                      to_dev(ref.layer(50, FULL)[0], wl.F32), y, _work(FULL, T, 4, st, wl.BF16), err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == bd.MAMBA_ERR_SEQLENS
    assert torch.equal(pool, before) and (y == 7.0).all()
