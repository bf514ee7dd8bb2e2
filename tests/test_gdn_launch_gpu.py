"""The gated delta rule's calls in captured graphs and with programmatic dependent launch off: the same bytes."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest

import gdn_ref as ref
from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import to_dev, to_i32
from test_gdn_gpu import FULL, _store_views, _vkq, _work, states

pytestmark = pytest.mark.gpu

TESTS = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(TESTS)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    bld.build()
    bd.lib()
    torch.cuda.set_device(0)


def replays(call, buffers, times):
    """The buffers after `times` eager calls and after as many replays of the call captured, both from what they hold."""
    import torch
    start = [b.clone() for b in buffers]
    for _ in range(times):
        call()
    torch.cuda.synchronize()
    eager = [b.clone() for b in buffers]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for b, s in zip(buffers, start):
        b.copy_(s)
    for _ in range(times):
        graph.replay()
    torch.cuda.synchronize()
    return start, eager, buffers


@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_the_scan_in_a_graph(st):
    import torch
    lens = [150, 1, 333]
    T = sum(lens)
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(70, FULL))
    x, r, b = (to_dev(a, d) for a, d in zip(ref.inputs(70, FULL, (T,), wl.BF16), (wl.BF16, wl.F32, wl.F32)))
    vkq = [t.contiguous() for t in _vkq(FULL, x)]
    pool, y = to_dev(states(70, FULL, 9, st), st), torch.zeros(T, 4, 128, dtype=torch.bfloat16, device="cuda")
    work, cu, slots = _work(FULL, T, 3, st, wl.BF16), to_i32(wl.cu_seqlens(lens)), to_i32([0, 1, 2])
    ckpt, one = to_i32([[3, 4], [-1, -1], [5, 6]]), torch.ones(3, dtype=torch.uint8, device="cuda")
    call = lambda: bd.gdn_chunk_scan(bd.layer_desc(FULL, state=st), pool, cu, slots, *vkq, r, b, A, y, work, dt_bias=bias,  # noqa: E731
                                     has_initial_state=one, ckpt_slots=ckpt, ckpt_interval=64)
    start, eager, got = replays(call, [pool, y], 3)
    for s, e, g in zip(start, eager, got):
        assert torch.equal(e, g) and not torch.equal(e, s)


def test_the_int8_step_in_a_graph():
    import torch
    desc = bd.layer_desc(FULL)
    store, codes, scales = _store_views(FULL, desc, 5)
    codes.copy_(torch.randint(-127, 128, codes.shape, device="cuda"))
    scales.fill_(0.01)
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(71, FULL))
    x, r, b = (to_dev(a, d) for a, d in zip(ref.inputs(71, FULL, (4,), wl.BF16), (wl.BF16, wl.F32, wl.F32)))
    y, entries = torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda"), to_i32([4, -1, 0, 2])
    call = lambda: bd.gdn_state_update_int8(desc, store, entries, x, r, b, A, y, dt_bias=bias)  # noqa: E731
    start, eager, got = replays(call, [store, y], 3)
    for s, e, g in zip(start, eager, got):
        assert torch.equal(e, g) and not torch.equal(e, s)


CHILD = textwrap.dedent("""
    import sys
    import numpy as np
    import torch
    sys.path[:0] = [{root!r}, {tests!r}]
    import gdn_ref as ref
    from recurrent_state_update_gb300 import binding as bd, build as bld, workloads as wl
    from gpu_util import to_dev, to_i32
    from test_gdn_gpu import FULL, _store_views, _vkq, _work, states
    bld.build()
    torch.cuda.set_device(0)
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(72, FULL))
    lens = [700, 64, 129]
    T = sum(lens)
    x, r, b = (to_dev(a, d) for a, d in zip(ref.inputs(72, FULL, (T,), wl.BF16), (wl.BF16, wl.F32, wl.F32)))
    vkq = [t.contiguous() for t in _vkq(FULL, x)]
    kept = []
    for st in (wl.BF16, wl.F32):  # prompts, single tokens, drafts and steps on entries, back to back on one stream
        desc = bd.layer_desc(FULL, state=st)
        pool, y = to_dev(states(72, FULL, 20, st), st), torch.zeros(T, 4, 128, dtype=torch.bfloat16, device="cuda")
        bd.gdn_chunk_scan(desc, pool, to_i32(wl.cu_seqlens(lens)), to_i32([0, 1, 2]), *vkq, r, b, A, y,
                          _work(FULL, T, 3, st, wl.BF16), dt_bias=bias)
        kept.append(y)
        for t in range(3):
            y = torch.zeros(3, 1, 512, dtype=torch.bfloat16, device="cuda")
            bd.gdn_state_update(desc, pool, to_i32([0, 1, 2]), x[None, 3 * t:3 * t + 3].transpose(0, 1).contiguous(),
                                r[3 * t:3 * t + 3, None], b[3 * t:3 * t + 3, None], A, y, dt_bias=bias)
            kept.append(y)
        y = torch.zeros(3, 4, 512, dtype=torch.bfloat16, device="cuda")
        bd.gdn_state_update(desc, pool, to_i32([0, 1, 2]), x[:12].view(3, 4, -1), r[:12].view(3, 4, -1), b[:12].view(3, 4, -1), A, y,
                            dt_bias=bias, scratch_slots=to_i32(np.arange(3, 15).reshape(3, 4)))
        store = _store_views(FULL, desc, 3)[0]
        bd.mamba_ckpt_store_int8(desc, pool, to_i32([0, 1, 2]), to_i32([2, 0, 1]), store)
        for t in range(3):
            z = torch.zeros(3, 512, dtype=torch.bfloat16, device="cuda")
            bd.gdn_state_update_int8(desc, store, to_i32([2, 0, 1]), x[20 + t:23 + t], r[20 + t:23 + t], b[20 + t:23 + t], A, z, dt_bias=bias)
            kept.append(z)
        kept += [y, pool, store]
    torch.cuda.synchronize()
    np.savez({path!r}, *[t.contiguous().view(torch.uint8).cpu().numpy() for t in kept])
""")


def test_results_identical_with_and_without_dependent_launch(tmp_path):
    outs = {}
    for pdl in ("1", "0"):
        path = str(tmp_path / f"pdl{pdl}.npz")
        r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, tests=TESTS, path=path)], capture_output=True, text=True,
                           env=dict(os.environ, MAMBA_PDL=pdl), timeout=600)
        assert r.returncode == 0, r.stderr[-3000:]
        outs[pdl] = np.load(path)
    assert len(outs["1"].files) == len(outs["0"].files) == 20
    for k in outs["1"].files:
        np.testing.assert_array_equal(outs["1"][k], outs["0"][k], err_msg=k)
