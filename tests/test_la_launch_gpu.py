"""Linear attention's calls and the batch plan in captured graphs, on other streams, twice at once, and with programmatic
dependent launch off: the same bytes.  What an fp32 pool holds to 24 bits; offsets past 2^31."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest

import la_ref as ref
from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import f64, to_dev, to_i32
from test_gdn_launch_gpu import replays

pytestmark = pytest.mark.gpu

TESTS = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(TESTS)
SHAPE = wl.LayerShape(nheads=4, head_dim=128, d_state=128, n_groups=2)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    bld.build()
    bd.lib()
    torch.cuda.set_device(0)


def scan_setup(seed, lens, st, shape=SHAPE, S=12):
    import torch
    T, n = sum(lens), len(lens)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = torch.randn(T, shape.conv_dim, dtype=torch.bfloat16, device="cuda", generator=g)
    desc = bd.layer_desc(shape, state=st)
    pool = 0.1 * torch.randn(S, shape.nheads, shape.head_dim, shape.d_state, device="cuda", generator=g)
    pool = pool.bfloat16() if st == wl.BF16 else pool
    y = torch.zeros(T, shape.nheads, shape.head_dim, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(bd.la_chunk_scan_workspace_bytes(desc, T, n), dtype=torch.uint8, device="cuda")
    cu, slots, one = to_i32(wl.cu_seqlens(np.asarray(lens, np.int32))), to_i32(range(n)), torch.ones(n, dtype=torch.uint8, device="cuda")
    decay = to_dev(ref.decays(seed, shape.nheads), wl.F32)
    v, k, q = ref.split(shape, rows)

    def call(**kw):
        bd.la_chunk_scan(desc, pool, cu, slots, v, k, q, decay, y, work, has_initial_state=one, **kw)
    return call, pool, y, rows


@pytest.mark.parametrize("lens", [[150, 1, 333], [2000]], ids=str)  # the second in segments
@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_the_scan_in_a_graph(st, lens):
    import torch
    call, pool, y, _ = scan_setup(70, lens, st)
    start, eager, got = replays(call, [pool, y], 3)
    for s, e, g in zip(start, eager, got):
        assert torch.equal(e, g) and not torch.equal(e, s)


def test_plan_norm_and_step_in_a_graph():
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    n, desc = 5, bd.layer_desc(SHAPE, state=wl.F32)
    new, past, table = torch.tensor([1, 1, 0, 1, 1], **i32), torch.tensor([0, 126, 7, 127, 300], **i32), torch.arange(20, **i32).view(5, 4)
    cu, slots, src, dst, pos = (torch.zeros(m, **i32) for m in (n + 1, n, n, n, n))
    g = torch.Generator(device="cuda").manual_seed(7)
    pool = torch.randn(20, 4, 128, 128, device="cuda", generator=g)
    x, y = torch.randn(n, 1, SHAPE.conv_dim, dtype=torch.bfloat16, device="cuda", generator=g), torch.zeros(n, 1, 512, dtype=torch.bfloat16, device="cuda")
    decay, freq = to_dev(ref.decays(71, 4), wl.F32), torch.rand(64, device="cuda", generator=g)
    _, k, q = ref.split(SHAPE, x[:, 0])

    def call():
        bd.mamba_batch_plan(new, past, table, 128, 20, cu_seqlens=cu, slot_ids=slots, copy_src=src, copy_dst=dst, positions=pos)
        bd.mamba_slot_copy(desc, pool, src, dst)
        bd.la_state_update(desc, pool, slots, x, decay, y, qk_norm=True, positions=past, inv_freq=freq)
        bd.la_qk_norm_rope(desc, k, q, k, q, positions=past, inv_freq=freq)
        past.add_(new)
    start, eager, got = replays(call, [past, pool, x, y], 3)
    for s, e, g in zip(start, eager, got):
        assert torch.equal(e, g) and not torch.equal(e, s)


def test_two_scans_at_once_on_two_streams():
    import torch
    calls = [scan_setup(72 + i, lens, wl.F32) for i, lens in enumerate(([1500], [90, 700, 3, 260]))]
    for call, *_ in calls:
        call()
    torch.cuda.synchronize()
    want = [(pool.clone(), y.clone()) for _, pool, y, _ in calls]
    again = [scan_setup(72 + i, lens, wl.F32) for i, lens in enumerate(([1500], [90, 700, 3, 260]))]
    streams = [torch.cuda.Stream() for _ in again]
    torch.cuda.synchronize()
    for (call, *_), s in zip(again, streams):
        call(stream=s)
    for (call, pool, y, _), s, (p0, y0) in zip(again, streams, want):
        s.synchronize()
        assert torch.equal(pool, p0) and torch.equal(y, y0)


@pytest.mark.parametrize("lens", [[129, 128, 1, 77, 300], [3000], [5] * 40], ids=lambda x: str(len(x)))
@pytest.mark.parametrize("N", [64, 128])
def test_an_fp32_pool_holds_24_bits(lens, N):
    """Keys' decays are split exactly to 24 bits and chunks are added with one rounding each: a state is off by a few 2^-24 of
    what it sums, 3000 tokens' random signs and all.  16 bits, or a part lost for some rows, are off by 1e-5."""
    shape = wl.LayerShape(nheads=2, head_dim=64, d_state=N, n_groups=2)
    import torch
    call, pool, y, rows = scan_setup(80, lens, wl.F32, shape, S=len(lens) + 1)
    start = f64(pool)
    call()
    v, k, q = ref.split(shape, f64(rows))
    at, decay = 0, ref.decays(80, 2).astype(np.float64)
    got = f64(pool)
    for i, n in enumerate(lens):
        back = np.exp(decay[None, :] * (n - 1 - np.arange(n))[:, None])  # (token, head)
        want = start[i] * np.exp(decay * n)[:, None, None] + np.einsum("th,thp,thn->hpn", back, v[at:at + n], k[at:at + n])
        err = np.sqrt(((got[i] - want) ** 2).sum((1, 2)) / (want ** 2).sum((1, 2)))
        assert (err <= 1e-6).all(), (i, n, err)
        at += n


def test_scan_past_2_to_31_elements():
    """The last tokens' values and outputs lie past 2^31 elements; what comes before decays away within the check."""
    import torch
    shape = wl.LayerShape(nheads=64, head_dim=64, d_state=64, n_groups=1)
    T = (1 << 31) // (64 * 64) + 300
    g = torch.Generator(device="cuda").manual_seed(9)
    v = torch.zeros(T, 64, 64, dtype=torch.bfloat16, device="cuda")
    k, q = (torch.randn(T, 1, 64, dtype=torch.bfloat16, device="cuda", generator=g) for _ in range(2))
    v[-700:] = torch.randn(700, 64, 64, dtype=torch.bfloat16, device="cuda", generator=g)
    y = torch.full((T, 64, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    desc = bd.layer_desc(shape, state=wl.F32)
    pool = torch.zeros(1, 64, 64, 64, device="cuda")
    work = torch.empty(bd.la_chunk_scan_workspace_bytes(desc, T, 1), dtype=torch.uint8, device="cuda")
    decay = np.full(64, -0.05, np.float32)
    bd.la_chunk_scan(desc, pool, to_i32([0, T]), to_i32([0]), v, k, q, to_dev(decay, wl.F32), y, work)
    S, want = ref.sequence(np.zeros((64, 64, 64)), f64(v[-700:]), f64(k[-700:]), f64(q[-700:]), decay)
    assert not (y[:-700] != 0).any()
    err = np.abs(f64(y[-700:]) - want).max() / np.abs(want).max()
    assert err <= 2.0 ** -8 + 5e-3
    assert np.abs(f64(pool[0]) - S[-1]).max() <= 1e-5 * np.abs(S[-1]).max()


CHILD = textwrap.dedent("""
    import sys
    import numpy as np
    import torch
    sys.path[:0] = [{root!r}, {tests!r}]
    from recurrent_state_update_gb300 import binding as bd, build as bld, workloads as wl
    import la_ref as ref
    from gpu_util import to_dev, to_i32
    from test_la_launch_gpu import SHAPE, scan_setup
    bld.build()
    torch.cuda.set_device(0)
    kept = []
    decay, freq = to_dev(ref.decays(1, 4), wl.F32), torch.full((64,), 0.3, device="cuda")
    for st in (wl.BF16, wl.F32):  # prompts, their keys, single tokens and drafts back to back on one stream
        desc = bd.layer_desc(SHAPE, state=st)
        for lens in ([700, 64, 129], [1800]):
            call, pool, y, rows = scan_setup(75, lens, st, S=20)
            _, k, q = ref.split(SHAPE, rows)
            bd.la_qk_norm_rope(desc, k, q, k, q, positions=to_i32(np.arange(len(rows))), inv_freq=freq)
            call()
            z = torch.zeros(3, 2, 512, dtype=torch.bfloat16, device="cuda")
            for t in range(3):
                bd.la_state_update(desc, pool, to_i32([0, 1, 2]), rows[6 * t:6 * t + 6].view(3, 2, -1), decay, z, positions=to_i32([[t, t + 1]] * 3),
                                   inv_freq=freq)
            bd.la_state_update(desc, pool, to_i32([0, 1, 2]), rows[:12].view(3, 4, -1), decay, torch.zeros(3, 4, 512, dtype=torch.bfloat16, device="cuda"),
                               scratch_slots=to_i32(np.arange(3, 15).reshape(3, 4)))
            kept += [y, pool, z, rows]
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
    assert len(outs["1"].files) == len(outs["0"].files) == 16
    for k in outs["1"].files:
        np.testing.assert_array_equal(outs["1"][k], outs["0"][k], err_msg=k)
