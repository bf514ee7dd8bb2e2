"""Linear attention's kernels against their 64-bit forms, through the binding.

Tolerances, as the largest error of a (row or token, head) tile over the tile's largest value:
  F32   fp32 throughout: a sum of 128 terms is off by at most 128 * 2^-24 = 7.7e-6 of its terms' sum, and a decay
        rounded to 2^-25 drifts by 500 of those over what a head remembers; 1e-4 covers both several times, as
        everywhere in these tests for fp32.
  BF16  a result rounded once to bf16 (2^-8 of itself at most) on top of F32.
  CHUNK bf16 results of the chunked form on tensor cores.  Its operands are rounded to bf16 in two places (scores or
        the state that queries read; decayed keys under a bf16 pool), each off by 2^-8/sqrt(3) rms of itself at
        most, so an output by sqrt(2) times that of its terms' length, 3.2e-3; the largest of a tile's few thousand errors is 4.5
        of them, and the tile's largest value at least 3 times its rms: 4.8e-3, on top of the result's own rounding.
        A single token's head has 64 values and no such largest value, so tiles are whole heads of a sequence.
"""
import numpy as np
import pytest

import la_ref as ref
from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import f64, guarded, tile_rel_err, to_dev, to_i32

pytestmark = pytest.mark.gpu

F32, BF16, CHUNK = 1e-4, 2.0 ** -8 + 1e-4, 2.0 ** -8 + 5e-3
FULL = wl.LayerShape(nheads=4, head_dim=128, d_state=128, n_groups=4)
SHAPES = [FULL, wl.LayerShape(nheads=8, head_dim=64, d_state=128, n_groups=2),
          wl.LayerShape(nheads=3, head_dim=64, d_state=64, n_groups=3),
          wl.LayerShape(nheads=6, head_dim=32, d_state=64, n_groups=1),
          wl.LayerShape(nheads=4, head_dim=16, d_state=16, n_groups=2)]
DTYPES = [(wl.BF16, wl.BF16), (wl.F32, wl.BF16), (wl.F32, wl.F32), (wl.BF16, wl.F32)]
ids = lambda s: f"{s.nheads}x{s.head_dim}x{s.d_state}g{s.n_groups}" if isinstance(s, wl.LayerShape) else str(s)  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    bld.build()
    bd.lib()
    torch.cuda.set_device(0)


def tol(dtype, chunked=False):
    return F32 if dtype == wl.F32 else CHUNK if chunked else BF16


def chunked(shape, act):
    return act == wl.BF16 and shape.head_dim >= 64 and shape.d_state >= 64


def states(seed, shape, n, dtype, scale=0.1):
    return wl.store(scale * wl.rng(seed, 7).standard_normal((n, shape.nheads, shape.head_dim, shape.d_state)), dtype)


def prep_args(seed, shape, positions, norm=True, rot=None, inter=False):
    """(keyword arguments of the calls, those of the 64-bit form) of one norm and rotation."""
    g, N = wl.rng(seed, 11), shape.d_state
    rot = N if rot is None else rot
    kw, qw = ((1 + 0.1 * g.standard_normal(N)).astype(np.float32) for _ in range(2))
    freq = (10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32) if rot else None
    call = dict(qk_norm=norm, interleaved=inter)
    if norm:
        call.update(k_weight=to_dev(kw, wl.F32), q_weight=to_dev(qw, wl.F32), eps=1e-5)
    if rot:
        call.update(positions=to_i32(positions), inv_freq=to_dev(freq, wl.F32))
    own = dict(eps=1e-5 if norm else None, positions=positions, inv_freq=freq, interleaved=inter)
    return call, (dict(own, weight=kw.astype(float)), dict(own, weight=qw.astype(float)))


# ---- the step ----

def run_step(seed, shape, st, act, slots, ntok=1, scratch=None, S=14, stride=None, scale=None, **prep):
    """One call on guarded buffers, checked against the 64-bit form; returns (pool before, pool after, error word)."""
    import torch
    slots = np.asarray(slots, np.int32)
    g = wl.rng(seed, 1)
    xbc = wl.store(g.standard_normal((len(slots), ntok, shape.conv_dim)), act)
    pos = (g.integers(0, 2 ** 17, (len(slots), 1)) + np.arange(ntok)).astype(np.int32)
    before = states(seed, shape, S, st)
    pool = guarded(to_dev(before, st))
    y = guarded(torch.full((len(slots), ntok, shape.nheads * shape.head_dim), 7.0, device="cuda",
                           dtype=torch.float32 if act == wl.F32 else torch.bfloat16))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    decay = ref.decays(seed, shape.nheads)
    call, (kp, qp) = prep_args(seed, shape, pos, **prep)
    bd.la_state_update(bd.layer_desc(shape, state=st, act=act), pool.t, to_i32(slots), to_dev(xbc, act), to_dev(decay, wl.F32),
                       y.t, scratch_slots=to_i32(scratch), scale=scale, err_word=err, **call)
    torch.cuda.synchronize()
    pool.check("pool")
    y.check("y")
    v, k, q = ref.split(shape, wl.upcast(xbc, act))
    k, q = ref.norm_rotate(k, **kp), ref.norm_rotate(q, **qp)
    before, after, y = wl.upcast(before, st), f64(pool.t), f64(y.t).reshape(v.shape)
    touched = set()
    for i, s in enumerate(slots):
        scr = None if scratch is None else np.asarray(scratch)[i]
        if s < 0 or s >= S or (scr is not None and ((scr < -1) | (scr >= S)).any()):
            assert (y[i] == 7.0).all()
            continue
        want, out = ref.sequence(before[s], v[i], k[i], q[i], decay, scale)
        assert tile_rel_err(y[i], out, 1) <= tol(act)
        for j in range(ntok):
            to = scr[j] if scr is not None else (s if j == ntok - 1 else -1)
            if to >= 0:
                touched.add(int(to))
                assert tile_rel_err(after[to], want[j], 2) <= tol(st)
    for s in set(range(S)) - touched:
        assert np.array_equal(after[s], before[s])
    return int(err.item())


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("st,act", DTYPES)
def test_step(shape, st, act):
    assert run_step(1, shape, st, act, [3, -1, 0, 11, 7]) == 0


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rot", [0, 16, None])
@pytest.mark.parametrize("inter", [False, True])
def test_step_norm_and_rotation(shape, norm, rot, inter):
    assert run_step(2, shape, wl.F32, wl.F32, [5, 2], norm=norm, rot=rot, inter=inter) == 0


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("ntok", [2, 3, 8])
def test_step_of_several_tokens(shape, ntok):
    assert run_step(3, shape, wl.F32, wl.BF16, [9, 1, -1], ntok=ntok) == 0


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_step_of_drafts(shape, st):
    scratch = [[3, 4, 5], [-1, -1, 6], [7, 8, 9], [10, -1, 11]]
    assert run_step(4, shape, st, wl.BF16, [0, 1, -1, 2], ntok=3, scratch=scratch) == 0


def test_step_flags_ids_outside_the_pool_and_leaves_their_rows():
    assert run_step(5, FULL, wl.BF16, wl.BF16, [0, 14, -2, 3]) == bd.MAMBA_ERR_SLOT_RANGE
    assert run_step(5, FULL, wl.F32, wl.BF16, [0, 1], ntok=2, scratch=[[5, 14], [6, 7]]) == bd.MAMBA_ERR_SLOT_RANGE


def test_step_scale():
    assert run_step(6, FULL, wl.F32, wl.F32, [1], scale=1.0) == 0


def test_step_of_a_large_batch_with_states_past_2_to_31_elements():
    import torch
    shape = wl.LayerShape(nheads=32, head_dim=128, d_state=128, n_groups=32)
    slots, S = [4150, 0, 4151, 17], 4152  # 4152 * 2^19 elements
    pool = torch.zeros(S, 32, 128, 128, dtype=torch.bfloat16, device="cuda")
    g = wl.rng(8, 0)
    xbc = wl.store(g.standard_normal((4, 1, shape.conv_dim)), wl.BF16)
    decay = ref.decays(8, 32)
    st = states(8, shape, 4, wl.BF16)
    pool[torch.tensor(slots, device="cuda")] = to_dev(st, wl.BF16)
    y = torch.empty(4, 1, 32 * 128, dtype=torch.bfloat16, device="cuda")
    bd.la_state_update(bd.layer_desc(shape), pool, to_i32(slots), to_dev(xbc, wl.BF16), to_dev(decay, wl.F32), y)
    v, k, q = ref.split(shape, wl.upcast(xbc, wl.BF16))
    for i, s in enumerate(slots):
        want, out = ref.sequence(wl.upcast(st, wl.BF16)[i], v[i], k[i], q[i], decay)
        assert tile_rel_err(f64(pool[s]), want[-1], 2) <= BF16
        assert tile_rel_err(f64(y[i]).reshape(out.shape), out, 1) <= BF16


# ---- norm and rotation on their own ----

@pytest.mark.parametrize("heads,N", [(1, 16), (3, 32), (5, 64), (2, 128), (32, 128), (40, 128), (7, 256)])
@pytest.mark.parametrize("act", [wl.BF16, wl.F32])
@pytest.mark.parametrize("tokens", [1, 37])
def test_norm_and_rotation(heads, N, act, tokens):
    import torch
    shape = wl.LayerShape(nheads=heads, head_dim=8, d_state=N, n_groups=heads)
    g = wl.rng(20, 0)
    row = wl.store(g.standard_normal((tokens, shape.conv_dim)), act)
    pos = g.integers(0, 2 ** 31 - 1, tokens).astype(np.int32)
    pos[tokens // 2:][:1] = -1 if tokens > 1 else 5
    for rot, inter, norm in ((N, False, True), (16, True, True), (N, True, False), (0, False, True)):
        rows = to_dev(row, act)
        _, k, q = ref.split(shape, rows)
        call, (kp, qp) = prep_args(20, shape, pos, norm, rot, inter)
        out = guarded(torch.full((tokens, 3, heads, N), 7.0, device="cuda", dtype=rows.dtype))
        bd.la_qk_norm_rope(bd.layer_desc(shape, act=act), k, q, out.t[:, 0], out.t[:, 2], **call)
        out.check("k and q")
        got = f64(out.t)
        assert (got[:, 1] == 7.0).all()
        _, k64, q64 = ref.split(shape, wl.upcast(row, act))
        live = pos >= 0 if rot else np.ones(tokens, bool)
        assert (got[~live] == 7.0).all()
        for i, (x, p) in enumerate(((k64, kp), (q64, qp))):
            want = ref.norm_rotate(x, **p)
            # angles are held to 2^-25 of a half turn (6e-8), the norm and the products to a few roundings
            bound = tol(act) * np.abs(want) + 1e-6 * np.abs(want).max() if act == wl.BF16 else 2e-6 * np.abs(want).max()
            assert (np.abs(got[:, 2 * i] - want) <= bound)[live].all()
        bd.la_qk_norm_rope(bd.layer_desc(shape, act=act), k, q, k, q, **call)  # in place
        assert torch.equal(k[torch.from_numpy(live).cuda()], out.t[:, 0][torch.from_numpy(live).cuda()])
        assert torch.equal(q[torch.from_numpy(live).cuda()], out.t[:, 2][torch.from_numpy(live).cuda()])
        assert np.array_equal(f64(ref.split(shape, rows)[0]), ref.split(shape, wl.upcast(row, act))[0])


# ---- the scan ----

def run_scan(seed, shape, st, act, lens, seeded=True, interval=0, slots=None, behind=0, apart=True, S=None, scale=None, edit=None,
             decay=None):
    """One call on guarded buffers, checked against the 64-bit form; returns the error word."""
    import torch
    g = wl.rng(seed, 2)
    nseq, T = len(lens), int(sum(lens))
    HP, GN = shape.nheads * shape.head_dim, shape.n_groups * shape.d_state
    rows = wl.store(g.standard_normal((T + behind, HP + 2 * GN)), act)
    init = np.array([(i + 1) % 3 > 0 for i in range(nseq)], np.uint8) if seeded else np.zeros(nseq, np.uint8)
    kept = [(n - 1) // interval if interval and n else 0 for n in lens]
    S = S or nseq + sum(kept) + 2
    order = g.permutation(S)
    slots = order[:nseq] if slots is None else np.asarray(slots)
    rest = [s for s in order if s not in set(slots.tolist())]
    ckpt = np.full((nseq, max(1, max(kept, default=0))), -1, np.int32)
    for i, n in enumerate(kept):
        for j in range(n):
            ckpt[i, j] = rest.pop()
    if interval and kept and max(kept) > 1:
        ckpt[int(np.argmax(kept)), 0] = -1
    before = states(seed, shape, S, st)
    pool = guarded(to_dev(before, st))
    dev_rows = to_dev(rows, act)
    if edit:
        edit(dev_rows, T)
    v, k, q = ref.split(shape, dev_rows)
    if not apart:
        v, k, q = v.contiguous(), k.contiguous(), q.contiguous()
    y = guarded(torch.full((T + behind, shape.nheads, shape.head_dim), 7.0, device="cuda", dtype=dev_rows.dtype))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    desc = bd.layer_desc(shape, state=st, act=act)
    ws = guarded(torch.full((bd.la_chunk_scan_workspace_bytes(desc, T + behind, nseq),), 0xFF, dtype=torch.uint8, device="cuda"))
    decay = ref.decays(seed, shape.nheads) if decay is None else np.asarray(decay, np.float32)
    cu = wl.cu_seqlens(np.asarray(lens, np.int32))
    bd.la_chunk_scan(desc, pool.t, to_i32(cu), to_i32(slots), v, k, q, to_dev(decay, wl.F32), y.t, ws.t,
                     has_initial_state=torch.from_numpy(init).cuda(), ckpt_slots=to_i32(ckpt) if interval else None,
                     ckpt_interval=interval, scale=scale, err_word=err)
    torch.cuda.synchronize()
    for b, n in ((pool, "pool"), (y, "y"), (ws, "workspace")):
        b.check(n)
    v, k, q = ref.split(shape, wl.upcast(rows, act))
    before, after, y = wl.upcast(before, st), f64(pool.t), f64(y.t)
    assert (y[T:] == 7.0).all()
    touched, ch = set(), chunked(shape, act)
    for i, n in enumerate(lens):
        a, s = int(cu[i]), int(slots[i])
        if s < -1 or s >= S:
            assert (y[a:a + n] == 7.0).all()
            continue
        if n == 0:
            continue
        start = before[s] if init[i] and s >= 0 else np.zeros_like(before[0])
        want, out = ref.sequence(start, v[a:a + n], k[a:a + n], q[a:a + n], decay, scale)
        assert tile_rel_err(y[a:a + n].swapaxes(0, 1), out.swapaxes(0, 1), 2) <= tol(act, ch), (i, n)
        for to, j in [(s, n)] + [(int(ckpt[i, m]), (m + 1) * interval) for m in range(kept[i])]:
            if to >= 0:
                touched.add(to)
                assert tile_rel_err(after[to], want[j - 1], 2) <= tol(st, ch), (i, n, j)
    for s in set(range(S)) - touched:
        assert np.array_equal(after[s], before[s])
    return int(err.item())


LENGTHS = [[1], [127], [128], [129], [5, 0, 300, 1, 64], [257, 128, 2]]


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("st,act", DTYPES)
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_scan(shape, st, act, lens):
    assert run_scan(30, shape, st, act, lens) == 0


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
@pytest.mark.parametrize("interval", [128, 256])
def test_scan_checkpoints(shape, st, interval):
    assert run_scan(31, shape, st, wl.BF16, [700, 256, 129, 1], interval=interval) == 0


@pytest.mark.parametrize("shape", SHAPES[:2], ids=ids)
@pytest.mark.parametrize("act", [wl.BF16, wl.F32])
def test_scan_of_dense_inputs_and_rows_behind_the_last_sequence(shape, act):
    import torch

    def spoil(rows, T):
        rows[T:] = float("nan")
    assert run_scan(32, shape, wl.F32, act, [70, 200], apart=False, behind=1) == 0
    assert run_scan(32, shape, wl.F32, act, [70, 201], behind=150, edit=spoil) == 0


def test_a_sequence_keeps_clear_of_its_neighbours_nan():
    """Whole tiles are loaded, the next sequence's first tokens with them."""
    import torch
    shape = wl.LayerShape(nheads=2, head_dim=128, d_state=128, n_groups=2)
    for lens in ([100, 60, 30], [1, 128, 5]):
        rows = torch.randn(sum(lens), shape.conv_dim, dtype=torch.bfloat16, device="cuda")
        outs = []
        for spoil in (False, True):
            if spoil:
                rows[lens[0]:lens[0] + lens[1]] = float("nan")
                rows[lens[0] + 1] = float("inf")
            v, k, q = ref.split(shape, rows)
            pool = torch.zeros(3, 2, 128, 128, device="cuda")
            y = torch.zeros(sum(lens), 2, 128, dtype=torch.bfloat16, device="cuda")
            desc = bd.layer_desc(shape, state=wl.F32)
            ws = torch.empty(bd.la_chunk_scan_workspace_bytes(desc, sum(lens), 3), dtype=torch.uint8, device="cuda")
            bd.la_chunk_scan(desc, pool, to_i32(wl.cu_seqlens(np.asarray(lens, np.int32))), to_i32([0, 1, 2]), v, k, q,
                             to_dev(ref.decays(33, 2), wl.F32), y, ws)
            outs.append((y, pool))
        (y0, p0), (y1, p1) = outs
        end = lens[0] + lens[1]
        assert torch.equal(y0[:lens[0]], y1[:lens[0]]) and torch.equal(y0[end:], y1[end:])
        assert torch.equal(p0[0], p1[0]) and torch.equal(p0[2], p1[2]) and p1[1].isnan().any()


@pytest.mark.parametrize("act", [wl.BF16, wl.F32])
def test_scan_without_states_to_write_and_with_bad_slots(act):
    assert run_scan(34, FULL, wl.F32, act, [150, 40, 3], slots=[-1, 2, -1], S=5) == 0
    assert run_scan(34, FULL, wl.F32, act, [150, 40, 3, 9], slots=[4, 5, 1, -2], S=5) == bd.MAMBA_ERR_SLOT_RANGE


@pytest.mark.parametrize("act", [wl.BF16, wl.F32])
@pytest.mark.parametrize("cu", [[1, 5, 20], [0, 30, 20], [0, 5, 21], [0, 2 ** 31 - 1, 20], [0, -3, 20]])
def test_scan_refuses_bad_boundaries_and_does_nothing(act, cu):
    import torch
    desc = bd.layer_desc(FULL, state=wl.F32, act=act)
    dt = torch.bfloat16 if act == wl.BF16 else torch.float32
    x = torch.zeros(20, 4, 128, dtype=dt, device="cuda")
    pool, y = torch.full((2, 4, 128, 128), 3.0, device="cuda"), torch.full_like(x, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(bd.la_chunk_scan_workspace_bytes(desc, 20, 2), dtype=torch.uint8, device="cuda")
    bd.la_chunk_scan(desc, pool, to_i32(cu), to_i32([0, 1]), x, x, x, torch.zeros(4, device="cuda"), y, ws, err_word=err)
    assert err.item() == bd.MAMBA_ERR_SEQLENS and (y == 7.0).all() and (pool == 3.0).all()


@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
@pytest.mark.parametrize("decay", [[0.0, -1e-4], [-1e-30, -0.5], [-3.0, -88.0], [-1e4, float("-inf")]], ids=str)
def test_scan_of_slow_and_fast_decays(st, decay):
    shape = wl.LayerShape(nheads=2, head_dim=64, d_state=128, n_groups=1)
    assert run_scan(35, shape, st, wl.BF16, [300, 130], decay=decay) == 0


@pytest.mark.parametrize("heads,lens", [(1, [2500]), (2, [3000, 1, 1290]), (5, [1, 1665])])
@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_scan_of_long_prompts_of_few_heads(heads, lens, st):
    """Few heads and long sequences: these are worked on in several segments side by side."""
    shape = wl.LayerShape(nheads=heads, head_dim=64, d_state=64, n_groups=heads)
    assert run_scan(36, shape, st, wl.BF16, lens, interval=512) == 0


def test_scan_of_many_sequences():
    shape = wl.LayerShape(nheads=1, head_dim=64, d_state=64, n_groups=1)
    lens = wl.rng(37, 0).integers(0, 5, 3000).tolist()
    assert run_scan(37, shape, wl.F32, wl.BF16, lens) == 0
    small = wl.LayerShape(nheads=1, head_dim=16, d_state=16, n_groups=1)
    assert run_scan(37, small, wl.F32, wl.F32, lens) == 0


@pytest.mark.parametrize("shape", SHAPES[:2], ids=ids)
@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_scan_of_more_sequences_than_blocks(shape, st):
    """Two or three sequences a block, one after the other, whose last chunks are of every length."""
    lens = wl.rng(39, 0).integers(1, 161, 90 * 4 // shape.nheads).tolist()
    assert run_scan(39, shape, st, wl.BF16, lens + [128, 256]) == 0


def test_scan_scale_and_no_tokens():
    import torch
    assert run_scan(38, FULL, wl.F32, wl.BF16, [40], scale=1.0) == 0
    assert run_scan(38, FULL, wl.F32, wl.BF16, [0, 0], seeded=False) == 0


def test_a_second_run_gives_the_same_bytes():
    import torch
    shape = wl.LayerShape(nheads=2, head_dim=128, d_state=128, n_groups=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = torch.randn(3000, shape.conv_dim, dtype=torch.bfloat16, device="cuda", generator=g)
    v, k, q = ref.split(shape, rows)
    desc = bd.layer_desc(shape, state=wl.F32)
    ws = torch.empty(bd.la_chunk_scan_workspace_bytes(desc, 3000, 3), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(3):
        pool = torch.zeros(3, 2, 128, 128, device="cuda")
        y = torch.empty(3000, 2, 128, dtype=torch.bfloat16, device="cuda")
        bd.la_chunk_scan(desc, pool, to_i32([0, 1500, 1501, 3000]), to_i32([2, 0, 1]), v, k, q, to_dev(ref.decays(1, 2), wl.F32), y, ws)
        outs.append((y, pool))
    for y, pool in outs[1:]:
        assert torch.equal(y, outs[0][0]) and torch.equal(pool, outs[0][1])
