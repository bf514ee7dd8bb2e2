"""The gated delta rule's kernels against its 64-bit form, through the binding.

Tolerances, as the largest error of a (row or token, head) tile over the tile's largest value:
  F32   fp32 throughout: a dot product of 128 terms is off by at most 128 * 2^-24 = 7.7e-6 of its terms'
        sum, and the delta rule damps what earlier tokens left; 1e-4 covers ten such terms, as
        everywhere in these tests for fp32.
  BF16  a result rounded once to bf16 (8 bits: 2^-8 of itself at most) on top of F32.
  CHUNK bf16 results of the chunked form on tensor cores, whose operands are rounded to 11 bits: four
        products in a row with two operands each, 2^-11/sqrt(3) rms a rounding, give 8e-4 of a tile's
        rms, and the largest of a tile's few thousand errors is 4.5 of them: 3.6e-3 of the rms, a third
        of that against the tile's largest value, and as much again for the state the errors have
        passed through: 3e-3 with room, on top of the result's own rounding.
  A stored bf16 state is compared after every call against the 64-bit sequence from the stored start.
"""
import numpy as np
import pytest

import gdn_ref as ref
from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import f64, guarded, tile_rel_err, to_dev, to_i32

pytestmark = pytest.mark.gpu

F32, BF16, CHUNK = 1e-4, 2.0 ** -8 + 1e-4, 2.0 ** -8 + 3e-3
FULL = wl.LayerShape(nheads=4, head_dim=128, d_state=128, n_groups=2)
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


def states(seed, shape, n, dtype, scale=0.1):
    g = wl.rng(seed, 7)
    return wl.store(scale * g.standard_normal((n, shape.nheads, shape.head_dim, shape.d_state)), dtype)


def run_step(seed, shape, st, act, slots, ntok=1, scratch=None, S=12, steps=None, dt="f32", edit=None, **kw):
    """One call on guarded buffers; returns (inputs, pool before, pool after, y, error word)."""
    import torch
    slots = np.asarray(slots, np.int32)
    A, bias = ref.layer(seed, shape)
    xbc, raw, beta = ref.inputs(seed, shape, (len(slots), ntok), act, dt, steps)
    before = states(seed, shape, S, st)
    if edit:
        edit(xbc, raw, beta, before)
    pool = guarded(to_dev(before, st))
    y = guarded(torch.full((len(slots), ntok, shape.nheads * shape.head_dim), 7.0, device="cuda",
                           dtype=torch.float32 if act == wl.F32 else torch.bfloat16))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    desc = bd.layer_desc(shape, state=st, act=act, dt=dt)
    bd.gdn_state_update(desc, pool.t, to_i32(slots), to_dev(xbc, act), to_dev(raw, dt), to_dev(beta, dt), to_dev(A, wl.F32),
                        y.t, dt_bias=to_dev(bias, wl.F32), scratch_slots=to_i32(scratch), err_word=err, **kw)
    torch.cuda.synchronize()
    pool.check("pool")
    y.check("y")
    inp = [wl.upcast(a, d) for a, d in ((xbc, act), (raw, dt), (beta, dt))]
    return inp, wl.upcast(before, st), f64(pool.t), f64(y.t), int(err.item()), (A.astype(float), bias.astype(float))


def check_step(shape, st, act, slots, r, scratch=None, flags={}):
    (xbc, dt, beta), before, after, y, err, (A, bias) = r
    assert err == 0
    v, k, q = ref.split(shape, xbc)
    want = before.copy()
    for i, s in enumerate(slots):
        if s < 0:
            assert (y[i] == 7.0).all()
            continue
        S, out = ref.sequence(before[s], v[i], k[i], q[i], dt[i], beta[i], A, bias, **flags)
        got = y[i].reshape(out.shape)
        assert tile_rel_err(got, out, 1) <= tol(act)
        writes = [(s, len(S) - 1)] if scratch is None else [(d, j) for j, d in enumerate(scratch[i]) if d >= 0]
        for d, j in writes:
            assert tile_rel_err(after[d], S[j], 2) <= tol(st)
            want[d] = after[d]
    np.testing.assert_array_equal(after, want)  # every other slot is untouched


@pytest.mark.parametrize("st,act", DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_step(shape, st, act):
    slots = [3, -1, 0, 11, 7]
    check_step(shape, st, act, slots, run_step(1, shape, st, act, slots))


@pytest.mark.parametrize("batch", [1, 2, 9, 40, 130])
@pytest.mark.parametrize("shape", SHAPES[:2], ids=ids)
def test_step_batches(shape, batch):
    slots = np.random.default_rng(batch).permutation(batch + 3)[:batch]
    check_step(shape, wl.BF16, wl.BF16, slots, run_step(batch, shape, wl.BF16, wl.BF16, slots, S=batch + 3))


@pytest.mark.parametrize("st,act", DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("ntok", [2, 5, 8])
def test_several_tokens_into_scratch_slots(shape, st, act, ntok):
    slots = [2, -1, 0]
    scratch = np.full((3, ntok), -1)
    scratch[0] = np.arange(4, 4 + ntok)
    scratch[2, 1:] = np.arange(12, 11 + ntok)
    check_step(shape, st, act, slots, run_step(2, shape, st, act, slots, ntok, scratch, S=24), scratch)


def test_several_tokens_in_place():
    slots = [5, 1]
    check_step(FULL, wl.F32, wl.BF16, slots, run_step(3, FULL, wl.F32, wl.BF16, slots, 4))


@pytest.mark.parametrize("steps", [wl.WIDE_STEPS, wl.LARGE_STEPS])
def test_step_sizes(steps):
    slots = [0, 4, 2]
    check_step(FULL, wl.F32, wl.F32, slots, run_step(4, FULL, wl.F32, wl.F32, slots, 6, steps=steps))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("softplus,sigmoid,l2norm,scale", [(False, True, True, None), (True, False, True, 1.0),
                                                           (True, True, False, 0.5), (False, False, False, 2.0)])
def test_step_switches(dt, softplus, sigmoid, l2norm, scale):
    def edit(xbc, raw, beta, before):
        if not softplus:  # the step itself: non-negative
            raw[...] = wl.store(np.abs(wl.upcast(raw, dt)) / 10 + 8, dt)  # dt_bias is about -5
        if not sigmoid:
            beta[...] = wl.store(np.clip(np.abs(wl.upcast(beta, dt)), 0, 1), dt)
        if not l2norm:  # keys of about unit length
            HP = FULL.nheads * FULL.head_dim
            xbc[..., HP:] = wl.store(wl.upcast(xbc[..., HP:], wl.BF16) / 8, wl.BF16)

    slots = [1, 3]
    r = run_step(5, FULL, wl.F32, wl.BF16, slots, 3, dt=dt, edit=edit, dt_softplus=softplus, beta_sigmoid=sigmoid,
                 qk_l2norm=l2norm, scale=scale)
    check_step(FULL, wl.F32, wl.BF16, slots, r, flags=dict(softplus=softplus, sigmoid=sigmoid, l2norm=l2norm, scale=scale))


def test_a_zero_key_writes_nothing_and_a_zero_query_reads_nothing():
    HP, GN = FULL.nheads * FULL.head_dim, FULL.n_groups * FULL.d_state

    def edit(xbc, raw, beta, before):
        xbc[0, :, HP:HP + GN] = 0
        xbc[1, :, HP + GN:] = 0

    slots = [0, 1]
    r = run_step(6, FULL, wl.F32, wl.F32, slots, edit=edit)
    check_step(FULL, wl.F32, wl.F32, slots, r)
    assert (r[3][1] == 0).all()


def test_no_step_and_no_write_leave_the_state_bit_for_bit():
    def edit(xbc, raw, beta, before):
        raw[...] = 0
        beta[...] = 0

    import torch
    for st in (wl.F32, wl.BF16):
        A, bias = ref.layer(7, FULL)
        xbc, raw, beta = ref.inputs(7, FULL, (2, 1), wl.BF16)
        edit(xbc, raw, beta, None)
        before = to_dev(states(7, FULL, 3, st), st)
        pool = before.clone()
        y = torch.zeros(2, 1, 512, dtype=torch.bfloat16, device="cuda")
        bd.gdn_state_update(bd.layer_desc(FULL, state=st), pool, to_i32([2, 0]), to_dev(xbc, wl.BF16), to_dev(raw, wl.F32),
                            to_dev(beta, wl.F32), to_dev(A, wl.F32), y, dt_softplus=False, beta_sigmoid=False)
        assert torch.equal(pool, before)
        bd.gdn_chunk_scan(bd.layer_desc(FULL, state=st), pool, to_i32([0, 2]), to_i32([1]),
                          *[t.contiguous() for t in _vkq(FULL, to_dev(xbc, wl.BF16)[:, 0])], to_dev(raw, wl.F32)[:, 0],
                          to_dev(beta, wl.F32)[:, 0], to_dev(A, wl.F32), y, _work(FULL, 2, 1, st, wl.BF16),
                          dt_softplus=False, beta_sigmoid=False,
                          has_initial_state=torch.ones(1, dtype=torch.uint8, device="cuda"))
        assert torch.equal(pool, before)


def test_bad_slots_are_flagged_and_their_rows_left_alone():
    slots = [1, 12, -2, 3]
    inp, before, after, y, err, _ = run_step(8, FULL, wl.BF16, wl.BF16, slots)
    assert err == bd.MAMBA_ERR_SLOT_RANGE
    assert (y[1] == 7.0).all() and (y[2] == 7.0).all() and (y[0] != 7.0).any() and (y[3] != 7.0).any()
    keep = [s for s in range(12) if s not in (1, 3)]
    np.testing.assert_array_equal(after[keep], before[keep])
    scratch = [[4, 5], [6, 12]]
    inp, before, after, y, err, _ = run_step(8, FULL, wl.BF16, wl.BF16, [0, 1], 2, scratch)
    assert err == bd.MAMBA_ERR_SLOT_RANGE and (y[1] == 7.0).all()
    np.testing.assert_array_equal(after[[0, 1, 2, 3, 6, 7]], before[[0, 1, 2, 3, 6, 7]])


def test_a_strided_pool_a_second_stream_and_a_graph():
    import torch
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(9, FULL))
    xbc, raw, beta = ref.inputs(9, FULL, (3, 1), wl.BF16)
    args = to_dev(xbc, wl.BF16), to_dev(raw, wl.F32), to_dev(beta, wl.F32), A
    start = to_dev(states(9, FULL, 5, wl.BF16), wl.BF16)
    desc, slots = bd.layer_desc(FULL), to_i32([4, 0, 2])

    def fresh():
        return start.clone(), torch.zeros(3, 1, 512, dtype=torch.bfloat16, device="cuda")

    plain, y0 = fresh()
    for _ in range(3):
        bd.gdn_state_update(desc, plain, slots, *args, y0, dt_bias=bias)
    wide = torch.zeros(5, 2, *start.shape[1:], dtype=torch.bfloat16, device="cuda")
    wide[:, 0] = start
    y1 = torch.zeros_like(y0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            bd.gdn_state_update(desc, wide[:, 0], slots, *args, y1, dt_bias=bias)
    torch.cuda.synchronize()
    assert torch.equal(wide[:, 0], plain) and torch.equal(y1, y0) and not wide[:, 1].any()
    pool, y2 = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.gdn_state_update(desc, pool, slots, *args, y2, dt_bias=bias)
    pool.copy_(start)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(pool, plain) and torch.equal(y2, y0)


def test_offsets_past_32_bits():
    """A pool of over 2^32 elements: the last slot's state and no other."""
    import torch
    n = (1 << 32) // (4 * 128 * 128) + 2
    pool = torch.zeros(n, 4, 128, 128, dtype=torch.bfloat16, device="cuda")
    first = to_dev(states(10, FULL, 1, wl.BF16), wl.BF16)
    pool[-1] = first[0]
    xbc, raw, beta = ref.inputs(10, FULL, (1, 1), wl.BF16)
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(10, FULL))
    ys = [torch.zeros(1, 1, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for p, s, y in ((pool, n - 1, ys[0]), (first, 0, ys[1])):
        bd.gdn_state_update(bd.layer_desc(FULL), p, to_i32([s]), to_dev(xbc, wl.BF16), to_dev(raw, wl.F32),
                            to_dev(beta, wl.F32), A, y, dt_bias=bias)
    assert torch.equal(ys[0], ys[1]) and torch.equal(pool[-1], first[0]) and not pool[:-1].any()


# ---- int8 entries ----

def _store_views(shape, desc, n):
    import torch
    size = bd.mamba_int8_entry_bytes(desc)
    store = torch.zeros(n, size, dtype=torch.uint8, device="cuda")
    H, P, N = shape.nheads, shape.head_dim, shape.d_state
    at = (H * P * N + 255) // 256 * 256
    return store, store[:, :H * P * N].view(torch.int8).view(n, H, P, N), store[:, at:at + 4 * H * N].view(torch.float32).view(n, H, N)


@pytest.mark.parametrize("act", [wl.BF16, wl.F32])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("steps", [None, wl.WIDE_STEPS])
def test_int8_step(shape, act, steps):
    """Codes are the 64-bit form's but where its value lies within fp32's error of a rounding boundary
    (about 1e-6 of the column's maximum, two boundaries a grid step of 1/127: under 1 in 1000), and
    there they are the neighbour."""
    import torch
    desc = bd.layer_desc(shape, act=act)
    entries = [4, -1, 0, 2]
    store, codes, scales = _store_views(shape, desc, 6)
    S0 = wl.upcast(states(20, shape, 6, wl.F32), wl.F32)
    S0[2, 0] = 0  # a head without a state yet
    sc, co = ref.int8_codes(S0)
    codes.copy_(torch.from_numpy(co))
    scales.copy_(torch.from_numpy(sc))
    store[:, -256:] = 91  # the conv windows
    held = guarded(store)
    codes, scales = (t.clone() for t in (codes, scales))
    A, bias = ref.layer(20, shape)
    xbc, raw, beta = ref.inputs(20, shape, (4, 1), act, steps=steps)
    y = torch.full((4, shape.nheads * shape.head_dim), 7.0, device="cuda", dtype=to_dev(xbc, act).dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.gdn_state_update_int8(desc, held.t, to_i32(entries), to_dev(xbc, act)[:, 0], to_dev(raw, wl.F32)[:, 0],
                             to_dev(beta, wl.F32)[:, 0], to_dev(A, wl.F32), y, dt_bias=to_dev(bias, wl.F32), err_word=err)
    torch.cuda.synchronize()
    held.check("store")
    assert int(err.item()) == 0
    v, k, q = ref.split(shape, wl.upcast(xbc, act))
    want = store.clone()
    H, P, N = shape.nheads, shape.head_dim, shape.d_state
    at = (H * P * N + 255) // 256 * 256
    for i, e in enumerate(entries):
        if e < 0:
            assert (y[i] == 7.0).all()
            continue
        S, out = ref.sequence(f64(codes[e]) * f64(scales[e])[:, None], v[i], k[i], q[i], raw[i].astype(float),
                              beta[i].astype(float), A.astype(float), bias.astype(float))
        assert tile_rel_err(f64(y[i]).reshape(out.shape[1:]), out[0], 1) <= tol(act)
        sc, co = ref.int8_codes(S[0])
        got_c = f64(held.t[e, :H * P * N].view(torch.int8)).reshape(H, P, N)
        got_s = f64(held.t[e, at:at + 4 * H * N].view(torch.float32)).reshape(H, N)
        np.testing.assert_allclose(got_s, sc, rtol=1e-5)
        off = np.abs(got_c - co)
        assert off.max() <= 1 and (off > 0).mean() <= 1e-3
        assert np.abs(got_c).max() <= 127
        want[e, :at + 4 * H * N] = held.t[e, :at + 4 * H * N]
    assert torch.equal(held.t, want)  # other entries and every conv window are untouched


@pytest.mark.parametrize("shape,batch", [(FULL, 330), (SHAPES[1], 200), (SHAPES[3], 450)], ids=ids)
def test_int8_large_batches(shape, batch):
    """Many rows: the same bytes as the rows' entries get in small calls, with padding rows and entries out
    of range among them."""
    import torch
    desc = bd.layer_desc(shape)
    n = batch + 5
    g = np.random.default_rng(batch)
    entries = g.permutation(n)[:batch].astype(np.int32)
    entries[g.permutation(batch)[:9]] = -1
    entries[g.permutation(batch)[:4]] = n + 3
    store, codes, scales = _store_views(shape, desc, n)
    codes.copy_(torch.randint(-127, 128, codes.shape, device="cuda"))
    scales.copy_(torch.rand(scales.shape, device="cuda") / 1000)
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(23, shape))
    x, r, b = (to_dev(a, d) for a, d in zip(ref.inputs(23, shape, (batch,), wl.BF16), (wl.BF16, wl.F32, wl.F32)))
    outs = []
    for step in (batch, 7):
        held = guarded(store)
        y = torch.full((batch, shape.nheads * shape.head_dim), 7.0, device="cuda", dtype=torch.bfloat16)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        for i in range(0, batch, step):
            bd.gdn_state_update_int8(desc, held.t, to_i32(entries[i:i + step]), x[i:i + step], r[i:i + step], b[i:i + step], A,
                                     y[i:i + step], dt_bias=bias, err_word=err)
        torch.cuda.synchronize()
        held.check("store")
        assert int(err.item()) == bd.MAMBA_ERR_SLOT_RANGE
        outs.append((held.t.clone(), y))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert not torch.equal(outs[0][0], store)


def test_int8_bad_entries_are_flagged():
    import torch
    desc = bd.layer_desc(FULL)
    store, codes, scales = _store_views(FULL, desc, 3)
    codes.copy_(torch.randint(-127, 128, codes.shape, device="cuda"))
    scales.fill_(0.01)
    before = store.clone()
    xbc, raw, beta = ref.inputs(21, FULL, (2,), wl.BF16)
    A, _ = ref.layer(21, FULL)
    y = torch.full((2, 512), 7.0, device="cuda", dtype=torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.gdn_state_update_int8(desc, store, to_i32([3, -5]), to_dev(xbc, wl.BF16), to_dev(raw, wl.F32), to_dev(beta, wl.F32),
                             to_dev(A, wl.F32), y, err_word=err)
    assert int(err.item()) == bd.MAMBA_ERR_SLOT_RANGE and torch.equal(store, before) and (y == 7.0).all()


def test_int8_follows_the_exact_chain():
    """64 steps: each rounds by a uniform error of half a grid step at most, 1/(254 sqrt 3) rms of a
    column's maximum (about 2.8 deviations of its values: 0.64 % rms), and the rule forgets them as it
    forgets values; the outputs of the 64-bit chain without any rounding are followed to 5 % rms
    (60 remembered errors)."""
    import torch
    T = 64
    desc = bd.layer_desc(FULL, state=wl.F32, act=wl.F32)
    pool = to_dev(states(22, FULL, 1, wl.F32), wl.F32)
    store, *_ = _store_views(FULL, desc, 1)
    bd.mamba_ckpt_store_int8(desc, pool, to_i32([0]), to_i32([0]), store)
    xbc, raw, beta = ref.inputs(22, FULL, (T, 1), wl.F32)
    A, bias = ref.layer(22, FULL)
    y = torch.zeros(T, 1, 512, device="cuda")
    dx, dr, db = to_dev(xbc, wl.F32), to_dev(raw, wl.F32), to_dev(beta, wl.F32)
    for t in range(T):
        bd.gdn_state_update_int8(desc, store, to_i32([0]), dx[t], dr[t], db[t], to_dev(A, wl.F32), y[t],
                                 dt_bias=to_dev(bias, wl.F32))
    bd.mamba_ckpt_load_int8(desc, pool, to_i32([0]), to_i32([0]), store)
    v, k, q = (a[:, 0] for a in ref.split(FULL, xbc.astype(float)))
    S, out = ref.sequence(wl.upcast(states(22, FULL, 1, wl.F32), wl.F32)[0], v, k, q, raw[:, 0].astype(float),
                          beta[:, 0].astype(float), A.astype(float), bias.astype(float))
    rms = lambda a, b: np.sqrt(((a - b) ** 2).sum() / (b ** 2).sum())  # noqa: E731
    assert rms(f64(y).reshape(out.shape), out) <= 0.05 and rms(f64(pool)[0], S[-1]) <= 0.05


# ---- the scan ----

def _vkq(shape, xbc):
    T = xbc.shape[0]
    HP, GN = shape.nheads * shape.head_dim, shape.n_groups * shape.d_state
    return (xbc[:, :HP].reshape(T, shape.nheads, shape.head_dim), xbc[:, HP:HP + GN].reshape(T, shape.n_groups, shape.d_state),
            xbc[:, HP + GN:].reshape(T, shape.n_groups, shape.d_state))


def _work(shape, T, nseq, st, act, dt="f32"):
    import torch
    return torch.full((bd.gdn_chunk_scan_workspace_bytes(bd.layer_desc(shape, state=st, act=act, dt=dt), T, nseq),), 255,
                      dtype=torch.uint8, device="cuda")


def run_scan(seed, shape, st, act, lens, slots, init=None, ckpt=None, interval=0, S=None, steps=None, dt="f32", edit=None,
             flags={}):
    """One call on guarded buffers (the workspace starts as NaN); checks everything against the 64-bit form."""
    import torch
    T, n = int(sum(lens)), len(lens)
    S = S or n + 2
    A, bias = ref.layer(seed, shape)
    xbc, raw, beta = ref.inputs(seed, shape, (T,), act, dt, steps)
    before = states(seed, shape, S, st)
    if edit:
        edit(xbc, raw, beta, before)
    pool = guarded(to_dev(before, st))
    y = guarded(torch.full((T, shape.nheads, shape.head_dim), 7.0, device="cuda",
                           dtype=torch.float32 if act == wl.F32 else torch.bfloat16))
    work = guarded(_work(shape, T, n, st, act, dt))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = wl.cu_seqlens(lens)
    bd.gdn_chunk_scan(bd.layer_desc(shape, state=st, act=act, dt=dt), pool.t, to_i32(cu), to_i32(slots),
                      *[t.contiguous() for t in _vkq(shape, to_dev(xbc, act))], to_dev(raw, dt), to_dev(beta, dt),
                      to_dev(A, wl.F32), y.t, work.t, dt_bias=to_dev(bias, wl.F32),
                      has_initial_state=None if init is None else torch.tensor(init, dtype=torch.uint8, device="cuda"),
                      ckpt_slots=to_i32(ckpt), ckpt_interval=interval, err_word=err,
                      **{{"softplus": "dt_softplus", "sigmoid": "beta_sigmoid", "l2norm": "qk_l2norm"}.get(k, k): w
                         for k, w in flags.items()})
    torch.cuda.synchronize()
    for b in (pool, y, work):
        b.check()
    assert int(err.item()) == 0
    before, after, got = wl.upcast(before, st), f64(pool.t), f64(y.t)
    v, k, q = ref.split(shape, wl.upcast(xbc, act))
    raw, beta = wl.upcast(raw, dt), wl.upcast(beta, dt)
    want = before.copy()
    for i, L in enumerate(lens):
        a, b = cu[i], cu[i + 1]
        if L == 0:
            continue
        S0 = before[slots[i]] if slots[i] >= 0 and init is not None and init[i] else np.zeros(before.shape[1:])
        St, out = ref.sequence(S0, v[a:b], k[a:b], q[a:b], raw[a:b], beta[a:b], A.astype(float), bias.astype(float), **flags)
        assert np.isfinite(got[a:b]).all()
        for c in range(0, L, 64):  # tiles of 64 tokens
            assert tile_rel_err(got[a + c:min(b, a + c + 64)].transpose(1, 0, 2), out[c:c + 64].transpose(1, 0, 2), 2) <= tol(act, True)
        writes = [(slots[i], L)] if slots[i] >= 0 else []
        if ckpt is not None:
            writes += [(d, (j + 1) * interval) for j, d in enumerate(ckpt[i]) if d >= 0 and (j + 1) * interval <= L]
        for d, at in writes:
            assert tile_rel_err(after[d], St[at - 1], 2) <= tol(st, True)
            want[d] = after[d]
    np.testing.assert_array_equal(after, want)
    return got, after


LENS = [1, 64, 0, 63, 130, 65, 2, 200]


@pytest.mark.parametrize("st,act", DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_scan_ragged(shape, st, act):
    run_scan(30, shape, st, act, LENS, [9, 0, 3, 1, 5, 2, -1, 4], init=[1, 0, 1, 1, 0, 1, 1, 1], S=11)


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_scan_checkpoints(shape, st):
    ckpt = [[5, -1, 6], [7, 8, 9], [10, 11, 12]]
    run_scan(31, shape, st, wl.BF16, [200, 63, 128], [2, 0, -1], init=[0, 1, 1], ckpt=ckpt, interval=64, S=14)


@pytest.mark.parametrize("st,act", [DTYPES[0], DTYPES[2]])
@pytest.mark.parametrize("steps", [wl.WIDE_STEPS, wl.LARGE_STEPS])
def test_scan_step_sizes(st, act, steps):
    """Decays from almost none to exp(-80) a token, mixed in one chunk."""
    run_scan(32, FULL, st, act, [150, 64], [0, 1], init=[1, 1], steps=steps)


@pytest.mark.parametrize("st,act", [DTYPES[0], DTYPES[2]])
def test_scan_almost_no_decay(st, act):
    def edit(xbc, raw, beta, before):
        raw -= 12

    run_scan(33, FULL, st, act, [300], [0], init=[1], edit=edit)


@pytest.mark.parametrize("st,act", [DTYPES[0], DTYPES[1]])
def test_scan_repeated_keys(st, act):
    """The same key all along: every row of I + L is full, and a value replaces the last one's."""
    HP, GN = FULL.nheads * FULL.head_dim, FULL.n_groups * FULL.d_state

    def edit(xbc, raw, beta, before):
        xbc[:, HP:HP + GN] = xbc[0, HP:HP + GN]
        beta += 3

    run_scan(34, FULL, st, act, [200], [0], edit=edit)


@pytest.mark.parametrize("st,act", [DTYPES[0], DTYPES[1]])
@pytest.mark.parametrize("exponent", [-30, 17, 40])
def test_scan_value_magnitudes(st, act, exponent):
    """Values and states of any size bf16 holds: outputs scale with them."""
    HP = FULL.nheads * FULL.head_dim

    def edit(xbc, raw, beta, before):
        xbc[:, :HP] = wl.store(wl.upcast(xbc[:, :HP], act) * 2.0 ** exponent, act)
        before[...] = wl.store(wl.upcast(before, st) * 2.0 ** exponent, st)

    run_scan(35, FULL, st, act, [90, 70], [0, 2], init=[1, 0], edit=edit)


@pytest.mark.parametrize("st,act", [DTYPES[0], DTYPES[1]])
def test_scan_zero_keys_and_queries(st, act):
    HP, GN = FULL.nheads * FULL.head_dim, FULL.n_groups * FULL.d_state

    def edit(xbc, raw, beta, before):
        xbc[10:40, HP:HP + GN] = 0
        xbc[30:90, HP + GN:] = 0
        xbc[90:, :HP] = 0

    got, _ = run_scan(36, FULL, st, act, [130], [0], init=[1], edit=edit)
    assert (got[30:90] == 0).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_scan_switches(st, dt):
    """The step, the gate and the lengths given as they are; queries of any length."""
    HP, GN = FULL.nheads * FULL.head_dim, FULL.n_groups * FULL.d_state

    def edit(xbc, raw, beta, before):
        raw[...] = wl.store(np.abs(wl.upcast(raw, dt)) / 10 + 8, dt)  # dt_bias is about -5
        beta[...] = wl.store(np.clip(np.abs(wl.upcast(beta, dt)), 0, 1), dt)
        xbc[:, HP:HP + GN] = wl.store(wl.upcast(xbc[:, HP:HP + GN], wl.BF16) / 8, wl.BF16)
        xbc[:, HP + GN:] = wl.store(wl.upcast(xbc[:, HP + GN:], wl.BF16) * 1e6, wl.BF16)

    run_scan(37, FULL, st, wl.BF16, [70, 20], [0, 1], init=[1, 1], dt=dt, edit=edit,
             flags=dict(softplus=False, sigmoid=False, l2norm=False, scale=1e-6))


@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_a_sequence_of_nan_leaves_its_neighbours_alone(st):
    """Sequences share tiles at their ends: what one holds may not reach another."""
    import torch
    lens = [70, 61, 33]
    T = sum(lens)
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(38, FULL))
    xbc, raw, beta = ref.inputs(38, FULL, (T,), wl.BF16)
    outs = []
    for poison in (False, True):
        x, r, b = to_dev(xbc, wl.BF16), to_dev(raw, wl.F32), to_dev(beta, wl.F32)
        pool = to_dev(states(38, FULL, 4, st), st)
        if poison:
            x[70:131], r[70:131], b[70:131], pool[1] = (float("nan"),) * 4
        y = torch.zeros(T, 4, 128, dtype=torch.bfloat16, device="cuda")
        bd.gdn_chunk_scan(bd.layer_desc(FULL, state=st), pool, to_i32(wl.cu_seqlens(lens)), to_i32([0, 1, 2]),
                          *[t.contiguous() for t in _vkq(FULL, x)], r, b, A, y, _work(FULL, T, 3, st, wl.BF16), dt_bias=bias,
                          has_initial_state=torch.ones(3, dtype=torch.uint8, device="cuda"))
        outs.append((torch.cat([y[:70], y[131:]]), pool[[0, 2, 3]]))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.isfinite(outs[1][0].float()).all()


@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_scan_refuses_bad_lengths_and_slots(st):
    import torch
    A, _ = ref.layer(39, FULL)
    xbc, raw, beta = ref.inputs(39, FULL, (90,), wl.BF16)
    vkq = [t.contiguous() for t in _vkq(FULL, to_dev(xbc, wl.BF16))]

    def call(cu, slots, ckpt=None):
        pool = to_dev(states(39, FULL, 4, st), st)
        y = torch.full((90, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        bd.gdn_chunk_scan(bd.layer_desc(FULL, state=st), pool, to_i32(cu), to_i32(slots), *vkq, to_dev(raw, wl.F32),
                          to_dev(beta, wl.F32), to_dev(A, wl.F32), y, _work(FULL, 90, len(slots), st, wl.BF16),
                          ckpt_slots=to_i32(ckpt), ckpt_interval=64 if ckpt else 0, err_word=err)
        return f64(pool), f64(y), int(err.item())

    before = wl.upcast(states(39, FULL, 4, st), st)
    for cu in ([0, 50, 89], [1, 50, 90], [0, 91, 90]):
        pool, y, err = call(cu, [0, 1])
        assert err == bd.MAMBA_ERR_SEQLENS and (y == 7.0).all()
        np.testing.assert_array_equal(pool, before)
    for bad in (4, -2):
        pool, y, err = call([0, 50, 90], [bad, 1])
        assert err == bd.MAMBA_ERR_SLOT_RANGE and (y[:50] == 7.0).all() and (y[50:] != 7.0).any()
        np.testing.assert_array_equal(pool[[0, 2, 3]], before[[0, 2, 3]])
    pool, y, err = call([0, 70, 90], [0, 1], ckpt=[[9], [3]])  # a bad checkpoint slot is skipped
    assert err == bd.MAMBA_ERR_SLOT_RANGE and (y != 7.0).any()
    np.testing.assert_array_equal(pool[[2, 3]], before[[2, 3]])


@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_only_empty_sequences(st):
    import torch
    pool = to_dev(states(40, FULL, 2, st), st)
    before = pool.clone()
    e = torch.zeros(0, device="cuda")
    bd.gdn_chunk_scan(bd.layer_desc(FULL, state=st), pool, to_i32([0, 0, 0]), to_i32([0, 1]), *[e.bfloat16()] * 3, e, e,
                      to_dev(ref.layer(40, FULL)[0], wl.F32), e.bfloat16(), _work(FULL, 0, 2, st, wl.BF16))
    torch.cuda.synchronize()
    assert torch.equal(pool, before)


@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
def test_scan_is_the_same_every_time_and_on_another_stream(st):
    import torch
    lens = [500, 1, 777, 64]
    T = sum(lens)
    shape = wl.LayerShape(nheads=16, head_dim=128, d_state=128, n_groups=4)
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(41, shape))
    x, r, b = (to_dev(a, d) for a, d in zip(ref.inputs(41, shape, (T,), wl.BF16), (wl.BF16, wl.F32, wl.F32)))
    vkq = [t.contiguous() for t in _vkq(shape, x)]
    first = None
    side = torch.cuda.Stream()
    for k in range(4):
        pool = to_dev(states(41, shape, 4, st), st)
        y = torch.zeros(T, 16, 128, dtype=torch.bfloat16, device="cuda")
        work = _work(shape, T, 4, st, wl.BF16)
        side.wait_stream(torch.cuda.current_stream())
        bd.gdn_chunk_scan(bd.layer_desc(shape, state=st), pool, to_i32(wl.cu_seqlens(lens)), to_i32([0, 1, 2, 3]), *vkq, r, b,
                          A, y, work, dt_bias=bias, stream=side if k % 2 else None)
        torch.cuda.synchronize()
        if first is None:
            first = (y, pool)
        assert torch.equal(y, first[0]) and torch.equal(pool, first[1])


@pytest.mark.parametrize("st,act", [DTYPES[0], DTYPES[2]])
def test_a_prompt_in_two_calls_and_a_step(st, act):
    """A prompt given in two calls and ended by a step: the state goes through the pool's rounding
    twice more than in one call, and both are within the 64-bit form's tolerance of it."""
    import torch
    T, cut = 211, 97
    A, bias = ref.layer(42, FULL)
    xbc, raw, beta = ref.inputs(42, FULL, (T,), act)
    x, r, b, dA, db = to_dev(xbc, act), to_dev(raw, wl.F32), to_dev(beta, wl.F32), to_dev(A, wl.F32), to_dev(bias, wl.F32)
    desc = bd.layer_desc(FULL, state=st, act=act)
    pool = to_dev(states(42, FULL, 1, st), st)
    y = torch.zeros(T, 4, 128, dtype=x.dtype, device="cuda")
    one = torch.ones(1, dtype=torch.uint8, device="cuda")
    for i, (lo, hi) in enumerate(((0, cut), (cut, T - 1))):
        bd.gdn_chunk_scan(desc, pool, to_i32([0, hi - lo]), to_i32([0]), *[t[lo:hi].contiguous() for t in _vkq(FULL, x)],
                          r[lo:hi], b[lo:hi], dA, y[lo:hi], _work(FULL, hi - lo, 1, st, act), dt_bias=db,
                          has_initial_state=one * i)
    bd.gdn_state_update(desc, pool, to_i32([0]), x[None, T - 1:], r[None, T - 1:], b[None, T - 1:], dA, y[T - 1:], dt_bias=db)
    v, k, q = ref.split(FULL, wl.upcast(xbc, act))
    S, out = ref.sequence(np.zeros((4, 128, 128)), v, k, q, raw.astype(float), beta.astype(float), A.astype(float),
                          bias.astype(float))
    assert tile_rel_err(f64(y)[:, :, None], out[:, :, None], 3) <= tol(act, True)
    assert tile_rel_err(f64(pool)[0], S[-1], 2) <= tol(st, True)


def test_scan_offsets_past_32_bits():
    """Values of over 2^32 bytes and elements past 2^31: the last sequence as if it were alone."""
    import torch
    shape = wl.LayerShape(nheads=128, head_dim=128, d_state=128, n_groups=2)
    T, L = 140000, 70
    x = torch.zeros(T, shape.conv_dim, dtype=torch.bfloat16, device="cuda")
    xbc, raw, beta = ref.inputs(43, shape, (L,), wl.BF16)
    x[-L:] = to_dev(xbc, wl.BF16)
    r = torch.zeros(T, 128, device="cuda")
    b = torch.zeros(T, 128, device="cuda")
    r[-L:], b[-L:] = to_dev(raw, wl.F32), to_dev(beta, wl.F32)
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(43, shape))
    outs = []
    for lens, lo in (([T - L, L], 0), ([L], T - L)):
        v, k, q = (t.contiguous() for t in _vkq(shape, x[lo:]))
        n = T - lo
        y = torch.zeros(n, 128, 128, dtype=torch.bfloat16, device="cuda")
        pool = torch.zeros(2, 128, 128, 128, dtype=torch.bfloat16, device="cuda")
        bd.gdn_chunk_scan(bd.layer_desc(shape), pool, to_i32(wl.cu_seqlens(lens)), to_i32([1, 0][-len(lens):]), v, k, q, r[lo:],
                          b[lo:], A, y, _work(shape, n, len(lens), wl.BF16, wl.BF16), dt_bias=bias)
        outs.append((y[-L:].clone(), pool[0].clone(), y[:-L].any()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1]) and not outs[0][2]
