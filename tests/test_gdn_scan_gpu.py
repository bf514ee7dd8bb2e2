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
from test_gdn_gpu import DTYPES, FULL, _vkq, _work, states, tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    bld.build()
    bd.lib()
    torch.cuda.set_device(0)


PAIR = wl.LayerShape(nheads=2, head_dim=128, d_state=128, n_groups=1)
NARROW = wl.LayerShape(nheads=2, head_dim=64, d_state=128, n_groups=1)
BOTH = [DTYPES[0], DTYPES[1]]  # bf16 states (in chunks) and fp32 states (token by token), bf16 activations
SMALLEST = 2.0 ** -100  # a tile below it holds what fp32 need not keep apart from zero


def tile_err(got, want):
    """Largest error of a head's tile over the tile's largest value: (heads, ..) arrays."""
    axes = tuple(range(1, want.ndim))
    return float((np.abs(got - want).max(axis=axes) / np.maximum(np.abs(want).max(axis=axes), SMALLEST)).max())


def follow(seed, shape, st, lens, edit=None, init=None, interval=0, act=wl.BF16, flags={}, skip=(), y_tol=None, s_tol=None):
    """One call on sequences of these lengths, each 64-token tile of the outputs, each final state and each checkpoint
    (one every `interval` tokens) against the 64-bit form.  edit(xbc, dt, beta, states) changes the inputs, as float64,
    before they are stored; tiles whose number is in skip are only asked to be finite."""
    import torch
    T, n = int(sum(lens)), len(lens)
    H, HP = shape.nheads, shape.nheads * shape.head_dim
    A, bias = ref.layer(seed, shape)
    xbc, raw, beta = (np.array(wl.upcast(a, d)) for a, d in zip(ref.inputs(seed, shape, (T,), act), (act, wl.F32, wl.F32)))
    kept = [L // interval if interval else 0 for L in lens]
    before = np.array(wl.upcast(states(seed, shape, n + sum(kept), st), st))
    if edit:
        edit(xbc, raw, beta, before)
    stored = [wl.store(a, d) for a, d in ((xbc, act), (raw, wl.F32), (beta, wl.F32), (before, st))]
    ckpt = np.full((n, max(1, max(kept))), -1)
    for i, k in enumerate(kept):
        ckpt[i, :k] = n + sum(kept[:i]) + np.arange(k)
    dx, dr, db, pool = (to_dev(a, d) for a, d in zip(stored, (act, wl.F32, wl.F32, st)))
    y = torch.zeros(T, H, shape.head_dim, dtype=dx.dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = wl.cu_seqlens(lens)
    bd.gdn_chunk_scan(bd.layer_desc(shape, state=st, act=act), pool, to_i32(cu), to_i32(np.arange(n)),
                      *[t.contiguous() for t in _vkq(shape, dx)], dr, db, to_dev(A, wl.F32), y, _work(shape, T, n, st, act),
                      dt_bias=to_dev(bias, wl.F32), has_initial_state=None if init is None else to_dev(np.array(init), wl.F32).byte(),
                      ckpt_slots=to_i32(ckpt) if interval else None, ckpt_interval=interval, err_word=err,
                      **{{"softplus": "dt_softplus", "sigmoid": "beta_sigmoid", "l2norm": "qk_l2norm"}.get(k, k): w
                         for k, w in flags.items()})
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    xbc, raw, beta, before = (wl.upcast(a, d) for a, d in zip(stored, (act, wl.F32, wl.F32, st)))
    got, after = f64(y), f64(pool)
    assert np.isfinite(got).all() and np.isfinite(after).all()
    y_tol, s_tol = y_tol or tol(act, True), s_tol or tol(st, True)
    v, k, q = ref.split(shape, xbc)
    rep = H // shape.n_groups
    k, q = (np.repeat(ref.unit(x, flags.get("l2norm", True)), rep, axis=1) for x in (k, q))
    a, b = ref.gates(raw, beta, A.astype(float), bias.astype(float), flags.get("softplus", True), flags.get("sigmoid", True))
    scale = flags.get("scale", shape.d_state ** -0.5)
    for i, L in enumerate(lens):
        S = before[i] if init is not None and init[i] else np.zeros(before.shape[1:])
        want = np.zeros((L, H, shape.head_dim))
        for t in range(L):
            S, want[t] = ref.step(S, v[cu[i] + t], k[cu[i] + t], q[cu[i] + t], a[cu[i] + t], b[cu[i] + t], scale)
            if interval and (t + 1) % interval == 0 and t // 64 not in skip:
                assert tile_err(after[ckpt[i, t // interval]], S) <= s_tol, f"checkpoint after {t + 1}"
        for c in range((L + 63) // 64):
            rows = slice(64 * c, min(L, 64 * c + 64))
            if c not in skip:
                assert tile_err(got[cu[i]:cu[i + 1]][rows].transpose(1, 0, 2), want[rows].transpose(1, 0, 2)) <= y_tol, f"tile {c}"
        assert tile_err(after[i], S) <= s_tol, "final state"


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


# ---- numbers whose size changes along a sequence ----

@pytest.mark.parametrize("shape", [PAIR, NARROW], ids=["128", "64"])
@pytest.mark.parametrize("st,act", BOTH)
@pytest.mark.parametrize("loud", [512.0, 1e36])
def test_values_after_a_state_that_vanished(shape, st, act, loud):
    """Loud values, a stretch whose steps wipe the state out while nothing is written, and ordinary values: more than
    2^126 lies between the largest numbers of chunk 0 and of chunk 16."""
    HP = shape.nheads * shape.head_dim

    def edit(xbc, raw, beta, before):
        xbc[:64, :HP] = np.sign(xbc[:64, :HP]) * loud
        xbc[14 * 64:18 * 64, :HP] = 0
        raw[14 * 64:18 * 64] = 300
        if loud > 512:  # what the loud values left has to be gone before the tiles that are compared
            raw[64:14 * 64], xbc[64:14 * 64, :HP] = 300, 0

    follow(51, shape, st, [20 * 64 + 5], edit, skip=range(18))


# ---- write gates and keys over the rule's whole domain, 0 <= b |k|^2 <= 2 ----

HP, GN = 256, 128  # of PAIR


@pytest.mark.parametrize("st,act", BOTH)
@pytest.mark.parametrize("logit", [-12, -14, -16, -18, -30])
@pytest.mark.parametrize("shape", [PAIR, NARROW], ids=["128", "64"])
def test_gates_nearly_closed(shape, st, act, logit):
    """Little is written and nothing was there: outputs and state are as small as the gates."""
    def edit(xbc, raw, beta, before):
        beta += logit

    follow(52, shape, st, [200, 64, 3], edit)


@pytest.mark.parametrize("st,act", BOTH)
def test_gates_that_open_and_close(st, act):
    def edit(xbc, raw, beta, before):
        beta[:100] -= 18
        beta[160:230:3] -= 40
        beta[260:] -= 12

    follow(53, PAIR, st, [300], edit, init=[1])


@pytest.mark.parametrize("st,act", BOTH)
@pytest.mark.parametrize("length,gate", [(1000.0, 1e-6), (3000.0, 1e-7), (1e8, 1e-16), (0.004, 6e4), (1e-8, 1e16), (None, 1.0)])
def test_keys_of_any_length(st, act, length, gate):
    """Keys and gates as they are: the product b |k|^2 is the rule's, whatever each of them is (None: lengths from
    1/1000 to 1000 side by side, their gates to match)."""
    def edit(xbc, raw, beta, before):
        k = xbc[:, HP:HP + GN]
        k /= np.sqrt((k * k).sum(1, keepdims=True))
        lengths = length or np.exp(wl.rng(54, 3).uniform(-7, 7, (len(k), 1)))
        k *= lengths
        beta[...] = wl.rng(54, 4).uniform(0.3, 1.0, beta.shape) * (gate if length else 1 / lengths ** 2)
        before *= gate * (length or 1)  # what such writes leave

    follow(54, PAIR, st, [200, 70], edit, init=[1, 0], flags=dict(sigmoid=False, l2norm=False))


@pytest.mark.parametrize("st,act", BOTH)
def test_full_reflections(st, act):
    """b |k|^2 = 2 and no decay: no write is forgotten, and no rounding either.  Five chunks' errors of 8e-4 rms, one
    sequence's tile being off by the root of their sum, stay within the scan's tolerance."""
    bias = ref.layer(55, PAIR)[1]

    def edit(xbc, raw, beta, before):
        raw[...] = -bias
        beta[...] = 2.0

    follow(55, PAIR, st, [300], edit, init=[1], flags=dict(softplus=False, sigmoid=False))


@pytest.mark.parametrize("st,act", BOTH)
def test_one_key_reflected_with_values_of_either_sign(st, act):
    """s <- -s + 2 v along one key: the state grows by 2 |v| a token, and a token's rounding stays in it.  In chunks
    64 roundings of twice 2^-12 / sqrt(3) of the state rms add up to 2.3e-3, over four chunks to 4.5e-3 and at the
    outside (4.5 deviations) to 2e-2; token by token in fp32 to 2^12 times less."""
    bias = ref.layer(56, PAIR)[1]

    def edit(xbc, raw, beta, before):
        raw[...] = -bias
        beta[...] = 2.0
        xbc[:, HP:HP + GN] = xbc[0, HP:HP + GN]
        xbc[:, :HP] = np.abs(xbc[:, :HP]) * np.where(np.arange(len(xbc)) % 2, 1, -1)[:, None]

    chunks = st == wl.BF16
    follow(56, PAIR, st, [200], edit, flags=dict(softplus=False, sigmoid=False), y_tol=2 ** -8 + 2e-2 if chunks else None,
           s_tol=2 ** -8 + 2e-2 if chunks else None)


@pytest.mark.parametrize("st,act", BOTH)
def test_reflections_keep_their_length(st, act):
    """The same over 300 tokens, for 16 keys: what a token's factor 1 - b |k|^2 = -1 is off by multiplies up with the
    tokens, so a key's rounding to 11 bits may not change its length (2^-12 of it would by itself be 600 * 2^-12 = 15 %
    at the end).  Five chunks' roundings as above: 2.3e-3 sqrt(5) rms, 4.5 deviations 2.3e-2."""
    shape = wl.LayerShape(nheads=16, head_dim=64, d_state=128, n_groups=16)
    at = shape.nheads * shape.head_dim
    bias = ref.layer(57, shape)[1]

    def edit(xbc, raw, beta, before):
        raw[...] = -bias
        beta[...] = 2.0
        xbc[:, at:at + 16 * 128] = xbc[0, at:at + 16 * 128]
        xbc[:, :at] = np.abs(xbc[:, :at]) * np.where(np.arange(len(xbc)) % 2, 1, -1)[:, None]

    chunks = st == wl.BF16
    follow(57, shape, st, [300], edit, flags=dict(softplus=False, sigmoid=False), y_tol=2 ** -8 + 2.3e-2 if chunks else None,
           s_tol=2 ** -8 + 2.3e-2 if chunks else None)


# ---- values that grow and shrink along a sequence ----

def decay_of(seed, shape, a):
    """(dt without softplus, flags) for a decay of a in every token and head."""
    A, bias = ref.layer(seed, shape)
    return np.log(a) / A - bias, dict(softplus=False)


@pytest.mark.parametrize("st,act", BOTH)
@pytest.mark.parametrize("shape", [PAIR, NARROW], ids=["128", "64"])
@pytest.mark.parametrize("exponent", [-17, -20, -23])
def test_values_and_state_that_fall(shape, st, act, exponent):
    """Values fall after 64 tokens and the state with them, by 0.74 a token."""
    dt, flags = decay_of(58, shape, 0.74)

    def edit(xbc, raw, beta, before):
        raw[...] = dt
        xbc[64:, :shape.nheads * shape.head_dim] *= 2.0 ** exponent

    follow(58, shape, st, [300], edit, init=[1], flags=flags)


@pytest.mark.parametrize("st,act", BOTH)
@pytest.mark.parametrize("a,power,chunks", [(0.98, 2, 20), (0.9, 10, 7), (0.9, -2, 20), (0.8, -3, 36), (0.5, -12, 6)])
def test_values_that_grow_and_shrink_by_the_chunk(st, act, a, power, chunks):
    dt, flags = decay_of(59, PAIR, a)

    def edit(xbc, raw, beta, before):
        raw[...] = dt
        xbc[:, :HP] *= 2.0 ** (power * (np.arange(len(xbc)) // 64))[:, None]

    follow(59, PAIR, st, [64 * chunks - 7], edit, flags=flags, interval=128)


@pytest.mark.parametrize("st,act", BOTH)
def test_a_loud_token_and_a_loud_seed(st, act):
    """One token, and one state from the pool, 2^15 times the rest."""
    dt, flags = decay_of(60, PAIR, 0.8)

    def edit(xbc, raw, beta, before):
        raw[...] = dt
        xbc[333, :HP] *= 2.0 ** 15
        before[1] *= 2.0 ** 15

    follow(60, PAIR, st, [700, 500], edit, init=[0, 1], flags=flags, interval=64)


@pytest.mark.parametrize("st,act", BOTH)
def test_nothing_written_for_twenty_chunks(st, act):
    """The state only decays, and what is written afterwards stands beside what is left of it."""
    dt, flags = decay_of(61, PAIR, 0.995)

    def edit(xbc, raw, beta, before):
        raw[...] = dt
        xbc[70:1300, :HP] = 0
        xbc[1300:, :HP] *= 2.0 ** -10

    follow(61, PAIR, st, [1400], edit, init=[1], flags=flags, interval=256)


@pytest.mark.parametrize("st,act", BOTH)
@pytest.mark.parametrize("shape", [PAIR, NARROW], ids=["128", "64"])
def test_many_chunks(shape, st, act):
    follow(62, shape, st, [2111, 1024, 1089], init=[1, 0, 1], interval=512)


@pytest.mark.parametrize("st,act", BOTH)
def test_what_lies_far_below_the_loudest_of_its_tokens(st, act):
    """Values that fall by 2^-40 while the state is halved with every token.  In chunks a row's numbers are held to
    2^-24 of the largest of the same 64 tokens: the chunk of the fall loses the quiet values, and the one after it starts
    from that loss.  From then on they are as exact as any."""
    dt, flags = decay_of(63, PAIR, 0.5)

    def edit(xbc, raw, beta, before):
        raw[...] = dt
        xbc[64:, :HP] *= 2.0 ** -40

    follow(63, PAIR, st, [320], edit, init=[1], flags=flags, skip=(1, 2) if st == wl.BF16 else ())


# ---- what is not a number ----

@pytest.mark.parametrize("what", ["value", "key", "query", "step", "gate"])
@pytest.mark.parametrize("st,act", BOTH)
def test_how_far_a_nan_reaches(st, act, what):
    """Later tokens of its sequence, and in chunks the other tokens of its own 64 too; never an earlier chunk, a
    checkpoint before it, another head (a value, a step or a gate) or another row of the state (a value)."""
    import torch
    T, bad = 200, 100
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(65, PAIR))
    xbc, raw, beta = ref.inputs(65, PAIR, (T,), act)
    outs = []
    for poison in (False, True):
        x, r, b = to_dev(xbc, act), to_dev(raw, wl.F32), to_dev(beta, wl.F32)
        if poison:
            at = {"value": (x, 5), "key": (x, HP + 3), "query": (x, HP + GN + 3), "step": (r, 0), "gate": (b, 0)}[what]
            at[0][bad, at[1]] = float("nan")
        pool = to_dev(states(65, PAIR, 4, st), st)
        y = torch.zeros(T, 2, 128, dtype=x.dtype, device="cuda")
        bd.gdn_chunk_scan(bd.layer_desc(PAIR, state=st, act=act), pool, to_i32([0, T]), to_i32([0]),
                          *[t.contiguous() for t in _vkq(PAIR, x)], r, b, A, y, _work(PAIR, T, 1, st, act), dt_bias=bias,
                          ckpt_slots=to_i32([[1, 2, 3]]), ckpt_interval=64)
        outs.append((f64(y), f64(pool)))
    (good, good_pool), (got, pool) = outs
    clean = 64 if st == wl.BF16 else bad
    np.testing.assert_array_equal(got[:clean], good[:clean])
    np.testing.assert_array_equal(pool[1], good_pool[1])
    assert np.isnan(got[bad, 0]).any()
    if what == "query":  # it is only read with
        np.testing.assert_array_equal(got[128:], good[128:])
        np.testing.assert_array_equal(pool, good_pool)
    else:
        assert np.isnan(got[bad + 1:, 0]).any(axis=1).all() and all(np.isnan(pool[i, 0]).any() for i in (0, 2, 3))
    if what in ("value", "step", "gate"):
        np.testing.assert_array_equal(got[:, 1], good[:, 1])
        np.testing.assert_array_equal(pool[:, 1], good_pool[:, 1])
    if what == "value":
        rows = [i for i in range(128) if i != 5]
        np.testing.assert_array_equal(got[:, 0, rows], good[:, 0, rows])
        np.testing.assert_array_equal(pool[:, 0, rows], good_pool[:, 0, rows])


# ---- heads that share keys in odd numbers ----

@pytest.mark.parametrize("st,act", BOTH)
@pytest.mark.parametrize("heads,head_dim,groups", [(3, 128, 3), (3, 128, 1), (5, 64, 5), (6, 64, 2), (1, 128, 1)])
def test_odd_numbers_of_heads_a_group(heads, head_dim, groups, st, act):
    shape = wl.LayerShape(nheads=heads, head_dim=head_dim, d_state=128, n_groups=groups)
    follow(66, shape, st, [200, 1, 64, 129], init=[1, 0, 1, 1], interval=64)


# ---- plans of many sequences ----

@pytest.mark.parametrize("st", [wl.BF16, wl.F32])
@pytest.mark.parametrize("nseq", [1030, 2500, 5000])
def test_many_sequences(nseq, st):
    """The same bytes as in calls of 200 sequences: over 1024 a thread of the plan numbers several, over 4096 they run
    in the order given."""
    import torch
    shape = wl.LayerShape(nheads=1, head_dim=64, d_state=128, n_groups=1)
    g = np.random.default_rng(nseq)
    lens = g.integers(0, 20, nseq)
    lens[g.permutation(nseq)[:40]] = g.integers(60, 200, 40)
    T, cu = int(lens.sum()), wl.cu_seqlens(lens)
    A, bias = (to_dev(a, wl.F32) for a in ref.layer(67, shape))
    xbc, raw, beta = ref.inputs(67, shape, (T,), wl.BF16)
    vkq = [t.contiguous() for t in _vkq(shape, to_dev(xbc, wl.BF16))]
    r, b = to_dev(raw, wl.F32), to_dev(beta, wl.F32)
    slots = g.permutation(nseq + 7)[:nseq].astype(np.int32)
    slots[g.permutation(nseq)[:20]] = -1
    init = torch.from_numpy(g.integers(0, 2, nseq).astype(np.uint8)).cuda()
    start = to_dev(states(67, shape, nseq + 7, st), st)
    outs = []
    for step in (nseq, 200):
        pool, y = start.clone(), torch.zeros(T, 1, 64, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        for i in range(0, nseq, step):
            j = min(nseq, i + step)
            lo, hi = int(cu[i]), int(cu[j])
            bd.gdn_chunk_scan(bd.layer_desc(shape, state=st), pool, to_i32(cu[i:j + 1] - lo), to_i32(slots[i:j]),
                              *[t[lo:hi] for t in vkq], r[lo:hi], b[lo:hi], A, y[lo:hi], _work(shape, hi - lo, j - i, st, wl.BF16),
                              dt_bias=bias, has_initial_state=init[i:j], err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        outs.append((y, pool))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert (outs[0][0] != 0).any(dim=2).all() and not torch.equal(outs[0][1], start)


# ---- steps of any size ----

@pytest.mark.parametrize("st,act", BOTH)
@pytest.mark.parametrize("step", [30.0, 1e3, 1e6, 3e38, float("inf")])
def test_steps_that_wipe_the_state_out(st, act, step):
    """Tokens whose decay is zero in any arithmetic among tokens of ordinary steps, in one chunk and at its ends: what
    comes after them decays as exactly as if they had not been that large."""
    def edit(xbc, raw, beta, before):
        raw[10:40] = step
        raw[63] = step
        raw[64] = step
        raw[100:190:9] = step
        raw[192:256] = step

    follow(68, PAIR, st, [300], edit, init=[1], interval=64)
