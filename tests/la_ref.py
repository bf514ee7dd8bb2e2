"""Linear attention with a fixed decay a head in 64 bits, one token after another, as its formulas read, and the
plan of a batch one request after another: what the tests compare the kernels with.  Inputs are numpy float64
arrays holding the stored values exactly."""
import math

import numpy as np

from recurrent_state_update_gb300 import workloads as wl


def norm_rotate(x, weight=None, eps=None, positions=None, inv_freq=None, interleaved=False):
    """Rows (..., heads, N) at positions (...); eps None: no norm, inv_freq None: no rotation."""
    if eps is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if weight is None else weight)
    if inv_freq is None:
        return x
    half = len(inv_freq)
    angle = np.asarray(positions, np.float64)[..., None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(angle), np.sin(angle)
    out = x.copy()
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    return out


def sequence(S, v, k, q, log_decay, scale=None):
    """A whole sequence from state S (H, P, N): v (T, H, P), k and q (T, G, N).  Returns the states after each
    token (T, H, P, N) and the outputs (T, H, P)."""
    rep = v.shape[1] // k.shape[1]
    k, q = (np.repeat(x, rep, axis=1) for x in (k, q))
    a = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    scale = 1 / math.sqrt(k.shape[-1]) if scale is None else scale
    states, ys = np.empty((v.shape[0],) + S.shape), np.empty(v.shape)
    for t in range(v.shape[0]):
        S = S * a + v[t][:, :, None] * k[t][:, None, :]
        states[t] = S
        ys[t] = scale * np.einsum("hpn,hn->hp", S, q[t])
    return states, ys


def decays(seed, heads):
    """Heads that forget over 1 to 500 tokens, the first one all at once and the last one nothing."""
    d = -np.exp(-wl.rng(seed, 3).uniform(0, math.log(500.0), heads)).astype(np.float32)
    if heads > 2:
        d[0], d[-1] = -40.0, 0.0
    return d


def split(shape, xbc):
    """v, k, q views of channels (..., conv_dim)."""
    HP, GN = shape.nheads * shape.head_dim, shape.n_groups * shape.d_state
    v = xbc[..., :HP].reshape(xbc.shape[:-1] + (shape.nheads, shape.head_dim))
    k = xbc[..., HP:HP + GN].reshape(xbc.shape[:-1] + (shape.n_groups, shape.d_state))
    q = xbc[..., HP + GN:].reshape(xbc.shape[:-1] + (shape.n_groups, shape.d_state))
    return v, k, q


def batch_plan(new, past, table, block, num_slots, max_tokens, max_ckpt):
    """(outputs by name, error bits) of mamba_batch_plan."""
    rows = len(new)
    err = 0
    if any(n < 0 or c < 0 or n + c >= 2 ** 31 for n, c in zip(new, past)) or sum(new) > max_tokens:
        new, past, err = [0] * rows, [0] * rows, 4
    o = dict(cu_seqlens=[0], slot_ids=[], has_initial_state=[], copy_src=[], copy_dst=[], ckpt_slots=[], positions=[], token_rows=[])
    for i, (n, c) in enumerate(zip(new, past)):
        def page(t):
            j = (t - 1) // block if block else 0
            return table[i][j] if j < len(table[i]) else -1
        to = page(c + n) if n else -1
        start = page(c) if n and c else to
        kept = [-1] * max_ckpt
        bad = n > 0 and not (0 <= to < num_slots and 0 <= start < num_slots)
        for m in range(1, max_ckpt + 1):
            if block and n and c % block == 0 and m * block < n:
                j = c // block + m - 1
                kept[m - 1] = table[i][j] if j < len(table[i]) else -2
                bad |= not -1 <= kept[m - 1] < num_slots
        if bad:
            err |= 1
        o["cu_seqlens"].append(o["cu_seqlens"][-1] + n)
        o["slot_ids"].append(-2 if bad else to)
        o["has_initial_state"].append(int(n > 0 and c > 0))
        moved = not bad and start != to
        o["copy_src"].append(start if moved else -1)
        o["copy_dst"].append(to if moved else -1)
        o["ckpt_slots"].append([-1] * max_ckpt if bad else kept)
        o["positions"] += range(c, c + n)
        o["token_rows"] += [i] * n
    for n in ("positions", "token_rows"):
        o[n] += [-1] * (max_tokens - len(o[n]))
    return o, err
