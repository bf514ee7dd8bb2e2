"""The gated delta rule in 64 bits, one token after another, as its formula reads: what the tests
compare the kernels with.  Inputs are numpy float64 arrays holding the stored values exactly."""
import math

import numpy as np

from recurrent_state_update_gb300 import workloads as wl


def unit(x, on=True):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6) if on else x


def gates(dt, beta, A, dt_bias, softplus=True, sigmoid=True):
    s = dt + (0.0 if dt_bias is None else dt_bias)
    step = np.where(s > 30, s, np.log1p(np.exp(np.minimum(s, 30)))) if softplus else s
    return np.exp(step * A), 1 / (1 + np.exp(-beta)) if sigmoid else beta


def step(S, v, k, q, a, b, scale):
    """States (H, P, N), v (H, P), k and q (H, N), a and b (H): the new states and the outputs."""
    S = S * a[:, None, None]
    u = b[:, None] * (v - np.einsum("hpn,hn->hp", S, k))
    S = S + u[:, :, None] * k[:, None, :]
    return S, scale * np.einsum("hpn,hn->hp", S, q)


def sequence(S, v, k, q, dt, beta, A, dt_bias, scale=None, softplus=True, sigmoid=True, l2norm=True):
    """A whole sequence from state S: v (T, H, P), k and q (T, G, N), dt and beta (T, H).  Returns the
    states after each token (T, H, P, N) and the outputs (T, H, P)."""
    rep = v.shape[1] // k.shape[1]
    k, q = (np.repeat(unit(x, l2norm), rep, axis=1) for x in (k, q))
    a, b = gates(dt, beta, A, dt_bias, softplus, sigmoid)
    scale = 1 / math.sqrt(k.shape[-1]) if scale is None else scale
    states, ys = [], []
    for t in range(v.shape[0]):
        S, y = step(S, v[t], k[t], q[t], a[t], b[t], scale)
        states.append(S)
        ys.append(y)
    T, H, P = v.shape
    return (np.array(states).reshape((T,) + S.shape), np.array(ys).reshape(T, H, P))


def int8_codes(S):
    """Scales (..., N) and codes (..., P, N) of states S."""
    top = np.abs(S).max(axis=-2)
    inv = np.where(top > 0, 127 / np.where(top > 0, top, 1), 0)
    return top / 127, np.rint(S * inv[..., None, :])


def layer(seed, shape):
    """A, dt_bias of a layer, as the package's workloads draw them."""
    prm = wl.layer_params(wl.rng(seed, 0), shape)
    return prm["A"], prm["dt_bias"]


def silu(x):
    return x / (1 + np.exp(-x))


def inputs(seed, shape, lead, act, dt="f32", steps=None):
    """Stored v | k | q channels (lead..., conv_dim), dt and beta (lead..., H)."""
    g = wl.rng(seed, 1)
    A, bias = layer(seed, shape)
    xbc = wl.store(silu(g.standard_normal(tuple(lead) + (shape.conv_dim,))), act)
    raw = wl.store(wl.step_dt(g, bias, tuple(lead), steps), dt)
    beta = wl.store(g.standard_normal(tuple(lead) + (shape.nheads,)), dt)
    return xbc, raw, beta


def split(shape, xbc):
    """v, k, q views of channels (..., conv_dim)."""
    HP, GN = shape.nheads * shape.head_dim, shape.n_groups * shape.d_state
    v = xbc[..., :HP].reshape(xbc.shape[:-1] + (shape.nheads, shape.head_dim))
    k = xbc[..., HP:HP + GN].reshape(xbc.shape[:-1] + (shape.n_groups, shape.d_state))
    q = xbc[..., HP + GN:].reshape(xbc.shape[:-1] + (shape.n_groups, shape.d_state))
    return v, k, q
