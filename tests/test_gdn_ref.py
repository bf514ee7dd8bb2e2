"""CPU checks of the gated delta rule's 64-bit form: what the mathematics fixes."""
import numpy as np

import gdn_ref as ref


def _case(seed, T=70, H=4, G=2, P=6, N=8):
    g = np.random.default_rng(seed)
    return dict(S=0.3 * g.standard_normal((H, P, N)), v=g.standard_normal((T, H, P)), k=g.standard_normal((T, G, N)),
                q=g.standard_normal((T, G, N)), dt=g.standard_normal((T, H)), beta=g.standard_normal((T, H)),
                A=-np.exp(g.uniform(0, 2, H)), dt_bias=g.standard_normal(H) - 3)


def test_orthonormal_keys_are_recalled():
    """No decay and a full write: after writing N orthonormal keys the state returns each value."""
    g = np.random.default_rng(1)
    N, P = 8, 5
    keys = np.linalg.qr(g.standard_normal((N, N)))[0]
    v = g.standard_normal((N, 1, P))
    S, y = ref.sequence(np.zeros((1, P, N)), v, keys[:, None], keys[:, None], np.zeros((N, 1)), np.ones((N, 1)),
                        np.array([-1.0]), None, scale=1.0, softplus=False, sigmoid=False, l2norm=False)
    np.testing.assert_allclose(S[-1][0] @ keys.T, v[:, 0].T, atol=1e-12)
    np.testing.assert_allclose(y, v, atol=1e-12)


def test_a_second_write_to_a_key_replaces_the_first():
    k = np.zeros((2, 1, 4))
    k[:, 0, 1] = 1
    v = np.array([[[1.0, 2.0]], [[5.0, -3.0]]])
    S, _ = ref.sequence(np.zeros((1, 2, 4)), v, k, k, np.zeros((2, 1)), np.ones((2, 1)), np.array([-1.0]), None,
                        softplus=False, sigmoid=False, l2norm=False)
    np.testing.assert_allclose(S[-1][0][:, 1], [5.0, -3.0])


def test_no_write_gate_leaves_only_the_decay():
    c = _case(2, T=3)
    c["beta"] = np.zeros_like(c["beta"])
    S, _ = ref.sequence(**c, sigmoid=False)
    a, _ = ref.gates(c["dt"], c["beta"], c["A"], c["dt_bias"])
    np.testing.assert_allclose(S[-1], c["S"] * a.prod(0)[:, None, None], rtol=1e-12)


def test_the_sequence_equals_its_matrix_form():
    """U = (I + L)^-1 diag(b) (V - diag(e^c) K S0^T), Y and the last state from U."""
    c = _case(3)
    S, y = ref.sequence(**c)
    a, b = ref.gates(c["dt"], c["beta"], c["A"], c["dt_bias"])
    T, H, _ = c["v"].shape
    for h in range(H):
        k, q = (ref.unit(c[n])[:, h // 2] for n in ("k", "q"))
        cum = np.cumsum(np.log(a[:, h]))
        E = np.tril(np.exp(cum[:, None] - cum[None]))
        L = b[:, h, None] * (k @ k.T) * np.tril(E, -1)
        r = c["v"][:, h] - np.exp(cum)[:, None] * (k @ c["S"][h].T)
        U = np.linalg.solve(np.eye(T) + L, b[:, h, None] * r)
        Y = (np.exp(cum)[:, None] * (q @ c["S"][h].T) + (E * (q @ k.T)) @ U) / np.sqrt(8)
        np.testing.assert_allclose(y[:, h], Y, rtol=1e-9, atol=1e-10)
        last = np.exp(cum[-1]) * c["S"][h] + U.T @ (np.exp(cum[-1] - cum)[:, None] * k)
        np.testing.assert_allclose(S[-1][h], last, rtol=1e-9, atol=1e-10)


def test_codes_of_a_decayed_state_do_not_move():
    """A decay scales every column's maximum with the column: codes stay, scales decay."""
    S = np.random.default_rng(4).standard_normal((2, 16, 8))
    s0, c0 = ref.int8_codes(S)
    s1, c1 = ref.int8_codes(0.9 * (c0 * s0[:, None]))
    np.testing.assert_array_equal(c0, c1)
    np.testing.assert_allclose(s1, 0.9 * s0, rtol=1e-12)
