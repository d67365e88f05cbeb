"""Hand-worked cases of the fp64 oracle of the convolution, the scan and draft
verification (CPU)."""
import numpy as np

import oracle


def test_conv_by_hand():
    x = np.array([[[1.0], [2.0], [3.0]]])
    w, b = np.array([[10.0, 100.0, 1000.0]]), np.array([0.5])
    st = np.array([[[7.0, 8.0]]])
    out, mag = oracle.causal_conv(x, w, b, st, silu=False)
    assert out[0, :, 0].tolist() == [1870.5, 2180.5, 3210.5] and (mag == out).all()
    assert st.tolist() == [[[2.0, 3.0]]]
    # one token: the state moves by one; none: it stays
    st = np.array([[[7.0, 8.0]]])
    oracle.causal_conv(x, w, b, st, ctx=np.array([1], np.int32))
    assert st.tolist() == [[[8.0, 1.0]]]
    oracle.causal_conv(x, w, b, st, ctx=np.array([0], np.int32))
    assert st.tolist() == [[[8.0, 1.0]]]
    out, _ = oracle.causal_conv(x * 0, w * 0, np.array([2.0]), st, ctx=np.array([2], np.int32))
    assert abs(out[0, 0, 0] - 2 / (1 + np.exp(-2))) < 1e-15 and out[0, 2, 0] == 0


def test_scan_by_hand():
    # dt' = 1 (no bias, no softplus), decay 1/2 and 1/4, B = 1 and 2, C = 1 and 10
    x, dt = np.array([[[3.0], [5.0]]]), np.ones((1, 2, 1))
    A = np.log(np.array([[0.5, 0.25]]))
    B = np.tile(np.array([1.0, 2.0]), (1, 2, 1, 1))
    C = np.tile(np.array([1.0, 10.0]), (1, 2, 1, 1))
    st = np.array([[[2.0, 4.0]]])
    out, _, _ = oracle.channel_scan(x, A, B, C, dt, st, softplus=False, D=np.array([100.0]))
    # h: (1+3, 1+6) -> (2+5, 1.75+10)
    np.testing.assert_allclose(out[0, :, 0], [4 + 70 + 300, 7 + 117.5 + 500], rtol=1e-15)
    np.testing.assert_allclose(st, [[[7.0, 11.75]]], rtol=1e-15)


def test_scan_is_the_head_recurrence_where_the_decays_agree():
    rng = np.random.default_rng(3)
    b, t, h, d, n = 2, 6, 3, 4, 16
    A1, dt1 = -rng.uniform(1, 8, h), rng.normal(size=(b, t, h)) * 0.5
    x, B, C = rng.normal(size=(b, t, h, d)), rng.normal(size=(b, t, 1, n)), rng.normal(size=(b, t, 1, n))
    D, z = rng.normal(size=h), rng.normal(size=x.shape)
    st = rng.normal(size=(b, h, d, n))
    st2, out2 = st.copy(), np.zeros(x.shape)
    oracle.prefill(x, A1, B, C, dt1, st2, out2, D=D, z=z, dt_bias=None)
    flat = st.reshape(b, h * d, n).copy()
    out, _, _ = oracle.channel_scan(
        x.reshape(b, t, -1), np.repeat(A1, d)[:, None].repeat(n, 1), B, C, np.repeat(dt1, d, 2), flat,
        D=np.repeat(D, d), z=z.reshape(b, t, -1))
    np.testing.assert_allclose(out, out2.reshape(b, t, -1), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(flat, st2.reshape(flat.shape), rtol=1e-12, atol=1e-12)


def test_verify_by_hand():
    p = np.array([[[0.5, 0.25, 0.25], [0.125, 0.375, 0.5], [0.0, 0.0, 1.0]]])
    q = np.array([[[0.25, 0.75, 0.0], [0.25, 0.25, 0.5]]])
    tok = np.array([[9, 0, 1]], np.int32)
    # 0.9 * 0.25 < 0.5 and 0.9 * 0.25 < 0.375: both stand, the last row draws
    acc, nxt, path = oracle.draft_verify(tok, p, np.array([[0.3, 0.9, 0.9]]), draft=q)
    assert (acc[0], nxt[0], path[0].tolist()) == (3, 2, [0, 1, 2])
    # token 1 instead: 0.5 * 0.75 > 0.25; residual of p - q = (0.25, 0, 0.25)
    tok = np.array([[9, 1, 1]], np.int32)
    for u0, want in ((0.0, 0), (0.49, 0), (0.5, 2), (0.99, 2)):
        acc, nxt, path = oracle.draft_verify(tok, p, np.array([[u0, 0.5, 0.1]]), draft=q)
        assert (acc[0], nxt[0], path[0].tolist()) == (1, want, [0, -1, -1])


def test_verify_tree_by_hand():
    # root with children 1 (token 0) and 2 (token 1), child 3 of node 2
    p = np.zeros((1, 4, 3))
    p[0, 0], p[0, 2], p[0, 3] = (0.5, 0.25, 0.25), (0.25, 0.5, 0.25), (0.0, 1.0, 0.0)
    tok, par = np.array([[9, 0, 1, 0]], np.int32), np.array([[-1, 0, 0, 2]], np.int32)
    u = np.array([[0.1, 0.6, 0.4, 0.2]])  # 0.6 >= 0.5: no; 0.4 * 0.5 < 0.25: yes; 0.2 < 0.25: yes
    acc, nxt, path = oracle.draft_verify(tok, p, u, parents=par)
    assert (acc[0], nxt[0], path[0].tolist()) == (3, 1, [0, 2, 3, -1])
    u = np.array([[0.1, 0.6, 0.5, 0.2]])  # 0.5 * 0.5 >= 0.25: no; what is left is token 2
    acc, nxt, path = oracle.draft_verify(tok, p, u, parents=par)
    assert (acc[0], nxt[0], path[0].tolist()) == (1, 2, [0, -1, -1, -1])
    acc, nxt, path = oracle.draft_verify(tok, p, u * 0, parents=par, max_accept=1)
    assert (acc[0], nxt[0], path[0].tolist()) == (1, 0, [0])


def test_verify_is_lossless():
    """The exact distribution of the next token over a fine grid of numbers."""
    p, q = np.array([0.4, 0.1, 0.5, 0.0]), np.array([0.1, 0.6, 0.1, 0.2])
    n = 200
    grid = (np.arange(n) + 0.5) / n
    u = np.stack(np.meshgrid(grid, grid), -1).reshape(-1, 2)
    got = np.zeros(4)
    for x in range(4):
        tok = np.tile(np.array([[0, x]], np.int32), (u.shape[0], 1))
        acc, nxt, _ = oracle.draft_verify(tok, np.tile(p, (u.shape[0], 2, 1)), u,
                                          draft=np.tile(q, (u.shape[0], 1, 1)))
        first = np.where(acc > 1, x, nxt)
        got += q[x] * np.bincount(first, minlength=4) / u.shape[0]
    np.testing.assert_allclose(got, p, atol=2.0 / n)  # a grid cell on either side of each step
