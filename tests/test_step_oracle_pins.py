"""Pins of the post-training step's fp64 oracle: closed forms, gradients
against central differences, and the packed order of block scales."""
import numpy as np
import pytest

from oracle import step_oracle as S


@pytest.mark.parametrize("fmt,fmax", [("e4m3", 448.0), ("e5m2", 57344.0)])
def test_block_scales_at_binade_edges(fmt, fmax):
    x = np.zeros((6, 128), np.float32)
    x[0, 3] = fmax                    # exactly representable: scale 1
    x[1, 3] = np.nextafter(np.float32(fmax), np.float32(np.inf))
    x[2, 0] = -fmax / 4
    x[3, 1] = 1e-44                   # below fmax 2^-126: the least scale
    x[5, 2] = np.inf
    q, s = S.block_quantize(x, 1, 128, fmt)
    assert s[:, 0].tolist() == [127, 128, 125, 1, 127, 255]
    assert (q[5] == 0x7F).all() and (q[4] == 0).all()
    v = S.block_dequantize(q, s, 1, 128, fmt)
    assert v[0, 3] == fmax and v[2, 0] == -fmax / 4 and np.isnan(v[5]).all()


def test_packed_order_is_a_bijection_of_words_per_row():
    rows, K = 300, 128 * 6
    ids = (np.arange(rows)[:, None] * 6 + np.arange(6)[None]) % 251
    p = S.pack_scales(ids.astype(np.uint8), rows, K)
    assert p.size == S.packed_bytes(rows, K) == 3 * 2 * 512
    # a 32-bit word holds a row's four consecutive blocks
    w = p.reshape(3, 2, 32, 4, 4)     # row chunk, block chunk, r % 32, (r % 128) / 32, block % 4
    for r in (0, 31, 32, 127, 128, 299):
        got = w[r // 128, :, r % 32, (r % 128) // 32].reshape(-1)
        assert got[:6].tolist() == ids[r].tolist() and (got[6:] == 127).all()


def test_qknorm_rope_keeps_the_norm_and_passes_v():
    rng = np.random.default_rng(0)
    M, nq, nk, D = 5, 2, 1, 16
    x = rng.standard_normal((M, (nq + 2 * nk) * D))
    y = S.qknorm_rope(x, np.ones(D), np.ones(D), np.arange(M), nq, nk, D, 0.0)
    h = y[:, :3 * D].reshape(M, 3, D)
    assert np.allclose((h * h).sum(2), D)       # unit rms, and a rotation keeps it
    assert (y[:, 3 * D:] == x[:, 3 * D:]).all()
    assert np.allclose(y[0, :D], x[0, :D] / np.sqrt((x[0, :D] ** 2).mean()))  # position 0


def test_qknorm_rope_backward_against_differences():
    rng = np.random.default_rng(1)
    M, nq, nk, D, eps = 3, 2, 1, 16, 1e-2
    x, d = rng.standard_normal((2, M, (nq + 2 * nk) * D))
    gq, gk = rng.uniform(0.5, 1.5, (2, D))
    pos = np.array([7, 0, 900])

    def f(x, gq, gk):
        return float((S.qknorm_rope(x, gq, gk, pos, nq, nk, D, eps) * d).sum())

    dx, dgq, dgk = S.qknorm_rope_backward(x, d, gq, gk, pos, nq, nk, D, eps)
    e = 1e-5
    for i in np.ndindex(x.shape):
        p = np.zeros_like(x)
        p[i] = e
        assert abs((f(x + p, gq, gk) - f(x - p, gq, gk)) / (2 * e) - dx[i]) < 1e-7
    for i in range(D):
        p = np.zeros(D)
        p[i] = e
        assert abs((f(x, gq + p, gk) - f(x, gq - p, gk)) / (2 * e) - dgq[i]) < 1e-7
        assert abs((f(x, gq, gk + p) - f(x, gq, gk - p)) / (2 * e) - dgk[i]) < 1e-7


@pytest.mark.parametrize("old,ref", [(True, True), (True, False), (False, True)])
def test_policy_loss_gradients_against_differences(old, ref):
    rng = np.random.default_rng(2)
    M, d, V, T = 7, 4, 11, 0.7
    H, W = rng.standard_normal((M, d)), rng.standard_normal((V, d))
    y = rng.integers(0, V, M)
    adv, w = rng.standard_normal(M), rng.uniform(0.1, 1.0, M)
    w[3], y[3] = 0.0, -100
    lp = S.policy_loss(H, W, y, adv, w, None, None, 0.2, 0.2, 0.0, T)["logp"]
    o = lp + rng.normal(0, 0.3, M) if old else lp
    f = lp + rng.normal(0, 0.5, M) if ref else None

    def loss(H, W):
        return S.policy_loss(H, W, y, adv, w, o, f, 0.2, 0.28, 0.1, T)["stats"][0]

    # without old log-probabilities the ratio is 1 but its gradient is that of exp(lp - stop(lp))
    r = S.policy_loss(H, W, y, adv, w, o if old else None, f, 0.2, 0.28, 0.1, T)
    e = 1e-6
    for A, G, which in ((H, r["dH"], 0), (W, r["dWt"], 1)):
        for i in np.ndindex(A.shape):
            p = np.zeros_like(A)
            p[i] = e
            num = (loss(H + p, W) - loss(H - p, W) if which == 0 else loss(H, W + p) - loss(H, W - p)) / (2 * e)
            assert abs(num - G[i]) < 1e-7
    assert (r["dH"][3] == 0).all()


def test_policy_terms_clip_both_sides():
    lp = np.log(np.array([1.5, 1.5, 0.5, 0.5, 1.1]))
    adv = np.array([1.0, -1.0, 1.0, -1.0, 2.0])
    loss, pg, kl, clipped, g = S.policy_terms(lp, adv, np.ones(5), np.zeros(5), None, 0.8, 1.2, 0.3)
    assert np.allclose(pg, [-1.2, 1.5, -0.5, 0.8, -2.2]) and (kl == 0).all()
    assert clipped.tolist() == [1, 0, 0, 1, 0]
    assert np.allclose(g, [0, 1.5, -0.5, 0, -2.2])
