"""Pins of the 64-bit oracle of the rotary, short-convolution and state-space entry points: closed
forms, and gradients against central differences of the oracle's own forward."""
import numpy as np
import pytest

from oracle import mixers


def rng(n):
    return np.random.default_rng(n)


def differences(fn, x, dout, h=1e-5):
    """d sum(dout * fn(x)) / dx by central differences, element by element."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[i] = h
        g[i] = (np.sum(dout * fn(x + e)) - np.sum(dout * fn(x - e))) / (2 * h)
    return g


def close(a, b, tol=1e-7):
    assert np.abs(a - b).max() <= tol * (1 + np.abs(b).max())


@pytest.mark.parametrize("half", [True, False])
def test_rope_keeps_norms_composes_and_depends_on_distance(half):
    r = rng(1)
    x = r.standard_normal((1, 6, 2, 16))
    f = 10000.0 ** (-np.arange(0, 12, 2) / 12)
    pos = r.integers(0, 1000, (1, 6, 1))
    kw = dict(begin=2, half=half)
    y = mixers.rope(x, f, (12,), pos, **kw)
    assert np.array_equal(y[..., :2], x[..., :2]) and np.array_equal(y[..., 14:], x[..., 14:])
    close(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), 1e-12)
    close(mixers.rope(y, f, (12,), pos, inverse=True, **kw), x, 1e-12)
    close(mixers.rope(y, f, (12,), pos, pos0=5, **kw), mixers.rope(x, f, (12,), 2 * pos, pos0=5, **kw), 1e-10)
    # scores of a rotated query and key depend on the distance of their positions alone
    q, k = x[:, :1], x[:, 1:2]
    s = [np.sum(mixers.rope(q, f, (12,), np.full((1, 1, 1), p), **kw)
                * mixers.rope(k, f, (12,), np.full((1, 1, 1), p + 7), **kw)) for p in (0, 3, 100)]
    assert np.ptp(s) < 1e-10


def test_rope_sections_turn_by_their_own_axis():
    x = rng(2).standard_normal((2, 3, 1, 12))
    f = np.array([1.0, 0.1, 0.5, 2.0])
    pos = rng(3).integers(0, 9, (2, 3, 2))
    y = mixers.rope(x, f, (4, 4), pos, half=False)
    close(y[..., :4], mixers.rope(x[..., :4], f[:2], (4,), pos[..., :1], half=False), 1e-14)
    close(y[..., 4:8], mixers.rope(x[..., 4:8], f[2:], (4,), pos[..., 1:], half=False), 1e-14)
    assert np.array_equal(y[..., 8:], x[..., 8:])


def test_rope_gradient_is_the_inverse_rotation():
    r = rng(4)
    x, do = r.standard_normal((1, 2, 1, 6)), r.standard_normal((1, 2, 1, 6))
    f, pos = np.array([0.7, 0.2]), np.array([[[3], [11]]])
    num = differences(lambda v: mixers.rope(v, f, (4,), pos, mscale=1.3), x, do)
    close(mixers.rope(do, f, (4,), pos, mscale=1.3, inverse=True), num)


@pytest.mark.parametrize("K,silu,lens", [(4, True, None), (3, False, None), (2, True, [0, 5]), (4, True, [2, 7])])
def test_short_conv_gradients_against_differences(K, silu, lens):
    r = rng(10 + K)
    B, L, D = 2, 7, 3
    x, w, bias = r.standard_normal((B, L, D)), r.standard_normal((D, K)), r.standard_normal(D)
    S0, do, dS = r.standard_normal((B, K - 1, D)), r.standard_normal((B, L, D)), r.standard_normal((B, K - 1, D))
    g = mixers.short_conv(x, w, bias, silu=silu, S0=S0, lens=lens, dout=do, dS_out=dS)

    def total(x=x, w=w, bias=bias, S0=S0):
        o = mixers.short_conv(x, w, bias, silu=silu, S0=S0, lens=lens)
        return np.sum(do * o["o"]) + np.sum(dS * o["S_out"])

    for name, arr in (("x", x), ("w", w), ("bias", bias), ("S0", S0)):
        close(g["d" + name], differences(lambda v: total(**{name: v}), arr, 1.0), 1e-6)


def test_short_conv_is_the_dense_product_and_its_state_carries():
    r = rng(20)
    x, w = r.standard_normal((1, 9, 2)), r.standard_normal((2, 4))
    o = mixers.short_conv(x, w, silu=False)
    for c in range(2):
        M = sum(w[c, j] * np.eye(9, k=-(3 - j)) for j in range(4))
        close(o["o"][0, :, c], M @ x[0, :, c], 1e-13)
    a = mixers.short_conv(x[:, :2], w)
    b = mixers.short_conv(x[:, 2:], w, S0=a["S_out"])
    both = mixers.short_conv(x, w)
    close(np.concatenate([a["o"], b["o"]], 1), both["o"], 1e-14)
    assert np.array_equal(b["S_out"], both["S_out"])


def _scan_inputs(r, B, L, C, N, G):
    x = {"u": r.standard_normal((B, L, C)), "dt": r.standard_normal((B, L, C)),
         "A": -np.exp(r.standard_normal((C, N))), "Bm": r.standard_normal((B, L, G, N)),
         "Cm": r.standard_normal((B, L, G, N)), "D": r.standard_normal(C),
         "z": r.standard_normal((B, L, C)), "dt_bias": r.standard_normal(C),
         "S0": r.standard_normal((B, C, N))}
    return x, r.standard_normal((B, L, C)), r.standard_normal((B, C, N))


@pytest.mark.parametrize("lens,G", [(None, 1), ([4, 0], 2), ([1, 3], 1)])
def test_scan_gradients_against_differences(lens, G):
    x, do, dS = _scan_inputs(rng(30 + G), 2, 4, 4, 3, G)
    g = mixers.ssm_scan(**x, lens=lens, dout=do, dS_out=dS)

    def total(**over):
        o = mixers.ssm_scan(**{**x, **over}, lens=lens)
        return np.sum(do * o["y"]) + np.sum(dS * o["S_out"])

    names = {"u": "du", "dt": "ddt", "A": "dA", "Bm": "dB", "Cm": "dC", "D": "dD", "z": "dz",
             "dt_bias": "ddt_bias", "S0": "dS0"}
    for k, n in names.items():
        close(g[n], differences(lambda v: total(**{k: v}), x[k], 1.0), 1e-6)


def test_scan_closed_form_and_carry():
    x, _, _ = _scan_inputs(rng(40), 1, 6, 2, 3, 1)
    o = mixers.ssm_scan(**x)
    d = np.log1p(np.exp(x["dt"] + x["dt_bias"]))[0]
    cum = np.cumsum(d, 0)
    for t in range(6):       # y_t as the sum over every token before it
        for c in range(2):
            w = np.exp(cum[t, c] * x["A"][c]) * x["S0"][0, c]
            for s in range(t + 1):
                w = w + np.exp((cum[t, c] - cum[s, c]) * x["A"][c]) * d[s, c] * x["u"][0, s, c] * x["Bm"][0, s, 0]
            y = (w @ x["Cm"][0, t, 0] + x["D"][c] * x["u"][0, t, c]) * x["z"][0, t, c] / (1 + np.exp(-x["z"][0, t, c]))
            assert abs(y - o["y"][0, t, c]) < 1e-12
    cut = lambda a, b: {k: (v[:, a:b] if k in ("u", "dt", "Bm", "Cm", "z") else v) for k, v in x.items()}  # noqa: E731
    p = mixers.ssm_scan(**cut(0, 4))
    q = mixers.ssm_scan(**{**cut(4, 6), "S0": p["S_out"]})
    close(np.concatenate([p["y"], q["y"]], 1), o["y"], 1e-13)
    close(q["S_out"], o["S_out"], 1e-13)


def test_scan_with_equal_decays_is_gated_linear_attention():
    """A the same for all channels and d the same for all channels: the state is k^T v with a scalar
    gate, which the library's GLA oracle computes."""
    import oracle
    r = rng(50)
    L, C, N = 12, 32, 32
    dt, A = np.repeat(r.standard_normal((1, L, 1)), C, 2), np.full((C, N), -0.7)
    u, Bm, Cm = r.standard_normal((1, L, C)), r.standard_normal((1, L, 1, N)), r.standard_normal((1, L, 1, N))
    d = np.log1p(np.exp(dt))
    alpha = np.repeat(np.exp(-0.7 * d[..., :1])[:, :, None], N, 3)
    o, _ = oracle.gla(Cm.astype(np.float32), Bm.astype(np.float32), (d * u)[:, :, None].astype(np.float32),
                      alpha.astype(np.float32))
    y = mixers.ssm_scan(u, dt, A, Bm, Cm)["y"]
    assert np.abs(o[:, :, 0] - y).max() < 1e-5 * np.abs(y).max()
