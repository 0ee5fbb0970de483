"""GPU parity of rotary positions, the short causal convolution and the selective state-space scan
(forward, backward, single tokens) against the 64-bit oracle, within its first-order bounds of an
fp32 evaluation and half a step of the output's type; and the calls around them: streams, graphs,
padded batches, rollouts, a layer that uses all three."""
import numpy as np
import pytest
import torch

from oracle import mixers

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def kta():
    from hybrid_linear_temporal_kta_b200 import build
    build.build()
    from hybrid_linear_temporal_kta_b200 import kta as mod
    return mod


def gpu(x, dtype=torch.float32):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


def host(t):
    return None if t is None else t.double().cpu().numpy()


def check(name, got, want, dtype=None):
    """got within half a step of its type and the oracle's bound."""
    val, bound = want
    g = host(got)
    assert g.shape == val.shape, name
    lim = mixers.rounded(val, bound, torch.finfo(dtype or got.dtype).eps) + 1e-35
    bad = ~(np.abs(g - val) <= lim)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(g - val) / lim):.2f} "
                           f"times its bound, first at {tuple(np.argwhere(bad)[0])}")


# ---------------------------------------------------------------------------------- rotary

ROPE = [
    # dtype, B, N, Hq, Hk, d, dims, begin, half, per_seq, pos0
    (torch.bfloat16, 1, 1, 1, None, 32, (32,), 0, True, False, 0),
    (torch.bfloat16, 2, 37, 3, 5, 128, (44, 42, 42), 0, False, True, 239),
    (torch.bfloat16, 2, 37, 3, 5, 128, (44, 42, 42), 0, True, False, 0),
    (torch.bfloat16, 1, 300, 4, 4, 128, (32, 48, 48), 0, True, True, 7),
    (torch.bfloat16, 3, 17, 2, None, 64, (48,), 8, True, True, 1 << 30),
    (torch.bfloat16, 1, 65, 1, 1, 64, (24,), 4, True, False, 0),
    (torch.bfloat16, 1, 65, 1, 1, 64, (2,), 62, True, False, -5),
    (torch.bfloat16, 1, 65, 2, 1, 64, (6,), 2, False, False, (1 << 31) - 4096),
    (torch.bfloat16, 1, 20, 2, None, 128, (20,), 106, False, False, 0),
    (torch.float32, 2, 33, 3, None, 64, (32,), 16, True, True, 211200),
    (torch.float32, 1, 129, 2, 7, 32, (6, 10, 4, 2), 4, False, True, 3),
    (torch.float32, 1, 129, 2, 2, 128, (120,), 4, True, True, 0),
    (torch.float32, 1, 5, 40, 40, 64, (12, 4), 0, True, False, 0),
]


@pytest.mark.parametrize("dtype,B,N,Hq,Hk,d,dims,begin,half,per_seq,pos0", ROPE)
@pytest.mark.parametrize("bwd", [False, True])
def test_rope_parity(kta, dtype, B, N, Hq, Hk, d, dims, begin, half, per_seq, pos0, bwd):
    r = np.random.default_rng(N + d + begin)
    xs = [gpu(r.standard_normal((B, N, H, d)), dtype) for H in (Hq, Hk) if H]
    freqs, _ = kta.rope_freqs(dims)
    pos = r.integers(-50, 4096, (B if per_seq else 1, N, len(dims)))
    tpos = torch.from_numpy(pos if per_seq else pos[0]).cuda()
    fn = kta.rope_bwd if bwd else kta.rope_fwd
    kw = dict(freqs=freqs, dims=dims, begin=begin, layout="half" if half else "interleaved", mscale=1.25, pos=tpos, pos0=pos0)
    got = fn(*xs, **kw)
    got = (got,) if len(xs) == 1 else got
    for x, g in zip(xs, got):
        want = mixers.rope(host(x), freqs.cpu().numpy(), dims, np.broadcast_to(pos, (B, N, len(dims))), begin=begin, half=half,
                           mscale=1.25, pos0=pos0, inverse=bwd, bounds=True)
        check("rope", g, want)
        still = [j for j in range(d) if not begin <= j < begin + sum(dims)]
        assert torch.equal(g[..., still], x[..., still])
    mine = [x.clone() for x in xs]                         # in place: the same bits
    fn(*mine, **kw, out=tuple(mine))
    assert all(torch.equal(a, b) for a, b in zip(mine, got))


def test_rope_head_range_defaults_and_non_finite_values(kta):
    x = torch.randn(2, 9, 6, 64, device="cuda")
    x[0, 3, 2, 5] = float("nan")
    x[0, 3, 2, 60] = float("inf")
    f, _ = kta.rope_freqs(32)
    full = kta.rope_fwd(x, freqs=f, dims=32, pos=torch.arange(9, device="cuda"))
    assert torch.equal(full.nan_to_num(), kta.rope_fwd(x, freqs=f, dims=32).nan_to_num())
    part = x.clone()
    kta.rope_fwd(part, freqs=f, dims=32, heads=(2, 5), out=part)
    assert torch.equal(part[:, :, 2:5].nan_to_num(), full[:, :, 2:5].nan_to_num())
    assert torch.equal(part[:, :, :2], x[:, :, :2]) and torch.equal(part[:, :, 5:], x[:, :, 5:])
    # a NaN reaches its pair alone, an infinity outside the part stays itself
    for layout, partner in (("half", 21), ("interleaved", 4)):
        y = kta.rope_fwd(x, freqs=f, dims=32, layout=layout)
        bad = ~torch.isfinite(y)
        assert bad[0, 3, 2, 5] and bad[0, 3, 2, partner] and y[0, 3, 2, 60] == float("inf") and bad.sum() == 3


# ---------------------------------------------------------------------------------- convolution

CONV = [
    # dtype, B, L, D, K, silu, bias, S0, lens
    (torch.bfloat16, 1, 1, 8, 4, True, True, False, None),
    (torch.bfloat16, 3, 2, 24, 4, True, True, True, None),
    (torch.bfloat16, 2, 257, 72, 4, True, True, True, [257, 0]),
    (torch.bfloat16, 5, 70, 200, 3, True, False, True, [1, 2, 70, 33, 64]),
    (torch.bfloat16, 2, 33, 8, 2, False, True, False, None),
    (torch.float32, 2, 300, 40, 4, True, True, True, None),
    (torch.float32, 3, 65, 16, 3, False, False, False, [-7, 99, 31]),
    (torch.float32, 1, 8, 136, 2, True, True, True, None),
    (torch.float32, 2, 3, 264, 4, True, True, False, [3, 1]),
]


def conv_case(r, dtype, B, L, D, K, bias, S0, lens):
    x = gpu(3 * r.standard_normal((B, L, D)), dtype)
    w, b = gpu(r.standard_normal((D, K))), gpu(r.standard_normal(D)) if bias else None
    s = gpu(r.standard_normal((B, K - 1, D)), dtype) if S0 else None
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    seen = None if lens is None else [min(max(v, 0), L) for v in lens]
    if seen:                                              # what lies behind a sequence is never read
        for i, v in enumerate(seen):
            x[i, v:] = float("nan")
    return x, w, b, s, n, seen


@pytest.mark.parametrize("dtype,B,L,D,K,silu,bias,S0,lens", CONV)
def test_short_conv_parity(kta, dtype, B, L, D, K, silu, bias, S0, lens):
    r = np.random.default_rng(L + D + K)
    x, w, b, s, n, seen = conv_case(r, dtype, B, L, D, K, bias, S0, lens)
    o, S = kta.short_conv_fwd(x, w, b, silu=silu, S0=s, lens=n, return_state=True)
    want = mixers.short_conv(np.nan_to_num(host(x)), host(w), host(b), silu=silu, S0=host(s), lens=seen, bounds=True)
    check("o", o, want["o"])
    assert np.array_equal(host(S), want["S_out"][0])
    mine = torch.full_like(x, 7.0)
    assert kta.short_conv_fwd(x, w, b, silu=silu, S0=s, lens=n, out=mine) is mine
    for i, v in enumerate(seen or [L] * B):
        assert torch.equal(mine[i, :v], o[i, :v]) and (mine[i, v:] == 7).all()


@pytest.mark.parametrize("dtype,B,L,D,K,silu,bias,S0,lens", CONV)
def test_short_conv_backward_parity(kta, dtype, B, L, D, K, silu, bias, S0, lens):
    r = np.random.default_rng(L + D + K)
    x, w, b, s, n, seen = conv_case(r, dtype, B, L, D, K, bias, S0, lens)
    do, dS = gpu(r.standard_normal((B, L, D)), dtype), gpu(r.standard_normal((B, K - 1, D)), dtype)
    for i, v in enumerate(seen or []):
        do[i, v:] = float("nan")
    for end in (None, dS):
        got = kta.short_conv_bwd(x, w, do, b, silu=silu, S0=s, lens=n, dS_out=end)
        want = mixers.short_conv(np.nan_to_num(host(x)), host(w), host(b), silu=silu, S0=host(s), lens=seen,
                                 dout=np.nan_to_num(host(do)), dS_out=host(end), bounds=True)
        for name, g in zip(("dx", "dw", "dbias", "dS0"), got):
            if g is not None:
                check(name, g, want[name])
        assert (got[2] is None) == (not bias) and (got[3] is None) == (not S0)
        again = kta.short_conv_bwd(x, w, do, b, silu=silu, S0=s, lens=n, dS_out=end)
        assert all(a is None or torch.equal(a, c) for a, c in zip(got, again))


def test_short_conv_backward_of_runs_that_fill_the_card(kta):
    """Enough rows and channels that the runs are stretched (100 tokens here on 148 SMs), with one sequence
    that ends inside a run."""
    x, w, b, s, n, seen = conv_case(np.random.default_rng(11), torch.bfloat16, 2, 3600, 4096, 4, True, True, [3600, 1551])
    do = gpu(np.random.default_rng(12).standard_normal(x.shape), torch.bfloat16)
    do[1, 1551:] = float("nan")
    got = kta.short_conv_bwd(x, w, do, b, S0=s, lens=n)
    want = mixers.short_conv(np.nan_to_num(host(x)), host(w), host(b), silu=True, S0=host(s), lens=seen,
                             dout=np.nan_to_num(host(do)), bounds=True)
    for name, g in zip(("dx", "dw", "dbias", "dS0"), got):
        check(name, g, want[name])


@pytest.mark.parametrize("dtype", TYPES)
def test_parameter_gradients_over_many_rows_and_few_channels(kta, dtype):
    """Hundreds of partial sums for a few columns: dw and dbias of the convolution, dA, dD and ddt_bias of the scan."""
    r = np.random.default_rng(21)
    x, w, b, _, n, seen = conv_case(r, dtype, 2, 4500, 8, 4, True, False, [4500, 4001])
    do = gpu(r.standard_normal(x.shape), dtype)
    do[1, 4001:] = float("nan")
    got = kta.short_conv_bwd(x, w, do, b, lens=n)
    want = mixers.short_conv(np.nan_to_num(host(x)), host(w), host(b), lens=seen, dout=np.nan_to_num(host(do)), bounds=True)
    for name, g in zip(("dx", "dw", "dbias"), got):
        check(name, g, want[name])
    x, kw, seen = scan_case(r, dtype, 2, 4500, 8, 4, 1, True, True, True, False, [4001, 4500])
    do = gpu(r.standard_normal(x["u"].shape), dtype)
    do[0, 4001:] = float("nan")
    got = kta.ssm_scan_bwd(**x, dout=do, **kw)
    want = scan_oracle(x, kw, seen, dout=np.nan_to_num(host(do)))
    for name, g in got.items():
        if g is not None:
            check(name, g, want[name])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [2, 3, 4])
def test_short_conv_backward_of_rows_behind_the_end(kta, dtype, K):
    """Rows behind a sequence add nothing to its gradients, whatever their windows hold: the state of a slot
    without rows, or a last row whose sum overflows behind the end alone."""
    r = np.random.default_rng(K)
    x, w, b, s, n, _ = conv_case(r, dtype, 2, 12, 16, K, True, True, [0, 12])
    do, dS = gpu(r.standard_normal((2, 12, 16)), dtype), gpu(r.standard_normal((2, K - 1, 16)), dtype)
    want = [kta.short_conv_bwd(x, w, do, b, S0=s, lens=n, dS_out=end) for end in (None, dS)]
    for bad in (float("nan"), float("inf"), float("-inf")):
        s[0] = bad
        for end, ok in zip((None, dS), want):
            got = kta.short_conv_bwd(x, w, do, b, S0=s, lens=n, dS_out=end)
            assert all(torch.equal(a, c) for a, c in zip(got, ok))
            assert torch.equal(got[3][0], torch.zeros_like(dS[0]) if end is None else dS[0])
    # the last row's own sum is 1e38 (the slope is 1 there), that of the row behind it infinite
    x, w = torch.zeros(1, 9, 8, device="cuda", dtype=dtype), torch.zeros(8, K, device="cuda")
    x[0, 8], w[:, K - 1], w[:, K - 2] = 2e38, 0.5, 2.0
    do = torch.ones_like(x)
    dx = kta.short_conv_bwd(x, w, do)[0]
    assert (dx[0, 8] == 0.5).all() and torch.isfinite(dx).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [2, 3, 4])
def test_short_conv_rollout_is_the_whole_sequence(kta, dtype, K):
    r = np.random.default_rng(K)
    x, w, b, s, _, _ = conv_case(r, dtype, 3, 11, 24, K, True, True, None)
    o, S = kta.short_conv_fwd(x, w, b, S0=s, return_state=True)
    state, other = s.clone(), torch.empty_like(s)
    for t in range(5):                                     # in place, then from one buffer to the other
        assert torch.equal(kta.short_conv_step(x[:, t].contiguous(), w, state, b), o[:, t])
    for t in range(5, 7):
        y = kta.short_conv_step(x[:, t].contiguous(), w, state, b, state_out=other)
        assert torch.equal(y, o[:, t])
        state, other = other, state
    y, state = kta.short_conv_fwd(x[:, 7:].contiguous(), w, b, S0=state, return_state=True)
    assert torch.equal(y, o[:, 7:]) and torch.equal(state, S)


# ---------------------------------------------------------------------------------- scan

SCAN = [
    # dtype, B, L, D, N, G, z, skip, bias, S0, lens
    (torch.bfloat16, 1, 1, 8, 16, 1, True, True, True, False, None),
    (torch.bfloat16, 2, 40, 72, 16, 1, True, True, True, True, None),
    (torch.bfloat16, 3, 130, 40, 16, 1, True, False, True, True, [130, 0, 77]),
    (torch.bfloat16, 1, 300, 8, 4, 1, False, False, False, False, None),
    (torch.bfloat16, 2, 65, 48, 8, 2, True, True, True, True, [64, 65]),
    (torch.bfloat16, 2, 33, 96, 32, 3, False, True, True, False, None),
    (torch.bfloat16, 1, 97, 16, 5, 2, True, True, False, True, None),
    (torch.float32, 2, 64, 32, 16, 1, True, True, True, True, None),
    (torch.float32, 3, 71, 24, 12, 3, True, True, True, True, [5, 71, 32]),
    (torch.float32, 1, 33, 40, 1, 1, False, True, True, False, None),
    (torch.float32, 1, 50, 8, 17, 1, True, False, True, True, [-3]),
    (torch.float32, 2, 9, 264, 3, 1, False, False, False, True, None),
    (torch.float32, 1, 1000, 16, 16, 1, True, True, True, True, None),
    (torch.bfloat16, 2, 45, 136, 12, 1, True, True, True, True, None),        # rows of 24 bytes
    (torch.bfloat16, 1, 70, 24, 6, 1, False, True, True, False, None),        # of 12
    (torch.bfloat16, 2, 40, 16, 24, 1, True, True, True, True, [40, 9]),
    (torch.float32, 1, 40, 48, 6, 2, True, False, True, True, None),
    (torch.bfloat16, 5, 100, 520, 16, 5, True, True, True, False, [0, 1, 31, 33, 100]),
]


def scan_case(r, dtype, B, L, D, N, G, z, skip, bias, S0, lens):
    dt0 = np.exp(r.uniform(np.log(1e-3), np.log(0.3), D))
    x = {"u": gpu(r.standard_normal((B, L, D)), dtype), "dt": gpu(r.standard_normal((B, L, D)) - (0 if bias else 3), dtype),
         "A": gpu(-np.exp(r.uniform(-1, 3, (D, N)))), "Bm": gpu(r.standard_normal((B, L, G, N)), dtype),
         "Cm": gpu(r.standard_normal((B, L, G, N)), dtype)}
    kw = {"D": gpu(r.standard_normal(D)) if skip else None, "z": gpu(2 * r.standard_normal((B, L, D)), dtype) if z else None,
          "dt_bias": gpu(np.log(np.expm1(dt0))) if bias else None,
          "S0": gpu(r.standard_normal((B, D, N))) if S0 else None}
    seen = None if lens is None else [min(max(v, 0), L) for v in lens]
    if seen:
        kw["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for i, v in enumerate(seen):
            for t in (x["u"], x["dt"], x["Bm"], x["Cm"], kw["z"]):
                if t is not None:
                    t[i, v:] = float("nan")
    return x, kw, seen


def scan_oracle(x, kw, seen, **more):
    clean = lambda t: None if t is None else np.nan_to_num(host(t))  # noqa: E731
    return mixers.ssm_scan(**{k: clean(v) for k, v in x.items()}, **{k: clean(v) for k, v in kw.items() if k != "lens"},
                           lens=seen, **more, bounds=True)


@pytest.mark.parametrize("dtype,B,L,D,N,G,z,skip,bias,S0,lens", SCAN)
def test_scan_parity(kta, dtype, B, L, D, N, G, z, skip, bias, S0, lens):
    x, kw, seen = scan_case(np.random.default_rng(L + D + N), dtype, B, L, D, N, G, z, skip, bias, S0, lens)
    y, S = kta.ssm_scan_fwd(**x, **kw, return_state=True)
    want = scan_oracle(x, kw, seen)
    check("S_out", S, want["S_out"])
    check("y", y, want["y"])
    mine = torch.full_like(x["u"], 7.0)
    assert kta.ssm_scan_fwd(**x, **kw, out=mine) is mine
    for i, v in enumerate(seen or [L] * B):
        assert torch.equal(mine[i, :v], y[i, :v]) and (mine[i, v:] == 7).all()


@pytest.mark.parametrize("dtype,B,L,D,N,G,z,skip,bias,S0,lens", SCAN)
def test_scan_backward_parity(kta, dtype, B, L, D, N, G, z, skip, bias, S0, lens):
    r = np.random.default_rng(L + D + N)
    x, kw, seen = scan_case(r, dtype, B, L, D, N, G, z, skip, bias, S0, lens)
    do, dS = gpu(r.standard_normal((B, L, D)), dtype), gpu(r.standard_normal((B, D, N)))
    for i, v in enumerate(seen or []):
        do[i, v:] = float("nan")
    for end in (None, dS):
        got = kta.ssm_scan_bwd(**x, dout=do, **kw, dS_out=end)
        want = scan_oracle(x, kw, seen, dout=np.nan_to_num(host(do)), dS_out=host(end))
        for name, there in (("dD", skip), ("dz", z), ("ddt_bias", bias), ("dS0", S0)):
            assert (got[name] is not None) == there, name
        for name, g in got.items():
            if g is not None:
                check(name, g, want[name])
        again = kta.ssm_scan_bwd(**x, dout=do, **kw, dS_out=end)
        assert all(a is None or torch.equal(a, again[n]) for n, a in got.items())
    mine = {n: torch.full_like(got[n], 7.0) for n in ("du", "ddt", "dB", "dC") + (("dz",) if z else ())}
    kta.ssm_scan_bwd(**x, dout=do, **kw, dS_out=end, out=mine)
    for n, t in mine.items():
        for i, v in enumerate(seen or [L] * B):
            assert torch.equal(t[i, :v], got[n][i, :v]) and (t[i, v:] == 7).all(), n


@pytest.mark.parametrize("dtype,B,D,N,G", [(torch.bfloat16, 5, 24, 16, 1), (torch.float32, 9, 16, 8, 2), (torch.bfloat16, 1, 40, 5, 1),
                                           (torch.float32, 4, 8, 32, 1), (torch.bfloat16, 3, 8, 2, 1), (torch.bfloat16, 4, 8, 32, 1)])
def test_scan_steps_follow_the_prompt(kta, dtype, B, D, N, G):
    x, kw, _ = scan_case(np.random.default_rng(D + N), dtype, B, 9, D, N, G, True, True, True, True, None)
    want = scan_oracle(x, kw, None)
    S0 = kw.pop("S0")
    cut = lambda a, b: ({k: v if k == "A" else v[:, a:b].contiguous() for k, v in x.items()},  # noqa: E731
                        {k: v[:, a:b].contiguous() if k == "z" else v for k, v in kw.items()})
    p, pk = cut(0, 5)
    y, state = kta.ssm_scan_fwd(**p, **pk, S0=S0, return_state=True)
    rows, other = [y], torch.empty_like(state)
    for t in range(5, 9):
        s, sk = cut(t, t + 1)
        s = {k: v if k == "A" else v[:, 0].contiguous() for k, v in s.items()}
        sk["z"] = sk["z"][:, 0].contiguous()
        if t < 7:
            rows.append(kta.ssm_scan_step(**s, state=state, **sk)[:, None])
        else:
            rows.append(kta.ssm_scan_step(**s, state=state, state_out=other, **sk)[:, None])
            state, other = other, state
    check("y", torch.cat(rows, 1), want["y"])
    check("state", state, want["S_out"])


def test_scan_long_segments_agree_with_pieces(kta):
    """A long sequence with few channels is cut into segments; in pieces short enough for one it is
    not. Both within the oracle's bound of each other."""
    x, kw, _ = scan_case(np.random.default_rng(5), torch.float32, 1, 3000, 8, 16, 1, True, True, True, True, None)
    y, S = kta.ssm_scan_fwd(**x, **kw, return_state=True)
    state, rows = kw["S0"], []
    for a in range(0, 3000, 100):
        p = {k: v if k == "A" else v[:, a:a + 100].contiguous() for k, v in x.items()}
        o, state = kta.ssm_scan_fwd(**p, D=kw["D"], z=kw["z"][:, a:a + 100].contiguous(), dt_bias=kw["dt_bias"], S0=state,
                                    return_state=True)
        rows.append(o)
    want = scan_oracle(x, kw, None)
    for name, t in (("y", y), ("y in pieces", torch.cat(rows, 1))):
        check(name, t, want["y"])
    check("S", S, want["S_out"])
    check("S in pieces", state, want["S_out"])


def test_scan_step_sizes_to_their_stated_error(kta):
    """With A = 0 and u = B = 1 the state after one token is d = log(1 + e^dt) itself. Relative error, in units of
    2^-24: |x| for the rounded argument of e^-|x| and 0.23 |x| for log2(e) in fp32; 4 for the exponential, 0.5 for
    the fit, 3 for its evaluation and 0.5 for the last sum."""
    x = torch.linspace(-80, 20, 100_000, dtype=torch.float64).float().cuda()[None, None]
    one = torch.ones(1, 1, 1, 1, device="cuda")
    _, S = kta.ssm_scan_fwd(torch.ones_like(x), x, torch.zeros(x.shape[2], 1, device="cuda"), one, one, return_state=True)
    step = kta.ssm_scan_step(torch.ones_like(x[0]), x[0], torch.zeros(x.shape[2], 1, device="cuda"), one[0], one[0],
                             torch.zeros(1, x.shape[2], 1, device="cuda"))
    want = np.logaddexp(0.0, host(x)[0, 0])
    lim = want * (1.25 * np.abs(host(x)[0, 0]) + 8) * 2.0 ** -24
    assert (np.abs(host(S)[0, :, 0] - want) <= lim).all()
    assert (np.abs(host(step)[0] - want) <= lim).all()


def test_scan_extreme_steps(kta):
    """Step sizes that under- and overflow: the state is kept exactly, or forgotten at once."""
    L, D, N = 40, 8, 16
    g = torch.Generator("cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    u, Bm, Cm, S0 = r(1, L, D), r(1, L, 1, N), r(1, L, 1, N), r(1, D, N)
    A = -torch.ones(D, N, device="cuda")
    y, S = kta.ssm_scan_fwd(u, torch.full_like(u, -200.0), A, Bm, Cm, S0=S0, return_state=True)
    assert torch.equal(S, S0) and torch.allclose(y[0], (S0[0][None] * Cm[0]).sum(-1), atol=1e-5)
    y, S = kta.ssm_scan_fwd(u, torch.full_like(u, 150.0), A, Bm, Cm, S0=S0, return_state=True)
    assert torch.allclose(S[0], 150 * u[0, -1][:, None] * Bm[0, -1], rtol=1e-5)
    gr = kta.ssm_scan_bwd(u, torch.full_like(u, 150.0), A, Bm, Cm, torch.ones_like(u), S0=S0)
    assert all(torch.isfinite(t).all() for t in gr.values() if t is not None)


def test_scan_of_growing_states_that_are_still_zero(kta):
    """A > 0 whose growth over a segment overflows: a state that no input has reached stays zero, and the
    last tokens come out as in a call of their own."""
    L, D, N = 512, 8, 16
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    u, Bm, Cm = r(1, L, D), r(1, L, 1, N), r(1, L, 1, N)
    u[:, :-2] = 0
    dt, A = torch.full_like(u, 3.5), torch.ones(D, N, device="cuda")   # exp(32 softplus(3.5)) > 2^128
    y, S = kta.ssm_scan_fwd(u, dt, A, Bm, Cm, return_state=True)
    last = [t[:, -2:].contiguous() for t in (u, dt, Bm, Cm)]
    y2, S2 = kta.ssm_scan_fwd(*last[:2], A, *last[2:], return_state=True)
    assert (y[:, :-2] == 0).all() and torch.equal(y[:, -2:], y2) and torch.equal(S, S2)
    assert torch.isfinite(S).all()


@pytest.mark.parametrize("dtype,B,L,D,N,lens", [
    (torch.float32, 1, 5, 8, 4, None), (torch.bfloat16, 2, 45, 40, 16, [45, 0]), (torch.float32, 1, 700, 16, 12, [333]),
    (torch.bfloat16, 1, 33, 8, 32, None), (torch.bfloat16, 3, 1, 8, 8, None)])
def test_scan_states_that_forget_at_once(kta, dtype, B, L, D, N, lens):
    """A = -inf is A = -1e30 to the last bit: rows that pad a tile (d = 0) or lie behind a sequence leave the
    state alone."""
    r = np.random.default_rng(L)
    x, kw, _ = scan_case(r, dtype, B, L, D, N, 1, True, True, True, True, lens)
    do, dS = gpu(r.standard_normal((B, L, D)), dtype), gpu(r.standard_normal((B, D, N)))
    some = torch.from_numpy(r.random((D, N)) < 0.5).cuda()
    outs = []
    for a in (-1e30, float("-inf")):
        x["A"] = torch.where(some, a, x["A"])
        y, S = kta.ssm_scan_fwd(**x, **kw, return_state=True)
        g = kta.ssm_scan_bwd(**x, dout=do, dS_out=dS, **kw)
        outs.append([y, S] + [t for t in g.values() if t is not None])
        if L == 1:
            one = {n: t if n == "A" else t[:, 0].contiguous() for n, t in x.items()}
            state = kw["S0"].clone()
            outs[-1] += [kta.ssm_scan_step(**one, state=state, D=kw["D"], z=kw["z"][:, 0].contiguous(),
                                           dt_bias=kw["dt_bias"]), state]
    assert all(torch.isfinite(t).all() for t in outs[0])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("scale", [1e-30, -1e-20, 2.0 ** -126])
def test_scan_of_small_states_that_grow(kta, scale):
    """A > 0: growth over one segment that overflows alone, while the state that it acts on stays finite; cut
    into segments or not, the state is the formula's."""
    L, D, N = 512, 8, 16
    r = np.random.default_rng(4)
    dt = np.full((1, L, D), -200.0)
    dt[:, 64:96] = np.log(np.expm1((90 if abs(scale) > 1e-25 else 96) / 32))        # e^90, e^96 over the 32 tokens
    x = {"u": torch.zeros(1, L, D, device="cuda"), "dt": gpu(dt), "A": torch.ones(D, N, device="cuda"),
         "Bm": gpu(r.standard_normal((1, L, 1, N))), "Cm": gpu(r.standard_normal((1, L, 1, N)))}
    kw = {"S0": gpu(scale * r.uniform(1, 2, (1, D, N)))}
    y, S = kta.ssm_scan_fwd(**x, **kw, return_state=True)
    want = scan_oracle(x, kw, None)
    check("S_out", S, want["S_out"])
    check("y", y, want["y"])
    state, rows = kw["S0"], []
    for a in range(0, L, 32):                               # one segment each
        piece = {n: t if n == "A" else t[:, a:a + 32].contiguous() for n, t in x.items()}
        o, state = kta.ssm_scan_fwd(**piece, S0=state, return_state=True)
        rows.append(o)
    check("S in pieces", state, want["S_out"])
    check("y in pieces", torch.cat(rows, 1), want["y"])


def test_rope_refuses_numbers_out_of_range(kta):
    q, f = torch.zeros(1, 4, 2, 64, device="cuda"), torch.ones(16, device="cuda", dtype=torch.float64)
    for kw in (dict(pos0=1 << 64), dict(pos0=0.5), dict(begin=1 << 40), dict(dims=(32.0,))):
        with pytest.raises(ValueError):
            kta.rope_fwd(q, freqs=f, **{"dims": 32, **kw})


def test_sizes_past_their_c_types_are_value_errors(kta):
    x = torch.empty(1, 1 << 31, 8, device="cuda", dtype=torch.bfloat16)     # 2^31 tokens
    with pytest.raises(ValueError):
        kta.short_conv_fwd(x, torch.zeros(8, 4, device="cuda"))
    b = x.view(-1)[:1 << 31].view(1, 1 << 31, 1, 1)
    with pytest.raises(ValueError):
        kta.ssm_scan_fwd(x, x, torch.zeros(8, 1, device="cuda"), b, b)


@pytest.mark.parametrize("dtype,N", [(torch.bfloat16, 16), (torch.bfloat16, 8), (torch.float32, 16)])
def test_scan_rows_of_b_and_c_at_any_address(kta, dtype, N):
    """B and C, and the buffers of their gradients, may begin at any element."""
    x, kw, _ = scan_case(np.random.default_rng(N), dtype, 1, 90, 24, N, 1, True, True, True, True, None)
    do = torch.ones_like(x["u"])
    want_y = kta.ssm_scan_fwd(**x, **kw)
    want_g = kta.ssm_scan_bwd(**x, dout=do, **kw)
    for off in (1, 2, 4):
        def moved(t):
            buf = torch.full((t.numel() + off,), float("nan"), dtype=t.dtype, device="cuda")
            buf[off:] = t.reshape(-1)
            return buf[off:].view(t.shape)
        y = {**x, "Bm": moved(x["Bm"]), "Cm": moved(x["Cm"])}
        assert torch.equal(kta.ssm_scan_fwd(**y, **kw), want_y)
        out = {"dB": moved(x["Bm"]), "dC": moved(x["Cm"])}
        g = kta.ssm_scan_bwd(**y, dout=do, **kw, out=out)
        assert g["dB"] is out["dB"] and all(torch.equal(g[n], want_g[n]) for n in g if g[n] is not None)


# ---------------------------------------------------------------------------------- calls

def train_step(kta, x, w, bias, scan, kw, do):
    """Convolution, silu and scan, forward and backward."""
    c = kta.short_conv_fwd(x, w, bias)
    y = kta.ssm_scan_fwd(c, *scan, **kw)
    g = kta.ssm_scan_bwd(c, *scan, do, **kw)
    dx, dw, db, _ = kta.short_conv_bwd(x, w, g["du"], bias)
    return [y, dx, dw, db] + [g[n] for n in ("ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")]


def step_inputs(seed, dtype=torch.bfloat16, B=2, L=700, D=64, N=16):
    r = np.random.default_rng(seed)
    x, kw, _ = scan_case(r, dtype, B, L, D, N, 1, True, True, True, False, None)
    kw.pop("S0")
    w, b = gpu(r.standard_normal((D, 4))), gpu(r.standard_normal(D))
    return x["u"], w, b, (x["dt"], x["A"], x["Bm"], x["Cm"]), kw, gpu(r.standard_normal((B, L, D)), dtype)


def test_graphs_of_two_calls_replay_at_once(kta):
    """Two captured training steps share no scratch: replayed together on two streams, over and over,
    each gives the bits of its eager call."""
    a, b = step_inputs(1), step_inputs(2)
    want = [[t.clone() for t in train_step(kta, *i)] for i in (a, b)]
    graphs, outs = [], []
    for i in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(train_step(kta, *i))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for t in outs[0] + outs[1]:
            t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(got, w))


def test_rollout_replayed_as_a_graph(kta):
    """Steps in place inside a graph: each replay moves rows and state on by one token."""
    x, kw, _ = scan_case(np.random.default_rng(8), torch.bfloat16, 3, 12, 40, 16, 1, True, True, True, True, None)
    w, b = torch.randn(40, 4, device="cuda"), torch.randn(40, device="cuda")
    rows, state = torch.randn(3, 3, 40, device="cuda").bfloat16(), kw.pop("S0")
    tok = {n: t[:, 0].contiguous() for n, t in {**x, "z": kw["z"]}.items() if n != "A"}

    def one(rows, state):
        u = kta.short_conv_step(tok["u"], w, rows, b)
        return kta.ssm_scan_step(u, tok["dt"], x["A"], tok["Bm"], tok["Cm"], state, D=kw["D"], z=tok["z"],
                                 dt_bias=kw["dt_bias"])

    def put(t):
        for n in tok:
            tok[n].copy_((x[n] if n in x else kw[n])[:, t])

    mine = rows.clone(), state.clone()
    want = []
    for t in range(12):
        put(t)
        want.append(one(*mine))
    one(rows.clone(), state.clone())
    g = torch.cuda.CUDAGraph()
    r2, s2 = rows.clone(), state.clone()
    with torch.cuda.graph(g):
        y = one(rows, state)
    rows.copy_(r2), state.copy_(s2)
    for t in range(12):
        put(t)
        g.replay()
        assert torch.equal(y, want[t])
    assert torch.equal(rows, mine[0]) and torch.equal(state, mine[1])


def test_calls_on_two_streams_at_once(kta):
    a, b = step_inputs(3), step_inputs(4)
    want = [train_step(kta, *i) for i in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for i, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(train_step(kta, *i))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))


def test_stream_argument(kta):
    x, w, b, scan, kw, do = step_inputs(5)
    q = torch.randn(1, 50, 2, 64, device="cuda")
    f, _ = kta.rope_freqs(64)
    want = (kta.short_conv_fwd(x, w, b), kta.ssm_scan_fwd(x, *scan, **kw), kta.rope_fwd(q, freqs=f, dims=64),
            kta.ssm_scan_bwd(x, *scan, do, **kw)["dA"], kta.short_conv_bwd(x, w, do, b)[1])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = (kta.short_conv_fwd(x, w, b, stream=s), kta.ssm_scan_fwd(x, *scan, **kw, stream=s),
           kta.rope_fwd(q, freqs=f, dims=64, stream=s), kta.ssm_scan_bwd(x, *scan, do, **kw, stream=s)["dA"],
           kta.short_conv_bwd(x, w, do, b, stream=s)[1])
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_binding_refusals(kta):
    x, w, b, scan, kw, do = step_inputs(6, L=20)
    for bad in (lambda: kta.short_conv_fwd(x[:, ::2], w, b), lambda: kta.short_conv_fwd(x, w.t(), b),
                lambda: kta.short_conv_fwd(x, w, b.bfloat16()), lambda: kta.short_conv_fwd(x, w, b.cpu()),
                lambda: kta.short_conv_fwd(x.half(), w, b),
                lambda: kta.short_conv_fwd(x, w, b, lens=torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: kta.short_conv_step(x[:, 0], w, None, b), lambda: kta.ssm_scan_fwd(x, scan[0][:, :5], *scan[1:]),
                lambda: kta.ssm_scan_fwd(x, *scan, S0=torch.zeros(2, 64, 16, dtype=torch.bfloat16, device="cuda")),
                lambda: kta.ssm_scan_bwd(x, *scan, do, out={"dz": torch.empty_like(x)}),
                lambda: kta.rope_fwd(x[:, :, None], freqs=torch.zeros(8, device="cuda"), dims=16),
                lambda: kta.rope_fwd(x[:, :, None], freqs=torch.zeros(8, dtype=torch.float64, device="cuda"), dims=16,
                                     pos=torch.zeros(21, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(kta.KtaError):
        kta.short_conv_fwd(x, torch.zeros(64, 5, device="cuda"))
    with pytest.raises(kta.KtaError):
        kta.short_conv_fwd(x, w, b, out=x)


def test_layer_rollout_matches_the_whole_sequence(kta):
    """The operators as a hybrid layer uses them: projected queries and keys turn by frame, row and
    column before the softmax heads, a state-space branch runs convolution and scan. The whole clip
    at once and frame by frame (the clip's positions are the frame's plus pos0; rings, rows and states
    carried) give the same layer."""
    F, P, H, d, D = 6, 24, 4, 64, 64
    g = torch.Generator("cuda").manual_seed(9)
    r = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    x = r(1, F * P, 256)
    q, k, v, alpha, _ = kta.qkv_gate_proj(x, (r(3 * H * d + d, 256) / 16), H=H, d=d, n_gla=1)
    t = torch.arange(F * P, device="cuda")
    pos = torch.stack([t // P, t % P // 6, t % 6], -1)
    dims = (24, 20, 20)
    f, _ = kta.rope_freqs(dims)
    cfg = kta.hybrid_cfg(B=1, F=F, P=P, d=d, n_swa=2, n_dswa=1, n_gla=1, W_swa=2, W_dswa=2, dil=2)
    heads = (0, 3)
    qr, kr = q.clone(), k.clone()
    kta.rope_fwd(qr, kr, freqs=f, dims=dims, pos=pos, heads=heads, out=(qr, kr))
    o = kta.hybrid_fwd(cfg, qr, kr, v, alpha)
    s_in = kta.linear(x, r(D, 256) / 16)
    w, bias, A = torch.randn(D, 4, device="cuda", generator=g), None, -torch.rand(D, 16, device="cuda", generator=g) - 0.5
    dt, Bm, Cm = r(1, F * P, D), r(1, F * P, 1, 16), r(1, F * P, 1, 16)
    c = kta.short_conv_fwd(s_in, w, bias)
    y = kta.ssm_scan_fwd(c, dt, A, Bm, Cm)
    stream = kta.Stream(cfg)
    rows, state = torch.zeros(1, 3, D, device="cuda", dtype=torch.bfloat16), None
    for fr in range(F):
        at = slice(fr * P, (fr + 1) * P)
        cut = lambda a: a[:, at].contiguous()  # noqa: E731
        qf, kf = kta.rope_fwd(cut(q), cut(k), freqs=f, dims=dims, pos=pos[:P].contiguous(), pos0=fr, heads=heads,
                              out=(cut(q), cut(k)))
        assert torch.equal(qf[:, :, :3], qr[:, at, :3]) and torch.equal(kf[:, :, :3], kr[:, at, :3])
        of = stream.step(qf, kf, cut(v), cut(alpha))
        assert (of.float() - o[:, at].float()).norm() <= 1e-2 * o[:, at].float().norm()
        cf, rows = kta.short_conv_fwd(cut(s_in), w, bias, S0=rows, return_state=True)
        assert torch.equal(cf, c[:, at])
        yf, state = kta.ssm_scan_fwd(cf, cut(dt), A, cut(Bm), cut(Cm), S0=state, return_state=True)
        # two roundings to bf16 (half a step each) of values that differ by fp32 rounding
        assert (yf.float() - y[:, at].float()).abs().max() <= 2 ** -7 * y.float().abs().max()
    torch.cuda.synchronize()
    kta.device_status()


def test_offsets_past_32_bits(kta):
    """More than 2^31 elements a tensor: the last rows come out as in a short call."""
    B, L, D = 2, 65537, 16392
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    x = torch.zeros(B, L, D, device="cuda", dtype=torch.bfloat16)
    x[:, -8:] = r(B, 8, D).to(torch.bfloat16)
    tail = x[:, -16:].contiguous()
    w = r(D, 4)
    o = kta.short_conv_fwd(x, w)
    assert torch.equal(o[:, -16:], kta.short_conv_fwd(tail, w))
    # the states before the last rows are zero, so the scan's last rows are those of a short call
    A, Bm = -torch.rand(D, 4, device="cuda", generator=g), r(B, L, 1, 4).to(torch.bfloat16)
    kta.ssm_scan_fwd(x, x, A, Bm, Bm, out=o)
    Bt = Bm[:, -16:].contiguous()
    torch.testing.assert_close(o[:, -16:], kta.ssm_scan_fwd(tail, tail, A, Bt, Bt), rtol=2 ** -7, atol=1e-5)
    del x, o
    H = 256
    q = torch.zeros(1, 131080, H, 64, device="cuda", dtype=torch.bfloat16)
    q[:, -3:] = r(1, 3, H, 64).to(torch.bfloat16)
    f, _ = kta.rope_freqs(64)
    last = kta.rope_fwd(q[:, -3:].contiguous(), freqs=f, dims=64, pos0=131077)
    assert torch.equal(kta.rope_fwd(q, freqs=f, dims=64, out=q)[:, -3:], last)


def zeros_but_the_last_rows(g, B, L, D, n):
    x = torch.zeros(B, L, D, device="cuda", dtype=torch.bfloat16)
    x[:, -n:] = torch.randn(B, n, D, device="cuda", generator=g).to(torch.bfloat16)
    return x


def test_backward_offsets_past_32_bits(kta):
    """More than 2^31 elements a tensor, zeros but for the last rows: their gradients and the parameters' are
    those of a call on the last rows alone."""
    B, L, D, N, n = 2, 65537, 16392, 4, 8
    g = torch.Generator("cuda").manual_seed(5)
    x = zeros_but_the_last_rows(g, B, L, D, n)
    tail = x[:, -n:].contiguous()
    r = np.random.default_rng(5)
    w, b = gpu(r.standard_normal((D, 4))), gpu(r.standard_normal(D))
    dx, dw, db, _ = kta.short_conv_bwd(x, w, x, b)
    want = mixers.short_conv(host(tail), host(w), host(b), dout=host(tail), bounds=True)
    for name, t in (("dx", dx[:, -n:]), ("dw", dw), ("dbias", db)):
        check(name, t, want[name])
    del dx
    A, Bm = gpu(-np.exp(r.uniform(-1, 1, (D, N)))), gpu(r.standard_normal((B, L, 1, N)), torch.bfloat16)
    kw = {"D": gpu(r.standard_normal(D)), "dt_bias": gpu(r.standard_normal(D))}
    got = kta.ssm_scan_bwd(x, x, A, Bm, Bm, x, **kw)
    Bt = Bm[:, -n:].contiguous()
    want = scan_oracle({"u": tail, "dt": tail, "A": A, "Bm": Bt, "Cm": Bt}, kw, None, dout=host(tail))
    for name, t in got.items():
        if t is not None:
            check(name, t[:, -n:] if name in ("du", "ddt", "dB", "dC") else t, want[name])


def test_segments_of_a_scan_with_offsets_past_32_bits(kta):
    """2^28 tokens of 8 channels, cut into segments. Between the first rows and the last d = 0, so the state
    stays as it is, and the ends come out as if they were neighbours."""
    L, D, N, n = (1 << 28) + 77, 8, 4, 16
    r = np.random.default_rng(6)
    ends = {k: gpu(r.standard_normal((1, 2 * n) + tail), torch.bfloat16)
            for k, tail in (("u", (D,)), ("dt", (D,)), ("Bm", (1, N)), ("Cm", (1, N)))}

    def stretch(t, fill):
        x = torch.full((1, L) + t.shape[2:], fill, device="cuda", dtype=t.dtype)
        x[:, :n], x[:, -n:] = t[:, :n], t[:, n:]
        return x

    A = gpu(-np.exp(r.uniform(-3, -1, (D, N))))
    x = {k: stretch(t, -200.0 if k == "dt" else 1.0) for k, t in ends.items()}
    y, S = kta.ssm_scan_fwd(**x, A=A, return_state=True)
    want = scan_oracle({**ends, "A": A}, {}, None)
    check("y", torch.cat([y[:, :n], y[:, -n:]], 1), want["y"])
    check("S_out", S, want["S_out"])
