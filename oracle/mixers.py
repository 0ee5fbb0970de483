"""64-bit oracle of the rotary, short-convolution and state-space entry points: plain numpy, token by
token, from the formulas in include/kta.h; shares nothing with the package.

Every function returns values, and with bounds=True pairs (value, bound): a first-order bound of what
an evaluation in fp32 may be off, element by element, before the result is rounded to its type. It
counts, for u = 2^-24: one u for each rounded operation, 2^-22 for an approximated exponential or
reciprocal (plus the rounding of its argument), n u for a sum of n terms, and carries the errors of
what a result is made of along the same recurrences. It is doubled once for second-order terms and
for sums split into segments.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
EXP = 2.0 ** -22


def _sig(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def _sig_rel(x):
    """Relative error of 1 / (1 + e^-x) in fp32: that of e^-x, of the sum and of the reciprocal."""
    return np.abs(x) * 4 * U + 2 * EXP + 2 * U


def rounded(value, bound, eps):
    """The bound after rounding to a type of machine epsilon eps (half a step of the value)."""
    return bound + (np.abs(value) + bound) * (eps / 2)


# ---------------------------------------------------------------------------------- rotary

def rope(x, freqs, dims, pos, *, begin=0, half=True, mscale=1.0, pos0=0, inverse=False, bounds=False):
    """x [B, N, H, d]; pos int [B, N, axes]; freqs [sum(dims) / 2]."""
    x = np.asarray(x, np.float64)
    y, err = x.copy(), np.zeros_like(x)
    at, k = begin, 0
    for a, r in enumerate(dims):
        p = pos[..., a].astype(np.int64) + (pos0 if a == 0 else 0)
        for i in range(r // 2):
            t = p.astype(np.float64) * freqs[k + i]
            c, s = mscale * np.cos(t)[..., None], mscale * np.sin(t)[..., None]
            s = -s if inverse else s
            lo, hi = (at + i, at + i + r // 2) if half else (at + 2 * i, at + 2 * i + 1)
            va, vb = x[..., lo], x[..., hi]
            y[..., lo], y[..., hi] = va * c - vb * s, va * s + vb * c
            # angle: three 64-bit roundings of pos * freq / 2 pi, one of the reduced turn; sine,
            # scaling, two products and a sum
            d = mscale * (np.abs(t) * 4 * 2.0 ** -53 + 6.3 * U + 4 * U)[..., None]
            err[..., lo] = err[..., hi] = (np.abs(va) + np.abs(vb)) * (d + mscale * 3 * U)
        at, k = at + r, k + r // 2
    return (y, 2 * err) if bounds else y


# ---------------------------------------------------------------------------------- convolution

def short_conv(x, w, bias=None, *, silu=True, S0=None, lens=None, dout=None, dS_out=None, bounds=False):
    """x [B, L, D]. Returns o and S_out, or with dout the gradients dx, dw, dbias, dS0, as a dict. Rows
    past a sequence's end come back as zeros."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    B, L, D = x.shape
    K = w.shape[1]
    bias = np.zeros(D) if bias is None else np.asarray(bias, np.float64)
    S0 = np.zeros((B, K - 1, D)) if S0 is None else np.asarray(S0, np.float64)
    lens = [L] * B if lens is None else [int(n) for n in lens]
    o, oe = np.zeros_like(x), np.zeros_like(x)
    S = np.zeros_like(S0)
    g = {n: np.zeros_like(v) for n, v in (("dx", x), ("dw", w), ("dbias", bias), ("dS0", S0))}
    ge = {n: np.zeros_like(v) for n, v in g.items()}
    for b in range(B):
        n = lens[b]
        full = np.concatenate([S0[b], x[b, :n]])
        S[b] = full[n:n + K - 1]
        df, de = np.zeros_like(full), np.zeros_like(full)
        for t in range(n):
            win = full[t:t + K]                           # rows t - K + 1 .. t
            pre = bias + (w.T * win).sum(0)
            pe = (K + 1) * U * (np.abs(bias) + np.abs(w.T * win).sum(0))
            s = _sig(pre) if silu else np.ones(D)
            if dout is None:
                o[b, t] = pre * s
                oe[b, t] = (1.1 * pe + np.abs(pre * s) * (_sig_rel(pre) + U)) if silu else pe
                continue
            dy = np.asarray(dout[b, t], np.float64)
            act = s * (1 + pre * (1 - s)) if silu else 1.0
            dp = dy * act
            # s (1 + x (1 - s)): its derivative is below 1/2; each product and sum is rounded
            pe = np.abs(dy) * (0.5 * pe + 3 * (s + np.abs(pre) * s) * (_sig_rel(pre) + 3 * U)) if silu else 0 * pe
            df[t:t + K] += w.T * dp
            de[t:t + K] += np.abs(w.T) * pe + (K + 1) * U * np.abs(w.T * dp)
            g["dw"] += (win * dp).T
            ge["dw"] += (np.abs(win) * pe + (64 + L * B / 64) * U * np.abs(win * dp)).T
            g["dbias"] += dp
            ge["dbias"] += pe + (64 + L * B / 64) * U * np.abs(dp)
        if dout is not None:
            if dS_out is not None:
                df[n:n + K - 1] += dS_out[b]
                de[n:n + K - 1] += 2 * U * (np.abs(dS_out[b]) + np.abs(df[n:n + K - 1]))
            g["dS0"][b], ge["dS0"][b] = df[:K - 1], de[:K - 1]
            g["dx"][b, :n], ge["dx"][b, :n] = df[K - 1:], de[K - 1:]
    if dout is None:
        r, e = {"o": o, "S_out": S}, {"o": oe, "S_out": np.zeros_like(S)}
    else:
        r, e = g, ge
    return {n: (r[n], 2 * e[n]) for n in r} if bounds else r


# ---------------------------------------------------------------------------------- scan

def ssm_scan(u, dt, A, Bm, Cm, *, D=None, z=None, dt_bias=None, S0=None, lens=None, dout=None,
             dS_out=None, bounds=False):
    """u, dt, z [B, L, D]; A [D, N]; Bm, Cm [B, L, G, N]. Returns y and S_out, or with dout the
    gradients, as a dict. Rows past a sequence's end come back as zeros."""
    f = lambda t: np.asarray(t, np.float64)  # noqa: E731
    u, dt, A, Bm, Cm = f(u), f(dt), f(A), f(Bm), f(Cm)
    B, L, C = u.shape
    N, G = A.shape[1], Bm.shape[2]
    rep = C // G
    wide = lambda t: np.repeat(t, rep, axis=0)  # noqa: E731  [G, N] -> [C, N]
    Dk = np.zeros(C) if D is None else f(D)
    bias = np.zeros(C) if dt_bias is None else f(dt_bias)
    S0 = np.zeros((B, C, N)) if S0 is None else f(S0)
    lens = [L] * B if lens is None else [int(n) for n in lens]
    y, ye = np.zeros_like(u), np.zeros_like(u)
    S, Se = S0.copy(), np.zeros_like(S0)
    names = {"du": u, "ddt": u, "dz": u, "dB": Bm, "dC": Cm, "dA": A, "dD": Dk, "ddt_bias": bias, "dS0": S0}
    g, ge = ({n: np.zeros_like(v) for n, v in names.items()} for _ in range(2))
    nb = 16 + (rep + 31) // 32                            # additions of a sum over channels
    nt = 96 + B * L / 256                                 # of a sum over tokens
    for b in range(B):
        n = lens[b]
        raw = dt[b] + bias
        d = np.maximum(raw, 0) + np.log1p(np.exp(-np.abs(raw)))
        dr = 2 * EXP + np.abs(raw) * 4 * U + (np.abs(dt[b]) + np.abs(bias)) * 2 * U   # relative
        if z is None:
            s, gate, gr = np.ones((L, C)), np.ones((L, C)), np.zeros((L, C))
            zb = np.zeros((L, C))
        else:
            zb = f(z[b])
            s = _sig(zb)
            gate, gr = zb * s, _sig_rel(zb) + U
        h, he = S0[b].copy(), np.zeros((C, N))
        H, HE, AH, AHE, AV, AR = [], [], [], [], [], []
        for t in range(n):
            x = d[t][:, None] * A
            a = np.exp(x)
            ar = np.abs(x) * (dr[t][:, None] + 4 * U) + EXP
            ah, ahe = a * h, a * he + a * np.abs(h) * (ar + U)
            v = (d[t] * u[b, t])[:, None] * wide(Bm[b, t])
            h = ah + v
            he = ahe + np.abs(v) * (dr[t][:, None] + 3 * U) + np.abs(h) * U
            if dout is not None:
                H.append(h), HE.append(he), AH.append(ah), AHE.append(ahe), AV.append(a), AR.append(ar)
            ch = wide(Cm[b, t]) * h
            core = ch.sum(1) + Dk * u[b, t]
            ce = (np.abs(wide(Cm[b, t])) * he).sum(1) + (N + 3) * U * (np.abs(ch).sum(1) + np.abs(Dk * u[b, t]))
            y[b, t] = core * gate[t]
            ye[b, t] = ce * np.abs(gate[t]) + np.abs(y[b, t]) * (gr[t] + 2 * U)
            if dout is not None and z is not None:
                act = s[t] * (1 + zb[t] * (1 - s[t]))
                ae = 3 * (s[t] + np.abs(zb[t]) * s[t]) * (_sig_rel(zb[t]) + 3 * U)
                do = f(dout[b, t])
                g["dz"][b, t] = do * core * act
                ge["dz"][b, t] = np.abs(do) * (ce * np.abs(act) + np.abs(core) * (ae + 3 * U))
        S[b], Se[b] = h, he
        if dout is None:
            continue
        gr_, gre = (np.zeros((C, N)), np.zeros((C, N))) if dS_out is None else (f(dS_out[b]).copy(), np.zeros((C, N)))
        for t in range(n - 1, -1, -1):
            dy = f(dout[b, t]) * gate[t]
            dye = np.abs(dy) * (gr[t] + 2 * U)
            Bw, Cw = wide(Bm[b, t]), wide(Cm[b, t])
            v = dy[:, None] * Cw
            gr_ = gr_ + v
            gre = gre + dye[:, None] * np.abs(Cw) + U * np.abs(v) + U * np.abs(gr_)
            q = dy[:, None] * H[t]
            qe = dye[:, None] * np.abs(H[t]) + np.abs(dy)[:, None] * HE[t] + nb * U * np.abs(q)
            g["dC"][b, t] = q.reshape(G, rep, N).sum(1)
            ge["dC"][b, t] = qe.reshape(G, rep, N).sum(1)
            du = (d[t] * u[b, t])[:, None]
            q = gr_ * du
            qe = gre * np.abs(du) + np.abs(q) * (dr[t][:, None] + (nb + 1) * U)
            g["dB"][b, t] = q.reshape(G, rep, N).sum(1)
            ge["dB"][b, t] = qe.reshape(G, rep, N).sum(1)
            dx = (gr_ * Bw).sum(1)
            dxe = (gre * np.abs(Bw)).sum(1) + (N + 1) * U * np.abs(gr_ * Bw).sum(1)
            w = gr_ * AH[t]
            we = gre * np.abs(AH[t]) + np.abs(gr_) * AHE[t] + U * np.abs(w)
            g["dA"] += w * d[t][:, None]
            ge["dA"] += (we + np.abs(w) * (dr[t][:, None] + nt * U)) * d[t][:, None]
            sw = (w * A).sum(1)
            swe = (we * np.abs(A)).sum(1) + (N + 1) * U * np.abs(w * A).sum(1)
            sg = _sig(raw[t])
            dd = (dx * u[b, t] + sw) * sg
            dde = (dxe * np.abs(u[b, t]) + swe + 2 * U * (np.abs(dx * u[b, t]) + np.abs(sw))) * sg + \
                np.abs(dd) * (_sig_rel(raw[t]) + 2 * U * (1 + np.abs(dt[b, t]) + np.abs(bias)))
            g["ddt"][b, t], ge["ddt"][b, t] = dd, dde
            g["ddt_bias"] += dd
            ge["ddt_bias"] += dde + nt * U * np.abs(dd)
            g["du"][b, t] = dx * d[t] + Dk * dy
            ge["du"][b, t] = dxe * d[t] + np.abs(dx * d[t]) * (dr[t] + 2 * U) + np.abs(Dk) * (dye + 2 * U * np.abs(dy))
            g["dD"] += dy * u[b, t]
            ge["dD"] += dye * np.abs(u[b, t]) + nt * U * np.abs(dy * u[b, t])
            gre = AV[t] * gre + AV[t] * np.abs(gr_) * (AR[t] + U)
            gr_ = AV[t] * gr_
        g["dS0"][b], ge["dS0"][b] = gr_, gre
    r, e = ({"y": y, "S_out": S}, {"y": ye, "S_out": Se}) if dout is None else (g, ge)
    return {n: (r[n], 2 * e[n]) for n in r} if bounds else r
