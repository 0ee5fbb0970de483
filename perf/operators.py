"""The token-mixer operators around the hybrid layer, as they are measured: rotary positions for the
softmax heads, the short causal convolution, and the selective state-space scan.

Each operator has its plain form here (elementary torch operations in 32 bits, angles in 64) and the
call that a user makes of the library (where `own` is true). Formulas, for channel c, state n:

  rotary       (a, b) -> m (a cos t - b sin t, a sin t + b cos t),  t = pos * freq
  convolution  y_t = act(bias + sum_j w_j x_{t-K+1+j}),  act = silu or identity
  scan         dt'_t = softplus(dt_t + dt_bias),  h_t = exp(dt'_t A) h_{t-1} + dt'_t u_t B_t,
               y_t = (C_t . h_t + D u_t) silu(z_t)
"""
import math

import torch

own = False

LOG_MIN_DT, LOG_MAX_DT = math.log(1e-3), math.log(1e-1)   # usual range of initial step sizes
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one 880-token frame of a streamed rollout: q and k of 16 softmax heads, three axes
        {"name": "rope frame", "op": "rope", "way": "fwd", "type": "bf16", "B": 1, "N": 880, "H": 16, "d": 128,
         "dims": "44,42,42", "begin": 0, "half": False, "two": True, "factor": 1.0, "pos0": 239},
        # q and k of the 16 softmax heads of a 21 x 1560-token clip
        {"name": "rope clip", "op": "rope", "way": "fwd", "type": "bf16", "B": 1, "N": 32760, "H": 16, "d": 128,
         "dims": "32,48,48", "begin": 0, "half": True, "two": True, "factor": 1.0, "pos0": 0},
        # gradients in training, far positions, scaled frequencies on part of the head
        {"name": "rope far bwd", "op": "rope", "way": "bwd", "type": "f32", "B": 2, "N": 4095, "H": 8, "d": 64,
         "dims": "32", "begin": 16, "half": True, "two": False, "factor": 8.0, "pos0": 211200},
        # two 65,536-token sequences of 16 heads of 128 channels
        {"name": "conv long", "op": "conv", "way": "fwd", "type": "bf16", "B": 2, "L": 65536, "D": 2048, "K": 4,
         "silu": True, "bias": True, "state": False, "ragged": False},
        # a training step over odd lengths
        {"name": "conv train", "op": "conv", "way": "bwd", "type": "bf16", "B": 2, "L": 8191, "D": 2048, "K": 4,
         "silu": True, "bias": True, "state": False, "ragged": False},
        # one token for each of 64 running sequences
        {"name": "conv token", "op": "conv", "way": "step", "type": "bf16", "B": 64, "L": 1, "D": 4096, "K": 4,
         "silu": True, "bias": True, "state": True, "ragged": False},
        # a batch of prompts
        {"name": "scan prompts", "op": "scan", "way": "fwd", "type": "bf16", "B": 4, "L": 2048, "D": 2048, "N": 16,
         "G": 1, "z": True, "skip": True, "state": False, "ragged": False},
        # one long sequence: the clip's tokens over the channels of 8 heads
        {"name": "scan clip", "op": "scan", "way": "fwd", "type": "bf16", "B": 1, "L": 32760, "D": 1024, "N": 16,
         "G": 1, "z": True, "skip": True, "state": False, "ragged": False},
        # prompts of unlike lengths in one padded batch, continued from states, full precision
        {"name": "scan ragged", "op": "scan", "way": "fwd", "type": "f32", "B": 5, "L": 777, "D": 328, "N": 8,
         "G": 1, "z": False, "skip": True, "state": True, "ragged": True},
        # a training step
        {"name": "scan train", "op": "scan", "way": "bwd", "type": "bf16", "B": 2, "L": 2048, "D": 2048, "N": 16,
         "G": 1, "z": True, "skip": True, "state": False, "ragged": False},
        # a small training step in full precision: groups, an odd state size, unlike lengths, carried states
        {"name": "scan train ragged", "op": "scan", "way": "bwd", "type": "f32", "B": 3, "L": 501, "D": 240, "N": 12,
         "G": 3, "z": True, "skip": True, "state": True, "ragged": True},
        # one token for each of 64 running sequences
        {"name": "scan token", "op": "scan", "way": "step", "type": "bf16", "B": 64, "L": 1, "D": 4096, "N": 16,
         "G": 1, "z": True, "skip": True, "state": True, "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, way = rng.choice([("rope", "fwd"), ("rope", "bwd"), ("conv", "fwd"), ("conv", "bwd"), ("conv", "step"),
                          ("scan", "fwd"), ("scan", "bwd"), ("scan", "step"), ("scan", "fwd"), ("scan", "bwd")])
    c = {"op": op, "way": way, "type": rng.choice(["bf16", "bf16", "f32"])}
    if op == "rope":
        d = rng.choice([32, 64, 128])
        half = rng.choice([True, False])
        axes = rng.choice([1, 1, 3])
        if axes == 1:
            dims = [rng.choice([d, d // 2, 2 * rng.randint(1, d // 2)])]
        else:
            one = 2 * rng.randint(1, d // 6)
            dims = [2 * rng.randint(1, (d - 2 * one) // 2), one, one]
        begin = 2 * rng.randint(0, (d - sum(dims)) // 2)
        B, H = rng.randint(1, 4), rng.randint(1, 24)
        N = _log(rng, 1, 32760 * 16 * 128 // (2 * B * H * d) + 1)
        c.update(B=B, N=N, H=H, d=d, dims=",".join(map(str, dims)), begin=begin, half=half, two=rng.choice([True, False]),
                 factor=rng.choice([1.0, 8.0]) if axes == 1 else 1.0, pos0=_log(rng, 1, 1 << 30) - 1)
        return c
    ragged = rng.choice([True, False])
    if op == "conv":
        c["K"] = rng.randint(2, 4)
        c.update(silu=rng.choice([True, False]), bias=rng.choice([True, False]))
        D = 8 * _log(rng, 1, 512)
        if way == "step":
            c.update(B=_log(rng, 1, 256), L=1, D=D, state=True, ragged=False)
        else:
            B = rng.randint(1, 8)
            c.update(B=B, L=_log(rng, 1, max(2, min(65536, (1 << 25) // (B * D)))), D=D, state=rng.choice([True, False]), ragged=ragged)
        return c
    N = rng.choice([4, 8, 12, 16, 16, 16, 24, 32])
    G = rng.choice([1, 1, 1, 2, 4])
    D = G * 8 * _log(rng, 1, 512 // G)
    c.update(N=N, G=G, z=rng.choice([True, False]), skip=rng.choice([True, False]))
    if way == "step":
        c.update(B=_log(rng, 1, 64), L=1, D=D, state=True, ragged=False)
    else:
        B = rng.randint(1, 8)
        most = (1 << 27) // (B * D * N)
        c.update(B=B, L=_log(rng, 1, max(2, min(8192, most))), D=D, state=rng.choice([True, False]), ragged=ragged)
    return c


# ------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ty = DTYPES[case["type"]]

    def randn(*shape, dtype=ty, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    st = {"case": dict(case)}
    if case["op"] == "rope":
        B, N, H, d = case["B"], case["N"], case["H"], case["d"]
        dims = [int(v) for v in case["dims"].split(",")]
        st["dims"] = tuple(dims)
        st["x"] = [randn(B, N, H, d) for _ in range(2 if case["two"] else 1)]
        f = [torch.pow(10000.0, -torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r) for r in dims]
        f, st["mscale"] = torch.cat(f), 1.0
        if case["factor"] != 1.0:   # by parts: long wavelengths stretched, short ones kept, a ramp between
            turns = 4096.0 * f / (2.0 * math.pi)
            keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
            f = f * (keep + (1.0 - keep) / case["factor"])
            st["mscale"] = 0.1 * math.log(case["factor"]) + 1.0
        st["freqs"] = f
        n = torch.arange(N, device="cuda")
        if len(dims) == 1:   # every sequence begins at a place of its own
            at = (rand(B, 1) * 4096).long()
            st["pos"] = (n[None] + at)[..., None].contiguous()
        else:                # rows of 40 tokens, 22 rows to a frame
            st["pos"] = torch.stack([n // 880, n % 880 // 40, n % 40], -1)[None].expand(B, -1, -1).contiguous()
        return st
    B, L, D = case["B"], case["L"], case["D"]
    st["lens"] = (rand(B) * (L + 1)).long().clamp(0, L).to(torch.int32) if case["ragged"] else None
    shape = (B, D) if case["way"] == "step" else (B, L, D)
    if case["op"] == "conv":
        K = case["K"]
        st["x"] = randn(*shape)
        st["w"] = randn(D, K, dtype=torch.float32, scale=K ** -0.5)
        st["bias"] = randn(D, dtype=torch.float32, scale=0.1) if case["bias"] else None
        st["S0"] = randn(B, K - 1, D) if case["state"] else None
    else:
        N, G = case["N"], case["G"]
        st["x"] = randn(*shape)
        st["dt"] = randn(*shape, scale=0.5)
        dt0 = torch.exp(rand(D) * (LOG_MAX_DT - LOG_MIN_DT) + LOG_MIN_DT)
        st["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))     # softplus(dt_bias) = dt0
        st["A"] = -torch.arange(1, N + 1, device="cuda").float()[None] * torch.exp(0.1 * randn(D, N, dtype=torch.float32))
        st["Bm"] = randn(*shape[:-1], G, N)
        st["Cm"] = randn(*shape[:-1], G, N)
        st["skip"] = randn(D, dtype=torch.float32, scale=0.1, shift=1.0) if case["skip"] else None
        st["z"] = randn(*shape) if case["z"] else None
        st["S0"] = randn(B, D, N, dtype=torch.float32) if case["state"] else None
    if case["way"] == "bwd":
        st["dout"] = randn(*shape)
    if st["lens"] is not None:   # rows past a sequence's end are left as they are: buffers that begin as zeros
        st["out"] = torch.zeros_like(st["x"])
        if case["way"] == "bwd" and case["op"] == "scan":
            st["out"] = {"du": torch.zeros_like(st["x"]), "ddt": torch.zeros_like(st["x"]),
                         "dz": torch.zeros_like(st["x"]) if case["z"] else None,
                         "dB": torch.zeros_like(st["Bm"]), "dC": torch.zeros_like(st["Cm"])}
    return st


# ------------------------------------------------------------------------------------- plain forms

def _rope_plain(st):
    """Rotates the pairs of each axis' section; the rest of the head passes through."""
    c = st["case"]
    pos, half, begin = st["pos"].double(), c["half"], c["begin"]
    pos[..., 0] += c["pos0"]
    on = {"device": pos.device}
    axis = torch.cat([torch.full((r // 2,), a, **on) for a, r in enumerate(st["dims"])])
    ang = pos[..., axis] * st["freqs"]                       # [B, N, pairs], 64 bits
    cos, sin = (torch.cos(ang) * st["mscale"]).float(), (torch.sin(ang) * st["mscale"]).float()
    if c["way"] == "bwd":
        sin = -sin
    starts = [begin + sum(st["dims"][:a]) for a in range(len(st["dims"]))]
    lo = torch.cat([s + torch.arange(r // 2, **on) * (1 if half else 2) for s, r in zip(starts, st["dims"])])
    step = torch.cat([torch.full((r // 2,), r // 2 if half else 1, **on) for r in st["dims"]])
    cos, sin = cos[:, :, None], sin[:, :, None]

    def turn(x):
        f = x.float()
        a, b = f[..., lo], f[..., lo + step]
        y = f.clone()
        y[..., lo] = a * cos - b * sin
        y[..., lo + step] = a * sin + b * cos
        return y.to(x.dtype)

    return [turn(x) for x in st["x"]]


def _live(st, L):
    """[B, L, 1] of the rows before each sequence's end, or None."""
    if st["lens"] is None:
        return None
    return (torch.arange(L, device="cuda")[None] < st["lens"][:, None])[..., None]


def _ends(rows, lens, K):
    """The last K - 1 of the first lens + K - 1 rows."""
    if lens is None:
        return rows[:, rows.shape[1] - (K - 1):]
    at = lens.long()[:, None] + torch.arange(K - 1, device=rows.device)
    return torch.gather(rows, 1, at[..., None].expand(-1, -1, rows.shape[2]))


def _conv_pre(st, x, K):
    B, L, D = x.shape
    S0 = st["S0"].float() if st["S0"] is not None else torch.zeros(B, K - 1, D, device=x.device)
    rows = torch.cat([S0, x.float()], 1)
    pre = sum(rows[:, j:j + L] * st["w"][:, j] for j in range(K))
    return rows, pre if st["bias"] is None else pre + st["bias"]


def _conv_plain(st):
    c, x = st["case"], st["x"]
    x = x[:, None] if c["way"] == "step" else x
    K, L = c["K"], x.shape[1]
    rows, pre = _conv_pre(st, x, K)
    live = _live(st, L)
    if c["way"] != "bwd":
        y = pre * torch.sigmoid(pre) if c["silu"] else pre
        y = (y if live is None else y * live).to(x.dtype)
        ends = _ends(rows, st["lens"], K).to(x.dtype)
        return [y[:, 0] if c["way"] == "step" else y, ends]
    dy = st["dout"].float()
    s = torch.sigmoid(pre)
    dp = dy * (s * (1.0 + pre * (1.0 - s))) if c["silu"] else dy
    dp = dp if live is None else dp * live
    pad = torch.cat([dp, torch.zeros_like(rows[:, :K - 1])], 1)      # rows t .. t + K - 1
    drows = torch.cat([torch.zeros_like(rows[:, :K - 1]), pad], 1)
    dr = sum(drows[:, K - 1 - j:K - 1 - j + L + K - 1] * st["w"][:, j] for j in range(K))
    dw = torch.stack([(dp * rows[:, j:j + L]).sum((0, 1)) for j in range(K)], 1)
    dx = dr[:, K - 1:].to(x.dtype)
    out = [dx, dw]
    if c["bias"]:
        out.append(dp.sum((0, 1)))
    if c["state"]:
        out.append(dr[:, :K - 1].to(x.dtype))
    return out


def _carry(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, by doubling."""
    s = 1
    while s < a.shape[1]:
        b = torch.cat([b[:, :s], torch.addcmul(b[:, s:], a[:, s:], b[:, :-s])], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _scan_plain(st):
    c, f = st["case"], lambda t: None if t is None else t.float()  # noqa: E731
    u, z, Bm, Cm = f(st["x"]), f(st["z"]), f(st["Bm"]), f(st["Cm"])
    raw = f(st["dt"]) + st["dt_bias"]
    step = c["way"] == "step"
    if step:
        u, raw, Bm, Cm = u[:, None], raw[:, None], Bm[:, None], Cm[:, None]
        z = None if z is None else z[:, None]
    B, L, D = u.shape
    N, G = c["N"], c["G"]
    live = _live(st, L)
    dt = torch.clamp(raw, min=0.0) + torch.log1p(torch.exp(-raw.abs()))
    dt = dt if live is None else dt * live
    Bx, Cx = (t[:, :, :, None].expand(-1, -1, -1, D // G, -1).reshape(B, L, D, N) for t in (Bm, Cm))
    a = torch.exp(dt[..., None] * st["A"])
    b = (dt * u)[..., None] * Bx
    h0 = st["S0"] if st["S0"] is not None else torch.zeros(B, D, N, device="cuda")
    b0 = b.clone() if L > 1 else b
    b0[:, 0] += a[:, 0] * h0
    h = _carry(a, b0)
    del b0, b
    y = (h * Cx).sum(-1)
    y = y if st["skip"] is None else y + st["skip"] * u
    s = None if z is None else torch.sigmoid(z)
    if c["way"] != "bwd":
        o = y if z is None else y * z * s
        o = (o if live is None else o * live).to(st["x"].dtype)
        return [o[:, 0] if step else o, h[:, -1].contiguous()]
    do = f(st["dout"])
    do = do if live is None else do * live
    dz = None if z is None else do * y * (s * (1.0 + z * (1.0 - s)))
    dy = do if z is None else do * z * s
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    G_ = _carry(nxt.flip(1), (dy[..., None] * Cx).flip(1)).flip(1)     # dL/dh_t
    del nxt
    group = lambda t: t.reshape(B, L, G, D // G, N).sum(3)  # noqa: E731
    dC = group(dy[..., None] * h)
    dB = group(G_ * (dt * u)[..., None])
    dx = (G_ * Bx).sum(-1)
    ah = a * torch.cat([h0[:, None], h[:, :-1]], 1)                     # a_t h_{t-1}
    del h
    dh0 = a[:, 0] * G_[:, 0]
    del a
    gah = G_ * ah
    del ah, G_
    ddt = dx * u + (gah * st["A"]).sum(-1)
    dA = (gah * dt[..., None]).sum((0, 1))
    du = dx * dt if st["skip"] is None else dx * dt + dy * st["skip"]
    ddt = ddt * torch.sigmoid(raw)
    ddt = ddt if live is None else ddt * live
    ty = st["x"].dtype
    out = {"du": du.to(ty), "ddt": ddt.to(ty), "dA": dA, "dB": dB.to(ty), "dC": dC.to(ty), "ddt_bias": ddt.sum((0, 1))}
    if z is not None:
        out["dz"] = dz.to(ty)
    if st["skip"] is not None:
        out["dD"] = (dy * u).sum((0, 1))
    if c["state"]:
        out["dS0"] = dh0
    return out


# ------------------------------------------------------------------------------------- the library's calls

def _rope_own(st):
    from hybrid_linear_temporal_kta_b200 import kta
    c = st["case"]
    fn = kta.rope_bwd if c["way"] == "bwd" else kta.rope_fwd
    o = fn(*st["x"], freqs=st["freqs"], dims=st["dims"], begin=c["begin"], layout="half" if c["half"] else "interleaved",
           mscale=st["mscale"], pos=st["pos"], pos0=c["pos0"])
    return list(o) if c["two"] else [o]


def _conv_own(st):
    from hybrid_linear_temporal_kta_b200 import kta
    c = st["case"]
    out = st["out"] if st["lens"] is not None else None
    if c["way"] == "step":
        state = torch.empty_like(st["S0"])
        return [kta.short_conv_step(st["x"], st["w"], st["S0"], st["bias"], silu=c["silu"], state_out=state), state]
    if c["way"] == "fwd":
        return list(kta.short_conv_fwd(st["x"], st["w"], st["bias"], silu=c["silu"], S0=st["S0"], lens=st["lens"],
                                       return_state=True, out=out))
    g = kta.short_conv_bwd(st["x"], st["w"], st["dout"], st["bias"], silu=c["silu"], S0=st["S0"], lens=st["lens"], out=out)
    return [t for t in g if t is not None]


def _scan_own(st):
    from hybrid_linear_temporal_kta_b200 import kta
    c = st["case"]
    args = st["x"], st["dt"], st["A"], st["Bm"], st["Cm"]
    more = {"D": st["skip"], "z": st["z"], "dt_bias": st["dt_bias"]}
    if c["way"] == "step":
        state = torch.empty_like(st["S0"])
        return [kta.ssm_scan_step(*args, st["S0"], state_out=state, **more), state]
    more.update(S0=st["S0"], lens=st["lens"])
    if c["way"] == "fwd":
        return list(kta.ssm_scan_fwd(*args, return_state=True, out=st["out"] if st["lens"] is not None else None, **more))
    g = kta.ssm_scan_bwd(*args, st["dout"], out=st["out"] if st["lens"] is not None else None, **more)
    return {k: v for k, v in g.items() if v is not None}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _rope_own, "conv": _conv_own, "scan": _scan_own}[op](state)
    return {"rope": _rope_plain, "conv": _conv_plain, "scan": _scan_plain}[op](state)


# ------------------------------------------------------------------------------------- work

def work(case):
    """Inputs once, outputs once. Rows past a sequence's end are counted: lengths are drawn from the seed."""
    s, way = SIZE[case["type"]], case["way"]
    if case["op"] == "rope":
        n = case["B"] * case["N"] * case["H"] * case["d"] * (2 if case["two"] else 1)
        axes = case["dims"].count(",") + 1
        return {"bytes": 2 * n * s + 8 * case["B"] * case["N"] * axes, "flops": 3 * n}
    B, L, D = case["B"], case["L"], case["D"]
    n = B * L * D
    if case["op"] == "conv":
        K = case["K"]
        par = 4 * D * (K + 1)
        st = B * (K - 1) * D * s
        if way == "bwd":
            return {"bytes": 3 * n * s + 2 * par + (2 * st if case["state"] else 0), "flops": n * (6 * K + 8)}
        return {"bytes": 2 * n * s + par + st * (2 if case["state"] else 1), "flops": n * (2 * K + 4)}
    N, G = case["N"], case["G"]
    rows, bc, par, st = n * s, 2 * B * L * G * N * s, 4 * D * (N + 2), 4 * B * D * N
    if way == "bwd":   # u, dt, dout (z) in, du, ddt (dz) out
        return {"bytes": rows * (5 + (2 if case["z"] else 0)) + 2 * bc + 2 * par + (2 * st if case["state"] else 0), "flops": 19 * n * N}
    return {"bytes": rows * (3 + (1 if case["z"] else 0)) + bc + par + st * (2 if case["state"] else 1), "flops": 7 * n * N}


# ------------------------------------------------------------------------------------- 64 bits

def _exact_rope(st):
    """The rotation as a complex product, one axis at a time."""
    c, outs = st["case"], []
    for x in st["x"]:
        y, at, k = x.double().clone(), c["begin"], 0
        for a, r in enumerate(st["dims"]):
            p = st["pos"][..., a] + (c["pos0"] if a == 0 else 0)
            t = p.double()[..., None] * st["freqs"][k:k + r // 2]
            w = torch.polar(torch.full_like(t, st["mscale"]), -t if c["way"] == "bwd" else t)[:, :, None]
            sec = x[..., at:at + r].double()
            sec = sec.unflatten(-1, (2, r // 2)).transpose(-1, -2) if c["half"] else sec.unflatten(-1, (r // 2, 2))
            v = torch.view_as_real(torch.view_as_complex(sec.contiguous()) * w)
            y[..., at:at + r] = (v.transpose(-1, -2) if c["half"] else v).flatten(-2)
            at, k = at + r, k + r // 2
        outs.append(y)
    return outs


def _exact_conv(st):
    """Each output row as a product over the window's rows; gradients by adding each row's share."""
    c = st["case"]
    x = st["x"].double()
    x = x[:, None] if c["way"] == "step" else x
    B, L, D = x.shape
    K, w = c["K"], st["w"].double()
    S0 = st["S0"].double() if st["S0"] is not None else torch.zeros(B, K - 1, D, dtype=torch.float64, device="cuda")
    full = torch.cat([S0, x], 1)
    lens = st["lens"].long() if st["lens"] is not None else torch.full((B,), L, device="cuda")
    mask = torch.arange(L, device="cuda")[None, :, None] < lens[:, None, None]
    bias = st["bias"].double() if st["bias"] is not None else 0.0
    pre = torch.einsum("bldk,dk->bld", full.unfold(1, K, 1), w) + bias
    if c["way"] != "bwd":
        y = pre / (1 + torch.exp(-pre)) if c["silu"] else pre
        y = torch.where(mask, y, 0.0)
        ends = torch.stack([full[b, int(n):int(n) + K - 1] for b, n in enumerate(lens.tolist())])
        return [y[:, 0] if c["way"] == "step" else y, ends]
    g = st["dout"].double()
    if c["silu"]:
        e = torch.exp(-pre)
        g = g * (1 / (1 + e) + pre * e / (1 + e) ** 2)
    g = torch.where(mask, g, 0.0)
    dfull = torch.zeros_like(full)
    dw = torch.zeros_like(w)
    for j in range(K):
        dfull[:, j:j + L] += g * w[:, j]
        dw[:, j] = torch.einsum("bld,bld->d", g, full[:, j:j + L])
    out = [dfull[:, K - 1:], dw]
    if c["bias"]:
        out.append(torch.einsum("bld->d", g))
    if c["state"]:
        out.append(dfull[:, :K - 1])
    return out


def _exact_scan(st):
    """The recurrence token by token; gradients token by token from the last."""
    c = st["case"]
    d = lambda t: None if t is None else t.double()  # noqa: E731
    u, raw, Bm, Cm, z = d(st["x"]), d(st["dt"]) + d(st["dt_bias"]), d(st["Bm"]), d(st["Cm"]), d(st["z"])
    if c["way"] == "step":
        u, raw, Bm, Cm = u[:, None], raw[:, None], Bm[:, None], Cm[:, None]
        z = None if z is None else z[:, None]
    B, L, D = u.shape
    N, G = c["N"], c["G"]
    A, skip = d(st["A"]), d(st["skip"])
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    lens = st["lens"].long() if st["lens"] is not None else torch.full((B,), L, device="cuda")
    live = torch.arange(L, device="cuda")[None] < lens[:, None]

    def wide(t):                                            # [B, G, N] -> [B, D, N]
        return t.repeat_interleave(D // G, 1)

    h = d(st["S0"]) if st["S0"] is not None else torch.zeros(B, D, N, dtype=torch.float64, device="cuda")
    bwd = c["way"] == "bwd"
    kept, ys = [h], []
    for t in range(L):
        new = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * u[:, t])[..., None] * wide(Bm[:, t])
        h = torch.where(live[:, t, None, None], new, h)
        ys.append(torch.einsum("bdn,bdn->bd", h, wide(Cm[:, t])))
        if bwd:
            kept.append(h)
    y = torch.stack(ys, 1)
    y = y if skip is None else y + skip * u
    gate = 1.0 if z is None else z / (1 + torch.exp(-z))
    if not bwd:
        o = torch.where(live[..., None], y * gate, 0.0)
        return [o[:, 0] if c["way"] == "step" else o, h]
    do = torch.where(live[..., None], d(st["dout"]), 0.0)
    dy = do * gate
    g = torch.zeros_like(h)
    dA = torch.zeros_like(A)
    du, ddt = torch.zeros_like(u), torch.zeros_like(u)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    for t in range(L - 1, -1, -1):
        on = live[:, t, None, None]
        a = torch.where(on, torch.exp(dt[:, t, :, None] * A), 1.0)
        g = g + dy[:, t, :, None] * wide(Cm[:, t])
        dC[:, t] = (dy[:, t, :, None] * kept[t + 1]).reshape(B, G, D // G, N).sum(2)
        m = torch.where(on, g, 0.0)
        dB[:, t] = (m * (dt[:, t] * u[:, t])[..., None]).reshape(B, G, D // G, N).sum(2)
        dx = (m * wide(Bm[:, t])).sum(-1)
        w = m * a * kept[t]
        dA += (w * dt[:, t, :, None]).sum(0)
        ddt[:, t] = dx * u[:, t] + (w * A).sum(-1)
        du[:, t] = dx * dt[:, t]
        g = g * a
    ddt = ddt / (1 + torch.exp(-raw))
    out = {"du": du if skip is None else du + dy * skip, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "ddt_bias": ddt.sum((0, 1))}
    if z is not None:
        e = torch.exp(-z)
        out["dz"] = do * y * (1 / (1 + e) + z * e / (1 + e) ** 2)
    if skip is not None:
        out["dD"] = (dy * u).sum((0, 1))
    if c["state"]:
        out["dS0"] = g
    return out


def exact(case, seed):
    if case["op"] == "scan" and case["way"] == "bwd" and case["B"] * case["L"] * case["D"] * case["N"] * 8 > 40e9:
        return None                                           # the kept states would not fit
    st = prepare(case, seed)
    return {"rope": _exact_rope, "conv": _exact_conv, "scan": _exact_scan}[case["op"]](st)
