"""Host-side checks of the rotary, short-convolution and state-space entry points (no GPU needed):
frequencies, workspace sizes, and refusals that come back before any CUDA call (the pointers are
never dereferenced)."""
import ctypes
import math

import numpy as np
import pytest

OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, 1, 2, 3
ST = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def kta():
    from hybrid_linear_temporal_kta_b200 import build
    build.build()
    from hybrid_linear_temporal_kta_b200 import kta as mod
    return mod


def at(n, off=0):
    """A fake device address, 16 GiB apart for each n."""
    return ctypes.c_void_p((n + 1 << 34) + off)


# ---------------------------------------------------------------------------------- frequencies

def test_rope_freqs_values(kta):
    f, m = kta.rope_freqs(64, device="cpu")
    want = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    assert m == 1.0 and np.allclose(f.numpy(), want, rtol=1e-14)
    f, m = kta.rope_freqs((8, 4), base=500.0, scaling="linear", factor=4.0, device="cpu")
    want = np.concatenate([500.0 ** (-np.arange(0, r, 2) / r) for r in (8, 4)]) / 4
    assert m == 1.0 and np.allclose(f.numpy(), want, rtol=1e-14)
    # raised base: the highest frequency stays, the lowest is divided by the factor
    f, m = kta.rope_freqs(32, scaling="base", factor=8.0, device="cpu")
    g, _ = kta.rope_freqs(32, device="cpu")
    assert m == 1.0 and f[0] == 1.0 and math.isclose(f[-1], g[-1] / 8, rel_tol=1e-12)
    # by parts: kept above beta_fast turns, divided below beta_slow, between them between
    f, m = kta.rope_freqs(64, scaling="by_parts", factor=8.0, orig_len=4096, device="cpu")
    g = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    turns = 4096 * g / (2 * math.pi)
    f = f.numpy()
    assert math.isclose(m, 0.1 * math.log(8) + 1, rel_tol=1e-6)
    assert np.allclose(f[turns >= 32], g[turns >= 32], rtol=1e-14)
    assert np.allclose(f[turns <= 1], g[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all(f[mid] < g[mid]) and np.all(f[mid] > g[mid] / 8)


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1, 0, 32, 1), (3, 1e4, 0, 1, 0, 32, 1), (130, 1e4, 0, 1, 0, 32, 1), (8, 0.0, 0, 1, 0, 32, 1),
    (8, math.inf, 0, 1, 0, 32, 1), (8, 1e4, 4, 1, 0, 32, 1), (8, 1e4, 1, 0.5, 0, 32, 1), (8, 1e4, 2, math.nan, 0, 32, 1),
    (8, 1e4, 3, 2, 0, 32, 1), (8, 1e4, 3, 2, 4096, 1, 1), (8, 1e4, 3, 2, 4096, 32, -1)])
def test_rope_freqs_refusals(kta, args):
    f, m = (ctypes.c_double * 64)(), ctypes.c_float()
    assert kta.raw_call("kta_rope_freqs", *args, ctypes.cast(f, ctypes.c_void_p), ctypes.byref(m)) == INVALID
    assert kta.raw_call("kta_rope_freqs", *args, None, None) == INVALID


# ---------------------------------------------------------------------------------- rotary

def rope_call(kta, x=at(0), o=at(1), x2=None, o2=None, s=None, H=2, ld=2, H2=0, ld2=0, axes=1, dims=(32,), begin=0,
              mscale=1.0, pos=at(5), freqs=at(6)):
    cfg = kta.Rope(axes, (ctypes.c_int * 4)(*dims), begin, 0, mscale, pos, 0, 0, freqs)
    s = s or kta.Shape(1, 2, 16, 64, 0)
    return kta.raw_call("kta_rope_fwd", ctypes.byref(cfg), x, o, x2, o2, s, H, ld, H2, ld2, ST)


def test_rope_refusals(kta):
    assert kta.raw_call("kta_rope_fwd", None, at(0), at(1), None, None, kta.Shape(1, 2, 16, 64, 0), 2, 2, 0, 0, ST) == INVALID
    for kw in (dict(x=None), dict(o=None), dict(freqs=None), dict(axes=0), dict(axes=5), dict(dims=(31,)),
               dict(dims=(0,)), dict(dims=(66,)), dict(begin=1), dict(begin=-2), dict(begin=34), dict(H=0), dict(H=3),
               dict(mscale=math.nan), dict(axes=2, dims=(32, 32), pos=None), dict(axes=2, dims=(32, 34)),
               dict(x2=at(2)), dict(x2=at(2), o2=at(3), H2=0, ld2=1), dict(x2=at(2), o2=at(3), H2=3, ld2=2),
               dict(s=kta.Shape(0, 2, 16, 64, 0)), dict(s=kta.Shape(1, 2, 16, 64, 7))):
        assert rope_call(kta, **kw) == INVALID, kw
    assert rope_call(kta, s=kta.Shape(1, 2, 16, 96, 0)) == UNSUPPORTED
    for kw in (dict(x=at(0, 2)), dict(freqs=at(6, 4)), dict(pos=at(5, 4)), dict(x2=at(2, 8), o2=at(3), H2=1, ld2=1)):
        assert rope_call(kta, **kw) == ALIGNMENT, kw


def test_rope_refuses_overlap(kta):
    row = 4 * 64 * 2
    assert rope_call(kta, o=at(0, row)) == INVALID                        # o a row behind x
    assert rope_call(kta, x2=at(1), o2=at(2), H2=2, ld2=2) == INVALID      # o is the second input
    assert rope_call(kta, x2=at(2), o2=at(1, 128), H2=2, ld2=2) == INVALID  # the outputs meet
    # heads of one tensor: [0, 2) into [1, 3) meet
    assert rope_call(kta, x=at(0), o=at(0, 128), H=2, ld=4) == INVALID


# ---------------------------------------------------------------------------------- convolution

def conv(kta, **kw):
    d = dict(B=2, L=9, D=16, K=4, dtype=0, silu=1, x=at(0), w=at(1), bias=at(2), S0=at(3), lens=None)
    d.update(kw)
    return kta.ShortConv(*d.values())


BAD_CONV = [(dict(B=0), INVALID), (dict(L=0), INVALID), (dict(D=0), INVALID), (dict(K=1), UNSUPPORTED),
            (dict(K=5), UNSUPPORTED), (dict(D=12), ALIGNMENT), (dict(dtype=2), INVALID), (dict(x=None), INVALID),
            (dict(w=None), INVALID), (dict(x=at(0, 8)), ALIGNMENT), (dict(w=at(1, 4)), ALIGNMENT),
            (dict(bias=at(2, 4)), ALIGNMENT), (dict(S0=at(3, 2)), ALIGNMENT), (dict(lens=at(4, 2)), ALIGNMENT),
            (dict(B=1 << 16, L=1 << 15), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", BAD_CONV)
def test_short_conv_refusals(kta, kw, want):
    c = conv(kta, **kw)
    assert kta.raw_call("kta_short_conv_fwd", ctypes.byref(c), at(8), at(9), ST) == want
    big = 1 << 33
    assert kta.raw_call("kta_short_conv_bwd", ctypes.byref(c), at(8), None, at(9), at(10), at(11), at(12), at(13), big, ST) == want


def test_short_conv_other_refusals(kta):
    c = conv(kta)
    fwd = lambda o, S: kta.raw_call("kta_short_conv_fwd", ctypes.byref(c), o, S, ST)  # noqa: E731
    assert kta.raw_call("kta_short_conv_fwd", None, at(8), at(9), ST) == INVALID
    assert fwd(None, None) == INVALID
    assert fwd(at(0), None) == INVALID                  # o = x: rows are read again
    assert fwd(at(8), at(3, 16)) == INVALID             # S_out partly over S0
    assert fwd(at(8), at(8)) == INVALID
    assert fwd(at(8, 4), None) == ALIGNMENT
    n = kta._lib.kta_short_conv_bwd_workspace(ctypes.byref(c))
    assert n >= 5 * 16 * 4
    bwd = lambda *a: kta.raw_call("kta_short_conv_bwd", ctypes.byref(c), *a, ST)  # noqa: E731
    assert bwd(at(8), None, at(9), at(10), at(11), at(12), at(13), n - 1) == INVALID
    assert bwd(at(8), None, at(9), at(10), at(11), at(12), None, n) == INVALID
    assert bwd(at(8), None, at(9), at(10), at(11), at(12), at(13, 8), n) == ALIGNMENT
    assert bwd(None, None, at(9), at(10), at(11), at(12), at(13), n) == INVALID
    assert bwd(at(8), None, at(8), at(10), at(11), at(12), at(13), n) == INVALID   # dx = dout
    assert bwd(at(8), None, at(9), at(9), at(11), at(12), at(13), n) == INVALID    # dw = dx
    c.S0 = None
    assert bwd(at(8), None, at(9), at(10), at(11), at(12), at(13), n) == INVALID   # dS0 without S0


# ---------------------------------------------------------------------------------- scan

def ssm(kta, **kw):
    d = dict(B=2, L=9, D=16, N=16, G=1, dtype=0, u=at(0), dt=at(1), A=at(2), Bm=at(3), Cm=at(4), D_skip=at(5), z=at(6),
             dt_bias=at(7), S0=at(8), lens=None)
    d.update(kw)
    return kta.Ssm(*d.values())


def grads(kta, **kw):
    d = dict(dout=at(20), dS_out=None, du=at(21), ddt=at(22), dA=at(23), dB=at(24), dC=at(25), dD_skip=at(26), dz=at(27),
             ddt_bias=at(28), dS0=at(29))
    d.update(kw)
    return kta.SsmGrads(*d.values())


BAD_SSM = [(dict(B=0), INVALID), (dict(L=0), INVALID), (dict(D=0), INVALID), (dict(N=0), INVALID), (dict(G=0), INVALID),
           (dict(N=33), UNSUPPORTED), (dict(G=3), INVALID), (dict(D=12), ALIGNMENT), (dict(G=4), ALIGNMENT),
           (dict(dtype=5), INVALID), (dict(u=None), INVALID), (dict(dt=None), INVALID), (dict(A=None), INVALID),
           (dict(Bm=None), INVALID), (dict(Cm=None), INVALID), (dict(u=at(0, 2)), ALIGNMENT), (dict(S0=at(8, 4)), ALIGNMENT),
           (dict(lens=at(9, 1)), ALIGNMENT), (dict(Bm=at(3, 1)), ALIGNMENT),
           (dict(Cm=at(4, 2), dtype=1), ALIGNMENT), (dict(B=1 << 16, L=1 << 15), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", BAD_SSM)
def test_ssm_refusals(kta, kw, want):
    c, g, big = ssm(kta, **kw), grads(kta), 1 << 33
    assert kta.raw_call("kta_ssm_scan_fwd", ctypes.byref(c), at(10), at(11), at(12), big, ST) == want
    assert kta.raw_call("kta_ssm_scan_bwd", ctypes.byref(c), ctypes.byref(g), at(12), big, ST) == want
    if kw != dict(L=0) and "lens" not in kw:
        c.L = 1 if c.L == 9 else c.L
        assert kta.raw_call("kta_ssm_scan_step", ctypes.byref(c), at(10), at(11), ST) == want


def test_ssm_other_refusals(kta):
    c, g = ssm(kta), grads(kta)
    fwd = lambda c, y, S: kta.raw_call("kta_ssm_scan_fwd", ctypes.byref(c), y, S, at(12), 1 << 33, ST)  # noqa: E731
    step = lambda c, y, S: kta.raw_call("kta_ssm_scan_step", ctypes.byref(c), y, S, ST)  # noqa: E731
    assert fwd(c, None, None) == INVALID
    assert fwd(c, at(0), None) == INVALID and fwd(c, at(6), None) == INVALID
    assert fwd(c, at(10), at(8)) == INVALID             # the state in place is the step's
    assert step(c, at(10), at(8)) == INVALID            # L = 9
    one = ssm(kta, L=1)
    assert step(one, at(10), None) == INVALID and step(one, at(10), at(8, 64)) == INVALID
    assert step(ssm(kta, L=1, S0=None), at(10), at(11)) == INVALID
    assert step(ssm(kta, L=1, lens=at(9)), at(10), at(11)) == INVALID
    n = kta._lib.kta_ssm_scan_bwd_workspace(ctypes.byref(c))
    bwd = lambda c, g, ws, n: kta.raw_call("kta_ssm_scan_bwd", ctypes.byref(c), ctypes.byref(g), ws, n, ST)  # noqa: E731
    assert n > 0 and bwd(c, g, at(12), n - 1) == INVALID and bwd(c, g, None, n) == INVALID
    assert kta.raw_call("kta_ssm_scan_bwd", ctypes.byref(c), None, at(12), n, ST) == INVALID
    for name in ("dout", "du", "ddt", "dA", "dB", "dC", "dz"):
        assert bwd(c, grads(kta, **{name: None}), at(12), n) == INVALID, name
    assert bwd(ssm(kta, z=None), g, at(12), n) == INVALID
    assert bwd(ssm(kta, D_skip=None), g, at(12), n) == INVALID
    assert bwd(c, grads(kta, du=at(20)), at(12), n) == INVALID
    assert bwd(c, grads(kta, dB=at(25)), at(12), n) == INVALID
    assert kta._lib.kta_ssm_scan_bwd_workspace(ctypes.byref(ssm(kta, N=40))) == 0


def test_binding_refuses_what_is_not_on_a_gpu(kta):
    import torch
    x, w = torch.zeros(2, 9, 16), torch.zeros(16, 4)
    with pytest.raises(ValueError):
        kta.short_conv_fwd(x, w)
    with pytest.raises(ValueError):
        kta.rope_fwd(torch.zeros(1, 4, 2, 64), freqs=torch.zeros(16, dtype=torch.float64), dims=32)
    with pytest.raises(ValueError):
        kta.ssm_scan_fwd(x, x, torch.zeros(16, 16), torch.zeros(2, 9, 1, 16), torch.zeros(2, 9, 1, 16))
    with pytest.raises(ValueError):
        kta.rope_freqs(32, scaling="other", device="cpu")


def test_token_counts_leave_room_for_what_ends_behind_the_last_row(kta):
    """Tokens are counted in 32 bits, and the ends of runs and segments are rounded up."""
    for L in ((1 << 31) - 1, (1 << 31) - (1 << 16)):
        c, s, g = conv(kta, B=1, L=L), ssm(kta, B=1, L=L), grads(kta)
        assert kta.raw_call("kta_short_conv_fwd", ctypes.byref(c), at(8), at(9), ST) == UNSUPPORTED
        assert kta._lib.kta_short_conv_bwd_workspace(ctypes.byref(c)) == 0
        assert kta.raw_call("kta_ssm_scan_fwd", ctypes.byref(s), at(10), at(11), at(12), 1 << 40, ST) == UNSUPPORTED
        assert kta.raw_call("kta_ssm_scan_bwd", ctypes.byref(s), ctypes.byref(g), at(12), 1 << 60, ST) == UNSUPPORTED
    assert kta._lib.kta_ssm_scan_bwd_workspace(ctypes.byref(ssm(kta, B=1, L=(1 << 31) - (1 << 16) - 1))) > 0


def test_trace_has_room_for_every_kernel_name(kta):
    import pathlib
    import re
    csrc = pathlib.Path(kta.__file__).parent / "csrc"
    names = {n for f in csrc.glob("*.cu*") for line in f.read_text().splitlines() if "TraceScope" in line
             for n in re.findall(r'"(\w+)"', line)}
    assert 30 < len(names) <= kta._TRACE_NAMES


@pytest.mark.parametrize("B,L,D,longer", [
    (2, 8191, 2048, True), (2, 3600, 4096, True), (2, 12000, 2048, True), (16, 1085, 3456, True), (8, 1759, 7936, True),
    (1, 65536, 2048, True), (8, 768, 5120, False), (16, 768, 2560, False), (24, 512, 4096, False), (8, 4096, 2048, False),
    (24, 5051, 1472, False), (16, 2048, 4096, False), (1, 64, 2048, False)])
def test_conv_backward_stretches_runs_where_measured_faster(kta, B, L, D, longer):
    """The workspace tells the blocks of a call (4 runs each) on 148 SMs: runs of 64 tokens where longer ones
    were measured to take as long or longer, fewer blocks where they were faster."""
    n = kta._lib.kta_short_conv_bwd_workspace(ctypes.byref(conv(kta, B=B, L=L, D=D)))
    blocks, of64 = n // (5 * D * 4), B * -(-L // 256)
    assert blocks < of64 if longer else blocks >= of64


def test_outputs_over_lengths_positions_or_frequencies_are_refused(kta):
    """They are read again while outputs are written."""
    big, n8 = 1 << 33, 2 * 9 * 16 * 2                       # bytes of x, o, u, y
    c = conv(kta, lens=at(9, n8 - 4))                       # the last element of an output at at(9)
    fwd = lambda c, o, S: kta.raw_call("kta_short_conv_fwd", ctypes.byref(c), o, S, ST)  # noqa: E731
    assert fwd(c, at(9), None) == INVALID and fwd(c, at(8), at(9, n8 - 16)) == INVALID
    c.lens = at(9, 4)
    for k in range(5):                                      # dx, dw, dbias, dS0, the workspace
        outs = [at(9) if i == k else at(20 + i) for i in range(5)]
        assert kta.raw_call("kta_short_conv_bwd", ctypes.byref(c), at(8), None, *outs, big, ST) == INVALID, k
    s = ssm(kta, lens=at(9, 4))
    assert kta.raw_call("kta_ssm_scan_fwd", ctypes.byref(s), at(9), at(11), at(12), big, ST) == INVALID
    assert kta.raw_call("kta_ssm_scan_fwd", ctypes.byref(s), at(10), at(9), at(12), big, ST) == INVALID
    many = ssm(kta, B=1, L=4096, lens=at(9, 4))             # cut into segments: it has a workspace
    assert kta._lib.kta_ssm_scan_fwd_workspace(ctypes.byref(many)) > 0
    assert kta.raw_call("kta_ssm_scan_fwd", ctypes.byref(many), at(10), at(11), at(9), big, ST) == INVALID
    for name in ("du", "ddt", "dA", "dB", "dC", "dD_skip", "dz", "ddt_bias", "dS0"):
        g = grads(kta, **{name: at(9)})
        assert kta.raw_call("kta_ssm_scan_bwd", ctypes.byref(s), ctypes.byref(g), at(12), big, ST) == INVALID, name
    assert kta.raw_call("kta_ssm_scan_bwd", ctypes.byref(s), ctypes.byref(grads(kta)), at(9), big, ST) == INVALID
    row = 2 * 16 * 2 * 64 * 2                               # bytes of o: 32 tokens of 2 heads of 64
    for kw in (dict(pos=at(1, row - 8)), dict(freqs=at(1, row - 8)), dict(o=at(5, 8 * 32 - 16)), dict(o=at(6, 8 * 16 - 16)),
               dict(x2=at(2), o2=at(3), H2=2, ld2=2, pos=at(3, 64)), dict(x2=at(2), o2=at(3), H2=2, ld2=2, freqs=at(3, 64)),
               dict(o=at(0), pos=at(0, 64))):
        assert rope_call(kta, **kw) == INVALID, kw


def test_import_without_torchs_private_cuda_names(kta):
    """A torch built without CUDA has no _cuda_* functions: the host-side checks are there all the same."""
    import pathlib
    import subprocess
    import sys
    code = ("import torch\n"
            "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "from hybrid_linear_temporal_kta_b200 import kta\n"
            "assert kta.version() > 0 and kta.rope_freqs(8, device='cpu')[0].numel() == 4\n")
    root = pathlib.Path(kta.__file__).parents[1]
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True)


STRUCTS = [("Rope", "kta_rope", "_ROPE"), ("ShortConv", "kta_short_conv", "_CONV"), ("Ssm", "kta_ssm", "_SSM"),
           ("SsmGrads", "kta_ssm_grads", "_GRADS")]


def test_struct_layouts_are_the_headers(kta, tmp_path):
    """Sizes and offsets of the ctypes structures as a C compiler lays them out."""
    import pathlib
    import subprocess
    lines = [f'printf("%zu", sizeof({c}));' + "".join(f' printf(" %zu", offsetof({c}, {f[0]}));' for f in getattr(kta, py)._fields_)
             + ' printf("\\n");' for py, c, _ in STRUCTS]
    src = "#include <stddef.h>\n#include <stdio.h>\n#include \"kta.h\"\nint main(void) {\n" + "\n".join(lines) + "\nreturn 0; }\n"
    (tmp_path / "a.c").write_text(src)
    inc = pathlib.Path(kta.__file__).parents[1] / "include"
    subprocess.run(["gcc", f"-I{inc}", "-o", tmp_path / "a", tmp_path / "a.c"], check=True)
    out = subprocess.run([tmp_path / "a"], check=True, capture_output=True, text=True).stdout.splitlines()
    for (py, _, _), line in zip(STRUCTS, out, strict=True):
        t = getattr(kta, py)
        assert [int(v) for v in line.split()] == [ctypes.sizeof(t)] + [getattr(t, f[0]).offset for f in t._fields_], py


def test_packed_structs_are_the_ctypes_structures(kta):
    """What calls pack natively is, byte for byte, the structure that the library is declared to take."""
    for py, _, packed in STRUCTS:
        t, flat, fields = getattr(kta, py), [], []
        for i, (name, ty) in enumerate(t._fields_):
            if name == "dims":
                v = [101, 102, 103, 104]
                fields.append((ctypes.c_int * 4)(*v))
                flat += v
            else:
                v = 0.25 + i if ty is ctypes.c_float else (7 + i << 33) + i if ctypes.sizeof(ty) == 8 else (1 << 20) + i
                fields.append(v)
                flat.append(v)
        assert getattr(kta, packed).pack(*flat) == bytes(t(*fields)), py
