"""Host-code checks of the sequence-mixing entry points for the sanitizer build of the library, run by
tests/test_host_sanitized_sequence.py in a child process with the sanitizer runtime preloaded: only ctypes,
and no device call (every compute call below is refused before any HIP call)."""
import ctypes
import sys

lib = ctypes.CDLL(sys.argv[1])
vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class Attn(ctypes.Structure):
    _fields_ = [(n, i32) for n in ("B", "T", "H", "H_kv", "D_k", "D_v", "dtype", "decay")] + [("scale", ctypes.c_double)] + \
               [(n, i64 * 3) for n in ("q_stride", "k_stride", "v_stride")] + \
               [("lens", vp), ("stream", vp), ("workspace", vp), ("workspace_bytes", ctypes.c_size_t)]


class Norm(ctypes.Structure):
    _fields_ = [(n, i32) for n in ("N", "L", "C", "groups", "dtype", "act")] + [("eps", ctypes.c_double)] + \
               [("lens", vp), ("stream", vp), ("workspace", vp), ("workspace_bytes", ctypes.c_size_t)]


P = ctypes.POINTER
for name, args, res in [
    ("pnr_linattn_workspace_bytes", [P(Attn)], ctypes.c_size_t),
    ("pnr_linattn_workspace_bytes_backward", [P(Attn)], ctypes.c_size_t),
    ("pnr_linattn_forward", [P(Attn)] + [vp] * 7, ctypes.c_int),
    ("pnr_linattn_step", [P(Attn)] + [vp] * 6 + [ctypes.c_int, vp, vp], ctypes.c_int),
    ("pnr_linattn_backward", [P(Attn)] + [vp] * 12, ctypes.c_int),
    ("pnr_groupnorm_workspace_bytes", [P(Norm)], ctypes.c_size_t),
    ("pnr_groupnorm_workspace_bytes_backward", [P(Norm)], ctypes.c_size_t),
    ("pnr_groupnorm", [P(Norm)] + [vp] * 7, ctypes.c_int),
    ("pnr_groupnorm_backward", [P(Norm)] + [vp] * 11, ctypes.c_int),
    ("pnr_last_error", [], ctypes.c_char_p),
]:
    f = getattr(lib, name)
    f.argtypes, f.restype = args, res

E_INVALID, E_UNSUPPORTED, E_WORKSPACE = -1, -2, -3
F64, F32, BF16 = 0, 1, 2
ADDR = 0x10000
fails = []


def expect(cond, what):
    if not cond:
        fails.append(what)


def attn(B=2, T=100, H=4, H_kv=2, D_k=64, D_v=64, dtype=BF16, decay=0, scale=0.125, ws=None, nbytes=0, stride=(25600, 256, 64)):
    s = (i64 * 3)(*stride)
    return Attn(B, T, H, H_kv, D_k, D_v, dtype, decay, scale, s, s, s, None, None, ws, nbytes)


def norm(N=2, L=10, C=64, groups=4, dtype=F32, act=1, eps=1e-5, ws=None, nbytes=0):
    return Norm(N, L, C, groups, dtype, act, eps, None, None, ws, nbytes)


def attn_calls(d):
    r = ctypes.byref(d)
    a = [ADDR] * 4
    return [lib.pnr_linattn_forward(r, *a, None, ADDR, None), lib.pnr_linattn_backward(r, *a, None, ADDR, *[None] * 6)]


def norm_calls(d):
    r = ctypes.byref(d)
    return [lib.pnr_groupnorm(r, ADDR, None, None, None, ADDR, None, None),
            lib.pnr_groupnorm_backward(r, ADDR, None, None, None, ADDR, ADDR, ADDR, ADDR, None, None, None)]


# workspace sizes over grids of shapes; each that is needed is asked for
for dtype in (F32, BF16):
    for B, H, Hkv in ((1, 1, 1), (1, 16, 16), (3, 6, 2), (64, 16, 4), (250, 32, 32), (8000000, 1, 1), (244, 32768, 32768)):
        for T in (0, 1, 63, 64, 65, 193, 2049, 65536, 1 << 30):
            for Dk, Dv in ((1, 1), (64, 64), (65, 7), (128, 128)):
                d = attn(B, T, H, Hkv, Dk, Dv, dtype)
                fwd, bwd = lib.pnr_linattn_workspace_bytes(ctypes.byref(d)), lib.pnr_linattn_workspace_bytes_backward(ctypes.byref(d))
                expect(bwd > 0 and bwd >= fwd, ("attn ws", dtype, B, H, T, Dk, Dv, fwd, bwd))
                expect(attn_calls(d)[1] == E_WORKSPACE, ("attn no ws", B, T))
                if fwd:
                    expect(attn_calls(d)[0] == E_WORKSPACE, ("attn fwd no ws", B, T))
                for ws, nb in ((ADDR + 8, bwd), (ADDR, bwd - 1)):
                    expect(attn_calls(attn(B, T, H, Hkv, Dk, Dv, dtype, ws=ws, nbytes=nb))[1] == E_WORKSPACE, ("attn ws", ws, nb))
    for N in (1, 7, 300, 65536, 16000000):
        for L in (0, 1, 2, 9, 1000, 1 << 20, 1 << 30):
            for C, groups in ((1, 1), (8, 8), (330, 11), (513, 1), (2048, 16), (4100, 2), (9001, 1), (1 << 20, 2), (1 << 26, 1)):
                d = norm(N, L, C, groups, dtype)
                fwd, bwd = lib.pnr_groupnorm_workspace_bytes(ctypes.byref(d)), lib.pnr_groupnorm_workspace_bytes_backward(ctypes.byref(d))
                big = N * groups > (1.6e7 if L != 1 or C // groups > 512 else 2e9) or N * L * C > 4.0e18
                expect((bwd > 0) == (not big), ("norm ws", dtype, N, L, C, groups, fwd, bwd))
                expect(norm_calls(d)[1] == (E_INVALID if big else E_WORKSPACE), ("norm no ws", N, L, C))

# refusals
for kw, code in ((dict(B=0), E_INVALID), (dict(T=-1), E_INVALID), (dict(T=(1 << 30) + 1), E_INVALID), (dict(H_kv=3), E_INVALID),
                 (dict(D_k=129), E_UNSUPPORTED), (dict(dtype=F64), E_UNSUPPORTED), (dict(dtype=-5), E_INVALID),
                 (dict(decay=9), E_INVALID), (dict(scale=float("nan")), E_INVALID), (dict(scale=1e300), E_INVALID),
                 (dict(stride=(-1, 1, 1)), E_INVALID), (dict(B=2 ** 31 - 1, H=2 ** 31 - 1, H_kv=2 ** 31 - 1), E_INVALID)):
    d = attn(**kw)
    expect(attn_calls(d) == [code, code] and lib.pnr_last_error() != b"", ("attn", kw))
    expect(lib.pnr_linattn_workspace_bytes_backward(ctypes.byref(d)) == 0, ("attn ws", kw))
for kw, code in ((dict(N=0), E_INVALID), (dict(L=-1), E_INVALID), (dict(L=2 ** 31 - 1), E_INVALID), (dict(C=2 ** 31 - 1, groups=1), E_INVALID),
                 (dict(groups=5), E_INVALID), (dict(act=7), E_INVALID), (dict(dtype=F64), E_UNSUPPORTED), (dict(eps=1e-300), E_INVALID),
                 (dict(eps=float("nan")), E_INVALID), (dict(N=2 ** 31 - 1, C=2 ** 26, L=2 ** 30), E_INVALID)):
    d = norm(**kw)
    expect(norm_calls(d) == [code, code] and lib.pnr_last_error() != b"", ("norm", kw))
    expect(lib.pnr_groupnorm_workspace_bytes_backward(ctypes.byref(d)) == 0, ("norm ws", kw))
d = attn()
for n_slots, slots in ((0, ADDR), (1, None), (-5, None)):
    expect(lib.pnr_linattn_step(ctypes.byref(d), *[ADDR] * 5, slots, n_slots, ADDR, ADDR) == E_INVALID, ("slots", n_slots))
for i in range(4):
    a = [ADDR] * 4
    for bad in (None, ADDR + 1):
        a[i] = bad
        expect(lib.pnr_linattn_forward(ctypes.byref(d), *a, None, ADDR, None) == E_INVALID, ("pointer", i, bad))
for f, n in ((lib.pnr_linattn_forward, 7), (lib.pnr_linattn_backward, 12), (lib.pnr_groupnorm, 7), (lib.pnr_groupnorm_backward, 11)):
    expect(f(None, *[ADDR] * n) == E_INVALID, "null descriptor")
for f in (lib.pnr_linattn_workspace_bytes, lib.pnr_linattn_workspace_bytes_backward, lib.pnr_groupnorm_workspace_bytes,
          lib.pnr_groupnorm_workspace_bytes_backward):
    expect(f(None) == 0, "null descriptor's workspace")

if fails:
    print("FAILED:", fails[:20])
    sys.exit(1)
print("host checks passed")
