"""Host-code checks of the selective scan, the causal convolution and the 8-bit copies for the sanitizer build of
the library, run by tests/test_host_sanitized_selscan.py in a child process with the sanitizer runtime
preloaded: only ctypes, and no device call (every compute call below is refused before any HIP call)."""
import ctypes
import sys

lib = ctypes.CDLL(sys.argv[1])
vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class Scan(ctypes.Structure):
    _fields_ = [(n, i32) for n in ("B", "T", "E", "N", "G", "dtype", "softplus")] + \
               [(n, i64 * 2) for n in ("u_stride", "dt_stride", "z_stride")] + [(n, i64 * 3) for n in ("B_stride", "C_stride")] + \
               [("lens", vp), ("stream", vp), ("workspace", vp), ("workspace_bytes", ctypes.c_size_t)]


class Conv(ctypes.Structure):
    _fields_ = [(n, i32) for n in ("B", "T", "E", "W", "dtype", "act")] + [("x_stride", i64 * 2)] + \
               [("lens", vp), ("stream", vp), ("workspace", vp), ("workspace_bytes", ctypes.c_size_t)]


class Checkpoint(ctypes.Structure):
    _fields_ = [(n, i32) for n in ("B", "T", "E", "dtype")] + [("x_stride", i64 * 2), ("stream", vp)]


P = ctypes.POINTER
for name, args, res in [
    ("pnr_selscan_workspace_bytes", [P(Scan)], ctypes.c_size_t),
    ("pnr_selscan_workspace_bytes_backward", [P(Scan)], ctypes.c_size_t),
    ("pnr_selscan_forward", [P(Scan)] + [vp] * 11, ctypes.c_int),
    ("pnr_selscan_step", [P(Scan)] + [vp] * 10 + [ctypes.c_int, vp, vp], ctypes.c_int),
    ("pnr_selscan_backward", [P(Scan)] + [vp] * 20, ctypes.c_int),
    ("pnr_conv_workspace_bytes_backward", [P(Conv)], ctypes.c_size_t),
    ("pnr_conv_forward", [P(Conv)] + [vp] * 7, ctypes.c_int),
    ("pnr_conv_step", [P(Conv)] + [vp] * 5 + [ctypes.c_int, vp, vp], ctypes.c_int),
    ("pnr_conv_backward", [P(Conv)] + [vp] * 11, ctypes.c_int),
    ("pnr_checkpoint_pack", [P(Checkpoint)] + [vp] * 3, ctypes.c_int),
    ("pnr_checkpoint_unpack", [P(Checkpoint)] + [vp] * 3, ctypes.c_int),
    ("pnr_last_error", [], ctypes.c_char_p),
]:
    f = getattr(lib, name)
    f.argtypes, f.restype = args, res

E_INVALID, E_UNSUPPORTED, E_WORKSPACE = -1, -2, -3
F64, F32, BF16 = 0, 1, 2
ADDR, CHANNELS, TOKENS = 0x10000, 1 << 20, 1 << 30
fails = []


def expect(cond, what):
    if not cond:
        fails.append(what)


def scan(B=2, T=100, E=64, N=16, G=1, dtype=BF16, soft=1, ws=None, nbytes=0, s2=(6400, 64), s3=(1600, 16, 16), lens=None):
    return Scan(B, T, E, N, G, dtype, soft, (i64 * 2)(*s2), (i64 * 2)(*s2), (i64 * 2)(*s2), (i64 * 3)(*s3), (i64 * 3)(*s3), lens, None, ws, nbytes)


def conv(B=2, T=100, E=64, W=4, dtype=BF16, act=1, ws=None, nbytes=0, s=(6400, 64)):
    return Conv(B, T, E, W, dtype, act, (i64 * 2)(*s), None, None, ws, nbytes)


def scan_calls(d):
    r = ctypes.byref(d)
    return [lib.pnr_selscan_forward(r, *[ADDR] * 5, *[None] * 4, ADDR, None),
            lib.pnr_selscan_backward(r, *[ADDR] * 5, *[None] * 4, ADDR, *[None] * 10)]


def conv_back(d):
    return lib.pnr_conv_backward(ctypes.byref(d), ADDR, None, ADDR, None, None, ADDR, *[None] * 5)


# workspace sizes over grids of shapes; each that is needed is asked for
for dtype in (F32, BF16):
    for B in (1, 3, 64, 4000000):
        for T in (0, 1, 16, 129, 2049, 65536, TOKENS):
            for E, G in ((1, 1), (64, 1), (65, 1), (330, 2), (4096, 4), (8192, 8192), (CHANNELS, 1), (CHANNELS, CHANNELS)):
                for lens in (None, ADDR):
                    for N in (1, 16, 33, 64):
                        d = scan(B, T, E, N, G, dtype, lens=lens)
                        fwd, bwd = lib.pnr_selscan_workspace_bytes(ctypes.byref(d)), lib.pnr_selscan_workspace_bytes_backward(ctypes.byref(d))
                        tiles = G * ((E // G + 63) // 64)
                        big = tiles > 65536 or B * tiles > 4000000
                        expect((bwd > 0) == (not big) and bwd >= fwd, ("scan ws", B, T, E, G, N, fwd, bwd))
                        got = scan_calls(d)
                        expect(got[1] == (E_INVALID if big else E_WORKSPACE), ("scan no ws", B, T, E, G, N, got))
                        if fwd or big:
                            expect(got[0] == (E_INVALID if big else E_WORKSPACE), ("scan fwd no ws", B, T, E, G, N, got))
                        if not big:
                            for ws, nb in ((ADDR + 8, bwd), (ADDR, bwd - 1)):
                                expect(scan_calls(scan(B, T, E, N, G, dtype, ws=ws, nbytes=nb, lens=lens))[1] == E_WORKSPACE, ("scan ws", ws, nb))
                for W in (1, 4, 8):
                    d = conv(B, T, E, W, dtype)
                    need = lib.pnr_conv_workspace_bytes_backward(ctypes.byref(d))
                    big = B * (E // 64 + 1) > 4000000
                    expect((need > 0) == (not big), ("conv ws", B, T, E, W, need))
                    expect(conv_back(d) == (E_INVALID if big else E_WORKSPACE), ("conv no ws", B, T, E, W))
                    if not big:
                        expect(conv_back(conv(B, T, E, W, dtype, ws=ADDR, nbytes=need - 1)) == E_WORKSPACE, ("conv small ws", B, T, E, W))

# refusals
for kw, code in ((dict(B=0), E_INVALID), (dict(T=-1), E_INVALID), (dict(T=TOKENS + 1), E_INVALID), (dict(E=CHANNELS + 1), E_INVALID),
                 (dict(G=5), E_INVALID), (dict(N=0), E_INVALID), (dict(N=65), E_UNSUPPORTED), (dict(dtype=F64), E_UNSUPPORTED), (dict(dtype=-5), E_INVALID),
                 (dict(soft=9), E_INVALID), (dict(s2=(-1, 1)), E_INVALID), (dict(s3=(1, 1, -1)), E_INVALID), (dict(s2=(0, 1 << 62)), E_UNSUPPORTED),
                 (dict(B=2 ** 31 - 1, E=2 ** 31 - 1, G=2 ** 31 - 1), E_INVALID)):
    d = scan(**kw)
    expect(scan_calls(d) == [code, code] and lib.pnr_last_error() != b"", ("scan", kw))
    expect(lib.pnr_selscan_workspace_bytes_backward(ctypes.byref(d)) == 0, ("scan ws", kw))
for kw, code in ((dict(B=0), E_INVALID), (dict(T=-1), E_INVALID), (dict(T=TOKENS + 1), E_INVALID), (dict(E=2 ** 31 - 1), E_INVALID), (dict(W=0), E_INVALID),
                 (dict(W=9), E_UNSUPPORTED), (dict(act=2), E_UNSUPPORTED), (dict(act=7), E_INVALID), (dict(s=(-1, 0)), E_INVALID)):
    d = conv(**kw)
    expect(conv_back(d) == code and lib.pnr_last_error() != b"", ("conv", kw))
    expect(lib.pnr_conv_forward(ctypes.byref(d), ADDR, None, ADDR, None, None, ADDR, None) == code, ("conv", kw))
for kw in (dict(B=0), dict(E=0), dict(T=-1), dict(B=2 ** 31 - 1, T=TOKENS, E=CHANNELS), dict(E=CHANNELS + 1), dict(dtype=9)):
    v = dict(B=1, T=1, E=1, dtype=F32)
    v.update(kw)
    d = Checkpoint(*v.values(), (i64 * 2)(0, 0), None)
    expect(lib.pnr_checkpoint_pack(ctypes.byref(d), ADDR, ADDR, ADDR) == E_INVALID, ("checkpoint", kw))
    expect(lib.pnr_checkpoint_unpack(ctypes.byref(d), ADDR, ADDR, ADDR) == E_INVALID, ("checkpoint", kw))
d = scan()
for n_slots, slots in ((0, ADDR), (1, None), (-5, None)):
    expect(lib.pnr_selscan_step(ctypes.byref(d), *[ADDR] * 5, *[None] * 3, ADDR, slots, n_slots, ADDR, ADDR) == E_INVALID, ("slots", n_slots))
for f, n in ((lib.pnr_selscan_forward, 11), (lib.pnr_selscan_backward, 20), (lib.pnr_conv_forward, 7), (lib.pnr_conv_backward, 11),
             (lib.pnr_checkpoint_pack, 3), (lib.pnr_checkpoint_unpack, 3)):
    expect(f(None, *[ADDR] * n) == E_INVALID, "null descriptor")
for f in (lib.pnr_selscan_workspace_bytes, lib.pnr_selscan_workspace_bytes_backward, lib.pnr_conv_workspace_bytes_backward):
    expect(f(None) == 0, "null descriptor's workspace")

if fails:
    print("FAILED:", fails[:20])
    sys.exit(1)
print("host checks passed")
