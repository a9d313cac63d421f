"""Single-token calls through their host code up to the launch, for the sanitizer build of the library, run by
tests/test_host_sanitized_steps.py in a child process that sees no device: the launch fails and is reported, and
no kernel runs.  What a single token does not read (T, token strides) holds what it likes."""
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


lib.pnr_conv_step.argtypes = [ctypes.POINTER(Conv)] + [vp] * 5 + [ctypes.c_int, vp, vp]
lib.pnr_selscan_step.argtypes = [ctypes.POINTER(Scan)] + [vp] * 10 + [ctypes.c_int, vp, vp]
lib.pnr_last_error.restype = ctypes.c_char_p
hip = ctypes.CDLL("libamdhip64.so")
count = ctypes.c_int(0)
if hip.hipGetDeviceCount(ctypes.byref(count)) == 0 and count.value:
    print("a device is visible: not run")
    sys.exit(3)

ADDR, MOST, LEAST = 0x10000, 2 ** 31 - 1, -2 ** 31
bad = []
for T in (MOST, MOST - 7, LEAST, -1, 0, 1):
    for far in (2 ** 63 - 1, -2 ** 63, 0):
        for E in (1, 64, 4096, 1 << 20):
            for W in (1, 4, 8):
                rc = lib.pnr_conv_step(ctypes.byref(Conv(2, T, E, W, 2, 1, (i64 * 2)(E, far), ADDR, None, None, 0)), ADDR, ADDR, None, ADDR, None, 2,
                                       ADDR, ADDR)
                if rc == 0 or b"step" not in lib.pnr_last_error():
                    bad.append(("conv", T, far, E, W, rc, lib.pnr_last_error()))
            s2, s3 = (i64 * 2)(E, far), (i64 * 3)(16, far, 16)
            rc = lib.pnr_selscan_step(ctypes.byref(Scan(2, T, E, 16, 1, 2, 1, s2, s2, s2, s3, s3, ADDR, None, None, 0)), *[ADDR] * 5, None, ADDR, None,
                                      ADDR, None, 2, ADDR, ADDR)
            if rc == 0 or b"step" not in lib.pnr_last_error():
                bad.append(("scan", T, far, E, rc, lib.pnr_last_error()))
if bad:
    print("FAILED:", bad[:10])
    sys.exit(1)
print("host checks passed")
