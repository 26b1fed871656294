"""Which kernels layer_norm, its gradients and newton_schulz launch, and how, without a GPU: their host code compiled with
lm_launches.cpp in place of the HIP runtime.  A call made through it records its launches."""
import collections
import ctypes
import functools
import os
import re
import subprocess
import tempfile

from lm_launches import HIPCC, ROOT, P, _i32, _i64, _vp

Launch = collections.namedtuple("Launch", "kernel grid block")
SCHULZ = (3.4445, -4.7750, 2.0315) * 5


@functools.lru_cache(maxsize=None)
def recorder():
    with tempfile.TemporaryDirectory() as tmp:
        objs = []
        for src in ("allgather_gemm_amd/csrc/lm_norm.hip", "allgather_gemm_amd/csrc/lm_ortho.hip", "tests/lm_launches.cpp"):
            objs.append(os.path.join(tmp, os.path.basename(src) + ".o"))
            subprocess.run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-I",
                            os.path.join(ROOT, "include"), "-c", os.path.join(ROOT, src), "-o", objs[-1]], check=True,
                           capture_output=True)
        undefined = subprocess.run(["nm", "-u"] + objs, check=True, capture_output=True, text=True).stdout
        binaries = sorted(set(re.findall(r"__hip_fatbin_\w+", undefined)))
        so = os.path.join(tmp, "norm_ortho_launches.so")
        subprocess.run(["g++", "-shared", "-o", so] + objs + ["-Wl,--defsym=%s=0" % b for b in binaries], check=True,
                       capture_output=True)
        L = ctypes.CDLL(so)
    L.rec_name.restype = L.rec_kernel.restype = ctypes.c_char_p
    L.layer_norm.argtypes = [_vp] * 4 + [_i64] * 2 + [ctypes.c_float] + [_vp] * 5
    L.layer_norm_bwd.argtypes = [_vp] * 6 + [_i64] * 2 + [_vp] * 4 + [_i64, _vp]
    L.newton_schulz.argtypes = [_vp, _i32] + [_i64] * 3 + [_vp, _i32, ctypes.c_float, _vp, _vp, _i64, _vp]
    for name, n in (("layer_norm_bwd_workspace", 2), ("newton_schulz_workspace", 3)):
        getattr(L, name).argtypes, getattr(L, name).restype = [_i64] * n, _i64
    return L


def _kernel(mangled):
    """Name and template arguments as the source has them: "ortho64<5,2,0>", "ortho_norm<f>"."""
    name, args = re.match(r".*_GLOBAL__N_1\d+(\w+?)_kernel(?:I((?:L[ib]\d+E|f|DF16b)+)E)?(?:E|v|P|N)", mangled).groups()
    return name + ("<%s>" % ",".join(a or b for a, b in re.findall(r"L[ib](\d+)E|(f|DF16b)", args)) if args else "")


def _record(call, cus=256):
    L = recorder()
    L.rec_start(cus)
    rc = call(L)
    assert rc == 0, rc
    out = []
    for i in range(L.rec_count()):
        dims = (_i64 * 6)()
        L.rec_dims(i, dims)
        out.append(Launch(_kernel(L.rec_name(i).decode()), tuple(dims[:3]), tuple(dims[3:])))
    return out


def kernels():
    L = recorder()
    return {_kernel(L.rec_kernel(i).decode()) for i in range(L.rec_kernels())}


def norm(rows, width):
    return _record(lambda L: L.layer_norm(P[0], P[1], P[2], P[3], rows, width, 1e-5, P[4], P[5], P[6], P[7], None))


def norm_bwd(rows, width, dx=True, dh=True, sums=True):
    n = recorder().layer_norm_bwd_workspace(rows, width)
    return _record(lambda L: L.layer_norm_bwd(P[0], P[1], P[2], P[3], P[4], P[5] if dh else None, rows, width, P[6] if dx else None,
                                              P[7] if sums else None, P[8] if sums else None, P[9], n, None))


def schulz(E, R, C, fp32=False, coefficients=SCHULZ):
    n = recorder().newton_schulz_workspace(E, R, C)
    q = (ctypes.c_float * len(coefficients))(*coefficients)
    return _record(lambda L: L.newton_schulz(P[0], int(fp32), E, R, C, q, len(coefficients) // 3, 1e-7, P[1], P[2], n, None))
