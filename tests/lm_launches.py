"""Which kernels the language-model operators launch, and how, without a GPU: their host code (entry points, plans,
launches) compiled with lm_launches.cpp in place of the HIP runtime.  A call made through it records its launches."""
import collections
import concurrent.futures
import ctypes
import functools
import os
import re
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCES = ["lm_api", "lm_nt", "lm_nn", "lm_tn", "lm_rows", "lm_small"]
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

# kernel: its name and template arguments ("nt256<1>"), as the source has them, or "nn256", "nn256 scaled"; args: M, N, K and what else the
# product's arguments say (None for kernels that are no product)
Launch = collections.namedtuple("Launch", "kernel grid block args")
Args = collections.namedtuple("Args", "M N K group E splits part accumulate")

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
P = [_vp(0x100000 + 0x1000 * i) for i in range(12)]       # never dereferenced: nothing runs


@functools.lru_cache(maxsize=None)
def recorder():
    with tempfile.TemporaryDirectory() as tmp:
        def compile_one(src):
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            subprocess.run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17", "-fPIC",
                            "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj], check=True, capture_output=True)
            return obj
        srcs = [os.path.join(ROOT, "allgather_gemm_amd", "csrc", s + ".hip") for s in SOURCES]
        srcs.append(os.path.join(ROOT, "tests", "lm_launches.cpp"))
        with concurrent.futures.ThreadPoolExecutor(4) as ex:
            objs = list(ex.map(compile_one, srcs))
        # the device code that is not there
        undefined = subprocess.run(["nm", "-u"] + objs, check=True, capture_output=True, text=True).stdout
        binaries = sorted(set(re.findall(r"__hip_fatbin_\w+", undefined)))
        so = os.path.join(tmp, "lm_launches.so")
        subprocess.run(["g++", "-shared", "-o", so] + objs + ["-Wl,--defsym=%s=0" % b for b in binaries], check=True,
                       capture_output=True)
        L = ctypes.CDLL(so)
    L.rec_name.restype = ctypes.c_char_p
    for name, types in (("gemm_bias_act_workspace", [_i64] * 3), ("gemm_xent_workspace", [_i64] * 3),
                        ("gemm_xent_bwd_workspace", [_i64] * 3), ("gemm_bias_act_bwd_workspace", [_i64] * 3 + [_i32])):
        getattr(L, name).argtypes, getattr(L, name).restype = types, _i64
    L.gemm_bias_act.argtypes = [_vp] * 4 + [_i64] * 3 + [_i32, _vp, _vp, _vp, _i64, _vp]
    L.gemm_bias_act_bwd.argtypes = [_vp] * 4 + [_i64] * 3 + [_i32] + [_vp] * 4 + [_i64, _vp]
    L.gemm_grouped.argtypes = [_vp] * 3 + [_i32] + [_i64] * 3 + [_vp, _vp]
    L.gemm_grouped_bwd.argtypes = [_vp] * 4 + [_i32] + [_i64] * 3 + [_vp, _vp, _vp]
    L.gemm_xent.argtypes = [_vp] * 3 + [_i64] * 3 + [_vp] * 3 + [_i64, _vp]
    L.gemm_xent_bwd.argtypes = [_vp] * 5 + [_i64] * 3 + [_vp] * 3 + [_i64, _vp]
    return L


def _kernel(mangled):
    name, targs = re.match(r".*_GLOBAL__N_1\d+(\w+?)_kernel(?:I((?:L[ib]\d+E)+)E)?", mangled).groups()
    if name[:2] in ("nn", "tn"):         # the sums alone, or times the unit of the d logits
        return name + {"Li3E": "", "Li4E": " scaled"}[targs]
    return name + ("<%s>" % ",".join(re.findall(r"L[ib](\d+)E", targs)) if targs else "")


def _record(call, cus=256):
    L = recorder()
    L.rec_start(cus)
    rc = call(L)
    assert rc == 0, rc
    out = []
    for i in range(L.rec_count()):
        dims, args = (_i64 * 6)(), (_i64 * 8)()
        L.rec_dims(i, dims)
        tile = L.rec_args(i, args)
        out.append(Launch(_kernel(L.rec_name(i).decode()), tuple(dims[:3]), tuple(dims[3:]), Args(*args) if tile else None))
    return out


def linear(M, K, Nc, act="none", bias=False, residual=False, pre=False):
    return _record(lambda L: L.gemm_bias_act(P[0], P[1], P[2] if bias else None, P[3] if residual else None, M, Nc, K, ACTS[act],
                                             P[4], P[5] if pre else None, P[6], 1 << 50, None))


def linear_bwd(M, K, Nc, act="none", dA=True, dB=True, dbias=True):
    return _record(lambda L: L.gemm_bias_act_bwd(P[0], P[1], P[2], P[3], M, Nc, K, ACTS[act], P[4] if dA else None,
                                                 P[5] if dB else None, P[6] if dbias else None, P[7], 1 << 50, None))


def grouped(E, M, K, Nc):
    return _record(lambda L: L.gemm_grouped(P[0], P[1], P[2], E, M, Nc, K, P[3], None))


def grouped_bwd(E, M, K, Nc):
    return _record(lambda L: L.gemm_grouped_bwd(P[0], P[1], P[2], P[3], E, M, Nc, K, P[4], P[5], None))


def xent(T, K, V):
    return _record(lambda L: L.gemm_xent(P[0], P[1], P[2], T, V, K, P[3], P[4], P[5], 1 << 60, None))


def xent_bwd(T, K, V, work_bytes=None, dA=True, dB=True):
    """work_bytes: as gemm_xent_bwd_workspace() asks for where None."""
    n = recorder().gemm_xent_bwd_workspace(T, V, K) if work_bytes is None else work_bytes
    return _record(lambda L: L.gemm_xent_bwd(P[0], P[1], P[2], P[3], P[4], T, V, K, P[5] if dA else None, P[6] if dB else None,
                                             P[7], n, None))


def kernels():
    """Every kernel of the operators."""
    L = recorder()
    L.rec_kernel.restype = ctypes.c_char_p
    return {_kernel(L.rec_kernel(i).decode()) for i in range(L.rec_kernels())}


def _sizes(ends, limit):
    """Rows of each group and, last, of none, a table's entries held to the range that their predecessors leave."""
    out, prev = [], 0
    for e in list(ends) + [limit]:
        e = max(prev, min(int(e), limit))
        out.append(e - prev)
        prev = e
    return out


def pieces(launch, ends=()):
    """What a 256 x 256 kernel's launch is cut into: tiles ("tile"), two groups' halves as one unit ("pair"), and in its
    tail halves or quarters ("half", "quarter") of tiles ("... of tile"), of pairs, or left over ("lone ...")."""
    L, a = recorder(), launch.args
    assert "256" in launch.kernel
    by_rows, by_k = a.group == 1, a.group == 2
    units, halves = [], 0              # units in their order
    for n in _sizes(ends, a.M) if by_rows else [a.M]:
        units += ["tile"] * L.rec_big_rows(n)
        if L.rec_half_rows(n):
            halves += 1
            if halves % 2 == 0:
                units.append("pair")
    if not by_rows:
        assert halves < 2
    parts = a.E if by_k else a.splits
    cols, quarter_cols, cut = (a.N + 255) // 256, (a.N + 127) // 128, (ctypes.c_int * 2)(0, 0)
    if not by_k:
        L.rec_tail(len(units), halves & 1, cols * parts, quarter_cols * parts, launch.grid[0], cut)
    kind = "quarter" if cut[1] else "half"
    whole, tail = units[:len(units) - cut[0]], units[len(units) - cut[0]:]
    return set(whole) | {"%s of %s" % (kind, u) for u in tail} | ({"lone " + kind} if halves & 1 else set())
