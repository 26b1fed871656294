"""What newton_schulz's plans choose for a stack's extents, without a GPU."""
import collections
import ctypes
import functools
import os
import re
import subprocess
import tempfile

from lm_launches import HIPCC, ROOT, _i64

CUS = 256
# epi: "gram" (X X^T), "square" (A A), "update" (B X, "thin" where B is formed next to it); size: width of the tiles; tiles: how
# many; cut: those that go in quarters; parts: of a reduction
Plan = collections.namedtuple("Plan", "epi size tiles cut parts")


@functools.lru_cache(maxsize=None)
def library():
    with tempfile.TemporaryDirectory() as tmp:
        objs = []
        for src in ("ortho_plans.cpp", "lm_launches.cpp"):
            objs.append(os.path.join(tmp, src + ".o"))
            subprocess.run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-I",
                            os.path.join(ROOT, "include"), "-c", os.path.join(ROOT, "tests", src), "-o", objs[-1]], check=True,
                           capture_output=True)
        undefined = subprocess.run(["nm", "-u"] + objs, check=True, capture_output=True, text=True).stdout
        binaries = sorted(set(re.findall(r"__hip_fatbin_\w+", undefined)))
        so = os.path.join(tmp, "ortho_plans.so")
        subprocess.run(["g++", "-shared", "-o", so] + objs + ["-Wl,--defsym=%s=0" % b for b in binaries], check=True,
                       capture_output=True)
        L = ctypes.CDLL(so)
    L.rec_start(CUS)
    L.plan_of.argtypes = [ctypes.c_int] + [_i64] * 4 + [ctypes.POINTER(_i64)]
    return L


@functools.lru_cache(maxsize=None)
def plan(epi, E, M, N, K):
    out = (_i64 * 4)()
    library().plan_of(epi, E, M, N, K, out)
    return Plan(("gram", "square", "update")[epi], out[0], out[3], out[1], out[2])


def plans(E, R, C):
    """Of the products of a step."""
    m, n = (-(-x // 128) * 128 for x in sorted((R, C)))
    first = plan(0, E, m, m, n)
    if m <= 256:
        return [first, Plan("thin", m, 0, 0, 1)]
    return [first, plan(1, E, m, m, m), plan(2, E, m, n, m)]


def ways(E, R, C, cus=CUS):
    """What tells one way through the kernels from another: the product, the width of its tiles, whether some of them go in
    quarters, whether two 64 x 64 ones share a CU, parts, and whether the result of the last product is turned."""
    out = set()
    for p in plans(E, R, C):
        two = p.size == 64 and (p.tiles * p.parts > cus)
        way = (p.epi, p.size, p.cut > 0, two, p.parts > 1)
        out.add(way + (R > C,) if p.epi in ("update", "thin") else way)
    return out
