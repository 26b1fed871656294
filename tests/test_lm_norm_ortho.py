"""layer_norm, its gradients and newton_schulz without a GPU: the C entry points' refusals, their workspace sizes, the
binding's checks of its arguments, what autograd is told, and that no kernel spills."""
import ctypes
import os
import re
import subprocess
import types

import pytest
import torch

import allgather_gemm_amd as ag

_vp = ctypes.c_void_p
P = [_vp(0x10000 + 0x1000 * i) for i in range(12)]     # never dereferenced: every call is refused or empty
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
BF16 = torch.bfloat16


def test_exports():
    names = ag.declared_functions()
    for n in ("layer_norm", "layer_norm_bwd", "layer_norm_bwd_workspace", "newton_schulz", "newton_schulz_workspace"):
        assert n in names and hasattr(ag.lib(), n)


def norm(**kw):
    a = dict(x=P[0], res=P[1], w=P[2], b=P[3], rows=64, width=64, eps=1e-5, y=P[4], h=P[5], mean=P[6], rstd=P[7])
    a.update(kw)
    return ag.lib().layer_norm(a["x"], a["res"], a["w"], a["b"], a["rows"], a["width"], a["eps"], a["y"], a["h"], a["mean"],
                               a["rstd"], None)


def test_norm_refusals():
    for kw in (dict(rows=-1), dict(width=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None),
               dict(y=None), dict(res=None), dict(x=_vp(0x10008)), dict(res=_vp(0x10002)), dict(w=_vp(0x10008)),
               dict(b=_vp(0x10008)), dict(y=_vp(0x10004)), dict(h=_vp(0x10008)), dict(mean=_vp(0x10002)), dict(rstd=_vp(0x10001))):
        assert norm(**kw) == ag.AG_EINVAL, kw
    for kw in (dict(width=(1 << 21) + 1), dict(rows=(1 << 30) + 1)):
        assert norm(**kw) == ag.AG_EUNSUPPORTED, kw
    assert norm(rows=0) == ag.AG_OK and norm(width=0) == ag.AG_OK


def test_norm_bwd_refusals():
    need = ag.lib().layer_norm_bwd_workspace(640, 64)
    assert need > 0

    def call(**kw):
        a = dict(dy=P[0], h=P[1], mean=P[2], rstd=P[3], w=P[4], dh=P[5], rows=640, width=64, dx=P[6], dw=P[7], db=P[8], work=P[9], n=need)
        a.update(kw)
        return ag.lib().layer_norm_bwd(a["dy"], a["h"], a["mean"], a["rstd"], a["w"], a["dh"], a["rows"], a["width"], a["dx"],
                                       a["dw"], a["db"], a["work"], a["n"], None)
    for kw in (dict(rows=-1), dict(width=-2), dict(dy=None), dict(h=None), dict(mean=None), dict(rstd=None), dict(dy=_vp(0x10008)),
               dict(h=_vp(0x10008)), dict(mean=_vp(0x10002)), dict(w=_vp(0x10008)), dict(dh=_vp(0x10008)), dict(dx=_vp(0x10008)),
               dict(dw=_vp(0x10002)), dict(db=_vp(0x10008)), dict(work=None), dict(work=_vp(0x10008)), dict(n=need - 1)):
        assert call(**kw) == ag.AG_EINVAL, kw
    for kw in (dict(width=(1 << 21) + 1), dict(rows=(1 << 30) + 1)):
        assert call(**kw) == ag.AG_EUNSUPPORTED, kw
    assert call(width=0) == ag.AG_OK and call(dx=None, dw=None, db=None, work=None, n=0) == ag.AG_OK
    for rows, width in ((1 << 30, 1 << 21), (1 << 30, 64), (5, 1 << 21)):       # the partial sums stay small
        assert ag.lib().layer_norm_bwd_workspace(rows, width) <= 1024 * width * 8


def schulz(**kw):
    steps = kw.pop("steps", [3.4445, -4.7750, 2.0315] * 5)
    a = dict(G=P[0], type=ag.TYPE_BF16, E=1, R=64, C=96, n_steps=len(steps) // 3, eps=1e-7, out=P[1], work=P[2], n=1 << 50,
             q=(ctypes.c_float * len(steps))(*steps))
    a.update(kw)
    return ag.lib().newton_schulz(a["G"], a["type"], a["E"], a["R"], a["C"], a["q"], a["n_steps"], a["eps"], a["out"], a["work"],
                                  a["n"], None)


def test_schulz_refusals():
    need = ag.lib().newton_schulz_workspace(1, 64, 96)
    assert need > 0
    nan, inf = float("nan"), float("inf")
    for kw in (dict(E=-1), dict(R=-1), dict(C=-1), dict(n_steps=0), dict(q=None), dict(type=2), dict(type=-1), dict(eps=-1.0),
               dict(eps=nan), dict(eps=inf), dict(steps=[1.0, nan, 0.0]), dict(steps=[inf, 0.0, 0.0]), dict(G=None), dict(out=None),
               dict(G=_vp(0x10008)), dict(out=_vp(0x10002)), dict(work=None), dict(work=_vp(0x10008)), dict(n=need - 1)):
        assert schulz(**kw) == ag.AG_EINVAL, kw
    for kw in (dict(C=(1 << 20) + 1), dict(E=65536), dict(R=1 << 19, C=1 << 19), dict(E=60000, R=8192, C=8192)):
        assert schulz(**kw) == ag.AG_EUNSUPPORTED, kw
        assert ag.lib().newton_schulz_workspace(kw.get("E", 1), kw.get("R", 64), kw.get("C", 96)) == 0
    # iterates that could leave fp16: downwards, by their size, by that of b t + c t^2, or at an extremum inside the range
    for steps in ([10.0, 0.0, 0.0] * 2, [1.0, -40.0, 0.0], [1.0, 0.0, 30.0], [3.5, 3.5, 3.5] * 2, [2.0, 120.0, -125.0],
                  [20.0, -36.0, 16.0] * 2, [0.015, 0.0, 0.0] * 2, [0.0, 0.0, 0.0] * 2):
        assert schulz(steps=steps) == ag.AG_EUNSUPPORTED, steps
    for kw in (dict(E=0), dict(R=0), dict(C=0)):
        assert schulz(**kw) == ag.AG_OK


def test_binding_refuses_before_the_library_sees_it():
    x = torch.zeros(4, 64, dtype=BF16)
    for call, why in ((lambda: ag.layer_norm(x), "device tensor"), (lambda: ag.layer_norm(x.float()), "x must be"),
                      (lambda: ag.layer_norm(x[0]), "dimensions"), (lambda: ag.layer_norm(x, h=x), "without a residual"),
                      (lambda: ag.layer_norm_bwd(x, x[0], None, None), "dimensions"),
                      (lambda: ag.layer_norm_bwd(x.float(), x, torch.zeros(4), torch.zeros(4)), "dy must be"),
                      (lambda: ag.newton_schulz(x), "device tensor"), (lambda: ag.newton_schulz(x[0]), "dimensions"),
                      (lambda: ag.newton_schulz(x.half()), "bfloat16 or float32"),
                      (lambda: ag.newton_schulz(x, coefficients=()), "at least one step"),
                      (lambda: ag.newton_schulz(x, coefficients=[(1.0, 2.0)]), "at least one step")):
        with pytest.raises(ValueError, match=why):
            call()


def test_outputs_that_the_caller_gives_count_as_written(monkeypatch):
    done = []
    fake = types.SimpleNamespace(layer_norm=lambda *a: done.append("norm") or 0, newton_schulz=lambda *a: done.append("schulz") or 0)
    monkeypatch.setattr(ag, "lib", lambda: fake)
    monkeypatch.setattr(ag, "_need", lambda t, *a, **k: None if t is None else t.data_ptr())
    monkeypatch.setattr(ag, "_work", lambda *a: (None, 0))
    monkeypatch.setattr(ag, "_stream_of", lambda device: 0)
    x, res, y, h = (torch.zeros(4, 8, dtype=BF16) for _ in range(4))
    mean, rstd = torch.zeros(4), torch.zeros(4)
    assert ag.layer_norm(x, residual=res, y=y, h=h, mean=mean, rstd=rstd) is y
    assert all(t._version == 1 for t in (y, h, mean, rstd)) and x._version == res._version == 0
    assert ag.newton_schulz(x, out=x) is x and x._version == 1
    assert done == ["norm", "schulz"]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
@pytest.mark.parametrize("src", ["lm_norm.hip", "lm_ortho.hip"])
def test_no_scratch_and_no_spills(tmp_path, src):
    out = tmp_path / "kernels.s"
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S",
           os.path.join(ROOT, "allgather_gemm_amd", "csrc", src), "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    blocks = out.read_text().split("  - .agpr_count")[1:]
    assert blocks
    for block in blocks:
        value = {k: int(re.search(r"\.%s:\s+(\d+)" % k, block).group(1))
                 for k in ("private_segment_fixed_size", "vgpr_spill_count", "group_segment_fixed_size")}
        name = re.search(r"\.name:\s+(\S+)", block).group(1)
        assert value["private_segment_fixed_size"] == 0 and value["vgpr_spill_count"] == 0, (name, value)
        assert value["group_segment_fixed_size"] <= 160 * 1024, (name, value)
