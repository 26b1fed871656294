"""The language-model operators without a GPU: the C entry points' refusals, their workspace sizes, the
binding's checks of its arguments."""
import ctypes

import pytest
import torch

import allgather_gemm_amd as ag

_vp = ctypes.c_void_p
P = [_vp(0x10000 + 0x1000 * i) for i in range(12)]     # never dereferenced: every call is refused or empty


def test_exports():
    names = ag.declared_functions()
    for n in ("gemm_bias_act", "gemm_bias_act_workspace", "gemm_bias_act_bwd", "gemm_bias_act_bwd_workspace", "gemm_grouped",
              "gemm_grouped_bwd", "gemm_xent", "gemm_xent_workspace", "gemm_xent_bwd", "gemm_xent_bwd_workspace"):
        assert n in names and hasattr(ag.lib(), n)


def linear(**kw):
    a = dict(A=P[0], B=P[1], bias=P[2], res=P[3], M=64, Nc=64, K=64, act=1, C=P[4], pre=P[5], work=P[6], n=1 << 40)
    a.update(kw)
    return ag.lib().gemm_bias_act(a["A"], a["B"], a["bias"], a["res"], a["M"], a["Nc"], a["K"], a["act"], a["C"],
                                  a["pre"], a["work"], a["n"], None)


def test_linear_refusals():
    for kw in (dict(M=-1), dict(Nc=-1), dict(K=-8), dict(K=60), dict(act=5), dict(act=-1), dict(A=None), dict(B=None),
               dict(C=None), dict(A=_vp(0x10008)), dict(B=_vp(0x10002)), dict(C=_vp(0x10004)), dict(bias=_vp(0x10002)),
               dict(res=_vp(0x10008)), dict(pre=_vp(0x10008))):
        assert linear(**kw) == ag.AG_EINVAL, kw
    for kw in (dict(K=(1 << 21) + 8), dict(Nc=(1 << 21) + 1), dict(M=(1 << 30) + 1)):
        assert linear(**kw) == ag.AG_EUNSUPPORTED, kw
    assert linear(M=0) == ag.AG_OK and linear(Nc=0) == ag.AG_OK
    # one row over a long reduction is split: its workspace must be there
    need = ag.lib().gemm_bias_act_workspace(500, 1003, 8192)
    if need:
        assert linear(M=500, Nc=1003, K=8192, n=need - 1) == ag.AG_EINVAL
        assert linear(M=500, Nc=1003, K=8192, work=None, n=need) == ag.AG_EINVAL
        assert linear(M=500, Nc=1003, K=8192, work=_vp(0x10008)) == ag.AG_EINVAL


def test_linear_bwd_refusals():
    def call(**kw):
        a = dict(dC=P[0], A=P[1], B=P[2], pre=P[3], M=64, Nc=64, K=64, act=2, dA=P[4], dB=P[5], db=P[6], work=P[7], n=1 << 40)
        a.update(kw)
        return ag.lib().gemm_bias_act_bwd(a["dC"], a["A"], a["B"], a["pre"], a["M"], a["Nc"], a["K"], a["act"], a["dA"],
                                          a["dB"], a["db"], a["work"], a["n"], None)
    for kw in (dict(M=-1), dict(K=12), dict(act=9), dict(dC=None), dict(A=None), dict(B=None), dict(pre=None),
               dict(dA=_vp(0x10008)), dict(dB=_vp(0x10008)), dict(db=_vp(0x10002)), dict(work=None), dict(n=0),
               dict(work=_vp(0x10004))):
        assert call(**kw) == ag.AG_EINVAL, kw
    assert call(K=(1 << 21) + 8) == ag.AG_EUNSUPPORTED
    # nothing wanted: nothing runs, and the operands of what is not wanted may be absent
    assert call(dA=None, dB=None, db=None, A=None, B=None) == ag.AG_OK


def test_grouped_refusals():
    def call(bwd=False, **kw):
        a = dict(dC=P[0], A=P[1], B=P[2], ends=P[3], E=4, M=64, Nc=64, K=64, C=P[4], dA=P[5], dB=P[6])
        a.update(kw)
        if bwd:
            return ag.lib().gemm_grouped_bwd(a["dC"], a["A"], a["B"], a["ends"], a["E"], a["M"], a["Nc"], a["K"], a["dA"],
                                             a["dB"], None)
        return ag.lib().gemm_grouped(a["A"], a["B"], a["ends"], a["E"], a["M"], a["Nc"], a["K"], a["C"], None)
    both = (dict(E=0), dict(E=-3), dict(M=-1), dict(Nc=12), dict(K=12), dict(ends=None), dict(ends=_vp(0x10002)),
            dict(A=None), dict(B=None), dict(A=_vp(0x10008)), dict(B=_vp(0x10008)))
    for kw in both + (dict(C=None), dict(C=_vp(0x10008))):
        assert call(**kw) == ag.AG_EINVAL, kw
    for kw in both + (dict(dC=None), dict(dA=_vp(0x10008)), dict(dB=_vp(0x10008))):
        assert call(True, **kw) == ag.AG_EINVAL, kw
    assert call(E=1025) == ag.AG_EUNSUPPORTED and call(True, E=1025) == ag.AG_EUNSUPPORTED
    assert call(M=0) == ag.AG_OK and call(Nc=0) == ag.AG_OK and call(True, dA=None, dB=None) == ag.AG_OK


def test_xent_refusals():
    need = ag.lib().gemm_xent_workspace(64, 1000, 64)
    assert need > 0

    def fwd(**kw):
        a = dict(A=P[0], B=P[1], y=P[2], T=64, V=1000, K=64, loss=P[3], lse=P[4], work=P[5], n=need)
        a.update(kw)
        return ag.lib().gemm_xent(a["A"], a["B"], a["y"], a["T"], a["V"], a["K"], a["loss"], a["lse"], a["work"], a["n"], None)
    for kw in (dict(V=0), dict(T=-1), dict(K=4), dict(A=None), dict(B=None), dict(y=None), dict(y=_vp(0x10004)),
               dict(loss=None), dict(lse=_vp(0x10002)), dict(work=None), dict(n=need - 1), dict(B=_vp(0x10008))):
        assert fwd(**kw) == ag.AG_EINVAL, kw
    assert fwd(V=(1 << 21) + 1) == ag.AG_EUNSUPPORTED and fwd(T=0) == ag.AG_OK

    def bwd(**kw):
        a = dict(g=P[0], A=P[1], B=P[2], y=P[3], lse=P[4], T=64, V=1000, K=64, dA=P[5], dB=P[6], work=P[7], n=1 << 30)
        a.update(kw)
        return ag.lib().gemm_xent_bwd(a["g"], a["A"], a["B"], a["y"], a["lse"], a["T"], a["V"], a["K"], a["dA"], a["dB"],
                                      a["work"], a["n"], None)
    for kw in (dict(V=0), dict(T=-1), dict(K=4), dict(g=None), dict(A=None), dict(B=None), dict(y=None), dict(lse=None),
               dict(dA=_vp(0x10008)), dict(dB=_vp(0x10008)), dict(work=None), dict(n=64 * 256 * 2 - 1)):
        assert bwd(**kw) == ag.AG_EINVAL, kw
    assert bwd(K=(1 << 21) + 8) == ag.AG_EUNSUPPORTED
    assert bwd(dA=None, dB=None) == ag.AG_OK


def test_xent_bwd_workspace_is_bounded_by_its_pieces():
    """The d logits held at a time stay under 512 MiB (or 256 columns) however large the vocabulary."""
    for T, V, K in ((1, 1, 8), (4096, 50257, 2048), (8192, 1 << 20, 4096), (1 << 20, 1 << 17, 1024)):
        n = ag.lib().gemm_xent_bwd_workspace(T, V, K)
        split = n - max(512 << 20, T * 256 * 2)
        assert 0 < n and split <= 64 * max(T, 1) * K * 4, (T, V, K, n)


def test_binding_refuses_before_the_library_sees_it():
    a, b = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        ag.gemm_bias_act(a, b)
    with pytest.raises(ValueError, match="A must be"):
        ag.gemm_bias_act(a.float(), b)
    with pytest.raises(ValueError, match="dimensions"):
        ag.gemm_bias_act(a[0], b)
    with pytest.raises(ValueError, match="dimensions"):
        ag.gemm_grouped(a, b, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        ag.gemm_xent(a, b, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="device tensor"):
        ag.gemm_grouped_bwd(a[:, :8].contiguous(), a, b[None], torch.zeros(1, dtype=torch.int32))
