"""What the binding of the language-model operators tells autograd of the tensors it writes, without a GPU: the library's
call and the checks of devices are replaced."""
import types

import pytest
import torch

import allgather_gemm_amd as ag


@pytest.fixture
def calls(monkeypatch):
    done = []
    fake = types.SimpleNamespace(gemm_bias_act=lambda *a: done.append("linear") or 0,
                                 gemm_grouped=lambda *a: done.append("grouped") or 0)
    monkeypatch.setattr(ag, "lib", lambda: fake)
    monkeypatch.setattr(ag, "_need", lambda t, *a, **k: None if t is None else t.data_ptr())
    monkeypatch.setattr(ag, "_work", lambda *a: (None, 0))
    monkeypatch.setattr(ag, "_stream_of", lambda device: 0)
    return done


def bf16(*shape, **kw):
    return torch.zeros(*shape, dtype=torch.bfloat16, **kw)


def test_outputs_that_the_caller_gives_count_as_written(calls):
    A, B, C, pre, bias, residual = bf16(4, 8), bf16(6, 8), bf16(4, 6), bf16(4, 6), bf16(6), bf16(4, 6)
    ag.gemm_bias_act(A, B, bias=bias, act="silu", residual=residual, C=C, pre=pre)
    assert C._version == 1 and pre._version == 1
    assert A._version == B._version == bias._version == residual._version == 0
    ag.gemm_bias_act(A, B, residual=C, C=C)
    assert C._version == 2
    W, ends = bf16(2, 6, 8), torch.zeros(2, dtype=torch.int32)
    ag.gemm_grouped(A, W, ends, C=C)
    assert C._version == 3 and W._version == ends._version == 0
    assert calls == ["linear", "linear", "grouped"]


def test_a_saved_tensor_that_a_call_overwrites_is_noticed(calls):
    A, B, C = bf16(4, 8), bf16(6, 8), bf16(4, 6)
    w = bf16(4, 6, requires_grad=True)
    loss = (w * C).sum()                       # keeps C for w's gradient
    ag.gemm_bias_act(A, B, residual=C, C=C)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_outputs_of_inference_mode_are_taken(calls):
    with torch.inference_mode():
        C = bf16(4, 6)
    assert ag.gemm_bias_act(bf16(4, 8), bf16(6, 8), C=C, pre=C) is C
