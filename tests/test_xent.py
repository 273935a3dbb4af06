"""Softmax cross entropy against a vocabulary on the host: every refusal and its
status, and the binding's own checks."""
from __future__ import annotations

import pytest
import torch

import matrix_multiply_gb300 as tg

T, H, V = 10, 64, 1000
AT = dict(X=1 << 20, W=1 << 40, targets=2 << 40, loss=3 << 40, lse=4 << 40, grad=5 << 40, dX=6 << 40, dW=7 << 40)


def forward(at=None, **kw):
    a = {**AT, **(at or {})}
    kw = {"tokens": T, "hidden": H, "vocab": V, "dtype": "bf16", **kw}
    return tg.tc_linear_xent_validate(tg.make_xent_desc(**kw), *(a[k] for k in ("X", "W", "targets", "loss", "lse")))


def backward(at=None, **kw):
    a = {**AT, **(at or {})}
    kw = {"tokens": T, "hidden": H, "vocab": V, "dtype": "bf16", **kw}
    return tg.tc_linear_xent_backward_validate(tg.make_xent_desc(**kw),
                                               *(a[k] for k in ("X", "W", "targets", "lse", "grad", "dX", "dW")))


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("kw,want", [
    ({}, tg.TC_OK), ({"dtype": "f16"}, tg.TC_OK), ({"grad_dtype": "f32"}, tg.TC_OK), ({"target_dtype": "i32"}, tg.TC_OK),
    ({"reduction": "none"}, tg.TC_OK), ({"reduction": "sum"}, tg.TC_OK), ({"tokens": 1, "hidden": 1, "vocab": 1}, tg.TC_OK),
    ({"ldx": 65, "ldw": 64, "lddx": 70, "lddw": 66}, tg.TC_OK), ({"z_weight": 1.0, "scale": 1e-6}, tg.TC_OK),
    ({"tokens": 0}, tg.TC_ERR_DIM), ({"hidden": -1}, tg.TC_ERR_DIM), ({"vocab": 0}, tg.TC_ERR_DIM),
    ({"dtype": "f32"}, tg.TC_ERR_DTYPE), ({"dtype": 99}, tg.TC_ERR_DTYPE), ({"grad_dtype": "f16"}, tg.TC_ERR_DTYPE),
    ({"target_dtype": "f32"}, tg.TC_ERR_DTYPE), ({"target_dtype": "i8"}, tg.TC_ERR_DTYPE),
    ({"reduction": 3}, tg.TC_ERR_EPILOGUE), ({"reduction": -1}, tg.TC_ERR_EPILOGUE),
    ({"ldx": 63}, tg.TC_ERR_LD), ({"ldw": -64}, tg.TC_ERR_LD), ({"lddx": 1}, tg.TC_ERR_LD), ({"lddw": 63}, tg.TC_ERR_LD),
    ({"scale": 0.0}, tg.TC_ERR_SCALAR), ({"scale": -1.0}, tg.TC_ERR_SCALAR), ({"scale": float("inf")}, tg.TC_ERR_SCALAR),
    ({"z_weight": -1e-9}, tg.TC_ERR_SCALAR), ({"z_weight": float("nan")}, tg.TC_ERR_SCALAR),
    ({"tokens": 2 ** 31 - 1, "vocab": 2 ** 31 - 1, "hidden": 1}, tg.TC_ERR_OVERFLOW),
])
def test_descriptor(call, kw, want):
    assert call(**kw) == want


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("dim", ["tokens", "hidden", "vocab"])
def test_largest(call, dim):
    """32 bits hold a dimension, its last partial tile included."""
    sizes = {"tokens": 1, "hidden": 1, "vocab": 1}
    at = {k: i << 50 for i, k in enumerate(AT, 1)}
    assert call(at, **{**sizes, dim: 2 ** 31 - 4097}) == tg.TC_OK
    for n in (2 ** 31 - 4096, 2 ** 31 - 1):
        assert call(at, **{**sizes, dim: n}) == tg.TC_ERR_OVERFLOW


def test_null():
    assert tg.tc_linear_xent_validate(None) == tg.TC_ERR_NULL
    assert tg.tc_linear_xent_backward_validate(None) == tg.TC_ERR_NULL
    for k in ("X", "W", "targets", "loss", "lse"):
        assert forward({k: 0}) == tg.TC_ERR_NULL, k
    for k in ("X", "W", "targets", "lse", "grad"):
        assert backward({k: 0}) == tg.TC_ERR_NULL, k
    assert backward({"dX": 0}) == tg.TC_OK and backward({"dW": 0}) == tg.TC_OK
    assert backward({"dX": 0, "dW": 0}) == tg.TC_ERR_NULL


def test_overlap():
    end = AT["X"] + T * H * 2
    assert forward({"lse": end}) == tg.TC_OK and forward({"lse": end - 4}) == tg.TC_ERR_OVERLAP
    assert forward({"loss": AT["W"]}) == tg.TC_ERR_OVERLAP
    assert forward({"loss": AT["targets"] + 8 * T - 4}) == tg.TC_ERR_OVERLAP
    assert forward({"loss": AT["lse"] + 4 * T - 4}) == tg.TC_ERR_OVERLAP
    assert forward({"loss": AT["lse"] - 4}) == tg.TC_OK                       # one float where reduced
    assert forward({"loss": AT["lse"] - 4}, reduction="none") == tg.TC_ERR_OVERLAP
    for k in ("X", "W", "targets", "lse", "grad", "dW"):
        assert backward({"dX": AT[k]}) == tg.TC_ERR_OVERLAP, k
    assert backward({"dX": AT["dW"] - T * H * 2}) == tg.TC_OK
    assert backward({"dX": AT["dW"] - T * H * 2}, grad_dtype="f32") == tg.TC_ERR_OVERLAP
    assert backward({"dW": AT["W"] + V * H * 2 - 2}) == tg.TC_ERR_OVERLAP


class FakeContext:
    ptr = None


def prepared(**kw):
    """The binding's checks run before any call: on host tensors they refuse the first."""
    a = dict(X=torch.zeros(T, H, dtype=torch.bfloat16), W=torch.zeros(V, H, dtype=torch.bfloat16),
             targets=torch.zeros(T, dtype=torch.int64), lse=torch.zeros(T))
    extra = {k: kw.pop(k) for k in list(kw) if k in ("loss", "grad", "dX", "dW")}
    a.update(kw)
    return tg.PreparedXent(FakeContext(), tg.make_xent_desc(T, H, V, "bf16"), a["X"], a["W"], a["targets"], a["lse"],
                           **extra)


def test_binding_refuses():
    with pytest.raises(ValueError, match="CUDA"):
        prepared(loss=torch.zeros(1))
    with pytest.raises(ValueError, match="give loss"):
        prepared()
    with pytest.raises(ValueError, match="grad comes with"):
        prepared(loss=torch.zeros(1), dX=torch.zeros(T, H))
    with pytest.raises(ValueError, match="grad comes with"):
        prepared(grad=torch.zeros(1))


def test_binding_without_a_stream_or_half():
    call = tg.PreparedXent(FakeContext(), tg.make_xent_desc(T, H, V, "bf16"), 1 << 20, 1 << 40, 2 << 40, 3 << 40, loss=4 << 40)
    with pytest.raises(ValueError, match="stream"):
        call.enqueue()
    with pytest.raises(ValueError, match="not prepared"):
        call.enqueue_backward()
