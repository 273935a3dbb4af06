"""The 4-bit weight entry points on the host: every refusal and its status."""
from __future__ import annotations

import ctypes

import pytest
import torch

import matrix_multiply_gb300 as tg
import q4_ref


def weight(N=64, K=96, group=32, scale=tg.TC_F16, ldw=0, lds=0, codes=1 << 32, scales=1 << 33, zeros=None):
    return tg.tc_q4_weight(N, K, group, scale, ldw, lds, codes, scales, zeros)


@pytest.mark.parametrize("kw,want", [
    ({}, tg.TC_OK), ({"zeros": 1 << 34}, tg.TC_OK), ({"K": 1, "N": 1}, tg.TC_OK),
    ({"ldw": 128, "lds": 80, "scale": tg.TC_BF16, "group": 128}, tg.TC_OK),
    ({"codes": None}, tg.TC_ERR_NULL), ({"scales": None}, tg.TC_ERR_NULL),
    ({"N": 0}, tg.TC_ERR_DIM), ({"K": -1}, tg.TC_ERR_DIM), ({"group": 48}, tg.TC_ERR_DIM), ({"group": 0}, tg.TC_ERR_DIM),
    ({"scale": tg.TC_F32}, tg.TC_ERR_DTYPE), ({"scale": 77}, tg.TC_ERR_DTYPE),
    ({"ldw": 64}, tg.TC_ERR_LD), ({"ldw": 100}, tg.TC_ERR_LD), ({"ldw": -32}, tg.TC_ERR_LD),
    ({"lds": 48}, tg.TC_ERR_LD), ({"lds": 72}, tg.TC_ERR_LD), ({"lds": -16}, tg.TC_ERR_LD),
    ({"codes": (1 << 32) + 8}, tg.TC_ERR_ALIGN_UNSUPPORTED), ({"scales": (1 << 33) + 2}, tg.TC_ERR_ALIGN_UNSUPPORTED),
    ({"zeros": (1 << 34) + 1}, tg.TC_ERR_ALIGN_UNSUPPORTED),
    ({"scales": (1 << 32) + 16}, tg.TC_ERR_OVERLAP), ({"zeros": (1 << 33) + 16}, tg.TC_ERR_OVERLAP),
])
def test_weight_checks(kw, want):
    assert tg.tc_q4_validate(weight(**kw)) == want


def test_matrix_checks():
    q = weight()
    assert tg.tc_q4_validate(None) == tg.TC_ERR_NULL
    assert tg.tc_q4_validate(q, W=0) == tg.TC_ERR_NULL
    assert tg.tc_q4_validate(q, tg.TC_I8) == tg.TC_ERR_DTYPE
    assert tg.tc_q4_validate(q, tg.TC_F32, 95) == tg.TC_ERR_LD
    assert tg.tc_q4_validate(q, tg.TC_F32, -1) == tg.TC_ERR_LD
    assert tg.tc_q4_validate(q, tg.TC_F32, 0, (1 << 32) - 64 * 96 * 4 + 1) == tg.TC_ERR_OVERLAP
    assert tg.tc_q4_validate(q, tg.TC_F32, 0, (1 << 32) - 64 * 96 * 4) == tg.TC_OK


def desc(M=4, N=64, K=96, a="f16", c="f16", **kw):
    kw = {"b_dtype": "i4", "transpose_b": True, **kw}
    return tg.make_desc(M, N, K, a, c, **kw)


@pytest.mark.parametrize("kw,want", [
    ({}, tg.TC_OK), ({"a": "bf16", "c": "f32"}, tg.TC_OK), ({"ldb": 96}, tg.TC_OK), ({"lda": 97, "ldc": 65}, tg.TC_OK),
    ({"M": 0}, tg.TC_ERR_DIM), ({"N": 63}, tg.TC_ERR_DIM), ({"K": 95}, tg.TC_ERR_DIM),
    ({"a": "f32", "c": "f32"}, tg.TC_ERR_DTYPE), ({"c": "bf16"}, tg.TC_ERR_DTYPE), ({"b_dtype": "i8"}, tg.TC_ERR_DTYPE),
    ({"transpose_b": False}, tg.TC_ERR_LAYOUT), ({"transpose_a": True}, tg.TC_ERR_LAYOUT),
    ({"ldb": 128}, tg.TC_ERR_LD), ({"lda": 95}, tg.TC_ERR_LD), ({"ldc": 63}, tg.TC_ERR_LD),
    ({"alpha": float("inf")}, tg.TC_ERR_SCALAR), ({"beta": float("nan")}, tg.TC_ERR_SCALAR),
])
def test_product_checks(kw, want):
    assert tg.tc_gemm_q4_weight_validate(desc(**kw), weight()) == want


def test_product_overlap():
    q = weight(zeros=1 << 34)
    for c in (1 << 20, (1 << 32) + 100, (1 << 33) + 2, (1 << 34) + 5):
        assert tg.tc_gemm_q4_weight_validate(desc(), q, X=1 << 20, C=c) == tg.TC_ERR_OVERLAP
    assert tg.tc_gemm_q4_weight_validate(desc(), weight(group=31)) == tg.TC_ERR_DIM
    # the plain GEMM and the int8 product do not take the type
    assert tg.tc_gemm_validate(desc(b_dtype="i4")) == tg.TC_ERR_DTYPE
    assert tg.tc_gemm_q8_weight_validate(desc()) == tg.TC_ERR_DTYPE


def moe(T=2, H=96, I=40, E=6, k=2, x="bf16", y=None, w1=None, w2=None, validate=None, **kw):
    d = tg.make_moe_desc(T, H, I, E, k, x, y, **kw)
    w1 = w1 or weight(N=max(1, E) * 2 * max(1, I), K=max(1, H), codes=1 << 32, scales=1 << 33)
    w2 = w2 or weight(N=max(1, E) * max(1, H), K=max(1, I), codes=1 << 35, scales=1 << 36)
    return tg.tc_moe_q4_validate(d, w1, w2, **(validate or {}))


@pytest.mark.parametrize("kw,want", [
    ({}, tg.TC_OK), ({"T": 32, "k": 6, "router_dtype": "bf16", "y": "f32"}, tg.TC_OK), ({"ldx": 97, "ldy": 101}, tg.TC_OK),
    ({"T": 0}, tg.TC_ERR_DIM), ({"T": 33}, tg.TC_ERR_DIM), ({"H": 0}, tg.TC_ERR_DIM), ({"I": 0}, tg.TC_ERR_DIM),
    ({"E": 0}, tg.TC_ERR_DIM), ({"E": 513}, tg.TC_ERR_DIM), ({"k": 0}, tg.TC_ERR_DIM), ({"k": 7}, tg.TC_ERR_DIM),
    ({"E": 40, "k": 17}, tg.TC_ERR_DIM),
    ({"w1": weight(N=481, K=96)}, tg.TC_ERR_DIM), ({"w1": weight(N=480, K=97)}, tg.TC_ERR_DIM),
    ({"w2": weight(N=577, K=40)}, tg.TC_ERR_DIM), ({"w2": weight(N=576, K=41)}, tg.TC_ERR_DIM),
    ({"w1": weight(N=480, K=96, group=64)}, tg.TC_ERR_DIM), ({"w2": weight(N=576, K=40, scale=tg.TC_BF16)}, tg.TC_ERR_DTYPE),
    ({"w1": weight(N=480, K=96, group=16)}, tg.TC_ERR_DIM), ({"w2": weight(N=576, K=40, ldw=48)}, tg.TC_ERR_LD),
    ({"x": "f32"}, tg.TC_ERR_DTYPE), ({"y": "f16"}, tg.TC_ERR_DTYPE), ({"router_dtype": "f16"}, tg.TC_ERR_DTYPE),
    ({"ldx": 95}, tg.TC_ERR_LD), ({"ld_router": 95}, tg.TC_ERR_LD), ({"ldy": -1}, tg.TC_ERR_LD),
    ({"validate": {"Y": 1 << 20}}, tg.TC_ERR_OVERLAP), ({"validate": {"Y": (1 << 30) + 4}}, tg.TC_ERR_OVERLAP),
    ({"validate": {"Y": (1 << 35) + 4}}, tg.TC_ERR_OVERLAP), ({"validate": {"ids": 3 << 40}}, tg.TC_ERR_OVERLAP),
    ({"validate": {"ids": 1 << 41, "weights": (1 << 41) + 8}}, tg.TC_ERR_OVERLAP),
    ({"validate": {"ids": 1 << 41, "weights": (1 << 41) + 16}}, tg.TC_OK),
    ({"validate": {"weights": (1 << 32) + 16}}, tg.TC_ERR_OVERLAP),
    ({"validate": {"X": 0}}, tg.TC_ERR_NULL), ({"validate": {"router": 0}}, tg.TC_ERR_NULL),
    ({"validate": {"Y": 0}}, tg.TC_ERR_NULL),
])
def test_moe_checks(kw, want):
    assert moe(**kw) == want


def test_null_structures():
    lib = tg.library()
    d, q = desc(), weight()
    assert lib.tc_gemm_q4_weight_validate(None, ctypes.byref(q), 1, 2) == tg.TC_ERR_NULL
    assert lib.tc_gemm_q4_weight_validate(ctypes.byref(d), None, 1, 2) == tg.TC_ERR_NULL
    assert lib.tc_gemm_q4_weight(None, ctypes.byref(d), ctypes.byref(q), 1, 2) == tg.TC_ERR_NULL
    assert lib.tc_quantize_q4(None, 1, 0, 1, ctypes.byref(q)) == tg.TC_ERR_NULL
    assert lib.tc_dequantize_q4(None, ctypes.byref(q), 1, 0, 1) == tg.TC_ERR_NULL
    assert lib.tc_moe_q4(None, None, 1, 1, None, None, 1, None, None) == tg.TC_ERR_NULL


def test_binding_checks_tensors():
    """Q4Weight takes CUDA tensors of the right types only."""
    codes, scales = torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(1, 16, dtype=torch.float16)
    with pytest.raises(ValueError):
        tg.Q4Weight(8, 32, 32, codes, scales)
    with pytest.raises(ValueError):
        tg.Q4Weight.empty(0, 32, 32)


@pytest.mark.parametrize("K", [1, 7, 8, 31, 32, 100])
def test_reference_packing_inverts(K):
    code = torch.randint(0, 16, (5, K), dtype=torch.uint8)
    assert torch.equal(q4_ref.unpack(q4_ref.pack(code, q4_ref.up(K, 32)), K), code)
    # elements 0 and 1 of a word in the low and high halves of a masked register
    b = q4_ref.pack(torch.arange(8, dtype=torch.uint8)[None], 32)[0, :4].to(torch.int64)
    word = int(b[0] + (b[1] << 8) + (b[2] << 16) + (b[3] << 24))
    for i in range(4):
        assert (word >> (4 * i)) & 0x000F000F == (2 * i) | ((2 * i + 1) << 16)
