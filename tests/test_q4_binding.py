"""The binding's checks of tensors for the 4-bit operators, on the host: CPU
tensors that claim to be CUDA ones reach every check and no launch."""
from __future__ import annotations

import types

import pytest
import torch

import matrix_multiply_gb300 as tg


class Cuda(torch.Tensor):
    is_cuda = property(lambda self: True)


def t(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Cuda)


def parts(N=64, K=96, group=32):
    return t(N, -(-K // 32) * 16), t(-(-K // group), N, dtype=torch.float16), t(-(-K // group), N)


# a context that the library refuses: a call that passes the binding's checks
# ends in TC_ERR_NULL
NO_CTX = types.SimpleNamespace(ptr=None)


def test_rows_of_the_right_stride_pass():
    codes, scales, zeros = parts()
    assert tg.Q4Weight(64, 96, 32, codes, scales, zeros).desc.ldw == 96
    wide = t(64, 80)[:, :48]
    assert tg.Q4Weight(64, 96, 32, wide, scales, zeros).desc.ldw == 160
    # one row has no stride
    tg.Q4Weight(1, 96, 32, t(48).expand(1, 48), scales[:, :1])
    tg.Q4Weight(64, 32, 32, t(64, 16), t(64, dtype=torch.float16).expand(1, 64))


def test_rows_that_share_memory_are_refused():
    """A row stride of 0, as expand gives it, means the default pitch to the
    library, which would run past the one row there is."""
    codes, scales, zeros = parts()
    with pytest.raises(ValueError):
        tg.Q4Weight(64, 96, 32, codes, scales[:1].expand(3, 64), zeros[:1].expand(3, 64))
    with pytest.raises(ValueError):
        tg.Q4Weight(64, 96, 32, codes, scales[:1].expand(3, 64))
    with pytest.raises(ValueError):
        tg.Q4Weight(64, 96, 32, codes[:1].expand(64, 48), scales)
    with pytest.raises(ValueError):
        tg.Q4Weight(64, 96, 32, t(4096).as_strided((64, 48), (16, 1)), scales)


F32 = torch.float32


@pytest.mark.parametrize("W", [t(1, 96, dtype=F32).expand(64, 96), t(1, 1, dtype=F32).expand(64, 96),
                               t(8192, dtype=F32).as_strided((64, 96), (32, 1))])
def test_matrices_whose_rows_share_memory_are_refused(W):
    q = tg.Q4Weight(64, 96, 32, *parts())
    for call in (lambda: tg.tc_quantize_q4(NO_CTX, W, q), lambda: tg.tc_dequantize_q4(NO_CTX, q, W)):
        with pytest.raises(ValueError):
            call()


def test_a_column_whose_rows_share_memory_is_refused():
    q = tg.Q4Weight(64, 1, 32, t(64, 16), t(1, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        tg.tc_quantize_q4(NO_CTX, t(1, 1, dtype=torch.float32).expand(64, 1), q)


def test_pitches_beyond_the_descriptor_are_refused():
    """A pitch that wraps in 32 bits (here to the default) names other memory."""
    codes = types.SimpleNamespace(is_cuda=True, dim=lambda: 2, stride=lambda i: (2 ** 31, 1)[i], shape=(2, 16),
                                  dtype=torch.uint8, data_ptr=lambda: 16)
    with pytest.raises(ValueError):
        tg.Q4Weight(2, 32, 32, codes, t(1, 16, dtype=torch.float16))
    W = types.SimpleNamespace(is_cuda=True, dim=lambda: 2, stride=lambda i: (2 ** 32, 1)[i], shape=(64, 96), dtype=F32,
                              data_ptr=lambda: 16)
    with pytest.raises(ValueError):
        tg.tc_quantize_q4(NO_CTX, W, tg.Q4Weight(64, 96, 32, *parts()))


def test_matrices_of_rows_apart_reach_the_library():
    q = tg.Q4Weight(64, 96, 32, *parts())
    for W in (t(64, 96, dtype=torch.float32), t(64, 100, dtype=torch.bfloat16)[:, :96]):
        with pytest.raises(tg.TcError) as err:
            tg.tc_quantize_q4(NO_CTX, W, q)
        assert err.value.status == tg.TC_ERR_NULL


@pytest.mark.parametrize("x,c", [(torch.float32, torch.float16), (torch.bfloat16, torch.float16), (torch.uint8, torch.float16),
                                 (torch.float16, torch.bfloat16), (torch.float16, torch.float32), (torch.float16, torch.uint8)])
def test_product_of_other_types_is_refused(x, c):
    """Elements are counted, so a tensor of a narrower type than the
    descriptor's would be too short."""
    q = tg.Q4Weight(64, 96, 32, *parts())
    d = tg.make_desc(4, 64, 96, "f16", "f16", b_dtype="i4", transpose_b=True)
    stream = types.SimpleNamespace(ptr=None)
    X, C = t(4, 96, dtype=x), t(4, 64, dtype=c)
    for call in (lambda: tg.tc_gemm_q4_weight(NO_CTX, d, X, q, C),
                 lambda: tg.tc_gemm_q4_weight_async(NO_CTX, d, X, q, C, stream),
                 lambda: tg.PreparedGemm(NO_CTX, d, X, q, C, stream)):
        with pytest.raises(ValueError):
            call()
    # addresses are the caller's word, and a type the library refuses is its to report
    with pytest.raises(tg.TcError):
        tg.tc_gemm_q4_weight(NO_CTX, d, 1 << 20, q, 1 << 30)
    with pytest.raises(tg.TcError):
        tg.tc_gemm_q4_weight(NO_CTX, tg.make_desc(4, 64, 96, "i8", "f32", b_dtype="i4", transpose_b=True), X, q,
                             t(4, 64, dtype=F32))


def test_longest_rows():
    """Quantising and reading back take K up to 65535 * 1024; a longer row is
    refused as a size, not as a failed launch."""
    K = 65535 * 1024
    for k, want in ((K, tg.TC_OK), (K + 1, tg.TC_ERR_DIM)):
        q = tg.tc_q4_weight(2, k, 32, tg.TC_F16, 0, 0, 1 << 32, 1 << 40, None)
        assert tg.tc_q4_validate(q, W=1 << 50) == want
