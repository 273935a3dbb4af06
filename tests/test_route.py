"""Routing of tokens to experts on the host: every refusal and its status, and
the binding's own checks."""
from __future__ import annotations

import pytest
import torch

import matrix_multiply_gb300 as tg

T, E, K = 10, 64, 4
AT = dict(logits=1 << 40, ids=2 << 40, weights=3 << 40, counts=4 << 40, losses=5 << 40, grad_weights=6 << 40,
          grad_losses=7 << 40, dlogits=8 << 40, valid=9 << 40)


def call(back, at=None, **kw):
    kw = {"tokens": T, "experts": E, "top_k": K, "logits_dtype": "f32", **kw}
    d = tg.make_route_desc(**kw)
    a = {**AT, **(at or {})}
    names = ("valid", "ids", "counts", "grad_weights", "grad_losses", "dlogits") if back else \
        ("valid", "ids", "weights", "counts", "losses")
    fn = tg.tc_moe_route_backward_validate if back else tg.tc_moe_route_validate
    return fn(d, a["logits"], *(a[n] for n in names))


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,want", [
    ({}, tg.TC_OK), ({"logits_dtype": "bf16"}, tg.TC_OK), ({"logits_dtype": "f16", "grad_dtype": "f32"}, tg.TC_OK),
    ({"experts": 512, "top_k": 16}, tg.TC_OK), ({"experts": 1, "top_k": 1, "tokens": 1}, tg.TC_OK),
    ({"ld_logits": 65, "ld_dlogits": 70, "renormalize": False}, tg.TC_OK),
    ({"tokens": 0}, tg.TC_ERR_DIM), ({"experts": 0}, tg.TC_ERR_DIM), ({"experts": 513}, tg.TC_ERR_DIM),
    ({"top_k": 0}, tg.TC_ERR_DIM), ({"top_k": 17}, tg.TC_ERR_DIM), ({"experts": 3}, tg.TC_ERR_DIM),
    ({"logits_dtype": "i8"}, tg.TC_ERR_DTYPE), ({"logits_dtype": "f32", "grad_dtype": "bf16"}, tg.TC_ERR_DTYPE),
    ({"logits_dtype": "f16", "grad_dtype": "bf16"}, tg.TC_ERR_DTYPE),
    ({"ld_logits": 63}, tg.TC_ERR_LD), ({"ld_dlogits": -1}, tg.TC_ERR_LD),
])
def test_descriptor(back, kw, want):
    assert call(back, **kw) == want


def test_null():
    assert tg.tc_moe_route_validate(None) == tg.TC_ERR_NULL
    assert tg.tc_moe_route_backward_validate(None) == tg.TC_ERR_NULL
    for n in ("logits", "ids", "weights", "counts", "losses"):
        assert call(False, {n: 0}) == tg.TC_ERR_NULL, n
    for n in ("logits", "ids", "counts", "dlogits"):
        assert call(True, {n: 0}) == tg.TC_ERR_NULL, n
    assert call(False, {"valid": 0}) == tg.TC_OK
    for n in ("valid", "grad_weights", "grad_losses"):
        assert call(True, {n: 0}) == tg.TC_OK, n


def test_overlap():
    outs = ("ids", "weights", "counts", "losses")
    for o in outs:
        for n in ("logits", "valid") + tuple(x for x in outs if x != o):
            assert call(False, {o: AT[n]}) == tg.TC_ERR_OVERLAP, (o, n)
    assert call(False, {"losses": AT["counts"] + 4 * (E + 1)}) == tg.TC_OK
    assert call(False, {"losses": AT["counts"] + 4 * E}) == tg.TC_ERR_OVERLAP      # the count of tokens is the last
    for n in ("logits", "valid", "ids", "counts", "grad_weights", "grad_losses"):
        assert call(True, {"dlogits": AT[n]}) == tg.TC_ERR_OVERLAP, n


class FakeContext:
    ptr = None


def test_binding_refuses():
    d = tg.make_route_desc(T, E, K)
    logits, ids, counts = torch.zeros(T, E), torch.zeros(T, K, dtype=torch.int32), torch.zeros(E + 1, dtype=torch.int32)
    for kw, what in (({}, "give weights"), ({"weights": logits}, "come with"), ({"losses": logits}, "come with"),
                     ({"grad_losses": 5, "weights": 1, "losses": 2}, "come with dlogits"),
                     ({"weights": 1, "losses": 2}, "CUDA")):
        with pytest.raises(ValueError, match=what):
            tg.PreparedRoute(FakeContext(), d, logits, ids, counts, **kw)
    call = tg.PreparedRoute(FakeContext(), d, 1 << 40, 2 << 40, 3 << 40, weights=4 << 40, losses=5 << 40)
    with pytest.raises(ValueError, match="stream"):
        call.enqueue()
    with pytest.raises(ValueError, match="not prepared"):
        call.enqueue_backward()
