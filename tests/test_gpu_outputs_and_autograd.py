"""Calls that write tensors through raw pointers, beside autograd: what it has
saved counts as changed, and a tensor that gradients are wanted of is not written."""

import numpy as np
import pytest
import torch

from rope_context_extension_scaled_b200 import _lib
from tests.test_gpu_kv_block import DEV, filled, gen, lens_of

pytestmark = pytest.mark.gpu


def rope_inputs():
    x = torch.randn(1, 5, 2, 32, generator=gen(1), device=DEV)
    return x, np.ones(16), np.zeros(16, np.int32), torch.arange(5, device=DEV)[None, None]


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("axes", [True, False])
def test_rotation_in_place_is_seen_by_autograd(which, axes):
    x, inv, axis, pos = rope_inputs()
    w = torch.ones_like(x, requires_grad=True)
    y = (w * x).sum()                                          # saves x
    before = x._version
    q, k = (x, None) if which == "q" else (None, x)
    if axes:
        _lib.rope_axes_apply(q, k, inv, axis, pos)
    else:
        _lib.rope_apply(q, k, inv)
    assert x._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_rotation_of_what_requires_grad():
    x, inv, axis, pos = rope_inputs()
    x.requires_grad_()
    old = x.detach().clone()
    with pytest.raises(ValueError, match="requires grad"):
        _lib.rope_axes_apply(x, None, inv, axis, pos)
    with pytest.raises(ValueError, match="requires grad"):
        _lib.rope_axes_apply(None, x, inv, axis, pos)
    assert torch.equal(x.detach(), old)
    y, _ = _lib.rope_axes_apply(x, None, inv, axis, pos, q_out=torch.empty_like(x, requires_grad=False))
    assert not torch.equal(y, old) and torch.equal(x.detach(), old)
    with torch.no_grad():
        _lib.rope_axes_apply(x, None, inv, axis, pos)
    assert torch.equal(x.detach(), y)


def test_rotation_of_inference_tensors():
    x, inv, axis, pos = rope_inputs()
    want, _ = _lib.rope_axes_apply(x, None, inv, axis, pos, q_out=torch.empty_like(x))
    with torch.inference_mode():
        z = x.clone()
        _lib.rope_axes_apply(z, None, inv, axis, pos)
    assert torch.equal(z, want)
    with torch.inference_mode():
        z = x.clone()
    _lib.rope_axes_apply(z, None, inv, axis, pos)
    assert torch.equal(z, want)


def test_given_outputs_of_the_cache_calls():
    c = filled([40], 16, 2, 64, "int8")
    q = torch.randn(1, 1, 4, 64, generator=gen(2), device=DEV).to(torch.bfloat16)
    o, lse = torch.empty_like(q), torch.empty(1, 4, 1, device=DEV)
    k, v = (torch.empty(1, 40, 2, 64, device=DEV) for _ in range(2))
    outs = (o, lse, k, v)
    before = [x._version for x in outs]
    _lib.attn_kv_block_fwd(q, c, lens_of([39]), o=o, lse=lse)
    _lib.kv_block_read(c, lens_of([40]), 40, dtype=torch.float32, k_out=k, v_out=v)
    assert all(x._version > b for x, b in zip(outs, before))
    for x in outs:
        x.requires_grad_()
    with pytest.raises(ValueError, match="requires grad"):
        _lib.attn_kv_block_fwd(q, c, lens_of([39]), o=o)
    with pytest.raises(ValueError, match="requires grad"):
        _lib.attn_kv_block_fwd(q, c, lens_of([39]), lse=lse)
    with pytest.raises(ValueError, match="requires grad"):
        _lib.kv_block_read(c, lens_of([40]), 40, dtype=torch.float32, k_out=k, v_out=v)
    q.requires_grad_()                                         # a query that requires grad: the result has no graph
    o2, _ = _lib.attn_kv_block_fwd(q, c, lens_of([39]))
    assert torch.equal(o2, o.detach()) and not o2.requires_grad
