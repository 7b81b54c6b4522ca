"""Multi-axis rotation on the GPU against the float64 oracle, and its inverse
as the gradient."""

import numpy as np
import pytest
import torch

from oracle import rcx_oracle as orc
from rope_context_extension_scaled_b200 import _lib
from tests._parity import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(B, N, Hq, Hkv, d, dtype, sections, inter, seed=0, span=1 << 20):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn(B, N, Hq, d, generator=g, device=DEV).to(dtype)
    k = torch.randn(B, N, Hkv, d, generator=g, device=DEV).to(dtype)
    pos = torch.randint(0, span, (len(sections), B, N), generator=g, device=DEV)
    inv, _ = _lib.rope_freqs(_lib.PLAIN, 5e5, d, 1, 1)
    return q, k, pos, inv, _lib.rope_axes_map(sections, inter)


def _check(x, y, pos, inv, axis, halves, inverse):
    """|error| <= angle error 5e-7 and four fp32 roundings times |pair|, plus one rounding to bf16."""
    for b in range(x.shape[0]):
        ref = orc.rope_rotate_axes(np64(x[b]), pos[:, b].cpu().numpy(), inv, axis, halves, inverse)
        mag = np.abs(np64(x[b])).max(initial=0)
        out = 2.0 ** -8 * np.abs(ref) if x.dtype == torch.bfloat16 else 0.0
        assert np.all(np.abs(np64(y[b]) - ref) <= 1.5 * mag * (5e-7 + 4 * 2.0 ** -24) + out)


@pytest.mark.parametrize("halves", [True, False])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("dtype,B,N,Hq,Hkv,d,sections,inter", [
    (torch.bfloat16, 1, 1, 1, 1, 16, [8], False), (torch.bfloat16, 3, 37, 5, 1, 64, [10, 11, 11], True),
    (torch.bfloat16, 2, 300, 40, 8, 128, [16, 24, 24], False), (torch.float32, 2, 65, 3, 2, 128, [1, 62, 1], True),
    (torch.float32, 1, 129, 7, 7, 8, [1, 1, 1, 1], False), (torch.bfloat16, 1, 700, 2, 1, 256, [100, 28], True),
    (torch.float32, 64, 1, 9, 3, 256, [128], False)])
def test_matches_oracle(dtype, B, N, Hq, Hkv, d, sections, inter, halves, inverse):
    q, k, pos, inv, axis = _inputs(B, N, Hq, Hkv, d, dtype, sections, inter)
    qo, ko = _lib.rope_axes_apply(q, k, inv, axis, pos, halves=halves, inverse=inverse, q_out=torch.empty_like(q),
                                  k_out=torch.empty_like(k))
    for x, y in ((q, qo), (k, ko)):
        _check(x, y, pos, inv, axis, halves, inverse)


def test_one_axis_equals_rope_apply():
    q, k, _, inv, axis = _inputs(2, 200, 4, 2, 128, torch.bfloat16, [64], False)
    pos = torch.arange(200, device=DEV)
    a, b = _lib.rope_apply(q, k, inv, positions=pos, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
    c, d = _lib.rope_axes_apply(q, k, inv, axis, pos.expand(1, 2, 200), q_out=torch.empty_like(q),
                                k_out=torch.empty_like(k))
    # The same angles; x c - y s may be contracted either way, fma(x, c, -fl(y s)) or fma(-y, s,
    # fl(x c)): each is within 2 * 2^-24 (|x| + |y|) of the exact value, |x| + |y| <= 2 max |q|, so the
    # two differ by at most 2^-21 max |q| before the rounding to bf16, which then falls to the same or
    # a neighbouring value: one more step, 2^-7 of the value.
    for got, want, x in ((c, a, q), (d, b, k)):
        far = (got.double() - want.double()).abs() - 2.0 ** -7 * want.double().abs()
        assert far.max() <= 2.0 ** -21 * x.abs().max().item()


@pytest.mark.parametrize("halves", [True, False])
def test_inverse_is_the_gradient(halves):
    """The rotation is linear: its derivative along e is R e, and the inverse of dy has to be R^T dy."""
    x, _, pos, inv, axis = _inputs(1, 5, 2, 1, 32, torch.float32, [9, 7], True, seed=3, span=5000)
    g = torch.Generator(device=DEV).manual_seed(4)
    dy = torch.randn(x.shape, generator=g, device=DEV)

    def rot(t, inverse=False):
        return _lib.rope_axes_apply(t, None, inv, axis, pos, halves=halves, inverse=inverse, q_out=torch.empty_like(t))[0]
    dx = rot(dy, inverse=True)
    n = x.numel()
    for i in range(0, n, 7):
        e = torch.zeros(n, device=DEV)
        e[i] = 0.5
        e = e.view_as(x)
        diff = (rot(x + e).double() - rot(x - e).double()).mul(dy.double()).sum().item()   # step 1
        # each of the two rotations: 1e-6 |pair| per component, times |dy|
        assert abs(diff - dx.flatten()[i].item()) <= 4e-6 * (1 + 2 * x.abs().max().item()) * dy.abs().max().item() * 2
    # and back: x again, within two rotations' error
    assert (rot(rot(x), inverse=True) - x).abs().max().item() <= 3e-6 * x.abs().max().item()


def test_strides_shared_positions_and_in_place():
    q, k, pos, inv, axis = _inputs(3, 50, 6, 2, 64, torch.bfloat16, [12, 20], False)
    wide = torch.zeros(3, 50, 9, 72, dtype=torch.bfloat16, device=DEV)
    wide[:, :, 2:8, :64] = q
    view = wide[:, :, 2:8, :64]
    shared = pos[:, :1].expand(2, 3, 50)                      # one row of positions for all sequences
    ref, _ = _lib.rope_axes_apply(q, None, inv, axis, pos[:, :1].repeat(1, 3, 1), halves=True, q_out=torch.empty_like(q))
    got, none = _lib.rope_axes_apply(view, None, inv, axis, shared, halves=True)
    assert none is None and got is view and torch.equal(view, ref)
    rest = wide.clone()
    rest[:, :, 2:8, :64] = 0
    assert not rest.any()                                     # nothing outside the view changed
    none, kk = _lib.rope_axes_apply(None, k, inv, axis, shared, k_out=torch.empty_like(k))
    _check(k, kk, shared, inv, axis, False, False)


def test_non_finite_values_stay_in_their_pairs():
    x, _, pos, inv, axis = _inputs(1, 3, 2, 1, 64, torch.float32, [32], False)
    y0, _ = _lib.rope_axes_apply(x, None, inv, axis, pos, q_out=torch.empty_like(x))
    x[0, 1, 1, 5] = float("nan")
    y1, _ = _lib.rope_axes_apply(x, None, inv, axis, pos, q_out=torch.empty_like(x))
    assert torch.isnan(y1[0, 1, 1, 4:6]).all()
    y1[0, 1, 1, 4:6] = y0[0, 1, 1, 4:6]
    assert torch.equal(y0, y1)


def test_captured_and_replayed_on_another_stream():
    q, k, pos, inv, axis = _inputs(4, 1, 8, 2, 128, torch.bfloat16, [20, 22, 22], True)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    _lib.rope_axes_apply(q, k, inv, axis, pos, q_out=qo, k_out=ko)     # loads the kernels
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        _lib.rope_axes_apply(q, k, inv, axis, pos, halves=True, q_out=qo, k_out=ko)
    for step in range(2):
        pos += 1 + step
        graph.replay()
        _check(q, qo, pos, inv, axis, True, False)
        _check(k, ko, pos, inv, axis, True, False)
