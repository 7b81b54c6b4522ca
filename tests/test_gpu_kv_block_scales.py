"""Attention over the block-scaled cache where scales lie far apart: O is bounded
by the values that a row sees, whatever stands in blocks that it does not see."""

import math

import numpy as np
import pytest
import torch

from oracle import rcx_oracle as orc
from rope_context_extension_scaled_b200 import _lib
from tests._parity import np64
from tests.test_gpu_kv_block import DEV, attend, filled, gen, lens_of, values

pytestmark = pytest.mark.gpu

# (heads of the group, tokens): the mma.sync kernel with one and several columns, the
# tcgen05 kernel with converters, and over tiles converted before the launch
SHAPES = [(4, 1), (8, 8), (16, 10), (16, 140)]
FEW, MANY = SHAPES[:2], SHAPES[2:]


def check_seen(c, q, o, lse, start, count, window=0, n_sink=0):
    """O and LSE against the oracle, bounded by what each row sees.

    A = the largest sum |q_i k_i| / sqrt(d) over the row's keys: logits are fp32
    sums of d exact products and a few roundings of factors, delta = (d + 8)
    2^-23 A.  A weight carries 2 delta, 2^-21 of the exponential and up to three
    half steps of fp16 (weight, V tile, V ratio), times the largest |v| of the
    row's keys; fp16's floor is 2^-25 of weights held as 2^7 p for a reference
    scale at most 2^4 above the block's own: 2^-28 a key.  O is rounded once."""
    N, Hq, d = q.shape[1:]
    o_type = 2.0 ** -8 if o.dtype == torch.bfloat16 else 2.0 ** -22
    for b in range(q.shape[0]):
        n0, n = start[b], count[b]
        og, lg = np64(o[b]), lse[b].double().cpu().numpy()
        assert np.isfinite(og).all() and not og[n:].any() and np.isneginf(lg[:, n:]).all()
        if n == 0:
            continue
        K, V = values(c, b, n0 + n)
        qq = np64(q[b, :n])
        i, j = n0 + np.arange(n)[:, None], np.arange(n0 + n)[None]
        seen = (j <= i) & ((window == 0) | (j > i - window) | (j < n_sink))
        O, L = orc.attention(qq, K, V, 1.0 / math.sqrt(d), window=window, n_sink=n_sink, q_index=n0 + np.arange(n),
                             k_index=np.arange(n0 + n))
        G = Hq // K.shape[1]
        for h in range(Hq):
            a = (np.abs(qq[:, h]) @ np.abs(K[:, h // G]).T) / math.sqrt(d)
            delta = (d + 8) * 2.0 ** -23 * np.where(seen, a, 0).max(1)
            top = np.where(seen, np.abs(V[:, h // G]).max(1)[None], 0).max(1)
            tol = top * (2 * delta + 2.0 ** -21 + 3 * 2.0 ** -11 + (n0 + n) * 2.0 ** -28)
            bad = np.abs(og[:n, h] - O[:, h]) - (o_type * np.abs(O[:, h]) + tol[:, None])
            assert bad.max() <= 0, (b, h, np.unravel_index(bad.argmax(), bad.shape), bad.max())
            far = np.abs(lg[h, :n] - L[h]) - (delta + 2.0 ** -21 + 2.0 ** -22 * np.abs(L[h]))
            assert far.max() <= 0, (b, h, far.max())


def unseen_blocks(n0, n, block, window, n_sink):
    """Blocks of a sequence's tokens that none of its rows sees."""
    first = max(0, n0 + 1 - window)
    return [j for j in range(-(-(n0 + n) // block)) if (j + 1) * block <= first and j * block >= n_sink]


def unseen_blocks(n0, n, block, window, n_sink):
    """Blocks of a sequence's tokens that none of its rows sees."""
    first = max(0, n0 + 1 - window)
    return [j for j in range(-(-(n0 + n) // block)) if (j + 1) * block <= first and j * block >= n_sink]


UNSEEN = [(16, 600, 100, 4), (32, 1000, 90, 40), (64, 600, 100, 4)]      # block, start, window, n_sink


def unseen(kind, G, N, block, start, window, n_sink, factor):
    """Windows and sinks that end inside a key tile: the scales of the tile's other blocks do not matter."""
    c = filled([start + N], block, 1, 64, kind)
    hidden = unseen_blocks(start, N, block, window, n_sink)
    assert hidden
    c.v_scale[c.table[0, hidden].long()] *= factor
    q, o, lse = attend(c, G, [start], [N], N, 64, window=window, n_sink=n_sink)
    check_seen(c, q, o, lse, [start], [N], window, n_sink)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("block,start,window,n_sink", UNSEEN)
@pytest.mark.parametrize("power", [1, 2, 10, 70])
def test_unseen_scales_over_converted_tiles(kind, block, start, window, n_sink, power):
    unseen(kind, 16, 140, block, start, window, n_sink, 2.0 ** power)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("G,N", SHAPES)
@pytest.mark.parametrize("start", [5, 3000, 40000])
@pytest.mark.parametrize("alike", [False, True])
def test_largest_scales_stay_finite(kind, G, N, start, alike):
    """Values up to 2^127 (the format's largest scales), random or all the same: their averages are finite."""
    c = filled([start + N], 64, 1, 64, kind)
    c.v_scale.fill_(2.0 ** 120 if kind == "int8" else 2.0 ** 118)
    if kind == "e4m3":
        c.v.copy_(c.v.float().clamp(-240, 240).to(c.v.dtype))
    if alike:
        c.v.copy_(torch.full(c.v.shape, 120.0, device=DEV).to(c.v.dtype))
    q, o, lse = attend(c, G, [start], [N], N, 64, out=torch.float32)
    check_seen(c, q, o, lse, [start], [N])


def later(kind, G, N, d, power):
    """The block of the last tokens has a V scale 2^power larger; the rows before do not see it."""
    block = 16
    start = 16 * 13 - max(2, N // 4)
    c = filled([start + N], block, 1, d, kind)
    late = sorted({start // block + 1, (start + N - 1) // block})
    c.v_scale[c.table[0, late].long()] *= 2.0 ** power
    q, o, lse = attend(c, G, [start], [N], N, d, out=torch.float32)
    check_seen(c, q, o, lse, [start], [N])


def rise_and_fall(kind, G, N, window, n_sink):
    """V scales from 2^-40 to 2^40 in random order, one of zero, for rows that see some of them."""
    block, start = 16, 700
    c = filled([start + N], block, 1, 64, kind, seed=2)
    row = c.table[0].long()
    e = torch.randint(-4, 5, (len(row), 1), generator=gen(8), device=DEV)
    c.v_scale[row] *= torch.exp2(10.0 * e)
    c.v_scale[row[43]] = 0
    q, o, lse = attend(c, G, [start], [N], N, 64, window=window, n_sink=n_sink, out=torch.float32)
    check_seen(c, q, o, lse, [start], [N], window, n_sink)


def behind_zero(kind, G, N):
    """Rows that see blocks of zero scale and small ones; only later rows see large ones."""
    block = 16
    start = 16 * 13 - max(2, N // 4)
    c = filled([start + N], block, 1, 64, kind)
    row = c.table[0].long()
    c.v_scale[row] *= 2.0 ** -40
    c.v_scale[row[:9]] = 0
    c.v_scale[row[(start + N - 1) // block]] = 1.0
    q, o, lse = attend(c, G, [start], [N], N, 64, out=torch.float32)
    check_seen(c, q, o, lse, [start], [N])


def no_entry(G, N):
    """Table entries of blocks that no row sees may be anything."""
    start, block, window, n_sink = 600, 16, 100, 4
    c = filled([start + N], block, 1, 64, "int8")
    q, o, lse = attend(c, G, [start], [N], N, 64, window=window, n_sink=n_sink)
    c.table[0, unseen_blocks(start, N, block, window, n_sink)] = -1
    _, o2, lse2 = attend(c, G, [start], [N], N, 64, window=window, n_sink=n_sink)      # device_status() is 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("G,N", FEW)
@pytest.mark.parametrize("block,start,window,n_sink", UNSEEN)
@pytest.mark.parametrize("power", [1, 10, 70])
def test_unseen_scales_of_few_rows(kind, G, N, block, start, window, n_sink, power):
    unseen(kind, G, N, block, start, window, n_sink, 2.0 ** power)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [10, 24, 30, 70])
def test_later_scales_of_few_rows(kind, d, power):
    later(kind, 8, 8, d, power)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("G,N", FEW)
@pytest.mark.parametrize("window,n_sink", [(0, 0), (70, 20)])
def test_scales_rise_and_fall_for_few_rows(kind, G, N, window, n_sink):
    rise_and_fall(kind, G, N, window, n_sink)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_small_scales_behind_zero_ones_for_few_rows(kind):
    behind_zero(kind, 8, 8)


@pytest.mark.parametrize("G,N", FEW)
def test_hidden_blocks_of_few_rows_need_no_entry(G, N):
    no_entry(G, N)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("block,start,window,n_sink", UNSEEN)
@pytest.mark.parametrize("power", [1, 10, 70])
def test_unseen_scales_of_many_rows(kind, block, start, window, n_sink, power):
    unseen(kind, 16, 10, block, start, window, n_sink, 2.0 ** power)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("G,N", MANY)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [10, 24, 30, 70])
def test_later_scales_of_many_rows(kind, G, N, d, power):
    later(kind, G, N, d, power)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("G,N", MANY + [(16, 60)])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (70, 20)])
def test_scales_rise_and_fall_for_many_rows(kind, G, N, window, n_sink):
    rise_and_fall(kind, G, N, window, n_sink)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("G,N", MANY)
def test_small_scales_behind_zero_ones_for_many_rows(kind, G, N):
    behind_zero(kind, G, N)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("G,N", [(16, 100), (16, 140)])
@pytest.mark.parametrize("power", [8, 40, 100])
def test_scales_that_grow_along_the_keys(kind, G, N, power):
    """From 2^-power to 2^power over 2000 tokens, the causal border inside the last tiles: the
    reference grows many times, and early rows see none of the last blocks."""
    block, start = 16, 2000
    c = filled([start + N], block, 1, 64, kind)
    row = c.table[0].long()
    c.v_scale[row] *= torch.exp2(torch.linspace(-power, power, len(row), device=DEV).round())[:, None]
    q, o, lse = attend(c, G, [start], [N], N, 64, out=torch.float32)
    check_seen(c, q, o, lse, [start], [N])


@pytest.mark.parametrize("G,N", MANY)
def test_hidden_blocks_of_many_rows_need_no_entry(G, N):
    no_entry(G, N)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("G,N", SHAPES)
def test_a_bad_block_number_reads_as_block_0(kind, G, N):
    start, block = 300, 32
    c = filled([start + N], block, 1, 64, kind)
    q = torch.randn(1, N, G, 64, generator=gen(5), device=DEV).to(torch.bfloat16)
    c.table[0, 3] = 0
    want = _lib.attn_kv_block_fwd(q, c, lens_of([start]))
    assert _lib.device_status() == 0
    for bad in (-7, c.k.shape[0], 2 ** 31 - 1):
        c.table[0, 3] = bad
        o, lse = _lib.attn_kv_block_fwd(q, c, lens_of([start]))
        assert _lib.device_status() == _lib.RCX_ERR_DEVICE_INDEX
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("G,N", SHAPES)
@pytest.mark.parametrize("start", [100, 9000])
def test_nan_scale_reaches_rows_that_give_it_no_weight(G, N, start):
    """A visible block of V scale NaN makes NaN, however small its weight (start = 9000:
    more partials than one warp of the merge loads at once)."""
    block, d = 16, 64
    c = filled([start + N], block, 1, d, "int8")
    q = torch.ones(1, N, G, d, dtype=torch.bfloat16, device=DEV)
    c.k.fill_(1)
    p = int(c.table[0, 2])
    c.k[c.table[0, :20].long() if start > 1000 else p] = -127  # logits 1024 below the others
    c.k_scale.fill_(1.0)
    o, lse = _lib.attn_kv_block_fwd(q, c, lens_of([start]))
    assert torch.isfinite(o.float()).all()
    c.v_scale[p] = float("nan")
    o2, lse2 = _lib.attn_kv_block_fwd(q, c, lens_of([start]))
    assert torch.isnan(o2).all() and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("G,N", SHAPES)
def test_one_key_takes_everything(kind, G, N):
    """Logits of 1e30 over scales far apart and zero: the winner's value, alone."""
    block, start = 16, 200
    c = filled([start + N], block, 1, 64, kind, seed=3)
    row = c.table[0].long()
    c.v_scale[row] *= torch.exp2(10.0 * torch.randint(-4, 5, (len(row), 1), generator=gen(8), device=DEV))
    c.v_scale[row[::3]] = 0
    q, o, lse = attend(c, G, [start], [N], N, 64, qscale=1e30, out=torch.float32)
    K, V = values(c, 0, start + N)
    checked = 0
    for h in range(G):
        z = np64(q[0, :, h]) @ K[:, 0].T
        for i in range(N):
            top = z[i, :start + 1 + i]
            best = int(top.argmax())
            if top[best] - np.partition(top, -2)[-2] > 1e-4 * np.abs(top[best]):   # fp32 sums cannot mistake the winner
                # three half steps of fp16 of its own value: no other key has any weight
                assert np.abs(np64(o[0, i, h]) - V[best, 0]).max() <= 3 * 2.0 ** -11 * np.abs(V[best, 0]).max()
                checked += 1
    assert checked


# ------------------------------------------------------------------ tables with room for more

@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("capacity", [1 << 20, (1 << 21) + 5000])
def test_many_rows_in_wide_tables(kind, capacity):
    """2240 rows where a table row has room for 1M tokens (the converted tiles of one
    sequence at a time fit the workspace) and for more than 2M (they do not fit)."""
    block, start, N, G = 128, [500, 90, 0], 140, 16
    c = filled([s + N for s in start], block, 1, 128, kind)
    table = torch.full((3, capacity // block), -1, dtype=torch.int32, device=DEV)
    table[:, :c.table.shape[1]] = c.table
    wide = _lib.KvBlockCache(c.k, c.v, c.k_scale, c.v_scale, table)
    count = [N, N - 1, N]
    for window, n_sink in ((0, 0), (130, 3)):
        q, o, lse = attend(wide, G, start, count, N, 128, window=window, n_sink=n_sink)
        check_seen(c, q, o, lse, start, count, window, n_sink)
