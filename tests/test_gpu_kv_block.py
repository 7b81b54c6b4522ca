"""Block-scaled 8-bit paged KV cache on the GPU: append and read bit for bit
against the oracle's rule, attention over the cache against the float64 oracle
over code * scale, and the calls together as a serving loop makes them."""

import math

import numpy as np
import pytest
import torch

from oracle import rcx_oracle as orc
from rope_context_extension_scaled_b200 import _lib
from tests._parity import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def table_of(lens, block, width, n_blocks, seed=0):
    """A table with shuffled blocks for sequences of `lens` tokens, -1 elsewhere."""
    order = np.random.default_rng(seed).permutation(n_blocks)
    t, at = np.full((len(lens), width), -1, dtype=np.int32), 0
    for b, n in enumerate(lens):
        m = -(-n // block)
        t[b, :m] = order[at:at + m]
        at += m
    assert at <= n_blocks
    return torch.from_numpy(t).to(DEV)


def pools(n_blocks, block, Hkv, d, kind, seed, tokens_first=False, spread=0.3):
    """Random codes and scales; a block of zero scale among them."""
    g = gen(seed)
    shape = (n_blocks, block, Hkv, d) if tokens_first else (n_blocks, Hkv, block, d)
    if kind == "int8":
        k, v = (torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8) for _ in range(2))
        unit = 1.0 / 73
    else:
        k, v = (torch.randn(shape, generator=g, device=DEV).mul(100).clamp(-448, 448).to(CODES[kind]) for _ in range(2))
        unit = 1.0 / 100
    if not tokens_first:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    ks, vs = (unit * torch.exp(spread * torch.randn(n_blocks, Hkv, generator=g, device=DEV)) for _ in range(2))
    if kind == "e4m3":
        ks, vs = (torch.exp2(torch.log2(s).round()) for s in (ks, vs))
    return k, v, ks.contiguous(), vs.contiguous()


def filled(lens, block, Hkv, d, kind, seed=1, extra=2, **kw):
    """A cache handle whose sequences have room for `lens` tokens, and its table on the host."""
    width = max(1, -(-max(lens) // block))
    n_blocks = sum(-(-n // block) for n in lens) + extra
    t = table_of(lens, block, width, n_blocks, seed)
    return _lib.KvBlockCache(*pools(n_blocks, block, Hkv, d, kind, seed, **kw), t)


def values(c, b, n):
    """K, V [n, Hkv, d] of sequence b in float64."""
    row = c.table[b].long()
    block = c.k.shape[1]
    j = torch.arange(n, device=DEV)
    p = row[j // block]
    return tuple((codes[p, j % block].double() * scale[p].double()[:, :, None]).cpu().numpy()
                 for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)))


def lens_of(xs):
    return torch.tensor(xs, dtype=torch.int64, device=DEV)


def check_attention(c, q, o, lse, start, count, window=0, n_sink=0, t=1.0):
    """O and LSE against the oracle, with bounds from the roundings on the way.

    A = the largest sum |q_i k_i| / (sqrt(d) t): the logits are fp32 sums of d
    exact products (2^-23 A each) and four roundings of factors, so delta =
    (d + 8) 2^-23 A.  A weight then carries 2 delta relative error, 2^-21 from
    the exponential, and up to three half steps of fp16 (weight, V tile, V
    ratio; 2^-11 each) plus fp16's floor, 2^-25 / 2^7 a key; all times max |v|.
    O is rounded once to its type; LSE sees delta, 2^-21 and its own rounding."""
    N, Hq, d = q.shape[1:]
    o_type = 2.0 ** -8 if o.dtype == torch.bfloat16 else 2.0 ** -22
    for b in range(q.shape[0]):
        n0, n = start[b], count[b]
        og, lg = np64(o[b]), lse[b].double().cpu().numpy()
        assert not og[n:].any() and np.isneginf(lg[:, n:]).all()
        if n == 0:
            continue
        K, V = values(c, b, n0 + n)
        qq = np64(q[b, :n])
        O, L = orc.attention(qq, K, V, 1.0 / (math.sqrt(d) * t), window=window, n_sink=n_sink,
                             q_index=n0 + np.arange(n), k_index=np.arange(n0 + n))
        G = Hq // K.shape[1]
        A = max(float((np.abs(qq[:, h]) @ np.abs(K[:, h // G]).T).max()) for h in range(Hq)) / (math.sqrt(d) * t)
        delta = (d + 8) * 2.0 ** -23 * A
        tol = np.abs(V).max() * (2 * delta + 2.0 ** -21 + 3 * 2.0 ** -11 + (n0 + n) * 2.0 ** -32)
        bad = np.abs(og[:n] - O) - (o_type * np.abs(O) + tol)
        assert bad.max() <= 0, (b, bad.max(), tol)
        far = np.abs(lg[:, :n] - L) - (delta + 2.0 ** -21 + 2.0 ** -22 * np.abs(L))
        assert far.max() <= 0, (b, far.max(), delta)


def attend(c, Hq, start, count, N, d, seed=5, window=0, n_sink=0, t=1.0, out=None, qscale=1.0, with_count=True):
    q = (qscale * torch.randn(len(start), N, Hq, d, generator=gen(seed), device=DEV)).to(torch.bfloat16)
    o = None if out is None else torch.full(q.shape, 7.0, dtype=out, device=DEV)
    o, lse = _lib.attn_kv_block_fwd(q, c, lens_of(start), lens_of(count) if with_count else None, o=o, window=window,
                                    n_sink=n_sink, temperature=t)
    assert _lib.device_status() == 0
    return q, o, lse


# ------------------------------------------------------------------ append, read

@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block,d,Hkv,tokens_first", [(16, 64, 1, False), (16, 128, 3, True), (32, 64, 2, False),
                                                      (64, 128, 2, True), (128, 128, 1, False), (128, 64, 2, False)])
def test_append_and_read_equal_the_rule(kind, dtype, block, d, Hkv, tokens_first):
    start, count, N = [0, 5, block - 1, block, 3 * block + 7, 2], [1, 0, 2, block, 2 * block + 1, 11], 2 * block + 1
    lens = [a + b for a, b in zip(start, count)]
    c = filled(lens, block, Hkv, d, kind, tokens_first=tokens_first)
    g = gen(3)
    k, v = (torch.randn(6, N, Hkv, d, generator=g, device=DEV).mul(torch.exp(torch.randn(6, N, 1, 1, generator=g, device=DEV)))
            .to(dtype) for _ in range(2))
    k[3, :, 0] = 0                                             # a block of zeros
    k[4, :4] *= 1e-3                                           # joins a block of larger scale
    if kind == "int8":
        v[0, 0, 0, :5] = torch.tensor([127.0, 2.5, -2.5, 3.5, -126.5]).to(dtype)   # ties at scale 1
        v[0, 0, 0, 5:] = 0.5
    before = [x.clone() for x in (c.k.float(), c.v.float(), c.k_scale, c.v_scale)]
    ref = [[x[:, :, h].double().cpu().numpy() if x.dim() == 4 else x[:, h].double().cpu().numpy() for h in range(Hkv)]
           for x in before]
    _lib.kv_block_append(k, v, c, lens_of(start), lens_of(count))
    assert _lib.device_status() == 0
    rows = c.table.cpu().numpy()
    for i, x in enumerate((k, v)):
        for h in range(Hkv):
            for b in range(6):
                orc.kv_block_append(ref[i][h], ref[2 + i][h], rows[b], np64(x[b, :count[b], h]), start[b], kind)
    # every block of the pool, those that no token fell into among them
    for i, (codes, scale) in enumerate(((c.k, c.k_scale), (c.v, c.v_scale))):
        assert np.array_equal(codes.float().cpu().numpy(), np.stack(ref[i], axis=2))
        assert np.array_equal(scale.cpu().numpy(), np.stack(ref[2 + i], axis=1).astype(np.float32))
    n = max(lens) + 3
    for out in (torch.bfloat16, torch.float32):
        kk, vv = _lib.kv_block_read(c, lens_of(lens), n, dtype=out)
        assert _lib.device_status() == 0
        for b in range(6):
            for y, full in zip((kk, vv), values(c, b, lens[b])):
                want = torch.from_numpy(full).float().to(out)          # code * scale in fp32, then the type
                assert torch.equal(y[b, :lens[b]].cpu(), want) and not y[b, lens[b]:].any()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_token_by_token_grows_like_the_rule(kind):
    block, d = 16, 64
    c = filled([40], block, 1, d, kind)
    g = gen(9)
    x = torch.randn(1, 40, 1, d, generator=g, device=DEV) * torch.linspace(0.01, 5, 40, device=DEV)[None, :, None, None]
    ref, sc = c.k[:, :, 0].double().cpu().numpy(), c.k_scale[:, 0].double().cpu().numpy()
    row = c.table[0].cpu().numpy()
    for t in range(40):
        _lib.kv_block_append(x[:, t:t + 1], x[:, t:t + 1], c, lens_of([t]))
        orc.kv_block_append(ref, sc, row, np64(x[0, t:t + 1, 0]), t, kind)
    assert np.array_equal(c.k[:, :, 0].float().cpu().numpy(), ref) and np.array_equal(c.k_scale[:, 0].cpu().numpy(), sc)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_extreme_and_non_finite_values(kind):
    c = filled([16] * 6, 16, 1, 64, kind)
    x = torch.randn(6, 16, 1, 64, generator=gen(2), device=DEV)
    x[0] *= 1e-42                                              # subnormal: the smallest scale
    x[1] *= 1e37
    x[2, 3, 0, 7] = float("nan")
    x[3, 3, 0, 7] = float("-inf")
    x[4, 1] *= 1e-30                                           # tiny beside large
    _lib.kv_block_append(x, x, c, lens_of([0] * 6))
    k, v = _lib.kv_block_read(c, lens_of([16] * 6), 16, dtype=torch.float32)
    assert torch.equal(k.nan_to_num(9e9), v.nan_to_num(9e9))
    assert torch.isnan(k[2:4]).all() and torch.isfinite(k[[0, 1, 4, 5]]).all()
    for b in (0, 1, 4, 5):
        s = orc.kv_block_scale(float(np.float32(x[b].abs().max().item())), kind)
        want = orc.kv_code_values(np64(x[b]) * float(np.float32(1 / s)), kind) * s
        assert np.array_equal(np64(k[b]), want.astype(np.float32).astype(np.float64))
    # a later token does not hide it; a block that starts again is clean
    y = torch.randn(6, 1, 1, 64, generator=gen(3), device=DEV)
    _lib.kv_block_append(y, y, c, lens_of([15] * 6))
    assert torch.isnan(_lib.kv_block_read(c, lens_of([16] * 6), 16)[0][2:4]).all()
    _lib.kv_block_append(y, y, c, lens_of([0] * 6))
    assert torch.isfinite(_lib.kv_block_read(c, lens_of([1] * 6), 1)[0]).all()


def test_bad_lengths_and_blocks_are_reported_and_followed_nowhere():
    block, d = 16, 64
    lens = [20, 20, 20, 20]
    c = filled(lens, block, 2, d, "int8", extra=4)
    c.table[1, 1] = c.k.shape[0]                               # one past the pool
    c.table[2, 0] = -1
    x = torch.randn(4, 2, 2, d, generator=gen(1), device=DEV)
    k0, s0 = c.k.clone(), c.k_scale.clone()
    _lib.kv_block_append(x, x, c, lens_of([18, 18, 0, 31]))    # the last would end at token 33 of 32
    assert _lib.device_status() == _lib.RCX_ERR_DEVICE_INDEX and _lib.device_status() == 0
    p = int(c.table[0, 1])
    changed = (c.k != k0).flatten(1).any(1) | (c.k_scale != s0).any(1)
    assert changed.nonzero().flatten().tolist() == [p]
    k, _ = _lib.kv_block_read(c, lens_of([20, 20, 20, -1]), 20)
    assert _lib.device_status() == _lib.RCX_ERR_DEVICE_INDEX
    good, _ = values(c, 0, 20)
    assert torch.equal(k[0].cpu(), torch.from_numpy(good).float().to(torch.bfloat16))
    assert not k[1, 16:].any() and not k[2, :16].any() and not k[3].any() and k[1, :16].any() and k[2, 16:].any()
    for N in (1, 60):                                          # both attention kernels
        q = torch.randn(4, N, 2, d, generator=gen(2), device=DEV).to(torch.bfloat16)
        n = min(N, 19)
        o, lse = _lib.attn_kv_block_fwd(q[:, :n], c, lens_of([20 - n, 20 - n, 20 - n, -5])) if N == 1 else \
            _lib.attn_kv_block_fwd(q[:, :32].repeat_interleave(2, 2).repeat_interleave(8, 2), c,
                                   lens_of([0, 0, 0, 4]), lens_of([20, 20, 20, 40]))
        assert _lib.device_status() == _lib.RCX_ERR_DEVICE_INDEX
        assert not o[3].any() and torch.isneginf(lse[3]).all() and torch.isfinite(o.float()).all()


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("block,d,Hq,Hkv,start", [
    (16, 128, 8, 1, [0, 1, 15, 16, 31, 32, 33, 500]), (64, 64, 6, 2, [0, 63, 64, 127, 128, 1000]),
    (32, 128, 3, 3, [7, 2000]), (128, 128, 28, 4, [300, 0, 0, 5000]), (16, 64, 32, 1, [777, 20]),
    (64, 128, 15, 1, [129])])
def test_single_tokens(kind, block, d, Hq, Hkv, start):
    c = filled([s + 1 for s in start], block, Hkv, d, kind)
    q, o, lse = attend(c, Hq, start, [1] * len(start), 1, d, with_count=False)
    check_attention(c, q, o, lse, start, [1] * len(start))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("block,d,Hq,Hkv,N,start,count", [
    (16, 128, 8, 2, 8, [0, 40, 3, 900], [8, 0, 5, 8]),          # 32 rows: one item of the one kernel
    (16, 128, 11, 1, 3, [0, 40, 3, 900], [3, 0, 1, 3]),         # 33: two
    (16, 128, 32, 2, 4, [0, 1000], [4, 3]), (64, 64, 5, 1, 13, [50, 0], [13, 12]),    # 64, and 65: the other kernel
    (32, 64, 8, 1, 16, [5, 0], [16, 9]), (32, 64, 43, 1, 3, [130, 2], [3, 2]),     # 128 and 129 rows
    (64, 128, 4, 1, 64, [64, 0, 1], [64, 33, 0]), (128, 64, 7, 1, 37, [1, 200], [37, 37]),   # 256 and 259
    (128, 128, 3, 3, 300, [0, 511], [300, 299]), (16, 64, 2, 1, 700, [0], [700]),
    (64, 128, 1, 1, 33, [0, 4000], [33, 1])])
def test_drafts_and_chunks(kind, block, d, Hq, Hkv, N, start, count):
    c = filled([a + b for a, b in zip(start, count)], block, Hkv, d, kind, extra=1)
    if N > c.table.shape[1] * block:
        pytest.fail("case")
    q, o, lse = attend(c, Hq, start, count, N, d)
    check_attention(c, q, o, lse, start, count)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("block,d,Hq,Hkv,N,start,count,window,n_sink", [
    (16, 64, 48, 2, 86, [0, 300, 7], [86, 50, 0], 0, 0),        # 2064 rows: tiles converted before the launch
    (64, 128, 16, 1, 140, [500, 0], [140, 139], 100, 40),
    (128, 128, 16, 1, 128, [129, 1000], [128, 1], 0, 0),        # 2048, the first of them
    (32, 64, 17, 1, 150, [2000], [150], 700, 0)])
def test_many_rows_over_converted_tiles(kind, block, d, Hq, Hkv, N, start, count, window, n_sink):
    c = filled([a + b for a, b in zip(start, count)], block, Hkv, d, kind, extra=1, spread=1.0)
    row = c.table[len(start) - 1 if count[-1] else 0].long()
    c.v_scale[row[:1]] = 0
    for out in (None, torch.float32):
        q, o, lse = attend(c, Hq, start, count, N, d, window=window, n_sink=n_sink, out=out)
        check_attention(c, q, o, lse, start, count, window, n_sink)


def test_nan_scale_over_converted_tiles():
    start, N, G = 60, 140, 16
    c = filled([start + N], 16, 1, 64, "e4m3")
    q, o, lse = attend(c, G, [start], [N], N, 64)
    c.v_scale[int(c.table[0, 96 // 16])] = float("nan")         # tokens 96 .. 111
    _, o2, lse2 = attend(c, G, [start], [N], N, 64)
    assert torch.isnan(o2[:, 36:]).all() and torch.equal(lse, lse2)
    # the other rows: V tiles relative to another scale at most, two roundings of fp16 each
    far = (o2[:, :36].double() - o[:, :36].double()).abs() - 2.0 ** -7 * o[:, :36].double().abs()
    assert far.max() <= 6 * 2.0 ** -11 * np.abs(values(c, 0, 96)[1]).max()


@pytest.mark.parametrize("N,Hq", [(1, 4), (4, 8), (50, 8)])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (16, 4), (100, 33), (129, 0), (5000, 7), (200, 10 ** 12), (2 ** 40, 3)])
def test_windows_and_sinks(N, Hq, window, n_sink):
    start = [0, 10, 700, 333]
    c = filled([s + N for s in start], 32, 1, 64, "int8")
    q, o, lse = attend(c, Hq, start, [N] * 4, N, 64, window=window, n_sink=n_sink, t=1.3)
    check_attention(c, q, o, lse, start, [N] * 4, window, n_sink, 1.3)


@pytest.mark.parametrize("N", [1, 70])
def test_fp32_output_and_lse_left_out(N):
    c = filled([400 + N], 64, 2, 128, "e4m3")
    q, o, lse = attend(c, 4, [400], [N], N, 128, out=torch.float32)
    check_attention(c, q, o, lse, [400], [N])
    o2, none = _lib.attn_kv_block_fwd(q, c, lens_of([400]), o=torch.empty_like(o), want_lse=False)
    assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("N", [1, 80])
def test_scales_far_apart(kind, N):
    """Blocks whose V scales rise and fall by 2^12 along the sequence, and a zero-scale block."""
    c = filled([600 + N], 16, 1, 128, kind)
    row = c.table[0].long()
    steps = torch.arange(len(row), device=DEV)
    c.v_scale[row] = torch.exp2(((steps * 5) % 13).float() - 12)[:, None] * c.v_scale[row]
    c.v_scale[row[:2]] = 0
    c.k_scale[row[7]] = 0
    q, o, lse = attend(c, 4, [600], [N], N, 128)
    check_attention(c, q, o, lse, [600], [N])


@pytest.mark.parametrize("N", [1, 64])
@pytest.mark.parametrize("qscale", [0.0, 1e-30, 40.0, 1e30])
def test_query_sizes(N, qscale):
    """From no query at all to one key taking everything (logits of 1e30 still order like exact ones)."""
    c = filled([200 + N], 32, 1, 64, "int8")
    q, o, lse = attend(c, 2, [200], [N], N, 64, qscale=qscale)
    if qscale <= 40:
        check_attention(c, q, o, lse, [200], [N])
    else:
        K, V = values(c, 0, 200 + N)
        for h in range(2):
            z = np64(q[0, :, h]) @ K[:, 0].T
            for i in range(N):
                top = z[i, :201 + i]
                best = top.argmax()
                gap = top[best] - np.partition(top, -2)[-2]
                if gap > 1e-4 * np.abs(top[best]):              # fp32 sums cannot mistake the winner
                    assert np.abs(np64(o[0, i, h]) - V[best, 0]).max() <= (2.0 ** -8 + 3 * 2.0 ** -11) * np.abs(V).max()


@pytest.mark.parametrize("N,G", [(1, 4), (40, 4)])
def test_unseen_places_do_not_matter(N, G):
    """Garbage behind the sequences, in other blocks and in scales that no row sees; NaN where one row sees it."""
    start = [30, 100, 250]
    c = filled([s + N for s in start], 64, 1, 64, "e4m3", extra=3)
    q, o, lse = attend(c, G, start, [N] * 3, N, 64, window=20)
    used = set(c.table.flatten().tolist())
    for p in set(range(c.k.shape[0])) - used:
        c.k_scale[p] = c.v_scale[p] = float("nan")
    bits = c.k.view(torch.uint8), c.v.view(torch.uint8)
    for b, s in enumerate(start):
        last = int(c.table[b, (s + N - 1) // 64])
        for x in bits:
            x[last, (s + N - 1) % 64 + 1:] = 0x7f              # rows behind the sequence: NaN codes
    first = int(c.table[2, 0])                                 # tokens 0 .. 63 of sequence 2: outside every window
    c.k_scale[first] = float("inf")
    c.v_scale[first] = float("nan")
    for x in bits:
        x[first] = 0x7f
    q2, o2, lse2 = attend(c, G, start, [N] * 3, N, 64, window=20)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("N,G", [(4, 4), (40, 4)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_scale_reaches_exactly_the_rows_that_see_it(N, G, which):
    start, block = 126, 16
    c = filled([start + N], block, 1, 64, "int8")
    q, o, lse = attend(c, G, [start], [N], N, 64)
    p = int(c.table[0, 128 // block])                          # tokens 128 .. 143
    (c.k_scale if which == "k" else c.v_scale)[p] = float("nan")
    _, o2, lse2 = attend(c, G, [start], [N], N, 64)
    assert torch.equal(o[:, :2], o2[:, :2]) and torch.isnan(o2[:, 2:]).all()
    assert torch.equal(lse[:, :, :2], lse2[:, :, :2])
    assert torch.isnan(lse2[:, :, 2:]).all() if which == "k" else torch.equal(lse, lse2)


@pytest.mark.parametrize("N", [1, 40])
def test_strides_layouts_and_shared_blocks(N):
    """Q, O and LSE views, both pool layouts, and two sequences that share their first blocks."""
    start, block, d = [200, 140], 32, 64
    c = filled([s + N for s in start], block, 2, d, "int8", extra=20)
    c.table[1, :4] = c.table[0, :4]
    q, o, lse = attend(c, 6, start, [N] * 2, N, d)
    check_attention(c, q, o, lse, start, [N] * 2)
    flat = _lib.KvBlockCache(c.k.contiguous(), c.v.contiguous(), c.k_scale, c.v_scale,
                             torch.cat([c.table, c.table], 1)[:, :c.table.shape[1]])
    wide = torch.full((2, N + 1, 9, 80), 5.0, dtype=torch.bfloat16, device=DEV)
    wide[:, :N, 1:7, 16:] = q
    out = torch.full((2, N, 8, 72), 9.0, dtype=torch.bfloat16, device=DEV)
    big = torch.full((2, 7, N + 3), 4.0, device=DEV)
    o2, l2 = _lib.attn_kv_block_fwd(wide[:, :N, 1:7, 16:], flat, lens_of(start), o=out[:, :, 2:, 4:68],
                                    lse=big[:, 1:, :N])
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    out[:, :, 2:, 4:68] = 9.0
    big[:, 1:, :N] = 4.0
    assert (out == 9).all() and (big == 4).all()               # nothing else written


def test_many_sequences_and_long_split():
    """More sequences than a warp scans at once, lengths from 0 to a split over the whole GPU."""
    B = 150
    start = [(i * 37) % 211 for i in range(B)]
    start[77] = 40000
    count = [1 - (i % 9 == 4) for i in range(B)]
    c = filled([s + 1 for s in start], 128, 1, 64, "int8")
    q, o, lse = attend(c, 2, start, count, 1, 64)
    check_attention(c, q, o, lse, start, count)


def test_more_sequences_than_a_launch_takes():
    """70,000 sequences of one token each, some with none: the attention of a single key is its value."""
    B, d = 70000, 64
    t = torch.randperm(B, generator=gen(1), device=DEV).int()[:, None].contiguous()
    k = torch.zeros(B, 16, 1, d, dtype=torch.int8, device=DEV)
    s = torch.full((B, 1), 9.0, device=DEV)
    c = _lib.KvBlockCache(k, k.clone(), s, s.clone(), t)
    x, y = (torch.randn(B, 1, 1, d, generator=gen(n), device=DEV) for n in (2, 3))
    start, count = torch.zeros(B, dtype=torch.int64, device=DEV), torch.ones(B, dtype=torch.int64, device=DEV)
    count[::7] = 0
    _lib.kv_block_append(x, y, c, start, count)
    kk, vv = _lib.kv_block_read(c, count, 1, dtype=torch.float32)
    live = count.bool()
    for got, want in ((kk, x), (vv, y)):                      # half a step of amax / 127
        assert ((got - want).abs() <= want.abs().amax(-1, keepdim=True) * (0.5001 / 127))[live].all()
        assert not got[~live].any()
    assert (c.k_scale[t[~live].long().flatten()] == 9).all()
    o, lse = _lib.attn_kv_block_fwd(x.to(torch.bfloat16), c, start, count, o=torch.empty_like(x))
    # weight 2^7 p over its own sum and V as it stands: roundings of fp32 only
    assert ((o - vv).abs() <= 2.0 ** -21 * vv.abs().amax(-1, keepdim=True))[live].all() and not o[~live].any()
    z = (x.to(torch.bfloat16).double() * kk.double()).sum(-1).flatten() / 8
    assert torch.isneginf(lse[~live]).all()
    assert (lse.flatten().double() - z)[live].abs().max() <= (d + 8) * 2.0 ** -23 * 40 + 2.0 ** -20
    assert _lib.device_status() == 0


def test_positions_past_32_bit_offsets():
    """A pool of more than 2^31 bytes of codes: the last blocks are reached."""
    block, d, H = 128, 128, 8
    n_blocks = (1 << 31) // (block * d * H) + 40
    k = torch.empty(n_blocks, block, H, d, dtype=torch.int8, device=DEV)
    ks = torch.zeros(n_blocks, H, device=DEV)
    t = torch.arange(n_blocks - 5, n_blocks, dtype=torch.int32, device=DEV)[None].contiguous()
    c = _lib.KvBlockCache(k, k.clone(), ks, ks.clone(), t)
    x, y = (torch.randn(1, 600, H, d, generator=gen(s), device=DEV).to(torch.bfloat16) for s in (1, 2))
    _lib.kv_block_append(x, y, c, lens_of([0]))
    kk, _ = _lib.kv_block_read(c, lens_of([600]), 600)
    # int8: half a step of amax / 127, and the output's rounding
    assert (kk - x).float().abs().max() <= (0.5 / 127 + 2 * 2.0 ** -8) * x.float().abs().max()
    q, o, lse = attend(c, H, [599], [1], 1, d)
    check_attention(c, q, o, lse, [599], [1])


@pytest.mark.parametrize("N,Hq", [(1, 8), (96, 8)])
def test_results_do_not_depend_on_the_run_or_the_workspace(N, Hq):
    start = [900, 20, 5000]
    c = filled([s + N for s in start], 64, 2, 128, "int8")
    q, o, lse = attend(c, Hq, start, [N] * 3, N, 128)
    ws = torch.full((_lib.attn_kv_block_workspace_size(q, c),), 255, dtype=torch.uint8, device=DEV)   # NaN everywhere
    for _ in range(2):
        o2, l2 = _lib.attn_kv_block_fwd(q, c, lens_of(start), workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    with pytest.raises(_lib.RcxError):
        _lib.attn_kv_block_fwd(q, c, lens_of(start), workspace=ws[:-256])


def test_two_streams_at_once():
    start = [3000, 100]
    c = filled([s + 64 for s in start], 64, 2, 128, "e4m3")
    one, many = (torch.randn(2, n, 8, 128, generator=gen(n), device=DEV).to(torch.bfloat16) for n in (1, 64))
    want = [_lib.attn_kv_block_fwd(x, c, lens_of(start)) for x in (one, many)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    st = lens_of(start)
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, x in zip(streams, (one, many)):
            with torch.cuda.stream(s):
                got.append(_lib.attn_kv_block_fwd(x, c, st))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_tensor_core_wait_that_runs_out_is_reported():
    c = filled([128], 64, 1, 128, "int8")
    q = torch.randn(1, 64, 2, 128, generator=gen(0), device=DEV).to(torch.bfloat16)
    assert _lib.device_status() == 0
    _lib.debug_inject_wait_timeout(20000)
    try:
        _lib.attn_kv_block_fwd(q, c, lens_of([64]))
        torch.cuda.synchronize()
        assert _lib.device_status() == _lib.RCX_ERR_DEVICE_TIMEOUT
    finally:
        _lib.debug_inject_wait_timeout(0)
    o, lse = _lib.attn_kv_block_fwd(q, c, lens_of([64]))
    check_attention(c, q, o, lse, [64], [64])


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_serving_loop_eager_and_captured(kind):
    """A prompt chunk, then decoding steps: rotate, append, attend.  The steps run from one
    captured graph whose lengths advance on the device, and give what eager calls give."""
    B, Hq, Hkv, d, block, N0, steps = 2, 8, 2, 128, 32, 75, 40
    inv, t = _lib.rope_freqs(_lib.YARN, 5e5, d, 8192, 131072)
    axis = _lib.rope_axes_map([24, 20, 20], interleaved=True)
    g = gen(11)
    total = N0 + steps
    q, k, v = (torch.randn(B, total, h, d, generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    pos = torch.stack([torch.arange(total, device=DEV) * m % 97 + m for m in (1, 5, 11)])[:, None].expand(3, B, total).contiguous()
    first = [N0, N0 - 20]

    def fresh():
        c = filled([total] * B, block, Hkv, d, kind, seed=4)
        n = lens_of(first)
        qq, kk = _lib.rope_axes_apply(q[:, :N0], k[:, :N0], inv, axis, pos[:, :, :N0], halves=True,
                                      q_out=torch.empty_like(q[:, :N0]), k_out=torch.empty_like(k[:, :N0]))
        _lib.kv_block_append(kk, v[:, :N0], c, lens_of([0, 0]), n)
        o, lse = _lib.attn_kv_block_fwd(qq, c, lens_of([0, 0]), n, window=50, n_sink=4, temperature=t)
        check_attention(c, qq, o, lse, [0, 0], first, 50, 4, t)
        return c, n
    c, n = fresh()
    s = dict(q=q[:, :1].clone(), k=k[:, :1].clone(), v=v[:, :1].clone(), p=pos[:, :, :1].clone())
    o, lse = torch.empty_like(s["q"]), torch.empty(B, Hq, 1, device=DEV)
    ws = torch.empty(_lib.attn_kv_block_workspace_size(s["q"], c), dtype=torch.uint8, device=DEV)

    def step(c, n):
        _lib.rope_axes_apply(s["q"], s["k"], inv, axis, s["p"], halves=True)
        _lib.kv_block_append(s["k"], s["v"], c, n)
        _lib.attn_kv_block_fwd(s["q"], c, n, o=o, lse=lse, window=50, n_sink=4, temperature=t, workspace=ws)
        n += 1

    def load(i):
        for name, x in (("q", q), ("k", k), ("v", v)):
            s[name].copy_(x[:, N0 + i:N0 + i + 1])
        s["p"].copy_(pos[:, :, N0 + i:N0 + i + 1])
    eager = []
    for i in range(steps):
        load(i)
        step(c, n)
        eager.append((o.clone(), lse.clone()))
        at = [x + i for x in first]
        check_attention(c, s["q"], o, lse, at, [1, 1], 50, 4, t)
    c2, n2 = fresh()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step(c2, n2)
    assert n2.tolist() == first                                # capture runs nothing
    for i in range(steps):
        load(i)
        graph.replay()
        assert torch.equal(o, eager[i][0]) and torch.equal(lse, eager[i][1])
    assert torch.equal(c.k.view(torch.uint8), c2.k.view(torch.uint8)) and torch.equal(c.v_scale, c2.v_scale)
    assert _lib.device_status() == 0


def test_python_refusals_on_the_gpu():
    c = filled([40], 16, 2, 64, "int8")
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        _lib.attn_kv_block_fwd(q, c, lens_of([3, 4]))
    with pytest.raises(ValueError):
        _lib.attn_kv_block_fwd(q, c, lens_of([3]).int())
    with pytest.raises(ValueError):
        _lib.attn_kv_block_fwd(q, c, torch.tensor([3]))                    # lengths on the host
    with pytest.raises(ValueError):
        _lib.attn_kv_block_fwd(q.cpu(), c, lens_of([3]))
    with pytest.raises(ValueError):
        _lib.kv_block_append(q[:, :, :2], q[:, :, :2].cpu(), c, lens_of([3]))   # V on the host
    with pytest.raises(_lib.RcxError):
        _lib.kv_block_append(q, q, c, lens_of([3]))                        # four heads, two in the cache
    with pytest.raises(TypeError):
        _lib.attn_kv_block_fwd(q.half(), c, lens_of([3]))
    with pytest.raises(AttributeError):
        c.table = c.table.clone()                                          # the view would still name the old one
