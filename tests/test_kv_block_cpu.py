"""CPU checks of the multi-axis rotation and of the block-scaled 8-bit KV cache:
the oracle's rules against closed forms, and the host's refusals, which come
before anything is launched."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import rcx_oracle as orc
from rope_context_extension_scaled_b200 import _lib

FAKE = 1 << 20            # never dereferenced: every refused call stops at its checks
ONES = (ctypes.c_double * 64)(*([1.0] * 64))
INV, UNS, ALI = _lib.RCX_ERR_INVALID_ARG, _lib.RCX_ERR_UNSUPPORTED, _lib.RCX_ERR_ALIGNMENT


def tensor(dtype, shape, stride=None, ptr=FAKE):
    if stride is None:
        stride = [1] * 4
        for i in (2, 1, 0):
            stride[i] = stride[i + 1] * shape[i + 1]
    return _lib.RcxTensor(ptr, dtype, tuple(shape), tuple(stride))


def cache(dtype=_lib.RCX_I8, shape=(10, 16, 2, 128), v=None, table=FAKE, B=2, width=5, scale=FAKE, k=None):
    k = tensor(dtype, shape) if k is None else k
    return _lib.RcxKvBlocks(k, tensor(dtype, shape) if v is None else v, scale, scale, table, B, width, width)


# ------------------------------------------------------------------ oracle

def test_e4m3_rule_equals_torch_conversion():
    x = torch.randn(20000, generator=torch.Generator().manual_seed(0), dtype=torch.float64)
    y = (x * torch.exp2(torch.arange(20000) % 20 - 12.0)).clamp(-448, 448).float()
    y[:6] = torch.tensor([0.0, 2.0 ** -10, 3 * 2.0 ** -10, 448.0, 17.0, -19.0])
    assert np.array_equal(orc.kv_code_values(y.numpy(), "e4m3"), y.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("kind,amax,s", [
    ("int8", 127.0, 1.0), ("int8", 0.0, 0.0), ("int8", 2.0 ** -130, 2.0 ** -120), ("e4m3", 448.0, 1.0),
    ("e4m3", 449.0, 2.0), ("e4m3", 224.0, 0.5), ("e4m3", 225.0, 1.0), ("e4m3", 3.4e38, 2.0 ** 120),
    ("e4m3", 2.0 ** -140, 2.0 ** -120), ("e4m3", 0.0, 0.0)])
def test_block_scale(kind, amax, s):
    assert orc.kv_block_scale(float(np.float32(amax)), kind) == s


def test_growing_block_keeps_values_within_a_step():
    rng = np.random.default_rng(0)
    for kind, rel in (("int8", 1 / 127), ("e4m3", 2.0 ** -3)):
        codes, scale = np.zeros((3, 16, 8)), np.zeros(3)
        x = rng.standard_normal((20, 8)) * np.linspace(0.1, 4, 20)[:, None]
        for t in range(20):
            orc.kv_block_append(codes, scale, [2, 0], x[t:t + 1], t, kind)
        y = orc.kv_block_tokens(codes, scale, [2, 0], 20)
        # half a step per rounding; up to 15 of them, each step at most the last one's
        assert np.abs(x - y).max() <= 16 * rel * np.abs(x).max()
        assert not codes[1].any() and scale[1] == 0


# ------------------------------------------------------------------ axes map

@pytest.mark.parametrize("sections,inter", [([16, 24, 24], False), ([24, 20, 20], True), ([64], True), ([1, 0, 3], True),
                                            ([5, 1, 2], False)])
def test_axes_map(lib, sections, inter):
    assert list(_lib.rope_axes_map(sections, interleaved=inter)) == orc.rope_axes_map(sections, inter)


def test_axes_map_refusals(lib):
    out = (ctypes.c_int32 * 64)()
    sec = (ctypes.c_int64 * 3)(16, 24, 24)
    assert lib.rcx_rope_axes_map(sec, 3, 0, 63, out) == INV            # sections do not add up
    assert lib.rcx_rope_axes_map(sec, 0, 0, 64, out) == INV
    assert lib.rcx_rope_axes_map(None, 3, 0, 64, out) == INV
    assert lib.rcx_rope_axes_map((ctypes.c_int64 * 2)(65, -1), 2, 0, 64, out) == INV
    assert lib.rcx_rope_axes_map((ctypes.c_int64 * 1)(129), 1, 0, 129, out) == INV


def test_rope_axes_refusals(lib):
    q = tensor(_lib.RCX_BF16, (2, 4, 3, 128))
    k32 = tensor(_lib.RCX_F32, (2, 4, 1, 128))
    null = _lib.RcxTensor()
    ax = (ctypes.c_int32 * 64)()

    def call(q=q, k=null, qo=None, ko=null, pos=FAKE, n_axes=1, sa=8, sb=4, inv=ONES, axis=ax, flags=0):
        return lib.rcx_rope_axes_apply(q, k, q if qo is None else qo, ko, pos, n_axes, sa, sb, inv, axis, flags, None)
    assert call(q=null, qo=null) == 0                                    # nothing to rotate
    assert call(inv=None) == INV and call(axis=None) == INV and call(pos=None) == INV
    assert call(n_axes=0) == INV and call(n_axes=257) == INV and call(sa=-1) == INV and call(flags=4) == INV
    assert call(axis=(ctypes.c_int32 * 64)(*([0] * 63 + [1]))) == INV    # an axis that is not there
    assert call(axis=(ctypes.c_int32 * 64)(*([0] * 63 + [-1]))) == INV
    assert call(k=k32, ko=k32) == INV                                    # two dtypes
    assert call(qo=tensor(_lib.RCX_BF16, (2, 4, 2, 128))) == INV
    assert call(q=tensor(_lib.RCX_BF16, (2, 4, 3, 24))) == UNS           # d not a multiple of 16
    assert call(q=tensor(_lib.RCX_F32, (2, 4, 3, 12))) == UNS
    assert call(q=tensor(_lib.RCX_BF16, (2, 4, 3, 128), (1560, 390, 130, 1))) == ALI
    assert call(q=tensor(_lib.RCX_BF16, (0, 4, 3, 128))) == 0 and call(q=tensor(_lib.RCX_BF16, (2, 0, 3, 128))) == 0


# ------------------------------------------------------------------ cache

BAD_CACHES = [
    (INV, dict(dtype=_lib.RCX_BF16)),
    (INV, dict(v=tensor(_lib.RCX_E4M3, (10, 16, 2, 128)))),              # two code types
    (INV, dict(v=tensor(_lib.RCX_I8, (10, 16, 3, 128)))),
    (INV, dict(scale=None)), (INV, dict(table=None)), (INV, dict(width=0)),
    (INV, dict(k=tensor(_lib.RCX_I8, (10, 16, 2, 128), (4096, 256, 128, 2)))),
    (UNS, dict(shape=(10, 8, 2, 128))), (UNS, dict(shape=(10, 48, 2, 128))), (UNS, dict(shape=(10, 256, 2, 128))),
    (UNS, dict(shape=(10, 16, 2, 96))), (UNS, dict(shape=(10, 16, 2, 256))),
    (UNS, dict(width=1 << 27)),                                          # 2^31 tokens
    (ALI, dict(k=tensor(_lib.RCX_I8, (10, 16, 2, 128), (4352, 272, 136, 1)))),
    (ALI, dict(k=tensor(_lib.RCX_I8, (10, 16, 2, 128), ptr=FAKE + 8))), (ALI, dict(scale=FAKE + 2)),
]


@pytest.mark.parametrize("status,bad", BAD_CACHES)
def test_bad_caches_are_refused(lib, status, bad):
    c = ctypes.byref(cache(**bad))
    shape = bad.get("shape", (10, 16, 2, 128))
    rows = tensor(_lib.RCX_BF16, (2, 3, 2, shape[3]))
    null = _lib.RcxTensor()
    assert lib.rcx_kv_block_append(rows, rows, c, FAKE, None, None) == status
    assert lib.rcx_kv_block_read(c, FAKE, rows, rows, None) == status
    assert lib.rcx_attn_kv_block_fwd(rows, c, FAKE, None, rows, null, 0, 0, 1.0, FAKE, 1 << 40, None) == status
    assert lib.rcx_attn_kv_block_workspace_size(rows, c) == -1


def test_append_and_read_refusals(lib):
    c = ctypes.byref(cache())
    rows = tensor(_lib.RCX_BF16, (2, 3, 2, 128))
    for bad, st in ((tensor(_lib.RCX_BF16, (1, 3, 2, 128)), INV), (tensor(_lib.RCX_BF16, (2, 3, 4, 128)), INV),
                    (tensor(_lib.RCX_BF16, (2, 3, 2, 64)), INV), (tensor(_lib.RCX_I8, (2, 3, 2, 128)), INV),
                    (tensor(_lib.RCX_BF16, (2, 3, 2, 128), ptr=FAKE + 8), ALI),
                    (tensor(_lib.RCX_BF16, (2, 3, 2, 128), (1000, 260, 130, 1)), ALI)):
        assert lib.rcx_kv_block_append(bad, bad, c, FAKE, None, None) == st
        assert lib.rcx_kv_block_read(c, FAKE, bad, bad, None) == st
    f32 = tensor(_lib.RCX_F32, (2, 3, 2, 128))
    assert lib.rcx_kv_block_append(rows, f32, c, FAKE, None, None) == INV        # K and V of two dtypes
    assert lib.rcx_kv_block_append(rows, rows, c, None, None, None) == INV
    assert lib.rcx_kv_block_read(c, None, rows, rows, None) == INV
    long = tensor(_lib.RCX_BF16, (2, 81, 2, 128))
    assert lib.rcx_kv_block_append(long, long, c, FAKE, None, None) == INV       # 81 tokens, 80 places
    none = tensor(_lib.RCX_BF16, (2, 0, 2, 128))
    assert lib.rcx_kv_block_append(none, none, c, None, None, None) == 0
    assert lib.rcx_kv_block_read(c, None, none, none, None) == 0


def test_attention_refusals(lib):
    c = ctypes.byref(cache())
    q = tensor(_lib.RCX_BF16, (2, 3, 8, 128))
    null = _lib.RcxTensor()

    def call(q=q, o=None, lse=null, start=FAKE, window=0, sink=0, t=1.0, ws=FAKE, n=1 << 40):
        return lib.rcx_attn_kv_block_fwd(q, c, start, None, q if o is None else o, lse, window, sink, t, ws, n, None)
    assert call(start=None) == INV and call(window=-1) == INV and call(sink=-1) == INV
    assert call(t=0.0) == INV and call(t=math.nan) == INV and call(t=math.inf) == INV
    assert call(ws=None) == INV and call(n=16) == INV and call(ws=FAKE + 16) == ALI
    assert call(q=tensor(_lib.RCX_BF16, (2, 3, 7, 128))) == INV                  # Hkv = 2 does not divide 7
    assert call(q=tensor(_lib.RCX_BF16, (1, 3, 8, 128))) == INV
    assert call(q=tensor(_lib.RCX_BF16, (2, 3, 8, 64))) == INV
    assert call(q=tensor(_lib.RCX_BF16, (2, 81, 8, 128))) == INV                 # more rows than tokens
    assert call(q=tensor(_lib.RCX_F32, (2, 3, 8, 128))) == UNS
    assert call(o=tensor(_lib.RCX_BF16, (2, 3, 4, 128))) == INV
    assert call(o=tensor(_lib.RCX_F32, (2, 3, 8, 128), ptr=FAKE + 8)) == ALI
    assert call(q=tensor(_lib.RCX_BF16, (2, 3, 8, 128), ptr=FAKE + 8)) == ALI
    assert call(lse=tensor(_lib.RCX_F32, (2, 8, 4, 1))) == INV
    assert call(q=tensor(_lib.RCX_BF16, (2, 0, 8, 128))) == 0                    # no rows: nothing to do
    need = lib.rcx_attn_kv_block_workspace_size(q, c)
    assert need > 0 and call(n=need - 1) == INV


def test_python_side_refusals(lib):
    k = torch.zeros(4, 16, 2, 64, dtype=torch.int8)
    s = torch.zeros(4, 2)
    t = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        _lib.KvBlockCache(k, k, s, s, t)                                         # not on a GPU
    with pytest.raises(ValueError):
        _lib.KvBlockCache(k, k, s[:, :1], s, t)
    with pytest.raises(ValueError):
        _lib.KvBlockCache(k, k, s, s, t.long())
    q = torch.zeros(1, 3, 2, 64)
    with pytest.raises(ValueError):
        _lib.rope_axes_apply(q, None, np.ones(32), np.zeros(32), torch.zeros(1, 1, 4, dtype=torch.int64))
    with pytest.raises(ValueError):
        _lib.rope_axes_apply(q, None, np.ones(31), np.zeros(32), torch.zeros(1, 1, 3, dtype=torch.int64))
    with pytest.raises(ValueError):
        _lib.rope_axes_apply(q, None, np.ones(32), np.zeros(32), torch.zeros(1, 1, 3))
    with pytest.raises(ValueError):
        _lib.rope_axes_apply(q, None, np.ones(32), np.zeros(32), torch.zeros(1, 1, 3, dtype=torch.int64))  # on the CPU
    assert _lib.rope_axes_apply(None, None, None, None, None) == (None, None)
