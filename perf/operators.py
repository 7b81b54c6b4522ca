"""Workloads of the multi-axis rotation and of the block-scaled 8-bit KV cache.

Three operators that a decoding step runs in this order: Q and K are rotated
by positions on several axes (``rope_axes``), K and V are quantised into the
blocks of a paged cache and read back (``kv_block``), and queries attend to
the cache (``attn_kv_block``).  ``run`` computes them in plain torch where
``own`` is false and through this package where it is true.

Cache format: a block is ``block`` tokens of one sequence and KV head and has
one fp32 scale for K and one for V.
  int8:  s = fl(amax / 127), code = rint(x * fl(1 / s)), the product unrounded;
  e4m3:  s = the smallest power of two with amax <= 448 s, code = e4m3(x / s).
A block that grows keeps the larger of its scale and the new tokens' scale; when
the scale grows the codes already there are rounded again to the new one.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ----------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 64 sequences of an image and video chat: three axes, 32 / 8 heads
        dict(name="rope_decode_step", op="rope", B=64, N=1, Hq=32, Hkv=8, d=128, type="bf16", halves=True,
             sections="16,24,24", interleaved=False, grad=False, span=131072),
        # a long video prompt, odd length, axes interleaved over the pairs, 64 / 8 heads
        dict(name="rope_video_prompt", op="rope", B=1, N=40007, Hq=64, Hkv=8, d=128, type="bf16", halves=True,
             sections="24,20,20", interleaved=True, grad=False, span=1048576),
        # the gradient of the rotation in fp32, adjacent pairs, two axes (image rows and columns)
        dict(name="rope_image_gradient", op="rope", B=2, N=8192, Hq=32, Hkv=8, d=64, type="f32", halves=False,
             sections="16,16", interleaved=False, grad=True, span=8192),
        # a decoding step's new token of 16 short sequences, then the sequences read back (moving them out)
        dict(name="kv_decode_step", op="kv", B=16, N=1, Hkv=8, d=128, block=32, codes="int8", type="bf16",
             lo=1, hi=160, ragged=False),
        # a 128K prompt written into the cache and read back
        dict(name="kv_prompt_128k", op="kv", B=1, N=131072, Hkv=8, d=128, block=64, codes="e4m3", type="bf16",
             lo=0, hi=0, ragged=False),
        # ragged chunks (one of them empty) behind cached contexts that end inside a block
        dict(name="kv_ragged_chunks", op="kv", B=9, N=1000, Hkv=8, d=64, block=16, codes="int8", type="f32",
             lo=0, hi=3000, ragged=True),
        # one user's next token at 8K context: latency
        dict(name="attn_step_8k", op="attn", B=1, N=1, Hq=32, Hkv=8, d=128, block=64, codes="int8", lo=8191, hi=8191,
             window=0, sinks=0, ragged=False),
        # a served batch: contexts from a few tokens to 32K
        dict(name="attn_batch_ragged", op="attn", B=32, N=1, Hq=64, Hkv=8, d=128, block=64, codes="e4m3", lo=3,
             hi=32768, window=0, sinks=0, ragged=False),
        # one token against a 1M-token cache, 64 / 8 heads
        dict(name="attn_step_1m", op="attn", B=1, N=1, Hq=64, Hkv=8, d=128, block=128, codes="int8", lo=1048575,
             hi=1048575, window=0, sinks=0, ragged=False),
        # a 4096-token window with 4 sinks over long contexts, 64-wide heads, small blocks
        dict(name="attn_window_sinks", op="attn", B=24, N=1, Hq=32, Hkv=8, d=64, block=16, codes="e4m3", lo=60000,
             hi=131072, window=4096, sinks=4, ragged=False),
        # five drafted tokens checked at once for 8 sequences
        dict(name="attn_draft_check", op="attn", B=8, N=5, Hq=32, Hkv=8, d=128, block=32, codes="int8", lo=9000,
             hi=24000, window=0, sinks=0, ragged=True),
        # the last 4096-token chunk of a 32K prompt over the 8-bit cache
        dict(name="attn_prompt_chunk", op="attn", B=1, N=4096, Hq=64, Hkv=8, d=128, block=128, codes="e4m3", lo=28672,
             hi=28672, window=0, sinks=0, ragged=False),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "kv", "attn", "attn"])
    Hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128])
    if op == "rope":
        N = _log(rng, 1, 20000)
        B = max(1, min(64, _log(rng, 1, 64), 20000 // N))
        pairs = d // 2
        n_axes = rng.choice([1, 2, 3, 4])
        cuts = sorted(rng.sample(range(1, pairs), n_axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        return dict(op=op, B=B, N=N, Hq=Hkv * rng.choice([1, 4, 5, 8]), Hkv=Hkv, d=d,
                    type=rng.choice(["bf16", "bf16", "f32"]), halves=rng.random() < 0.5,
                    sections=",".join(map(str, sections)), interleaved=rng.random() < 0.4, grad=rng.random() < 0.4,
                    span=_log(rng, 512, 1048576))
    block, codes = rng.choice([16, 32, 64, 128]), rng.choice(["int8", "e4m3"])
    if op == "kv":
        N = _log(rng, 1, 40000)
        B = max(1, min(32, _log(rng, 1, 32), 40000 // N))
        return dict(op=op, B=B, N=N, Hkv=Hkv, d=d, block=block, codes=codes, type=rng.choice(["bf16", "bf16", "f32"]),
                    lo=0, hi=_log(rng, 1, 2000), ragged=rng.random() < 0.6)
    G = rng.choice([1, 3, 4, 7, 8])
    N = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 2000)])
    B = _log(rng, 1, 32) if N < 9 else rng.randint(1, 3)
    hi = _log(rng, 16, 262144 // B if N < 9 else 20000 // B)
    window = rng.choice([0, 0, _log(rng, 1, 8192)])
    return dict(op=op, B=B, N=N, Hq=Hkv * G, Hkv=Hkv, d=d, block=block, codes=codes, lo=rng.randint(0, hi), hi=hi,
                window=window, sinks=rng.choice([0, 4, rng.randint(1, 100)]) if window else 0,
                ragged=N > 1 and rng.random() < 0.6)


# ----------------------------------------------------------------- inputs

def _lens(case, g):
    """Cached tokens before the call and new tokens of each sequence (host lists)."""
    B, N = case["B"], case["N"]
    start = [int(x) for x in torch.randint(case["lo"], case["hi"] + 1, (B,), generator=g)]
    if case["ragged"]:
        count = [int(x) for x in torch.randint(0, N + 1, (B,), generator=g)]
        count[0] = N
        if B > 2:
            count[1] = 0
    else:
        count = [N] * B
    return start, count


def _inv_freq(d):
    return [500000.0 ** (-2.0 * i / d) for i in range(d // 2)]


def _pair_axis(case):
    """Axis of each pair: the sections one after another, or dealt out in turn."""
    left = [int(x) for x in case["sections"].split(",")]
    if not case["interleaved"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _rows(shape, g, heads):
    """N(0, 1) rows with a different size for every channel, as keys have."""
    d = shape[-1]
    size = torch.exp(0.4 * torch.randn(heads, d, generator=g, device=DEV))
    return torch.randn(shape, generator=g, device=DEV) * size


def _block_scale(amax, codes):
    """The scale of blocks whose largest magnitude is amax (fp32, correctly rounded)."""
    if codes == "int8":
        s = (amax.double() / 127.0).float()
        return torch.where(amax > 0, s.clamp_min(2.0 ** -120), torch.zeros_like(s))
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).int()).clamp(-120, 120)
    s = ((e + 127) << 23).view(torch.float32)
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _code_values(x, s, codes):
    """Values of the codes of x (float64) for scales s (fp32, broadcast), as float32."""
    inv = torch.where(s > 0, 1.0 / s.double(), torch.zeros_like(s, dtype=torch.float64)).float()
    y = x.double() * inv.double()
    if codes == "int8":
        return torch.round(y).clamp(-127, 127).float()
    # y is exact in fp32 (a power of two times an fp32 value)
    return y.float().clamp(-448, 448).to(torch.float8_e4m3fn).float()


def _filled_pool(n_blocks, Hkv, block, d, codes, g):
    """Codes [n_blocks, Hkv, block, d] and scales [n_blocks, Hkv] of random rows."""
    c = torch.empty(n_blocks, Hkv, block, d, dtype=CODES[codes], device=DEV)
    s = torch.empty(n_blocks, Hkv, dtype=torch.float32, device=DEV)
    size = torch.exp(0.4 * torch.randn(Hkv, 1, d, generator=g, device=DEV))
    step = max(1, (1 << 26) // (Hkv * block * d))
    for i in range(0, n_blocks, step):
        n = min(step, n_blocks - i)
        x = torch.randn(n, Hkv, block, d, generator=g, device=DEV).mul_(size)
        s[i:i + n] = _block_scale(x.abs().amax((2, 3)), codes)
        y = x.div_(s[i:i + n, :, None, None])
        c[i:i + n] = (y.round_() if codes == "int8" else y).to(CODES[codes])
    return c, s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(1000003 * seed + 17)
    gc = torch.Generator().manual_seed(seed + 5)
    B, N, Hkv, d = case["B"], case["N"], case["Hkv"], case["d"]
    st = dict(case=dict(case))
    if case["op"] == "rope":
        dt = TYPES[case["type"]]
        st["q"] = _rows((B, N, case["Hq"], d), g, case["Hq"]).to(dt)
        st["k"] = _rows((B, N, Hkv, d), g, Hkv).to(dt)
        axes = len(case["sections"].split(","))
        # a clip: the first axis is time, the others walk over each frame
        first = torch.randint(0, max(1, case["span"] - N), (axes, B, 1), generator=gc)
        width = 1 + case["span"] % 61
        t = torch.arange(N)[None, :]
        pos = [first[a] + (t // width if a == 0 else (t * (a + 1)) % width if axes > 1 else t) for a in range(axes)]
        st["pos"] = torch.stack([p.expand(B, N) for p in pos]).contiguous().to(DEV)
        st["inv"] = _inv_freq(d)
        st["axis"] = _pair_axis(case)
        if own:
            from rope_context_extension_scaled_b200 import _lib
            import numpy as np
            st["plan"] = (np.asarray(st["inv"]), np.asarray(st["axis"], dtype=np.int32))
            assert list(_lib.rope_axes_map([int(x) for x in case["sections"].split(",")],
                                           interleaved=case["interleaved"])) == st["axis"]
        return st
    start, count = _lens(case, gc)
    block, codes = case["block"], case["codes"]
    total = [a + b for a, b in zip(start, count)]
    per = [max(1, -(-t // block)) for t in total]
    width = -(-(case["hi"] + N) // block)                    # a pool with room for every sequence at its longest
    n_blocks = B * width + 3
    order = torch.randperm(n_blocks, generator=gc)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :per[b]] = order[at:at + per[b]].int()
        at += per[b]
    st.update(start_list=start, count_list=count, table=table.to(DEV),
              start=torch.tensor(start, dtype=torch.int64, device=DEV),
              count=torch.tensor(count, dtype=torch.int64, device=DEV))
    for n in "kv":
        c, s = _filled_pool(n_blocks, Hkv, block, d, codes, g)
        st[n + "_codes"], st[n + "_scale"] = c.transpose(1, 2), s      # [n_blocks, block, Hkv, d]
    if case["op"] == "kv":
        dt = TYPES[case["type"]]
        st["k"] = (1.2 * _rows((B, N, Hkv, d), g, Hkv)).to(dt)
        st["v"] = _rows((B, N, Hkv, d), g, Hkv).to(dt)
    else:
        st["q"] = _rows((B, N, case["Hq"], d), g, case["Hq"]).to(torch.bfloat16)
    if own:
        from rope_context_extension_scaled_b200 import _lib
        st["cache"] = _lib.KvBlockCache(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"], st["table"])
        if case["op"] == "attn":
            need = _lib.attn_kv_block_workspace_size(st["q"], st["cache"])
            st["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return st


# ----------------------------------------------------------------- one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from rope_context_extension_scaled_b200 import _lib
    case = st["case"]
    if case["op"] == "rope":
        inv, axis = st["plan"]
        q, k = _lib.rope_axes_apply(st["q"], st["k"], inv, axis, st["pos"], halves=case["halves"],
                                    inverse=case["grad"], q_out=torch.empty_like(st["q"]),
                                    k_out=torch.empty_like(st["k"]))
        return {"q": q, "k": k}
    count = st["count"] if case["ragged"] else None
    if case["op"] == "kv":
        _lib.kv_block_append(st["k"], st["v"], st["cache"], st["start"], count)
        k, v = _lib.kv_block_read(st["cache"], st["start"] + st["count"], _read_len(st), dtype=TYPES[case["type"]])
        return {"k": k, "v": v, "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    o, lse = _lib.attn_kv_block_fwd(st["q"], st["cache"], st["start"], count, window=case["window"],
                                    n_sink=case["sinks"], workspace=st["workspace"])
    return {"o": o, "lse": lse}


def _read_len(st):
    """Tokens that every sequence of the case fits in."""
    return st["case"]["hi"] + st["case"]["N"]


def _run_plain(st):
    return {"rope": _plain_rope, "kv": _plain_kv, "attn": _plain_attn}[st["case"]["op"]](st)


def _plain_rope(st):
    """Pair i turns by pos[axis_i] inv_freq_i; the gradient turns back."""
    case = st["case"]
    half = case["d"] // 2
    axis = torch.tensor(st["axis"], device=DEV)
    inv = torch.tensor(st["inv"], dtype=torch.float64, device=DEV)
    phi = st["pos"][axis].permute(1, 2, 0).double() * inv        # [B, N, d/2]
    c, s = phi.cos().float()[:, :, None], phi.sin().float()[:, :, None]
    if case["grad"]:
        s = -s
    out = {}
    for name in "qk":
        x = st[name].float()
        if case["halves"]:
            a, b = x[..., :half], x[..., half:]
            y = torch.cat([a * c - b * s, a * s + b * c], -1)
        else:
            a, b = x[..., 0::2], x[..., 1::2]
            y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
        out[name] = y.to(st[name].dtype)
    return out


def _plain_append(st, x, codes, scale):
    """Quantise the new tokens of x [B, N, Hkv, d] into the blocks they fall in."""
    case = st["case"]
    B, N, block, kind = case["B"], case["N"], case["block"], case["codes"]
    start, count, table = st["start"], st["count"], st["table"]
    nb = (N + block - 2) // block + 1
    slot = (start // block)[:, None] + torch.arange(nb, device=DEV)                   # [B, nb]
    tok = slot[:, :, None] * block + torch.arange(block, device=DEV)                  # [B, nb, block]
    new = tok - start[:, None, None]
    is_new = (new >= 0) & (new < count[:, None, None])
    is_old = tok < start[:, None, None]
    live = is_new.any(-1)
    phys = table.long().gather(1, slot.clamp(max=table.shape[1] - 1))
    b, j = live.nonzero(as_tuple=True)
    phys, is_new, is_old, new = phys[b, j], is_new[b, j], is_old[b, j], new[b, j]
    xn = x[b[:, None], new.clamp(0, N - 1)].float()                                   # [n, block, Hkv, d]
    mask = is_new[:, :, None, None]
    amax = torch.where(mask, xn.abs(), torch.zeros_like(xn)).amax((1, 3))             # [n, Hkv]
    s_old = torch.where(is_old.any(-1)[:, None], scale[phys], torch.zeros_like(amax))
    s = torch.maximum(s_old, _block_scale(amax, kind))
    ratio = torch.where(s > 0, s_old.double() / s.double(), torch.zeros_like(s, dtype=torch.float64)).float()
    old = codes[phys].float()
    again = _round_codes(old.double() * ratio.double()[:, None, :, None], kind)
    keep = torch.where((s > s_old)[:, None, :, None], again, old)
    val = torch.where(mask, _code_values(xn, s[:, None, :, None], kind),
                      torch.where(is_old[:, :, None, None], keep, old))
    codes[phys] = val.to(codes.dtype)
    scale[phys] = s


def _round_codes(y, kind):
    if kind == "int8":
        return torch.round(y).clamp(-127, 127).float()
    return y.float().to(torch.float8_e4m3fn).float()


def _plain_read(st, codes, scale, total, n, dtype):
    block, table = st["case"]["block"], st["table"].long()
    t = torch.arange(n, device=DEV)
    ok = t[None] < total[:, None]                                                     # [B, n]
    phys = table[:, (t // block).clamp(max=table.shape[1] - 1)].clamp_min(0)
    x = codes[phys, (t % block)[None].expand_as(phys)].float() * scale[phys][..., None]
    return torch.where(ok[:, :, None, None], x, torch.zeros_like(x)).to(dtype)


def _plain_kv(st):
    out = {}
    for n in "kv":
        _plain_append(st, st[n], st[n + "_codes"], st[n + "_scale"])
        out[n] = _plain_read(st, st[n + "_codes"], st[n + "_scale"], st["start"] + st["count"], _read_len(st),
                             TYPES[st["case"]["type"]])
        out[n + "_scale"] = st[n + "_scale"]
    return out


def _plain_attn(st):
    """softmax(q k^T / sqrt(d)) v over the dequantised cache; rows past a sequence's count give 0 and -inf."""
    case = st["case"]
    B, N, Hq, Hkv, d, block = (case[x] for x in ("B", "N", "Hq", "Hkv", "d", "block"))
    G = Hq // Hkv
    o = torch.zeros(B, N, Hq, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, Hq, N), -math.inf, dtype=torch.float32, device=DEV)
    for b in range(B):
        n0, n = st["start_list"][b], st["count_list"][b]
        if n == 0:
            continue
        L = n0 + n
        low = max(0, n0 + 1 - case["window"]) if case["window"] else 0
        keys = torch.arange(low, L, device=DEV)
        if low:
            keys = torch.cat([torch.arange(min(case["sinks"], low), device=DEV), keys])
        rows = n0 + torch.arange(n, device=DEV)
        hide = keys[None] > rows[:, None]
        if case["window"]:
            hide |= (keys[None] <= rows[:, None] - case["window"]) & (keys[None] >= case["sinks"])
        hide = hide if bool(case["window"]) or n > 1 else None
        phys = st["table"][b].long()[keys // block]
        for h in range(Hkv):
            K = st["k_codes"][phys, keys % block, h].float() * st["k_scale"][phys, h][:, None]
            q = st["q"][b, :n, h * G:(h + 1) * G].float().transpose(0, 1) / math.sqrt(d)     # [G, n, d]
            S = q @ K.T
            if hide is not None:
                S = S.masked_fill_(hide, -math.inf)
            m = S.amax(-1, keepdim=True)
            P = S.sub_(m).exp_()
            l = P.sum(-1, keepdim=True)
            V = st["v_codes"][phys, keys % block, h].float() * st["v_scale"][phys, h][:, None]
            o[b, :n, h * G:(h + 1) * G] = (P @ V / l).transpose(0, 1).to(torch.bfloat16)
            lse[b, h * G:(h + 1) * G, :n] = (m + l.log())[..., 0]
            del K, V, S, P
    return {"o": o, "lse": lse}


# ----------------------------------------------------------------- in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "kv": _exact_kv, "attn": _exact_attn}[case["op"]](st)


def _exact_rope(st):
    """Each pair as a complex number times exp(+-i phi)."""
    case = st["case"]
    pos = st["pos"].double()
    half = case["d"] // 2
    out = {}
    for name in "qk":
        x = st[name].double()
        y = torch.empty_like(x)
        for i in range(half):
            i0, i1 = (i, i + half) if case["halves"] else (2 * i, 2 * i + 1)
            phi = pos[st["axis"][i]] * st["inv"][i]
            turn = torch.polar(torch.ones_like(phi), -phi if case["grad"] else phi)[..., None]
            z = torch.complex(x[..., i0], x[..., i1]) * turn
            y[..., i0], y[..., i1] = z.real, z.imag
        out[name] = y
    return out


def _exact_kv(st):
    """Sequence by sequence and block by block."""
    case = st["case"]
    block, kind, n = case["block"], case["codes"], _read_len(st)
    out = {}
    for name in "kv":
        codes, scale = st[name + "_codes"].double(), st[name + "_scale"].clone()
        res = torch.zeros(case["B"], n, case["Hkv"], case["d"], dtype=torch.float64, device=DEV)
        for b in range(case["B"]):
            n0, n1 = st["start_list"][b], st["start_list"][b] + st["count_list"][b]
            table = st["table"][b].tolist()
            whole = -(-n0 // block) * block                  # blocks from here on hold new tokens only
            if n1 > n0 and n0 % block:
                p, f, end = table[n0 // block], n0 % block, min(n1 - n0 // block * block, block)
                x = st[name][b, :end - f].double()                              # [r, Hkv, d]
                s0 = scale[p].double()
                s1 = _scale64(x.abs().amax((0, 2)), kind)
                s = torch.maximum(s0, s1)
                grown = codes[p, :f] * (s0 / s).float().double()[:, None]
                codes[p, :f] = torch.where((s > s0)[:, None], _nearest(grown, kind), codes[p, :f])
                codes[p, f:end] = _nearest(x * _inverse(s)[:, None], kind)
                scale[p] = s.float()
            if n1 > whole:
                x = st[name][b, whole - n0:n1 - n0].double()
                fill = -len(x) % block
                x = torch.cat([x, x.new_zeros(fill, *x.shape[1:])]).unflatten(0, (-1, block))
                p = torch.tensor(table[whole // block:whole // block + len(x)], device=DEV)
                s = _scale64(x.abs().amax((1, 3)), kind)
                y = _nearest(x * _inverse(s)[:, None, :, None], kind)
                last = codes[p[-1]].clone()
                codes[p] = y
                if fill:
                    codes[p[-1], block - fill:] = last[block - fill:]
                scale[p] = s.float()
            if n1:                                           # rows behind the sequence stay 0
                p = torch.tensor(table[:-(-n1 // block)], device=DEV)
                res[b, :n1] = (codes[p] * scale[p].double()[:, None, :, None]).flatten(0, 1)[:n1]
        out[name], out[name + "_scale"] = res, scale.double()
        del codes
    return out


def _scale64(amax, kind):
    """Block scale as a float64 that fp32 holds exactly."""
    if kind == "int8":
        s = (amax / 127).float().double()
    else:
        s = torch.exp2(torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448)))
        s = torch.where(amax > 448 * s, 2 * s, torch.where(amax <= 224 * s, s / 2, s))
    return torch.where(amax > 0, s.clamp_min(2.0 ** -120), torch.zeros_like(s))


def _inverse(s):
    return torch.where(s > 0, (1 / s).float().double(), torch.zeros_like(s))


def _nearest(y, kind):
    """The nearest code value, ties to even."""
    if kind == "int8":
        return y.round().clamp(-127, 127)
    _, e = torch.frexp(y)                                    # |y| in [2^(e-1), 2^e)
    step = torch.exp2((e.double() - 4).clamp_min(-9))        # e4m3: 3 bits behind the point, subnormals from 2^-9
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_attn(st):
    case = st["case"]
    B, N, Hq, Hkv, d, block = (case[x] for x in ("B", "N", "Hq", "Hkv", "d", "block"))
    G, w = Hq // Hkv, case["window"]
    o = torch.zeros(B, N, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, N), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        n0, n = st["start_list"][b], st["count_list"][b]
        if n == 0:
            continue
        table = st["table"][b, :-(-(n0 + n) // block)].long()
        for h in range(Hkv):
            K = (st["k_codes"][table, :, h].double() * st["k_scale"][table, h].double()[:, None, None]).flatten(0, 1)
            V = (st["v_codes"][table, :, h].double() * st["v_scale"][table, h].double()[:, None, None]).flatten(0, 1)
            j = torch.arange(n0 + n, device=DEV)
            K, V = K[:n0 + n], V[:n0 + n]
            for r0 in range(0, n, 512):
                r1 = min(n, r0 + 512)
                i = n0 + torch.arange(r0, r1, device=DEV)[:, None]
                seen = (j <= i) if not w else (j <= i) & ((j > i - w) | (j < case["sinks"]))
                q = st["q"][b, r0:r1, h * G:(h + 1) * G].double()
                S = torch.einsum("rgd,kd->grk", q, K) * d ** -0.5
                S = torch.where(seen, S, -math.inf)
                L = torch.logsumexp(S, -1)
                o[b, r0:r1, h * G:(h + 1) * G] = torch.einsum("grk,kd->rgd", torch.exp(S - L[..., None]), V)
                lse[b, h * G:(h + 1) * G, r0:r1] = L
    return {"o": o, "lse": lse}


# ----------------------------------------------------------------- work

def _visible(case, i):
    """Keys that token i sees."""
    w = case["window"]
    if not w or i + 1 <= w:
        return i + 1
    return w + min(case["sinks"], i + 1 - w)


def work(case):
    B, N, Hkv, d = case["B"], case["N"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        n = B * N * (case["Hq"] + Hkv) * d
        axes = len(case["sections"].split(","))
        return {"bytes": 2 * n * (2 if case["type"] == "bf16" else 4) + 8 * axes * B * N, "flops": 3 * n}
    block = case["block"]
    mean = (case["lo"] + case["hi"]) // 2
    new = N if not case["ragged"] else N // 2
    if case["op"] == "kv":
        e = 2 if case["type"] == "bf16" else 4
        row = 2 * Hkv * d                                     # K and V of a token
        read_rows = B * (mean + new)
        scales = 2 * Hkv * 4 * B * (-(-(mean + new) // block))
        return {"bytes": B * new * row * (e + 1) + read_rows * row * (1 + e) + 2 * scales,
                "flops": 3 * B * new * row + read_rows * row}
    pairs = sum(_visible(case, mean + i) for i in range(new or 1)) * B
    keys = min(mean + new, _visible(case, mean + new - 1) + (new - 1 if case["window"] else 0)) if new else mean
    return {"bytes": B * (keys * 2 * Hkv * d + 2 * Hkv * 4 * -(-keys // block) + 4 * -(-keys // block) +
                          new * case["Hq"] * (4 * d + 4)),
            "flops": 4 * pairs * case["Hq"] * d}
