"""The cache operators of long-running sequences: what each computes, in plain torch, and how it is called.

A serving program keeps the keys and values of many sequences in pools of pages of 32 positions, found
through a block table.  Four operators work on such a pool, held in bfloat16 or in 4 bits:

- "attend": grouped-query attention of the last rows of every sequence over its cached positions, the row at
  position p seeing key j if j <= p and (no window, or j > p - window, or j < sinks);
- "append": new key and value rows written to the positions they belong to (quantised in a 4-bit pool), then
  read back;
- "copy": whole pages copied inside the pools of all layers, as a forked sequence or a shrunk pool needs it.

A 4-bit page of one KV head holds 32 rows: 32 D / 2 bytes of e2m1 codes, then 32 D / 16 e4m3 block scales, then
32 float32 row scales.  K: codes [32][D / 2] (the even element in the low nibble), block scales [32][D / 16].
V, with position 8 t + 2 j + i of the page: codes [j][D / 16][t][16 elements] (position i = 0 in the low nibble,
i = 1 in the high one), block scales [D / 16][32].  A row is quantised in float32 steps: s = amax / 2688 (0 for a row of zeros), b = e4m3(min(amax of 16 /
(6 s), 448)), code = e2m1(clamp(x / (b s), -6, 6)) with ties to the even code; its value is e2m1 * b * s.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 32
BF16, NVFP4 = "bf16", "nvfp4"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def _attend(name, fmt, dtype, heads, kv_heads, dim, seqs, rows, length, ragged, window, sinks):
    return {"name": name, "op": "attend", "fmt": fmt, "type": dtype, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "seqs": seqs, "rows": rows, "len": length, "ragged": ragged, "window": window,
            "sinks": sinks}


def _append(name, fmt, dtype, kv_heads, dim, seqs, rows, length, ragged):
    return {"name": name, "op": "append", "fmt": fmt, "type": dtype, "heads": kv_heads, "kv_heads": kv_heads,
            "dim": dim, "seqs": seqs, "rows": rows, "len": length, "ragged": ragged, "window": 0, "sinks": 0}


def _copy(name, fmt, kv_heads, dim, pools, pages, moves):
    return {"name": name, "op": "copy", "fmt": fmt, "kv_heads": kv_heads, "dim": dim, "pools": pools,
            "pages": pages, "moves": moves}


def listed():
    return [
        # one sequence decoding with a window and a few sinks: latency counts
        _attend("window_decode_1", BF16, "f32", 32, 8, 128, 1, 1, 1024, False, 256, 4),
        # a full batch of streams past the length they were given, all windows full or filling
        _attend("window_decode_32", BF16, "f32", 32, 8, 128, 32, 1, 8192, True, 2048, 4),
        # a chunk of a long prompt with a window, bfloat16 activations
        _attend("window_prompt", BF16, "bf16", 32, 8, 128, 4, 1024, 8192, True, 1024, 16),
        # a small model's prompt without a window: 64-wide heads, odd lengths
        _attend("prompt_dim64", BF16, "bf16", 4, 2, 64, 3, 333, 1999, True, 0, 0),
        # one sequence decoding over a 4-bit cache
        _attend("kv4_decode_1", NVFP4, "f32", 32, 8, 128, 1, 1, 4096, False, 0, 0),
        # the largest serving batch: 32 streams of very different lengths in 4 bits
        _attend("kv4_decode_32", NVFP4, "bf16", 32, 8, 128, 32, 1, 32768, True, 0, 0),
        # five drafted frames per sequence looked at in one pass, with a window
        _attend("kv4_rows_5", NVFP4, "f32", 32, 8, 128, 16, 5, 4096, True, 1000, 4),
        # a prompt chunk over positions already held in 4 bits
        _attend("kv4_prompt", NVFP4, "bf16", 32, 8, 128, 2, 1024, 5120, False, 0, 0),
        # one new row per sequence written to the 4-bit pool in a decode step
        _append("append_32", NVFP4, "f32", 8, 128, 32, 1, 4096, True),
        # whole prompts written to the 4-bit pool
        _append("append_prompt", NVFP4, "bf16", 8, 128, 16, 512, 512, False),
        # a fork: one partly filled page in the K and V pools of 36 layers
        _copy("copy_fork", NVFP4, 8, 128, 72, 64, 1),
        # a pool shrunk: live pages moved down in all layers
        _copy("copy_many", BF16, 8, 128, 72, 192, 64),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    case = _draw(rng)
    while work(case)["bytes"] > 6e8 or work(case)["flops"] > 1.5e11:  # no more than the largest listed ones
        case = _draw(rng)
    return case


def _draw(rng):
    kind = rng.choice(("decode", "decode", "rows", "prompt", "append", "copy"))
    fmt = rng.choice((BF16, NVFP4))
    dim = rng.choice((64, 128, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    ratio = rng.choice((1, 2, 3, 4, 8))
    if kind == "copy":
        pages = _spread(rng, 8, 192)
        return _copy(None, fmt, kv_heads, dim, _spread(rng, 2, 72), pages, rng.randint(1, max(1, pages // 3)))
    if kind == "append":
        rows = _spread(rng, 1, 512)
        return _append(None, fmt, rng.choice(("f32", "bf16")), kv_heads, dim, rng.randint(1, 16), rows,
                       rows + _spread(rng, 1, 512), rng.random() < 0.7)
    window = rng.choice((0, _spread(rng, 16, 2048)))
    sinks = rng.choice((0, 1, 4, rng.randint(2, 64))) if window else 0
    if kind == "decode":
        seqs = _spread(rng, 1, 32)
        return _attend(None, fmt, rng.choice(("f32", "bf16")), kv_heads * ratio, kv_heads, dim, seqs, 1,
                       _spread(rng, 16, 16384), rng.random() < 0.8, window, sinks)
    if kind == "rows":
        return _attend(None, fmt, rng.choice(("f32", "bf16")), kv_heads * ratio, kv_heads, dim,
                       rng.randint(1, 16), rng.randint(2, 12), _spread(rng, 16, 4096), True, window, sinks)
    rows = _spread(rng, 48, 700)
    return _attend(None, fmt, "bf16", min(kv_heads * ratio, 32), kv_heads, dim, rng.randint(1, 3), rows,
                   rows + _spread(rng, 1, 2048), rng.random() < 0.7, window, sinks)


def _sizes(case):
    """Cached positions and rows of every sequence; the case alone decides them."""
    n, rows, length = case["seqs"], case["rows"], case["len"]
    if not case["ragged"]:
        return [length] * n, [rows] * n
    lens, counts = [], []
    for i in range(n):
        f = (0.6180339887 * i) % 1.0
        r = rows if i == 0 else max(1, rows - int(f * rows * 0.5))
        l = length if i == 0 else max(r, int(length * (1.0 - f)))
        if case["op"] == "attend" and rows == 1 and i == 2:
            l = 0                               # a slot that holds nothing yet
        lens.append(l)
        counts.append(r)
    return lens, counts


def _seen(case, first, last):
    """Cached positions that the rows at positions first..last see, and the (row, position) pairs of them."""
    w, s = case["window"], case["sinks"]
    if last < 0:
        return 0, 0
    pairs = 0
    for p in range(max(first, 0), last + 1):
        pairs += p + 1 if not w else min(p + 1, w) + max(0, min(s, p + 1 - w))
    low = 0 if not w else max(0, max(first, 0) - w + 1)
    return last + 1 - low + min(s, low), pairs


def _row_bytes(case):
    d = case["dim"]
    return 2 * d if case["fmt"] == BF16 else d // 2 + d // 16 + 4


def page_bytes(case):
    return case["kv_heads"] * PAGE * _row_bytes(case)


def work(case):
    if case["op"] == "copy":
        return {"bytes": 2 * case["pools"] * case["moves"] * page_bytes(case), "flops": 0}
    lens, counts = _sizes(case)
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "append":
        n = sum(counts) * case["kv_heads"] * 2
        return {"bytes": n * (case["dim"] * (size + 4) + _row_bytes(case)), "flops": n * case["dim"] * 4}
    keys = pairs = 0
    for l, r in zip(lens, counts):
        k, p = _seen(case, l - r, l - 1)
        keys, pairs = keys + k, pairs + p
    return {"bytes": keys * case["kv_heads"] * 2 * _row_bytes(case)
            + 2 * sum(counts) * case["heads"] * case["dim"] * size,
            "flops": 4 * case["heads"] * case["dim"] * pairs}


# ---------------------------------------------------------------- the pool's 4-bit form
def _quantise(x):
    """float32 rows [..., D] -> e2m1 codes [..., D], block scales [..., D / 16] (both bytes), row scales [...]."""
    c = lambda v: torch.full((), v, device=x.device)  # a tensor: a division by a number becomes a product
    b16 = x.unflatten(-1, (-1, 16))
    amax = x.abs().amax(-1)
    s = amax / c(2688.0)
    s6 = (s * 6.0).unsqueeze(-1)
    b = torch.where(s6 > 0, (b16.abs().amax(-1) / s6).clamp(max=448.0), 0.0).to(torch.float8_e4m3fn)
    step = (b.float() * s.unsqueeze(-1)).unsqueeze(-1)
    r = torch.where(step > 0, (b16 / step).clamp(-6.0, 6.0), 0.0).flatten(-2)
    a = r.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8) + ((r < 0).to(torch.uint8) << 3))
    return code, b.view(torch.uint8), s


def _split_page(pool, case, v):
    """Views of a 4-bit pool [..][bytes]: packed codes (K [.., 32, D / 2], V [.., 4, D / 16, 4, 16]), block scales
    [.., 32, D / 16] and row scales [.., 32]."""
    d = case["dim"]
    codes = pool[..., :PAGE * d // 2].unflatten(-1, (4, d // 16, 4, 16) if v else (PAGE, d // 2))
    scales = pool[..., PAGE * d // 2:PAGE * (d // 2 + d // 16)]
    scales = scales.unflatten(-1, (d // 16, PAGE)).transpose(-1, -2) if v else scales.unflatten(-1, (PAGE, d // 16))
    return codes, scales, pool.view(torch.float32)[..., PAGE * (d // 2 + d // 16) // 4:]


def _pack(code, v):
    """Codes of whole pages [.., 32, D] as the pages hold them."""
    if not v:
        return code[..., 0::2] | (code[..., 1::2] << 4)
    c = code.unflatten(-2, (4, 4, 2)).unflatten(-1, (-1, 16))  # [.., t, j, i, D / 16, 16]
    return (c[..., 0, :, :] | (c[..., 1, :, :] << 4)).movedim(-4, -2)


def _unpack(codes, v):
    """Codes [.., 32, D] of whole pages."""
    both = torch.stack((codes & 15, codes >> 4), -1)
    if not v:
        return both.flatten(-2)
    return both.movedim(-3, -5).movedim(-1, -3).flatten(-5, -3).flatten(-2)  # [.., t, j, i, D / 16, 16]


def _values(code, scales, s):
    """float32 values of quantised rows."""
    table = torch.tensor(E2M1 + tuple(-e for e in E2M1), device=code.device)
    x = table[code.int()].unflatten(-1, (-1, 16))
    return ((x * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)) * s.unsqueeze(-1)


def _whole(pool, case, v, table):
    """Every position of every sequence, float32 [seqs, Hkv, positions, D]."""
    pages = pool[table.long()].transpose(1, 2)  # [seqs, Hkv, pages, ...]
    if case["fmt"] == BF16:
        return pages.flatten(2, 3).float()
    codes, scales, s = _split_page(pages, case, v)
    return _values(_unpack(codes, v), scales.contiguous(), s).flatten(2, 3)


# ---------------------------------------------------------------- inputs
def _store(pool, case, v, lo, x):
    """Fills pages lo.. of a pool with float32 rows x [pages][Hkv][32][D]."""
    if case["fmt"] == BF16:
        pool[lo:lo + x.shape[0]] = x.to(torch.bfloat16)
    else:
        code, b, s = _quantise(x)
        for p, y in zip(_split_page(pool[lo:lo + x.shape[0]], case, v), (_pack(code, v), b, s)):
            p.copy_(y)


def _pool(case, n_pages, gen, v):
    h, d = case["kv_heads"], case["dim"]
    if case["fmt"] == BF16:
        pool = torch.empty((n_pages, h, PAGE, d), dtype=torch.bfloat16, device="cuda")
    else:
        pool = torch.empty((n_pages, h, PAGE * _row_bytes(case)), dtype=torch.uint8, device="cuda")
    # keys have channels of unequal size, values are smaller
    size = torch.exp(0.5 * torch.randn(h, 1, d, device="cuda", generator=gen)) * (0.25 if v else 0.8)
    for lo in range(0, n_pages, 2048):
        n = min(2048, n_pages - lo)
        _store(pool, case, v, lo, torch.randn((n, h, PAGE, d), device="cuda", generator=gen) * size)
    return pool


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    host = np.random.default_rng(seed)
    if case["op"] == "copy":
        shape = (case["pools"], case["pages"], page_bytes(case))
        pools = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=gen)
        order = host.permutation(case["pages"]).astype(np.int32)
        n = case["moves"]
        return {"case": case, "pools": pools, "bases": [p.data_ptr() for p in pools.unbind(0)],
                "src": order[:n].copy(), "dst": order[n:2 * n].copy()}
    lens, counts = _sizes(case)
    dtype = TYPES[case["type"]]
    stride = max(1, max((l + PAGE - 1) // PAGE for l in lens))
    n_pages = 1 + sum((l + PAGE - 1) // PAGE for l in lens)
    order = host.permutation(n_pages - 1).astype(np.int32) + 1
    table = np.zeros((case["seqs"], stride), np.int32)
    used = 0
    for i, l in enumerate(lens):
        n = (l + PAGE - 1) // PAGE
        table[i, :n] = order[used:used + n]
        used += n
    starts = np.concatenate(([0], np.cumsum(counts)))
    state = {"case": case, "K": _pool(case, n_pages, gen, False), "V": _pool(case, n_pages, gen, True),
             "table": torch.from_numpy(table).cuda(), "n_pages": n_pages,
             "lengths": torch.tensor(lens, dtype=torch.int32, device="cuda"),
             "row_start": torch.tensor(starts, dtype=torch.int32, device="cuda"),
             "n_rows": int(starts[-1]), "max_rows": max(counts), "max_length": max(max(lens), 1)}
    n, h, d = state["n_rows"], case["heads"], case["dim"]
    if case["op"] == "attend":
        state["q"] = torch.randn((n, h, d), device="cuda", generator=gen).to(dtype)
        state["out"] = torch.empty((n, h, d), dtype=dtype, device="cuda")
    else:
        for name, size in (("k", 0.8), ("v", 0.25)):
            channel = torch.exp(0.5 * torch.randn(h, d, device="cuda", generator=gen)) * size
            state[name] = (torch.randn((n, h, d), device="cuda", generator=gen) * channel).to(dtype)
            state["read_" + name] = torch.empty((n, h, d), device="cuda")
    return state


# ---------------------------------------------------------------- one pass
def _rows(st):
    """Sequence and position of every row."""
    i = torch.arange(st["n_rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(st["row_start"], i, right=True) - 1
    return seq, st["lengths"][seq] - st["row_start"][seq + 1] + i


def _plain_attend(st):
    case = st["case"]
    h, hk, d, r = case["heads"], case["kv_heads"], case["dim"], st["max_rows"]
    seq, pos = _rows(st)
    at = (torch.arange(st["n_rows"], device="cuda") - st["row_start"][seq])  # row's place in its sequence
    q = torch.zeros((case["seqs"], r, h, d), device="cuda")
    q[seq, at] = st["q"].float()
    p = torch.full((case["seqs"], r), -1, device="cuda", dtype=torch.int32)
    p[seq, at] = pos.int()
    q = q.unflatten(2, (hk, h // hk)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [seqs, Hkv, G * r, D]
    k, v = _whole(st["K"], case, False, st["table"]), _whole(st["V"], case, True, st["table"])
    z = torch.matmul(q, k.transpose(-1, -2)) * (d ** -0.5)
    j = torch.arange(k.shape[2], device="cuda", dtype=torch.int32)
    see = j <= p[..., None]
    if case["window"]:
        see &= (j > p[..., None] - case["window"]) | (j < case["sinks"])
    see = see[:, None, None].expand(-1, 1, h // hk, -1, -1).flatten(2, 3)  # [seqs, 1, G * r, positions]
    z = z.masked_fill(~see, float("-inf"))
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(top == float("-inf"), 0.0, top))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    o = o.unflatten(2, (h // hk, r)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return o[seq, at].to(TYPES[case["type"]])


def _plain_append(st):
    case = st["case"]
    seq, pos = _rows(st)
    page, slot = st["table"][seq, (pos // PAGE).long()].long(), (pos % PAGE).long()

    def one(pool, x, v):
        if case["fmt"] == BF16:
            pool[page, :, slot] = x.to(torch.bfloat16)
            return pool[page, :, slot].float()
        codes, scales, s = _split_page(pool, case, v)
        code, scales[page, :, slot], s[page, :, slot] = _quantise(x.float())
        if v:  # a byte holds two positions: what each nibble changes by is added to it
            t, j, shift = slot // 8, slot // 2 % 4, (slot % 2 * 4).to(torch.uint8)[:, None, None, None]
            at = codes[page, :, j, :, t] >> shift & 15
            h, g, e = (torch.arange(n, device="cuda") for n in (codes.shape[1], codes.shape[3], 16))
            of = lambda x: x[:, None, None, None]
            codes.index_put_((of(page), h[:, None, None], of(j), g[:, None], of(t), e),
                             (code.unflatten(-1, (-1, 16)) - at) << shift, accumulate=True)
            code = (codes[page, :, j, :, t] >> shift & 15).flatten(-2)
        else:
            codes[page, :, slot] = code[..., 0::2] | (code[..., 1::2] << 4)
            code = torch.stack((codes[page, :, slot] & 15, codes[page, :, slot] >> 4), -1).flatten(-2)
        return _values(code, scales[page, :, slot], s[page, :, slot])

    return one(st["K"], st["k"], False), one(st["V"], st["v"], True)


def _cache(st):
    import dual_ar_decode_gb300 as tf
    case = st["case"]
    return tf.kv_cache(case["fmt"], case["kv_heads"], case["dim"], st["K"].data_ptr(), st["V"].data_ptr(),
                       st["n_pages"], st["table"].data_ptr(), st["table"].shape[1], case["seqs"],
                       st["lengths"].data_ptr(), st["row_start"].data_ptr(), st["n_rows"], st["max_rows"],
                       st["max_length"])


def run(state):
    case = state["case"]
    if own:
        import dual_ar_decode_gb300 as tf
        stream = torch.cuda.current_stream().cuda_stream
        if case["op"] == "copy":
            tf.op_cache_copy(state["bases"], page_bytes(case), case["pages"], state["src"], state["dst"], stream)
            return state["pools"]
        if case["op"] == "append":
            cache = _cache(state)
            tf.op_cache_append(cache, state["k"].data_ptr(), state["v"].data_ptr(), case["type"], stream)
            tf.op_cache_read(cache, state["read_k"].data_ptr(), state["read_v"].data_ptr(), "f32", stream)
            return state["read_k"], state["read_v"]
        tf.op_attention_cache(_cache(state), state["q"].data_ptr(), state["out"].data_ptr(), case["type"],
                              case["heads"], case["window"], case["sinks"], stream=stream)
        return state["out"]
    if case["op"] == "copy":
        pools = state["pools"]
        src, dst = (torch.from_numpy(state[n]).cuda().long() for n in ("src", "dst"))
        pools[:, dst] = pools[:, src]
        return pools
    if case["op"] == "append":
        return _plain_append(state)
    return _plain_attend(state)


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_page_values(st, which, i, n):
    """float64 [n, Hkv, D]: the first n cached positions of sequence i, decoded byte by byte."""
    case = st["case"]
    hk, d = case["kv_heads"], case["dim"]
    pages = st[which][st["table"][i, :(n + PAGE - 1) // PAGE].long()]
    if case["fmt"] == BF16:
        return pages.double().permute(0, 2, 1, 3).reshape(-1, hk, d)[:n]
    raw = pages.long()
    if which == "K":
        nib = torch.stack((raw[..., :16 * d] % 16, raw[..., :16 * d] // 16), -1).reshape(-1, hk, PAGE, d)
    else:
        pos, dim = torch.meshgrid(torch.arange(PAGE), torch.arange(d), indexing="ij")
        byte = ((pos // 2 % 4 * (d // 16) + dim // 16) * 4 + pos // 8) * 16 + dim % 16
        nib = (raw[..., byte.cuda()] // 16 ** (pos % 2).cuda()) % 16
    mag = nib % 8
    e, m = mag // 2, mag % 2
    x = torch.where(e == 0, m * 0.5, (1 + 0.5 * m.double()) * 2.0 ** (e - 1).double()) * (1 - 2 * (nib // 8)).double()
    sb = raw[..., 16 * d:18 * d]
    sb = sb.reshape(-1, hk, d // 16, PAGE).transpose(2, 3) if which == "V" else sb.reshape(-1, hk, PAGE, d // 16)
    e, m = sb // 8 % 16, sb % 8
    scale = torch.where(e == 0, m.double() / 512, (1 + m.double() / 8) * 2.0 ** (e - 7).double())
    bits = raw[..., 18 * d:].reshape(-1, hk, PAGE, 4)
    bits = bits[..., 0] + bits[..., 1] * 256 + bits[..., 2] * 65536 + bits[..., 3] * 16777216
    row = bits.to(torch.int32).view(torch.float32).double()
    y = x.reshape(-1, hk, PAGE, d // 16, 16) * scale[..., None] * row[..., None, None]
    return y.reshape(-1, hk, PAGE, d).permute(0, 2, 1, 3).reshape(-1, hk, d)[:n]


def _exact_rows(x):
    """What a 4-bit pool holds of rows [.., D], in 64 bits with the float32 steps that the format names."""
    f32 = lambda a: a.astype(np.float32).astype(np.float64)
    x = x.double().cpu().numpy()
    s = f32(np.abs(x).max(-1) / 2688.0)[..., None, None]
    y = x.reshape(*x.shape[:-1], -1, 16)
    with np.errstate(divide="ignore", invalid="ignore"):
        b = np.minimum(np.nan_to_num(f32(np.abs(y).max(-1, keepdims=True) / f32(6.0 * s))), 448.0)
        # e4m3: three bits after the leading one, none below 2^-9
        ulp = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(b, 2.0 ** -20))), -6) - 3)
        b = np.rint(b / ulp) * ulp
        r = np.clip(np.nan_to_num(f32(y / f32(b * s))), -6.0, 6.0)
    ulp = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(r), 2.0 ** -20))), 0) - 1)
    r = np.rint(r / ulp) * ulp  # e2m1: one bit after the leading one, none below 1 / 2
    return (np.where(b > 0, r, 0.0) * b * s).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "copy":
        return None
    if case["op"] == "append":
        if case["fmt"] == BF16:
            return tuple(st[n].to(torch.bfloat16).double() for n in ("k", "v"))
        return tuple(torch.from_numpy(_exact_rows(st[n])) for n in ("k", "v"))
    lens, counts = _sizes(case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros((st["n_rows"], h, d), dtype=torch.float64, device="cuda")
    row = 0
    for i, (n, r) in enumerate(zip(lens, counts)):
        if n:
            k, v = _exact_page_values(st, "K", i, n), _exact_page_values(st, "V", i, n)
            q = st["q"][row:row + r].double().reshape(r, hk, h // hk, d)
            p = torch.arange(n - r, n, device="cuda")[:, None]
            j = torch.arange(n, device="cuda")
            hidden = j > p
            if case["window"]:
                hidden |= (j <= p - case["window"]) & (j >= case["sinks"])
            for g in range(hk):
                z = torch.einsum("rad,jd->raj", q[:, g], k[:, g]) / math.sqrt(d)
                w = torch.softmax(z.masked_fill(hidden[:, None], float("-inf")), -1)
                w = w.masked_fill(hidden.all(-1)[:, None, None], 0.0)
                out[row:row + r, g * (h // hk):(g + 1) * (h // hk)] = torch.einsum("raj,jd->rad", w, v[:, g])
        row += r
    return out
