"""The 4-bit operators, case by case: microscaled 4-bit rows (quantised, read back and
multiplied) and a paged key/value cache held in low-bit codes (appended to and read back).

``run`` computes a case in elementary torch operations, or, where ``own`` is true, with
the package's kernels.  Both read and write the same stored forms:

* microscaled rows: ``codes`` int32 (rows, ceil(cols/32)*4), eight 4-bit codes per word,
  column 8w+i in bits 4i..4i+3; a code is sign<<3 | index into 0, .5, 1, 1.5, 2, 3, 4, 6.
  One scale 2^(e-127) per 32 columns, e held as a byte in 128x4 tiles: ``scales`` uint8
  (ceil(rows/128), ceil(cols/128), 32, 16), the byte of row r and block k at
  [r//128, k//4, r%32, 4*((r%128)//32) + k%4].
* cache: pages of tokens, (pages, page, heads, words) codes packed like the rows above
  (or four 8-bit codes per word), and per group of the head dimension a float32 pair
  (scale, zero), or the byte e per 32 values for microscaled blocks.  Row i of sequence s
  among the rows of a call (cu[s] <= row < cu[s+1]) is position start[s] + i, which lives
  in page table[s, position // page].
"""
import math

import torch

own = False

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


def listed():
    return [
        # one token's activations on their way into a 4-bit product: latency
        {"name": "round trip, one token", "op": "round_trip", "rows": 1, "cols": 4096, "ld": 4096, "x": "bf16", "y": "bf16"},
        # a ragged batch whose rows end inside a block, in a buffer with longer rows
        {"name": "round trip, ragged", "op": "round_trip", "rows": 1999, "cols": 11003, "ld": 11016, "x": "fp16", "y": "fp32"},
        # the largest layer's weights, quantised once and read back to compare
        {"name": "round trip, 49152x12288", "op": "round_trip", "rows": 49152, "cols": 12288, "ld": 12288, "x": "fp16", "y": "fp16"},
        # decoding: one token through a square projection
        {"name": "product, one token", "op": "product", "tokens": 1, "rows": 4096, "cols": 4096, "y": "bf16"},
        # decoding a small batch through the widest layer: the weights' bytes count
        {"name": "product, 16 tokens, widest", "op": "product", "tokens": 16, "rows": 12288, "cols": 49152, "y": "fp16"},
        # a ragged chunk of a prompt, columns that end inside a 128-column tile, full-precision output
        {"name": "product, ragged chunk", "op": "product", "tokens": 333, "rows": 11008, "cols": 4104, "y": "fp32"},
        # one sequence of the calibration length
        {"name": "product, 2048 tokens", "op": "product", "tokens": 2048, "rows": 13824, "cols": 5120, "y": "bf16"},
        # a large prefill batch
        {"name": "product, 8192 tokens", "op": "product", "tokens": 8192, "rows": 12288, "cols": 12288, "y": "bf16"},
        # one new token for each of 64 running sequences, 8-bit cache
        {"name": "append, one token each", "op": "append", "seqs": 64, "tokens": 64, "past": 4096, "heads": 8, "dim": 128, "page": 16,
         "kind": "grid", "bits": 8, "group": 0, "sym": False, "x": "bf16"},
        # prompts of several sequences written at once, microscaled cache
        {"name": "append, prompts", "op": "append", "seqs": 7, "tokens": 16384, "past": 100, "heads": 32, "dim": 128, "page": 64,
         "kind": "mx", "bits": 4, "group": 32, "sym": False, "x": "fp16"},
        # a few short sequences read back, a head dimension that is no power of two, pages of 24
        {"name": "read, short", "op": "read", "seqs": 3, "tokens": 300, "past": 40, "heads": 8, "dim": 80, "page": 24,
         "kind": "grid", "bits": 4, "group": 32, "sym": False, "x": "fp32"},
        # the whole context of 32 long sequences
        {"name": "read, long", "op": "read", "seqs": 32, "tokens": 131072, "past": 0, "heads": 8, "dim": 128, "page": 32,
         "kind": "grid", "bits": 4, "group": 64, "sym": False, "x": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["round_trip", "product", "product", "append", "read"])
    if op == "round_trip":
        cols = _log(rng, 32, 49152)
        rows = _log(rng, 1, min(49152, 49152 * 12288 // cols))
        return {"op": op, "rows": rows, "cols": cols, "ld": cols + rng.choice([0, 0, 1, 8]),
                "x": rng.choice(sorted(DT)), "y": rng.choice(["bf16", "fp32"])}
    if op == "product":
        cols = _log(rng, 32, 49152)
        rows = _log(rng, 16, min(49152, 49152 * 12288 // cols))
        tokens = _log(rng, 1, max(1, min(8192, 8192 * 12288 * 12288 // (rows * cols))))
        return {"op": op, "tokens": tokens, "rows": rows, "cols": cols, "y": rng.choice(sorted(DT))}
    heads, dim = rng.choice([1, 2, 5, 8, 16, 32]), rng.choice([64, 80, 96, 128, 192, 256])
    kind = rng.choice(["grid", "grid", "mx"])
    most = 131072 * 8 * 128 // (heads * dim)
    seqs = _log(rng, 1, 256)
    tokens = seqs if op == "append" and rng.random() < 0.5 else _log(rng, max(2, seqs), max(2, seqs, min(131072, most)))
    return {"op": op, "seqs": seqs, "tokens": tokens, "past": _log(rng, 1, 4096) - 1, "heads": heads, "dim": dim,
            "page": rng.choice([1, 16, 24, 32, 64, 128]), "kind": kind, "bits": 4 if kind == "mx" else rng.choice([4, 8]),
            "group": 32 if kind == "mx" else rng.choice([0, 32, 64, 128]), "sym": kind == "grid" and rng.random() < 0.3,
            "x": rng.choice(sorted(DT))}


# ------------------------------------------------------------------ the plain forms
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _cdiv(a, b):
    return -(-a // b)


def _pack(q, bits):
    """Codes (..., n) as int32 words of 32/bits codes each, lowest bits first."""
    per = 32 // bits
    q = q.to(torch.int64).reshape(*q.shape[:-1], q.shape[-1] // per, per)
    w = (q << (bits * torch.arange(per, device=q.device))).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _unpack(words, bits):
    per = 32 // bits
    q = (words.unsqueeze(-1) >> (bits * torch.arange(per, device=words.device, dtype=torch.int32))) & (2 ** bits - 1)
    return q.reshape(*words.shape[:-1], -1)


def _mx_codes(x):
    """4-bit codes and scale bytes of float32 values (..., 32 n), block by block: the scale is
    2^(floor(log2 of the largest magnitude) - 2), each value / scale goes to the nearest level (ties to
    the even code, beyond 6 to 6)."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    e = ((b.abs().amax(-1).contiguous().view(torch.int32) >> 23) - 2).clamp(min=0)
    y = b * ((254 - e) << 23).view(torch.float32).unsqueeze(-1)  # times 2^(127 - e)
    m = y.abs()
    i = (m > 0.25).to(torch.uint8)
    for border, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        i += (m >= border) if up else (m > border)
    q = i | (torch.signbit(y).to(torch.uint8) << 3)
    return q.reshape(x.shape), e.to(torch.uint8)


def _mx_values(q, e):
    """float32 values of codes (..., 32 n) and scale bytes (..., n)."""
    levels = torch.tensor(LEVELS + [-v for v in LEVELS], device=q.device)
    v = levels[q.long()].reshape(*e.shape, 32)
    return torch.ldexp(v, e.to(torch.int32).unsqueeze(-1) - 127).reshape(q.shape)


def _tile(e):
    """Scale bytes (rows, blocks) in 128x4 tiles, zero where there is no row or block."""
    r, k = e.shape
    t = torch.zeros(_cdiv(r, 128) * 128, _cdiv(k, 4) * 4, dtype=torch.uint8, device=e.device)
    t[:r, :k] = e
    return t.reshape(_cdiv(r, 128), 4, 32, _cdiv(k, 4), 4).permute(0, 3, 2, 1, 4).reshape(_cdiv(r, 128), _cdiv(k, 4), 32, 16).contiguous()


def _untile(t, r, k):
    a, b = t.shape[:2]
    return t.reshape(a, b, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(a * 128, b * 4)[:r, :k]


def _mx_rows(x):
    """The stored form of (rows, cols) values."""
    r, c = x.shape
    p = torch.zeros(r, _cdiv(c, 32) * 32, device=x.device)
    p[:, :c] = x
    q, e = _mx_codes(p)
    return _pack(q, 4), _tile(e)


def _mx_dense(codes, scales, cols):
    r, w = codes.shape
    return _mx_values(_unpack(codes, 4), _untile(scales, r, w // 4))[:, :cols]


def _grid_codes(x, bits, group, sym):
    """Codes (..., groups, g), scales and zeros (..., groups) of float32 values (..., dim): per group the
    min-max grid that contains 0, in float32 throughout."""
    dim = x.shape[-1]
    g = group if group > 0 else dim
    n = _cdiv(dim, g)
    p = torch.zeros(*x.shape[:-1], n * g, device=x.device)
    p[..., :dim] = x
    p = p.reshape(*x.shape[:-1], n, g)
    lo, hi = p.amin(-1).clamp(max=0), p.amax(-1).clamp(min=0)
    most = torch.full((), float(2 ** bits - 1), device=x.device)  # on the device: a division, not a product with 1/most
    if sym:
        m = torch.maximum(-lo, hi)
        m = torch.where(m == 0, torch.ones_like(m), m)
        s = (m + m) / most
        z = torch.full_like(s, 2.0 ** (bits - 1))
    else:
        flat = (lo == 0) & (hi == 0)
        lo, hi = torch.where(flat, -1.0, lo), torch.where(flat, 1.0, hi)
        s = (hi - lo) / most
        z = torch.round(-lo / s)
    q = (torch.round(p / s.unsqueeze(-1)) + z.unsqueeze(-1)).clamp(0, 2 ** bits - 1)
    return q, s, z


def _words(c):
    return _cdiv(c["dim"], 32) * 4 if c["kind"] == "mx" else _cdiv(c["dim"] * c["bits"], 32)


def _store(c, x, codes, grids, at):
    """Rows x (rows, heads, dim) into the cache's slots `at`."""
    x = x.float()
    dim, words = c["dim"], _words(c)
    if c["kind"] == "mx":
        p = torch.zeros(*x.shape[:-1], words * 8, device=x.device)
        p[..., :dim] = x
        q, e = _mx_codes(p)
        grids.reshape(-1, *grids.shape[2:])[at] = e
    else:
        q, s, z = _grid_codes(x, c["bits"], c["group"], c["sym"])
        grids.reshape(-1, *grids.shape[2:])[at] = torch.stack([s, z], -1)
        q = q.flatten(-2)[..., :dim]
        per = 32 // c["bits"]
        p = torch.zeros(*x.shape[:-1], words * per, device=x.device)
        p[..., :dim] = q
        q = p
    codes.reshape(-1, *codes.shape[2:])[at] = _pack(q, c["bits"])


def _load(c, codes, grids, at):
    dim = c["dim"]
    q = _unpack(codes.reshape(-1, *codes.shape[2:])[at], c["bits"])
    f = grids.reshape(-1, *grids.shape[2:])[at]
    if c["kind"] == "mx":
        return _mx_values(q, f)[..., :dim].to(DT[c["x"]])
    g = c["group"] if c["group"] > 0 else dim
    of = torch.arange(dim, device=q.device) // g
    return (f[..., 0][..., of] * (q[..., :dim].float() - f[..., 1][..., of])).to(DT[c["x"]])


def _slots(c, s):
    """The slot (page * page size + place in it) of every row of a call."""
    row = torch.arange(c["tokens"], device=s["cu"].device)
    seq = torch.searchsorted(s["cu"], row.to(torch.int32), right=True) - 1
    pos = s["start"][seq].long() + row - s["cu"][seq].long()
    return s["table"][seq, pos // c["page"]].long() * c["page"] + pos % c["page"]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _acts(shape, gen, dtype):
    """Activations: heavier tails than a normal's, and a few channels twenty times as large."""
    n = torch.randn(shape, generator=gen, device="cuda")
    n = n / (torch.rand(shape, generator=gen, device="cuda") * 0.8 + 0.2)
    big = 1 + 19.0 * (torch.rand(shape[-1], generator=gen, device="cuda") < 0.01)
    return (n * big).to(dtype)


def _lengths(c, seed):
    """How many rows each sequence has in this call, and how many it had before."""
    g = torch.Generator().manual_seed(seed)
    n, t = c["seqs"], c["tokens"]
    if n == t:
        new = [1] * n
    else:
        cuts = torch.sort(torch.randint(0, t + 1, (n - 1,), generator=g)).values.tolist()
        new = [b - a for a, b in zip([0] + cuts, cuts + [t])]
    return new, torch.randint(0, c["past"] + 1, (n,), generator=g).tolist()


def prepare(case, seed):
    c, gen = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "round_trip":
        x = torch.zeros(c["rows"], c["ld"], dtype=DT[c["x"]], device="cuda")
        x[:, :c["cols"]] = _acts((c["rows"], c["cols"]), gen, DT[c["x"]])
        s["x"] = x[:, :c["cols"]]
        s["codes"] = torch.zeros(c["rows"], _cdiv(c["cols"], 32) * 4, dtype=torch.int32, device="cuda")
        s["scales"] = torch.zeros(_cdiv(c["rows"], 128), _cdiv(c["cols"], 128), 32, 16, dtype=torch.uint8, device="cuda")
        s["y"] = torch.zeros(c["rows"], c["cols"], dtype=DT[c["y"]], device="cuda")
    elif c["op"] == "product":
        s["xc"], s["xs"] = _mx_rows(_acts((c["tokens"], c["cols"]), gen, torch.bfloat16).float())
        w = torch.empty(c["rows"], c["cols"], device="cuda").normal_(0, 0.02, generator=gen)
        s["wc"], s["ws"] = _mx_rows(w)
        s["y"] = torch.zeros(c["tokens"], c["rows"], dtype=DT[c["y"]], device="cuda")
    else:
        new, past = _lengths(c, seed)
        need = [_cdiv(p + n, c["page"]) for p, n in zip(past, new)]
        pages = sum(need) + 1
        table = torch.full((c["seqs"], max(1, _cdiv(c["past"] + c["tokens"], c["page"]))), -1, dtype=torch.int32)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        s["table"] = table.cuda()
        s["cu"] = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
        s["start"] = torch.tensor(past, dtype=torch.int32).cuda()
        h, d, dt = c["heads"], c["dim"], DT[c["x"]]
        g = 32 if c["kind"] == "mx" else c["group"] or d
        shape = (pages, c["page"], h, _cdiv(d, g))
        for n in ("k", "v"):
            s[n + "_codes"] = torch.zeros(pages, c["page"], h, _words(c), dtype=torch.int32, device="cuda")
            s[n + "_grids"] = torch.zeros(shape, dtype=torch.uint8, device="cuda") if c["kind"] == "mx" else torch.zeros(*shape, 2, device="cuda")
        kv = _acts((c["tokens"], 2, h, d), gen, dt)  # keys and values beside each other, as one projection leaves them
        if c["op"] == "append":
            s["k"], s["v"] = kv[:, 0], kv[:, 1]
        else:
            at = _slots(c, s)
            for i, n in enumerate(("k", "v")):
                _store(c, kv[:, i], s[n + "_codes"], s[n + "_grids"], at)
        s["k_out"], s["v_out"] = (torch.zeros(c["tokens"], h, d, dtype=dt, device="cuda") for _ in range(2))
    return s


# ------------------------------------------------------------------ one pass
def _own_run(s):
    from post_weight_quantization_20_b200 import kv_cache, mx
    c = s["case"]
    if c["op"] == "round_trip":
        mx.gptq_mx_quantize(s["x"], s["codes"], s["scales"])
        mx.gptq_mx_dequantize(s["codes"], s["scales"], s["y"])
        return s["y"]
    if c["op"] == "product":
        mx.gptq_mx_matmul(s["xc"], s["xs"], s["wc"], s["ws"], c["cols"], s["y"])
        return s["y"]
    cfg = kv_cache.make_cache_config(c["kind"], bits=c["bits"], group_size=c["group"], sym=c["sym"])
    cache = (s["k_codes"], s["k_grids"], s["v_codes"], s["v_grids"])
    if c["op"] == "append":
        kv_cache.gptq_cache_write(s["k"], s["v"], cfg, *cache, s["table"], s["cu"], s["start"])
    kv_cache.gptq_cache_read(cfg, *cache, s["table"], s["cu"], s["start"], s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


def run(state):
    if own:
        return _own_run(state)
    s, c = state, state["case"]
    if c["op"] == "round_trip":
        s["codes"], s["scales"] = _mx_rows(s["x"].float())
        return _mx_dense(s["codes"], s["scales"], c["cols"]).to(DT[c["y"]])
    if c["op"] == "product":
        return (_mx_dense(s["xc"], s["xs"], c["cols"]) @ _mx_dense(s["wc"], s["ws"], c["cols"]).T).to(DT[c["y"]])
    at = _slots(c, s)
    if c["op"] == "append":
        _store(c, s["k"], s["k_codes"], s["k_grids"], at)
        _store(c, s["v"], s["v_codes"], s["v_grids"], at)
    return _load(c, s["k_codes"], s["k_grids"], at), _load(c, s["v_codes"], s["v_grids"], at)


def work(case):
    c = case
    if c["op"] == "round_trip":
        n, blocks = c["rows"] * c["cols"], c["rows"] * _cdiv(c["cols"], 32)
        return {"bytes": n * (SIZE[c["x"]] + SIZE[c["y"]]) + 17 * blocks, "flops": 4 * n}
    if c["op"] == "product":
        blocks = _cdiv(c["cols"], 32)
        return {"bytes": 17 * blocks * (c["tokens"] + c["rows"]) + c["tokens"] * c["rows"] * SIZE[c["y"]],
                "flops": 2 * c["tokens"] * c["rows"] * c["cols"]}
    n = 2 * c["tokens"] * c["heads"]
    g = 32 if c["kind"] == "mx" else c["group"] or c["dim"]
    stored = n * (4 * _words(c) + _cdiv(c["dim"], g) * (1 if c["kind"] == "mx" else 8))
    rows = n * c["dim"] * SIZE[c["x"]]
    return {"bytes": stored + rows * (2 if c["op"] == "append" else 1), "flops": 4 * n * c["dim"]}


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_mx(x):
    """The value that each of x (rows, cols; float64) stands for after microscaled 4-bit rounding."""
    r, c = x.shape
    out = torch.empty_like(x)
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    for r0 in range(0, r, 4096):
        part = torch.nn.functional.pad(x[r0:r0 + 4096], (0, -c % 32)).unflatten(1, (-1, 32))
        top = part.abs().amax(2, keepdim=True)
        power = torch.frexp(top).exponent.double() - 3                   # floor(log2 top) - 2
        scale = torch.exp2(torch.where(top > 0, power.clamp(min=-127), -127.0))
        mag = (part.abs() / scale).clamp(max=6.0)
        up = torch.searchsorted(levels, mag.contiguous()).clamp(max=7)   # first level >= mag
        down = (up - 1).clamp(min=0)
        a, b = mag - levels[down], levels[up] - mag
        pick = torch.where((a < b) | ((a == b) & (down % 2 == 0)), down, up)
        out[r0:r0 + 4096] = (torch.copysign(levels[pick], part) * scale).flatten(1)[:, :c]
    return out


def _exact_rows(codes, scales, cols):
    """float64 values of stored rows, byte by byte: two codes to a byte, the scales through their address."""
    r = codes.shape[0]
    by = codes.contiguous().view(torch.uint8).long()
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=codes.device)
    sign = torch.tensor([1.0, -1.0], dtype=torch.float64, device=codes.device)
    v = torch.empty(r, 2 * by.shape[1], dtype=torch.float64, device=codes.device)
    v[:, 0::2] = levels[by & 7] * sign[(by >> 3) & 1]
    v[:, 1::2] = levels[(by >> 4) & 7] * sign[by >> 7]
    row = torch.arange(r, device=codes.device)[:, None]
    k = torch.arange(v.shape[1] // 32, device=codes.device)[None, :]
    byte = ((row // 128) * scales.shape[1] + k // 4) * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + k % 4
    v = v.unflatten(1, (-1, 32)) * torch.exp2(scales.reshape(-1)[byte].double() - 127).unsqueeze(2)
    return v.flatten(1)[:, :cols]


def _exact_grid(x, bits, group, sym):
    """The value that each of x (..., dim; float64) stands for on its group's grid; the scale, the quotient
    and the zero are 32-bit numbers by definition, each rounded once from 64 bits."""
    out, step = torch.empty_like(x), group or x.shape[-1]
    r32 = lambda t: t.float().double()  # noqa: E731
    for j in range(0, x.shape[-1], step):
        part = x[..., j:j + step]
        lo = part.amin(-1, keepdim=True).clamp(max=0)
        hi = part.amax(-1, keepdim=True).clamp(min=0)
        none = (hi - lo) == 0
        if sym:
            hi = torch.maximum(hi, -lo)
            hi = torch.where(none, 1.0, hi)
            scale, zero = r32(r32(2 * hi) / (2 ** bits - 1)), 2.0 ** (bits - 1)
        else:
            lo, hi = torch.where(none, -1.0, lo), torch.where(none, 1.0, hi)
            scale = r32(r32(hi - lo) / (2 ** bits - 1))
            zero = torch.round(r32(-lo / scale))
        code = (torch.round(r32(part / scale)) + zero).clamp(0, 2 ** bits - 1)
        out[..., j:j + step] = scale * (code - zero)
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "round_trip":
        return _exact_mx(s["x"].double())
    if c["op"] == "product":
        return _exact_rows(s["xc"], s["xs"], c["cols"]) @ _exact_rows(s["wc"], s["ws"], c["cols"]).T
    if c["op"] == "append":
        k, v = s["k"].double(), s["v"].double()
    else:  # what was stored, from the same draw as prepare()'s
        kv = _acts((c["tokens"], 2, c["heads"], c["dim"]), _gen(seed), DT[c["x"]]).double()
        k, v = kv[:, 0], kv[:, 1]
    if c["kind"] == "mx":
        return tuple(_exact_mx(t.reshape(-1, c["dim"])).reshape(t.shape) for t in (k, v))
    return tuple(_exact_grid(t, c["bits"], c["group"], c["sym"]) for t in (k, v))
