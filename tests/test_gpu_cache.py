"""The paged low-bit cache on the GPU against the float64 definition (oracle/lowbit_ref.py).

A grid's decisions are float32 by definition, so codes, scales, zeros and scale bytes must be
equal bit for bit, and what is read back is s (code - z) or level * 2^(e-127) formed in
float32 (code - z is exact, one product) and rounded once to its type: equal as well."""
import numpy as np
import pytest
import torch

from oracle import gptq_ref as o
from oracle import lowbit_ref as L
from post_weight_quantization_20_b200 import gptq as G
from post_weight_quantization_20_b200 import kv_cache as KV
from tests.guards import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.float16, torch.bfloat16]
CONFIGS = [("grid", 4, 0, False), ("grid", 4, 32, False), ("grid", 4, 64, True), ("grid", 4, 128, False),
           ("grid", 8, 0, False), ("grid", 8, 0, True), ("grid", 8, 64, False), ("mx", 4, 32, False)]


def _define(x, kind, bits, group, sym):
    """(packed words, grids, float32 values) of x (rows, heads, dim)."""
    n, h, d = x.shape
    if kind == "mx":
        c, e = L.mx_quantize(x.reshape(n * h, d))
        vals = L.mx_values(c, e)[:, :d].astype(np.float32)
        return (o.pack(c.astype(np.int64), 4).reshape(n, h, -1), e.reshape(n, h, -1),
                vals.reshape(n, h, d))
    c, s, z = L.grid_quantize(x, bits, group, sym)
    g = group if group > 0 else d
    of = np.arange(d) // g
    with np.errstate(invalid="ignore"):
        vals = s[..., of] * (np.float32(c) - z[..., of])         # float32, one rounding
    return (o.pack(c.reshape(n * h, d), bits).reshape(n, h, -1), np.stack([s, z], -1), vals)


class Call:
    """Rows of a few sequences (one of them empty, `extra` rows of padding behind the last)."""

    def __init__(self, new, past, page, seed, extra=0, spare=2):
        rng = np.random.default_rng(seed)
        need = [-(-(p + n) // page) for p, n in zip(past, new)]
        self.pages, self.page, self.rows = sum(need) + spare, page, sum(new) + extra
        self.table = np.full((len(new), max(need) + 1), -1, np.int32)
        order, at = rng.permutation(self.pages).astype(np.int32), 0
        for i, k in enumerate(need):
            self.table[i, :k] = order[at:at + k]
            at += k
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.start = np.array(past, np.int32)
        self.slots = L.slots(self.rows, self.table, self.cu, self.start, page, self.pages)

    def args(self):
        return tuple(torch.from_numpy(a).to(DEV) for a in (self.table, self.cu, self.start))


def _pools(cfg, call, heads, dim, guarded=True):
    words = KV._words(cfg, dim)
    shape, dt = KV._grid_shape(cfg, call.pages, call.page, heads, dim)
    cs = (call.pages, call.page, heads, words)
    return [Guarded(s, d, DEV, fill=torch.full(s, f, dtype=d)) for _ in range(2)
            for s, d, f in ((cs, torch.int32, 0x11111111), (shape, dt, 7))]


def _input(rows, heads, dim, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, heads, dim)) * np.exp2(rng.integers(-4, 5, (rows, heads, 1)))
    x[rng.random(x.shape) < 0.02] *= 20
    return torch.from_numpy(x).to(dtype)


def _bits(a):
    return np.ascontiguousarray(a).view(np.uint8)


@pytest.mark.parametrize("conf", CONFIGS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("heads,dim", [(1, 64), (8, 128), (3, 80), (5, 256), (2, 8), (1, 200)])
@pytest.mark.parametrize("dtype", TYPES)
def test_write_and_read_are_the_definition(conf, heads, dim, dtype):
    call = Call([1, 0, 13, 40, 1], [0, 5, 20, 3, 31], 16, seed=heads * dim, extra=3)
    cfg = KV.make_cache_config(*conf)
    # keys and values beside each other in one buffer, with a spare head between
    fused = torch.full((call.rows, 2 * heads + 1, dim), float("nan"), dtype=dtype)
    k, v = _input(call.rows, heads, dim, dtype, 1), _input(call.rows, heads, dim, dtype, 2)
    fused[:, :heads], fused[:, heads + 1:] = k, v
    fused[-3:] = float("nan")                               # padding rows are ignored
    fused = fused.to(DEV)
    K, V = fused[:, :heads], fused[:, heads + 1:]
    pools = _pools(cfg, call, heads, dim)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    KV.gptq_cache_write(K, V, cfg, *(p.t for p in pools), *call.args(), st)
    assert int(st) == 0 and all(p.intact() for p in pools)
    live = call.slots >= 0
    slots = call.slots[live]
    untouched = np.setdiff1d(np.arange(call.pages * call.page), slots)
    want = []
    for x, codes, grids in ((k, *pools[:2]), (v, *pools[2:])):
        words, g, vals = _define(x.double().numpy()[live], *conf)
        want.append(vals)
        c = codes.t.cpu().numpy().reshape(-1, heads, words.shape[-1])
        np.testing.assert_array_equal(c[slots].view(np.uint32), words)
        assert (c[untouched] == 0x11111111).all()
        gr = grids.t.cpu().numpy().reshape(-1, *g.shape[1:])
        np.testing.assert_array_equal(_bits(gr[slots]), _bits(g.astype(gr.dtype)))
        assert (gr[untouched] == 7).all()
    for dt in TYPES:
        outs = [Guarded((call.rows, heads, dim + 8), dt, DEV,
                        fill=torch.full((call.rows, heads, dim + 8), 7.0, dtype=dt)) for _ in range(2)]
        KV.gptq_cache_read(cfg, *(p.t for p in pools), *call.args(), *(t.t[..., :dim] for t in outs), st)
        assert int(st) == 0
        for out, vals in zip(outs, want):
            got = out.t.cpu()
            ref = torch.from_numpy(vals).to(dt)
            assert torch.equal(got[:len(slots), :, :dim], ref) and out.intact()
            assert (got[..., dim:] == 7.0).all() and (got[len(slots):] == 7.0).all()


def _check(call, conf, pools, rows, read):
    """The cache's live slots and what `read` gave hold the definition of the rows (K, V)."""
    live = call.slots >= 0
    for x, codes, grids, got in zip(rows, pools[::2], pools[1::2], read):
        words, g, vals = _define(x.double().cpu().numpy()[live], *conf)
        c = codes.t.cpu().numpy().reshape(-1, *words.shape[1:])[call.slots[live]]
        np.testing.assert_array_equal(c.view(np.uint32), words)
        gr = grids.t.cpu().numpy().reshape(-1, *g.shape[1:])[call.slots[live]]
        np.testing.assert_array_equal(_bits(gr), _bits(g.astype(gr.dtype)))
        assert torch.equal(got.cpu()[torch.from_numpy(live)], torch.from_numpy(vals).to(got.dtype))
    assert all(p.intact() for p in pools)


LAYOUTS = {
    # (rows, heads, dim) views of a buffer of `rows * (heads + 1) * (dim + 8) + 1` elements
    "off 16 bytes": lambda b, n, h, d: b[1:1 + n * h * d].view(n, h, d),
    "odd rows": lambda b, n, h, d: b[:n * (h * d + 1)].view(n, h * d + 1)[:, :h * d].unflatten(1, (h, d)),
    "head-major": lambda b, n, h, d: b[:n * h * d].view(h, n, d).transpose(0, 1),
    "head-major, padded, off 16 bytes":
        lambda b, n, h, d: b[1:1 + n * h * (d + 1)].view(h, n, d + 1)[..., :d].transpose(0, 1),
}


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("conf", [CONFIGS[1], CONFIGS[2], CONFIGS[4], CONFIGS[7]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("heads,dim", [(3, 80), (8, 128)])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_other_alignments_and_orders(layout, conf, heads, dim, dtype):
    # values and keys of layouts of their own, written from one and read into the other
    call = Call([1, 30, 9], [3, 0, 20], 16, seed=dim)
    n, cfg = call.rows, KV.make_cache_config(*conf)
    size = n * (heads + 1) * (dim + 8) + 1

    def views(dt, swap):
        a, b = (Guarded((size,), dt, DEV, fill=torch.full((size,), 7.0, dtype=dt)) for _ in range(2))
        odd, even = LAYOUTS[layout](a.t, n, heads, dim), b.t[:n * heads * dim].view(n, heads, dim)
        return (a, b), ((even, odd) if swap else (odd, even))

    _, (K, V) = views(dtype, False)
    K.copy_(_input(n, heads, dim, dtype, 1))
    V.copy_(_input(n, heads, dim, dtype, 2))
    pools = _pools(cfg, call, heads, dim)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    KV.gptq_cache_write(K, V, cfg, *(p.t for p in pools), *call.args(), st)
    for swap in (False, True):
        bufs, out = views(dtype, swap)
        KV.gptq_cache_read(cfg, *(p.t for p in pools), *call.args(), *out, st)
        _check(call, conf, pools, (K, V), out)
        # nothing beside the rows is written
        for t in out:
            t.fill_(7.0)
        assert all(b.intact() and (b.t == 7.0).all() for b in bufs)
    assert int(st) == 0


@pytest.mark.parametrize("conf", CONFIGS[1:4] + CONFIGS[6:], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("heads,dim", [(2, 264), (3, 512), (1, 4096), (5, 1000)])
@pytest.mark.parametrize("dtype", TYPES)
def test_wide_heads(conf, heads, dim, dtype):
    # up to the largest head; a row of more lanes than a CTA among them
    call = Call([1, 0, 18], [3, 0, 20], 16, seed=dim)
    n, cfg = call.rows, KV.make_cache_config(*conf)
    K, V = (_input(n, heads, dim, dtype, i).to(DEV) for i in range(2))
    pools = _pools(cfg, call, heads, dim)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    KV.gptq_cache_write(K, V, cfg, *(p.t for p in pools), *call.args(), st)
    out = torch.zeros_like(K), torch.zeros_like(V)
    KV.gptq_cache_read(cfg, *(p.t for p in pools), *call.args(), *out, st)
    _check(call, conf, pools, (K, V), out)
    assert int(st) == 0


@pytest.mark.parametrize("page", [1, 7, 24, 128])
@pytest.mark.parametrize("conf", [CONFIGS[1], CONFIGS[4], CONFIGS[7]], ids=lambda c: "-".join(map(str, c)))
def test_rows_one_by_one_equal_a_whole_prompt(conf, page):
    # a prompt of each length appended at once, and the same rows a token per sequence and call
    cfg, heads, dim = KV.make_cache_config(*conf), 2, 96
    lens = [9, 30, 1, 17]
    call = Call(lens, [0, 0, 0, 0], page, seed=page)
    k = _input(sum(lens), heads, dim, torch.float16, 3).to(DEV)
    a, b = (KV.KVCache.alloc(cfg, call.pages, page, heads, dim) for _ in range(2))
    table, cu, start = call.args()
    a.write(k, -k, table, cu, start)
    for i in range(max(lens)):
        has = [i < n for n in lens]
        rows = torch.tensor([int(call.cu[s]) + i for s in range(4) if has[s]], device=DEV)
        cu1 = torch.tensor(np.concatenate([[0], np.cumsum(has)]), dtype=torch.int32, device=DEV)
        st1 = torch.full((4,), i, dtype=torch.int32, device=DEV)
        x = k[rows]
        b.write(x, -x, table, cu1, st1)
    for n in ("k_codes", "k_grids", "v_codes", "v_grids"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    K, V = a.read(table, cu, start, sum(lens), torch.float32)
    K2, V2 = b.read(table, cu, start, sum(lens), torch.float32)
    assert torch.equal(K, K2) and torch.equal(V, V2)
    # a part of each sequence, from the middle on
    cu2 = torch.tensor([0, 4, 24, 24, 30], dtype=torch.int32, device=DEV)
    st2 = torch.tensor([5, 10, 0, 11], dtype=torch.int32, device=DEV)
    P, _ = a.read(table, cu2, st2, 30, torch.float32)
    want = torch.cat([K[5:9], K[9 + 10:9 + 30], K[40 + 11:40 + 17]])
    assert torch.equal(P, want)


@pytest.mark.parametrize("conf", [CONFIGS[0], CONFIGS[2], CONFIGS[4], CONFIGS[7]], ids=lambda c: "-".join(map(str, c)))
def test_values_at_the_edges(conf):
    f = np.float32
    x = np.zeros((14, 1, 32), dtype=f)
    x[1] = 5.0                                                # one sign only: the grid still holds 0
    x[2] = -5.0
    x[3, 0, 3] = np.nan
    x[4, 0, 9] = np.inf
    x[5, 0, 31] = -np.inf
    x[6, 0, :2] = [3e38, -3e38]                               # range beyond fp32
    x[7, 0, :2] = [2.0 ** -149, 0]                            # underflows
    x[8, 0, :3] = [1e-40, -1e-40, 5e-41]
    x[9, 0] = np.linspace(-1, 1, 32)
    x[10, 0] = np.arange(32) * 0.5                            # halves: ties on the 8-bit grid's quotients
    x[11, 0] = (np.arange(32) - 16) * f(1 / 3)
    x[12, 0] = -0.0
    x[13, 0, :4] = [1e30, -1e-30, 1e29, -1e30]
    cfg = KV.make_cache_config(*conf)
    words, g, vals = _define(x.astype(np.float64), *conf)
    call = Call([14], [0], 16, 0)
    pool = KV.KVCache.alloc(cfg, call.pages, 16, 1, 32)
    X = torch.from_numpy(x).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pool.write(X, X, *call.args(), st)
    assert int(st) == G.GPTQ_ERR_NONFINITE
    c = pool.k_codes.cpu().numpy().reshape(-1, 1, words.shape[-1])[call.slots]
    np.testing.assert_array_equal(c.view(np.uint32), words)
    K, V = pool.read(*call.args(), 14, torch.float32)
    for got in (K.cpu().numpy(), V.cpu().numpy()):
        np.testing.assert_array_equal(np.isnan(got), np.isnan(vals))
        np.testing.assert_array_equal(np.nan_to_num(got, nan=0.0), np.nan_to_num(vals, nan=0.0))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("conf", [CONFIGS[1], CONFIGS[2], CONFIGS[4], CONFIGS[7]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("order", ["near", "mixed"])
def test_every_16_bit_value(dtype, conf, order):
    # every bit pattern once, in groups of neighbours and of far-apart magnitudes
    bits = np.arange(65536, dtype=np.uint16)
    if order == "mixed":
        bits = np.random.default_rng(0).permutation(bits)
    t = torch.from_numpy(bits.view(np.int16)).view(dtype).reshape(512, 1, 128)
    with np.errstate(all="ignore"):
        words, g, vals = _define(t.double().numpy(), *conf)
    call = Call([512], [0], 64, 0)
    pool = KV.KVCache.alloc(KV.make_cache_config(*conf), call.pages, 64, 1, 128)
    pool.write(t.to(DEV), t.to(DEV), *call.args())
    c = pool.k_codes.cpu().numpy().reshape(-1, 1, words.shape[-1])[call.slots]
    np.testing.assert_array_equal(c.view(np.uint32), words)
    K, V = pool.read(*call.args(), 512, torch.float32)
    for got in (K.cpu().numpy(), V.cpu().numpy()):
        np.testing.assert_array_equal(np.isnan(got), np.isnan(vals))
        np.testing.assert_array_equal(np.nan_to_num(got, nan=0.0), np.nan_to_num(vals, nan=0.0))


@pytest.mark.parametrize("power", [-95, -60, -1, 40, 88])
@pytest.mark.parametrize("sym", [False, True])
@pytest.mark.parametrize("bits", [4, 8])
def test_quotients_across_the_range_of_scales(bits, sym, power):
    # ranges from below to above those that the kernel's products hold (2^-90 .. 2^90), among
    # them ones whose width is a rounding away from a power of two
    rng = np.random.default_rng([bits, power + 200])
    x = (rng.standard_normal((300, 2, 64)) * 2.0 ** power).astype(np.float32)
    x[:, 0] *= np.float32(1) + np.float32(2.0 ** -23)
    x[::3] = np.rint(x[::3] / np.float32(2.0 ** (power - 4))) * np.float32(2.0 ** (power - 4))
    conf = ("grid", bits, 32, sym)
    with np.errstate(all="ignore"):
        words, g, _ = _define(x.astype(np.float64), *conf)
    call = Call([300], [0], 64, 0)
    pool = KV.KVCache.alloc(KV.make_cache_config(*conf), call.pages, 64, 2, 64)
    X = torch.from_numpy(x).to(DEV)
    pool.write(X, X, *call.args())
    c = pool.k_codes.cpu().numpy().reshape(-1, 2, words.shape[-1])[call.slots]
    np.testing.assert_array_equal(c.view(np.uint32), words)
    gr = pool.v_grids.cpu().numpy().reshape(-1, 2, 2, 2)[call.slots]
    np.testing.assert_array_equal(gr, g)


def test_rounding_near_ties_takes_the_exact_quotient():
    # values a few float32 steps around every half step of their group's 8-bit grid
    rng = np.random.default_rng(0)
    x = np.zeros((400, 4, 128), dtype=np.float32)
    for r in range(400):
        for h in range(4):
            lo, hi = -rng.random() * 2 - 0.1, rng.random() * 2 + 0.1
            s = np.float32(np.float32(np.float32(hi) - np.float32(lo)) / np.float32(255))
            z = np.rint(np.float32(-np.float32(lo) / s))
            k = rng.integers(-int(z) + 1, 255 - int(z), 126)
            t = ((k + 0.5) * np.float64(s)).astype(np.float32)
            x[r, h, :126] = np.clip(t + rng.integers(-3, 4, 126) * np.spacing(t), np.float32(lo), np.float32(hi))
            x[r, h, 126:] = lo, hi
    conf = ("grid", 8, 0, False)
    words, g, _ = _define(x.astype(np.float64), *conf)
    call = Call([400], [0], 64, 0)
    pool = KV.KVCache.alloc(KV.make_cache_config(*conf), call.pages, 64, 4, 128)
    X = torch.from_numpy(x).to(DEV)
    pool.write(X, X, *call.args())
    c = pool.v_codes.cpu().numpy().reshape(-1, 4, 32)[call.slots]
    np.testing.assert_array_equal(c.view(np.uint32), words)


@pytest.mark.parametrize("dtype", TYPES)
def test_read_every_code_and_scale(dtype):
    # formed in fp32 (6 * 2^127 overflows there), then rounded once
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    e = np.arange(256, dtype=np.uint8)[:, None]
    cfg = KV.make_cache_config("mx")
    pool = KV.KVCache.alloc(cfg, 1, 256, 1, 32)
    for c, g in ((pool.k_codes, pool.k_grids), (pool.v_codes, pool.v_grids)):
        c.copy_(torch.from_numpy(o.pack(codes.astype(np.int64), 4).view(np.int32)).reshape(c.shape))
        g.copy_(torch.from_numpy(e).reshape(g.shape))
    i32 = dict(dtype=torch.int32, device=DEV)
    K, V = pool.read(torch.zeros(1, 1, **i32), torch.tensor([0, 256], **i32), torch.zeros(1, **i32),
                     256, dtype)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(L.mx_values(codes, e).astype(np.float32)).to(dtype)[:, None]
    for got in (K.cpu(), V.cpu()):
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


def test_bad_positions_and_pages_are_left_out():
    # negative starts, positions past the table, pages that do not exist: those rows are left
    # out and reported, the others are done
    call = Call([4, 4, 4, 4], [0, 0, 0, 0], 4, 1)
    call.table[1, 0] = call.pages
    call.table[2, 0] = -5
    call.start[3] = -2
    call.slots = L.slots(16, call.table, call.cu, call.start, 4, call.pages)
    assert (call.slots[4:] == -2).all() and (call.slots[:4] >= 0).all()
    cfg = KV.make_cache_config("grid", 8, 0)
    pools = _pools(cfg, call, 2, 64)
    X = _input(16, 2, 64, torch.float32, 0).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    KV.gptq_cache_write(X, X, cfg, *(p.t for p in pools), *call.args(), st)
    assert int(st) == G.GPTQ_ERR_INVALID_ARG and all(p.intact() for p in pools)
    c = pools[0].t.cpu().numpy().reshape(-1, 2, 16)
    rest = np.setdiff1d(np.arange(len(c)), call.slots[:4])
    assert (c[rest] == 0x11111111).all() and not (c[call.slots[:4]] == 0x11111111).all()
    st.zero_()
    K = torch.full((16, 2, 64), 7.0, device=DEV)
    V = K.clone()
    KV.gptq_cache_read(cfg, *(p.t for p in pools), *call.args(), K, V, st)
    assert int(st) == G.GPTQ_ERR_INVALID_ARG
    assert (K[4:] == 7.0).all() and (V[4:] == 7.0).all() and not (K[:4] == 7.0).any()
    # past the table's width
    far = torch.tensor([4 * call.table.shape[1] - 1] * 4, dtype=torch.int32, device=DEV)
    table, cu, _ = call.args()
    st.zero_()
    KV.gptq_cache_read(cfg, *(p.t for p in pools), table, cu, far, K, V, st)
    assert int(st) == G.GPTQ_ERR_INVALID_ARG
    # an empty cache and an empty table have no page at all
    none = KV.KVCache.alloc(cfg, 0, 4, 2, 64)
    st.zero_()
    none.write(X, X, *call.args(), st)
    none.write(X, X, torch.empty(4, 0, dtype=torch.int32, device=DEV), cu, far, st)
    assert int(st) == G.GPTQ_ERR_INVALID_ARG


def test_many_sequences_and_empty_calls():
    rng = np.random.default_rng(2)
    new = rng.integers(0, 4, 700).tolist()
    call = Call(new, rng.integers(0, 50, 700).tolist(), 16, 5)
    conf = ("grid", 4, 64, False)
    cfg = KV.make_cache_config(*conf)
    pool = KV.KVCache.alloc(cfg, call.pages, 16, 1, 128)
    X = _input(call.rows, 1, 128, torch.bfloat16, 4)
    pool.write(X.to(DEV), -X.to(DEV), *call.args())
    K, V = pool.read(*call.args(), call.rows, torch.float32)
    np.testing.assert_array_equal(K.cpu().numpy(), _define(X.double().numpy(), *conf)[2])
    np.testing.assert_array_equal(V.cpu().numpy(), _define(-X.double().numpy(), *conf)[2])
    n = G.gptq_launch_count()
    pool.write(X[:0].to(DEV), X[:0].to(DEV), *call.args())
    i32 = dict(dtype=torch.int32, device=DEV)
    pool.read(torch.empty(0, 3, **i32), torch.zeros(1, **i32), torch.empty(0, **i32), 5)
    assert G.gptq_launch_count() == n


def test_slots_past_32_bit_offsets():
    # 4.5 GB of codes per side: the last page's words lie past 2^32 bytes and 2^30 words
    cfg, heads, dim, page = KV.make_cache_config("grid", 8, 0), 8, 128, 128
    pages = 4_500_000_000 // (page * heads * dim)
    pool = KV.KVCache.alloc(cfg, pages, page, heads, dim)
    X = _input(6, heads, dim, torch.bfloat16, 9).to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.tensor([[0, pages - 1]], **i32)
    cu, start = torch.tensor([0, 6], **i32), torch.tensor([page - 3], **i32)
    pool.write(X, -X, table, cu, start)
    K, V = pool.read(table, cu, start, 6, torch.float32)
    want = _define(X.double().cpu().numpy(), "grid", 8, 0, False)[2]
    np.testing.assert_array_equal(K.cpu().numpy(), want)
    assert int(pool.k_codes[pages - 1, 3:].count_nonzero()) == 0
    assert int(pool.k_codes[1:pages - 1].count_nonzero()) == 0
    assert int(pool.v_codes[pages - 1, :3].count_nonzero()) > 0


def test_graph_replay_with_growing_sequences():
    # one decoding step captured: a token of each sequence is appended and the whole context
    # read; lengths live on the device and grow between replays
    cfg, heads, dim = KV.make_cache_config("mx"), 4, 64
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.arange(8, **i32).reshape(2, 4)
    pool = KV.KVCache.alloc(cfg, 8, 4, heads, dim)
    X = torch.randn(2, heads, dim, device=DEV)
    one, start = torch.tensor([0, 1, 2], **i32), torch.tensor([0, 3], **i32)
    cu, zero = torch.zeros(3, **i32), torch.zeros(2, **i32)
    K, V = (torch.zeros(32, heads, dim, device=DEV) for _ in range(2))
    args = (cfg, pool.k_codes, pool.k_grids, pool.v_codes, pool.v_grids)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pool.write(X, -X, table, one, start)
        KV.gptq_cache_read(*args, table, cu, zero, K, V)
        start.add_(1)
    seen = [[], []]
    pool.k_codes.zero_()
    start.copy_(torch.tensor([0, 0], **i32))
    for step in range(9):
        X.copy_(torch.randn(2, heads, dim, generator=torch.Generator().manual_seed(step)))
        for s in range(2):
            seen[s].append(_define(X[s:s + 1].double().cpu().numpy(), "mx", 4, 32, False)[2])
        cu.copy_(torch.tensor([0, step + 1, 2 * step + 2], **i32))
        g.replay()
        torch.cuda.synchronize()
        want = np.concatenate(seen[0] + seen[1])
        np.testing.assert_array_equal(K[:2 * step + 2].cpu().numpy(), want)
        np.testing.assert_array_equal(V[:2 * step + 2].cpu().numpy(), -want)


@pytest.mark.parametrize("rows", [2, 300, 6000])
def test_calls_back_to_back_see_each_others_results(rows):
    # each call starts while the one before it drains; the same slots are rewritten again and again
    call = Call([rows], [3], 16, 1)
    cfg = KV.make_cache_config("grid", 4, 64)
    pool = KV.KVCache.alloc(cfg, call.pages, 16, 8, 128)
    args = call.args()
    xs = [_input(rows, 8, 128, torch.bfloat16, i).to(DEV) for i in range(3)]
    want, negs = [], [-x for x in xs]
    for x in xs:
        pool.write(x, -x, *args)
        torch.cuda.synchronize()
        want.append(pool.read(*args, rows, torch.float32))
        torch.cuda.synchronize()
    outs = [[torch.zeros(rows, 8, 128, device=DEV) for _ in range(2)] for _ in range(20)]
    arrays = (pool.k_codes, pool.k_grids, pool.v_codes, pool.v_grids)
    torch.cuda.synchronize()
    for i, o2 in enumerate(outs):
        KV.gptq_cache_write(xs[i % 3], negs[i % 3], cfg, *arrays, *args)
        KV.gptq_cache_read(cfg, *arrays, *args, *o2)
    torch.cuda.synchronize()
    for i, (K, V) in enumerate(outs):
        assert torch.equal(K, want[i % 3][0]) and torch.equal(V, want[i % 3][1]), i


def test_two_caches_on_two_streams():
    call = Call([50, 30], [0, 0], 16, 7)
    pools, xs = [], []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, conf in enumerate((("grid", 4, 32, False), ("grid", 8, 0, False))):
        pools.append((conf, KV.KVCache.alloc(KV.make_cache_config(*conf), call.pages, 16, 8, 128)))
        xs.append(_input(80, 8, 128, torch.float16, i).to(DEV))
    args = call.args()
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for (conf, pool), x, s in zip(pools, xs, streams):
            pool.write(x, x, *args, stream=s)
            outs.append((conf, x, pool.read(*args, 80, torch.float32, stream=s)))
    torch.cuda.synchronize()
    for conf, x, (K, V) in outs:
        want = _define(x.double().cpu().numpy(), *conf)[2]
        np.testing.assert_array_equal(K.cpu().numpy(), want)
        np.testing.assert_array_equal(V.cpu().numpy(), want)


@pytest.mark.parametrize("conf", [CONFIGS[4], CONFIGS[7]], ids=lambda c: "-".join(map(str, c)))
def test_a_layer_runs_from_activations_to_the_cache_and_back(conf):
    # prompts, then single tokens: activations are quantised, multiplied by 4-bit weights into
    # keys and values beside the queries, appended where they lie and read back; every step
    # equals the definitions applied to what it was given
    from post_weight_quantization_20_b200 import mx as MX
    heads, dim, cols, page = 2, 64, 1000, 16
    gen = torch.Generator(device=DEV).manual_seed(1)
    w = MX.mx_quantize(torch.randn(6 * heads * dim // 2, cols, generator=gen, device=DEV).half() * 0.03)
    wv = L.mx_values(*L.mx_quantize(MX.mx_dequantize(w).double().cpu().numpy()))[:, :cols]
    cfg = KV.make_cache_config(*conf)
    lens = [20, 5, 33]
    call = Call([n + 4 for n in lens], [0, 0, 0], page, 3)
    table = torch.from_numpy(call.table).to(DEV)
    cache = KV.KVCache.alloc(cfg, call.pages, page, heads, dim)
    i32 = dict(dtype=torch.int32, device=DEV)
    kept = [[], [], []]
    have = [0, 0, 0]
    for step in range(5):
        new = lens if step == 0 else [1, 1, 1]
        X = torch.randn(sum(new), cols, generator=gen, device=DEV).bfloat16()
        Y = MX.mx_linear(X, w)                                   # (rows, (q, k, v) heads * dim)
        qx = L.mx_values(*L.mx_quantize(X.double().cpu().numpy()))[:, :cols]
        want, S = qx @ wv.T, np.abs(qx) @ np.abs(wv).T
        bound = 50 * 2.0 ** -23 * S
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)       # rounded to bf16: half a step
        assert np.all(np.abs(Y.double().cpu().numpy() - want) <= bound)
        K, V = Y.view(len(Y), 3, heads, dim)[:, 1], Y.view(len(Y), 3, heads, dim)[:, 2]
        cu = torch.tensor([0, *np.cumsum(new)], **i32)
        cache.write(K, V, table, cu, torch.tensor(have, **i32))
        at = 0
        for s, n in enumerate(new):
            kept[s].append((K[at:at + n].double().cpu().numpy(), V[at:at + n].double().cpu().numpy()))
            at += n
            have[s] += n
        total = torch.tensor([0, *np.cumsum(have)], **i32)
        k, v = cache.read(table, total, torch.zeros(3, **i32), sum(have), torch.float32)
        for got, i in ((k, 0), (v, 1)):
            rows = np.concatenate([r[i] for s in kept for r in s])
            np.testing.assert_array_equal(got.cpu().numpy(), _define(rows, *conf)[2])
