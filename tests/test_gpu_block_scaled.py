"""Microscaled 4-bit rows on the GPU against the float64 definition (oracle/lowbit_ref.py).

Quantisation is exact by definition, so codes and scales must be equal bit for bit, and
read-back must be the definition's value rounded once.  The product's bound: products of
codes and scales are exact; a 64-column MMA and each of its additions to the running sum may
cut the sum to 24 bits by truncation, 2^-23 of at most S = sum |x w| each, twice per step;
joining the splits of a long K adds at most one rounding per split; the result is rounded
once more to its type, half a step eps/2."""
import numpy as np
import pytest
import torch

from oracle import gptq_ref as o
from oracle import lowbit_ref as L
from post_weight_quantization_20_b200 import gptq as G
from post_weight_quantization_20_b200 import mx as MX
from tests.guards import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def _values(R, C, dtype, seed):
    """Values over many binades, exact in dtype, as a torch tensor and in float64."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, C)) * np.exp2(rng.integers(-6, 7, (R, 1)))
    x[rng.random((R, C)) < 0.05] = 0.0
    t = torch.from_numpy(x).to(dtype)
    return t, t.double().numpy()


def _stored(R, C, seed, e_lo=120, e_hi=131):
    """A random stored form: tensors on the device, and its float64 values."""
    rng = np.random.default_rng(seed)
    nb = -(-C // 32)
    codes = rng.integers(0, 16, (R, nb * 32)).astype(np.uint8)
    codes[:, C:] = 0
    e = rng.integers(e_lo, e_hi, (R, nb)).astype(np.uint8)
    return (*_device(codes, e, C), L.mx_values(codes, e)[:, :C])


def _device(codes, e, C, fill=0):
    R = codes.shape[0]
    words = torch.from_numpy(o.pack(codes.astype(np.int64), 4).view(np.int32)).to(DEV)
    scales = torch.from_numpy(L.mx_tile(e, fill)).reshape(MX.mx_scale_shape(R, C)).to(DEV)
    return words, scales


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("R,C,pad", [(1, 1, 0), (1, 32, 0), (3, 31, 1), (5, 33, 3), (128, 128, 0),
                                     (129, 1100, 4), (300, 1000, 8), (2, 5000, 0), (33, 4104, 0)])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_is_the_definition_bit_for_bit(R, C, pad, dtype):
    t, x = _values(R, C, dtype, R * 7 + C)
    buf = torch.full((R, C + pad), float("nan"), dtype=dtype)       # what lies between rows is not read
    buf[:, :C] = t
    X = buf.to(DEV)[:, :C]
    codes = Guarded((R, MX.mx_words(C)), torch.int32, DEV)
    scales = Guarded(MX.mx_scale_shape(R, C), torch.uint8, DEV,
                     fill=torch.full(MX.mx_scale_shape(R, C), 0x5A, dtype=torch.uint8))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    MX.gptq_mx_quantize(X, codes.t, scales.t, st)
    c, e = L.mx_quantize(x)
    np.testing.assert_array_equal(codes.t.cpu().numpy().view(np.uint32), o.pack(c.astype(np.int64), 4))
    # rows past the last one keep what was there
    np.testing.assert_array_equal(scales.t.cpu().numpy().ravel(), L.mx_tile(e, 0x5A))
    assert codes.intact() and scales.intact() and int(st) == 0
    for dt in TYPES:
        out = Guarded((R, C + pad), dt, DEV, fill=torch.full((R, C + pad), 7.0, dtype=dt))
        MX.gptq_mx_dequantize(codes.t, scales.t, out.t[:, :C])
        want = torch.from_numpy(L.mx_values(c, e)[:, :C]).to(dt)
        assert torch.equal(out.t[:, :C].cpu(), want) and out.intact()
        assert (out.t[:, C:] == 7.0).all()


@pytest.mark.parametrize("R,C,ld", [(9, 1100, 1101), (9, 515, 517), (140, 700, 703), (9, 2049, 2055),
                                    (9, 129, 131), (9, 513, 513), (9, 4096, 4097)])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_at_every_offset_from_16_bytes(R, C, ld, dtype):
    # ld is odd, so nine rows start at each multiple of the element size from a 16-byte boundary;
    # the buffer itself starts at an odd element.  What lies between rows is not read or written
    t, x = _values(R, C, dtype, R + C)
    c, e = L.mx_quantize(x)

    def view(flat):
        return flat[1:1 + R * ld].view(R, ld)[:, :C]

    flat = torch.full((R * ld + 1,), float("nan"), dtype=dtype, device=DEV)
    view(flat).copy_(t)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = MX.mx_quantize(view(flat), st)
    np.testing.assert_array_equal(q.codes.cpu().numpy().view(np.uint32), o.pack(c.astype(np.int64), 4))
    at = [[L.mx_scale_index(r, k, e.shape[1]) for k in range(e.shape[1])] for r in range(R)]
    np.testing.assert_array_equal(q.scales.cpu().numpy().ravel()[at], e)
    assert int(st) == 0
    for dt in TYPES:
        out = Guarded((R * ld + 1,), dt, DEV, fill=torch.full((R * ld + 1,), 7.0, dtype=dt))
        MX.gptq_mx_dequantize(q.codes, q.scales, view(out.t))
        want = torch.full((R * ld + 1,), 7.0, dtype=dt)
        view(want).copy_(torch.from_numpy(L.mx_values(c, e)[:, :C]).to(dt))
        assert torch.equal(out.t.cpu(), want) and out.intact()


def test_quantize_edges():
    f = np.float32
    rows = np.zeros((12, 64), dtype=f)
    rows[0, :12] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, -0.0]      # ties
    rows[1, :4] = [np.finfo(f).max, -np.finfo(f).max, 1e30, 2.0 ** -126]
    rows[2, :4] = [2.0 ** -149, -2.0 ** -149, 0, 0]                                      # subnormals
    rows[3, :4] = [2.0 ** -126, 2.0 ** -127, 2.0 ** -128, -2.0 ** -129]
    rows[4, :3] = [np.nextafter(f(8), f(0)), -7.99, 6.01]                                # above 6 scales
    rows[5, 3] = np.nan
    rows[6, 40] = np.inf
    rows[7, 63] = -np.inf
    rows[8, :2] = [-np.nan, np.inf]
    rows[9] = -0.0
    rows[10] = 2.0 ** -125
    x = rows.astype(np.float64)
    c, e = L.mx_quantize(x)
    assert [int(v) for v in e[5:9].ravel()] == [255, 0, 0, 255, 0, 255, 255, 0]
    X = torch.from_numpy(rows).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = MX.mx_quantize(X, st)
    np.testing.assert_array_equal(q.codes.cpu().numpy().view(np.uint32), o.pack(c.astype(np.int64), 4))
    got = q.scales.cpu().numpy().ravel()
    for r in range(12):
        for k in range(2):
            assert got[L.mx_scale_index(r, k, 2)] == e[r, k], (r, k)
    assert int(st) == G.GPTQ_ERR_NONFINITE
    MX.mx_quantize(X)                                       # a NULL status word is allowed
    y = MX.mx_dequantize(q).cpu().numpy()
    want = L.mx_values(c, e).astype(np.float32)
    np.testing.assert_array_equal(np.isnan(y), np.isnan(want))
    np.testing.assert_array_equal(np.nan_to_num(y, nan=0.0), np.nan_to_num(want, nan=0.0))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("order", ["near", "mixed"])
def test_quantize_every_16_bit_value(dtype, order):
    # every bit pattern once, in blocks of neighbours and in blocks of far-apart magnitudes
    bits = np.arange(65536, dtype=np.uint16)
    if order == "mixed":
        bits = np.random.default_rng(0).permutation(bits)
    t = torch.from_numpy(bits.view(np.int16)).view(dtype).reshape(-1, 32)
    with np.errstate(invalid="ignore"):
        c, e = L.mx_quantize(t.double().numpy())
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = MX.mx_quantize(t.to(DEV), st)
    np.testing.assert_array_equal(q.codes.cpu().numpy().view(np.uint32), o.pack(c.astype(np.int64), 4))
    got = q.scales.cpu().numpy().ravel()
    np.testing.assert_array_equal(got[[L.mx_scale_index(r, 0, 1) for r in range(len(t))]], e[:, 0])
    assert int(st) == G.GPTQ_ERR_NONFINITE


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_every_code_and_scale(dtype):
    e = np.arange(256, dtype=np.uint8)[:, None]
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    words, scales = _device(codes, e, 32)
    Y = torch.empty(256, 32, dtype=dtype, device=DEV)
    MX.gptq_mx_dequantize(words, scales, Y)
    # formed in fp32 (6 * 2^127 overflows there), then rounded once
    with np.errstate(over="ignore"):
        want = torch.from_numpy(L.mx_values(codes, e).astype(np.float32)).to(dtype)
    got = Y.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0.0, 1.0, -1.0), want.nan_to_num(0.0, 1.0, -1.0))
    assert torch.equal(got.isinf(), want.isinf())


def test_empty_calls_launch_nothing():
    n = G.gptq_launch_count()
    q = MX.mx_quantize(torch.empty(0, 64, device=DEV))
    assert MX.mx_dequantize(q).shape == (0, 64)
    w = MX.mx_quantize(torch.empty(0, 64, device=DEV))
    assert MX.mx_matmul(q, w).shape == (0, 0)
    assert G.gptq_launch_count() == n


def test_rows_past_32_bit_offsets():
    # 66000 x 65664 codes are 2.2 GB and the values 4.3e9 elements: corners only
    R, C = 66000, 65664
    X = torch.zeros(R, C, dtype=torch.bfloat16, device=DEV)
    spots = [(0, 0), (R - 1, C - 1), (R - 1, 0), (R // 2, 40000), (65500, 65000)]
    for i, (r, c) in enumerate(spots):
        X[r, c] = float(i + 1)
    q = MX.mx_quantize(X)
    X.zero_()
    MX.gptq_mx_dequantize(q.codes, q.scales, X)
    for i, (r, c) in enumerate(spots):
        assert float(X[r, c]) == {1: 1, 2: 2, 3: 3, 4: 4, 5: 4}[i + 1]      # 5 is a tie: to even
    for r in {r for r, _ in spots} | {1, R - 2}:
        assert int(X[r].count_nonzero()) == sum(1 for s in spots if s[0] == r)


# ------------------------------------------------------------------ product
SHAPES = [(1, 128, 64), (1, 1, 1), (2, 130, 32), (1, 513, 4128), (3, 100, 96), (16, 128, 128),
          (17, 256, 300), (33, 70, 1000), (64, 384, 512), (65, 129, 2080), (127, 128, 257),
          (129, 300, 640), (256, 256, 1024), (300, 200, 4104), (257, 1000, 160), (700, 515, 1056),
          (1, 4096, 12288), (5, 640, 20000), (520, 130, 8200),
          # every width of a token tile, tiles that start in the middle of 128 tokens among them
          (256, 5120, 96), (384, 9472, 96), (500, 9472, 64), (700, 9472, 33),
          # few tiles and a long K, which several pairs share
          (100, 300, 20000), (333, 513, 8200), (700, 130, 33000), (65, 2000, 1056), (129, 4000, 2100),
          (70, 100, 9000), (70, 129, 9000)]


@pytest.mark.parametrize("M,R,C", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_product_within_its_bound(M, R, C, dtype):
    xc, xs, x = _stored(M, C, M + C)
    wc, ws, w = _stored(R, C, R + 3 * C)
    out = Guarded((M, R + 5), dtype, DEV, fill=torch.full((M, R + 5), 7.0, dtype=dtype))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    MX.gptq_mx_matmul(xc, xs, wc, ws, C, out.t[:, :R], st)
    got = out.t.double().cpu().numpy()
    want, S = x @ w.T, np.abs(x) @ np.abs(w).T
    steps = -(-C // 64)
    bound = (2 * steps + 16) * 2.0 ** -23 * S
    bound = bound + torch.finfo(dtype).eps / 2 * (np.abs(want) + bound) + 1e-30
    if dtype == torch.float16:
        big = np.abs(want) > 65000
        got, want, bound = got[:, :R], np.where(big, 0, want), np.where(big, np.inf, bound)
    assert int(st) == 0
    err = np.abs(got[:, :R] - want)
    assert np.all(err <= bound), np.max(err / bound)
    assert out.intact() and (out.t[:, R:] == 7.0).all()


@pytest.mark.parametrize("M,R,C", [(1, 200, 4128), (40, 300, 2080), (130, 257, 1056), (513, 514, 5152),
                                   (100, 300, 9000), (300, 1030, 4160)])
def test_product_of_small_whole_numbers_is_exact(M, R, C):
    # every scale 1: products are multiples of 1/4 and every sum stays below 2^24 of them
    xc, xs, x = _stored(M, C, 1, 127, 128)
    wc, ws, w = _stored(R, C, 2, 127, 128)
    Y = torch.empty(M, R, device=DEV)
    MX.gptq_mx_matmul(xc, xs, wc, ws, C, Y)
    np.testing.assert_array_equal(Y.cpu().numpy().astype(np.float64), x @ w.T)


@pytest.mark.parametrize("M,R,C", [(5, 300, 4128), (16, 130, 9000), (130, 300, 700), (100, 300, 9000)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ex,ew", [((0, 30), (85, 125)), ((60, 100), (0, 30)), ((225, 255), (80, 109)),
                                   ((0, 2), (253, 255)), ((253, 255), (0, 2))])
def test_product_at_the_ends_of_the_scales(M, R, C, dtype, ex, ew):
    # the bound of test_product_within_its_bound where products and sums lie about fp32's least or
    # below its largest number: each of the cuts counted there is at least one of 2^-149, and the
    # last rounding at least half of the type's least subnormal
    xc, xs, x = _stored(M, C, 1, *ex)
    wc, ws, w = _stored(R, C, 2, *ew)
    Y = torch.empty(M, R, dtype=dtype, device=DEV)
    MX.gptq_mx_matmul(xc, xs, wc, ws, C, Y)
    got, want, S = Y.double().cpu().numpy(), x @ w.T, np.abs(x) @ np.abs(w).T
    assert S.max() < 2.0 ** 127                            # no sum overflows
    f = torch.finfo(dtype)
    bound = (2 * -(-C // 64) + 16) * (2.0 ** -23 * S + 2.0 ** -149)
    bound = bound + f.eps / 2 * (np.abs(want) + bound) + f.smallest_normal * f.eps / 2
    if dtype == torch.float16:
        edge = 65520.0                                     # what rounds to 65504 or less in magnitude
        inf = np.abs(want) - bound >= edge
        assert np.array_equal(np.isinf(got) & inf, inf)
        near = ~inf & (np.abs(want) + bound >= edge)       # either
        got = np.where(inf | near, 0, got)
        want = np.where(inf | near, 0, want)
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("M", [3, 100])
def test_product_past_the_range_is_infinite(M):
    # sums of one sign: beyond fp32's range an infinity of that sign, whatever their order
    R, C = 140, 1000
    rng = np.random.default_rng(0)
    cx, cw = (rng.integers(1, 8, (n, 1024)).astype(np.uint8) for n in (M, R))
    cw[1::2] |= 8
    cx[:, C:], cw[:, C:] = 0, 0
    ex, ew = np.full((M, 32), 254, np.uint8), np.full((R, 32), 254, np.uint8)
    ex[1] = 0                                              # 2^-127 x 2^127: an ordinary sum
    Y = torch.empty(M, R, device=DEV)
    MX.gptq_mx_matmul(*_device(cx, ex, C), *_device(cw, ew, C), C, Y)
    y, want = Y.double().cpu().numpy(), L.mx_values(cx, ex)[:, :C] @ L.mx_values(cw, ew)[:, :C].T
    np.testing.assert_array_equal(y[1], want[1])           # multiples of 1/4, below 2^24 of them
    rest = np.arange(M) != 1
    assert np.all(np.abs(want[rest]) > 2.0 ** 128)
    np.testing.assert_array_equal(y[rest], np.where(want[rest] > 0, np.inf, -np.inf))


@pytest.mark.parametrize("M,R,C", [(700, 9572, 64), (256, 25601, 32), (130, 6273, 160)])
def test_product_of_pairs_whose_second_half_has_no_rows(M, R, C):
    # R % 256 in 1 .. 128: in the last row tile rank 1 of a pair only hands the accumulator back,
    # and the pair parts at once; call upon call, each starting as the one before it drains
    xc, xs, x = _stored(M, C, 1, 127, 128)
    wc, ws, w = _stored(R, C, 2, 127, 128)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    Y = [torch.empty(M, R, device=DEV) for _ in range(4)]
    for i in range(40):
        MX.gptq_mx_matmul(xc, xs, wc, ws, C, Y[i % 4], st)
    want = torch.from_numpy(x @ w.T).to(DEV)          # multiples of 1/4, far below 2^24 of them
    assert int(st) == 0 and all(torch.equal(y.double(), want) for y in Y)


@pytest.mark.parametrize("M", [1, 20, 200])
def test_product_one_hot_reads_single_weights(M):
    # token t picks column t of W: any mistake in the order of columns, rows or scales shows
    R, C = 300, 640
    wc, ws, w = _stored(R, C, 5, 100, 150)
    hot = np.zeros((M, C))
    hot[np.arange(M), (np.arange(M) * 37) % C] = 1.0
    x = MX.mx_quantize(torch.from_numpy(hot).float().to(DEV))
    Y = torch.empty(M, R, device=DEV)
    MX.gptq_mx_matmul(x.codes, x.scales, wc, ws, C, Y)
    np.testing.assert_array_equal(Y.cpu().numpy().astype(np.float64), w[:, (np.arange(M) * 37) % C].T)


def test_product_leaves_unwritten_scales_and_bad_rows_to_their_rows():
    # bytes of rows past the last one may be anything (here 255, not a number), and a
    # block that is not a number spoils its own row only
    M, R, C = 3, 130, 160
    rng = np.random.default_rng(0)
    cx, ex = rng.integers(0, 16, (M, C)).astype(np.uint8), np.full((M, C // 32), 127, np.uint8)
    cw, ew = rng.integers(0, 16, (R, C)).astype(np.uint8), np.full((R, C // 32), 127, np.uint8)
    ex[1, 2] = 255
    ew[129, 4] = 255
    Y = torch.empty(M, R, device=DEV)
    MX.gptq_mx_matmul(*_device(cx, ex, C, 255), *_device(cw, ew, C, 255), C, Y)
    y = Y.cpu().numpy()
    want = L.mx_values(cx, ex) @ L.mx_values(cw, ew).T
    np.testing.assert_array_equal(np.isnan(y), np.isnan(want))
    ok = ~np.isnan(want)
    np.testing.assert_array_equal(y[ok], want[ok])
    assert ok.sum() == 2 * 129


def test_product_of_quantized_activations():
    # the path of a layer: activations and weights quantised on the device, then multiplied
    gen = torch.Generator(device=DEV).manual_seed(3)
    X = torch.randn(37, 1000, generator=gen, device=DEV, dtype=torch.bfloat16)
    W = torch.randn(300, 1000, generator=gen, device=DEV).half() * 0.02
    w = MX.mx_quantize(W)
    Y = MX.mx_linear(X, w)
    assert Y.dtype == torch.bfloat16
    qx = L.mx_values(*L.mx_quantize(X.double().cpu().numpy()))[:, :1000]
    qw = L.mx_values(*L.mx_quantize(W.double().cpu().numpy()))[:, :1000]
    want, S = qx @ qw.T, np.abs(qx) @ np.abs(qw).T
    bound = 40 * 2.0 ** -23 * S + 2.0 ** -8 * np.abs(want) * 1.01
    assert np.all(np.abs(Y.double().cpu().numpy() - want) <= bound)
    # and the quantised layer is near the layer: each side is off by at most a quarter (a value
    # above 6 scales; 1/6 between levels) of its own magnitude or half a step of the smallest levels
    full = X.double() @ W.double().T
    rel = float((Y.double() - full).norm() / full.norm())
    assert rel < 0.5


def test_product_repeats_bit_for_bit_and_on_two_streams():
    M, R, C = 5, 1000, 9000
    xc, xs, _ = _stored(M, C, 1)
    wc, ws, _ = _stored(R, C, 2)
    ref = torch.empty(M, R, device=DEV)
    MX.gptq_mx_matmul(xc, xs, wc, ws, C, ref)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = [torch.empty(M, R, device=DEV) for _ in range(8)]
    for i, y in enumerate(out):
        MX.gptq_mx_matmul(xc, xs, wc, ws, C, y, stream=streams[i % 2])
    torch.cuda.synchronize()
    for y in out:
        assert torch.equal(y, ref)


@pytest.mark.parametrize("M,R,C", [(3, 300, 700), (150, 700, 1000), (2000, 300, 4000)])
def test_calls_back_to_back_see_each_others_results(M, R, C):
    # each call starts while the one before it drains; one pair of buffers is rewritten again and
    # again, so a read of anything but the latest contents shows
    X = [torch.randn(M, C, device=DEV).half() for _ in range(3)]
    w = MX.mx_quantize(torch.randn(R, C, device=DEV))
    q = MX.mx_quantize(X[0])
    want = []
    for x in X:
        one = MX.mx_quantize(x)
        torch.cuda.synchronize()
        want.append((MX.mx_dequantize(one, torch.float16), MX.mx_matmul(one, w)))
        torch.cuda.synchronize()
    n = 30
    out = torch.empty(n, M, C, dtype=torch.float16, device=DEV)
    Y = torch.empty(n, M, R, device=DEV)
    torch.cuda.synchronize()
    for i in range(n):
        MX.gptq_mx_quantize(X[i % 3], q.codes, q.scales)
        if i % 2:
            MX.gptq_mx_dequantize(q.codes, q.scales, out[i])
            MX.gptq_mx_matmul(q.codes, q.scales, w.codes, w.scales, C, Y[i])
        else:
            MX.gptq_mx_matmul(q.codes, q.scales, w.codes, w.scales, C, Y[i])
            MX.gptq_mx_dequantize(q.codes, q.scales, out[i])
    torch.cuda.synchronize()
    for i in range(n):
        assert torch.equal(out[i], want[i % 3][0]) and torch.equal(Y[i], want[i % 3][1]), i


@pytest.mark.parametrize("M,R,C", [(4, 700, 1000), (300, 600, 2000)])
def test_graph_replay_sees_new_inputs(M, R, C):
    X = torch.randn(M, C, device=DEV)
    w = MX.mx_quantize(torch.randn(R, C, device=DEV))
    q = MX.mx_quantize(X)
    Y = torch.empty(M, R, device=DEV)
    MX.gptq_mx_matmul(q.codes, q.scales, w.codes, w.scales, C, Y)       # warm-up
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        MX.gptq_mx_quantize(X, q.codes, q.scales)
        MX.gptq_mx_matmul(q.codes, q.scales, w.codes, w.scales, C, Y)
    for seed in range(3):
        X.copy_(torch.randn(M, C, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        want = MX.mx_matmul(MX.mx_quantize(X), w)
        torch.cuda.synchronize()
        assert torch.equal(Y, want)


def test_product_output_past_32_bit_offsets():
    M, R, C = 8200, 270000, 32                       # 2.2e9 outputs
    hot = torch.zeros(M, C, device=DEV)
    hot[:, 0] = 1.0
    hot[M - 1, 0] = 2.0
    x = MX.mx_quantize(hot)
    W = torch.ones(R, C, device=DEV, dtype=torch.bfloat16)
    W[R - 1] = 3.0
    w = MX.mx_quantize(W)
    Y = MX.mx_matmul(x, w, torch.bfloat16)
    assert float(Y[0, 0]) == 1 and float(Y[M - 1, R - 1]) == 6 and float(Y[M - 1, 0]) == 2
    assert float(Y[M - 2, R - 1]) == 3 and float(Y[M // 2].float().sum()) == R + 2


@pytest.mark.parametrize("M,R,C,shared", [(4, 1500, 49152, False), (512, 1500, 49152, False),
                                          (16, 300, 49152, True), (300, 1000, 49152, True)])
def test_product_waits_give_up_and_drain(M, R, C, shared):
    # with a limit of one poll the waits run out during normal work: the status says so, the
    # context stays usable and the same call then computes the right values.  Where CTAs share
    # a tile's K (`shared`) a poll may outlast the work; then the values are right at once
    xc, xs, x = _stored(M, C, 1, 127, 128)
    wc, ws, w = _stored(R, C, 2, 127, 128)
    Y = torch.empty(M, R, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    old = G.gptq_debug_set_wait_limit(1)
    try:
        for _ in range(3):
            MX.gptq_mx_matmul(xc, xs, wc, ws, C, Y, st)
        torch.cuda.synchronize()
    finally:
        G.gptq_debug_set_wait_limit(0)
    assert old > 1 and int(st) in ((0, G.GPTQ_ERR_TIMEOUT) if shared else (G.GPTQ_ERR_TIMEOUT,))
    if int(st):
        st.zero_()
        MX.gptq_mx_matmul(xc, xs, wc, ws, C, Y, st)
    # multiples of 1/4 whose sums stay below 2^24 of them
    rows = slice(0, 300)
    np.testing.assert_array_equal(Y[:, rows].double().cpu().numpy(), x @ w[rows].T)
    assert int(st) == 0


@pytest.mark.parametrize("M,R,C,stage", [
    # one CTA a tile; K split over eight CTAs of a cluster
    (4, 9600, 4096, 0), (4, 9600, 4096, 6), (16, 300, 49152, 0), (16, 300, 49152, 3), (16, 300, 49152, 11),
    (60, 300, 20000, 2),
    # a pair a tile, of several tiles each; pairs that share a tile's K
    (512, 9500, 2080, 0), (512, 9500, 2080, 4), (2000, 2000, 5120, 7),
    (300, 1000, 49152, 0), (300, 1000, 49152, 5), (300, 1000, 49152, 20), (65, 200, 9000, 1)])
def test_product_that_gives_up_at_a_stage_stops_as_one(M, R, C, stage):
    # the last CTA or pair of each cluster stops in the middle of its work: the status says so every
    # time, and the same calls then compute the right values
    xc, xs, x = _stored(M, C, 1, 127, 128)
    wc, ws, w = _stored(R, C, 2, 127, 128)
    Y = torch.empty(M, R, device=DEV)
    st = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert MX.gptq_mx_debug_give_up(stage) == -1
    try:
        for i in range(3):
            MX.gptq_mx_matmul(xc, xs, wc, ws, C, Y, st[i:i + 1])
        torch.cuda.synchronize()
    finally:
        assert MX.gptq_mx_debug_give_up(-1) == stage
    assert st.tolist() == [G.GPTQ_ERR_TIMEOUT] * 3
    st.zero_()
    Y.fill_(float("nan"))
    MX.gptq_mx_matmul(xc, xs, wc, ws, C, Y, st[:1])
    rows = slice(0, 300)                              # multiples of 1/4, sums below 2^24 of them
    np.testing.assert_array_equal(Y[:, rows].double().cpu().numpy(), x @ w[rows].T)
    assert int(st[0]) == 0 and not Y.isnan().any()
