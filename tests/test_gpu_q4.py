"""4-bit block products on the GPU against the float64 oracle.

Tolerances.  Quantising is exact: codes and scale bytes must be the oracle's, and
so is reading back.  A product of two 4-bit operands: a product of two codes is a
multiple of 1/4 up to 36, so a block's 32 products sum exactly in 13 bits; an
instruction adds four blocks and the sum so far in fp32, at most five additions,
each off by at most one unit in the last place, 2^-23 of a partial sum that never
exceeds the sum of magnitudes S.  So with ceil(n / 128) instructions for n terms
and at most 25 more additions (pieces, waves, base) |error| <= (5 ceil(n / 128) +
25) 2^-23 S.  With bf16 rows every product of two operands (8 and 2 significant
bits) fits fp32 and its sum of n terms takes at most n additions: n 2^-23 S.  The
one rounding of the result adds half a step: 2^-8 of it for bf16, 2^-24 for fp32."""

import numpy as np
import pytest
import torch

import newton_schulz_dmuon_amd as nsd
from newton_schulz_dmuon_amd import _lib
from oracle import q4 as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def values(rng, rows, cols, dtype, std=1.0):
    """Rows of differing size, some of them zero, a few large channels."""
    x = rng.standard_normal((rows, cols)) * std * np.exp(rng.standard_normal((rows, 1)))
    x[:, rng.random(cols) < 0.02] *= 30.0
    x[rng.random(rows) < 0.1] = 0.0
    return torch.from_numpy(x).to(dtype)


def host(t):
    return t.detach().cpu().double().numpy()


def check_bytes(got, want, what):
    g = got.cpu().numpy()
    assert g.shape == want.shape and np.array_equal(g, want), (what, np.argwhere(g != want)[:4], g[g != want][:4], want[g != want][:4])


def check_matrix(q, x, random=None, plain=True, transposed=True):
    """q's forms are x's (fp64), bit for bit."""
    assert (q.rows, q.cols) == x.shape
    for on, codes, scales, v, r, what in ((plain, q.codes, q.scales, x, random, "plain"),
                                          (transposed, q.codes_t, q.scales_t, x.T, None if random is None else random.T, "transposed")):
        if not on:
            assert codes is None and scales is None
            continue
        c, s = ref.quantize(v, r)
        check_bytes(scales, s, (what, "scales", x.shape))
        check_bytes(codes, ref.pack(c), (what, "codes", x.shape))


def check_sum(got, want, mag, adds, what):
    """adds: additions in fp32 that a result takes."""
    g = host(got)
    assert g.shape == want.shape, what
    bound = adds * 2.0 ** -23 * mag + HALF_STEP[got.dtype] * np.abs(want) * (1 + 2.0 ** -7) + 1e-37
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], g[bad][:4], want[bad][:4], bound[bad][:4])


def adds(terms):
    return 5 * -(-terms // 128) + 25


def device(codes, scales):
    return torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(scales).cuda()


def rows_of(rng, t, k, std=1.0):
    """A matrix on the GPU in its plain form, made by the oracle, and its values."""
    c, s = ref.quantize(host(values(rng, t, k, BF16, std)))
    return nsd.Q4Matrix(t, k, *device(c, s)), ref.values(c, s)[:, :k]


def transposed_of(rng, t, k, std=1.0):
    """... in its transposed form."""
    c, s = ref.quantize(host(values(rng, t, k, BF16, std)).T)
    return nsd.Q4Matrix(t, k, None, None, *device(c, s)), ref.values(c, s)[:, :t].T


def weight_of(rng, n, k, transpose=False):
    return (transposed_of if transpose else rows_of)(rng, n, k, 0.02)


# ----------------------------------------------------------- quantising --

SIZES = [(1, 1), (1, 31), (1, 4096), (2, 32), (3, 33), (4, 1000), (5, 1024), (8, 128), (17, 2050), (33, 513), (130, 384),
         (257, 136), (300, 1001), (513, 40)]


@pytest.mark.parametrize("t,k", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("by_bytes", [False, True])
def test_quantise(t, k, dtype, by_bytes):
    print(f"quantise {t}x{k} {dtype} {by_bytes}", flush=True)
    rng = np.random.default_rng(t * 10007 + k)
    x = values(rng, t, k, dtype)
    r = rng.integers(0, 256, (t, k)).astype(np.uint8) if by_bytes else None
    rt = None if r is None else torch.from_numpy(r).cuda()
    for plain, transposed in ((True, True), (True, False), (False, True)):
        q = nsd.q4_quantize(x.cuda(), transposed=transposed, plain=plain, random=rt)
        torch.cuda.synchronize()
        check_matrix(q, host(x), r, plain, transposed)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_random_bytes_at_the_smallest_scales(dtype):
    """2^(10 - e) is more than fp32 holds for e below -117: blocks on both sides of
    that, and zero ones, beside each other in both directions."""
    print(f"smallest scales {dtype}", flush=True)
    rng = np.random.default_rng(12)
    for t, k in ((300, 520), (512, 512), (37, 1001)):
        e = rng.integers(-132, -100, (-(-t // 40), -(-k // 24)))
        e[rng.random(e.shape) < 0.1] = -1000
        scale = np.exp2(e.astype(np.float64)).repeat(40, 0).repeat(24, 1)[:t, :k]
        x = torch.from_numpy(rng.standard_normal((t, k)) * scale).to(dtype)
        r = rng.integers(0, 256, (t, k)).astype(np.uint8)
        q = nsd.q4_quantize(x.cuda(), transposed=True, random=torch.from_numpy(r).cuda())
        torch.cuda.synchronize()
        check_matrix(q, host(x), r)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("transposed", [True, False])
def test_weights(dtype, transposed):
    print(f"weights {dtype} {transposed}", flush=True)
    rng = np.random.default_rng(5)
    # more matrices than one launch takes, one of them without rows
    ws = [values(rng, n, k, dtype, 0.02) for n, k in SIZES[4:] * 4] + [torch.empty(0, 40, dtype=dtype)]
    ws.insert(3, torch.empty(0, 300, dtype=dtype))
    got = nsd.q4_quantize_weights([w.cuda() for w in ws], transposed=transposed)
    torch.cuda.synchronize()
    for w, q in zip(ws, got):
        if w.shape[0]:
            check_matrix(q, host(w), None, True, transposed)


def test_weights_of_both_types():
    """Types that change along the list, and with them the launches."""
    print("weights of both types", flush=True)
    rng = np.random.default_rng(6)
    ws = [values(rng, n, k, F32 if i % 3 == 1 else BF16, 0.02) for i, (n, k) in enumerate(SIZES)]
    got = nsd.q4_quantize_weights([w.cuda() for w in ws])
    torch.cuda.synchronize()
    for w, q in zip(ws, got):
        check_matrix(q, host(w))


def test_quantise_every_tie_and_range_end():
    """Every code, every tie between two codes and their fp32 neighbours, at the
    largest, the smallest and a middle scale; blocks of subnormals, zeros and the
    largest finite values, NaN and infinities."""
    print("ties and range ends", flush=True)
    fin = np.unique(ref.code_values(np.arange(16, dtype=np.uint8)))
    mid = (fin[1:] + fin[:-1]) / 2
    m32 = mid.astype(np.float32)
    v = np.concatenate([fin, mid, np.nextafter(m32, np.float32(np.inf)), np.nextafter(m32, np.float32(-np.inf))])
    rows = []
    for e in (0, -125, 125, 13, -60):
        block = np.zeros(-(-v.size // 31) * 32).reshape(-1, 32)
        block[:, 0] = 6.0  # fixes the scale
        block[:, 1:].flat[:v.size] = v
        rows.append((block * 2.0 ** e).reshape(1, -1))
    x = np.concatenate(rows).astype(np.float32)
    assert np.isfinite(x).all()
    extra = np.zeros((6, x.shape[1]), np.float32)
    extra[0, ::3] = 2.0 ** -149
    extra[1, ::5] = np.finfo(np.float32).max
    extra[2, 1], extra[2, 40], extra[2, 41] = np.nan, np.inf, -np.inf
    extra[2, 2], extra[2, 43] = 3.0, -5.0
    extra[3] = -0.0
    extra[4, ::2] = -np.finfo(np.float32).max
    extra[4, 1::2] = np.linspace(2.0 ** 124, 2.0 ** 127, extra[4, 1::2].size)
    extra[5] = np.float32(2.0 ** -126) * np.linspace(-6, 6, extra.shape[1])
    x = torch.from_numpy(np.concatenate([x, extra]))
    q = nsd.q4_quantize(x.cuda(), transposed=True)
    b = nsd.q4_quantize(x.to(BF16).cuda(), transposed=True)
    torch.cuda.synchronize()
    check_matrix(q, host(x))
    check_matrix(b, host(x.to(BF16)))
    r = np.random.default_rng(0).integers(0, 256, x.shape).astype(np.uint8)
    q = nsd.q4_quantize(x.cuda(), transposed=True, random=torch.from_numpy(r).cuda())
    torch.cuda.synchronize()
    check_matrix(q, host(x), r)


def test_random_bytes_cover_every_threshold():
    """Each value against all 256 bytes, values at and beside each byte's
    threshold among them."""
    print("thresholds", flush=True)
    part = (np.arange(256) + 0.5) / 256
    base = np.array([0.0, 0.5, 1.5, 2.0, 3.0, 4.0, 0.0, 4.0])[:, None]
    step = np.array([0.5, 0.5, 0.5, 1.0, 1.0, 2.0, 0.5, 2.0])[:, None]
    v = (base + step * part).astype(np.float32)
    v[6], v[7] = np.nextafter(v[6], np.float32(0)), np.nextafter(v[7], np.float32(9))
    x = np.zeros((256, 8 * 264), np.float32)
    x.reshape(256, 8, 264)[:, :, 8:] = v[None]
    x[:, ::32] = 6.0
    x[1::2] *= -1
    r = np.repeat(np.arange(256, dtype=np.uint8)[:, None], x.shape[1], 1)
    q = nsd.q4_quantize(torch.from_numpy(x).cuda(), transposed=True, random=torch.from_numpy(r).cuda())
    torch.cuda.synchronize()
    check_matrix(q, x.astype(np.float64), r)


@pytest.mark.parametrize("t,k", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dequantise(t, k, dtype):
    print(f"dequantise {t}x{k} {dtype}", flush=True)
    rng = np.random.default_rng(t + 31 * k)
    x = rng.standard_normal((t, k)) * 2.0 ** rng.integers(-120, 120, (t, k))
    x[rng.random((t, k)) < 0.3] = 0
    if t * k > 40:
        x[t // 2, k // 2] = np.nan
    c, s = ref.quantize(x)
    ct, st = ref.quantize(x.T)
    q = nsd.Q4Matrix(t, k, *device(c, s), *device(ct, st))
    got, got_t = nsd.q4_dequantize(q, dtype=dtype), nsd.q4_dequantize(q, transpose=True, dtype=dtype)
    torch.cuda.synchronize()
    assert got.dtype == dtype and np.array_equal(host(got), ref.values(c, s)[:, :k], equal_nan=True)
    assert np.array_equal(host(got_t), ref.values(ct, st)[:, :t], equal_nan=True)


def test_the_largest_values_read_back_as_infinite():
    print("largest values", flush=True)
    for dtype in (BF16, F32):
        x = torch.full((1, 64), torch.finfo(dtype).max, dtype=dtype)
        x[0, 32:] = -1.0
        q = nsd.q4_quantize(x.cuda())
        check_matrix(q, host(x), transposed=False)
        got = host(nsd.q4_dequantize(q, dtype=dtype))
        assert np.isposinf(got[0, :32]).all() and (got[0, 32:] == -1).all()


# ------------------------------------------------------------- products --

PRODUCT_SIZES = [(1, 1, 1), (1, 128, 128), (1, 1001, 513), (2, 16, 4096), (3, 17, 130), (15, 129, 257), (16, 256, 1024),
                 (17, 40, 128), (33, 300, 640), (64, 512, 2048), (65, 130, 1000), (100, 1024, 384), (129, 257, 2100),
                 (200, 640, 128), (256, 256, 256), (257, 520, 1030), (520, 264, 300), (700, 900, 1), (5, 9000, 130),
                 (40, 8200, 257), (60, 8200, 260), (1100, 1500, 700), (1100, 300, 6000)]


@pytest.mark.parametrize("t,n,k", PRODUCT_SIZES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product(t, n, k, transpose, dtype):
    print(f"product {t} {n} {k} {transpose} {dtype}", flush=True)
    rng = np.random.default_rng(t * 7 + n * 11 + k * 13 + transpose)
    w, wv = weight_of(rng, n, k, transpose)
    wv = wv if transpose else wv.T
    inner = n if transpose else k
    a, av = rows_of(rng, t, inner)
    x = values(rng, t, inner, BF16)
    out = nsd.q4_matmul(a, w, transpose=transpose, dtype=dtype)
    mixed = nsd.q4_matmul(x.cuda(), w, transpose=transpose, dtype=dtype)
    torch.cuda.synchronize()
    check_sum(out, av @ wv, np.abs(av) @ np.abs(wv), adds(inner), (t, n, k, transpose))
    check_sum(mixed, host(x) @ wv, np.abs(host(x)) @ np.abs(wv), inner + 25, (t, n, k, transpose, "bf16 rows"))


def any_codes(rng, rows, cols, spread):
    """Every code, and scales of 1 to 2^(spread - 1): codes, scales and values."""
    cp = ref.up(cols, ref.PAD)
    c = rng.integers(0, 16, (rows, cp)).astype(np.uint8)
    c[:, cols:] = 0
    s = rng.integers(127, 128 + spread, (cp // 32, ref.up(rows, 16))).astype(np.uint8)
    return c, s, ref.values(c, s)[:, :cols]


@pytest.mark.parametrize("t,n,k", PRODUCT_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sums_that_fp32_holds_are_exact(t, n, k, dtype):
    """Every code with scales of 1 to 4: all sums are multiples of 1/4 below 2^22
    (asserted), exact in fp32 in any order, so the result is the exact sum rounded
    once, where large products cancel too."""
    print(f"exact sums {t} {n} {k} {dtype}", flush=True)
    rng = np.random.default_rng(t + n + k)
    ca, sa, av = any_codes(rng, t, k, 3)
    cb, sb, bv = any_codes(rng, n, k, 3)
    w = nsd.Q4Matrix(n, k, *device(cb, sb))
    x = torch.from_numpy(np.rint(rng.standard_normal((t, k)) * 4)).to(BF16)
    for a, v in ((nsd.Q4Matrix(t, k, *device(ca, sa)), av), (x.cuda(), host(x))):
        want = v @ bv.T
        assert (np.abs(v) @ np.abs(bv).T).max() < 2.0 ** 22
        got, want = host(nsd.q4_matmul(a, w, dtype=dtype)), torch.from_numpy(want).to(dtype).double().numpy()
        assert np.array_equal(got, want), (np.argwhere(got != want)[:4], got[got != want][:4], want[got != want][:4])


WGRAD_SIZES = [(1, 1, 1), (1, 128, 128), (2, 300, 513), (3, 17, 130), (31, 64, 64), (32, 65, 129), (33, 256, 256),
               (64, 257, 200), (65, 40, 1000), (127, 1001, 33), (200, 136, 384), (333, 520, 513), (1000, 129, 257),
               (1025, 256, 512), (2100, 8, 128), (3000, 700, 300), (450, 8200, 2100)]


@pytest.mark.parametrize("t,n,k", WGRAD_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("base", ["none", "other", "out"])
def test_weight_grad(t, n, k, dtype, base):
    print(f"weight grad {t} {n} {k} {dtype} {base}", flush=True)
    rng = np.random.default_rng(t * 7 + n * 11 + k * 13)
    x, xv = transposed_of(rng, t, k)
    dy, dv = transposed_of(rng, t, n, 1e-2)
    b = values(rng, n, k, dtype, 0.05).cuda()
    b0 = host(b)
    out = b if base == "out" else None
    got = nsd.q4_weight_grad(dy, x, out=out, dtype=dtype, base=None if base == "none" else b)
    torch.cuda.synchronize()
    want, mag = ref.matmul(dv.T, xv.T, None if base == "none" else b0)
    check_sum(got, want, mag, adds(t), (t, n, k, base))
    if base == "other":
        assert np.array_equal(host(b), b0)


def unpacked(codes, scales, rows, cols):
    """The values of codes on the GPU, in fp64."""
    c = torch.stack((codes & 15, codes >> 4), 2).view(rows, -1)
    table = torch.from_numpy(ref.code_values(np.arange(16, dtype=np.uint8))).cuda()
    s = (scales[:, :rows].t().to(torch.int64) - 127 + 1023 << 52).view(torch.float64)
    return (table[c.int()] * s.repeat_interleave(32, 1))[:, :cols]


# (tiles of every shape: whole, split, both)
TILE_SIZES = [(1505, 2801, 131), (1500, 1000, 9001), (2230, 3602, 903), (2309, 3424, 133), (4200, 4301, 8003), (300, 4100, 5000)]


@pytest.mark.parametrize("t,n,k", TILE_SIZES)
def test_large_products(t, n, k):
    """Against float64 products on the GPU of the values that the codes stand for."""
    print(f"large products {t} {n} {k}", flush=True)
    torch.manual_seed(t)
    x = torch.randn(t, k, device="cuda").to(BF16)
    w = (0.02 * torch.randn(n, k, device="cuda")).to(BF16)
    x4, w4 = nsd.q4_quantize(x), nsd.q4_quantize_weights([w])[0]
    wv = unpacked(w4.codes, w4.scales, n, k).t().contiguous()
    for a, v, count in ((x4, unpacked(x4.codes, x4.scales, t, k), adds(k)), (x, x.double(), k + 25)):
        want, mag = (v @ wv).cpu().numpy(), (v.abs() @ wv.abs()).cpu().numpy()
        for dtype in (BF16, F32):
            check_sum(nsd.q4_matmul(a, w4, dtype=dtype), want, mag, count, (t, n, k, dtype))
    # n columns of gradients and k of activations, summed over t tokens
    dy = (0.01 * torch.randn(t, n, device="cuda")).to(BF16)
    d4, z4 = nsd.q4_quantize(dy, transposed=True, plain=False), nsd.q4_quantize(x, transposed=True, plain=False)
    dv, zv = unpacked(d4.codes_t, d4.scales_t, n, t), unpacked(z4.codes_t, z4.scales_t, k, t).t().contiguous()
    want, mag = dv @ zv, dv.abs() @ zv.abs()
    for dtype in (BF16, F32):
        check_sum(nsd.q4_weight_grad(d4, z4, dtype=dtype), want.cpu().numpy(), mag.cpu().numpy(), adds(t), (t, n, k, dtype))
        b = torch.randn(n, k, device="cuda").to(dtype)
        want_b, mag_b = (want + b.double()).cpu().numpy(), (mag + b.double().abs()).cpu().numpy()
        check_sum(nsd.q4_weight_grad(d4, z4, out=b, base=b), want_b, mag_b, adds(t), (t, n, k, dtype, "in place"))


# (every work-group of the streaming kernels, with rings that turn, and every tile:
# whole, split, both)
EVERY_KERNEL = [(10, 33, 1117), (1, 17, 1408), (9, 5, 6797), (1, 30, 4703), (17, 2180, 1248), (1, 5006, 1511), (81, 1457, 1154),
                (432, 603, 1114), (70, 6226, 1166), (10174, 136, 1161), (6306, 20, 13207), (5629, 676, 4018),
                (272, 13686, 1182), (6069, 1352, 4022), (1070, 40, 1285), (1289, 10, 4785), (8204, 193, 13635),
                (1671, 4760, 1199), (6738, 2463, 3873), (4, 20, 1813), (5, 40, 1118), (3, 4108, 1278), (6, 4720, 1383),
                (9, 10357, 1144), (1, 13032, 1134), (4, 9356, 1472), (5, 9980, 1598), (9283, 4, 6531), (638, 6649, 1798),
                (3720, 1543, 1202), (10351, 2, 13646), (724, 11302, 1331), (2637, 30, 1245), (12, 1, 13681),
                (2326, 882, 1510), (6785, 131, 19804), (1208, 13114, 1424), (1, 4706, 5292)]


@pytest.mark.parametrize("t,n,k", EVERY_KERNEL)
def test_every_kernel(t, n, k):
    """Against float64 products on the GPU of the values that the codes stand for,
    onto a base too."""
    print(f"every kernel {t} {n} {k}", flush=True)
    torch.manual_seed(t + n)
    x = (torch.randn(t, k, device="cuda") * torch.exp2(torch.randint(-8, 9, (t, 1), device="cuda"))).to(BF16)
    w = (0.02 * torch.randn(n, k, device="cuda") * torch.exp2(torch.randint(-8, 9, (1, k), device="cuda"))).to(BF16)
    x4, w4 = nsd.q4_quantize(x), nsd.q4_quantize_weights([w])[0]
    wv = unpacked(w4.codes, w4.scales, n, k).t().contiguous()
    for a, v, count in ((x4, unpacked(x4.codes, x4.scales, t, k), adds(k)), (x, x.double(), k + 25)):
        want, mag = v @ wv, v.abs() @ wv.abs()
        for dtype in (BF16, F32):
            check_sum(nsd.q4_matmul(a, w4, dtype=dtype), want.cpu().numpy(), mag.cpu().numpy(), count, (t, n, k, dtype))
    # the same sums as a weight gradient: t outputs by n columns over k tokens
    d4, z4 = nsd.Q4Matrix(k, t, None, None, x4.codes, x4.scales), nsd.Q4Matrix(k, n, None, None, w4.codes, w4.scales)
    v = unpacked(x4.codes, x4.scales, t, k)
    want, mag = v @ wv, v.abs() @ wv.abs()
    for dtype in (BF16, F32):
        b = torch.randn(t, n, device="cuda").to(dtype)
        want_b, mag_b = (want + b.double()).cpu().numpy(), (mag + b.double().abs()).cpu().numpy()
        check_sum(nsd.q4_weight_grad(d4, z4, base=b), want_b, mag_b, adds(k), (t, n, k, dtype, "onto a base"))


# rows of whole 16-byte chunks that end inside a kernel's step, for every kernel that
# multiplies bf16 rows
CHUNK_SIZES = [(10, 33, 1128), (1, 17, 1416), (4, 20, 1816), (5, 40, 1128), (17, 2180, 1256), (1, 5006, 1512), (3, 4108, 1288),
               (6, 4720, 1384), (9, 10357, 1144), (1, 13032, 1144), (4, 9356, 1480), (5, 9980, 1608), (10174, 136, 1168),
               (9283, 4, 6536), (638, 6649, 1800), (3720, 1543, 1208), (10351, 2, 13656), (724, 11302, 1336),
               (2637, 30, 1256), (12, 1, 13688), (2326, 882, 1512), (1671, 4760, 1208), (6785, 131, 19816),
               (1208, 13114, 1432), (3, 50, 8), (70, 90, 24), (300, 300, 72), (130, 70, 136), (33, 40, 248)]


@pytest.mark.parametrize("t,n,k", CHUNK_SIZES)
def test_rows_of_whole_chunks(t, n, k):
    """No workspace holds a copy of them; nothing of the next row, here NaN, reaches a
    row's sums."""
    print(f"rows of whole chunks {t} {n} {k}", flush=True)
    torch.manual_seed(t + n)
    x = torch.randn(t + 1, k, device="cuda").to(BF16)
    x[1::2] = float("nan")
    x[t] = float("nan")
    x = x[:t]
    w = (0.02 * torch.randn(n, k, device="cuda")).to(BF16)
    w4 = nsd.q4_quantize_weights([w])[0]
    wv = unpacked(w4.codes, w4.scales, n, k).t().contiguous()
    rows = x[::2].double()
    want, mag = (rows @ wv).cpu().numpy(), (rows.abs() @ wv.abs()).cpu().numpy()
    for dtype in (BF16, F32):
        got = nsd.q4_matmul(x, w4, dtype=dtype)
        assert got[1::2].isnan().all()
        check_sum(got[::2].contiguous(), want, mag, k + 25, (t, n, k, dtype))


def test_no_rows():
    print("no rows", flush=True)
    rng = np.random.default_rng(1)
    w, _ = weight_of(rng, 130, 200)
    x = nsd.q4_quantize(torch.empty(0, 200, dtype=BF16, device="cuda"), transposed=True)
    assert x.codes.shape == (0, 128) and x.codes_t.shape == (200, 0)
    assert nsd.q4_matmul(x, w).shape == (0, 130) and nsd.q4_dequantize(x).shape == (0, 200)
    assert nsd.q4_dequantize(x, transpose=True).shape == (200, 0)
    assert nsd.q4_matmul(torch.empty(0, 200, dtype=BF16, device="cuda"), w).shape == (0, 130)
    dy = nsd.q4_quantize(torch.empty(0, 130, dtype=BF16, device="cuda"), transposed=True)
    base = values(rng, 130, 200, F32).cuda()
    zero = nsd.q4_weight_grad(dy, x, out=torch.full((130, 200), 7.0, device="cuda"))
    same = nsd.q4_weight_grad(dy, x, base=base)
    kept = base.clone()
    nsd.q4_weight_grad(dy, x, out=kept, base=kept)
    torch.cuda.synchronize()
    assert not zero.any() and torch.equal(same, base) and same.dtype == F32 and torch.equal(kept, base)


@pytest.mark.parametrize("t", [3, 70, 300])
def test_non_finite_reach_only_their_outputs(t):
    """A NaN or infinite element makes its block NaN, and with it its row's outputs
    (forward), its column's (weight gradient) and no others; in the last row, whose
    copies stand in for the rows behind it, too."""
    print(f"non-finite {t}", flush=True)
    rng = np.random.default_rng(t)
    n, k = 140, 260
    wt = torch.from_numpy(rng.standard_normal((n, k)) * 0.02).to(BF16)
    wt[n - 1, 3] = float("nan")
    w = nsd.q4_quantize_weights([wt.cuda()])[0]
    x = torch.from_numpy(rng.standard_normal((t, k))).to(BF16)
    x[1, 129], x[t - 1, 7] = float("nan"), float("inf")
    q = nsd.q4_quantize(x.cuda(), transposed=True)
    dy = torch.from_numpy(rng.standard_normal((t, n)) * 0.01).to(BF16)
    dy[t - 1, 5] = float("-inf")
    d = nsd.q4_quantize(dy.cuda(), transposed=True)
    bad = np.zeros((t, n), bool)
    bad[1], bad[t - 1], bad[:, n - 1] = True, True, True
    for dtype in (BF16, F32):
        assert np.array_equal(np.isnan(host(nsd.q4_matmul(q, w, dtype=dtype))), bad)
        y = host(nsd.q4_matmul(x.cuda(), w, dtype=dtype))
        assert np.array_equal(~np.isfinite(y), bad) and np.isnan(y[1]).all() and np.isnan(y[:, n - 1]).all()
        g = host(nsd.q4_weight_grad(d, q, dtype=dtype))
        want = np.zeros((n, k), bool)
        want[5], want[:, 129], want[:, 7] = True, True, True
        assert np.array_equal(np.isnan(g), want)
        dx = host(nsd.q4_matmul(d, w, transpose=True, dtype=dtype))
        want = np.zeros((t, k), bool)
        want[t - 1], want[:, 3] = True, True
        assert np.array_equal(np.isnan(dx), want)


def test_extreme_scales():
    """Scales at both ends of the range pass through the products: 2^-125 against
    2^100 and the like, the largest values against small and zero ones."""
    print("extreme scales", flush=True)
    for t in (3, 40, 300):
        n, k = 130, 320
        rng = np.random.default_rng(3)
        x = rng.standard_normal((t, k)).astype(np.float32)
        x[:, :128] *= 2.0 ** -124
        x[:, 128:256] *= 2.0 ** -100
        x[:, 256:] = 0
        x[0, 256:] = torch.finfo(BF16).max
        w = rng.standard_normal((n, k)).astype(np.float32)
        w[:64] *= 2.0 ** 100
        w[64:, :256] = torch.finfo(BF16).min
        w[:, 256:] = 2.0 ** -120 * rng.standard_normal((n, 64))
        w[5, 256:] = 0
        xb, wb = torch.from_numpy(x).to(BF16), torch.from_numpy(w).to(BF16)
        q, w4 = nsd.q4_quantize(xb.cuda(), transposed=True), nsd.q4_quantize_weights([wb.cuda()])[0]
        xv, wv = ref.quantized(host(xb)), ref.quantized(host(wb))
        for dtype in (BF16, F32):
            # results beyond bf16's range are infinite in both
            for a, v, count in ((q, xv, adds(k)), (xb.cuda(), host(xb), k + 25)):
                want, mag = ref.matmul(v, wv)
                got = nsd.q4_matmul(a, w4, dtype=dtype)
                assert np.isfinite(want.astype(np.float32)).all()
                check_sum(got, want, mag, count, (t, dtype))
        dy = torch.from_numpy(rng.standard_normal((t, n)) * 2.0 ** 40).to(BF16)
        dy[:, 7] = 2.0 ** -120
        dy[0] = 0  # the largest x by a large gradient is no fp32 number
        dyv, xt = ref.quantized(host(dy).T), ref.quantized(host(xb).T)
        d = nsd.q4_quantize(dy.cuda(), transposed=True)
        check_sum(nsd.q4_weight_grad(d, q, dtype=F32), *ref.matmul(dyv, xt), adds(t), "gradient")


def test_offsets_beyond_32_bits():
    """More than 2^32 bytes of codes and 2^32 outputs: the rows at the far end,
    alone and in the gradient, where all other rows are zero."""
    print("offsets beyond 32 bits", flush=True)
    t, k, n, far = (1 << 21) + 5, 4352, 40, 70
    rng = np.random.default_rng(77)
    x = torch.zeros(t, k, dtype=BF16, device="cuda")
    xf = values(rng, far, k, BF16)
    x[t - far:] = xf.cuda()
    q = nsd.q4_quantize(x, transposed=True)
    c, s = ref.quantize(host(xf))
    check_bytes(q.codes[t - far:], ref.pack(c), "codes")
    check_bytes(q.scales[:, t - far:t], s[:, :far], "scales")
    assert not q.codes[:1000].any() and (q.scales[:, :1000] == 2).all()
    back = nsd.q4_dequantize(q)
    assert np.array_equal(host(back[t - far:]), ref.values(c, s)[:, :k]) and not back[:t - far].any()
    back = nsd.q4_dequantize(q, transpose=True)
    lead = (t - far) % 32  # the far rows' first block begins this far before them
    xt = ref.quantized(np.concatenate([np.zeros((lead, k)), host(xf)]).T)[:, lead:]
    assert np.array_equal(host(back[:, t - far:]), xt) and not back[:, :t - far].any()
    del back
    w, wv = weight_of(rng, n, k)
    for a, v, count in ((q, ref.values(c, s)[:, :k], adds(k)), (x, host(xf), k + 25)):
        y = nsd.q4_matmul(a, w, dtype=F32)
        check_sum(y[t - far:], *ref.matmul(v, wv), count, "product")
        assert not y[:t - far].any()
    del x, y
    dy = torch.zeros(t, n, dtype=BF16, device="cuda")
    dyf = values(rng, far, n, BF16)
    dy[t - far:] = dyf.cuda()
    d = nsd.q4_quantize(dy, transposed=True, plain=False)
    dv = ref.quantized(np.concatenate([np.zeros((lead, n)), host(dyf)]).T)[:, lead:]
    g = nsd.q4_weight_grad(d, q, dtype=F32)
    # all other products are zeros
    check_sum(g, *ref.matmul(dv, xt), adds(far + 31), "gradient")
    del q, d, dy
    # as rows of the result: more than 2^32 outputs
    w2, _ = weight_of(rng, k, 8)
    one = torch.ones(t, 8, dtype=BF16, device="cuda")
    for a in (nsd.q4_quantize(one), one):
        y2 = nsd.q4_matmul(a, w2)
        assert torch.equal(y2[t - 1], y2[0]) and torch.equal(y2[t // 2], y2[0]) and y2[0].any()
        del y2


# ----------------------------------------------------- buffers and bounds --

GUARD = 512


def guarded_like(t, fill):
    """A tensor of t's shape inside a larger buffer of fill bytes."""
    raw = torch.full((t.numel() * t.element_size() + 2 * GUARD,), fill, dtype=torch.uint8, device="cuda")
    return raw, raw[GUARD:GUARD + t.numel() * t.element_size()].view(t.dtype).view(t.shape)


def check_guards(raw, fill, what):
    assert (raw[:GUARD] == fill).all() and (raw[-GUARD:] == fill).all(), what


@pytest.mark.parametrize("t,n,k", [(1, 130, 200), (5, 129, 257), (19, 1001, 520), (70, 300, 130), (300, 270, 1100),
                                   (515, 780, 520)])
def test_outputs_stay_in_their_buffers(t, n, k):
    """Every result written into its place of a larger buffer: the bytes around it
    stay, the result is that of a fresh tensor, and no result takes anything from
    the bytes around its operands (0xA5 and 0x7F make large values and NaN)."""
    print(f"guards {t} {n} {k}", flush=True)
    rng = np.random.default_rng(t + n)
    x = values(rng, t, k, BF16).cuda()
    wt = values(rng, n, k, F32, 0.02).cuda()
    dy = values(rng, t, n, BF16).cuda()
    r = torch.from_numpy(rng.integers(0, 256, (t, n)).astype(np.uint8)).cuda()

    def step(place):
        q, w, d = (place(name, nsd.Q4Matrix.empty(a, b, "cuda")) for name, a, b in (("x", t, k), ("w", n, k), ("dy", t, n)))
        xx, dd, rr = place("x in", x), place("dy in", dy), place("random", r)
        xx.copy_(x)
        dd.copy_(dy)
        rr.copy_(r)
        nsd.q4_quantize(xx, out=q)
        nsd.q4_quantize_weights([wt], out=[w])
        nsd.q4_quantize(dd, out=d, random=rr)
        new = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        return [*q.tensors(), *w.tensors(), *d.tensors(), nsd.q4_matmul(q, w, out=place("y", new(t, n))),
                nsd.q4_matmul(d, w, transpose=True, out=place("dx", new(t, k, dtype=F32))),
                nsd.q4_matmul(xx, w, out=place("z", new(t, n))),
                nsd.q4_matmul(dd, w, transpose=True, out=place("dz", new(t, k, dtype=F32))),
                nsd.q4_weight_grad(d, q, out=place("g", new(n, k))),
                nsd.q4_dequantize(w, out=place("v", new(n, k))),
                nsd.q4_dequantize(w, transpose=True, out=place("vt", new(k, n, dtype=F32)))]

    want = step(lambda name, like: like.clone() if isinstance(like, torch.Tensor) else like)
    for fill in (0xA5, 0x7F):
        bufs = []

        def place(name, like):
            if isinstance(like, nsd.Q4Matrix):
                return nsd.Q4Matrix(like.rows, like.cols, *(place(name, v) for v in like.tensors()))
            raw, view = guarded_like(like, fill)
            bufs.append((name, raw))
            return view

        got = step(place)
        torch.cuda.synchronize()
        for name, raw in bufs:
            check_guards(raw, fill, name)
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_overwritten_results_take_the_new_matrix():
    print("overwritten", flush=True)
    rng = np.random.default_rng(4)
    a, b = values(rng, 50, 300, BF16), values(rng, 50, 290, BF16)
    q = nsd.q4_quantize(a.cuda())
    nsd.q4_quantize(b.cuda(), out=q)
    check_matrix(q, host(b), transposed=False)
    w = nsd.q4_quantize_weights([a.cuda()], transposed=False)
    nsd.q4_quantize_weights([b.cuda()], out=w)
    check_matrix(w[0], host(b), transposed=False)
    assert nsd.q4_matmul(q, w[0]).shape == (50, 50) and nsd.q4_dequantize(q).shape == (50, 290)


def test_results_repeat_bit_for_bit():
    print("repeat", flush=True)
    rng = np.random.default_rng(8)
    for t, n, k in ((1, 1024, 2048), (24, 512, 4096), (300, 512, 2048), (2048, 256, 512)):
        x, w, dy = (values(rng, a, b, BF16).cuda() for a, b in ((t, k), (n, k), (t, n)))
        x4, d4 = nsd.q4_quantize(x, transposed=True), nsd.q4_quantize(dy, transposed=True)
        w4 = nsd.q4_quantize_weights([w])[0]
        calls = [lambda: nsd.q4_matmul(x4, w4, dtype=F32), lambda: nsd.q4_matmul(x, w4, dtype=F32),
                 lambda: nsd.q4_weight_grad(d4, x4, dtype=F32)]
        for call in calls:
            want = call()
            for _ in range(3):
                assert torch.equal(want, call())


def test_rows_are_independent():
    """A row's output does not depend on the rows beside it, nor on a padded
    batch's zero rows, where the same kernel runs both."""
    print("independent rows", flush=True)
    rng = np.random.default_rng(9)
    w, _ = weight_of(rng, 300, 700)
    x = values(rng, 48, 700, BF16).cuda()
    z = x.clone()
    z[40:] = 0
    for a, b in ((nsd.q4_quantize(x), nsd.q4_quantize(z)), (x, z)):
        y, yz = nsd.q4_matmul(a, w), nsd.q4_matmul(b, w)
        assert torch.equal(y[:40], yz[:40]) and not yz[40:].any()


# ------------------------------------------------------------ gradients --

def test_gradients_are_differences_of_the_forward_product():
    """With L = sum dy * y, y = x w^T is linear in each code's value, so a changed
    code gives dL / dvalue exactly, but for fp32 sums.  The operands are values that
    both forms of the format hold (blocks of 32 x 32 whose largest is 6), so the
    forward product, the input's gradient and the weight's are of the same L."""
    print("differences", flush=True)
    t, n, k = 64, 160, 320
    rng = np.random.default_rng(12)

    def both_forms(r, c):
        v = rng.choice(ref.code_values(np.arange(16, dtype=np.uint8)), (r, c))
        v[::32, :] = 6.0
        v[:, ::32] = 6.0
        v *= np.repeat(np.repeat(2.0 ** rng.integers(-3, 4, (r // 32, c // 32)), 32, 0), 32, 1)
        q = nsd.q4_quantize(torch.from_numpy(v).float().cuda(), transposed=True)
        assert np.array_equal(host(nsd.q4_dequantize(q)), v) and np.array_equal(host(nsd.q4_dequantize(q, transpose=True)), v.T)
        return q, v

    x, xv = both_forms(t, k)
    w, wv = both_forms(n, k)
    dy, dv = both_forms(t, n)
    grad = host(nsd.q4_weight_grad(dy, x, dtype=F32))
    dx = host(nsd.q4_matmul(dy, w, transpose=True, dtype=F32))
    y0 = host(nsd.q4_matmul(x, w, dtype=F32))
    mag = np.abs(xv) @ np.abs(wv).T
    check_sum(nsd.q4_matmul(x, w, dtype=F32), xv @ wv.T, mag, adds(k), "forward")

    def changed(q, v, i, j):
        """q with another code at (i, j), and its value's step."""
        codes = q.codes.clone()
        old = int(codes[i, j // 2]) >> (4 * (j % 2)) & 15
        new = 0 if old & 7 > 2 else 7
        codes[i, j // 2] = int(codes[i, j // 2]) & (0xF0 if j % 2 == 0 else 0x0F) | new << (4 * (j % 2))
        table = ref.code_values(np.arange(16, dtype=np.uint8))
        step = (table[new] - table[old]) * 2.0 ** (int(q.scales[j // 32, i]) - 127)
        return nsd.Q4Matrix(q.rows, q.cols, codes, q.scales), step

    for _ in range(8):
        i, j = int(rng.integers(n)), int(rng.integers(k))
        w1, step = changed(w, wv, i, j)
        y1 = host(nsd.q4_matmul(x, w1, dtype=F32))
        slope = (dv * (y1 - y0)).sum() / step
        # both products are off by at most adds(k) 2^-23 S + 2^-24 |y|, S growing by |x step|
        s = mag[:, i] + np.abs(xv[:, j] * step)
        noise = (np.abs(dv[:, i]) * 2 * ((adds(k) + 1) * 2.0 ** -23) * s).sum() / abs(step)
        exact = (np.abs(dv[:, i]) * np.abs(xv[:, j])).sum() * (adds(t) + 1) * 2.0 ** -23
        assert abs(slope - grad[i, j]) <= noise + exact, ("w", i, j, slope, grad[i, j], noise)
        r, c = int(rng.integers(t)), int(rng.integers(k))
        x1, step = changed(x, xv, r, c)
        y1 = host(nsd.q4_matmul(x1, w, dtype=F32))
        slope = (dv * (y1 - y0)).sum() / step
        s = mag[r] + np.abs(wv[:, c] * step)
        noise = (np.abs(dv[r]) * 2 * ((adds(k) + 1) * 2.0 ** -23) * s).sum() / abs(step)
        exact = (np.abs(dv[r]) * np.abs(wv[:, c])).sum() * (adds(n) + 1) * 2.0 ** -23
        assert abs(slope - dx[r, c]) <= noise + exact, ("x", r, c, slope, dx[r, c], noise)


def test_layer_step_with_muon():
    """Two linear layers run together as a training step would run them: 4-bit
    forward, both gradients from 4-bit operands (the incoming gradient rounded by
    random bytes) into the packed gradient buffer, the Muon step on it, the updated
    params quantised again, and then served with bf16 rows.  Every stage is checked
    against the oracle on the values the stage before gave."""
    print("layer step with muon", flush=True)
    from oracle import muon
    from synth import update_scale
    rng = np.random.default_rng(21)
    t, d, h = 200, 256, 384
    shapes = [(h, d), (d, h)]  # up, down
    params = [values(rng, r, c, BF16, 0.02).cuda() for r, c in shapes]
    offs, total = nsd.pack_offsets([r * c for r, c in shapes])
    packed = torch.zeros(total, dtype=F32, device="cuda")
    grads = [packed[o:o + r * c].view(r, c) for o, (r, c) in zip(offs, shapes)]
    momenta = [torch.zeros(r, c, device="cuda") for r, c in shapes]
    scales = [update_scale(r, c) for r, c in shapes]
    w4 = nsd.q4_quantize_weights(params)
    grads_want, mags = [0.0, 0.0], [0.0, 0.0]
    for micro in range(2):
        x = values(rng, t, d, BF16).cuda()
        dz = values(rng, t, d, BF16, 1e-2).cuda()
        rz, ru = (rng.integers(0, 256, (t, c)).astype(np.uint8) for c in (d, h))
        x4 = nsd.q4_quantize(x, transposed=True)
        up = nsd.q4_matmul(x4, w4[0])
        u4 = nsd.q4_quantize(up, transposed=True)
        z = nsd.q4_matmul(u4, w4[1])
        z4 = nsd.q4_quantize(dz, transposed=True, random=torch.from_numpy(rz).cuda())
        nsd.q4_weight_grad(z4, u4, out=grads[1], base=grads[1])
        dup = nsd.q4_matmul(z4, w4[1], transpose=True)
        d4 = nsd.q4_quantize(dup, transposed=True, plain=False, random=torch.from_numpy(ru).cuda())
        nsd.q4_weight_grad(d4, x4, out=grads[0], base=grads[0])
        torch.cuda.synchronize()
        wv = [ref.quantized(host(p)) for p in params]
        check_sum(up, *ref.matmul(ref.quantized(host(x)), wv[0]), adds(d), "up")
        check_sum(z, *ref.matmul(ref.quantized(host(up)), wv[1]), adds(h), "down")
        check_sum(dup, *ref.matmul(ref.quantized(host(dz), rz), ref.quantized(host(params[1]).T)), adds(d), "gradient of up")
        for i, (g, r, v) in enumerate(((host(dup), ru, host(x)), (host(dz), rz, host(up)))):
            want, mag = ref.matmul(ref.quantized(g.T, r.T), ref.quantized(v.T))
            grads_want[i] = grads_want[i] + want
            mags[i] = mags[i] + mag
    for i in range(2):
        # two sums, the second added to the first's fp32 result
        check_sum(grads[i], grads_want[i], mags[i], 2 * adds(t), ("grad", i))
    p0, g0 = [host(p) for p in params], [host(g) for g in grads]
    outs = [torch.empty_like(p) for p in params]
    # the fp32 chain: a spread spectrum, on which the bf16 chain's own error says
    # nothing about the gradient that the step was given
    nsd.muon_step(params, grads, momenta, scales, nsd.StepOptions(ns_fp32=True), orth_out=outs)
    nsd.q4_quantize_weights(params, out=w4)
    served = nsd.q4_matmul(x[:3], w4[0])
    torch.cuda.synchronize()
    _, _, want = muon.muon_step(p0, g0, [np.zeros(s) for s in shapes], scales, muon.StepConfig())
    for i, (r, c) in enumerate(shapes):
        err = np.linalg.norm(host(outs[i]) - want[i]) / np.linalg.norm(want[i])
        assert err <= 1e-4 + 2.0 ** -8, (i, err)  # and the rounding of orth_out to bf16
        check_matrix(w4[i], host(params[i]))
    check_sum(served, *ref.matmul(host(x[:3]), ref.quantized(host(params[0]))), d + 25, "served")


# ------------------------------------------------------------- refusals --

def status(fn, *a, **kw):
    with pytest.raises(nsd.DmuonError) as e:
        fn(*a, **kw)
    return e.value.status


def test_binding_refusals():
    print("refusals", flush=True)
    bad, dt = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED_DTYPE
    x = torch.zeros(8, 256, dtype=BF16, device="cuda")
    w = torch.zeros(128, 256, dtype=BF16, device="cuda")
    r = torch.zeros(8, 256, dtype=torch.uint8, device="cuda")
    q, w4 = nsd.q4_quantize(x), nsd.q4_quantize_weights([w])[0]
    assert status(nsd.q4_quantize, x.half()) == dt
    assert status(nsd.q4_quantize, x.t()) == bad  # not contiguous
    assert status(nsd.q4_quantize, x[:, :0]) == bad
    assert status(nsd.q4_quantize, x, plain=False) == bad
    assert status(nsd.q4_quantize, x, random=r.int()) == dt
    assert status(nsd.q4_quantize, x, random=r[:7]) == bad
    assert status(nsd.q4_quantize, x, random=r.cpu()) == bad
    assert status(nsd.q4_quantize, x, out=nsd.Q4Matrix.empty(9, 256, "cuda")) == bad
    assert status(nsd.q4_quantize, x, out=nsd.Q4Matrix(8, 256)) == bad
    assert status(nsd.q4_quantize, x, out=nsd.Q4Matrix(8, 256, q.codes)) == bad
    assert status(nsd.q4_quantize, x.flatten()[8 * 256 - 255:].view(1, 255)) == _lib.ERR_MISALIGNED
    assert status(nsd.q4_quantize_weights, [x, w.cpu()]) == bad
    assert status(nsd.q4_quantize_weights, [w[0]]) == bad
    assert status(nsd.q4_quantize_weights, [w], out=[nsd.Q4Matrix.empty(128, 257, "cuda")]) == bad
    assert status(nsd.q4_quantize_weights, [w], out=[]) == bad
    assert status(nsd.q4_quantize_weights, [w, w], out=[w4, w4]) == _lib.ERR_ALIAS
    for a in (q, x):
        assert status(nsd.q4_matmul, a, w4, transpose=True) == bad  # 256 columns against 128
        assert status(nsd.q4_matmul, a, w4, out=torch.zeros(8, 127, device="cuda")) == bad
        assert status(nsd.q4_matmul, a, w4, dtype=torch.float16) == dt
        assert status(nsd.q4_matmul, a, w4, dtype=F32, out=torch.zeros(8, 128, dtype=BF16, device="cuda")) == bad
    assert status(nsd.q4_matmul, x.float(), w4) == dt and status(nsd.q4_matmul, x.t(), w4, transpose=True) == bad
    assert status(nsd.q4_matmul, nsd.Q4Matrix(8, 256, q.codes, q.scales[:1]), w4) == bad
    assert status(nsd.q4_matmul, nsd.Q4Matrix(8, 256, q.codes.view(torch.int8), q.scales), w4) == dt
    assert status(nsd.q4_dequantize, q, dtype=torch.float16) == dt
    assert status(nsd.q4_dequantize, q, out=torch.zeros(8, 255, device="cuda")) == bad
    x4 = nsd.q4_quantize(x, transposed=True)
    dy = torch.zeros(8, 128, dtype=BF16, device="cuda")
    d4, d7 = nsd.q4_quantize(dy, transposed=True), nsd.q4_quantize(dy[:7], transposed=True)
    assert status(nsd.q4_weight_grad, d7, x4) == bad
    assert status(nsd.q4_weight_grad, d4, x4, out=torch.zeros(128, 255, device="cuda")) == bad
    assert status(nsd.q4_weight_grad, d4, x4, dtype=F32, base=torch.zeros(128, 256, dtype=BF16, device="cuda")) == dt
    tracked = torch.zeros(128, 256, dtype=BF16, device="cuda", requires_grad=True)
    assert status(nsd.q4_weight_grad, d4, x4, base=tracked) == bad
    assert status(nsd.q4_matmul, tracked, w4) == bad
    buf = torch.zeros(128 * 256 + 64, device="cuda")
    assert status(nsd.q4_weight_grad, d4, x4, out=buf[:128 * 256].view(128, 256),
                  base=buf[64:].view(128, 256)) == _lib.ERR_ALIAS
    torch.cuda.synchronize()


def test_a_matrix_against_itself():
    print("a matrix against itself", flush=True)
    torch.manual_seed(4)
    for t, k in ((5, 64), (130, 300), (700, 1000)):
        x = torch.randn(t, k, device="cuda").to(BF16)
        x4 = nsd.q4_quantize(x, transposed=True)
        v, c = unpacked(x4.codes, x4.scales, t, k), unpacked(x4.codes_t, x4.scales_t, k, t)
        for dtype in (BF16, F32):
            check_sum(nsd.q4_matmul(x4, x4, dtype=dtype), (v @ v.t()).cpu().numpy(), (v.abs() @ v.abs().t()).cpu().numpy(),
                      adds(k), (t, k, dtype))
            check_sum(nsd.q4_weight_grad(x4, x4, dtype=dtype), (c @ c.t()).cpu().numpy(), (c.abs() @ c.abs().t()).cpu().numpy(),
                      adds(t), (t, k, dtype, "weight gradient"))


def test_more_rows_than_a_launch_reads_back():
    """2^28 rows are read back a launch."""
    rows = (1 << 28) + 77
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("not enough memory")
    print("rows of two launches", flush=True)
    q = nsd.Q4Matrix.empty(rows, 1, "cuda", True, False)
    q.codes.zero_()
    q.scales.fill_(127)
    q.codes[:, 0] = 2  # the code of 1
    q.codes[-100:, 0] = 4  # of 2
    got = nsd.q4_dequantize(q)
    assert (got[:-100] == 1).all() and (got[-100:] == 2).all()
    del q, got
    torch.cuda.empty_cache()
