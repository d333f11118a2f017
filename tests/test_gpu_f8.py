"""The 8-bit operands: fp4q_f8_quantize and fp4q_f8_gemm.

Bars:
- fp4q_f8_quantize: scales and codes bit-exact against the definition s =
  fp32(amax / 448) (1 when amax = 0), code = e4m3(fp32(x / s)), computed with
  IEEE division on the CPU;
- fp4q_f8_gemm, integer operands under power-of-two scales (every partial sum
  exact in fp32): bit-exact;
- any other operands, against the product in 64 bits: a block's sum is rounded
  (or truncated: a whole ulp, 2^-23) at most once per 16 products the tensor
  core adds, 8 times a block; the scale product rounds once (2^-24) and every
  block is added with one rounding of the running sum (2^-24 of at most the sum
  of magnitudes, ceil(k / 128) times); the result rounds once more:
  |y - y64| <= (16 + 1 + ceil(k / 128)) 2^-24 sum |a sA b sB| + u |y64|, u half
  an ulp of the output type.
"""
import numpy as np
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu
ROW, TILE = "row", "tile"


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import microscaling_fp4_quantization_block_b200 as m
    m.lib()
    return m


def quantize_oracle(x: torch.Tensor, grain: str):
    """Codes (uint8) and scales by the definition, on the CPU."""
    x = x.cpu()
    rows, cols = x.shape
    h = 1 if grain == ROW else 128
    p = torch.nn.functional.pad(x.float(), (0, -cols % 128, 0, -rows % h))
    t = p.view(p.shape[0] // h, h, p.shape[1] // 128, 128)
    a = t.abs().amax(dim=(1, 3))                                    # NaN propagates
    s = torch.where(a == 0, torch.ones_like(a), a / torch.full_like(a, 448.0))
    q = (t / s[:, None, :, None]).reshape(p.shape)[:rows, :cols].contiguous()
    return q.to(torch.float8_e4m3fn), s


def same(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Equal values, signs of zeros included, any NaN equal to any NaN."""
    a, b = a.cpu().float(), b.cpu().float()
    nan = torch.isnan(a) & torch.isnan(b)
    return bool((nan | (a.view(torch.int32) == b.view(torch.int32))).all())


@pytest.mark.parametrize("grain", [ROW, TILE])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (127, 128), (128, 256), (129, 400), (7, 5120),
                                       (300, 3584), (1024, 1040), (2048, 5120), (9500, 128), (40, 5120 * 3 + 16)])
def test_quantize_exact(fq, grain, rows, cols):
    x, _ = workloads.student_t_outliers_bf16(rows, cols, seed=rows * 31 + cols, n_outlier=min(8, cols))
    c, s = fq.fp4q_f8_quantize(x.cuda(), grain)
    wc, ws = quantize_oracle(x, grain)
    assert same(s, ws) and same(c, wc)


@pytest.mark.parametrize("grain", [ROW, TILE])
def test_quantize_extremes(fq, grain):
    """Zero groups, subnormals, the largest finite values, infinities and NaN, each in groups of their own."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn((1024, 256), generator=g)
    x[0:128] = 0.0
    x[128:256] *= 2.0 ** -131
    x[256:384] *= 3.0e38 / x[256:384].abs().max()
    x[384:512] *= 2.0 ** -115                                  # scales just outside the reciprocal's range
    x[512 + 3, 5] = float("inf")
    x[640 + 3, 5] = float("nan")
    x[640 + 4, 6] = float("-inf")
    x[768 + 9, 200] = float("-inf")
    x[896:, ::2] = -0.0
    x = x.to(torch.bfloat16)
    c, s = fq.fp4q_f8_quantize(x.cuda(), grain)
    wc, ws = quantize_oracle(x, grain)
    assert same(s, ws) and same(c, wc)


def test_quantize_views_streams_outputs(fq):
    """A strided view, given outputs, another stream; rows that are not asked for stay as they were."""
    x, _ = workloads.student_t_outliers_bf16(200, 512, seed=9)
    xd = x.cuda()
    view = xd[:, 128:400]
    c, s = fq.fp4q_f8_quantize(view, ROW)
    wc, ws = quantize_oracle(x[:, 128:400].contiguous(), ROW)
    assert same(s, ws) and same(c, wc)
    codes = torch.full((300, 512), 7, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.full((300, 4), -3.0, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fq.fp4q_f8_quantize(xd, ROW, codes=codes[:200], scales=scales[:200], stream=side)
    side.synchronize()
    wc, ws = quantize_oracle(x, ROW)
    assert same(codes[:200], wc) and same(scales[:200], ws)
    assert bool((codes[200:].view(torch.uint8) == 7).all()) and bool((scales[200:] == -3.0).all())


def test_quantize_empty_and_refusals(fq):
    c, s = fq.fp4q_f8_quantize(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert c.shape == (0, 64) and s.shape == (0, 1)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fq.Fp4qError):
        fq.fp4q_f8_quantize(x[:, :24].contiguous())
    with pytest.raises(fq.Fp4qError):
        fq.fp4q_f8_quantize(x.view(-1)[8:8 + 128].view(2, 64))        # 16 bytes past a 32-byte boundary
    with pytest.raises(ValueError):
        fq.fp4q_f8_quantize(x.float())
    with pytest.raises(ValueError):
        fq.fp4q_f8_quantize(x, codes=torch.empty((4, 64), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fq.fp4q_f8_quantize(x.cpu())


# ------------------------------------------------------------------ the product
def widen(c, s, rows_per_scale):
    s = s.double().repeat_interleave(rows_per_scale, 0)[:c.shape[0]]
    return c.cpu().float().double() * s.cpu().repeat_interleave(128, 1)[:, :c.shape[1]]


def check_product(y, a, sa, b, sb, out):
    A, B = widen(a, sa.cpu(), 1), widen(b, sb.cpu(), 128)
    want, mag = A @ B.T, A.abs() @ B.abs().T
    kb = -(-a.shape[1] // 128)
    u = torch.finfo(out).eps / 2
    tol = (17 + kb) * 2.0 ** -24 * mag * (1 + u) + u * want.abs()
    err = (y.cpu().double() - want).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


SHAPES = [(1, 1, 16), (1, 128, 128), (2, 130, 144), (7, 257, 112), (16, 384, 5120), (33, 100, 1040), (64, 1000, 2064),
          (65, 129, 640), (128, 256, 128), (129, 512, 272), (300, 641, 1024), (513, 77, 4112), (1, 4097, 3584)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_against_64_bits(fq, m, n, k, out):
    x, _ = workloads.student_t_outliers_bf16(m, k, seed=m + k, n_outlier=min(8, k))
    w = workloads.gaussian_bf16(n, k, 0.02, seed=n + k)
    a, sa = fq.fp4q_f8_quantize(x.cuda(), ROW)
    b, sb = fq.fp4q_f8_quantize(w.cuda(), TILE)
    y = fq.fp4q_f8_gemm(a, sa, b, sb, out)
    torch.cuda.synchronize()
    assert fq.fp4q_device_fault() == 0
    check_product(y, a, sa, b, sb, out)


@pytest.mark.parametrize("m,n,k", [(5, 300, 400), (130, 520, 256), (2048, 5120, 384), (4097, 2500, 128)])
def test_gemm_exact_on_integers(fq, m, n, k):
    """Integers up to 8 under power-of-two scales: every sum is exact in fp32, many tiles per CTA included."""
    g = torch.Generator(device="cuda").manual_seed(m + n)
    a = torch.randint(-8, 9, (m, k), generator=g, device="cuda").float()
    b = torch.randint(-8, 9, (n, k), generator=g, device="cuda").float()
    kb = -(-k // 128)
    sa = torch.exp2(torch.randint(-2, 3, (m, kb), generator=g, device="cuda").float())
    sb = torch.exp2(torch.randint(-2, 3, (-(-n // 128), kb), generator=g, device="cuda").float())
    y = fq.fp4q_f8_gemm(a.to(torch.float8_e4m3fn), sa, b.to(torch.float8_e4m3fn), sb, torch.float32)
    A = a.double() * sa.double().repeat_interleave(128, 1)[:, :k]
    B = b.double() * sb.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    assert torch.equal(y.double(), A @ B.T)
    assert fq.fp4q_device_fault() == 0


@pytest.mark.parametrize("m,n,k", [(2049, 3001, 128), (2300, 2200, 272), (6200, 1030, 144), (40000, 70, 144), (200, 40000, 144)])
def test_gemm_bands_of_tiles(fq, m, n, k):
    """Tiles are walked in bands of 16 rows of tiles: a last band of one, two and fewer rows than a band, one column, one band."""
    test_gemm_exact_on_integers(fq, m, n, k)


@pytest.mark.parametrize("m", [1, 40, 200])
def test_gemm_keeps_rows_apart(fq, m):
    """A row of A, or of B, that holds NaN or an infinite scale changes its own row, or column, alone."""
    n, k = 300, 512
    x, w = workloads.gaussian_bf16(m, k, 1.0, seed=1), workloads.gaussian_bf16(n, k, 0.02, seed=2)
    a, sa = fq.fp4q_f8_quantize(x.cuda(), ROW)
    b, sb = fq.fp4q_f8_quantize(w.cuda(), TILE)
    clean = fq.fp4q_f8_gemm(a, sa, b, sb)
    a2, b2 = a.clone(), b.clone()
    a2.view(torch.uint8)[m // 2, 7] = 0x7F
    b2.view(torch.uint8)[129, 300] = 0x7F
    y = fq.fp4q_f8_gemm(a2, sa, b2, sb)
    hit = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    hit[m // 2], hit[:, 129] = True, True
    assert bool(torch.isnan(y[hit]).all()) and torch.equal(y[~hit], clean[~hit])
    sa2 = sa.clone()
    sa2[m // 2, 1] = float("inf")
    y = fq.fp4q_f8_gemm(a, sa2, b, sb)
    assert not bool(torch.isfinite(y[m // 2]).any())
    keep = torch.arange(m, device="cuda") != m // 2
    assert torch.equal(y[keep], clean[keep])


def test_gemm_is_the_same_every_time(fq):
    for m, n, k in [(3, 640, 5120), (50, 3584, 4096), (300, 1000, 2048)]:
        a, sa = fq.fp4q_f8_quantize(workloads.gaussian_bf16(m, k, 1.0, seed=m).cuda(), ROW)
        b, sb = fq.fp4q_f8_quantize(workloads.gaussian_bf16(n, k, 0.02, seed=n).cuda(), TILE)
        first = fq.fp4q_f8_gemm(a, sa, b, sb, torch.float32)
        for _ in range(5):
            assert torch.equal(first, fq.fp4q_f8_gemm(a, sa, b, sb, torch.float32))


def test_gemm_strided_side_stream_and_graph(fq):
    m, n, k = 70, 520, 768
    x, w = workloads.gaussian_bf16(m, k, 1.0, seed=3).cuda(), workloads.gaussian_bf16(n, k, 0.02, seed=4).cuda()
    a, sa = fq.fp4q_f8_quantize(x, ROW)
    b, sb = fq.fp4q_f8_quantize(w, TILE)
    want = fq.fp4q_f8_gemm(a, sa, b, sb)
    # strided codes and scales, rows behind the result left alone, another stream
    wide = torch.zeros((m, k + 64), dtype=torch.uint8, device="cuda")
    wide[:, :k] = a.view(torch.uint8)
    ws = torch.zeros((m, 2 * sa.shape[1]), device="cuda")
    ws[:, ::2] = sa
    y = torch.full((m + 9, n), 3.0, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fq.fp4q_f8_gemm(wide[:, :k], ws[:, ::2], b, sb, y=y[:m], stream=side)
    side.synchronize()
    assert torch.equal(y[:m], want) and bool((y[m:] == 3.0).all())
    # quantize and multiply, captured once and replayed on new inputs
    graph = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(graph):
        ca, csa = fq.fp4q_f8_quantize(xs, ROW)
        out = fq.fp4q_f8_gemm(ca, csa, b, sb)
    x2 = workloads.gaussian_bf16(m, k, 2.0, seed=5).cuda()
    xs.copy_(x2)
    graph.replay()
    a2, sa2 = fq.fp4q_f8_quantize(x2, ROW)
    assert torch.equal(out, fq.fp4q_f8_gemm(a2, sa2, b, sb))


def test_gemm_empty_and_refusals(fq):
    a, sa = fq.fp4q_f8_quantize(torch.ones((4, 64), dtype=torch.bfloat16, device="cuda"), ROW)
    b, sb = fq.fp4q_f8_quantize(torch.ones((8, 64), dtype=torch.bfloat16, device="cuda"), TILE)
    assert fq.fp4q_f8_gemm(a[:0], sa[:0], b, sb).shape == (0, 8)
    assert fq.fp4q_f8_gemm(a, sa, b[:0], sb[:0]).shape == (4, 0)
    y = fq.fp4q_f8_gemm(a[:, :0], sa[:, :0], b[:, :0], sb[:, :0])
    assert y.shape == (4, 8) and not y.any()
    with pytest.raises(ValueError):
        fq.fp4q_f8_gemm(a, sa[:2], b, sb)
    with pytest.raises(ValueError):
        fq.fp4q_f8_gemm(a, sa, b[:, :48], sb)
    with pytest.raises(ValueError):
        fq.fp4q_f8_gemm(a, sa, b, sb, torch.float16)
    with pytest.raises(ValueError):
        fq.fp4q_f8_gemm(a, sa, b, sb, y=torch.empty((8, 4), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(fq.Fp4qError):
        fq.fp4q_f8_gemm(a[:, :24].contiguous(), sa, b[:, :24].contiguous(), sb)


def test_past_32_bits(fq):
    """Operands and results of more than 2^31 values: every tile of the integers' product, bit for
    bit where it is looked at (the first and last rows, and a sample between)."""
    m, n, k = 70000, 33024, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randint(-8, 9, (m, k), generator=g, device="cuda").float()
    b = torch.randint(-8, 9, (n, k), generator=g, device="cuda").float()
    sa = torch.exp2(torch.randint(-2, 3, (m, 1), generator=g, device="cuda").float())
    sb = torch.exp2(torch.randint(-2, 3, (-(-n // 128), 1), generator=g, device="cuda").float())
    y = fq.fp4q_f8_gemm(a.to(torch.float8_e4m3fn), sa, b.to(torch.float8_e4m3fn), sb)
    rows = torch.cat([torch.arange(3), torch.randint(0, m, (200,)), torch.arange(m - 3, m)]).cuda()
    want = (a[rows].double() * sa[rows].double()) @ (b.double() * sb.double().repeat_interleave(128, 0)[:n]).T
    assert torch.equal(y[rows].double(), want.to(torch.bfloat16).double())
    # the result as an input: rows past the 2^31st value quantized like any other
    c, s = fq.fp4q_f8_quantize(y, ROW)
    last = y[-130:].clone()
    wc, ws = fq.fp4q_f8_quantize(last, ROW)
    assert torch.equal(c[-130:].view(torch.uint8), wc.view(torch.uint8)) and torch.equal(s[-130:], ws)
    wc, ws = quantize_oracle(last[-4:], ROW)
    assert same(c[-4:], wc) and same(s[-4:], ws)
    c, s = fq.fp4q_f8_quantize(y, TILE)
    wc, ws = quantize_oracle(y[m // 128 * 128:].cpu(), TILE)
    assert same(c[m // 128 * 128:], wc) and same(s[-1:], ws)
    assert fq.fp4q_device_fault() == 0


# ------------------------------------------------------------------ the product, every kernel and split
# What the choice in fp4q_f8_gemm makes of them, by m, n and k:
EVERY = [
    # tiles of 128 x 256, many blocks of k and a short last one: n odd, a multiple of 16 alone; two and more tiles a CTA
    (700, 4001, 2064), (700, 4112, 2064), (2500, 3001, 2064), (1100, 2999, 4112),
    # tiles of 128 x 128, likewise; SMs without a tile
    (1300, 7000, 1040), (1000, 1000, 2320), (200, 3584, 4880),
    # 17 to 32 rows, alone and over clusters of 8; more CTAs because the scales do not fit one; not even in eight
    (17, 257, 112), (24, 1000, 2064), (31, 131, 5136), (32, 20000, 1040), (25, 20000, 14608), (20, 130, 115856),
    # up to 16 and up to 64 rows: the same two
    (5, 20000, 26256), (3, 40, 209056), (40, 20000, 6160), (64, 19100, 11920), (64, 130, 46224), (33, 301, 46224),
    # more than 64 rows in tiles of 64 over clusters
    (130, 130, 9232), (300, 300, 9232),
]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", EVERY)
def test_gemm_every_kernel_on_integers(fq, m, n, k, out):
    """Integers up to 8 under scales of 1/2 to 2: multiples of 1/4 below 2^20, so every fp32 sum in any order is exact
    and the result is the exact one rounded once."""
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    a = torch.randint(-8, 9, (m, k), generator=g, device="cuda").float()
    b = torch.randint(-8, 9, (n, k), generator=g, device="cuda").float()
    kb = -(-k // 128)
    sa = torch.exp2(torch.randint(-1, 2, (m, kb), generator=g, device="cuda").float())
    sb = torch.exp2(torch.randint(-1, 2, (-(-n // 128), kb), generator=g, device="cuda").float())
    guard = torch.full((m + 2, n), 7.0, dtype=out, device="cuda")
    y = fq.fp4q_f8_gemm(a.to(torch.float8_e4m3fn), sa, b.to(torch.float8_e4m3fn), sb, out, y=guard[1:m + 1])
    A = a.double() * sa.double().repeat_interleave(128, 1)[:, :k]
    B = b.double() * sb.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    want = A @ B.T
    assert float(want.abs().max()) < 2.0 ** 20
    assert torch.equal(y, want.to(out))
    assert bool((guard[0] == 7.0).all()) and bool((guard[m + 1] == 7.0).all())
    assert fq.fp4q_device_fault() == 0


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", EVERY)
def test_gemm_every_kernel_against_64_bits(fq, m, n, k, out):
    """Operands as the quantizer makes them, the bar of the product at the top; on the GPU."""
    x, _ = workloads.student_t_outliers_bf16(m, k, seed=m + k, n_outlier=8, device="cuda")
    w = workloads.gaussian_bf16(n, k, 0.02, seed=n + k, device="cuda")
    a, sa = fq.fp4q_f8_quantize(x, ROW)
    b, sb = fq.fp4q_f8_quantize(w, TILE)
    y = fq.fp4q_f8_gemm(a, sa, b, sb, out)
    A = a.double() * sa.double().repeat_interleave(128, 1)[:, :k]
    B = b.double() * sb.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    want, mag = A @ B.T, A.abs() @ B.abs().T
    u = torch.finfo(out).eps / 2
    tol = (17 + sa.shape[1]) * 2.0 ** -24 * mag * (1 + u) + u * want.abs()
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-300)).max())
    assert fq.fp4q_device_fault() == 0
