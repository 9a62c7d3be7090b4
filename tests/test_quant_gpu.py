"""The 8-bit calls on the GPU against the formulas in 64 bits.

Bounds, with u = 2^-24 the half step of fp32 relative to a value:
  * e4m3 has 4 significant bits and its quantum is at least 2^-9, so a value v is
    rounded by at most 2^(max(floor(log2 |v|), -6) - 4).
  * Exact grids: small integers with power-of-two scales, whose sums of products
    are exact in fp32 in any order; d is then the 64-bit result rounded once.
  * Products in general: 128 products are summed in the tensor core, each
    addition off by at most 2^-23 of the sum of magnitudes (2^-16 in all), and
    the blocks are added with one rounding each: |error| <= (2^-16 + (blocks + 4)
    u) S with S = sum |a w|, then half a step of d's type.
"""
import numpy as np
import pytest
import torch

import glu_activation_mlps_gb300 as glu

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    glu.build()
    yield
    assert glu.glu_wait_timeouts() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def half_step(v):
    """Largest rounding of |v| to e4m3."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -60))).clamp_min(-6)
    return torch.exp2(e - 4)


def expand(scale, rows, M, K):
    s = scale.double()
    if rows > 1:
        s = s.repeat_interleave(rows, -2)[..., :M, :]
    return s.repeat_interleave(128, -1)[..., :K]


def block_max(y, rows):
    M, K = y.shape
    p = torch.zeros(-(-M // rows) * rows, -(-K // 128) * 128, dtype=torch.float64, device=y.device)
    p[:M, :K] = y.abs()
    return p.view(-1, rows, p.shape[1] // 128, 128).amax((1, 3))


def check_quantised(q, scale, y, rows, rel, slack=0.0):
    """q, scale against y in 64 bits; rel: relative error of the values and of
    the scale before the rounding to e4m3; slack: an absolute error of y."""
    M, K = y.shape
    assert q.dtype == FP8 and tuple(q.shape) == (M, K) and tuple(scale.shape) == (-(-M // rows), -(-K // 128))
    top = block_max(y, rows).clamp_min(2.0 ** -100)
    top_slack = block_max(slack, rows) if torch.is_tensor(slack) else slack
    assert torch.all((scale.double() * 448 - top).abs() <= rel * top + top_slack)
    s = expand(scale, rows, M, K)
    err = (q.double() * s - y).abs()
    allow = half_step((y / s).abs() * (1 + 2.0 ** -20) + slack / s) * s * (1 + 2.0 ** -20) + rel * y.abs() + slack
    assert torch.all(err <= allow), float((err / allow).max())


def padded(q):
    """q with rows on 16-byte boundaries."""
    K = q.shape[-1]
    wide = torch.zeros((*q.shape[:-1], K + -K % 16), dtype=FP8, device=q.device)
    wide[..., :K] = q
    return wide[..., :K]


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 127), (129, 129), (5, 1000), (300, 272), (2, 20011),
                                       (130, 4096), (1, 40000), (257, 24)])
def test_quantize(rows, cols, dt, block):
    g = gen(rows * 100000 + cols)
    x = (randn(g, rows, cols) * torch.exp(2 * randn(g, rows, cols))).clamp(-60000, 60000).to(DT[dt])
    q, s = glu.quantize(x, block_rows=block)
    # scale: one rounding; the quotient: corrected to a few u, whatever the order
    check_quantised(q, s, x.double(), block, 4 * U)


def test_quantize_ties_go_to_even():
    """3/4 of a block's largest value lies exactly between two e4m3 numbers
    whatever that value is: 336 of 448, between 320 (1.25 * 256, even) and 352."""
    top = torch.arange(1, 129, device="cuda", dtype=torch.float32)[:, None] / 16 + 1
    frac = torch.tensor([1.0, 0.75, 0.375, -0.75, 0.1875], device="cuda")
    x = (top * frac).to(torch.float16)      # at most 9 significant bits
    assert torch.equal(x.float(), top * frac)
    q, s = glu.quantize(x)
    assert torch.equal(q.float(), torch.tensor([448.0, 320.0, 160.0, -320.0, 80.0], device="cuda").expand(128, 5))


def test_quantize_zeros_tiny_and_not_finite():
    x = torch.zeros(4, 300, device="cuda")
    x[1, 5], x[1, 200] = 2.0 ** -120, 1.0
    x[2, 7], x[2, 9], x[2, 299] = float("nan"), 3.0, -5.0
    x[3, 140] = float("inf")
    x[3, 3] = 3e38
    q, s = glu.quantize(x)
    floor = torch.tensor(2.0 ** -100, device="cuda") / 448
    assert torch.all(s[0] == floor) and torch.all(q[0].float() == 0)
    assert s[1, 0] == floor and q[1, 5].float() == 0 and q[1, 200].float() == 448
    # a NaN stays a NaN and does not reach the scale
    assert torch.isnan(q[2, 7].float()) and s[2, 0] * 448 == 3 and q[2, 9].float() == 448
    assert q[2, 299].float() == -448 and torch.isfinite(q[2, 8].float())
    assert q[3, 3].float() == 448 and torch.all(torch.isfinite(q[3, :128].float()))
    assert torch.all(torch.isnan(q[3, 128:256].float()))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("block", [1, 128])
def test_quantize_strided_and_guarded(dt, block):
    """Column slices in and out; nothing outside the outputs is written."""
    g = gen(5)
    for off, cols in ((0, 256), (3, 200), (8, 136)):
        x = randn(g, 200, 512).to(DT[dt])[:, off:off + cols]
        qb = torch.full((204, 600), 0x55, dtype=torch.uint8, device="cuda")
        q = qb.view(FP8)[2:202, 16:16 + cols]
        srows = 200 if block == 1 else 2
        sb = torch.full((srows + 2, 9), 7.0, device="cuda")
        s = sb[1:1 + srows, 3:3 + -(-cols // 128)]
        glu.quantize(x, block_rows=block, q=q, scale=s)
        check_quantised(q, s, x.double(), block, 4 * U)
        mask = torch.ones_like(qb, dtype=torch.bool)
        mask[2:202, 16:16 + cols] = False
        assert torch.all(qb[mask] == 0x55)
        mask = torch.ones_like(sb, dtype=torch.bool)
        mask[1:1 + srows, 3:3 + -(-cols // 128)] = False
        assert torch.all(sb[mask] == 7.0)


def test_quantize_weights_of_experts_and_batches():
    g = gen(6)
    w = randn(g, 3, 200, 300).to(torch.bfloat16)
    q, s = glu.quantize(w, block_rows=128)
    assert q.stride(-2) % 16 == 0 and tuple(s.shape) == (3, 2, 3)
    for e in range(3):
        check_quantised(q[e], s[e], w[e].double(), 128, 4 * U)
    x = randn(g, 2, 5, 256)
    q, s = glu.quantize(x)
    assert q.shape == x.shape and tuple(s.shape) == (2, 5, 2)
    check_quantised(q.view(10, 256), s.view(10, 2), x.view(10, 256).double(), 1, 4 * U)


def test_quantize_past_32_bit_offsets():
    rows, cols = 70000, 65536            # 4.6e9 values
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(cols, device="cuda").to(torch.bfloat16)
    x[rows // 2, 17] = 3.0
    q, s = glu.quantize(x)
    check_quantised(q[-1:], s[-1:], x[-1:].double(), 1, 4 * U)
    assert q[rows // 2, 17].float() == 448 and int((q.view(torch.uint8)[:-1] != 0).sum()) == 1
    del q, s
    q, s = glu.quantize(x, block_rows=128)
    check_quantised(q[-112:], s[-1:], x[-112:].double(), 128, 4 * U)


@pytest.mark.parametrize("dt,cols", [("f32", 1 << 28), ("bf16", (1 << 28) - 1), ("f32", (1 << 27) + 5)])
def test_quantize_the_widest_rows(dt, cols):
    """Rows with more stretches than one dimension of a grid counts: every block's scale and values."""
    g = gen(cols % 1000)
    x = torch.randint(-7, 8, (1, cols), generator=g, device="cuda", dtype=torch.int8).to(DT[dt])
    at = torch.arange(0, cols, 128, device="cuda")
    x[0, at] = (8 + at // 128 % 119).to(DT[dt])         # each block's maximum, 8 to 126
    top = x[0, at].float()
    sbuf = torch.full((1, at.numel() + 8), 3.0, device="cuda")
    qbuf = torch.full((1, cols + 256), 0x55, dtype=torch.uint8, device="cuda")
    q, s = glu.quantize(x, q=qbuf.view(FP8)[:, :cols], scale=sbuf[:, :at.numel()])
    assert torch.equal(s[0], top / torch.full_like(top, 448))
    assert torch.all(q[0, at].float() == 448)
    assert torch.all(sbuf[0, at.numel():] == 3.0) and torch.all(qbuf[0, cols:] == 0x55)
    for lo in range(0, cols, 1 << 24):
        part = slice(lo, min(cols, lo + (1 << 24)))
        check_quantised(q[:, part], s[:, lo // 128:-(-part.stop // 128)], x[:, part].double(), 1, 4 * U)


# ---------------------------------------------------------------- add + RMSNorm

# y = s * rstd * gamma: the sum of squares has at most 64 / 2 chained roundings
# per thread, 10 in its joining and 4 behind it, halved by the root, then two
# products and the scale's division: below 32 u
NORM_REL = 32 * U


def check_norm(x, res, gamma, eps, h, q, s, rstd=None):
    ssum = x.double() + res.double()
    dt = x.dtype
    want = ssum.to(torch.float32).to(dt) if dt != torch.float32 else (x + res)
    assert torch.equal(h, want)
    r = 1 / torch.sqrt((ssum ** 2).mean(-1, keepdim=True) + eps)
    check_quantised(q, s, ssum * r * gamma.double(), 1, NORM_REL)
    if rstd is not None:
        assert torch.all((rstd.double() - r[:, 0]).abs() <= NORM_REL * r[:, 0])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (7, 127), (3, 128), (1, 129), (65, 1000), (33, 512), (5, 4096), (4, 4104),
                                       (9, 5000), (2, 8191), (3, 16384), (2, 16400), (1, 32768), (2, 32767)])
def test_add_rmsnorm_q(rows, cols, dt):
    g = gen(rows * 7 + cols)
    x, res = randn(g, rows, cols).to(DT[dt]), (3 * randn(g, rows, cols)).to(DT[dt])
    gamma = (1 + 0.3 * randn(g, cols)).to(DT[dt])
    h, q, s, rstd = glu.add_rmsnorm_q(x, res, gamma, 1e-5, rstd=True)
    check_norm(x, res, gamma, 1e-5, h, q, s, rstd)
    # the same h and rstd as the call without quantisation, h in place
    x2, r2 = x.clone(), res.clone()
    h2, q2, s2 = glu.add_rmsnorm_q(x2, r2, gamma, 1e-5, h=x2)
    assert h2 is x2 and torch.equal(x2, h) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8))
    glu.add_rmsnorm_q(x, r2, gamma, 1e-5, h=r2, q=q2, scale=s2)
    assert torch.equal(r2, h) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [256, 264, 251])
def test_add_rmsnorm_q_strided_and_guarded(dt, cols):
    g = gen(cols)
    x, res = (randn(g, 130, 600).to(DT[dt])[:, 8:8 + cols] for _ in range(2))
    gamma = randn(g, cols).to(DT[dt])
    hb = torch.full((134, 700), 9.0, dtype=DT[dt], device="cuda")
    qb = torch.full((134, 700), 0x33, dtype=torch.uint8, device="cuda")
    sb = torch.full((134, 9), 5.0, device="cuda")
    h, q, s = hb[2:132, 5:5 + cols], qb.view(FP8)[2:132, 7:7 + cols], sb[2:132, 1:1 + -(-cols // 128)]
    glu.add_rmsnorm_q(x, res, gamma, 1e-6, h=h, q=q, scale=s)
    check_norm(x, res, gamma, 1e-6, h, q, s)
    for buf, fill, sl in ((hb, 9.0, slice(5, 5 + cols)), (qb, 0x33, slice(7, 7 + cols)),
                          (sb, 5.0, slice(1, 1 + -(-cols // 128)))):
        mask = torch.ones(buf.shape, dtype=torch.bool, device="cuda")
        mask[2:132, sl] = False
        assert torch.all(buf[mask] == fill)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_add_rmsnorm_q_tiny_values(dt):
    """Rows, and blocks of gamma, next to nothing: the scale's floor holds y."""
    g = gen(77)
    x = randn(g, 6, 512) * torch.tensor([1.0, 1e-15, 1e-25, 1e-31, 1e-36, 0.0], device="cuda")[:, None]
    x = x.to(DT[dt])
    gamma = torch.ones(512, device="cuda")
    gamma[128:256], gamma[256:384] = 1e-20, 1e-33
    gamma = (gamma * (1 + 0.1 * randn(g, 512))).to(DT[dt])
    for eps in (1e-5, 1e-30):
        h, q, s = glu.add_rmsnorm_q(x, torch.zeros_like(x), gamma, eps)
        r = 1 / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + float(np.float32(eps)))
        # squares below 2^-149 vanish in the sum: where the mean square is not far
        # above that, rstd is eps's
        y = x.double() * r * gamma.double()
        keep = (x.double() ** 2).mean(-1) > 2.0 ** -110
        keep |= (x.double() ** 2).mean(-1) < 2.0 ** -30 * eps
        # values of 2^-149 quanta, and a product of that size: an absolute slack
        check_quantised(q[keep], s[keep], y[keep], 1, NORM_REL, 2.0 ** -120)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_add_rmsnorm_q_large_gammas(dt):
    """Gammas just below 2^100 on rows from 2^-9 to 2^14 (rstd in the scale, or
    with the values), one value of a row far above the rest."""
    g = gen(78)
    x = randn(g, 24, 8192) * torch.exp2(torch.arange(-9, 15, device="cuda").float())[:, None]
    x[:, 77] *= 64
    x = x.to(DT[dt])
    gamma = (2.0 ** 100 * (1 - 2.0 ** -8) * (1 - torch.rand(8192, generator=g, device="cuda") / 4)).to(DT[dt])
    assert float(gamma.max()) < 2.0 ** 100
    h, q, s, rstd = glu.add_rmsnorm_q(x, torch.zeros_like(x), gamma, 1e-5, rstd=True)
    check_norm(x, torch.zeros_like(x), gamma, 1e-5, h, q, s, rstd)


def test_add_rmsnorm_q_zero_rows_and_nan():
    x = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    x[1, 3] = float("nan")
    x[2] = 2.0
    gamma = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    h, q, s = glu.add_rmsnorm_q(x, torch.zeros_like(x), gamma, 1e-5)
    assert torch.all(q[0].float() == 0) and torch.all(torch.isnan(q[1].float())) and torch.all(q[2].float() == 448)


# ---------------------------------------------------------------- products

def grid(g, M, K, rows):
    """Small integers and power-of-two scales."""
    v = torch.randint(-4, 5, (M, K), generator=g, device="cuda").to(torch.float32)
    s = torch.exp2(torch.randint(-1, 2, (-(-M // rows), -(-K // 128)), generator=g, device="cuda").float())
    return padded(v.to(FP8)), s


def value(q, s, rows):
    return q.double() * expand(s, rows, *q.shape[-2:])


# rows around the tiles' sizes (16, 32, 64, 128, 256), K and N around 128 and
# through several splits of K
SHAPES = [(1, 128, 128), (1, 1, 1), (2, 5000, 40), (15, 300, 130), (16, 128, 4096), (17, 2048, 256), (32, 1024, 384),
          (33, 16, 500), (64, 4100, 129), (65, 512, 1000), (100, 9000, 128), (128, 640, 257), (129, 256, 1024),
          (255, 384, 264), (256, 128, 256), (257, 1000, 8), (300, 130, 2000), (513, 2000, 300), (1030, 129, 513),
          (2000, 256, 4096)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_gemm_q_nt_exact_grid(M, K, N, dt):
    g = gen(M + K + N)
    a, sa = grid(g, M, K, 1)
    b, sb = grid(g, N, K, 128)
    d = glu.gemm_q_nt(a, sa, b, sb, dtype=DT[dt])
    want = value(a, sa, 1) @ value(b, sb, 128).T
    assert torch.equal(d, want.to(torch.float32).to(DT[dt]))
    assert torch.equal(d, glu.gemm_q_nt(a, sa, b, sb, dtype=DT[dt]))


def random_q(g, M, K, rows, spread=1.0):
    v = randn(g, M, K) * torch.exp(spread * randn(g, K))
    return glu.quantize(v, block_rows=rows)


def product64(a, sa, b, sb):
    A, B = value(a, sa, 1), value(b, sb, 128)
    blocks = -(-a.shape[1] // 128)
    return A @ B.T, (2.0 ** -16 + (blocks + 4) * U) * (A.abs() @ B.abs().T)


@pytest.mark.parametrize("M,K,N", [(3, 4096, 1000), (40, 1500, 300), (200, 3000, 520), (600, 777, 640)])
def test_gemm_q_nt_random(M, K, N):
    g = gen(M)
    a, sa = random_q(g, M, K, 1)
    b, sb = random_q(g, N, K, 128)
    for dt in (torch.float16, torch.bfloat16):
        d = glu.gemm_q_nt(a, sa, b, sb, dtype=dt)
        want, err = product64(a, sa, b, sb)
        if dt == torch.float16 and want.abs().max() > 60000:
            continue
        half = torch.finfo(dt).eps / 2
        assert torch.all((d.double() - want).abs() <= err + half * (want.abs() + err) + 2.0 ** -25)


def guarded_out(M, N, dt, pad=3):
    buf = torch.full((M + 4, N + 2 * pad), 7.0, device="cuda").to(dt)
    return buf, buf[2:M + 2, pad:pad + N]


def outside(buf, M, N, pad=3):
    mask = torch.ones(buf.shape, dtype=torch.bool, device="cuda")
    mask[2:M + 2, pad:pad + N] = False
    return mask


@pytest.mark.parametrize("M,K,N,pad", [(5, 300, 200, 3), (40, 256, 130, 8), (300, 256, 250, 3), (300, 256, 256, 8)])
def test_gemm_q_nt_strided_and_guarded(M, K, N, pad):
    g = gen(N)
    wide = torch.randint(-4, 5, (M, 512), generator=g, device="cuda").float().to(FP8)
    a = wide[:, 32:32 + K]
    sa = torch.exp2(torch.randint(-1, 2, (M, 9), generator=g, device="cuda").float())[:, 2:2 + -(-K // 128)]
    b = torch.randint(-4, 5, (N, 640), generator=g, device="cuda").float().to(FP8)[:, 64:64 + K]
    sb = torch.exp2(torch.randint(-1, 2, (-(-N // 128), 7), generator=g, device="cuda").float())[:, 1:1 + -(-K // 128)]
    buf, d = guarded_out(M, N, torch.bfloat16, pad)
    glu.gemm_q_nt(a, sa, b, sb, d=d)
    want = (value(a, sa, 1) @ value(b, sb, 128).T).float().to(torch.bfloat16)
    assert torch.equal(d, want) and torch.all(buf[outside(buf, M, N, pad)] == 7.0)


def test_gemm_q_nt_empty_sums_and_sizes():
    a, sa = torch.empty(5, 0, dtype=FP8, device="cuda"), torch.empty(5, 0, device="cuda")
    b, sb = torch.empty(40, 0, dtype=FP8, device="cuda"), torch.empty(1, 0, device="cuda")
    d = torch.full((5, 40), 3.0, dtype=torch.bfloat16, device="cuda")
    glu.gemm_q_nt(a, sa, b, sb, d=d)
    assert torch.all(d == 0)
    a, sa = torch.empty(0, 256, dtype=FP8, device="cuda"), torch.empty(0, 2, device="cuda")
    b, sb = torch.empty(40, 256, dtype=FP8, device="cuda"), torch.empty(1, 2, device="cuda")
    assert glu.gemm_q_nt(a, sa, b, sb).shape == (0, 40)
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = torch.full((3, 40), 3.0, dtype=torch.bfloat16, device="cuda")
    x, sx = torch.zeros(3, 256, dtype=FP8, device="cuda"), torch.ones(3, 2, device="cuda")
    glu.gemm_q_nt(x, sx, torch.empty(0, 40, 256, dtype=FP8, device="cuda"), torch.empty(0, 1, 2, device="cuda"), d=d,
                  offsets=off)
    assert torch.all(d == 3.0)


ACT64 = {
    "silu": lambda g: g * torch.special.expit(g),
    "gelu_erf": lambda g: g * torch.special.ndtr(g),
    "gelu_tanh": lambda g: g * torch.special.expit(2 * (2 / np.pi) ** 0.5 * (g + 0.044715 * g ** 3)),
    "relu": lambda g: g.clamp_min(0),
}


def gated64(x, sx, wg, sg, wu, su, act):
    """y in 64 bits and a bound of its fp32 error: the products' errors through
    act (whose slope is below 1.13) and u, and the activation's own (2^-20 of
    |u| times |act| or, in the tails, of 0.6 |u|)."""
    G, eg = product64(x, sx, wg, sg)
    Up, eu = product64(x, sx, wu, su)
    a = ACT64[act](G)
    y = a * Up
    err = 1.13 * eg * (Up.abs() + eu) + a.abs() * eu + 2.0 ** -20 * (Up.abs() + eu) * (a.abs() + 0.6)
    return y, err


def check_gated(y, ys, x, sx, wg, sg, wu, su, act):
    want, err = gated64(x, sx, wg, sg, wu, su, act)
    check_quantised(y, ys, want, 1, 8 * U, err)


@pytest.mark.parametrize("act", ["silu", "gelu_erf", "gelu_tanh", "relu"])
@pytest.mark.parametrize("M,K,I", [(1, 128, 128), (1, 4096, 512), (3, 300, 70), (16, 1024, 300), (17, 700, 129), (32, 256, 1),
                                   (33, 512, 384), (130, 1000, 200), (256, 128, 128), (300, 2000, 1030), (700, 256, 144)])
def test_gemm_q_fwd(M, K, I, act):
    g = gen(M + I)
    x, sx = random_q(g, M, K, 1, 0.5)
    wg, sg = glu.quantize(randn(g, I, K) / K ** 0.5, block_rows=128)
    wu, su = glu.quantize(randn(g, I, K) / K ** 0.5, block_rows=128)
    y, ys = glu.gemm_q_fwd(x, sx, wg, sg, wu, su, act=act)
    check_gated(y, ys, x, sx, wg, sg, wu, su, act)
    y2, ys2 = glu.gemm_q_fwd(x, sx, wg, sg, wu, su, act=act)
    assert torch.equal(y.view(torch.uint8), y2.view(torch.uint8)) and torch.equal(ys, ys2)
    # into a padded, odd place
    buf = torch.full((M + 4, I + 6), 0x44, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((M + 4, ys.shape[1] + 6), 7.0, device="cuda")
    yo, so = buf.view(FP8)[2:M + 2, 3:3 + I], sbuf[2:M + 2, 3:3 + ys.shape[1]]
    glu.gemm_q_fwd(x, sx, wg, sg, wu, su, y=yo, y_scale=so, act=act)
    assert torch.equal(yo.float().nan_to_num(), y.float().nan_to_num()) and torch.equal(so, ys)
    assert torch.all(buf[outside(buf, M, I)] == 0x44) and torch.all(sbuf[outside(sbuf, M, ys.shape[1])] == 7.0)


@pytest.mark.parametrize("act", ["silu", "gelu_erf", "gelu_tanh", "relu"])
@pytest.mark.parametrize("M", [8, 300])
def test_gated_nan_stays_alone(M, act):
    """A NaN in some rows of the gate and up weights is a NaN in those columns of
    y and takes no part in the scales: everything else has the bits of weights
    whose rows are zeros there, in the narrow kernel (8 rows) and the wide one."""
    g = gen(M)
    K, I = 384, 300
    x, sx = random_q(g, M, K, 1, 0.5)
    nans, zeros = [], []
    cols = [5, 130, 299], [66, 131, 257]        # of the gate, of up
    for at in cols:
        w, s = glu.quantize(randn(g, I, K) / K ** 0.5, block_rows=128)
        for out, byte in ((nans, 0x7F), (zeros, 0)):
            v = w.clone()
            v.view(torch.uint8)[at] = byte
            out += [v, s]
    y, ys = glu.gemm_q_fwd(x, sx, *nans, act=act)
    y0, ys0 = glu.gemm_q_fwd(x, sx, *zeros, act=act)
    hit = torch.zeros(I, dtype=torch.bool, device="cuda")
    hit[cols[0] + cols[1]] = True
    assert torch.all(torch.isnan(y.float()[:, hit]))
    assert torch.equal(y.view(torch.uint8)[:, ~hit], y0.view(torch.uint8)[:, ~hit])
    assert torch.equal(ys, ys0)


# ---------------------------------------------------------------- by expert

LOADS = [[5], [0, 3, 0, 1], [16, 16], [17, 0, 40, 1, 0], [200, 0, 3], [256, 256], [1, 700, 90, 0, 255, 257],
         [0, 0, 0], [2] * 70, [130] * 9]


def experts(g, E, N, K):
    qs = [grid(g, N, K, 128) for _ in range(E)]
    w = torch.zeros(E, N, K + -K % 16, dtype=FP8, device="cuda")[..., :K]
    for e, (q, _) in enumerate(qs):
        w[e] = q
    return w, torch.stack([s for _, s in qs])


def cuts(loads, first=0):
    return torch.tensor(np.cumsum([first, *loads]), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("N,K", [(128, 256), (300, 200), (264, 1024)])
@pytest.mark.parametrize("loads", LOADS, ids=lambda v: "x".join(map(str, v[:6])))
def test_grouped_nt_exact_grid(loads, N, K):
    g = gen(sum(loads) + N)
    first, behind = 3, 9                # rows that no expert has, on either side
    M = first + sum(loads) + behind
    a, sa = grid(g, M, K, 1)
    for rows in (a[:first], a[M - behind:]):
        rows.copy_(torch.full(rows.shape, float("nan"), device="cuda").to(FP8))     # may hold anything
    w, sw = experts(g, len(loads), N, K)
    off = cuts(loads, first)
    buf, d = guarded_out(M, N, torch.bfloat16)
    glu.gemm_q_nt(a, sa, w, sw, d=d, offsets=off)
    lo = first
    assert torch.all(d[:first] == 7.0) and torch.all(d[M - behind:] == 7.0)
    assert torch.all(buf[outside(buf, M, N)] == 7.0)
    for e, n in enumerate(loads):
        want = value(a[lo:lo + n], sa[lo:lo + n], 1) @ value(w[e], sw[e], 128).T
        assert torch.equal(d[lo:lo + n], want.float().to(torch.bfloat16)), e
        lo += n
    # into an aligned place too (the copy engine's stores stop at an expert's last row)
    d2 = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    glu.gemm_q_nt(a, sa, w, sw, d=d2, offsets=off)
    assert torch.equal(d2, d)


@pytest.mark.parametrize("act", ["silu", "relu"])
@pytest.mark.parametrize("loads", LOADS, ids=lambda v: "x".join(map(str, v[:6])))
def test_grouped_fwd(loads, act):
    g = gen(sum(loads))
    I, K, behind = 200, 260, 4
    M = sum(loads) + behind
    x, sx = random_q(g, M, K, 1, 0.5)
    ws = [glu.quantize(randn(g, len(loads), I, K) / K ** 0.5, block_rows=128) for _ in range(2)]
    y = torch.full((M, I + 8), 0x11, dtype=torch.uint8, device="cuda").view(FP8)[:, :I]
    ys = torch.full((M, 2), 7.0, device="cuda")
    glu.gemm_q_fwd(x, sx, *ws[0], *ws[1], y=y, y_scale=ys, act=act, offsets=cuts(loads))
    lo = 0
    for e, n in enumerate(loads):
        if n:
            check_gated(y[lo:lo + n], ys[lo:lo + n], x[lo:lo + n], sx[lo:lo + n], ws[0][0][e], ws[0][1][e], ws[1][0][e],
                        ws[1][1][e], act)
        lo += n
    assert torch.all(y.view(torch.uint8)[lo:] == 0x11) and torch.all(ys[lo:] == 7.0)


def test_many_experts_many_rows_long_sums():
    """The most experts (and one more is refused), a hundred thousand rows, a
    sum of 70000 terms: exact grids, both kernels."""
    g = gen(41)
    E, N, K = 1024, 130, 128
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").float().to(FP8)
    sw = torch.exp2(torch.randint(-1, 2, (E, 2, 1), generator=g, device="cuda").float())
    for per in (1, 40, 100):
        loads = torch.randint(0, 2 * per + 1, (E,), generator=g, device="cuda")
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[1:] = loads.cumsum(0)
        M = int(off[-1])
        a, sa = grid(g, M, K, 1)
        d = glu.gemm_q_nt(a, sa, w, sw, offsets=off)
        e = torch.repeat_interleave(torch.arange(E, device="cuda"), loads)
        for lo in range(0, M, 20000):       # each row with its own expert's weights
            sl = slice(lo, min(M, lo + 20000))
            scale = sw[e[sl]].repeat_interleave(128, 1)[:, :N, 0].double()
            want = torch.einsum("mk,mnk->mn", a[sl].float(), w.float()[e[sl]]).double() * sa[sl].double() * scale
            assert torch.equal(d[sl], want.float().to(torch.bfloat16))
    with pytest.raises(glu.GluError) as err:
        glu.gemm_q_nt(a, sa, torch.empty(1025, N, K, dtype=FP8, device="cuda"), torch.empty(1025, 2, 1, device="cuda"),
                      offsets=torch.zeros(1026, dtype=torch.int32, device="cuda"))
    assert err.value.status == -2
    for M, K, N in ((100003, 200, 72), (5, 70000, 200), (300, 70000, 264)):
        a, sa = grid(g, M, K, 1)
        b, sb = grid(g, N, K, 128)
        assert torch.equal(glu.gemm_q_nt(a, sa, b, sb, dtype=torch.float16),
                           (value(a, sa, 1) @ value(b, sb, 128).T).float().half())


def test_grouped_agrees_with_dense():
    """One expert with every row is the dense product bit for bit where both
    take the same kernel (sums do not depend on the tile order)."""
    g = gen(3)
    for M in (300, 600):
        a, sa = random_q(g, M, 640, 1)
        w, sw = random_q(g, 1000, 640, 128)
        off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        d = glu.gemm_q_nt(a, sa, w, sw)
        assert torch.equal(d, glu.gemm_q_nt(a, sa, w[None], sw[None], offsets=off))


def test_offsets_out_of_order_stay_inside():
    """Decreasing, negative or too large offsets give no access outside the
    operands: the guards around d keep their values."""
    g = gen(4)
    for M in (40, 900):
        a, sa = grid(g, M, 256, 1)
        w, sw = experts(g, 4, 136, 256)
        for bad in ([0, M, 5, M, 2], [-7, 3, -100, 2 ** 31 - 1, 9], [2 ** 31 - 1] * 5, [M, 0, M, 0, M], [0] * 5):
            off = torch.tensor(bad, dtype=torch.int32, device="cuda")
            buf, d = guarded_out(M, 136, torch.bfloat16)
            glu.gemm_q_nt(a, sa, w, sw, d=d, offsets=off)
            assert torch.all(buf[outside(buf, M, 136)] == 7.0)


def test_experts_weights_past_32_bit_offsets():
    """40 experts of 112 MB: the last one's weights lie past 4 GB."""
    E, N, K = 40, 8192, 14336
    w = torch.zeros(E, N, K, dtype=FP8, device="cuda")
    sw = torch.ones(E, N // 128, K // 128, device="cuda")
    g = gen(9)
    for e in (0, E - 1):
        w[e] = torch.randint(-1, 2, (N, K), generator=g, device="cuda").float().to(FP8)
    for n in (5, 70):
        a = torch.randint(-2, 3, (2 * n, K), generator=g, device="cuda").float().to(FP8)
        sa = torch.ones(2 * n, K // 128, device="cuda")
        off = torch.tensor([0] + [n] * (E - 1) + [2 * n], dtype=torch.int32, device="cuda")
        d = glu.gemm_q_nt(a, sa, w, sw, offsets=off, dtype=torch.float16)
        assert torch.equal(d[:n], (a[:n].float() @ w[0].float().T).half())
        assert torch.equal(d[n:], (a[n:].float() @ w[-1].float().T).half())


# ---------------------------------------------------------------- the MLP, a run of them, streams and graphs

def test_mlp_is_its_two_products():
    g = gen(12)
    for M, H, I in ((1, 256, 384), (20, 500, 300), (300, 384, 1000)):
        x, sx = random_q(g, M, H, 1, 0.5)
        wg, wu = (glu.quantize(randn(g, I, H) / H ** 0.5, block_rows=128) for _ in range(2))
        wd = glu.quantize(randn(g, H, I) / I ** 0.5, block_rows=128)
        out = glu.mlp_q_fwd(x, sx, *wg, *wu, *wd, act="gelu_tanh", dtype=torch.float16)
        y, ys = glu.gemm_q_fwd(x, sx, *wg, *wu, act="gelu_tanh")
        assert torch.equal(out, glu.gemm_q_nt(y, ys, *wd, dtype=torch.float16))


def test_mlp_by_expert():
    g = gen(13)
    loads, H, I = [0, 30, 200, 1], 272, 400
    M = sum(loads) + 5
    x, sx = random_q(g, M, H, 1, 0.5)
    wg, wu = (glu.quantize(randn(g, 4, I, H) / H ** 0.5, block_rows=128) for _ in range(2))
    wd = glu.quantize(randn(g, 4, H, I) / I ** 0.5, block_rows=128)
    off = cuts(loads)
    out = torch.full((M, H), 7.0, dtype=torch.bfloat16, device="cuda")
    glu.mlp_q_fwd(x, sx, *wg, *wu, *wd, out=out, offsets=off)
    y, ys = glu.gemm_q_fwd(x, sx, *wg, *wu, offsets=off)
    want = torch.full((M, H), 7.0, dtype=torch.bfloat16, device="cuda")
    glu.gemm_q_nt(y, ys, *wd, d=want, offsets=off)
    assert torch.equal(out, want) and torch.all(out[sum(loads):] == 7.0)


def test_without_experts():
    """A part of a model that holds no expert: every row of the outputs is left as it was."""
    M, H, I = 5, 256, 384
    x, sx = random_q(gen(2), M, H, 1)

    def none(n, k):
        return torch.empty(0, n, k, dtype=FP8, device="cuda"), torch.empty(0, -(-n // 128), -(-k // 128), device="cuda")

    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((M, H), 7.0, dtype=torch.bfloat16, device="cuda")
    y, ys = torch.full((M, I), 0x11, dtype=torch.uint8, device="cuda").view(FP8), torch.full((M, 3), 7.0, device="cuda")
    glu.mlp_q_fwd(x, sx, *none(I, H), *none(I, H), *none(H, I), out=out, offsets=off)
    glu.gemm_q_fwd(x, sx, *none(I, H), *none(I, H), y=y, y_scale=ys, offsets=off)
    assert torch.all(out == 7.0) and torch.all(y.view(torch.uint8) == 0x11) and torch.all(ys == 7.0)


def block(x, res, gamma, wg, wu, wd):
    """One decoder sub-block: norm, MLP, and the next norm over its result."""
    h, q, s = glu.add_rmsnorm_q(x, res, gamma)
    out = glu.mlp_q_fwd(q, s, *wg, *wu, *wd)
    return glu.add_rmsnorm_q(out, h, gamma)


@pytest.mark.parametrize("M", [1, 24, 200])
def test_a_block_on_a_side_stream_and_in_graphs(M):
    """The run a user makes, eagerly, on another stream and replayed from two
    captured graphs that follow each other: the same bits."""
    g = gen(M)
    H, I = 512, 1100
    x, res = (randn(g, M, H).to(torch.bfloat16) for _ in range(2))
    gamma = (1 + 0.1 * randn(g, H)).to(torch.bfloat16)
    wg, wu = (glu.quantize(randn(g, I, H) / H ** 0.5, block_rows=128) for _ in range(2))
    wd = glu.quantize(randn(g, H, I) / I ** 0.5, block_rows=128)
    want = [t.clone() for t in block(x, res, gamma, wg, wu, wd)]

    def same(got):
        return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block(x, res, gamma, wg, wu, wd)
    torch.cuda.current_stream().wait_stream(side)
    assert same(got)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = block(x, res, gamma, wg, wu, wd)
        graphs.append((gr, out))
    for _ in range(3):
        for gr, _ in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert all(same(out) for _, out in graphs)
    x.add_(1.0)
    want = [t.clone() for t in block(x, res, gamma, wg, wu, wd)]
    for gr, _ in graphs:
        gr.replay()
    assert all(same(out) for _, out in graphs)


def test_stream_argument():
    """Calls given another stream: their results, and the workspace of the MLP,
    are not handed out again while that stream still works."""
    g = gen(17)
    M, H, I = 64, 512, 700
    x, sx = random_q(g, M, H, 1, 0.5)
    wg, wu = (glu.quantize(randn(g, I, H) / H ** 0.5, block_rows=128) for _ in range(2))
    wd = glu.quantize(randn(g, H, I) / I ** 0.5, block_rows=128)
    want = glu.mlp_q_fwd(x, sx, *wg, *wu, *wd)
    xb = randn(g, M, H).to(torch.bfloat16)
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    norm = glu.add_rmsnorm_q(xb, xb, gamma, rstd=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        outs = []
        for _ in range(20):
            outs.append(glu.mlp_q_fwd(x, sx, *wg, *wu, *wd, stream=stream))
            torch.full((M * 1024,), 0x7F, dtype=torch.uint8, device="cuda")     # would land in a freed workspace
        got = glu.add_rmsnorm_q(xb, xb, gamma, rstd=True, stream=stream)
        q, s = glu.quantize(xb, stream=stream)
        side.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, norm))
        check_quantised(q, s, xb.double(), 1, 4 * U)


def test_results_wait_for_the_memory_they_take():
    """Given another stream, a call's results and workspace may come from memory
    that work still queued on the current stream uses: a late fill of a freed
    tensor of the same size must not land in them."""
    g = gen(19)
    M, H, I = 2048, 1024, 1024          # every result of 2 MB or more, so that a freed block is taken whole
    xb = randn(g, M, H).to(torch.bfloat16)
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    x, sx = glu.quantize(xb)
    wg, wu = (glu.quantize(randn(g, I, H) / H ** 0.5, block_rows=128) for _ in range(2))
    wd = glu.quantize(randn(g, H, I) / I ** 0.5, block_rows=128)
    experts = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    stacked = [t[None] for w in (wg, wu, wd) for t in w]
    calls = {
        "quantize rows": lambda **k: glu.quantize(xb, **k),
        "quantize blocks": lambda **k: glu.quantize(xb, block_rows=128, **k),
        "add_rmsnorm_q": lambda **k: glu.add_rmsnorm_q(xb, xb, gamma, rstd=True, **k),
        "gemm_q_nt": lambda **k: (glu.gemm_q_nt(x, sx, *wg, **k),),
        "gemm_q_fwd": lambda **k: glu.gemm_q_fwd(x, sx, *wg, *wu, **k),
        "mlp_q_fwd": lambda **k: (glu.mlp_q_fwd(x, sx, *wg, *wu, *wd, **k),),
        "mlp_q_fwd by expert": lambda **k: (glu.mlp_q_fwd(x, sx, *stacked, offsets=experts, **k),),
    }
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = [t.clone() for t in call()]
        sizes = [t.untyped_storage().nbytes() for t in want]
        sizes.append(glu.glu_mlp_q_workspace_bytes(M, I))
        for stream in (side, side.cuda_stream):
            torch.cuda.synchronize()
            torch.cuda.empty_cache()
            held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
            torch.cuda._sleep(100_000_000)          # some 50 ms
            for t in held:
                t.fill_(0x55)
            del held, t
            got = call(stream=stream)
            torch.cuda.synchronize()
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want)), name
            del got


def test_results_of_another_stream_are_kept_for_this_one():
    """A result made on another stream and read on the current one: once freed,
    its memory goes to no later call on that stream before the reading is done."""
    g = gen(23)
    xb = randn(g, 2048, 1024).to(torch.bfloat16)
    want, scale = glu.quantize(xb)
    zeros = torch.zeros_like(xb)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for stream in (side, side.cuda_stream):
        q, s = glu.quantize(xb, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(100_000_000)
        got, got_scale = q.view(torch.uint8).clone(), s.clone()
        del q, s
        for _ in range(3):
            glu.quantize(zeros, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want.view(torch.uint8)) and torch.equal(got_scale, scale)


def test_stream_argument_is_the_default_stream():
    """Handle 0, the default stream, from inside another one."""
    g = gen(29)
    xb = randn(g, 64, 512).to(torch.bfloat16)
    want = glu.quantize(xb)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for stream in (0, torch.cuda.default_stream()):
            q, s = glu.quantize(xb, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s, want[1])
    # and errors leave the current stream as it was
    here = torch.cuda.current_stream()
    with pytest.raises(ValueError):
        glu.quantize(xb, block_rows=3, stream=torch.cuda.Stream())
    assert torch.cuda.current_stream() == here


def test_stream_argument_in_a_graph():
    """Two calls on a stream that joins a capture, replayed on other inputs."""
    g = gen(37)
    M, H, I = 300, 512, 700
    wg, wu = (glu.quantize(randn(g, I, H) / H ** 0.5, block_rows=128) for _ in range(2))
    wd = glu.quantize(randn(g, H, I) / I ** 0.5, block_rows=128)
    xb = randn(g, M, H).to(torch.bfloat16)

    def run(stream=None):
        q, s = glu.quantize(xb, stream=stream)
        return [glu.mlp_q_fwd(q, s, *wg, *wu, *wd, stream=stream) for _ in range(2)]

    run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        side.wait_stream(torch.cuda.current_stream())
        outs = run(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        xb.copy_(randn(g, M, H))
        gr.replay()
        assert all(torch.equal(o, w) for o, w in zip(outs, run()))


def test_two_calls_at_once():
    """Products on two streams at the same time do not disturb each other."""
    g = gen(31)
    cases = []
    for M in (8, 500):
        a, sa = grid(g, M, 4096, 1)
        w, sw = grid(g, 1024, 4096, 128)
        cases.append((a, sa, w, sw, glu.gemm_q_nt(a, sa, w, sw)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for k, (st, c) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(st):
                got[k].append(glu.gemm_q_nt(*c[:4]))
    torch.cuda.synchronize()
    assert all(torch.equal(d, c[4]) for k, c in enumerate(cases) for d in got[k])


@pytest.mark.parametrize("bits", [8, 16])
def test_a_long_product_counts_no_timeout(bits):
    """A product that takes more than the second a wait may last (no single wait
    does): the right result, and no timeout is counted."""
    n, K = (131072, 163840) if bits == 8 else (98304, 131072)
    need = 2 * n * K * bits // 8 + 2 * n * n
    if torch.cuda.mem_get_info()[0] < need + (4 << 30):
        pytest.skip(f"needs {need >> 30} GB")
    before = glu.glu_wait_timeouts()
    if bits == 8:
        a, b = (torch.full((n, K), v, dtype=torch.uint8, device="cuda").view(FP8) for v in (0x38, 0x40))   # 1 and 2
        d = glu.gemm_q_nt(a, torch.full((n, K // 128), 2.0 ** -10, device="cuda"), b,
                          torch.full((n // 128, K // 128), 2.0 ** -8, device="cuda"))
        want = 2 * K * 2.0 ** -18
    else:
        a, b = (torch.full((n, K), v, dtype=torch.bfloat16, device="cuda") for v in (1.0, 2.0 ** -18))
        d = glu.gemm_nt(a, b)
        want = K * 2.0 ** -18
    torch.cuda.synchronize()
    assert glu.glu_wait_timeouts() == before
    assert float(d.min()) == float(d.max()) == want
    del a, b, d
    torch.cuda.empty_cache()


def test_modules():
    from glu_activation_mlps_gb300.autograd import FusedAddRMSNorm, GatedMLP, QuantGatedMLP
    torch.manual_seed(0)
    mlps = [GatedMLP(320, 500, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    norm = FusedAddRMSNorm(320, device="cuda", dtype=torch.bfloat16)
    x, res = (torch.randn(40, 320, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    h, q, s = norm.quantized(x, res)
    one = QuantGatedMLP.from_mlp(mlps[0])
    out = one(q, s)
    h2, y = norm(x, res)
    assert torch.equal(h, h2) and out.dtype == torch.bfloat16
    gate, up = (w.detach().double() for w in mlps[0]._gate_up_weights())
    y = y.double()
    ref = (ACT64["silu"](y @ gate.T) * (y @ up.T)) @ mlps[0].down_proj.weight.detach().double().T
    # three roundings to e4m3 (x, y, weights), each at most 2^-4 of a value and
    # about a third of that in the mean: far below this
    assert float(((out.double() - ref).norm() / ref.norm()).detach()) < 0.12
    many = QuantGatedMLP.from_mlps(mlps)
    off = cuts([10, 0, 30])
    got = many(q, s, off)
    # expert by expert: the same kernel gives the same bits; a module of one
    # expert may split its sums over K, which moves a y that lies next to a
    # border by one step, 2^-3 of it, so few of the products' terms
    assert torch.equal(got[:10], many(q[:10], s[:10], cuts([10, 0, 0])))
    assert torch.equal(got[10:], many(q[10:], s[10:], cuts([0, 0, 30])))
    for part, mlp, rows in ((got[:10], mlps[0], slice(0, 10)), (got[10:], mlps[2], slice(10, 40))):
        alone = QuantGatedMLP.from_mlp(mlp)(q[rows], s[rows]).double()
        assert float((part.double() - alone).norm() / alone.norm()) < 2.0 ** -5
    assert set(one.state_dict()) == {f"{n}_{k}" for n in ("gate", "up", "down") for k in ("weight", "scale")}


def test_module_from_f32_weights():
    """Weights of torch's default type: results come in bf16, or in the type asked for."""
    from glu_activation_mlps_gb300.autograd import GatedMLP, QuantGatedMLP
    torch.manual_seed(1)
    mlp = GatedMLP(256, 300, device="cuda")
    x = torch.randn(9, 256, device="cuda")
    for module, dt in ((QuantGatedMLP.from_mlp(mlp), torch.bfloat16),
                       (QuantGatedMLP.from_mlps([mlp, mlp]), torch.bfloat16),
                       (QuantGatedMLP.from_mlp(mlp, dtype=torch.float16), torch.float16)):
        off = None if module.gate_weight.dim() == 2 else cuts([4, 5])
        out = module(x, offsets=off)
        q, s = glu.quantize(x)
        names = ("gate", "up", "down")
        want = glu.mlp_q_fwd(q, s, *(getattr(module, f"{n}_{k}") for n in names for k in ("weight", "scale")),
                             dtype=dt, offsets=off)
        assert out.dtype == dt and torch.equal(out, want)
    with pytest.raises(ValueError):
        QuantGatedMLP.from_mlp(mlp, dtype=torch.float32)


def test_module_is_moved_and_cast():
    """Casting the module leaves the 8-bit weights and their scales as they are
    and sets the type of its results; moving it keeps rows on 16-byte boundaries
    at sizes that are no multiple of 16."""
    import copy
    from glu_activation_mlps_gb300.autograd import GatedMLP, QuantGatedMLP
    torch.manual_seed(2)
    mlps = [GatedMLP(250, 301, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    x = torch.randn(9, 250, device="cuda", dtype=torch.bfloat16)
    for module, off in ((QuantGatedMLP.from_mlp(mlps[0]), None), (QuantGatedMLP.from_mlps(mlps), cuts([4, 5]))):
        held = {k: v.clone() for k, v in module.state_dict().items()}
        want = {dt: copy.deepcopy(module) for dt in (torch.bfloat16, torch.float16)}
        for dt, m in want.items():
            m.dtype = dt
        want = {dt: m(x, offsets=off) for dt, m in want.items()}
        steps = [(lambda m: m.half(), torch.float16), (lambda m: m.to(torch.bfloat16), torch.bfloat16),
                 (lambda m: m.float(), torch.bfloat16), (lambda m: m.double(), torch.bfloat16),
                 (lambda m: m.cpu().cuda(), torch.bfloat16), (lambda m: m.to("cpu").to("cuda", torch.float16), torch.float16),
                 (copy.deepcopy, torch.float16)]
        for step, dt in steps:
            module = step(module)
            for k, v in module.state_dict().items():
                assert v.dtype == held[k].dtype and torch.equal(v.view(torch.uint8), held[k].view(torch.uint8)), k
            out = module(x, offsets=off)
            assert out.dtype == dt and torch.equal(out, want[dt])
        # inside another module, as a model casts its parts
        model = torch.nn.Sequential(module).to(torch.bfloat16)
        assert torch.equal(model[0](x, offsets=off), want[torch.bfloat16])
        # another module's weights
        other = QuantGatedMLP.from_mlp(mlps[1]) if off is None else QuantGatedMLP.from_mlps(mlps[::-1])
        other.load_state_dict(module.state_dict())
        assert torch.equal(other(x, offsets=off), want[torch.bfloat16])
        with pytest.raises(TypeError):
            module.type(torch.float16)


def test_refusals():
    x = torch.zeros(4, 256, device="cuda", dtype=torch.bfloat16)
    q, s = glu.quantize(x)
    w, sw = glu.quantize(torch.zeros(256, 256, device="cuda"), block_rows=128)
    with pytest.raises(ValueError):
        glu.quantize(x, q=torch.empty(4, 255, dtype=FP8, device="cuda"))
    with pytest.raises(ValueError):
        glu.quantize(x, scale=torch.empty(4, 3, device="cuda"))
    with pytest.raises(ValueError):
        glu.gemm_q_nt(q, s[:, :1], w, sw)
    with pytest.raises(ValueError):
        glu.gemm_q_nt(q, s, w, sw[:1])
    with pytest.raises(ValueError):
        glu.gemm_q_nt(q, s, w[:, :128], sw)
    with pytest.raises(TypeError):
        glu.gemm_q_nt(x, s, w, sw)
    with pytest.raises(ValueError):
        glu.gemm_q_nt(q.cpu(), s, w, sw)
    with pytest.raises(ValueError):
        glu.gemm_q_nt(q, s, w, sw.cpu())
    with pytest.raises(ValueError):     # 64-bit offsets, and the wrong number of them
        glu.gemm_q_nt(q, s, w[None], sw[None], offsets=torch.tensor([0, 4], device="cuda"))
    with pytest.raises(ValueError):
        glu.gemm_q_nt(q, s, w[None], sw[None], offsets=torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda"))
    with pytest.raises(glu.GluError) as e:      # f32 results
        glu.gemm_q_nt(q, s, w, sw, dtype=torch.float32)
    assert e.value.status == -5
    with pytest.raises(glu.GluError) as e:      # rows that do not start on 16-byte boundaries
        odd = torch.zeros(4, 264, dtype=FP8, device="cuda")[:, :256]
        glu.gemm_q_nt(odd, s, w, sw)
    assert e.value.status == -3
    with pytest.raises(glu.GluError) as e:      # d over b
        glu.gemm_q_nt(q, s, w, sw, d=torch.as_strided(w.view(torch.bfloat16), (4, 256), (256, 1)))
    assert e.value.status == -4
    pinned = torch.zeros(4, 256, dtype=torch.bfloat16).pin_memory()
    st = glu.glu_gemm_q_nt(q.data_ptr(), 256, s.data_ptr(), 2, w.data_ptr(), 256, sw.data_ptr(), 2,
                           pinned.data_ptr(), 256, 4, 256, 256, 2, None)
    assert st == -8                             # an output that is not in device memory
    assert glu.glu_last_launch()["path"] != 0
