"""Argument rules of the 8-bit calls on the CPU: every refusal happens on the
host, before any CUDA call, so fake device addresses are enough (they are passed
only where no GPU is present)."""
import pytest
import torch

import glu_activation_mlps_gb300 as glu

OK, NULL, SHAPE, STRIDE, ALIAS, ENUM, CUDA, WORKSPACE, VALUE = 0, -1, -2, -3, -4, -5, -6, -7, -8
F32, F16, BF16 = 0, 1, 2
BASE = 1 << 32
MB = 1 << 20

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake device addresses")


@pytest.fixture(scope="module", autouse=True)
def built():
    glu.build()
    glu.lib()


def quantize(x=BASE, sx=256, q=BASE + MB, sq=256, s=BASE + 2 * MB, ss=2, rows=4, cols=256, block=1, dtype=BF16):
    return glu.glu_quantize(x, sx, q, sq, s, ss, rows, cols, block, dtype, None)


def test_quantize():
    assert quantize(dtype=3) == ENUM and quantize(block=2) == VALUE and quantize(block=0) == VALUE
    assert quantize(rows=-1) == SHAPE and quantize(cols=-1) == SHAPE and quantize(cols=1 << 31) == SHAPE
    assert quantize(rows=1 << 60, sx=1 << 20) == SHAPE
    assert quantize(x=None) == NULL and quantize(q=None) == NULL and quantize(s=None) == NULL
    assert quantize(sx=255) == STRIDE and quantize(sq=255) == STRIDE and quantize(ss=1) == STRIDE
    assert quantize(s=BASE + 2 * MB + 2) == STRIDE
    # any overlap of an output with another operand
    assert quantize(q=BASE) == ALIAS and quantize(s=BASE + 4 * 512 - 4) == ALIAS and quantize(s=BASE + MB + 8) == ALIAS
    assert quantize(x=None, q=None, s=None, rows=0) == OK and quantize(cols=0) == OK
    assert glu.glu_last_launch()["launched"] == 0
    # a single row's and a single block row's strides do not count
    assert quantize(rows=1, sx=0, sq=0, ss=0) == CUDA
    assert quantize(rows=100, block=128, ss=0) == CUDA
    assert quantize() == CUDA and quantize(block=128, dtype=F32, sx=300) == CUDA


def test_quantize_the_widest_rows():
    """Up to 2^28 columns, whatever the accesses: whole pieces of 32 and 16
    bytes, single elements for odd widths and bases."""
    far = {"q": BASE + (1 << 31), "s": BASE + (1 << 32)}
    for cols in ((1 << 28) - 1, 1 << 28, (1 << 27) - 1, (1 << 27) + 8, 134215681):
        for dtype in (F32, F16, BF16):
            for block in (1, 128):
                assert quantize(rows=1, cols=cols, dtype=dtype, block=block, **far) == CUDA, (cols, dtype, block)
                assert quantize(x=BASE + 4, rows=1, cols=cols, dtype=dtype, block=block, **far) == CUDA
    assert quantize(rows=1, cols=(1 << 28) + 1, **far) == SHAPE


def norm(x=BASE, sx=256, r=BASE + MB, sr=256, g=BASE + 2 * MB, h=BASE + 3 * MB, sh=256, q=BASE + 4 * MB, sq=256,
         s=BASE + 5 * MB, ss=2, rstd=BASE + 6 * MB, rows=4, cols=256, eps=1e-5, dtype=BF16):
    return glu.glu_add_rmsnorm_q(x, sx, r, sr, g, h, sh, q, sq, s, ss, rstd, rows, cols, eps, dtype, None)


def test_add_rmsnorm_q():
    assert norm(dtype=7) == ENUM
    assert norm(eps=0.0) == VALUE and norm(eps=float("nan")) == VALUE and norm(eps=float("inf")) == VALUE
    assert norm(rows=-1) == SHAPE and norm(cols=32769, sx=40000, sr=40000, sh=40000, sq=40000, ss=300) == SHAPE
    for k in ("x", "r", "g", "h", "q", "s"):
        assert norm(**{k: None}) == NULL, k
    for k in ("sx", "sr", "sh", "sq"):
        assert norm(**{k: 255}) == STRIDE, k
    assert norm(ss=1) == STRIDE and norm(s=BASE + 5 * MB + 1) == STRIDE and norm(rstd=BASE + 6 * MB + 2) == STRIDE
    assert norm(h=BASE + 2) == ALIAS and norm(h=BASE + 2 * MB) == ALIAS
    for other in (BASE, BASE + MB, BASE + 2 * MB, BASE + 3 * MB, BASE + 6 * MB):
        assert norm(q=other) == ALIAS and norm(s=other) == ALIAS
    assert norm(q=BASE + 5 * MB) == ALIAS and norm(rstd=BASE) == ALIAS
    assert norm(rows=0, x=None, q=None) == OK
    # in place over x or the residual; no rstd
    assert norm(h=BASE) == CUDA and norm(h=BASE + MB) == CUDA and norm(rstd=None) == CUDA and norm() == CUDA


def test_operands_off_their_elements_boundary():
    """An access of an element that is not at a multiple of its size would fault."""
    for off in (1, 3):
        assert quantize(x=BASE + off) == STRIDE and quantize(x=BASE + off, block=128, dtype=F16) == STRIDE
        for k, at in (("x", BASE), ("r", BASE + MB), ("g", BASE + 2 * MB), ("h", BASE + 3 * MB)):
            assert norm(**{k: at + off}) == STRIDE, k
            assert norm(**{k: at + off}, dtype=F32, sx=300, sr=300, sh=300) == STRIDE, k
    assert quantize(x=BASE + 2, dtype=F32) == STRIDE and norm(g=BASE + 2 * MB + 2, dtype=F32) == STRIDE
    # on their boundary, and q anywhere
    assert quantize(x=BASE + 2, q=BASE + MB + 1) == CUDA and quantize(x=BASE + 4, dtype=F32) == CUDA
    assert norm(x=BASE + 2, r=BASE + MB + 6, g=BASE + 2 * MB + 2, h=BASE + 3 * MB + 2, q=BASE + 4 * MB + 3) == CUDA


def nt(a=BASE, sa=256, s=BASE + MB, ss=2, b=BASE + 2 * MB, sb=256, t=BASE + 3 * MB, st=2, d=BASE + 4 * MB, sd=384,
       M=8, K=256, N=384, dtype=BF16):
    return glu.glu_gemm_q_nt(a, sa, s, ss, b, sb, t, st, d, sd, M, K, N, dtype, None)


def test_gemm_q_nt():
    assert nt(dtype=F32) == ENUM and nt(dtype=5) == ENUM
    assert nt(M=-1) == SHAPE and nt(K=-1) == SHAPE and nt(N=-1) == SHAPE and nt(M=1 << 31) == SHAPE
    assert nt(K=(1 << 31) - 10, sa=1 << 31, sb=1 << 31, ss=1 << 24, st=1 << 24) == SHAPE
    for k in ("a", "s", "b", "t", "d"):
        assert nt(**{k: None}) == NULL, k
    assert nt(sa=255) == STRIDE and nt(sb=240) == STRIDE and nt(sd=383) == STRIDE
    assert nt(ss=1) == STRIDE and nt(st=1) == STRIDE
    # the copy engine's rules: 16-byte bases and strides; scales and d by element
    assert nt(a=BASE + 8) == STRIDE and nt(b=BASE + 2 * MB + 1) == STRIDE and nt(sa=264) == STRIDE and nt(sb=257) == STRIDE
    assert nt(s=BASE + MB + 2) == STRIDE and nt(t=BASE + 3 * MB + 3) == STRIDE and nt(d=BASE + 4 * MB + 1) == STRIDE
    for other in (BASE, BASE + MB, BASE + 2 * MB, BASE + 3 * MB):
        assert nt(d=other) == ALIAS
    assert nt(M=0, a=None, d=None) == OK and nt(N=0, b=None) == OK
    assert glu.glu_last_launch()["launched"] == 0
    # valid calls end at the missing device: an odd K with padded rows, one row,
    # one column block (whose scale stride separates nothing), K = 0
    assert nt(K=241) == CUDA and nt(M=1, sa=0, ss=0, sd=0) == CUDA and nt(N=100, sd=100, st=0) == CUDA
    assert nt(K=0, a=None, s=None, b=None, t=None) == CUDA and nt() == CUDA


def fwd(x=BASE, sx=256, s=BASE + MB, ss=2, g=BASE + 2 * MB, u=BASE + 3 * MB, sw=256, gs=BASE + 4 * MB,
        us=BASE + 5 * MB, sws=2, y=BASE + 6 * MB, sy=384, ys=BASE + 7 * MB, sys_=3, M=8, K=256, I=384, act=0):
    return glu.glu_gemm_q_fwd(x, sx, s, ss, g, u, sw, gs, us, sws, y, sy, ys, sys_, M, K, I, act, None)


def test_gemm_q_fwd():
    assert fwd(act=4) == ENUM and fwd(act=-1) == ENUM
    for k in ("x", "s", "g", "u", "gs", "us", "y", "ys"):
        assert fwd(**{k: None}) == NULL, k
    assert fwd(sy=383) == STRIDE and fwd(sys_=2) == STRIDE and fwd(sws=1) == STRIDE and fwd(u=BASE + 3 * MB + 4) == STRIDE
    assert fwd(ys=BASE + 7 * MB + 2) == STRIDE
    for other in (BASE, BASE + MB, BASE + 2 * MB, BASE + 3 * MB, BASE + 4 * MB, BASE + 5 * MB):
        assert fwd(y=other) == ALIAS and fwd(ys=other) == ALIAS
    assert fwd(ys=BASE + 6 * MB) == ALIAS
    assert fwd(M=0) == OK and fwd(I=0) == OK
    assert fwd(y=BASE + 6 * MB + 1, sy=385) == CUDA and fwd(K=0) == CUDA and fwd() == CUDA


def grouped(offsets=BASE + 8 * MB, n=3, wg=384 * 256, wsg=6, M=8, K=256, N=384, d=BASE + 16 * MB):
    return glu.glu_gemm_q_grouped_nt(BASE, 256, BASE + MB, 2, BASE + 2 * MB, 256, wg, BASE + 12 * MB, 2, wsg, d, 384,
                                     M, K, N, offsets, n, BF16, None)


def test_grouped():
    assert grouped(n=-1) == SHAPE and grouped(n=1025) == SHAPE
    assert grouped(offsets=None) == NULL and grouped(offsets=BASE + 8 * MB + 2) == STRIDE
    # experts' weights may not overlap; their distance is a multiple of 16 bytes
    assert grouped(wg=384 * 256 - 16) == STRIDE and grouped(wsg=5) == STRIDE and grouped(wg=384 * 256 + 8) == STRIDE
    # the footprint of d against every expert's weights, and against the offsets
    assert grouped(d=BASE + 2 * MB + 2 * 384 * 256) == ALIAS and grouped(d=BASE + 8 * MB) == ALIAS
    assert grouped(n=0) == OK and grouped(n=0, offsets=None) == OK and grouped(M=0) == OK
    assert grouped(n=1, wg=0, wsg=0) == CUDA and grouped() == CUDA


def test_grouped_extents_overflow():
    """Experts so far apart that their bytes wrap around 64 bits."""
    for wsg in (1 << 62, (1 << 62) + 6, 1 << 61, (1 << 63) - 1):
        assert grouped(wsg=wsg) == SHAPE, wsg
    assert grouped(wg=(1 << 63) - 16) == STRIDE and grouped(wg=1 << 40) == STRIDE


def mlp(x=BASE, out=BASE + 32 * MB, so=256, M=8, H=256, I=384, ws=BASE + 64 * MB, wb=None, offsets=None, n=0, act=0,
        dtype=BF16, wd=BASE + 8 * MB):
    wb = glu.glu_mlp_q_workspace_bytes(M, I) if wb is None else wb
    return glu.glu_mlp_q_fwd(x, 256, BASE + MB, 2, BASE + 2 * MB, BASE + 4 * MB, 256, 384 * 256, BASE + 6 * MB,
                             BASE + 7 * MB, 2, 6, wd, 384, 256 * 384, BASE + 12 * MB, 3, 6, out, so, M, H, I, offsets,
                             n, act, dtype, ws, wb, None)


def test_mlp():
    assert glu.glu_mlp_q_workspace_bytes(8, 384) == 8 * (384 + 12)
    assert glu.glu_mlp_q_workspace_bytes(3, 130) == 3 * (144 + 8)
    assert glu.glu_mlp_q_workspace_bytes(0, 5) == 0 and glu.glu_mlp_q_workspace_bytes(5, -1) == 0
    assert mlp(act=9) == ENUM and mlp(dtype=F32) == ENUM and mlp(M=-2) == SHAPE
    assert mlp(ws=None) == WORKSPACE and mlp(wb=8 * 396 - 1) == WORKSPACE and mlp(ws=BASE + 64 * MB + 8) == STRIDE
    assert mlp(out=BASE) == ALIAS and mlp(out=BASE + MB) == ALIAS and mlp(out=BASE + 8 * MB) == ALIAS
    assert mlp(out=BASE + 64 * MB) == ALIAS and mlp(ws=BASE + 2 * MB) == ALIAS and mlp(ws=BASE) == ALIAS
    assert mlp(out=None) == NULL and mlp(wd=None) == NULL and mlp(so=255) == STRIDE
    assert mlp(M=0) == OK and mlp(H=0) == OK
    assert mlp(offsets=BASE + 63 * MB, n=2000) == SHAPE
    assert mlp(I=0) == CUDA and mlp() == CUDA and mlp(offsets=BASE + 63 * MB, n=2) == CUDA


def test_mlp_without_experts():
    """Offsets and no expert: no work, as in the grouped products, not the dense MLP."""
    off = BASE + 63 * MB
    assert mlp(offsets=off, n=0) == OK and glu.glu_last_launch()["launched"] == 0
    assert mlp(offsets=off, n=0, I=0) == OK
    # there are no weights to point to, nor rows for a workspace to hold
    assert mlp(offsets=off, n=0, wd=None, ws=None, out=None, x=None) == OK
    assert mlp(offsets=off, n=-1) == SHAPE and mlp(offsets=off, n=0, act=9) == ENUM
    assert mlp(offsets=off, n=0, M=-1) == SHAPE
    assert mlp(n=0) == CUDA             # without offsets it is the dense one


def test_mlp_overlaps():
    """out and the workspace (the gaps between its rows too) overlap no operand of
    either product, dense or in any expert's part."""
    off = BASE + 63 * MB
    # x, its scales, gate and up weights and scales, down weights and scales: first and last bytes
    ends = {BASE: 8 * 256, BASE + MB: 8 * 8, BASE + 2 * MB: 384 * 256, BASE + 4 * MB: 384 * 256, BASE + 6 * MB: 24,
            BASE + 7 * MB: 24, BASE + 8 * MB: 256 * 384, BASE + 12 * MB: 24}
    for at, size in ends.items():
        for last in (0, size - 16 & ~15):
            assert mlp(out=at + last) == ALIAS, (at - BASE, last)
            assert mlp(ws=at + last) == ALIAS, (at - BASE, last)
            assert mlp(out=at + last, offsets=off, n=1) == ALIAS and mlp(ws=at + last, offsets=off, n=1) == ALIAS
        # just behind it
        assert mlp(out=at + (size + 15 & ~15)) == CUDA and mlp(ws=at + (size + 15 & ~15)) == CUDA
    for at, group in ((2 * MB, 384 * 256), (4 * MB, 384 * 256), (6 * MB, 24), (7 * MB, 24), (8 * MB, 256 * 384),
                      (12 * MB, 24)):
        third = BASE + at + 2 * group
        assert mlp(out=third, offsets=off, n=3) == ALIAS and mlp(ws=third, offsets=off, n=3) == ALIAS
        assert mlp(out=BASE + at + (3 * group + 15 & ~15), offsets=off, n=3) == CUDA
    assert mlp(out=off, offsets=off, n=3) == ALIAS and mlp(ws=off, offsets=off, n=3) == ALIAS
    # the workspace: 8 rows of 384 + 12 bytes
    assert mlp(out=BASE + 64 * MB + 8 * 396 - 2) == ALIAS and mlp(out=BASE + 64 * MB + 8 * 396) == CUDA
    # no columns between the products: the weights are not read
    assert mlp(I=0, out=BASE + 8 * MB) == CUDA and mlp(I=0, out=BASE + 2 * MB, offsets=off, n=3) == CUDA


def test_python_layer_refuses():
    x = torch.zeros(4, 256)
    q, s = torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.zeros(4, 2)
    with pytest.raises(ValueError):     # not on a CUDA device
        glu.quantize(x)
    with pytest.raises(ValueError):
        glu.quantize(x, block_rows=64)
    with pytest.raises(TypeError):
        glu.quantize(x.double())
    with pytest.raises(ValueError):
        glu.add_rmsnorm_q(x, x, x[0])
    with pytest.raises(ValueError):
        glu.gemm_q_nt(q, s, q, s)


def test_experts_of_one_activation():
    """A module of experts has one activation: MLPs of different ones are refused."""
    from glu_activation_mlps_gb300.autograd import GatedMLP, QuantGatedMLP
    mlps = [GatedMLP(16, 32, act=act) for act in ("silu", "relu", "silu")]
    with pytest.raises(ValueError, match="one activation"):
        QuantGatedMLP.from_mlps(mlps)
    with pytest.raises(ValueError, match="CUDA"):       # past that check, at weights that are not on a device
        QuantGatedMLP.from_mlps([mlps[0], mlps[2]])
