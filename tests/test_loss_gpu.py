"""The losses over a vocabulary (linear_ce, linear_distill and their gradients)
against the formulas in 64 bits.

Bounds, with u the largest relative rounding of the type (bf16 2^-8, f16 2^-11)
and A = |x| |w|^T:
  * a logit, summed in fp32 over H products, is off by dz <= H 2^-23 A (0 on
    grids whose sums are exact in fp32);
  * log sum exp moves by at most max dz (with dz / T); forming it: 300 terms are
    added one after the other at most (2^-24 each), exp2 and its argument are off
    by less than 2^-20 relative, and the result's own rounding is a few 2^-24 of
    its size;
  * an entry g = c (p - t) with |c p| (2 max dz + 2^-19) from the exponential, the
    rounding u |g|, and half a step of the type's smallest value: 2^-134, in f16
    under the scale, 2^-25 max |c| / 2^13;
  * dx = g w: what g is off by times |w|, V 2^-23 |g| |w| of the fp32 sums, one
    rounding u; dw alike.
"""
import math

import pytest
import torch

import glu_activation_mlps_gb300 as glu

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SIZES = [(1, 1, 1), (1, 8, 1), (3, 9, 2), (1, 64, 1000), (7, 40, 130), (128, 64, 256), (129, 100, 257), (300, 72, 1000),
         (64, 512, 5000), (257, 1030, 3001), (1000, 130, 129), (5, 2048, 20000), (520, 256, 40), (2000, 192, 700),
         # K of dx and dw in parts of uneven numbers of slices
         (128, 256, 4160), (129, 520, 8200), (4160, 64, 300), (600, 1100, 9000),
         # x transposed before dw
         (2048, 136, 32768)]


def matrix(rows, cols, dtype, g, scale=1.0, pad=True, grid=False):
    if grid:
        v = torch.randint(-8, 9, (rows, cols), generator=g, device="cuda") / 8
    else:
        v = torch.randn(rows, cols, generator=g, device="cuda") * scale
    wide = torch.zeros(rows, cols + (-cols % 8 if pad else 0), dtype=dtype, device="cuda")
    wide[:, :cols] = v
    return wide[:, :cols]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def shares_of(index, logit, V, T):
    """(valid rows, dense (N, V) shares, sum of p log p) in 64 bits."""
    N = index.shape[0]
    has = (index >= 0) & (index < V) & (logit != -math.inf)
    valid = has.any(1)
    t = logit.double()
    top = torch.where(has, t, -math.inf).amax(1)
    d = torch.where(has, (t - torch.where(valid, top, 0.0)[:, None]) / T, -math.inf)
    p = torch.softmax(torch.where(valid[:, None], d, 0.0), 1) * valid[:, None]
    dense = torch.zeros(N, V, dtype=torch.float64, device=index.device)
    r, k = has.nonzero(as_tuple=True)
    dense.index_put_((r, index[r, k]), p[r, k], accumulate=True)
    return has, valid, dense, -torch.special.entr(p).sum(1)


def reference(x, w, shares, valid, ent, T, dloss=None, exact=False):
    x64 = torch.where(valid[:, None], x.double(), 0.0)
    w64 = w.double()
    H, V = w.shape[1], w.shape[0]
    s = x64 @ w64.T / T
    lse = torch.logsumexp(s, 1) * valid
    log_q = s - lse[:, None]
    loss = (ent - (shares * log_q).sum(1)) * valid
    A = x64.abs() @ w64.abs().T
    dz = (0.0 if exact else 1.0) * H * 2.0 ** -23 * A / T
    off = dz.amax(1)
    tol = 2 * off + 300 * 2.0 ** -24 + 2.0 ** -20 + 8 * 2.0 ** -24 * (lse.abs() + ent.abs() + s.abs().amax(1))
    out = {"loss": loss, "lse": lse, "tol": tol, "z": s * T, "z_tol": dz * T + 2.0 ** -23 * (s * T).abs()}
    if dloss is not None:
        c = torch.where(valid, dloss.double(), 0.0) / T
        p = torch.exp(log_q)
        g = c[:, None] * (p - shares) * valid[:, None]
        u = U[x.dtype]
        # at a named token the exponential or, for the cross entropy, expm1 of the loss
        eg = c.abs()[:, None] * p * (2 * off[:, None] + tol[:, None] + 2.0 ** -19)
        eg = eg + c.abs()[:, None] * shares * (tol[:, None] + 2.0 ** -20)
        eg = eg + u * (g.abs() + eg)
        eg = eg + 2.0 ** -134 * valid[:, None]        # bf16's own smallest step
        if x.dtype == torch.float16:
            eg = eg + (2.0 ** -25 * c.abs().max() / 2.0 ** 13) * valid[:, None]
        ga = g.abs() + eg
        for name, val, err in (("dx", g @ w64, eg @ w64.abs() + V * 2.0 ** -23 * (ga @ w64.abs())),
                               ("dw", g.T @ x64, eg.T @ x64.abs() + len(x) * 2.0 ** -23 * (ga.T @ x64.abs()))):
            tiny = 2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -134
            out[name] = val
            out[name + "_tol"] = err + u * (val.abs() + err) + tiny
    return out


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} for {want[bad][0].item()}, allowed {tol.expand_as(want)[bad][0].item()}")


def targets(N, V, g, masked):
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    if masked == "some":
        t[torch.rand(N, generator=g, device="cuda") < 0.5] = -100
        t[N // 2] = V           # just behind the vocabulary
        t[0] = -1
    elif masked == "all":
        t[:] = -100
    elif masked == "last":
        t[:] = -1
        t[-1] = V - 1
    return t


def check_ce(x, w, target, dloss, exact=False, **kw):
    V = w.shape[0]
    valid = (target >= 0) & (target < V)
    shares = torch.zeros(len(x), V, dtype=torch.float64, device="cuda")
    shares[valid.nonzero()[:, 0], target[valid]] = 1.0
    ref = reference(x, w, shares, valid, torch.zeros(len(x), device="cuda").double(), 1.0, dloss, exact)
    loss, lse = glu.linear_ce(x, w, target)
    close(loss, ref["loss"], ref["tol"], "loss")
    close(lse, ref["lse"], ref["tol"], "lse")
    dx, dw = glu.linear_ce_bwd(dloss, x, w, target, loss, lse, **kw)
    close(dx, ref["dx"], ref["dx_tol"], "dx")
    close(dw, ref["dw"], ref["dw_tol"], "dw")
    assert glu.glu_wait_timeouts() == 0
    return loss, lse, dx, dw


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,H,V", SIZES)
def test_ce(N, H, V, dtype):
    g = gen(N * 7 + H * 3 + V)
    x, w = matrix(N, H, dtype, g), matrix(V, H, dtype, g, 2.0 / math.sqrt(H))
    t = targets(N, V, g, "none")
    check_ce(x, w, t, torch.randn(N, generator=g, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,H,V", [(1, 64, 300), (100, 64, 1000), (300, 72, 1000), (700, 136, 515), (2000, 64, 200),
                                   (2500, 72, 33000), (70000, 64, 300)])
@pytest.mark.parametrize("masked", ["some", "all", "last"])
def test_ce_rows_without_target(N, H, V, masked, dtype):
    g = gen(N + V)
    x, w = matrix(N, H, dtype, g), matrix(V, H, dtype, g, 0.3)
    t = targets(N, V, g, masked)
    dloss = torch.randn(N, generator=g, device="cuda")
    none = (t < 0) | (t >= V)
    x[none] = math.nan          # what such rows hold is not used
    dloss[none] = math.nan
    loss, lse, dx, _ = check_ce(x, w, t, dloss)
    for v in (loss, lse, dx):
        assert torch.all(v[none] == 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,H,V", [(33, 64, 777), (200, 200, 1500), (400, 1024, 300)])
def test_ce_on_exact_sums(N, H, V, dtype):
    g = gen(5)
    x, w = matrix(N, H, dtype, g, grid=True), matrix(V, H, dtype, g, grid=True)
    check_ce(x, w, targets(N, V, g, "some"), torch.randint(1, 5, (N,), generator=g, device="cuda").float(), exact=True)


@pytest.mark.parametrize("N,steps", [(64, 16), (300, 64)])
def test_logits_are_summed_in_segments(N, steps):
    """The logits of 4096 products: `steps` steps of 16 products in one accumulator, each of
    which may drop two units of 2^-23 of what is in it, and one rounded addition a segment."""
    H, V, K = 4096, 1000, 16
    g = gen(N)
    x, w = matrix(N, H, torch.bfloat16, g), matrix(V, H, torch.bfloat16, g, 0.1)
    index = torch.randint(0, V, (N, K), generator=g, device="cuda")
    _, _, top = glu.linear_distill(x, w, index, torch.zeros(N, K, device="cuda"))
    z, A = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
    segments = H // (16 * steps)
    close(top, z.gather(1, index), ((2 * steps + segments) * 2.0 ** -23 * A).gather(1, index), "top_logits")


def test_ce_confident_rows():
    """Where the target has nearly all the probability the loss and the target's
    gradient are small differences: to 2^-10 relative of what 64 bits give, on exact sums."""
    N, H, V = 64, 128, 2000
    g = gen(9)
    w = matrix(V, H, torch.float16, g, grid=True)
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    x = (w[t].float() * (torch.arange(N, device="cuda")[:, None] % 4 + 1) / 4).half()
    x = torch.round(x.float() * 8).div(8).half()
    loss, lse = glu.linear_ce(x, w, t)
    s = x.double() @ w.double().T
    s_t = s.gather(1, t[:, None])
    others = torch.exp(s - s_t).scatter_(1, t[:, None], 0.0).sum(1)
    want = torch.log1p(others)
    assert want.min() < 1e-3
    # the sum is 1 + others in fp32, off by 300 roundings of 2^-24 at most
    assert torch.all((loss.double() - want).abs() <= 300 * 2.0 ** -24 + 2.0 ** -20 * want)
    # g's entry at the target, -(1 - exp(-loss)) = expm1(-loss), seen alone: dw of a token that only it names
    dx, dw = glu.linear_ce_bwd(torch.ones(N, device="cuda"), x, w, t, loss, lse)
    p = torch.exp(s - torch.logsumexp(s, 1)[:, None])
    gg = p.scatter(1, t[:, None], torch.expm1(-loss.double())[:, None])
    err = (2.0 ** -11 + 2.0 ** -18) * gg.abs() + 2.0 ** -38
    for got, val, tol in ((dx, gg @ w.double(), err @ w.double().abs()), (dw, gg.T @ x.double(), err.T @ x.double().abs())):
        close(got, val, tol * 1.01 + 2.0 ** -11 * val.abs() + 2.0 ** -24 + V * 2.0 ** -23 * 1e-3, "gradient")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,H,V", [(50, 64, 3000), (300, 256, 5000), (600, 64, 1000), (1100, 200, 2500)])
@pytest.mark.parametrize("masked", ["none", "some"])
def test_ce_in_pieces(N, H, V, masked, dtype):
    """A small workspace: many pieces of the vocabulary, partial results added up."""
    g = gen(11)
    x, w = matrix(N, H, dtype, g), matrix(V, H, dtype, g, 0.2)
    t = targets(N, V, g, masked)
    dloss = torch.rand(N, generator=g, device="cuda")
    full = glu.glu_linear_ce_workspace_bytes(N, H, V, 1)
    for part in (0.9, 0.8, 0.7, 0.6, 0.4):
        ws = torch.full((int(full * part),), 255, dtype=torch.uint8, device="cuda")
        try:
            check_ce(x, w, t, dloss, workspace=ws)
        except glu.GluError as e:
            assert e.status == -7 and part < 0.7
    with pytest.raises(glu.GluError):
        loss, lse = glu.linear_ce(x, w, t)
        glu.linear_ce_bwd(dloss, x, w, t, loss, lse, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_ce_of_more_than_one_piece_by_default():
    """g of the whole vocabulary would take more than 1 GiB."""
    N, H, V = 8200, 64, 70000
    assert 2 * N * V > 1 << 30
    g = gen(13)
    x, w = matrix(N, H, torch.bfloat16, g), matrix(V, H, torch.bfloat16, g, 0.2)
    check_ce(x, w, targets(N, V, g, "none"), torch.rand(N, generator=g, device="cuda"))


def teacher(N, V, K, g, logit_dtype, kind):
    index = torch.randint(0, V, (N, K), generator=g, device="cuda")        # tokens may occur twice
    logit = (torch.randn(N, K, generator=g, device="cuda") * 3).to(logit_dtype)
    if kind == "ragged":
        index[torch.rand(N, K, generator=g, device="cuda") < 0.4] = -1
        logit[torch.rand(N, K, generator=g, device="cuda") < 0.1] = -math.inf
        index[0] = V            # rows without an entry
        logit[N // 2] = -math.inf
        logit[N - 1] = torch.finfo(logit_dtype).min
        index[N - 1, 0] = 0
    elif kind == "same":
        index[:] = index[:, :1]
    return index, logit


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,H,V,K", [(1, 8, 1, 1), (5, 40, 130, 3), (64, 128, 1000, 8), (130, 72, 2000, 33), (300, 256, 515, 100),
                                     (40, 64, 300, 1024), (600, 64, 1000, 64)])
@pytest.mark.parametrize("kind,T", [("plain", 1.0), ("ragged", 2.0), ("same", 0.5), ("ragged", 1.0)])
def test_distill(N, H, V, K, kind, T, dtype):
    g = gen(N + K)
    x, w = matrix(N, H, dtype, g), matrix(V, H, dtype, g, 0.3)
    logit_dtype = {"plain": torch.float32, "ragged": torch.bfloat16, "same": torch.float16}[kind]
    index, logit = teacher(N, V, K, g, logit_dtype, kind)
    dloss = torch.randn(N, generator=g, device="cuda")
    has, valid, shares, ent = shares_of(index, logit, V, T)
    x[~valid] = math.nan
    dloss[~valid] = math.nan
    ref = reference(x, w, shares, valid, ent, T, dloss)
    loss, lse, top = glu.linear_distill(x, w, index, logit, T)
    close(loss, ref["loss"], ref["tol"], "loss")
    close(lse, ref["lse"], ref["tol"], "lse")
    at = torch.where(has, index, 0)
    close(top, torch.where(has, ref["z"].gather(1, at), 0.0), ref["z_tol"].gather(1, at) + 2.0 ** -126, "top_logits")
    dx, dw = glu.linear_distill_bwd(dloss, x, w, index, logit, lse, top, T)
    close(dx, ref["dx"], ref["dx_tol"], "dx")
    close(dw, ref["dw"], ref["dw_tol"], "dw")
    assert glu.glu_wait_timeouts() == 0


@pytest.mark.parametrize("T", [2.0 ** -6, 100.0])
def test_distill_far_temperatures(T):
    N, H, V, K = 40, 64, 500, 9
    g = gen(17)
    x, w = matrix(N, H, torch.bfloat16, g, grid=True), matrix(V, H, torch.bfloat16, g, grid=True)
    index, logit = teacher(N, V, K, g, torch.float32, "plain")
    dloss = torch.rand(N, generator=g, device="cuda")
    has, valid, shares, ent = shares_of(index, logit, V, T)
    ref = reference(x, w, shares, valid, ent, T, dloss, exact=True)
    loss, lse, top = glu.linear_distill(x, w, index, logit, T)
    # logits over T of some hundreds: c1 z is one rounding of that size (in ref's bound), p's of d / T another
    slack = 2.0 ** -23 * (ref["z"].abs().amax(1) + 32.0) / T
    close(loss, ref["loss"], ref["tol"] + slack, "loss")
    close(lse, ref["lse"], ref["tol"] + slack, "lse")
    dx, dw = glu.linear_distill_bwd(dloss, x, w, index, logit, lse, top, T)
    more = 2 * slack.max() * dloss.max().double() / T * 2
    close(dx, ref["dx"], ref["dx_tol"] + more * w.double().abs().sum(0).max(), "dx")
    close(dw, ref["dw"], ref["dw_tol"] + more * x.double().abs().sum(0).max(), "dw")


def test_two_calls_at_once():
    """Two streams, each call with its own workspace and its own results."""
    N, H, V = 700, 512, 9000
    g = gen(31)
    w = matrix(V, H, torch.bfloat16, g, 0.1)
    xs = [matrix(N, H, torch.bfloat16, g) for _ in range(2)]
    ts = [targets(N, V, g, "some") for _ in range(2)]
    d = torch.rand(N, generator=g, device="cuda")

    def step(x, t):
        loss, lse = glu.linear_ce(x, w, t)
        return (loss, lse, *glu.linear_ce_bwd(d, x, w, t, loss, lse))

    want = [step(x, t) for x, t in zip(xs, ts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = step(xs[i], ts[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for u, v in zip(a, b):
            assert torch.equal(u, v)
    assert glu.glu_wait_timeouts() == 0


def test_rows_of_a_wider_matrix():
    """x and w as columns of wider matrices, dx and dw into columns of others."""
    N, H, V = 260, 80, 600
    g = gen(41)
    x = torch.randn(N, 3 * H, generator=g, device="cuda").half()[:, H:2 * H]
    w = (torch.randn(V, 2 * H, generator=g, device="cuda") * 0.2).half()[:, H:]
    t = targets(N, V, g, "some")
    dx = torch.zeros(N, 2 * H, device="cuda").half()[:, :H]
    dw = torch.zeros(V, 3 * H, device="cuda").half()[:, H:2 * H]
    check_ce(x, w, t, torch.rand(N, generator=g, device="cuda"), dx=dx, dw=dw)


def test_distill_strided_entries_and_pieces():
    N, H, V, K, T = 70, 64, 3000, 20, 1.5
    g = gen(3)
    x, w = matrix(N, H, torch.bfloat16, g), matrix(V, H, torch.bfloat16, g, 0.3)
    index = torch.randint(-1, V, (N, K + 7), generator=g, device="cuda")[:, 3:3 + K]
    logit = torch.randn(N, 2 * K, generator=g, device="cuda")[:, :K]
    dloss = torch.randn(N, generator=g, device="cuda")
    has, valid, shares, ent = shares_of(index, logit, V, T)
    ref = reference(x, w, shares, valid, ent, T, dloss)
    loss, lse, top = glu.linear_distill(x, w, index, logit, T)
    close(loss, ref["loss"], ref["tol"], "loss")
    full = glu.glu_linear_distill_workspace_bytes(N, H, V, K, 1)
    ws = torch.full((int(full * 0.8),), 255, dtype=torch.uint8, device="cuda")
    dx, dw = glu.linear_distill_bwd(dloss, x, w, index, logit, lse, top, T, workspace=ws)
    close(dx, ref["dx"], ref["dx_tol"], "dx")
    close(dw, ref["dw"], ref["dw_tol"], "dw")


@pytest.mark.parametrize("N", [100, 700])
def test_distill_in_pieces(N):
    H, V, K, T = 96, 2500, 12, 2.0
    g = gen(N)
    x, w = matrix(N, H, torch.float16, g), matrix(V, H, torch.float16, g, 0.3)
    index, logit = teacher(N, V, K, g, torch.float32, "ragged")
    dloss = torch.randn(N, generator=g, device="cuda")
    has, valid, shares, ent = shares_of(index, logit, V, T)
    ref = reference(x, w, shares, valid, ent, T, dloss)
    loss, lse, top = glu.linear_distill(x, w, index, logit, T)
    full = glu.glu_linear_distill_workspace_bytes(N, H, V, K, 1)
    for part in (0.9, 0.8, 0.7):
        ws = torch.full((int(full * part),), 255, dtype=torch.uint8, device="cuda")
        dx, dw = glu.linear_distill_bwd(dloss, x, w, index, logit, lse, top, T, workspace=ws)
        close(dx, ref["dx"], ref["dx_tol"], "dx")
        close(dw, ref["dw"], ref["dw_tol"], "dw")


@pytest.mark.parametrize("N", [60, 300])
def test_outputs_at_odd_places(N):
    """dx and dw off 16-byte boundaries and with gaps; what lies around them stays."""
    H, V = 77, 333
    g = gen(21)
    x, w = matrix(N, H, torch.bfloat16, g), matrix(V, H, torch.bfloat16, g, 0.3)
    for masked in ("none", "some"):
        t = targets(N, V, g, masked)
        dloss = torch.rand(N, generator=g, device="cuda")
        bx = torch.full((N + 2, H + 6), 7.0, dtype=torch.bfloat16, device="cuda")
        bw = torch.full((V + 2, H + 4), 7.0, dtype=torch.bfloat16, device="cuda")
        check_ce(x, w, t, dloss, dx=bx[1:-1, 3:3 + H], dw=bw[1:-1, 1:1 + H])
        bx[1:-1, 3:3 + H] = 7.0
        bw[1:-1, 1:1 + H] = 7.0
        assert torch.all(bx == 7.0) and torch.all(bw == 7.0)


def test_one_gradient_only():
    N, H, V = 200, 128, 900
    g = gen(1)
    x, w = matrix(N, H, torch.bfloat16, g), matrix(V, H, torch.bfloat16, g, 0.3)
    t = targets(N, V, g, "some")
    loss, lse = glu.linear_ce(x, w, t)
    d = torch.rand(N, generator=g, device="cuda")
    dx, dw = glu.linear_ce_bwd(d, x, w, t, loss, lse)
    only_x, none = glu.linear_ce_bwd(d, x, w, t, loss, lse, dw=False)
    assert none is None and torch.equal(only_x, dx)
    none, only_w = glu.linear_ce_bwd(d, x, w, t, loss, lse, dx=False)
    assert none is None and torch.equal(only_w, dw)
    assert glu.linear_ce_bwd(d, x, w, t, loss, lse, dx=False, dw=False) == (None, None)


def test_same_results_again_and_from_a_graph():
    N, H, V, K = 300, 256, 3000, 16
    g = gen(2)
    x, w = matrix(N, H, torch.bfloat16, g), matrix(V, H, torch.bfloat16, g, 0.1)
    t = targets(N, V, g, "some")
    index, logit = teacher(N, V, K, g, torch.float32, "ragged")
    d = torch.rand(N, generator=g, device="cuda")

    def step():
        loss, lse = glu.linear_ce(x, w, t)
        a = (loss, lse, *glu.linear_ce_bwd(d, x, w, t, loss, lse))
        loss, lse, top = glu.linear_distill(x, w, index, logit, 2.0)
        return (*a, loss, lse, top, *glu.linear_distill_bwd(d, x, w, index, logit, lse, top, 2.0))

    first = [v.clone() for v in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(2):
        graph.replay()
        for a, b in zip(first, captured):
            assert torch.equal(a, b)
    # new inputs in the same places
    x.copy_(matrix(N, H, torch.bfloat16, g))
    t.copy_(targets(N, V, g, "none"))
    graph.replay()
    again = step()
    for a, b in zip(again, captured):
        assert torch.equal(a, b)
    assert glu.glu_wait_timeouts() == 0


def test_another_stream():
    N, H, V = 200, 128, 900
    g = gen(4)
    x, w = matrix(N, H, torch.float16, g), matrix(V, H, torch.float16, g, 0.3)
    t = targets(N, V, g, "some")
    d = torch.rand(N, generator=g, device="cuda")
    loss, lse = glu.linear_ce(x, w, t)
    want = (loss, lse, *glu.linear_ce_bwd(d, x, w, t, loss, lse))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss2, lse2 = glu.linear_ce(x, w, t, stream=side)
    got = (loss2, lse2, *glu.linear_ce_bwd(d, x, w, t, loss2, lse2, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_no_rows():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(100, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = glu.linear_ce(x, w, t)
    assert loss.shape == (0,)
    dw = torch.full_like(w, 3.0)
    dx, dw = glu.linear_ce_bwd(loss, x, w, t, loss, lse, dw=dw)
    assert dx.shape == (0, 64) and torch.all(dw == 0)


def test_leading_shapes():
    g = gen(6)
    x = matrix(24, 64, torch.bfloat16, g).view(2, 3, 4, 64)
    w = matrix(500, 64, torch.bfloat16, g, 0.3)
    t = targets(24, 500, g, "none")
    a = glu.linear_ce(x, w, t.view(2, 3, 4))
    b = glu.linear_ce(x.view(24, 64), w, t)
    assert a[0].shape == (2, 3, 4) and torch.equal(a[0].flatten(), b[0])
    one = glu.linear_ce(x[0, 0, 0], w, t[0])
    assert one[0].shape == () and abs(one[0].item() - b[0][0].item()) < 1e-4


def test_directional_difference():
    """The gradients against differences of the loss itself, along one direction, on
    exact sums: the step is a grid step, the curvature bounded by its square."""
    N, H, V = 40, 64, 300
    g = gen(8)
    x, w = matrix(N, H, torch.float16, g, grid=True), matrix(V, H, torch.float16, g, grid=True)
    x, w = x * 0.25, w * 0.25
    t = targets(N, V, g, "none")
    loss, lse = glu.linear_ce(x, w, t)
    dx, dw = glu.linear_ce_bwd(torch.ones(N, device="cuda"), x, w, t, loss, lse)
    h = 2.0 ** -9
    v = torch.randint(0, 2, x.shape, generator=g, device="cuda").half() * 2 - 1
    up, down = glu.linear_ce(x + h * v, w, t)[0].double(), glu.linear_ce(x - h * v, w, t)[0].double()
    slope = (dx.double() * v.double()).sum(1)
    # third derivative of log sum exp along v: at most 8 max |w v|^3 / 6 h^2; the losses' own 2^-15 / h; 64 f16 entries of dx
    step = (v.double() @ w.double().T).abs().amax(1)
    tol = 8 * step ** 3 / 6 * h * h + 2.0 ** -15 / h + 64 * 2.0 ** -10 * dx.double().abs().amax(1)
    assert torch.all(((up - down) / (2 * h) - slope).abs() <= tol)


def test_offsets_past_32_bits():
    """A projection of more than 2^31 elements: the last tokens' logits and gradients."""
    N, H, V = 16, 4096, 540000
    x = torch.randn(N, H, generator=gen(1), device="cuda").bfloat16()
    w = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    last = V - 600
    w[last:] = torch.randn(600, H, generator=gen(2), device="cuda").bfloat16() * 0.05
    t = torch.arange(V - N, V, device="cuda")
    loss, lse = glu.linear_ce(x, w, t)
    d = torch.ones(N, device="cuda")
    dx, dw = glu.linear_ce_bwd(d, x, w, t, loss, lse)
    s = x.double() @ w[last:].double().T
    want = torch.logsumexp(torch.cat([s, torch.full((N, 1), math.log(last), device="cuda", dtype=torch.float64)], 1), 1)
    dz = (H * 2.0 ** -23 * (x.double().abs() @ w[last:].double().abs().T)).amax(1)
    # 4219 tiles: 132 in a chain of the join, 300 added at most elsewhere
    tol = 2 * dz + 500 * 2.0 ** -24 + 8 * 2.0 ** -24 * want
    assert torch.all((lse.double() - want).abs() <= tol)
    p = torch.exp(s - want[:, None])
    p[torch.arange(N), t - last] -= 1
    err = p.abs() * (2.0 ** -8 + 2 * tol[:, None] + 2.0 ** -18) + tol[:, None] * (p + 1).abs() * 2.0 ** -3
    val = p.T @ x.double()
    close(dw[last:], val, err.T @ x.double().abs() + 2.0 ** -8 * val.abs() + 1e-6, "dw")
    val = p @ w[last:].double()
    # the tokens before hold zeros and add nothing
    close(dx, val, err @ w[last:].double().abs() * 1.01 + 2.0 ** -8 * val.abs() + 1e-6, "dx")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N", [1, 64, 300])
def test_ce_confident_rows_relative_to_the_loss(N, dtype):
    """Rows whose target has nearly all the probability, on exact sums: the loss, the other
    tokens' share, is good relative to itself, down to 1e-17, and so is the target's gradient.

    A term 2^-d of the target's is off by four roundings of d 2^-24 (the product with
    log2 e, its constant, the differences in a tile and between tiles) and 2^-22 for each
    of two exponentials; their sum by 300 roundings; log1p and expm1 by 2^-22."""
    H, V = 128, 2000
    g = gen(N)
    w = matrix(V, H, dtype, g, grid=True)
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    x = torch.round(w[t].float() * (torch.arange(1, N + 1, device="cuda")[:, None] % 4 + 1) / 4 * 8).div(8).to(dtype)
    loss, lse = glu.linear_ce(x, w, t)
    s = x.double() @ w.double().T
    d = s - s.gather(1, t[:, None])
    want = torch.log1p(torch.exp(d).scatter_(1, t[:, None], 0.0).sum(1))
    assert N == 1 or (want.min() < 1e-13 and want.max() > 1e-4)
    rel = (4 * d.abs().amax(1) * math.log2(math.e) + 300) * 2.0 ** -24 + 4 * 2.0 ** -22
    assert torch.all(loss >= 0)
    close(loss, want, rel * want, "loss")
    # one row's gradient alone: dw of its target is g x, three roundings (g, the product's sum is exact, dw)
    for i in sorted({0, N // 3, N // 2, N - 1}):
        dloss = torch.zeros(N, device="cuda")
        dloss[i] = 2.0 ** 12
        dw = glu.linear_ce_bwd(dloss, x, w, t, loss, lse, dx=False)[1]
        val = 2.0 ** 12 * torch.expm1(-want[i]) * x[i].double()
        u = U[dtype]
        tol = (2.1 * u + rel[i]) * val.abs()
        if dtype == torch.float16:      # steps of f16: dw's, and g's under its scale (2^12 goes to 2^13)
            tol = tol + 2.0 ** -25 + 2.0 ** -26 * x[i].double().abs()
        close(dw[t[i]], val, tol, "dw")


def test_f16_scale_with_a_low_temperature():
    """The power of two that g is scaled by times 1 / T may pass the largest float."""
    N, H, V, K, T = 40, 64, 300, 5, 2.0 ** -10
    g = gen(19)
    x, w = matrix(N, H, torch.float16, g, 0.01), matrix(V, H, torch.float16, g, 0.1)
    index, logit = teacher(N, V, K, g, torch.float32, "plain")
    loss, lse, top = glu.linear_distill(x, w, index, logit, T)
    for dloss in (2.0 ** -118, 2.0 ** -140):
        dx, dw = glu.linear_distill_bwd(torch.full((N,), dloss, device="cuda"), x, w, index, logit, lse, top, T)
        # below half of f16's smallest step
        assert torch.all(dx == 0) and torch.all(dw == 0)


def test_very_many_rows():
    """Rows that one block lists in more than one stretch."""
    N, H, V = 512 * 4096 + 300001, 8, 3
    g = gen(23)
    x, w = matrix(N, H, torch.bfloat16, g), matrix(V, H, torch.bfloat16, g)
    for masked in ("some", "last"):
        check_ce(x, w, targets(N, V, g, masked), torch.rand(N, generator=g, device="cuda"))


def test_time_of_very_many_rows():
    """Eight times the rows take about eight times as long (not 64 times: the rows were
    counted anew for every 4096 of them)."""
    H, V = 8, 2
    w = torch.randn(V, H, device="cuda").half()
    took = []
    for N in (1 << 21, 1 << 24):
        x = torch.randn(N, H, device="cuda").half()
        t = torch.randint(-1, V, (N,), device="cuda")
        ws = torch.empty(glu.glu_linear_ce_workspace_bytes(N, H, V, 0), dtype=torch.uint8, device="cuda")
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            glu.linear_ce(x, w, t, workspace=ws)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        took.append(min(times))
    assert took[1] <= 20 * took[0], took


def test_no_rows_and_one_token():
    """The row stride of a matrix of one row says nothing, with no rows of x either."""
    w = torch.ones(1, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    t, f = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    dw = torch.full((64,), 3.0, dtype=torch.bfloat16, device="cuda").as_strided((1, 64), (1, 1))
    glu.linear_ce_bwd(f, x, w, t, f, f, dw=dw)
    assert torch.all(dw == 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N", [50, 300])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_gradients_that_are_not_finite_come_through(bad, N, dtype):
    """What a gradient scaler must see: dloss of infinity or NaN in rows that take part."""
    H, V, K = 72, 700, 5
    g = gen(29)
    x, w = matrix(N, H, dtype, g), matrix(V, H, dtype, g, 0.2)
    x[x == 0] = 1.0
    t = targets(N, V, g, "some")
    t[3], t[N // 2 + 1] = 1, 2
    index, logit = teacher(N, V, K, g, torch.float32, "plain")
    dloss = torch.rand(N, generator=g, device="cuda") + 0.5
    rows = torch.zeros(N, dtype=torch.bool, device="cuda")
    rows[[3, N // 2 + 1]] = True
    hurt, without = dloss.masked_fill(rows, bad), dloss.masked_fill(rows, 0.0)
    loss, lse = glu.linear_ce(x, w, t)
    kd, klse, top = glu.linear_distill(x, w, index, logit, 2.0)
    for grads in (lambda d: glu.linear_ce_bwd(d, x, w, t, loss, lse),
                  lambda d: glu.linear_distill_bwd(d, x, w, index, logit, klse, top, 2.0)):
        (dx, dw), (dx0, dw0) = grads(hurt), grads(without)
        assert not torch.isfinite(dx[rows]).any() and not torch.isfinite(dw).any()
        assert torch.equal(dx[~rows], dx0[~rows]) and torch.isfinite(dx0).all() and torch.isfinite(dw0).all()


def test_f16_gradients_far_apart():
    """dloss over 2^24: a row all of whose g is at least 2^-27 of the largest |dloss| keeps
    f16's relative rounding; smaller entries are rounded to multiples of 2^-37 of it at most."""
    N, H, V = 200, 64, 300
    g = gen(37)
    x, w = matrix(N, H, torch.float16, g), matrix(V, H, torch.float16, g, 0.1)
    t = targets(N, V, g, "none")
    dloss = 2.0 ** (10 - torch.arange(N, device="cuda") % 25).float()
    check_ce(x, w, t, dloss)            # with those steps, absolute
    loss, lse = glu.linear_ce(x, w, t)
    dx = glu.linear_ce_bwd(dloss, x, w, t, loss, lse, dw=False)[0]
    x64, w64 = x.double(), w.double()
    z = x64 @ w64.T
    q = torch.softmax(z, 1)
    q[torch.arange(N, device="cuda"), t] -= 1
    gg = q * dloss.double()[:, None]
    normal = gg.abs().amin(1) >= 2.0 ** -27 * dloss.max().double()
    assert 50 < int(normal.sum()) < N - 50
    dz = (H * 2.0 ** -23 * (x64.abs() @ w64.abs().T)).amax(1)[:, None]
    # the exponential (lse's bound and the logit's), g's rounding, V products of fp32 sums, dx's rounding
    rel = 4 * dz + 300 * 2.0 ** -24 + 2.0 ** -17 + 2.0 ** -11 * 1.01 + V * 2.0 ** -23
    tol = (rel * gg.abs() + (gg < 0) * dloss[:, None].double() * (4 * dz + 2.0 ** -15)) @ w64.abs()
    val = gg @ w64
    close(dx[normal], val[normal], (tol * (1 + 2.0 ** -11) + 2.0 ** -11 * val.abs() + 2.0 ** -25)[normal], "dx")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N", [60, 300])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_rows_that_are_not_finite(bad, N, dtype):
    """Infinity or NaN in hidden rows that take part stays in those rows' losses and dx, and is in all of dw, as 64 bits have it."""
    H, V, K = 72, 700, 5
    g = gen(43)
    x, w = matrix(N, H, dtype, g), matrix(V, H, dtype, g, 0.2)
    w[w == 0] = 0.125
    t = targets(N, V, g, "some")
    t[5], t[N - 2] = 1, 699
    index, logit = teacher(N, V, K, g, torch.float32, "plain")
    d = torch.rand(N, generator=g, device="cuda") + 0.5
    rows = torch.zeros(N, dtype=torch.bool, device="cuda")
    rows[[5, N - 2]] = True
    hurt = matrix(N, H, dtype, g)
    hurt.copy_(x)
    hurt[5, 7] = bad
    hurt[N - 2, H - 1] = bad

    def ce(x):
        loss, lse = glu.linear_ce(x, w, t)
        return (loss, lse, *glu.linear_ce_bwd(d, x, w, t, loss, lse))

    def distill(x):
        loss, lse, top = glu.linear_distill(x, w, index, logit, 2.0)
        return (loss, lse, *glu.linear_distill_bwd(d, x, w, index, logit, lse, top, 2.0))

    for f in (ce, distill):
        got, want = f(hurt), f(x)
        for a, b in zip(got[:3], want[:3]):
            assert torch.equal(a[~rows], b[~rows]) and not torch.isfinite(a[rows]).any()
        assert not torch.isfinite(got[3]).any()


def test_tokens_that_are_not_finite():
    """A projection row of NaN is in every row's softmax; one of infinities makes logits of
    -inf, which have no share, or +inf, which leave nothing finite."""
    N, H, V = 150, 64, 400
    g = gen(47)
    x, w = matrix(N, H, torch.bfloat16, g), matrix(V, H, torch.bfloat16, g, 0.2)
    x[x == 0] = 1.0
    t = targets(N, V, g, "none") % (V - 1)
    d = torch.ones(N, device="cuda")
    w[V - 1] = 0.0
    w[V - 1, 3] = math.nan
    loss, lse = glu.linear_ce(x, w, t)
    dx, dw = glu.linear_ce_bwd(d, x, w, t, loss, lse)
    for v in (loss, lse, dx, dw):
        assert not torch.isfinite(v).any()
    w[V - 1] = 0.0
    x[:, 4] = torch.where(torch.arange(N, device="cuda") % 2 == 0, -1.0, 1.0)
    w[V - 1, 4] = math.inf              # 0 elsewhere: logits of -inf and +inf in turn
    loss, lse = glu.linear_ce(x, w, t)
    low = x[:, 4] < 0
    want = glu.linear_ce(x, w[:V - 1], t)
    tol = 600 * 2.0 ** -24 + 2.0 ** -19 + 16 * 2.0 ** -24 * want[1].abs().double()
    close(loss[low], want[0][low].double(), tol[low], "loss")
    close(lse[low], want[1][low].double(), tol[low], "lse")
    assert not torch.isfinite(loss[~low]).any()


def test_distill_on_another_stream_and_one_gradient_only():
    N, H, V, K, T = 200, 128, 900, 9, 1.5
    g = gen(53)
    x, w = matrix(N, H, torch.float16, g), matrix(V, H, torch.float16, g, 0.3)
    index, logit = teacher(N, V, K, g, torch.float32, "ragged")
    d = torch.rand(N, generator=g, device="cuda")
    loss, lse, top = glu.linear_distill(x, w, index, logit, T)
    dx, dw = glu.linear_distill_bwd(d, x, w, index, logit, lse, top, T)
    for kw in ({"dx": False}, {"dw": False}, {"dx": False, "dw": False}):
        a, b = glu.linear_distill_bwd(d, x, w, index, logit, lse, top, T, **kw)
        assert a is None if "dx" in kw else torch.equal(a, dx)
        assert b is None if "dw" in kw else torch.equal(b, dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss2, lse2, top2 = glu.linear_distill(x, w, index, logit, T, stream=side)
    got = glu.linear_distill_bwd(d, x, w, index, logit, lse2, top2, T, stream=side)
    only = glu.linear_distill_bwd(d, x, w, index, logit, lse2, top2, T, dx=False, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((loss, lse, top, dx, dw, dw), (loss2, lse2, top2, *got, only[1])):
        assert torch.equal(a, b)
    assert only[0] is None


@pytest.mark.parametrize("H,wide", [(64, 64), (77, 80), (1, 8), (1030, 1032)])
def test_gradients_have_rows_on_16_bytes(H, wide):
    """dx and dw that are allocated here lie as x and w must: rows on 16-byte boundaries,
    views of wider rows where H is no multiple of 8; the values are those of plain matrices."""
    g = gen(59)
    x, w = matrix(30, H, torch.float16, g).unflatten(0, (5, 6)), matrix(200, H, torch.float16, g, 0.2)
    t = targets(30, 200, g, "none").view(5, 6)
    loss, lse = glu.linear_ce(x, w, t)
    d = torch.rand(5, 6, generator=g, device="cuda")
    dx, dw = glu.linear_ce_bwd(d, x, w, t, loss, lse)
    assert dx.shape == x.shape and dx.stride() == (6 * wide, wide, 1) and dx.data_ptr() % 16 == 0
    assert dw.shape == w.shape and dw.stride() == (wide, 1) and dw.data_ptr() % 16 == 0
    px, pw = torch.empty(5, 6, H, dtype=x.dtype, device="cuda"), torch.empty(200, H, dtype=x.dtype, device="cuda")
    glu.linear_ce_bwd(d, x, w, t, loss, lse, dx=px, dw=pw)
    assert torch.equal(px, dx) and torch.equal(pw, dw)


@pytest.mark.parametrize("N", [64, 300])
def test_dx_is_summed_in_segments(N):
    """dx over a large vocabulary, logits on exact sums: 256 steps of 16 products in one
    accumulator, each of which may drop two units of 2^-23 of what is in it, and one rounded
    addition a segment or part (32 and 16 at most); beside it g's own rounding."""
    H, V = 64, 131072
    g = gen(61)
    x = matrix(N, H, torch.float16, g, grid=True) * 0.125
    w = matrix(V, H, torch.float16, g, grid=True)
    t = targets(N, V, g, "none")
    dloss = torch.full((N,), 1024.0, device="cuda")
    loss, lse = glu.linear_ce(x, w, t)
    dx = glu.linear_ce_bwd(dloss, x, w, t, loss, lse, dw=False)[0]
    z = x.double() @ w.double().T
    gg = torch.softmax(z, 1)
    gg[torch.arange(N, device="cuda"), t] -= 1
    gg *= 1024.0
    # g: the exponential and its argument (2^-19), lse (V / 128 parts joined, a few hundred roundings), 2^-11
    rel = 2.0 ** -11 + 2.0 ** -19 + 600 * 2.0 ** -24 + 8 * 2.0 ** -24 * lse.abs().max().double()
    rel = rel * 1.01 + (2 * 256 + 48) * 2.0 ** -23
    val = gg @ w.double()
    close(dx, val, rel * (gg.abs() @ w.double().abs()) + 2.0 ** -11 * val.abs() * 1.01 + 2.0 ** -25, "dx")


@pytest.mark.parametrize("N,H,V", [(2048, 640, 32768), (1000, 1030, 40000), (16384, 264, 16000), (300, 2056, 51111)])
@pytest.mark.parametrize("masked", ["none", "some", "last"])
def test_x_transposed_before_dw(N, H, V, masked):
    """N H (V - 9400) above 2.5e10: dw's product reads x transposed."""
    assert N * H * (V - 9400) > 2.5e10
    g = gen(N + H)
    x, w = matrix(N, H, torch.bfloat16, g), matrix(V, H, torch.bfloat16, g, 1.0 / math.sqrt(H))
    t = targets(N, V, g, masked)
    dloss = torch.rand(N, generator=g, device="cuda")
    none = (t < 0) | (t >= V)
    x[none] = math.nan
    dloss[none] = math.nan
    loss, lse, dx, dw = check_ce(x, w, t, dloss)
    # in pieces the transposed rows are read again
    ws = torch.full((int(glu.glu_linear_ce_workspace_bytes(N, H, V, 1) * 0.8),), 255, dtype=torch.uint8, device="cuda")
    check_ce(x, w, t, dloss, workspace=ws)


def test_transposed_or_not_the_same_sums():
    """Rows that take part give the same dw whichever way x is read: 700 rows of a batch that is
    transposed, alone in one that is not."""
    H, V, n = 1024, 32000, 700
    g = gen(67)
    x, w = matrix(1200, H, torch.bfloat16, g), matrix(V, H, torch.bfloat16, g, 0.05)
    t = targets(1200, V, g, "none")
    t[n:] = -1
    assert n * H * (V - 9400) < 2.5e10 < 1200 * H * (V - 9400)
    d = torch.rand(1200, generator=g, device="cuda")
    loss, lse = glu.linear_ce(x, w, t)
    a = glu.linear_ce_bwd(d, x, w, t, loss, lse, dx=False)[1]
    b = glu.linear_ce_bwd(d[:n].contiguous(), x[:n], w, t[:n].contiguous(), loss[:n].contiguous(), lse[:n].contiguous(), dx=False)[1]
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N", [40, 300])
def test_mean_over_any_number_of_rows(N, dtype):
    """Every row's dloss is one number that 16 bits do not hold, the target's probability is
    below half a step and only its token has a row in the projection that is not 0: g is
    -dloss to 2^-12, so dx is its exact value rounded once, but for 2^-12 of it."""
    H, V = 64, 20000
    g = gen(71)
    x = matrix(N, H, dtype, g, 0.1)
    w = torch.zeros(V, H, dtype=dtype, device="cuda")
    w[777] = matrix(1, H, dtype, g, 0.3)[0]
    t = torch.full((N,), 777, device="cuda")
    dloss = torch.full((N,), 1024 / 3000, device="cuda")
    loss, lse = glu.linear_ce(x, w, t)
    dx = glu.linear_ce_bwd(dloss, x, w, t, loss, lse, dw=False)[0]
    share = torch.softmax(x.double() @ w.double().T, 1)[:, 777:778]
    assert share.max() < 2.0 ** -12
    val = (share - 1) * dloss.double()[:, None] * w[777].double()
    half_step = torch.exp2(torch.floor(torch.log2(val.abs()))) * U[dtype]
    close(dx, val, half_step + (2.0 ** -12 + 2.0 ** -16) * val.abs() + 2.0 ** -25, "dx")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N", [1, 16, 50, 64])
@pytest.mark.parametrize("op", ["ce", "distill"])
@pytest.mark.parametrize("pieces", [False, True])
def test_few_rows_have_g_in_two_parts(pieces, op, N, dtype):
    """Up to 64 rows dx and dw see g rounded to twice the type's bits (2^-16 or 2^-22, in f16
    under the scale 2^-38 of the largest at least), on exact sums: beside their own rounding
    remain the exponential and the loss (as in ``reference``) and the sums, at most 256 steps of
    two units of 2^-23 and 64 rounded additions."""
    H, V, K, T = 72, 3100, 8, 1.5 if op == "distill" else 1.0
    g = gen(N + 73)
    x = matrix(N, H, dtype, g, grid=True) * 0.25
    w = matrix(V, H, dtype, g, grid=True)
    dloss = torch.rand(N, generator=g, device="cuda") + 0.5
    if op == "ce":
        t = targets(N, V, g, "none")
        valid = torch.ones(N, dtype=torch.bool, device="cuda")
        shares = torch.zeros(N, V, dtype=torch.float64, device="cuda").scatter_(1, t[:, None], 1.0)
        ent = torch.zeros(N, dtype=torch.float64, device="cuda")
        loss, lse = glu.linear_ce(x, w, t)
        full = glu.glu_linear_ce_workspace_bytes(N, H, V, 1)
    else:
        index, logit = teacher(N, V, K, g, torch.float32, "plain")
        _, valid, shares, ent = shares_of(index, logit, V, T)
        loss, lse, top = glu.linear_distill(x, w, index, logit, T)
        full = glu.glu_linear_distill_workspace_bytes(N, H, V, K, 1)
    ws = torch.full((int(full * 0.8) if pieces else full,), 255, dtype=torch.uint8, device="cuda")
    if op == "ce":
        dx, dw = glu.linear_ce_bwd(dloss, x, w, t, loss, lse, workspace=ws)
    else:
        dx, dw = glu.linear_distill_bwd(dloss, x, w, index, logit, lse, top, T, workspace=ws)
    ref = reference(x, w, shares, valid, ent, T, exact=True)
    x64, w64, c = x.double(), w.double(), dloss.double()[:, None] / T
    p = torch.softmax(x64 @ w64.T / T, 1)
    gg, tol = c * (p - shares), ref["tol"][:, None]
    u = U[dtype]
    eg = c * (p * (tol + 2.0 ** -19) + shares * (tol + 2.0 ** -20))
    eg = eg + u * u * (gg.abs() + eg) + (2.0 ** -38 * c.max() if dtype == torch.float16 else 0.0)
    sums = (2 * 256 + 64) * 2.0 ** -23
    for got, val, err, size, what in ((dx, gg @ w64, eg @ w64.abs(), gg.abs() @ w64.abs(), "dx"),
                                      (dw, gg.T @ x64, eg.T @ x64.abs(), gg.abs().T @ x64.abs(), "dw")):
        err = 1.01 * err + sums * size
        close(got, val, err + u * (val.abs() + err) + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134), what)


@pytest.mark.parametrize("N", [40, 70, 300])
def test_very_large_projection_rows(N):
    """bf16's range: a projection of 2^116 and hidden rows of 2^-116 have ordinary logits, and a
    dx of 2^116 times the ordinary one."""
    H, V = 64, 900
    g = gen(79)
    x, w = matrix(N, H, torch.bfloat16, g, grid=True), matrix(V, H, torch.bfloat16, g, grid=True)
    t = targets(N, V, g, "none")
    d = torch.rand(N, generator=g, device="cuda") + 0.5

    def step(x, w):
        loss, lse = glu.linear_ce(x, w, t)
        return loss, lse, glu.linear_ce_bwd(d, x, w, t, loss, lse, dw=False)[0]

    big = 2.0 ** 116
    got, want = step(x / big, w * big), step(x, w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isfinite(got[2]).all() and torch.equal(got[2] / big, want[2])


@pytest.mark.parametrize("N", [4, 80, 300])
def test_bf16_shares_at_the_lower_end_of_its_range(N):
    """Probabilities down to 2^-132 under a dloss of 100: g keeps bf16's steps where fp32 has them."""
    H, V = 64, 500
    x = torch.zeros(N, H, device="cuda").bfloat16()
    x[:, 0], x[:, 1] = 5.75, 1.0
    w = torch.zeros(V, H, device="cuda").bfloat16()
    w[:, 0] = -(torch.arange(V, device="cuda") % 256) / 16
    w[:, 2] = 1.0
    t = torch.zeros(N, dtype=torch.int64, device="cuda")
    dloss = torch.full((N,), 0.01, device="cuda")
    dloss[:4] = torch.tensor([100.0, 50.0, 3.0, 0.1])
    check_ce(x, w, t, dloss, exact=True)
