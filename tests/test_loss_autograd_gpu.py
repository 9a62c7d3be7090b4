"""The losses over a vocabulary as autograd functions and in a small model: norm, gated
MLP, norm, loss.  The model's own gradients are those of its parts' tests; here the
loss's gradients at the hidden rows and the projection are compared with the formula in
64 bits, and what runs behind them must be what those hidden gradients give."""
import math

import pytest
import torch

import glu_activation_mlps_gb300 as glu
from glu_activation_mlps_gb300 import autograd as ag

pytestmark = pytest.mark.gpu
H, V, N = 256, 3000, 300


def model(seed=0):
    torch.manual_seed(seed)
    kw = {"device": "cuda", "dtype": torch.bfloat16}
    return (ag.FusedAddRMSNorm(H, **kw), ag.GatedMLP(H, 512, **kw), ag.FusedAddRMSNorm(H, **kw), ag.VocabLoss(H, V, **kw))


def hidden_rows(parts, x, res):
    norm, mlp, last, _ = parts
    h, y = norm(x, res)
    return last(mlp(y), h)[1]


def inputs():
    x = torch.randn(N, H, device="cuda").bfloat16().requires_grad_()
    res = torch.randn(N, H, device="cuda").bfloat16().requires_grad_()
    target = torch.randint(0, V, (N,), device="cuda")
    target[: N // 3] = -100
    return x, res, target


@pytest.mark.parametrize("loss_kind", ["ce", "distill"])
def test_model_gradients(loss_kind):
    parts = model()
    x, res, target = inputs()
    head = parts[3]
    index = torch.randint(0, V, (N, 7), device="cuda")
    logit = torch.randn(N, 7, device="cuda")
    index[target < 0] = -1
    T = 2.0

    def loss_of(rows):
        return head(rows, target) if loss_kind == "ce" else head.distill(rows, index, logit, T)

    rows = hidden_rows(parts, x, res)
    rows.retain_grad()
    loss = loss_of(rows)
    assert loss.dtype == torch.float32 and loss.shape == ()
    loss.backward()
    # the formula in 64 bits from the same hidden rows
    r64 = rows.detach().double().requires_grad_()
    w64 = head.weight.detach().double().requires_grad_()
    z = r64 @ w64.T
    valid = target >= 0
    n = int(valid.sum())
    if loss_kind == "ce":
        ref = (torch.logsumexp(z, 1) - z.gather(1, target.clamp_min(0)[:, None])[:, 0])[valid].sum() / n
        share = torch.zeros_like(z).scatter_(1, target.clamp_min(0)[:, None], 1.0)
    else:
        p = torch.softmax(logit.double() / T, 1)
        lq = torch.log_softmax(z / T, 1).gather(1, index.clamp_min(0))
        ref = (p * (p.log() - lq)).sum(1)[valid].sum() / n
        share = torch.zeros_like(z).scatter_add_(1, index.clamp_min(0), p)
    ref.backward()
    dz = (H * 2.0 ** -23 * (r64.detach().abs() @ w64.detach().abs().T)).max().item()
    assert abs(loss.item() - ref.item()) <= 2 * dz + 2.0 ** -14 + 2.0 ** -20 * abs(ref.item())
    t = T if loss_kind == "distill" else 1.0
    with torch.no_grad():
        q = torch.softmax(z / t, 1)
        # entries of g: 16 bits, and the exponential's and the loss's errors
        eg = (2.0 ** -8 * (q - share).abs() + (4 * dz + 2.0 ** -13) * (q + share)) / (n * t) * valid[:, None]
        for got, want, err in ((rows.grad, r64.grad, eg @ w64.abs()), (head.weight.grad, w64.grad, eg.T @ r64.abs())):
            slack = err * 1.01 + 2.0 ** -8 * (want.abs() + err) + 2.0 ** -60
            assert torch.all((got.double() - want).abs() <= slack)
    assert torch.all(rows.grad[~valid] == 0)
    # the rest of the model from those gradients alone
    first = [x.grad.clone(), res.grad.clone(), parts[1].down_proj.weight.grad.clone()]
    grad = rows.grad.clone()
    for p_ in (x, res, *parts[1].parameters()):
        p_.grad = None
    hidden_rows(parts, x, res).backward(grad)
    for a, b in zip(first, [x.grad, res.grad, parts[1].down_proj.weight.grad]):
        assert torch.equal(a, b)


def test_reductions_and_broadcast_gradients():
    head = model()[3]
    _, _, target = inputs()
    x = torch.randn(N, H, device="cuda").bfloat16().requires_grad_()
    each = head(x, target, reduction="none")
    valid = target >= 0
    assert each.shape == (N,) and torch.all(each[~valid] == 0)
    total, mean = head(x, target, reduction="sum"), head(x, target)
    assert abs(total.item() - each.double().sum().item()) <= 2.0 ** -16 * total.item()
    assert abs(mean.item() - total.item() / int(valid.sum())) <= 2.0 ** -20 * mean.item()
    with pytest.raises(ValueError):
        head(x, target, reduction="median")
    total.backward()            # one scalar gradient, broadcast over the rows
    a = x.grad.clone()
    x.grad = None
    each2 = head(x, target, reduction="none")
    each2.backward(torch.ones(N, device="cuda"))
    assert torch.equal(a, x.grad)
    none = head(x.detach(), torch.full_like(target, -100))
    assert none.item() == 0.0


def test_only_wanted_gradients():
    head = model()[3]
    _, _, target = inputs()
    x = torch.randn(N, H, device="cuda").bfloat16()
    head(x, target).backward()              # x wants none
    assert x.grad is None and head.weight.grad is not None
    w = head.weight.detach()
    x.requires_grad_()
    ag.linear_cross_entropy(x, w, target).backward()
    assert x.grad is not None and w.grad is None
    with torch.no_grad():
        assert head(x, target).requires_grad is False


def test_module_is_a_projection():
    lin = torch.nn.Linear(H, V, bias=False, device="cuda", dtype=torch.bfloat16)
    head = ag.VocabLoss.from_linear(lin)
    assert head.weight is lin.weight
    x = torch.randn(4, H, device="cuda").bfloat16()
    assert torch.equal(head.logits(x), glu.gemm_nt(x, lin.weight))
    with pytest.raises(ValueError):
        ag.VocabLoss(12, V)
    with pytest.raises(ValueError):
        ag.VocabLoss.from_linear(torch.nn.Linear(H, 16, device="cuda"))


def test_training_step_in_a_graph():
    """Forward and backward captured on a side stream and replayed with new inputs."""
    head = model()[3]
    x = torch.randn(N, H, device="cuda").bfloat16().requires_grad_()
    target = torch.randint(0, V, (N,), device="cuda")

    def step():
        loss = head(x, target)
        return (loss, *torch.autograd.grad(loss, (x, head.weight)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    with torch.no_grad():
        x.copy_(torch.randn(N, H, device="cuda"))
        target.copy_(torch.randint(0, V, (N,), device="cuda"))
    graph.replay()
    got = [v.clone() for v in captured]
    for a, b in zip(got, step()):
        assert torch.equal(a, b)
    assert math.isfinite(got[0].item())


@pytest.mark.parametrize("hidden,dtype", [(64, torch.bfloat16), (75, torch.float16)])
def test_shifted_targets(hidden, dtype):
    """A batch of sequences, each row's target the next token: slices that have no single
    row stride give what their copies give, values and gradients."""
    B, S, V_, K = 3, 21, 500, 6
    torch.manual_seed(1)
    wide = hidden + -hidden % 8
    w = (torch.randn(V_, wide, device="cuda") * 0.2).to(dtype)[:, :hidden].requires_grad_()
    x = torch.randn(B, S, wide, device="cuda").to(dtype)[..., :hidden].requires_grad_()
    tokens = torch.randint(0, V_, (B, S), device="cuda")
    index, logit = torch.randint(0, V_, (B, S, K), device="cuda"), torch.randn(B, S, K, device="cuda")
    d = torch.rand(B, S - 1, device="cuda")

    def padded(t):
        return torch.nn.functional.pad(t, (0, wide - hidden))[..., :hidden]

    for f, slices in ((ag.linear_cross_entropy, (tokens[:, 1:],)),
                      (ag.linear_distillation, (index[:, 1:], logit[:, 1:]))):
        loss = f(x[:, :-1], w, *slices, reduction="none")
        got = torch.autograd.grad(loss, (x, w), d)
        flat = padded(x.detach()[:, :-1].reshape(-1, hidden)).requires_grad_()
        want_loss = f(flat, w, *(v.reshape(B * (S - 1), *v.shape[2:]) for v in slices), reduction="none")
        dx, dw = torch.autograd.grad(want_loss, (flat, w), d.flatten())
        assert loss.shape == (B, S - 1) and torch.equal(loss.flatten(), want_loss)
        assert torch.equal(got[0][:, :-1].reshape(-1, hidden), dx) and torch.equal(got[1], dw)
        assert torch.all(got[0][:, -1] == 0)
        assert torch.isfinite(f(x[:, :-1], w, *slices))


def test_rows_that_do_not_lie_side_by_side():
    """Transposed, broadcast and unaligned hidden rows, transposed and broadcast entries."""
    torch.manual_seed(2)
    w = (torch.randn(300, 64, device="cuda") * 0.2).bfloat16()
    target = torch.randint(0, 300, (10,), device="cuda")
    base = torch.randn(64 * 10 + 1, device="cuda").bfloat16()
    views = (base[:-1].view(64, 10).t(), base[:64].expand(10, 64), base[1:].view(10, 64))
    index = torch.randint(0, 300, (4, 10), device="cuda").t()
    logit = torch.randn(4, device="cuda").expand(10, 4)
    for x in views:
        x = x.detach().requires_grad_()
        y = x.detach().contiguous().clone().requires_grad_()
        for f, a, b in ((ag.linear_cross_entropy, (target,), (target,)),
                        (ag.linear_distillation, (index, logit), (index.contiguous(), logit.contiguous()))):
            got, want = f(x, w, *a), f(y, w, *b)
            assert torch.equal(got, want)
            assert torch.equal(torch.autograd.grad(got, x)[0], torch.autograd.grad(want, y)[0])


def test_last_row_of_each_sequence():
    """x[:, -1:], whose innermost leading dimension has one entry: its stride says nothing."""
    torch.manual_seed(3)
    head = model()[3]
    x = torch.randn(5, 9, H, device="cuda").bfloat16()
    last, flat = x[:, -1:], x[:, -1].contiguous()
    assert torch.equal(head.logits(last)[:, 0], head.logits(flat))
    target = torch.randint(0, V, (5,), device="cuda")
    loss, lse = glu.linear_ce(last, head.weight, target[:, None])
    want = glu.linear_ce(flat, head.weight, target)
    assert torch.equal(loss[:, 0], want[0]) and torch.equal(lse[:, 0], want[1])
    assert torch.equal(head(last, target[:, None]), head(flat, target))
    assert torch.equal(glu.fwd(last, last)[:, 0], glu.fwd(flat, flat))
    q, s = glu.quantize(last)
    assert torch.equal(q[:, 0].float(), glu.quantize(flat)[0].float())


def test_module_as_the_readme_has_it():
    torch.manual_seed(4)
    x = torch.randn(20, 64, device="cuda").bfloat16().requires_grad_()
    head = ag.VocabLoss(64, 100, device="cuda")
    head(x, torch.randint(0, 100, (20,), device="cuda")).backward()
    assert x.grad.dtype == head.weight.grad.dtype == torch.bfloat16


def test_logits_of_slices():
    head = model()[3]
    x = torch.randn(4, 7, H, device="cuda").bfloat16()
    want = head.logits(x)
    assert torch.equal(head.logits(x[:, :-1]), want[:, :-1])
    assert torch.equal(head.logits(x.transpose(0, 1)), want.transpose(0, 1))
