"""Argument rules of the losses over a vocabulary: host checks, no GPU.

Every refusal comes before any CUDA call, so made-up addresses do; calls whose
arguments are in order get as far as asking for the device, which a machine
without one refuses (GLU_ERR_CUDA)."""
import math

import pytest

import glu_activation_mlps_gb300 as glu

N, H, V, K = 300, 128, 1000, 8
BF16, F16, F32 = 2, 1, 0
NULL, SHAPE, STRIDE, ALIAS, ENUM, CUDA, WORKSPACE, VALUE = -1, -2, -3, -4, -5, -6, -7, -8
BIG = 1 << 30
AT = {n: (i + 1) * (1 << 34) for i, n in enumerate(
    ("x", "w", "target", "index", "logit", "loss", "lse", "top_logits", "dloss", "dx", "dw", "workspace"))}

ORDER = {
    "ce_fwd": "x x_stride w w_stride target loss lse N H V dtype workspace workspace_bytes stream",
    "ce_bwd": "dloss x x_stride w w_stride target loss lse dx dx_stride dw dw_stride N H V dtype workspace "
              "workspace_bytes stream",
    "distill_fwd": "x x_stride w w_stride index index_stride logit logit_stride temperature loss lse top_logits N H V K "
                   "dtype logit_dtype workspace workspace_bytes stream",
    "distill_bwd": "dloss x x_stride w w_stride index index_stride logit logit_stride temperature lse top_logits dx "
                   "dx_stride dw dw_stride N H V K dtype logit_dtype workspace workspace_bytes stream",
}
GOOD = dict(AT, x_stride=H, w_stride=H, dx_stride=H, dw_stride=H, index_stride=K, logit_stride=K, temperature=1.0, N=N,
            H=H, V=V, K=K, dtype=BF16, logit_dtype=F32, workspace_bytes=BIG, stream=None)


def call(which, **kw):
    a = dict(GOOD, **kw)
    return getattr(glu, f"glu_linear_{which}")(*(a[n] for n in ORDER[which].split()))


BAD = [
    (dict(dtype=F32), ENUM), (dict(dtype=7), ENUM), (dict(N=-1), SHAPE), (dict(H=0), SHAPE), (dict(V=0), SHAPE),
    (dict(V=1 << 31), SHAPE), (dict(H=1 << 31), SHAPE), (dict(N=1 << 31), SHAPE),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(lse=None), NULL), (dict(workspace=None), NULL),
    (dict(x_stride=H - 8), STRIDE), (dict(x_stride=H + 4), STRIDE), (dict(w_stride=H + 2), STRIDE),
    (dict(w_stride=-H), STRIDE), (dict(x=AT["x"] + 8), STRIDE), (dict(w=AT["w"] + 2), STRIDE),
    (dict(lse=AT["lse"] + 2), STRIDE), (dict(workspace=AT["workspace"] + 128), STRIDE), (dict(w_stride=1 << 39), STRIDE),
    (dict(workspace=AT["x"]), ALIAS), (dict(workspace=AT["w"] - 256), ALIAS),
    (dict(workspace_bytes=1000), WORKSPACE), (dict(x=(1 << 64) - 4096), SHAPE),
    (dict(workspace_bytes=(1 << 64) - 1), SHAPE),
]
FORWARD = [
    (dict(loss=None), NULL), (dict(loss=AT["loss"] + 1), STRIDE), (dict(loss=AT["lse"] + 400), ALIAS),
    (dict(lse=AT["x"] + 64), ALIAS), (dict(loss=AT["w"] + 64), ALIAS), (dict(lse=AT["workspace"]), ALIAS),
]
BACKWARD = [
    (dict(dloss=None), NULL), (dict(dloss=AT["dloss"] + 2), STRIDE), (dict(dx_stride=H - 1), STRIDE),
    (dict(dw_stride=H - 1), STRIDE), (dict(dx=AT["dx"] + 1), STRIDE), (dict(dw=AT["dw"] + 1), STRIDE),
    (dict(dx=AT["x"]), ALIAS), (dict(dw=AT["w"]), ALIAS), (dict(dx=AT["dw"] + 256), ALIAS), (dict(dw=AT["lse"]), ALIAS),
    (dict(dx=AT["dloss"]), ALIAS), (dict(dw=AT["workspace"] + 512), ALIAS),
]
CE = [(dict(target=None), NULL), (dict(target=AT["target"] + 4), STRIDE)]
CE_FWD = [(dict(loss=AT["target"]), ALIAS), (dict(workspace=AT["target"]), ALIAS)]
CE_BWD = [(dict(loss=None), NULL), (dict(dx=AT["target"]), ALIAS), (dict(dx=AT["loss"]), ALIAS)]
DISTILL = [
    (dict(index=None), NULL), (dict(logit=None), NULL), (dict(top_logits=None), NULL), (dict(K=0), SHAPE),
    (dict(K=1025, index_stride=1025, logit_stride=1025), SHAPE), (dict(logit_dtype=3), ENUM),
    (dict(temperature=0.0), VALUE), (dict(temperature=-1.0), VALUE), (dict(temperature=math.nan), VALUE),
    (dict(temperature=math.inf), VALUE), (dict(temperature=2048.0), VALUE), (dict(temperature=2.0 ** -11), VALUE),
    (dict(index_stride=K - 1), STRIDE), (dict(logit_stride=K - 1), STRIDE), (dict(index=AT["index"] + 4), STRIDE),
    (dict(logit=AT["logit"] + 2), STRIDE), (dict(top_logits=AT["top_logits"] + 2), STRIDE),
    (dict(workspace=AT["index"]), ALIAS), (dict(workspace=AT["logit"]), ALIAS),
]
DISTILL_FWD = [(dict(top_logits=AT["index"]), ALIAS), (dict(top_logits=AT["logit"] + 4), ALIAS),
               (dict(loss=AT["top_logits"]), ALIAS)]
DISTILL_BWD = [(dict(dw=AT["top_logits"]), ALIAS), (dict(dx=AT["index"]), ALIAS)]

CASES = ([("ce_fwd", c) for c in BAD + FORWARD + CE + CE_FWD] + [("ce_bwd", c) for c in BAD + BACKWARD + CE + CE_BWD] +
         [("distill_fwd", c) for c in BAD + FORWARD + DISTILL + DISTILL_FWD] +
         [("distill_bwd", c) for c in BAD + BACKWARD + DISTILL + DISTILL_BWD])


@pytest.mark.parametrize("which,case", CASES, ids=lambda v: v if isinstance(v, str) else ",".join(v[0]) + str(v[1]))
def test_refused(which, case):
    assert call(which, **case[0]) == case[1]


@pytest.mark.parametrize("which", ORDER)
def test_nothing_to_do(which):
    kw = dict.fromkeys(AT, None)
    assert call(which, **kw, N=0) == 0
    if which.endswith("bwd"):
        assert call(which, dx=None, dw=None) == 0


@pytest.mark.parametrize("backward", [0, 1])
def test_workspace_bytes(backward):
    ce, kd = glu.glu_linear_ce_workspace_bytes, glu.glu_linear_distill_workspace_bytes
    for bad in ((0, H, V), (N, 0, V), (N, H, 0), (-1, H, V), (1 << 31, H, V)):
        assert ce(*bad, backward) == 0 and kd(*bad, K, backward) == 0
    assert kd(N, H, V, 0, backward) == 0 and kd(N, H, V, 1025, backward) == 0
    assert 0 < ce(N, H, V, backward) < kd(N, H, V, K, backward)
    # never the logits: at most a piece of 1 GiB, the listed rows and partial gradients
    big = ce(8192, 4096, 1 << 20, backward)
    assert big < (2 << 30) < 8192 * (1 << 20) * 2
    # a forward call keeps 16 bytes a row for each tile of 128 tokens or more
    assert ce(1 << 20, 64, 1 << 17, backward) < (1 << 20) * (1 << 17) * 2 / 15


@pytest.mark.parametrize("which", ["ce_bwd", "distill_bwd"])
def test_less_workspace_is_taken(which):
    """Down to what one piece of 256 tokens needs; one byte less is refused."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    wants = [b for b in range(256, 4 << 20, 256) if call(which, V=50000, workspace_bytes=b) != WORKSPACE]
    full = (glu.glu_linear_ce_workspace_bytes(N, H, 50000, 1) if which == "ce_bwd"
            else glu.glu_linear_distill_workspace_bytes(N, H, 50000, K, 1))
    assert wants and wants[0] < full / 4
    assert call(which, V=50000, workspace_bytes=wants[0] - 1) == WORKSPACE
    assert call(which, V=50000, workspace_bytes=wants[0]) == CUDA


def test_python_refusals():
    import torch
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(9, 8, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        glu.linear_ce(x, w, t)              # not on a GPU
    with pytest.raises(ValueError):
        glu._loss_in(x, w[:, :7])
    with pytest.raises(ValueError):
        glu._loss_in(x, w.half())
    with pytest.raises(ValueError):
        glu._target(t.int(), (4,))
    with pytest.raises(ValueError):
        glu._target(t, (5,))
    with pytest.raises(ValueError):
        glu._target(torch.zeros(8, dtype=torch.int64)[::2], (4,))
    with pytest.raises(ValueError):
        glu._per_row(torch.zeros(4, dtype=torch.float64), (4,), "loss", x)
    with pytest.raises(ValueError):
        glu._teacher(t[:, None], torch.zeros(4, 2), (4,))
    with pytest.raises(ValueError):
        glu._gradient(torch.zeros(4, 8), x, "dx")
    with pytest.raises(ValueError):
        glu._loss_workspace(torch.zeros(4), x, 4, 8, 9, 0, 0)


def test_module_without_a_type():
    """VocabLoss(hidden, vocab) has a type that its calls take."""
    import torch
    from glu_activation_mlps_gb300.autograd import VocabLoss
    assert VocabLoss(16, 9).weight.dtype == torch.bfloat16
    assert VocabLoss(16, 9, dtype=torch.float16).weight.dtype == torch.float16
    before = torch.get_default_dtype()
    try:
        torch.set_default_dtype(torch.float16)
        assert VocabLoss(16, 9).weight.dtype == torch.float16
    finally:
        torch.set_default_dtype(before)
    lin = torch.nn.Linear(16, 9, bias=False)
    assert VocabLoss.from_linear(lin).weight is lin.weight


def test_forward_of_few_rows_has_no_room_for_x():
    """Up to 128 rows nothing is listed, so no copy of x is made room for."""
    for n in (1, 100, 128):
        assert glu.glu_linear_ce_workspace_bytes(n, 65536, 1000, 0) < n * 65536
        assert glu.glu_linear_distill_workspace_bytes(n, 65536, 1000, K, 0) < n * 65536 + 4096
    assert glu.glu_linear_ce_workspace_bytes(129, 65536, 1000, 0) > 2 * 129 * 65536


def test_pieces_of_g():
    """1 GiB of g at most, whatever its parts, or 256 tokens of it where those are more."""
    for n in (1, 63, 64, 65, 4096):
        assert glu.glu_linear_ce_workspace_bytes(n, 64, 1 << 30, 1) < (1 << 30) + (300 << 20)
    n = 1 << 23
    assert 512 * n < glu.glu_linear_ce_workspace_bytes(n, 8, 1 << 20, 1) < 512 * n + n * (128 + 64) + (300 << 20)
