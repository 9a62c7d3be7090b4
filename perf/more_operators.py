"""Cases that measure the losses over a vocabulary, taken straight from hidden rows.

x (N, H) are the rows behind the last norm, w (V, H) the output projection, and
z = x @ w^T the logits, which are not kept.  Operators:

  ce       loss[n] = lse[n] - z[n, target[n]],   lse[n] = log sum_v exp z[n, v]
  distill  a teacher's top logits t[n, k] at index[n, k], p = softmax over k of t / T:
           loss[n] = sum_k p[n, k] (log p[n, k] - log q[n, index[n, k]]),
           q[n] = softmax over the whole vocabulary of z[n] / T

A row whose target (whose every index) lies outside 0 .. V - 1 takes no part: its
loss, its lse and its gradients are 0.  "step" cases run the forward and the
backward pass, dloss[n] the gradient that arrives at loss[n]:

  dz[n, v] = dloss[n] (exp(z[n, v] - lse[n]) - [v = target[n]])
  dx = dz @ w,   dw = dz^T @ x          (distill: softmax at T, p in place of 1, / T)

``own`` picks the side ``run`` computes: the plain form in elementary torch
operations, or the calls a user makes of this library.
"""
import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one token's loss on a small model: launch latency
        {"name": "score one", "op": "ce", "step": False, "dtype": "f16", "rows": 1, "hidden": 1024, "vocab": 8192},
        # a serving step that scores one token of 8 sequences: the projection's bytes
        {"name": "score decode", "op": "ce", "step": False, "dtype": "bf16", "rows": 8, "hidden": 4096, "vocab": 32768},
        # no size a multiple of a tile, rows padded to 16 bytes, prompt tokens without a target
        {"name": "score odd", "op": "ce", "step": False, "dtype": "f16", "rows": 333, "hidden": 1999, "vocab": 50001,
         "masked": 0.2},
        # perplexity of one batch over a large vocabulary: tensor cores
        {"name": "perplexity", "op": "ce", "step": False, "dtype": "bf16", "rows": 4096, "hidden": 4096,
         "vocab": 131072},
        # a training step of few tokens: the projection is read, its gradient written
        {"name": "train few", "op": "ce", "step": True, "dtype": "bf16", "rows": 64, "hidden": 4096, "vocab": 32768},
        # a training step with odd sizes, gradients scaled for half precision
        {"name": "train odd", "op": "ce", "step": True, "dtype": "f16", "rows": 777, "hidden": 1030, "vocab": 30001,
         "masked": 0.1},
        # fine-tuning on answers: most of the batch is prompt, without a target
        {"name": "train masked", "op": "ce", "step": True, "dtype": "bf16", "rows": 8192, "hidden": 2048,
         "vocab": 65536, "masked": 0.6},
        # one training batch over a large vocabulary: the largest
        {"name": "train", "op": "ce", "step": True, "dtype": "bf16", "rows": 4096, "hidden": 4096, "vocab": 131072},
        # distillation of a small model, few tokens
        {"name": "distill few", "op": "distill", "step": True, "dtype": "bf16", "rows": 16, "hidden": 1024,
         "vocab": 8192, "top": 8, "temperature": 1.0},
        # how far a student is from its teacher on held-out text
        {"name": "distill eval", "op": "distill", "step": False, "dtype": "bf16", "rows": 1024, "hidden": 4096,
         "vocab": 32768, "top": 32, "temperature": 1.0},
        # rows of uneven numbers of entries (a teacher cut at a probability), padding rows
        {"name": "distill ragged", "op": "distill", "step": True, "dtype": "f16", "rows": 1500, "hidden": 1536,
         "vocab": 50001, "top": 100, "temperature": 1.5, "masked": 0.2, "ragged": True},
        # a batch of distillation over a large vocabulary
        {"name": "distill train", "op": "distill", "step": True, "dtype": "bf16", "rows": 4096, "hidden": 2048,
         "vocab": 131072, "top": 64, "temperature": 2.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = {"op": rng.choice(["ce", "distill"]), "step": rng.random() < 0.6, "dtype": rng.choice(["bf16", "f16"]),
            "rows": _log(rng, 1, 8192), "hidden": _log(rng, 64, 8192), "vocab": _log(rng, 1000, 160000),
            "masked": rng.choice([0.0, 0.1, 0.6])}
    if rng.random() < 0.5:          # half of the models have widths that are multiples of 64
        case["hidden"] = -(-case["hidden"] // 64) * 64
    while case["rows"] * case["hidden"] * case["vocab"] > 4096 * 4096 * 131072:
        case["rows"] //= 2
    if case["op"] == "distill":
        case.update(top=_log(rng, 1, 256), temperature=rng.choice([1.0, 1.5, 2.0, 4.0]), ragged=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------- the state

def _valid_rows(case):
    """Which rows take part: runs without a target at the head of every sequence of up to 512 rows."""
    n, masked = case["rows"], case.get("masked", 0.0)
    return [i % 512 >= int(masked * min(512, n - i // 512 * 512)) for i in range(n)]


def _matrix(v, dtype):
    """v in its type, rows on 16-byte boundaries as a user lays out an odd width."""
    H = v.shape[1]
    if H % 8 == 0:
        return v.to(dtype)
    out = torch.zeros(v.shape[0], H + -H % 8, dtype=dtype, device=v.device)
    out[:, :H] = v
    return out[:, :H]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    N, H, V, t = case["rows"], case["hidden"], case["vocab"], TYPES[case["dtype"]]
    w = torch.randn(V, H, generator=g, device="cuda") * (2.5 / math.sqrt(H))
    x = torch.randn(N, H, generator=g, device="cuda")
    valid = torch.tensor(_valid_rows(case), device="cuda")
    if case["op"] == "ce":
        target = torch.randint(0, V, (N,), generator=g, device="cuda")
        # the model expects some targets more than others
        x = x + 2 * torch.rand(N, 1, generator=g, device="cuda") * w[target]
        st["target"] = torch.where(valid, target, -100)
    else:
        K, T = min(case["top"], V), case["temperature"]
        # K different tokens a row, the teacher's logits in descending order
        step = torch.randint(1, max(2, V // K + 1), (N, K), generator=g, device="cuda")
        index = (torch.randint(0, V, (N, 1), generator=g, device="cuda") + step.cumsum(1)) % V
        index = index[:, torch.randperm(K, generator=g, device="cuda")]
        logit = 12 - torch.rand(N, K, generator=g, device="cuda").mul_(12 / K).cumsum(1)
        x = x + torch.rand(N, 1, generator=g, device="cuda") * w[index[:, 0]]
        keep = torch.ones(N, K, dtype=torch.bool, device="cuda")
        if case.get("ragged"):
            keep = torch.arange(K, device="cuda") < torch.randint(1, K + 1, (N, 1), generator=g, device="cuda")
        st["index"] = torch.where(keep & valid[:, None], index, -1)
        st["logit"] = logit
    st["x"], st["w"] = _matrix(x, t), _matrix(w, t)
    if case["step"]:
        # the mean over the rows that take part, scaled for half precision
        scale = (1024.0 if case["dtype"] == "f16" else 1.0) / max(1, sum(_valid_rows(case)))
        st["dloss"] = torch.full((N,), scale, device="cuda")
    return st


# ---------------------------------------------------------------- the plain forms

def _softmax_sums(z):
    top = z.amax(1)
    return top + torch.log(torch.exp(z - top[:, None]).sum(1))


def _plain(st):
    x, w, V = st["x"].float(), st["w"].float(), st["vocab"]
    z = x @ w.T
    if st["op"] == "ce":
        valid = (st["target"] >= 0) & (st["target"] < V)
        at = torch.where(valid, st["target"], 0)[:, None]
        share, T = valid.float()[:, None], 1.0
        lse = torch.where(valid, _softmax_sums(z), 0.0)
        out = [torch.where(valid, lse - z.gather(1, at)[:, 0], 0.0), lse]
    else:
        T = st["temperature"]
        here = (st["index"] >= 0) & (st["index"] < V)
        valid = here.any(1)
        at = torch.where(here, st["index"], 0)
        t = torch.where(here, st["logit"] / T, -math.inf)
        t = t - torch.where(valid, t.amax(1), 0.0)[:, None]
        e = torch.where(here, torch.exp(t), 0.0)
        total = torch.where(valid, e.sum(1), 1.0)[:, None]
        share = e / total
        top = torch.where(here, z.gather(1, at), 0.0)
        z = z / T
        lse = torch.where(valid, _softmax_sums(z), 0.0)
        log_p = torch.where(here, t - torch.log(total), 0.0)
        out = [torch.where(valid, (share * (log_p - top / T + lse[:, None])).sum(1), 0.0), lse, top]
    if not st["step"]:
        return tuple(out)
    d = torch.where(valid, st["dloss"] / T, 0.0)[:, None]
    dz = z.sub_(lse[:, None]).exp_().mul_(d)
    dz.scatter_add_(1, at, -d * share)
    return out[0], (dz @ w).to(st["x"].dtype), (dz.T @ x).to(st["w"].dtype)


def run(state):
    if not own:
        return _plain(state)
    import glu_activation_mlps_gb300 as glu
    st = state
    if st["op"] == "ce":
        loss, lse = glu.linear_ce(st["x"], st["w"], st["target"])
        if not st["step"]:
            return loss, lse
        return (loss, *glu.linear_ce_bwd(st["dloss"], st["x"], st["w"], st["target"], loss, lse))
    loss, lse, top = glu.linear_distill(st["x"], st["w"], st["index"], st["logit"], st["temperature"])
    if not st["step"]:
        return loss, lse, top
    return (loss, *glu.linear_distill_bwd(st["dloss"], st["x"], st["w"], st["index"], st["logit"], lse, top,
                                          st["temperature"]))


# ---------------------------------------------------------------- work and the 64-bit values

def work(case):
    """The logits' product, and in a step those of the two gradients, over the rows that take part; every matrix once."""
    N, H, V = case["rows"], case["hidden"], case["vocab"]
    n = sum(_valid_rows(case))
    entries = case["op"] == "distill" and N * min(case["top"], V)
    small = 4 * n * 2 + (12 * entries if entries else 8 * N)
    if case["step"]:
        return {"bytes": 2 * (n * H + 2 * V * H + N * H) + small + 4 * N, "flops": 6.0 * n * H * V}
    return {"bytes": 2 * (n * H + V * H) + small + (4 * entries if entries else 0), "flops": 2.0 * n * H * V}


def exact(case, seed):
    N, H, V = case["rows"], case["hidden"], case["vocab"]
    if (3 if case["step"] else 1) * 2.0 * N * H * V > 1.5e13:
        return None
    st = prepare(case, seed)
    T = case.get("temperature", 1.0)
    w = st["w"].double()
    loss, lse = (torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(2))
    top = None if case["op"] == "ce" else torch.zeros(st["index"].shape, dtype=torch.float64, device="cuda")
    dx = torch.zeros(N, H, dtype=torch.float64, device="cuda")
    dw = torch.zeros(V, H, dtype=torch.float64, device="cuda")
    for lo in range(0, N, 1024):
        part = slice(lo, min(N, lo + 1024))
        x = st["x"][part].double()
        z = torch.matmul(x, w.t())
        # the weights of the formula, one dense row each: 1 at the target, or the teacher's shares
        p = torch.zeros_like(z)
        if case["op"] == "ce":
            t = st["target"][part]
            takes = (t >= 0) & (t < V)
            rows = takes.nonzero()[:, 0]
            p[rows, t[rows]] = 1.0
            entropy = torch.zeros(len(t), dtype=torch.float64, device="cuda")
        else:
            idx = st["index"][part]
            has = (idx >= 0) & (idx < V)
            takes = has.any(1)
            logit = st["logit"][part].double().masked_fill(~has, -math.inf)
            logit[~takes] = 0.0
            q = torch.softmax(logit / T, 1) * takes[:, None]
            entropy = torch.special.entr(q).sum(1)
            r, k = has.nonzero(as_tuple=True)
            p.index_put_((r, idx[r, k]), q[r, k], accumulate=True)
            top[part][r, k] = z[r, idx[r, k]]
        log_q = torch.log_softmax(z / T, 1)
        mine = -(p * log_q).sum(1) - entropy
        loss[part] = mine.masked_fill(~takes, 0.0)
        lse[part] = torch.logsumexp(z / T, 1).masked_fill(~takes, 0.0)
        if case["step"]:
            d = st["dloss"][part].double() * takes / T
            dz = (torch.exp(log_q) - p) * d[:, None]
            dx[part] = torch.matmul(dz, w)
            dw += torch.matmul(dz.t(), x)
    if case["step"]:
        return loss, dx, dw
    return (loss, lse) if case["op"] == "ce" else (loss, lse, top)
