"""Cases that measure the operators of the gated MLP in 8-bit floating point.

A value v of a matrix is held as an e4m3 number q and a float scale shared by a
block of the matrix, v ~ q * scale: 1 x 128 blocks along a row for activations,
128 x 128 blocks for weights, scale = max(amax, 2^-100) / 448 with amax the
block's largest magnitude.  Operators:

  norm     h = x + residual, then rmsnorm(h) * gamma quantised by rows
  quant    a matrix quantised by rows (1 x 128) or by blocks (128 x 128)
  nt       d = a @ b^T of two quantised matrices, d in f16 or bf16
  gated    act(x @ w_gate^T) * (x @ w_up^T) of quantised matrices, quantised by rows
  nt, gated with "experts": the rows of a (x) are sorted by expert, expert e's
           rows offsets[e] .. offsets[e + 1] are multiplied by its own weights,
           and rows behind the last offset are left as they were

``own`` picks the side ``run`` computes: the plain form in elementary torch
operations, or the calls a user makes of this library.
"""
import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
ACTS = ("silu", "gelu_erf", "gelu_tanh", "relu")
FLOOR = 2.0 ** -100


def listed():
    return [
        # a serving step of 8 sequences: launch latency
        {"name": "norm decode", "op": "norm", "dtype": "bf16", "rows": 8, "cols": 4096},
        # one prefill or training batch of 4096 tokens at hidden size 4096: HBM traffic
        {"name": "norm prefill", "op": "norm", "dtype": "bf16", "rows": 4096, "cols": 4096},
        # f32 rows that are no whole number of blocks
        {"name": "norm ragged f32", "op": "norm", "dtype": "f32", "rows": 1000, "cols": 5000},
        # activations that no norm precedes (the MLP's inner rows, by hand)
        {"name": "quant rows", "op": "quant", "dtype": "bf16", "rows": 4096, "cols": 14336, "block": 1},
        # one weight matrix of a checkpoint loaded in 16 bits
        {"name": "quant weights", "op": "quant", "dtype": "bf16", "rows": 14336, "cols": 4096, "block": 128},
        # down projection of a serving step: the weights' bytes
        {"name": "down decode", "op": "nt", "dtype": "bf16", "rows": 16, "k": 14336, "n": 4096, "experts": 0},
        # down projection of a prefill: tensor cores
        {"name": "down prefill", "op": "nt", "dtype": "bf16", "rows": 4096, "k": 14336, "n": 4096, "experts": 0},
        # a projection with no size a multiple of a tile
        {"name": "nt odd f16", "op": "nt", "dtype": "f16", "rows": 333, "k": 2000, "n": 1500, "experts": 0},
        # gate and up projections of one token
        {"name": "gated decode", "op": "gated", "act": "silu", "rows": 1, "k": 4096, "n": 14336, "experts": 0},
        # gate and up projections of a prefill: the largest product
        {"name": "gated prefill", "op": "gated", "act": "silu", "rows": 4096, "k": 4096, "n": 14336, "experts": 0},
        # a serving step of 32 sequences, two experts of eight each
        {"name": "experts decode", "op": "gated", "act": "silu", "rows": 64, "k": 4096, "n": 14336, "experts": 8, "ragged": 1},
        # a prefill over many small experts, with uneven loads
        {"name": "experts prefill", "op": "nt", "dtype": "bf16", "rows": 8192, "k": 2048, "n": 4096, "experts": 32, "ragged": 2},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "nt", "gated", "nt experts", "gated experts"])
    if op == "norm":
        return {"op": "norm", "dtype": rng.choice(["bf16", "f16", "f32"]), "rows": _log(rng, 1, 8192),
                "cols": _log(rng, 64, 16384)}
    if op == "quant":
        return {"op": "quant", "dtype": rng.choice(["bf16", "f16", "f32"]), "rows": _log(rng, 1, 8192),
                "cols": _log(rng, 16, 16384), "block": rng.choice([1, 128])}
    experts = _log(rng, 1, 128) if "experts" in op else 0
    k, n = _log(rng, 128, 16384), _log(rng, 64, 16384)
    # weights of at most a billion values, products of at most the listed largest
    while max(1, experts) * k * n > 2 ** 29:
        k, n = max(128, k // 2), max(64, n // 2)
    rows = _log(rng, 1, 8192)
    while rows * k * n > 4096 * 4096 * 14336:
        rows //= 2
    if op.startswith("nt"):
        case = {"op": "nt", "dtype": rng.choice(["bf16", "f16"]), "rows": rows, "k": k, "n": n, "experts": experts}
    else:
        case = {"op": "gated", "act": rng.choice(ACTS), "rows": rows, "k": k, "n": n, "experts": experts}
    if experts:
        case["ragged"] = rng.randrange(1 << 20)
    return case


def _loads(case):
    """Rows of each expert: uneven, some without any, and a few rows (of a padded batch) behind the last."""
    rng = random.Random(case["ragged"])
    left = case["rows"] - (case["rows"] // 16 if case["ragged"] % 2 else 0)
    weight = [rng.expovariate(1.0) + 0.05 for _ in range(case["experts"])]
    total, cuts, run_ = sum(weight), [0], 0.0
    for w in weight:
        run_ += w
        cuts.append(min(left, int(round(left * run_ / total))))
    return [b - a for a, b in zip(cuts, cuts[1:])]


# ---------------------------------------------------------------- the state

def _split_blocks(v, rows):
    """v (..., M, K) padded with zeros and viewed as (..., M / rows, rows, K / 128, 128)."""
    M, K = v.shape[-2:]
    v = torch.nn.functional.pad(v, (0, -K % 128, 0, -M % rows))
    return v.unflatten(-1, (-1, 128)).unflatten(-3, (-1, rows))


def _quantize(v, rows):
    """float32 v (M, K) as (q, scale), blocks of rows x 128."""
    M, K = v.shape
    b = _split_blocks(v, rows)
    scale = b.abs().amax((1, 3), keepdim=True).clamp_min(FLOOR) / 448
    q = (b / scale).to(FP8).flatten(0, 1).flatten(1, 2)[:M, :K]
    return q, scale[:, 0, :, 0].contiguous()


def _padded(q):
    """q with rows on 16-byte boundaries, as a user lays out an odd width."""
    K = q.shape[-1]
    if K % 16 == 0:
        return q.contiguous()
    out = torch.zeros((*q.shape[:-1], K + -K % 16), dtype=q.dtype, device=q.device)
    out.view(torch.uint8)[..., :K] = q.view(torch.uint8)
    return out[..., :K]


def _activations(g, rows, cols):
    """Normal rows with channels of uneven size, a few far above the rest."""
    ch = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    return torch.randn(rows, cols, generator=g, device="cuda") * ch


def _weights(g, case):
    """One weight matrix (N, K), or (E, N, K), quantised by 128 x 128 blocks."""
    n, k, E = case["n"], case["k"], case["experts"]
    qs, ss = [], []
    for _ in range(max(1, E)):
        q, s = _quantize(torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k), 128)
        qs.append(_padded(q))
        ss.append(s)
    if not E:
        return qs[0], ss[0]
    if k % 16 == 0:
        return torch.stack([q.view(torch.uint8) for q in qs]).view(FP8), torch.stack(ss)
    out = torch.zeros(E, n, k + -k % 16, dtype=FP8, device="cuda")
    for e in range(E):
        out[e, :, :k].view(torch.uint8).copy_(qs[e].view(torch.uint8))
    return out[..., :k], torch.stack(ss)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    if case["op"] == "norm":
        t = TYPES[case["dtype"]]
        st["x"] = torch.randn(case["rows"], case["cols"], generator=g, device="cuda").to(t)
        st["res"] = _activations(g, case["rows"], case["cols"]).to(t)
        st["gamma"] = (1 + 0.2 * torch.randn(case["cols"], generator=g, device="cuda")).to(t)
        st["eps"] = 1e-5
        return st
    if case["op"] == "quant":
        st["x"] = _activations(g, case["rows"], case["cols"]).to(TYPES[case["dtype"]])
        return st
    q, s = _quantize(_activations(g, case["rows"], case["k"]), 1)
    st["a"], st["a_scale"] = _padded(q), s
    st["w"] = [_weights(g, case) for _ in range(2 if case["op"] == "gated" else 1)]
    st["offsets"] = None
    if case["experts"]:
        loads = _loads(case)
        cuts = [0]
        for v in loads:
            cuts.append(cuts[-1] + v)
        st["offsets"] = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        st["most"] = max(1, max(loads))
        R, n = case["rows"], case["n"]
        if case["op"] == "nt":
            st["out"] = torch.zeros(R, n, dtype=TYPES[case["dtype"]], device="cuda")
        else:
            st["out"] = torch.zeros(R, n, dtype=FP8, device="cuda")
            st["out_scale"] = torch.zeros(R, -(-n // 128), device="cuda")
    return st


# ---------------------------------------------------------------- the plain forms

def _act(name, g):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    if name == "gelu_erf":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    return g.clamp_min(0)


def _values(q, scale, rows):
    """The float32 values of a quantised matrix (..., M, K)."""
    M, K = q.shape[-2:]
    s = scale.repeat_interleave(rows, -2)[..., :M, :] if rows > 1 else scale
    return q.to(torch.float32) * s.repeat_interleave(128, -1)[..., :K]


def _product(st, a, w):
    """a @ w^T in float32, rows by expert where there are experts."""
    q, s = w
    if st["offsets"] is None:
        return a @ _values(q, s, 128).mT
    # each expert's rows side by side in a padded batch
    off, R = st["offsets"].to(torch.int64), a.shape[0]
    at = off[:-1, None] + torch.arange(st["most"], device=a.device)
    here = at < off[1:, None]
    d = a[at.clamp_max(R - 1)] @ _values(q, s, 128).mT
    out = torch.zeros(R, d.shape[-1], device=a.device)
    out[at[here]] = d[here]
    return out


def _plain(st):
    if st["op"] == "norm":
        s = st["x"].float() + st["res"].float()
        y = s * (1 / torch.sqrt((s * s).mean(-1, keepdim=True) + st["eps"])) * st["gamma"].float()
        return (s.to(st["x"].dtype), *_quantize(y, 1))
    if st["op"] == "quant":
        return _quantize(st["x"].float(), st["block"])
    a = _values(st["a"], st["a_scale"], 1)
    if st["op"] == "nt":
        return _product(st, a, st["w"][0]).to(TYPES[st["dtype"]])
    q, s = _quantize(_act(st["act"], _product(st, a, st["w"][0])) * _product(st, a, st["w"][1]), 1)
    if st["offsets"] is not None:
        s = torch.where((torch.arange(len(s), device=s.device) < st["offsets"][-1])[:, None], s, 0.0)
    return q, s


def run(state):
    if not own:
        return _plain(state)
    import glu_activation_mlps_gb300 as glu
    st = state
    if st["op"] == "norm":
        return glu.add_rmsnorm_q(st["x"], st["res"], st["gamma"], st["eps"])
    if st["op"] == "quant":
        return glu.quantize(st["x"], block_rows=st["block"])
    if st["op"] == "nt":
        return glu.gemm_q_nt(st["a"], st["a_scale"], *st["w"][0], offsets=st["offsets"], d=st.get("out"),
                             dtype=TYPES[st["dtype"]])
    return glu.gemm_q_fwd(st["a"], st["a_scale"], *st["w"][0], *st["w"][1], act=st["act"], offsets=st["offsets"],
                          y=st.get("out"), y_scale=st.get("out_scale"))


# ---------------------------------------------------------------- work and the 64-bit values

def work(case):
    rows = case["rows"]
    if case["op"] == "norm":
        n, E = rows * case["cols"], BYTES[case["dtype"]]
        return {"bytes": n * (3 * E + 1) + case["cols"] * E + 4 * rows * -(-case["cols"] // 128), "flops": 8 * n}
    if case["op"] == "quant":
        n = rows * case["cols"]
        blocks = -(-rows // case["block"]) * -(-case["cols"] // 128)
        return {"bytes": n * (BYTES[case["dtype"]] + 1) + 4 * blocks, "flops": 3 * n}
    k, n = case["k"], case["n"]
    used, mats = 1, 2 if case["op"] == "gated" else 1
    if case["experts"]:
        loads = _loads(case)
        used, rows = sum(v > 0 for v in loads), sum(loads)
    weights = used * mats * (n * k + 4 * -(-n // 128) * -(-k // 128))
    out = rows * (2 * n if case["op"] == "nt" else n + 4 * -(-n // 128))
    return {"bytes": rows * (k + 4 * -(-k // 128)) + weights + out + 4 * case["experts"],
            "flops": 2.0 * mats * rows * n * k}


def _e4m3(v):
    """float64 v (magnitudes up to 448) rounded to the nearest e4m3 value, ties to even: 4 significant bits, quantum at least 2^-9."""
    quantum = torch.ldexp(torch.ones_like(v), torch.frexp(v)[1].clamp_min(-5) - 4)
    return (torch.round(v / quantum) * quantum).clamp(-448, 448)


def _q64(y, rows):
    """Quantised y in float64: block by block along the columns."""
    M, K = y.shape
    q, s = torch.empty_like(y), torch.empty(-(-M // rows), -(-K // 128), dtype=torch.float64, device=y.device)
    group = torch.arange(M, device=y.device) // rows
    for j in range(s.shape[1]):
        part = y[:, 128 * j:128 * j + 128]
        top = torch.zeros(s.shape[0], dtype=torch.float64, device=y.device)
        top = top.scatter_reduce(0, group, part.abs().amax(1), "amax")
        s[:, j] = torch.maximum(top, torch.full_like(top, FLOOR)) / 448
        q[:, 128 * j:128 * j + 128] = _e4m3(part / s[group, j][:, None])
    return q, s


def _w64(q, s):
    v = q.double()
    for j in range(s.shape[1]):
        v[:, 128 * j:128 * j + 128] *= torch.repeat_interleave(s[:, j].double(), 128)[: v.shape[0], None]
    return v


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        s = st["x"].double() + st["res"].double()
        rms = torch.sqrt(torch.sum(s ** 2, 1, keepdim=True) / s.shape[1] + st["eps"])
        return (s, *_q64(s / rms * st["gamma"].double(), 1))
    if case["op"] == "quant":
        return _q64(st["x"].double(), st["block"])
    a = st["a"].double()
    for j in range(st["a_scale"].shape[1]):
        a[:, 128 * j:128 * j + 128] *= st["a_scale"][:, j:j + 1].double()
    cuts = [0, case["rows"]] if not case["experts"] else st["offsets"].tolist()
    prods = [torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda") for _ in st["w"]]
    for p, (q, s) in zip(prods, st["w"]):
        for e, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
            if hi > lo:
                p[lo:hi] = a[lo:hi] @ (_w64(q[e], s[e]) if case["experts"] else _w64(q, s)).mT
    if case["op"] == "nt":
        return prods[0]
    g, u = prods
    act = {"silu": lambda: g * torch.special.expit(g),
           "gelu_erf": lambda: g * torch.special.ndtr(g),
           "gelu_tanh": lambda: g * torch.special.expit(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)),
           "relu": lambda: torch.where(g > 0, g, 0.0)}[case["act"]]()
    q, s = _q64(act * u, 1)
    s[cuts[-1]:] = 0
    return q, s
