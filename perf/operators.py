"""Cases of the serving-head operators: what they are fed, what they return and what they cost.

Three operators, in the order a decode step runs them:

  quantize_rows    RMS norm and symmetric 8-bit quantisation of hidden states, one scale per token
  linear_i8        the vocabulary projection in 8-bit integers, scaled by token and channel
  sample_filtered  temperature, top-k, top-p and min-p sampling from given uniform numbers

Case kinds: "sample" (sample_filtered on given logits), "linear" (linear_i8 on given integers) and "head"
(quantize_rows, then linear_i8, as Int8Head.logits runs them). `run` computes a case with elementary torch
operations, or with the package's kernels when `own` is set.
"""
import math

import torch

own = False

DEV = "cuda"
FLT_MAX = 3.4028234663852886e38
ONE = 2.0 ** 31  # weight of a row's largest logit in the integer weights of sample_filtered
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # One request of a small-codebook model (1024 codes and a mask token): latency is the call.
        {"name": "sample one row 1025", "kind": "sample", "n": 1, "V": 1025, "dtype": "bf16", "mode": "mixed"},
        # A diffusion canvas of that model, every position drawn in one call.
        {"name": "sample canvas 15510x1025", "kind": "sample", "n": 15510, "V": 1025, "dtype": "bf16", "mode": "mixed"},
        # A ragged batch over an odd vocabulary with fp32 logits; rows with masked tokens and each kind of filter.
        {"name": "sample 37x70001 f32", "kind": "sample", "n": 37, "V": 70001, "dtype": "f32", "mode": "mixed"},
        # Single-stream decoding over a large vocabulary, nucleus sampling.
        {"name": "sample one row 248320", "kind": "sample", "n": 1, "V": 248320, "dtype": "bf16", "mode": "top_p"},
        # A large serving batch over the large vocabulary: nucleus sampling alone needs the whole row's mass.
        {"name": "sample 256x248320 top-p", "kind": "sample", "n": 256, "V": 248320, "dtype": "bf16", "mode": "top_p"},
        # The same batch with requests of every kind side by side.
        {"name": "sample 256x248320 mixed", "kind": "sample", "n": 256, "V": 248320, "dtype": "bf16", "mode": "mixed"},
        # One token through eight 1025-way output heads stacked into one weight: the smallest projection.
        {"name": "head 1 token 8200x1024", "kind": "head", "n": 1, "N": 8200, "K": 1024, "dtype": "bf16"},
        # A decode batch through the large vocabulary projection: the weight's bytes are the call.
        {"name": "head 24 x 248320x2048", "kind": "head", "n": 24, "N": 248320, "K": 2048, "dtype": "bf16"},
        # The largest serving batch through the large vocabulary projection.
        {"name": "head 256 x 248320x2048", "kind": "head", "n": 256, "N": 248320, "K": 2048, "dtype": "bf16"},
        # The product alone, fp32 logits, sizes that divide nothing.
        {"name": "linear 5 x 70001x1000 f32", "kind": "linear", "n": 5, "N": 70001, "K": 1000, "dtype": "f32"},
        # Every position of a canvas through the eight stacked heads.
        {"name": "linear 1939 x 8200x1024", "kind": "linear", "n": 1939, "N": 8200, "K": 1024, "dtype": "bf16"},
        # A long prefill scored through an odd-sized vocabulary.
        {"name": "linear 777 x 20011x4096", "kind": "linear", "n": 777, "N": 20011, "K": 4096, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["sample", "sample", "linear", "head"])
    if kind == "sample":
        V = _log_int(rng, 33, 248320)
        n = _log_int(rng, 1, max(1, min(16384, 15_000_000 // V)))
        return {"kind": kind, "n": n, "V": V, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "mode": rng.choice(["mixed", "mixed", "top_p", "top_k", "free"])}
    K = _log_int(rng, 64, 4096)
    if rng.random() < 0.5:
        K = max(64, K // 64 * 64)
    N = _log_int(rng, 64, min(248320, 500_000_000 // K))
    n = _log_int(rng, 1, max(1, min(4096, 120_000_000_000 // (N * K), 60_000_000 // N)))
    return {"kind": kind, "n": n, "N": N, "K": K, "dtype": "bf16" if kind == "head" else rng.choice(["bf16", "f32"])}


# ------------------------------------------------------------------ inputs
def _pick(values, n, g):
    v = torch.tensor(values, device=DEV)
    return v[torch.randint(0, len(values), (n,), generator=g, device=DEV)]


def _sample_inputs(case, g):
    n, V, mode = case["n"], case["V"], case["mode"]
    x = torch.randn((n, V), generator=g, device=DEV)
    x *= 3.0 if V < 4096 else 4.0
    if mode == "mixed":
        tau = _pick([0.0, 0.5, 0.7, 0.9, 1.0, 1.0, 1.1, 1.3], n, g)
        k = _pick([0, 0, 0, 1, 20, 50, 50, 200], n, g).to(torch.int32)
        p = _pick([1.0, 1.0, 0.95, 0.9, 0.8, 0.5], n, g)
        mp = _pick([0.0, 0.0, 0.0, 0.02, 0.05, 0.1], n, g)
        # a quarter of the rows come from a constrained grammar: half of their tokens are masked, with -inf or
        # with the type's lowest value; of 16 rows and more, one row has nothing left
        masked = torch.nonzero(torch.rand((n,), generator=g, device=DEV) < 0.25).reshape(-1)
        for half, low in ((masked[0::2], -math.inf), (masked[1::2], float(torch.finfo(DTYPES[case["dtype"]]).min))):
            if half.numel():
                cut = torch.rand((half.numel(), V), generator=g, device=DEV) < 0.5
                x[half] = torch.where(cut, torch.full_like(cut, low, dtype=torch.float32), x[half])
        if n >= 16:
            x[n // 2] = -math.inf
    else:
        tau = torch.full((n,), {"top_p": 0.8, "top_k": 1.0, "free": 1.0}[mode], device=DEV)
        k = torch.full((n,), 50 if mode == "top_k" else 0, device=DEV, dtype=torch.int32)
        p = torch.full((n,), 0.9 if mode == "top_p" else 1.0, device=DEV)
        mp = torch.zeros((n,), device=DEV)
    u = torch.rand((n,), generator=g, device=DEV)
    return {"x": x.to(DTYPES[case["dtype"]]), "tau": tau, "k": k, "p": p, "mp": mp, "u": u}


def _ints(shape, sigma, g):
    """Normal integers in [-127, 127], made a slab of rows at a time."""
    out = torch.empty(shape, dtype=torch.int8, device=DEV)
    rows = max(1, (1 << 27) // shape[1])
    for i in range(0, shape[0], rows):
        part = out[i:i + rows]
        z = torch.randn(part.shape, generator=g, device=DEV)
        part.copy_(z.mul_(sigma).round_().clamp_(-127, 127))
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": dict(case)}
    if case["kind"] == "sample":
        s.update(_sample_inputs(case, g))
        return s
    n, N, K = case["n"], case["N"], case["K"]
    s["w"] = _ints((N, K), 32.0, g)
    s["sw"] = (0.75 + 0.5 * torch.rand((N,), generator=g, device=DEV)) * (4.0 / (32.0 * math.sqrt(K)))
    if case["kind"] == "head":
        s["h"] = (torch.randn((n, K), generator=g, device=DEV) * 1.7).to(torch.bfloat16)
        s["gain"] = 1.0 + 0.1 * torch.randn((K,), generator=g, device=DEV)
    else:
        s["a"] = _ints((n, K), 36.0, g)
        s["sa"] = (0.75 + 0.5 * torch.rand((n,), generator=g, device=DEV)) / 36.0
    if own:
        import vocab_wide_logit_gb300 as ds
        # a serving program lays its weights out once, when it loads them
        if case["kind"] == "head":
            s["plan"] = ds.Int8Head(s["w"], s["sw"], gain=s["gain"], eps=EPS)
        else:
            s["plan"] = ds.pack_i8(s["w"], s["sw"])
    return s


# ------------------------------------------------------------------ one pass
def _plain_sample(s):
    x = s["x"].float()
    n, V = x.shape
    m = x.amax(dim=1, keepdim=True)
    total = (x - m).exp().sum(dim=1, keepdim=True)
    lse = m + total.log()
    val, idx = torch.sort(x, dim=1, descending=True, stable=True)
    tau = s["tau"][:, None]
    greedy = tau == 0
    r = torch.where(greedy, torch.ones_like(tau), (1.0 / tau).clamp(max=FLT_MAX))
    w = torch.round(((val - m) * r).exp() * ONE)
    w = torch.where(torch.isnan(w), torch.zeros_like(w), w).to(torch.int64)
    k = s["k"][:, None]
    rank = torch.arange(V, device=x.device)[None, :]
    w = torch.where((k <= 0) | (rank < k), w, torch.zeros_like(w))
    cum = w.cumsum(dim=1)
    keep = (cum - w).double() < s["p"][:, None].double() * cum[:, -1:].double()
    keep &= w.double() >= s["mp"][:, None].double() * ONE
    w = torch.where(keep, w, torch.zeros_like(w))
    cum = w.cumsum(dim=1)
    t = (s["u"][:, None].double() * cum[:, -1:].double()).floor().to(torch.int64)
    at = (cum <= t).sum(dim=1, keepdim=True).clamp(max=V - 1)
    at = torch.where(greedy, torch.zeros_like(at), at)
    tokens = idx.gather(1, at)
    logprobs = val.gather(1, at) - lse
    none = ~torch.isfinite(total)
    tokens = torch.where(none, torch.full_like(tokens, -1), tokens)
    return {"tokens": tokens[:, 0].to(torch.int32), "logprobs": logprobs[:, 0]}


def _plain_linear(a, sa, w, sw, dtype):
    acc = a.float() @ w.float().t()
    return ((acc * sa[:, None]) * sw[None, :]).to(dtype)


def _plain_quantize(h, gain):
    x = h.float()
    y = x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS) * gain[None, :]
    amax = y.abs().amax(dim=1, keepdim=True)
    return torch.round(y * (127.0 / amax)), (amax / 127.0)[:, 0]


def run(state):
    case = state["case"]
    if case["kind"] == "sample":
        if own:
            import vocab_wide_logit_gb300 as ds
            tokens, logprobs = ds.sample_filtered(state["x"], state["tau"], state["u"], top_k=state["k"],
                                                  top_p=state["p"], min_p=state["mp"])
            return {"tokens": tokens, "logprobs": logprobs}
        return _plain_sample(state)
    dtype = DTYPES[case["dtype"]]
    if case["kind"] == "head":
        if own:
            return {"logits": state["plan"].logits(state["h"], dtype=dtype)}
        q, sa = _plain_quantize(state["h"], state["gain"])
        return {"logits": _plain_linear(q, sa, state["w"], state["sw"], dtype)}
    if own:
        import vocab_wide_logit_gb300 as ds
        return {"logits": ds.linear_i8(state["a"], state["sa"], state["plan"], dtype=dtype)}
    return {"logits": _plain_linear(state["a"], state["sa"], state["w"], state["sw"], dtype)}


def work(case):
    n = case["n"]
    if case["kind"] == "sample":
        V = case["V"]
        # the logits once, five parameters and two results a row; a subtraction, a product, an exponential and
        # a sum for each logit, twice (the row's log-sum-exp and its tempered weights)
        return {"bytes": n * V * (2 if case["dtype"] == "bf16" else 4) + 28 * n, "flops": 8 * n * V}
    N, K = case["N"], case["K"]
    out = n * N * (2 if case["dtype"] == "bf16" else 4)
    left = 2 * n * K + 4 * K if case["kind"] == "head" else n * K + 4 * n
    return {"bytes": N * K + 4 * N + left + out, "flops": 2 * n * N * K}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_sample(s):
    tokens, logprobs = [], []
    rows = max(1, (1 << 25) // s["x"].shape[1])
    for i in range(0, s["x"].shape[0], rows):
        x = s["x"][i:i + rows].double()
        tau, k, p, mp, u = (s[q][i:i + rows].double()[:, None] for q in ("tau", "k", "p", "mp", "u"))
        m = x.max(dim=1, keepdim=True).values
        lse = torch.logsumexp(x, dim=1, keepdim=True)
        val, idx = torch.sort(x, dim=1, descending=True, stable=True)
        prob = ((val - m) / torch.where(tau == 0, torch.ones_like(tau), tau)).exp()
        prob = torch.nan_to_num(prob, nan=0.0)
        rank = torch.arange(x.shape[1], device=x.device, dtype=torch.float64)[None, :]
        prob = prob * ((k <= 0) | (rank < k))
        before = prob.cumsum(dim=1) - prob
        keep = (before < p * prob.sum(dim=1, keepdim=True) * (1 - 1e-15)) | (rank == 0)
        keep = keep & (prob >= mp)
        run_ = (prob * keep).cumsum(dim=1)
        at = torch.searchsorted(run_, u * run_[:, -1:], right=True).clamp(max=x.shape[1] - 1)
        at = torch.where(tau == 0, torch.zeros_like(at), at)
        none = ~torch.isfinite(m)
        tokens.append(torch.where(none, torch.full_like(at, -1), idx.gather(1, at))[:, 0].to(torch.int32))
        lp = val.gather(1, at) - lse
        logprobs.append(torch.where(none, torch.full_like(lp, math.nan), lp)[:, 0])
    return {"tokens": torch.cat(tokens), "logprobs": torch.cat(logprobs)}


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    if case["kind"] == "sample":
        return _exact_sample(s)
    if case["kind"] == "head":
        x = s["h"].double()
        y = x / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS) * s["gain"].double()[None, :]
        scale = y.abs().amax(dim=1, keepdim=True) / 127
        a, sa = torch.round(y / scale), scale
    else:
        a, sa = s["a"].double(), s["sa"].double()[:, None]
    w, sw = s["w"], s["sw"].double()
    n, N = a.shape[0], w.shape[0]
    if float(n) * N * a.shape[1] > 2e11:
        return None
    out = torch.empty((n, N), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 28) // max(n, a.shape[1]))
    for j in range(0, N, step):
        out[:, j:j + step] = (a @ w[j:j + step].double().t()) * sa * sw[None, j:j + step]
    return {"logits": out}
