"""Cases of what stands around the sampler of the serving head: what they are fed, what they return and what they cost.

Three operators:

  score_tokens       log-probabilities of given tokens with the row's log-sum-exp and entropy, the token's rank and
                     the most likely alternatives
  score_tokens_grad  the gradient of log-probabilities and entropies with respect to the logits
  add_adapters       a low-rank adapter of each request's own, added to the logits of the shared projection

Case kinds: "score", "grad" and "adapters", one for each. `run` computes a case with elementary torch operations, or
with the package's kernels when `own` is set.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # One token of a small-codebook model (1024 codes and a mask token) with five alternatives: latency is the call.
        {"name": "score one row 1025", "kind": "score", "n": 1, "V": 1025, "dtype": "bf16", "top": 5},
        # A diffusion canvas of that model, every position's token scored in one call.
        {"name": "score canvas 15510x1025", "kind": "score", "n": 15510, "V": 1025, "dtype": "bf16", "top": 8},
        # A ragged batch over an odd vocabulary with fp32 logits, masked rows among them, the usual twenty alternatives.
        {"name": "score 37x70001 f32", "kind": "score", "n": 37, "V": 70001, "dtype": "f32", "top": 20},
        # A prompt's logprobs, or a large decode batch, over the large vocabulary.
        {"name": "score 256x248320", "kind": "score", "n": 256, "V": 248320, "dtype": "bf16", "top": 20},
        # Tuning a small-codebook model on a few positions.
        {"name": "grad 24x1025", "kind": "grad", "n": 24, "V": 1025, "dtype": "bf16", "entropy": True},
        # fp32 logits of an odd vocabulary, with an entropy bonus.
        {"name": "grad 300x70001 f32", "kind": "grad", "n": 300, "V": 70001, "dtype": "f32", "entropy": True},
        # A batch of positions over the large vocabulary, log-probabilities alone (a likelihood loss).
        {"name": "grad 256x248320", "kind": "grad", "n": 256, "V": 248320, "dtype": "bf16", "entropy": False},
        # One request with an adapter on eight 1025-way output heads stacked into one weight: the smallest call.
        {"name": "adapters 1 token 8200x1024", "kind": "adapters", "n": 1, "N": 8200, "K": 1024, "R": 16, "L": 4,
         "dtype": "bf16", "norm": True, "order": "mixed"},
        # A decode batch over the large vocabulary, eight adapters in any order.
        {"name": "adapters 24 x 248320x2048", "kind": "adapters", "n": 24, "N": 248320, "K": 2048, "R": 16, "L": 8,
         "dtype": "bf16", "norm": True, "order": "mixed"},
        # A large decode batch with many adapters of a higher rank: the adapters' bytes are the call.
        {"name": "adapters 256 x 248320x2048", "kind": "adapters", "n": 256, "N": 248320, "K": 2048, "R": 64, "L": 32,
         "dtype": "bf16", "norm": True, "order": "mixed"},
        # Positions of five requests one behind the other through the stacked heads.
        {"name": "adapters 1939 x 8200x1024", "kind": "adapters", "n": 1939, "N": 8200, "K": 1024, "R": 8, "L": 5,
         "dtype": "bf16", "norm": False, "order": "runs"},
        # fp32 logits, sizes and a rank that divide nothing.
        {"name": "adapters 37 x 70001x1000 f32", "kind": "adapters", "n": 37, "N": 70001, "K": 1000, "R": 5, "L": 6,
         "dtype": "f32", "norm": False, "order": "mixed"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["score", "score", "grad", "adapters", "adapters"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "adapters":
        R = rng.choice([1, 4, 5, 8, 8, 13, 16, 16, 24, 32, 64, 100, 128])
        L = _log_int(rng, 1, 32)
        K = _log_int(rng, 64, 4096)
        if rng.random() < 0.5:
            K = max(64, K // 64 * 64)
        N = _log_int(rng, 64, min(248320, 500_000_000 // (R * L)))
        n = _log_int(rng, 1, max(1, min(4096, 60_000_000 // N, 100_000_000_000 // (R * L * (N + K)))))
        return {"kind": kind, "n": n, "N": N, "K": K, "R": R, "L": L, "dtype": dtype, "norm": rng.random() < 0.5,
                "order": rng.choice(["mixed", "runs"])}
    V = _log_int(rng, 33, 248320)
    n = _log_int(rng, 1, max(1, min(16384, 60_000_000 // V // (2 if kind == "grad" and dtype == "f32" else 1))))
    if kind == "grad":
        return {"kind": kind, "n": n, "V": V, "dtype": dtype, "entropy": rng.random() < 0.5}
    return {"kind": kind, "n": n, "V": V, "dtype": dtype, "top": min(V, rng.choice([0, 1, 5, 8, 20, 20, 32, 64, 128]))}


# ------------------------------------------------------------------ inputs
def _logits(n, V, dtype, g):
    x = torch.randn((n, V), generator=g, device=DEV)
    x *= 3.0 if V < 4096 else 4.0
    # tokens drawn from these rows, as a program scores what was sampled; one in four comes from elsewhere (a prompt)
    tokens = torch.empty((n,), dtype=torch.int64, device=DEV)
    rows = max(1, (1 << 25) // V)
    for i in range(0, n, rows):
        u = torch.rand(x[i:i + rows].shape, generator=g, device=DEV).clamp_(min=1e-20)
        tokens[i:i + rows] = (x[i:i + rows] - u.log_().neg_().log_()).argmax(dim=1)
    other = torch.randint(0, V, (n,), generator=g, device=DEV)
    tokens = torch.where(torch.rand((n,), generator=g, device=DEV) < 0.25, other, tokens)
    # an eighth of the rows come from a constrained grammar: half of the tokens beside the given one are masked, with -inf
    # or with the type's lowest value; of 16 rows and more, one row has nothing left and one is padding without a token
    masked = torch.nonzero(torch.rand((n,), generator=g, device=DEV) < 0.125).reshape(-1)
    for half, low in ((masked[0::2], -math.inf), (masked[1::2], float(torch.finfo(dtype).min))):
        for i in range(0, half.numel(), rows):
            at = half[i:i + rows]
            cut = torch.rand((at.numel(), V), generator=g, device=DEV) < 0.5
            cut.scatter_(1, tokens[at][:, None], False)
            x[at] = torch.where(cut, torch.full_like(cut, low, dtype=torch.float32), x[at])
    if n >= 16:
        x[n // 2] = -math.inf
        tokens[n // 3] = -1
    return x.to(dtype), tokens.to(torch.int32)


def _adapter_rows(case):
    """(rows with an adapter, adapters in use): one row in eight has none."""
    rows = case["n"] - case["n"] // 8
    return rows, min(rows, case["L"])


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": dict(case)}
    dtype = DTYPES[case["dtype"]]
    n = case["n"]
    if case["kind"] == "adapters":
        N, K, R, L = case["N"], case["K"], case["R"], case["L"]
        rows, _ = _adapter_rows(case)
        ids = torch.full((n,), -1, device=DEV)
        if case["order"] == "runs":
            ids[:rows] = torch.arange(rows, device=DEV) * min(rows, L) // rows
        else:
            ids[torch.randperm(n, generator=g, device=DEV)[:rows]] = torch.arange(rows, device=DEV) % L
        s["ids"] = ids.to(torch.int32)
        s["hidden"] = (torch.randn((n, K), generator=g, device=DEV) * 1.7).to(torch.bfloat16)
        s["gain"] = 1.0 + 0.1 * torch.randn((K,), generator=g, device=DEV) if case["norm"] else None
        s["base"] = (torch.randn((n, N), generator=g, device=DEV) * 4.0).to(dtype)
        s["a"] = (torch.randn((L, R, K), generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16)
        s["b"] = torch.empty((L, N, R), dtype=torch.bfloat16, device=DEV)
        for i in range(L):
            s["b"][i] = torch.randn((N, R), generator=g, device=DEV) * (0.5 * R ** -0.5)
        s["scale"] = 0.5 + torch.rand((L,), generator=g, device=DEV)
        if own:
            import vocab_wide_logit_gb300 as ds
            # a serving program keeps its loaded adapters in such stacks
            s["adapters"] = ds.Adapters(s["a"], s["b"], s["scale"])
        return s
    s["x"], s["tokens"] = _logits(n, case["V"], dtype, g)
    if case["kind"] == "grad":
        # what the forward pass left behind, and the loss's gradient by its outputs
        s["lse"], s["entropy"] = _lse_entropy(s["x"])
        s["g_logprobs"] = torch.randn((n,), generator=g, device=DEV)
        s["g_entropy"] = 0.1 * torch.randn((n,), generator=g, device=DEV) if case["entropy"] else None
    return s


def _lse_entropy(logits):
    """float32 log-sum-exp (-inf for a row with nothing) and entropy of each row, made in 64 bits."""
    lse, entropy = [], []
    rows = max(1, (1 << 25) // logits.shape[1])
    for i in range(0, logits.shape[0], rows):
        x = logits[i:i + rows].double()
        z = torch.logsumexp(x, dim=1)
        p = (x - z[:, None]).exp()
        lse.append(z)
        entropy.append(-torch.where(p > 0, p * (x - z[:, None]), torch.zeros_like(x)).sum(dim=1))
    entropy = torch.cat(entropy)
    lse = torch.cat(lse)
    return lse.float(), torch.where(torch.isfinite(lse), entropy, torch.full_like(entropy, math.nan)).float()


# ------------------------------------------------------------------ one pass
def _plain_score(s):
    x = s["x"].float()
    n, V = x.shape
    top = s["case"]["top"]
    tokens = s["tokens"].long()[:, None]
    m = x.amax(dim=1, keepdim=True)
    d = x - m
    e = d.exp()
    total = e.sum(dim=1, keepdim=True)
    lse = m + total.log()
    entropy = total.log() - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(dim=1, keepdim=True) / total
    given = tokens.clamp(min=0)
    at = x.gather(1, given)
    ids = torch.arange(V, device=x.device)[None, :]
    ranks = ((x > at) | ((x == at) & (ids < given))).sum(dim=1, keepdim=True)
    none = torch.isneginf(m)
    unknown = none | (tokens < 0)
    nan = torch.full_like(lse, math.nan)
    if top:
        val, idx = torch.sort(x, dim=1, descending=True, stable=True)
        val, idx = val[:, :top] - lse, idx[:, :top]
    else:
        val, idx = x[:, :0], tokens[:, :0]
    return {"logprobs": torch.where(unknown, nan, at - lse)[:, 0],
            "lse": torch.where(none, m, lse)[:, 0],
            "entropy": torch.where(none, nan, entropy)[:, 0],
            "ranks": torch.where(unknown, torch.full_like(ranks, -1), ranks)[:, 0].to(torch.int32),
            "top_ids": torch.where(none, torch.full_like(idx, -1), idx).to(torch.int32),
            "top_logprobs": torch.where(none, torch.full_like(val, math.nan), val)}


def _plain_grad(s):
    x = s["x"].float()
    tokens = s["tokens"].long()[:, None]
    lse = s["lse"][:, None]
    logp = x - lse
    p = logp.exp()
    g = torch.where(tokens < 0, torch.zeros_like(lse), s["g_logprobs"][:, None])
    ids = torch.arange(x.shape[1], device=x.device)[None, :]
    out = g * ((ids == tokens).float() - p)
    if s["g_entropy"] is not None:
        bend = torch.where(p > 0, p * (logp + s["entropy"][:, None]), torch.zeros_like(p))
        out = out - s["g_entropy"][:, None] * bend
    return torch.where(torch.isneginf(lse), torch.zeros_like(out), out).to(s["x"].dtype)


def _plain_adapters(s):
    y = s["hidden"].float()
    if s["gain"] is not None:
        y = y * torch.rsqrt((y * y).mean(dim=1, keepdim=True) + EPS) * s["gain"][None, :]
    out = s["base"].float()
    for i in range(s["case"]["L"]):
        t = y @ s["a"][i].float().t()
        t = torch.where((s["ids"] == i)[:, None], t * s["scale"][i], torch.zeros_like(t))
        out = out + t @ s["b"][i].float().t()
    return out.to(s["base"].dtype)


def run(state):
    case = state["case"]
    if own:
        import vocab_wide_logit_gb300 as ds
        if case["kind"] == "score":
            r = ds.score_tokens(state["x"], state["tokens"], top=case["top"])
            return {"logprobs": r.logprobs, "lse": r.lse, "entropy": r.entropy, "ranks": r.ranks, "top_ids": r.top_ids,
                    "top_logprobs": r.top_logprobs}
        if case["kind"] == "grad":
            return {"grad": ds.score_tokens_grad(state["x"], state["tokens"], state["lse"], entropy=state["entropy"],
                                                 g_logprobs=state["g_logprobs"], g_entropy=state["g_entropy"])}
        return {"logits": ds.add_adapters(state["base"], state["hidden"], state["adapters"], state["ids"],
                                          gain=state["gain"], eps=EPS)}
    if case["kind"] == "score":
        return _plain_score(state)
    if case["kind"] == "grad":
        return {"grad": _plain_grad(state)}
    return {"logits": _plain_adapters(state)}


def work(case):
    n = case["n"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "score":
        V = case["V"]
        # the logits and tokens once, four results a row and two for each alternative; a difference, an exponential,
        # two sums with a product and a comparison for each logit
        return {"bytes": n * V * size + 20 * n + 8 * n * case["top"], "flops": 6 * n * V}
    if case["kind"] == "grad":
        V = case["V"]
        # the logits once, their gradient once, three to five values a row
        return {"bytes": 2 * n * V * size + (20 if case["entropy"] else 12) * n, "flops": (7 if case["entropy"] else 4) * n * V}
    N, K, R = case["N"], case["K"], case["R"]
    rows, used = _adapter_rows(case)
    # the base logits once, the result once, the hidden states and ids once, each adapter in use once
    return {"bytes": 2 * n * N * size + 2 * n * K + 4 * n + (4 * K if case["norm"] else 0) + used * (2 * R * (N + K) + 4),
            "flops": 2 * rows * R * (N + K) + n * N}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_score(s):
    parts = []
    x_all, top = s["x"], s["case"]["top"]
    V = x_all.shape[1]
    rows = max(1, (1 << 25) // V)
    for i in range(0, x_all.shape[0], rows):
        x, t = x_all[i:i + rows].double(), s["tokens"][i:i + rows].long()
        z = torch.logsumexp(x, dim=1)
        logp = x - z[:, None]
        p = logp.exp()
        h = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(dim=1)
        here = t.clamp(min=0)
        at = x[torch.arange(x.shape[0], device=DEV), here][:, None]
        before = torch.arange(V, device=DEV)[None, :] < here[:, None]
        rank = (x > at).sum(dim=1) + ((x == at) & before).sum(dim=1)
        dead = torch.isneginf(z)
        hide = dead | (t < 0)
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
        best = logp.gather(1, order)
        parts.append((torch.where(hide, math.nan, (at[:, 0] - z)), z, torch.where(dead, math.nan, h),
                      torch.where(hide, -1, rank).to(torch.int32),
                      torch.where(dead[:, None], -1, order).to(torch.int32),
                      torch.where(dead[:, None], math.nan, best)))
    names = ("logprobs", "lse", "entropy", "ranks", "top_ids", "top_logprobs")
    return {name: torch.cat([q[j] for q in parts]) for j, name in enumerate(names)}


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    if case["kind"] == "score":
        return _exact_score(s)
    n = case["n"]
    if case["kind"] == "grad":
        out = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
        rows = max(1, (1 << 25) // case["V"])
        for i in range(0, n, rows):
            live = torch.nonzero(torch.isfinite(s["lse"][i:i + rows])).reshape(-1) + i
            x, t = s["x"][live].double(), s["tokens"][live].long()
            p = (x - s["lse"][live].double()[:, None]).exp()
            gl = s["g_logprobs"][live].double() * (t >= 0)
            dx = -gl[:, None] * p
            dx[torch.arange(live.numel(), device=DEV), t.clamp(min=0)] += gl
            if s["g_entropy"] is not None:
                plogp = torch.where(p > 0, p * (x - s["lse"][live].double()[:, None]), torch.zeros_like(p))
                dx -= s["g_entropy"][live].double()[:, None] * (plogp + p * s["entropy"][live].double()[:, None])
            out[live] = dx
        return {"grad": out}
    h = s["hidden"].double()
    if s["gain"] is not None:
        h = h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["gain"].double()[None, :]
    out = s["base"].double()
    for i in range(case["L"]):
        mine = torch.nonzero(s["ids"] == i).reshape(-1)
        if mine.numel():
            t = h[mine] @ s["a"][i].double().t() * s["scale"][i].double()
            out[mine] += t @ s["b"][i].double().t()
    return {"logits": out}
