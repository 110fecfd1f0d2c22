"""ds_score_tokens and ds_score_tokens_grad against the definition in 64 bits."""
import math

import pytest
import torch

import vocab_wide_logit_gb300 as pkg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dev():
    assert torch.cuda.is_available(), "needs a GPU"
    return torch.device("cuda", 0)


def _reference(x, tokens, top):
    """The definition in float64; rows must hold no NaN and no +inf."""
    x, t = x.double(), tokens.long()
    V = x.shape[1]
    m = x.max(dim=1, keepdim=True).values
    d = x - m  # not x - lse: log s is lost beside a maximum of 1e38, in 64 bits too
    log_s = d.exp().sum(1).log()
    lse, logp = torch.where(torch.isneginf(m[:, 0]), m[:, 0], m[:, 0] + log_s), d - log_s[:, None]
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    here = t.clamp(0, V - 1)
    at = x.gather(1, here[:, None])
    ids = torch.arange(V, device=x.device)[None]
    ranks = ((x > at) | ((x == at) & (ids < here[:, None]))).sum(1)
    order = torch.sort(x + 0.0, dim=1, descending=True, stable=True).indices[:, :top]  # -0 and +0 tie
    dead = torch.isneginf(lse)
    hide = dead | (t < 0) | (t >= V)
    nan, none = torch.full_like(lse, math.nan), torch.full_like(ranks, -1)
    return pkg.TokenScores(torch.where(hide, nan, logp.gather(1, here[:, None])[:, 0]), lse, torch.where(dead, nan, entropy),
                           torch.where(hide, none, ranks), torch.where(dead[:, None], none[:, None], order),
                           torch.where(dead[:, None], nan[:, None], logp.gather(1, order)))


def _sum_tolerance(V, spread):
    """Relative error of a sum of exponentials. An exponential is off by 2^-22, and its argument d by three roundings of
    |d| 2^-24; weighted by probability |d| stays below the spread lse - mean, itself below log V for what counts. A sum is
    kept by a thread over at most V / 256 + 128 terms and joined in 24 steps (an exponential and a product each, twice)."""
    return (4 + 3 * spread + V / 256 + 128 + 4 * 24) * 2.0 ** -24


def _close(got, want, tol, name):
    # beyond fp32's range (1e38 - the lowest value) the nearest fp32 number is the infinity
    got = got.double()
    same = (got == want) | (got == want.float().double()) | (torch.isnan(got) & torch.isnan(want))
    off = (got - want).abs()
    bad = ~(same | (off <= tol))
    assert not bool(bad.any()), (name, int(bad.sum()), float(off[bad].max()), torch.nonzero(bad)[:4].tolist())


def _check(x, tokens, top, r, rows=None):
    V = x.shape[1]
    want = _reference(x, tokens, top)
    if rows is not None:
        x, tokens = x[rows], tokens[rows]
        want = pkg.TokenScores(*(w[rows] for w in want))
        r = pkg.TokenScores(*(g[rows] for g in r))
    rel = _sum_tolerance(V, math.log(max(V, 2)))
    # lse = m + log s: a rounding of the sum and one of the logarithm (2 ulp) beside the relative error of s
    z = rel + (want.lse.abs() + math.log(max(V, 2))) * 2.0 ** -22
    z = torch.where(torch.isfinite(z), z, torch.zeros_like(z))
    _close(r.lse, want.lse, z, "lse")
    _close(r.logprobs, want.logprobs, z + want.logprobs.abs().nan_to_num(0, 0) * 2.0 ** -24, "logprobs")
    # log s - t / s, both sides up to log V
    _close(r.entropy, want.entropy, (2 + 2 * math.log(max(V, 2))) * rel, "entropy")
    assert torch.equal(r.ranks.long(), want.ranks), "ranks"
    assert r.top_ids.shape == (x.shape[0], top) and torch.equal(r.top_ids.long(), want.top_ids), "top_ids"
    _close(r.top_logprobs, want.top_logprobs, z[:, None] + want.top_logprobs.abs().nan_to_num(0, 0) * 2.0 ** -24, "top_logprobs")


def _inputs(n, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((n, V), generator=g) * spread).to(DT[dtype])
    tokens = torch.randint(0, V, (n,), generator=g).to(torch.int32)
    return x.to(_dev()), tokens.to(_dev())


# every launch rule, below and above; the sizes around a chunk, a warp's and a block's share
# and a power of two with a few more
SIZES = [(9, 505), (9, 512), (9, 516), (9, 540), (9, 541), (9, 545), (40, 770), (40, 1017), (40, 1024), (40, 1049), (40, 1050), (40, 1053),
         (40, 1056), (1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 31), (7, 33), (2, 64), (9, 127), (3, 255), (5, 257), (33, 1000), (1, 1025),
         (700, 1025), (6, 2048), (5, 2049), (3, 4096), (4, 4097), (300, 4099), (2, 8191), (17, 8200), (1, 32000), (170, 32001),
         (37, 70001), (1, 248320), (3, 248319), (160, 248320), (1, 1000003)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V", SIZES)
def test_sizes(n, V, dtype):
    x, tokens = _inputs(n, V, dtype, n + V)
    for top in sorted({min(V, t) for t in ((0, 5, 128) if n * V < 4000000 else (20,))}):
        _check(x, tokens, top, pkg.score_tokens(x, tokens, top=top))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [1, 2, 8, 20, 31, 32, 33, 63, 64, 65, 100, 127, 128])
def test_alternatives(top, dtype):
    for n, V in ((40, 129), (300, 1025), (5, 9001), (2, 131072)):
        x, tokens = _inputs(n, V, dtype, top)
        _check(x, tokens, top, pkg.score_tokens(x, tokens, top=top))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [129, 1025, 1040, 5000, 40001])
@pytest.mark.parametrize("kind", ["constant", "zeros", "few", "ascending", "descending", "comb", "one block", "low", "huge",
                                  "tiny", "one", "late"])
def test_orders_and_ties(kind, V, dtype):
    """Rows where candidates are many, tie, or meet in one thread's share."""
    n = 6
    g = torch.Generator().manual_seed(V)
    x = torch.randn((n, V), generator=g)
    if kind == "constant":
        x[:] = 1.25
    elif kind == "zeros":  # -0 and +0 tie
        x = torch.where(x > 0, 0.0, -0.0)
    elif kind == "few":
        x = torch.round(x)
    elif kind == "ascending":
        x = torch.sort(x, dim=1).values
    elif kind == "descending":
        x = torch.sort(x, dim=1, descending=True).values
    elif kind == "comb":  # the largest ones meet in the same lanes whatever the stride between a thread's chunks
        for i, step in enumerate((32, 64, 256, 1024, 2048, 4096)):
            x[i, 5::step] += 20
            x[i, 6::step] += 20
    elif kind == "one block":
        x[:, V // 3:V // 3 + 100] += 30
    elif kind == "low":  # nothing but the type's lowest value, and rows with one or two others
        x[:] = float(torch.finfo(DT[dtype]).min)
        x[1, V - 1] = -5
        x[2, 0] = -2e38
        x[3, 1:3] = 1e38
    elif kind == "huge":
        x *= 5e37
    elif kind == "tiny":
        x *= 1e-38
    elif kind == "one":  # one probable token
        x[:, V // 2] = 200
    else:
        x[:, -3:] = 50
    x = x.to(DT[dtype]).to(_dev())
    tokens = torch.tensor([0, V - 1, V // 2, V // 3 + 50, 5, V // 2], dtype=torch.int32, device=_dev())
    for top in (5, 32, 128):
        _check(x, tokens, top, pkg.score_tokens(x, tokens, top=top))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,team,share", [(3900, 32, 24), (3900, 32, 20), (9000, 128, 64), (9000, 128, 40), (22000, 256, 128),
                                          (36000, 512, 128), (36000, 512, 256), (150001, 512, 128)])
def test_largest_logits_in_few_threads(V, team, share, dtype):
    """Chunks of 16 bytes go round a team of threads: rows whose largest logits are all in some threads' shares, so that a
    bound from the threads' maxima lists thousands."""
    E = 8 if dtype == "bf16" else 4
    V = V * E // 8
    x, tokens = _inputs(5, V, dtype, V + share)
    # rows of a new tensor start on a chunk when V is a multiple of its logits: here the first one does
    few = (torch.arange(V, device=_dev()) // E) % team < share
    x[0] = torch.where(few, x[0].abs() + 20, x[0])
    x[1] = x[0].flip(0)
    x[2] = torch.where(few, torch.full_like(x[2], 9.0), x[2])
    x[3] = torch.where(few, torch.round(x[3].float()).to(x.dtype) + 30, x[3])
    for top in (20, 24, 32, 128):
        _check(x, tokens, top, pkg.score_tokens(x, tokens, top=top))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 1025, 9001, 70001])
def test_masks(V, dtype):
    """Masked by -inf or the type's lowest value: all but none, one, a few, half; whole leading and trailing parts."""
    low = float(torch.finfo(DT[dtype]).min)
    x, tokens = _inputs(12, V, dtype, V)
    half = torch.rand((V,), generator=torch.Generator().manual_seed(1)).to(_dev()) < 0.5
    for i, value in ((0, -math.inf), (6, low)):
        x[i] = value
        x[i + 1, torch.arange(V, device=_dev()) != V // 2] = value
        x[i + 2, 3:] = value
        x[i + 3, half] = value
        x[i + 4, :V - 2] = value
        x[i + 5, V // 4:] = value
    tokens[1] = tokens[7] = V // 2
    tokens[2] = tokens[8] = V - 1  # a masked one
    for top in (1, 20, min(V, 128)):
        _check(x, tokens, top, pkg.score_tokens(x, tokens, top=top))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [17, 520, 1025, 1045, 9001, 248320])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_that_are_not_numbers(V, bad, dtype):
    x, tokens = _inputs(5, V, dtype, V)
    x[1, V - 1] = bad
    x[3, 0] = bad
    x[3, 1:] = -math.inf
    status = torch.zeros(1, dtype=torch.int32, device=_dev())
    r = pkg.score_tokens(x, tokens, top=4, d_status=status)
    assert int(status) == pkg.DS_DEV_ERR_LOGITS
    for i in (1, 3):
        for t in (r.logprobs, r.lse, r.entropy, r.top_logprobs):
            assert bool(torch.isnan(t[i]).all())
        assert int(r.ranks[i]) == -1 and bool((r.top_ids[i] == -1).all())
    good = torch.tensor([0, 2, 4], device=_dev())
    clean = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    _check(clean, tokens, 4, r, rows=good)


@pytest.mark.parametrize("V", [1025, 9001])
def test_rows_without_a_token(V):
    x, tokens = _inputs(6, V, "bf16", V)
    tokens[1], tokens[2], tokens[4] = -1, -(2 ** 31), -1
    x[4] = -math.inf
    status = torch.zeros(1, dtype=torch.int32, device=_dev())
    _check(x, tokens, 7, pkg.score_tokens(x, tokens, top=7, d_status=status))
    assert int(status) == 0
    tokens[3], tokens[5] = V, 2 ** 31 - 1
    _check(x, tokens, 7, pkg.score_tokens(x, tokens, top=7, d_status=status))
    assert int(status) == pkg.DS_DEV_ERR_PARAM


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,pad,offset", [(1025, 0, 1), (1025, 3, 5), (1000, 8, 0), (4200, 1, 7), (33, 2, 3), (70001, 6, 1)])
def test_strides(V, pad, offset, dtype):
    n, g = 9, torch.Generator().manual_seed(V + pad)
    # what lies between the rows is larger than anything in them
    buf = torch.full((n * (V + pad) + offset + 16,), 1e30).to(DT[dtype]).to(_dev())
    x = buf[offset:offset + n * (V + pad)].view(n, V + pad)[:, :V]
    x.copy_((torch.randn((n, V), generator=g) * 3).to(_dev()))
    tokens = torch.randint(0, V, (n,), generator=g).to(torch.int32).to(_dev())
    _check(x, tokens, 20, pkg.score_tokens(x, tokens, top=20))


def test_offsets_beyond_32_bits():
    n, V, ld = 4, 5003, 2 ** 31 - 5
    buf = torch.empty(3 * ld + V, dtype=torch.bfloat16, device=_dev())
    x = buf.as_strided((n, V), (ld, 1))
    fresh, tokens = _inputs(n, V, "bf16", 3)
    x.copy_(fresh)
    r = pkg.score_tokens(x, tokens, top=10)
    _check(fresh, tokens, 10, r)
    dx = pkg.score_tokens_grad(x, tokens, r.lse, g_logprobs=torch.ones(n, device=_dev()))
    assert torch.equal(dx, pkg.score_tokens_grad(fresh, tokens, r.lse, g_logprobs=torch.ones(n, device=_dev())))
    pkg.score_tokens_grad(x, tokens, r.lse, g_logprobs=torch.ones(n, device=_dev()), out=x)
    assert torch.equal(x.contiguous(), dx)


@pytest.mark.parametrize("dtype,V", [("bf16", 2 ** 31 - 1), ("f32", 2 ** 30 + 3)])
def test_one_row_of_the_longest(V, dtype):
    """Positions and byte offsets beyond 32 bits within a row; its sums are known: all logits are 0 but three."""
    x = torch.zeros((1, V), dtype=DT[dtype], device=_dev())
    x[0, V - 1], x[0, 5], x[0, V // 2] = 3, 2, -math.inf
    tokens = torch.tensor([V - 1], dtype=torch.int32, device=_dev())
    r = pkg.score_tokens(x, tokens, top=4)
    assert r.top_ids[0].tolist() == [V - 1, 5, 0, 1] and int(r.ranks[0]) == 0
    lse = math.log(V - 3 + math.exp(3) + math.exp(2))
    # a thread's chain of at most V / 16384 + 200 additions, each off by 2^-24 at most
    tol = (V / 16384 + 200) * 2.0 ** -24 + lse * 2.0 ** -23
    assert abs(float(r.lse[0]) - lse) <= tol and abs(float(r.logprobs[0]) - (3 - lse)) <= tol
    p3, p2 = math.exp(3 - lse), math.exp(2 - lse)
    entropy = lse - 3 * p3 - 2 * p2
    assert abs(float(r.entropy[0]) - entropy) <= (2 + 2 * lse) * tol
    tokens[0] = V - 2
    r = pkg.score_tokens(x, tokens, top=1)
    assert int(r.ranks[0]) == V - 2  # the three others are V - 1, 5 and -inf: V - 3 zeros, of which it is the last
    gl = torch.ones(1, device=_dev())
    out = pkg.score_tokens_grad(x, tokens, r.lse, g_logprobs=gl, out=x)
    # 0 - lse has lse's own half ulp in it, the exponential 2^-22, and bf16 half a step
    p = math.exp(-float(r.lse[0]))
    rel = (3 * lse + 10) * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0)
    for i, want in ((0, -p), (5, -p * math.exp(2)), (V - 1, -p * math.exp(3)), (V // 2, 0.0), (V - 2, 1 - p), (V - 3, -p)):
        assert abs(float(out[0, i]) - want) <= abs(want) * rel, i


@pytest.mark.parametrize("dtype,V", [("bf16", 2 ** 31 - 1), ("bf16", 2 ** 31 - 20), ("f32", 2 ** 31 - 1)])
def test_last_tokens_of_the_longest_rows(V, dtype):
    """All logits tie: a token's rank is its number, for the last ones of two rows, the second of which starts between two
    chunks; the sum of ones is V itself."""
    x = torch.zeros((2, V), dtype=DT[dtype], device=_dev())
    for back in (1, 2, 7, 8, 9, 16, 31, 32, 33):
        tokens = torch.tensor([V - back, V - back - 1], dtype=torch.int32, device=_dev())
        r = pkg.score_tokens(x, tokens)
        assert r.ranks.tolist() == tokens.tolist()
        # V ones in sums of less than V / 16384 + 200 additions, then the logarithm and its sum
        tol = (V / 16384 + 200) * 2.0 ** -24 + math.log(V) * 2.0 ** -22
        assert float((r.lse.double() - math.log(V)).abs().max()) <= tol
        assert float((r.logprobs.double() + math.log(V)).abs().max()) <= tol


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at_once", [8, 16, 32])
def test_sums_of_long_rows_in_a_large_batch(at_once, dtype):
    """More rows than SMs, each long: one logit of 0, the others so low that `at_once` of their exponentials are below half a
    step of a sum of 1. An addition of no more of them is lost where the sum has the 0; the stated number of additions bounds
    what is."""
    n, V = torch.cuda.get_device_properties(0).multi_processor_count + 8, 1 << 24
    low = torch.tensor(-math.log(at_once) - 24.05 * math.log(2)).to(DT[dtype])
    e = math.exp(float(low))
    assert at_once * e < 2.0 ** -24
    x = torch.full((n, V), float(low), dtype=DT[dtype], device=_dev())
    x[:, 0] = 0
    s = 1 + (V - 1) * e
    r = pkg.score_tokens(x, torch.zeros(n, dtype=torch.int32, device=_dev()))
    # additions, the exponentials (2^-22, three roundings of their argument), the logarithm and its sum
    tol = (V / 16384 + 200 + 4 + 3 * abs(float(low)) + 8) * 2.0 ** -24
    off = max(float((r.lse.double() - math.log(s)).abs().max()), float((r.logprobs.double() + math.log(s)).abs().max()))
    assert off <= tol, off / tol


def test_results_can_be_saved(tmp_path):
    """Results share their memory by type; what a program does with tensors works on them."""
    x, tokens = _inputs(3, 100, "f32", 1)
    for top in (0, 4):
        r = pkg.score_tokens(x, tokens, top=top)
        torch.save(tuple(r), tmp_path / "scores.pt")
        for a, b in zip(r, torch.load(tmp_path / "scores.pt")):
            assert torch.equal(a, b)
        kept = [t.clone() for t in r]
        for t in r[:3]:
            t.add_(1)
        assert torch.equal(r.ranks, kept[3]) and torch.equal(r.top_ids, kept[4]) and torch.equal(r.logprobs, kept[0] + 1)


# ------------------------------------------------------------------ gradient
def _grad_reference(x, tokens, lse, entropy, gl, gh):
    x, t, z = x.double(), tokens.long(), lse.double()[:, None]
    logp = x - z
    p = logp.exp()
    given = (t >= 0) & (t < x.shape[1])
    g = torch.zeros_like(z) if gl is None else torch.where(given, gl.double(), torch.zeros_like(z[:, 0]))[:, None]
    hit = torch.arange(x.shape[1], device=x.device)[None] == t[:, None]
    out = g * (hit.double() - p)
    size = g.abs() * (hit.double() + p)
    if gh is not None:
        bend = torch.where(p > 0, p * (logp + entropy.double()[:, None]), torch.zeros_like(p))
        out = out - gh.double()[:, None] * bend
        size = size + gh.double().abs()[:, None] * torch.where(
            p > 0, p * (logp.abs() + entropy.double().abs()[:, None]), torch.zeros_like(p))
    dead = torch.isneginf(z)
    return torch.where(dead, torch.zeros_like(out), out), torch.where(dead, torch.zeros_like(size), size), logp


def _check_grad(got, x, tokens, lse, entropy, gl, gh):
    want, size, logp = _grad_reference(x, tokens, lse, entropy, gl, gh)
    # p: exponential 2^-22, its argument three roundings of |log p|; five roundings of terms and sums; the type's own
    # half step; a p below fp32's normal range is 0
    d = logp.abs().clamp(max=110)
    scale = torch.zeros_like(lse) if gl is None else gl.abs().nan_to_num(0)
    tol = size * (4 + 3 * d + 6) * 2.0 ** -24 + 2.0 ** -126 * (1 + scale.double()[:, None])
    if gh is not None:
        tol = tol + gh.double().abs()[:, None] * 2.0 ** -126 * 256
    if got.dtype == torch.bfloat16:
        tol = tol + want.abs() * 2.0 ** -8 * (1 + 2.0 ** -10) + 2.0 ** -134
    _close(got, want, tol, "grad")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V", [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 33), (24, 1025), (700, 1025), (5, 4096), (17, 8200),
                                 (37, 70001), (2, 248319), (40, 248320)])
def test_grad(n, V, dtype):
    x, tokens = _inputs(n, V, dtype, n + V)
    if n > 3:
        tokens[2] = -1
        x[3] = -math.inf
        x[1, ::2] = -math.inf
        x[0, 1::3] = float(torch.finfo(DT[dtype]).min)
    r = pkg.score_tokens(x, tokens)
    g = torch.Generator().manual_seed(n)
    gl, gh = torch.randn((n,), generator=g).to(_dev()), torch.randn((n,), generator=g).to(_dev())
    if n > 3:
        gl[2] = math.nan  # no token: whatever is there
    for a, b in ((gl, None), (gl, gh), (None, gh)):
        dx = pkg.score_tokens_grad(x, tokens, r.lse, entropy=None if b is None else r.entropy, g_logprobs=a, g_entropy=b)
        assert dx.dtype == x.dtype and dx.is_contiguous()
        _check_grad(dx, x, tokens, r.lse, r.entropy, a, b)
        if n > 3:
            assert float(dx[3].abs().max()) == 0
    kept = x.clone()
    assert pkg.score_tokens_grad(x, tokens, r.lse, r.entropy, gl, gh, out=x) is x
    assert not bool(x.isnan().any())
    _check_grad(x, kept, tokens, r.lse, r.entropy, gl, gh)


@pytest.mark.parametrize("V", [5, 40])
def test_grad_against_differences(V):
    """Central differences of the forward formula in 64 bits; the gradient is fp32's."""
    n = 3
    x, tokens = _inputs(n, V, "f32", V, spread=1.5)
    r = pkg.score_tokens(x, tokens)
    g = torch.Generator().manual_seed(9)
    gl, gh = torch.randn((n,), generator=g).to(_dev()), torch.randn((n,), generator=g).to(_dev())
    dx = pkg.score_tokens_grad(x, tokens, r.lse, r.entropy, gl, gh)

    def loss(y):
        want = _reference(y, tokens, 0)
        return gl.double() * want.logprobs + gh.double() * want.entropy

    h = 1e-5
    for j in range(V):
        up, down = x.double().clone(), x.double().clone()
        up[:, j] += h
        down[:, j] -= h
        # a truncation of h^2 / 6 times third derivatives below 50 here, and 1e-14 / h of rounding
        assert float((dx[:, j].double() - (loss(up) - loss(down)) / (2 * h)).abs().max()) < 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,pad,offset,opad,ooffset", [(1025, 0, 1, 0, 1), (1025, 3, 5, 0, 0), (1000, 8, 0, 4, 2), (33, 2, 3, 7, 1)])
def test_grad_strides(V, pad, offset, opad, ooffset, dtype):
    n = 9
    fresh, tokens = _inputs(n, V, dtype, V + pad)
    buf = torch.full((n * (V + pad) + offset,), 7.0, dtype=DT[dtype], device=_dev())
    x = buf[offset:].view(n, V + pad)[:, :V]
    x.copy_(fresh)
    obuf = torch.full((n * (V + opad) + ooffset + 9,), 7.0, dtype=DT[dtype], device=_dev())
    out = obuf[ooffset:ooffset + n * (V + opad)].view(n, V + opad)[:, :V]
    lse = pkg.score_tokens(x, tokens).lse
    gl = torch.ones(n, device=_dev())
    pkg.score_tokens_grad(x, tokens, lse, g_logprobs=gl, out=out)
    _check_grad(out, fresh, tokens, lse, None, gl, None)
    out.zero_()
    assert float((obuf == 7.0).sum()) == ooffset + 9 + n * opad  # nothing beside the rows was written
    pkg.score_tokens_grad(x, tokens, lse, g_logprobs=gl, out=x)
    _check_grad(x, fresh, tokens, lse, None, gl, None)
    x.zero_()
    assert float((buf == 7.0).sum()) == offset + n * pad


@pytest.mark.parametrize("bend", [False, True])
@pytest.mark.parametrize("dtype,V", [("bf16", 2 ** 31 - 1), ("bf16", 2 ** 31 - 8), ("f32", 2 ** 31 - 1)])
def test_grad_of_the_longest_rows(V, dtype, bend):
    """Two rows of tied logits, the second of which starts between two chunks: every gradient is written, the first ones and
    the last ones of both."""
    lse = torch.full((2,), math.log(V), device=_dev())
    gl, gh = torch.tensor([1.0, -2.0], device=_dev()), torch.tensor([0.5, 0.25], device=_dev())
    for tokens in ((V - 1, 3), (0, V - 1)):
        x = torch.zeros((2, V), dtype=DT[dtype], device=_dev())
        out = torch.full((2, V), math.nan, dtype=DT[dtype], device=_dev())
        t = torch.tensor(tokens, dtype=torch.int32, device=_dev())
        pkg.score_tokens_grad(x, t, lse, lse if bend else None, gl, gh if bend else None, out=out)
        del x
        p = math.exp(-float(lse[0]))  # log p + H is 0
        # p: exponential 2^-22, its argument three roundings of log V; five roundings of terms of up to |gl| + |gh| log V
        rel = (4 + 3 * math.log(V) + 6) * 2.0 ** -24
        half = 2.0 ** -8 if dtype == "bf16" else 0.0
        for i in range(2):
            want = -p * float(gl[i])
            tol = p * (abs(float(gl[i])) + (float(gh[i]) * 2 * math.log(V) if bend else 0)) * rel + abs(want) * half * (1 + 2.0 ** -10)
            hit = float(out[i, tokens[i]])
            assert abs(hit - float(gl[i]) * (1 - p)) <= abs(float(gl[i])) * (half + 2.0 ** -22)
            out[i, tokens[i]] = want  # (rounded to the type it stays within the tolerance)
            least, most = float(out[i].amin()), float(out[i].amax())  # a NaN shows in both
            assert abs(least - want) <= tol and abs(most - want) <= tol, (i, least, most, want)
        del out


def test_grad_bad_rows():
    x, tokens = _inputs(4, 100, "f32", 1)
    x[1, 5] = math.nan
    tokens[2] = 100
    status = torch.zeros(1, dtype=torch.int32, device=_dev())
    r = pkg.score_tokens(x, tokens)
    dx = pkg.score_tokens_grad(x, tokens, r.lse, g_logprobs=torch.ones(4, device=_dev()), d_status=status)
    assert int(status) == pkg.DS_DEV_ERR_PARAM
    assert bool(dx[1].isnan().all()) and float(dx[2].abs().max()) == 0
    assert bool(torch.isfinite(dx[0]).all()) and bool(torch.isfinite(dx[3]).all())


# ------------------------------------------------------------------ how it is called
@pytest.mark.parametrize("V", [1025, 20011, 100003])
def test_a_row_in_other_batches(V):
    """Ranks and alternatives are the same whatever the batch; fp32 results within their own error."""
    x, tokens = _inputs(320, V, "bf16", V)
    whole = pkg.score_tokens(x, tokens, top=16)
    for i, n in ((0, 1), (3, 2), (7, 40), (0, 320)):
        part = pkg.score_tokens(x[i:i + n], tokens[i:i + n], top=16)
        assert torch.equal(part.ranks, whole.ranks[i:i + n]) and torch.equal(part.top_ids, whole.top_ids[i:i + n])
    again = pkg.score_tokens(x, tokens, top=16)
    for a, b in zip(whole, again):
        assert torch.equal(a, b)  # run to run: bit for bit


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1025, 20011, 100003])
def test_float_results_in_other_batches(V, dtype):
    """The batch decides how many threads and CTAs a row has: log-probabilities, sums and entropies of each batch are as near
    to the definition, so that those of two batches differ by twice that at most."""
    x, tokens = _inputs(320, V, dtype, V)
    whole = pkg.score_tokens(x, tokens, top=16)
    _check(x, tokens, 16, whole)
    rel = _sum_tolerance(V, math.log(V))
    z = rel + (whole.lse.double().abs() + math.log(V)) * 2.0 ** -22  # as in _check()
    for i, n in ((0, 1), (3, 2), (7, 40), (20, 100), (100, 160)):
        part = pkg.score_tokens(x[i:i + n], tokens[i:i + n], top=16)
        _check(x[i:i + n], tokens[i:i + n], 16, part)
        for a, b, tol in ((part.lse, whole.lse, z), (part.entropy, whole.entropy, (2 + 2 * math.log(V)) * rel + 0 * z),
                          (part.logprobs, whole.logprobs, z + whole.logprobs.double().abs() * 2.0 ** -24)):
            assert bool(((a.double() - b[i:i + n].double()).abs() <= 2 * tol[i:i + n]).all())


def test_no_rows():
    x = torch.empty((0, 50), dtype=torch.bfloat16, device=_dev())
    none = torch.empty(0, dtype=torch.int32, device=_dev())
    r = pkg.score_tokens(x, none, top=3)
    assert r.logprobs.shape == (0,) and r.top_ids.shape == (0, 3)
    assert pkg.score_tokens_grad(x, none, r.lse, g_logprobs=r.logprobs).shape == (0, 50)


def test_another_stream_and_a_graph():
    """Captured and replayed on new inputs, two graphs at once among them."""
    n, V, s = 5, 9001, torch.cuda.Stream()
    x, tokens = _inputs(n, V, "bf16", 1)
    gl, gh = torch.randn(n, device=_dev()), torch.randn(n, device=_dev())

    def step(x, tokens, stream=None):
        r = pkg.score_tokens(x, tokens, top=6, stream=stream)
        return r, pkg.score_tokens_grad(x, tokens, r.lse, r.entropy, gl, gh, stream=stream)

    s.wait_stream(torch.cuda.current_stream())
    r, dx = step(x, tokens, s)
    torch.cuda.current_stream().wait_stream(s)
    _check(x, tokens, 6, r)
    _check_grad(dx, x, tokens, r.lse, r.entropy, gl, gh)
    graphs = []
    for seed in (2, 3):
        y, t = _inputs(n, V, "bf16", seed)
        step(y, t)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(y, t)
        graphs.append((graph, y, t, out))
    for k, (graph, y, t, _) in enumerate(graphs):
        fresh, ft = _inputs(n, V, "bf16", 10 + k)
        y.copy_(fresh)
        t.copy_(ft)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for (graph, _, _, _), stream in zip(graphs, (s, other)):
        with torch.cuda.stream(stream):
            for _ in range(3):
                graph.replay()
    torch.cuda.synchronize()
    for _, y, t, (r, dx) in graphs:
        _check(y, t, 6, r)
        _check_grad(dx, y, t, r.lse, r.entropy, gl, gh)


def test_both_ways_of_a_call():
    """The calls that ds_calls runs, and the same through the checks in Python (as with a status word)."""
    status = torch.zeros(1, dtype=torch.int32, device=_dev())
    for n, V, dtype, top in ((5, 1025, "bf16", 4), (3, 9001, "f32", 0), (1, 40, "f32", 40)):
        x, tokens = _inputs(n, V, dtype, n)
        fast, slow = pkg.score_tokens(x, tokens, top=top), pkg.score_tokens(x, tokens, top=top, d_status=status)
        assert type(fast) is type(slow) is pkg.TokenScores
        for a, b in zip(fast, slow):
            assert torch.equal(a, b) and a.dtype == b.dtype and a.shape == b.shape
        gl = torch.randn(n, device=_dev())
        assert torch.equal(pkg.score_tokens_grad(x, tokens, fast.lse, fast.entropy, gl, gl),
                           pkg.score_tokens_grad(x, tokens, fast.lse, fast.entropy, gl, gl, d_status=status))
    for bad in (dict(tokens=None), dict(tokens=tokens.long()), dict(tokens=tokens.cpu()), dict(top=41), dict(top=-1),
                dict(logits=x.half()), dict(logits=x[:, ::2])):
        with pytest.raises(ValueError):
            pkg.score_tokens(**{**dict(logits=x, tokens=tokens, top=1), **bad})
    for bad in (dict(lse=None), dict(lse=fast.lse.double()), dict(g_logprobs=None), dict(g_logprobs=None, g_entropy=gl),
                dict(g_logprobs=gl.cpu())):
        with pytest.raises(ValueError):
            pkg.score_tokens_grad(**{**dict(logits=x, tokens=tokens, lse=fast.lse, g_logprobs=gl), **bad})


def test_c_names():
    n, V, top = 4, 2000, 9
    x, tokens = _inputs(n, V, "f32", 5)
    f = lambda *shape: torch.empty(shape, device=_dev())  # noqa: E731
    i = lambda *shape: torch.empty(shape, dtype=torch.int32, device=_dev())  # noqa: E731
    got = pkg.TokenScores(f(n), f(n), f(n), i(n), i(n, top), f(n, top))
    pkg.ds_score_tokens(x, tokens, got.logprobs, got.lse, got.entropy, got.ranks, got.top_ids, got.top_logprobs)
    want = pkg.score_tokens(x, tokens, top=top)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    alone = f(n)
    pkg.ds_score_tokens(x, tokens, alone)  # the results that may be left out are
    assert torch.equal(alone, want.logprobs)
    gl, out = torch.randn(n, device=_dev()), f(n, V)
    pkg.ds_score_tokens_grad(x, tokens, want.lse, out, g_logprobs=gl)
    assert torch.equal(out, pkg.score_tokens_grad(x, tokens, want.lse, g_logprobs=gl))
