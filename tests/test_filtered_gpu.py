"""ds_sample_filtered against plain implementations: the integer definition (tokens equal), and the real-number
distribution in 64 bits (the drawn token's interval of the cumulative distribution holds u)."""
import math

import numpy as np
import pytest
import torch

import vocab_wide_logit_gb300 as pkg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dev():
    assert torch.cuda.is_available(), "needs a GPU"
    return torch.device("cuda", 0)


def _params(n, seed, greedy=True):
    g = np.random.Generator(np.random.PCG64(seed))
    tau = g.choice(np.array(([0.0] if greedy else []) + [0.3, 0.7, 1.0, 1.5, 8.0], np.float32), n)
    k = g.choice(np.array([0, 0, 0, 1, 2, 17, 50, 1000, 1 << 30], np.int32), n)
    p = g.choice(np.array([1.0, 1.0, 0.99, 0.9, 0.5, 1e-3], np.float32), n)
    mp = g.choice(np.array([0.0, 0.0, 0.02, 0.2, 1.0], np.float32), n)
    u = g.random(n, dtype=np.float32)
    u[: min(n, 2)] = [0.0, np.float32(1 - 2.0 ** -24)][: min(n, 2)]
    return tau, k, p, mp, u


def _logits(n, V, sigma, seed, dtype, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, V), generator=g) * sigma
    if kind == "few":        # a handful of distinct values: ties everywhere
        x = torch.round(x)
        x[x == 0] = torch.where(torch.rand((int((x == 0).sum()),), generator=g) < 0.5, 0.0, -0.0)
    elif kind == "equal":
        x[:] = 1.25
    elif kind == "masked":   # half of the tokens at -inf or at the type's lowest value; one row with one token left
        low = torch.where(torch.arange(n)[:, None] % 2 == 0, -math.inf, float(torch.finfo(dtype).min))
        x = torch.where(torch.rand((n, V), generator=g) < 0.5, low, x)
        x[n // 2] = -math.inf
        x[n // 2, V // 2] = -3.0
    elif kind == "peaked":   # one token holds nearly all of the mass
        x[torch.arange(n), torch.randint(0, V, (n,), generator=g)] += 60.0
    return x.to(dtype)


def _run(x, tau, k, p, mp, u, status=None, stream=None):
    dev = x.device
    up = lambda v: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).to(dev)  # noqa: E731
    tok, lp = pkg.sample_filtered(x, up(tau), up(u), top_k=up(k), top_p=up(p), min_p=up(mp), d_status=status)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), lp.cpu().numpy()


def _integer_definition(x, tau, k, p, mp, u):
    """Tokens by the integer definition: fp32 exponentials (torch's), everything after them exact."""
    dev = x.device
    up = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(dev)[:, None]  # noqa: E731
    tau, k, p, mp, u = up(tau), up(k), up(p).double(), up(mp).double(), up(u).double()
    x = x.float()
    V = x.shape[1]
    val, idx = torch.sort(x, dim=1, descending=True, stable=True)
    r = torch.where(tau == 0, torch.ones_like(tau), (1.0 / tau).clamp(max=3.4028234663852886e38))
    w = torch.round(((val - val[:, :1]) * r).exp() * 2.0 ** 31).nan_to_num().long()
    w = torch.where((k <= 0) | (torch.arange(V, device=dev)[None] < k), w, 0)
    cum = w.cumsum(1)
    keep = ((cum - w).double() < p * cum[:, -1:].double()) & (w.double() >= mp * 2.0 ** 31)
    w = torch.where(keep, w, 0)
    cum = w.cumsum(1)
    t = (u * cum[:, -1:].double()).floor().long()
    at = (cum <= t).sum(1, keepdim=True).clamp(max=V - 1)
    at = torch.where(tau == 0, 0, at)
    tok = idx.gather(1, at)[:, 0]
    tok = torch.where(torch.isinf(val[:, 0]), -1, tok)
    return tok.cpu().numpy()


def _check_real(x, tok, lp, tau, k, p, mp, u):
    """The drawn token against the distribution in 64 bits. A weight's relative error: y = (x - m) / tau has three
    roundings of 2^-24 each and |y| < 22.2 wherever the weight is not zero, so 22.2 * 3 * 2^-24 = 4e-6; the fp32
    exponential and the scaling add under 3e-7; rounding to the integer adds 2^-32 of the largest weight, once per
    logit."""
    xs = x.float().cpu().numpy().astype(np.float64)
    V = xs.shape[1]
    for i in range(xs.shape[0]):
        row = xs[i]
        m = row.max()
        if m == -np.inf:
            assert tok[i] == -1 and np.isnan(lp[i])
            continue
        lse = m + math.log(np.exp(row - m).sum())
        assert 0 <= tok[i] < V
        # fp32 sums of at most V terms, taken in a tree: under 4e-6 relative, then the rounding of two values
        assert abs(lp[i] - (row[tok[i]] - lse)) <= 4e-6 + 2 * 2.0 ** -24 * (abs(row[tok[i]]) + abs(lse) + abs(m))
        order = np.lexsort((np.arange(V), -row))
        if tau[i] == 0:
            assert tok[i] == order[0]
            continue
        w = np.exp((row[order] - m) / float(tau[i]))
        d = 5e-6 + V * 2.0 ** -32
        kk = V if k[i] <= 0 or k[i] >= V else int(k[i])
        w[kk:] = 0
        cum = np.cumsum(w)
        before = cum - w
        total = cum[-1]
        lens = []
        for s in (-1.0, 1.0):
            keep = (before < float(p[i]) * total * (1 + s * d) + s * d) & (w >= float(mp[i]) * (1 - s * d))
            keep[0] = True
            lens.append(int(keep.sum()) if keep.all() else int(np.argmin(keep)))
        at = int(np.nonzero(order == tok[i])[0][0])
        assert at < min(lens[1], kk), (i, at, lens)
        lo = before[at] / cum[max(lens[1], 1) - 1]
        hi = cum[at] / cum[max(lens[0], 1) - 1]
        assert lo - 2 * d <= float(u[i]) <= hi + 2 * d, (i, lo, float(u[i]), hi)


CASES = [(1, 1, "normal"), (3, 2, "normal"), (5, 7, "few"), (33, 33, "normal"), (17, 255, "masked"), (64, 1025, "normal"),
         (40, 1025, "few"), (40, 1025, "masked"), (8, 1025, "equal"), (9, 2055, "peaked"), (24, 4097, "normal"),
         (24, 4097, "few"), (6, 20000, "masked"), (6, 32768, "normal"), (5, 70001, "normal"), (3, 70001, "equal"),
         (4, 131072, "few"), (3, 248320, "normal"), (2, 248320, "masked"), (2, 524281, "normal")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,kind", CASES)
def test_tokens_and_logprobs(n, V, kind, dtype):
    x = _logits(n, V, 3.0, n * 7 + V, DT[dtype], kind).to(_dev())
    par = _params(n, V + n)
    tok, lp = _run(x, *par)
    assert np.array_equal(tok, _integer_definition(x, *par))
    _check_real(x, tok, lp, *par)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sigma", [0.0, 1e-3, 0.1, 1.0, 4.0, 30.0])
@pytest.mark.parametrize("V", [1025, 50000])
def test_every_spread_and_filter_alone(sigma, V, dtype):
    """Flat to peaked rows, each filter alone, none, and temperatures from 1e-30 to 1e30."""
    n = 48
    x = _logits(n, V, sigma, V, DT[dtype]).to(_dev())
    g = np.random.Generator(np.random.PCG64(9))
    one, zero = np.ones(n, np.float32), np.zeros(n, np.float32)
    u = g.random(n, dtype=np.float32)
    tau = np.array([1e-30, 1e-3, 0.5, 1.0, 1.0, 3.0, 1e3, 1e30], np.float32)[np.arange(n) % 8]
    none = np.zeros(n, np.int32)
    for k, p, mp in ((none, one, zero), (none + 40, one, zero), (none, one * np.float32(0.8), zero),
                     (none, one, one * np.float32(0.1)), (none + V - 1, one * np.float32(0.999), zero)):
        par = (tau, k, p, mp, u)
        tok, lp = _run(x, *par)
        assert np.array_equal(tok, _integer_definition(x, *par))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V", [(1300, 33), (1300, 1025), (1301, 2048), (1300, 2049), (700, 5003), (160, 9001),
                                 (80, 20000), (100, 70001)])
@pytest.mark.parametrize("kind", ["normal", "few", "masked", "equal", "peaked"])
def test_batches_that_fill_the_gpu(n, V, kind, dtype):
    """Enough rows that each gets one warp or one CTA, and several in turn; rows that take further passes among them."""
    x = _logits(n, V, 3.0, V, DT[dtype], kind)
    x[::7] *= 0.01
    if kind == "peaked":  # further yet than a sum of exponentials reaches from the other logits
        x[3::11] = torch.where(x[3::11] > 30, x[3::11] + 200, x[3::11])
    x = x.to(_dev())
    par = _params(n, V)
    tok, _ = _run(x, *par)
    assert np.array_equal(tok, _integer_definition(x, *par))


def test_filters_left_out_are_off():
    n, V = 16, 1025
    x = _logits(n, V, 2.0, 1, torch.bfloat16).to(_dev())
    u = np.random.Generator(np.random.PCG64(2)).random(n, dtype=np.float32)
    tau, one, zero = np.ones(n, np.float32), np.ones(n, np.float32), np.zeros(n, np.float32)
    a = _run(x, tau, None, None, None, u)
    b = _run(x, tau, np.zeros(n, np.int32), one, zero, u)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,pad,offset", [(1025, 0, 1), (1025, 7, 3), (1000, 24, 0), (4097, 3, 5), (33333, 11, 1)])
def test_strides_and_alignment(V, pad, offset, dtype):
    """Rows that start anywhere and lie apart; what lies between the rows is not read as logits."""
    n, ld = 6, V + pad
    dense = _logits(n, V, 3.0, V, DT[dtype]).to(_dev())
    buf = torch.full((n * ld + offset + 8,), 80.0, dtype=DT[dtype], device=_dev())
    x = buf[offset:offset + n * ld].view(n, ld)[:, :V]
    x.copy_(dense)
    par = _params(n, 5)
    a, b = _run(dense, *par), _run(x, *par)
    assert np.array_equal(a[0], b[0])
    np.testing.assert_allclose(a[1], b[1], rtol=0, atol=1e-5)


def test_a_row_does_not_depend_on_its_batch():
    V, n = 50001, 40
    x = _logits(n, V, 3.0, 4, torch.bfloat16).to(_dev())
    par = _params(n, 6)
    whole, _ = _run(x, *par)
    for i in (0, 7, 39):
        alone, _ = _run(x[i:i + 1], *(v[i:i + 1] for v in par))
        assert alone[0] == whole[i]
    again, _ = _run(x, *par)
    assert np.array_equal(again, whole)


def test_offsets_beyond_32_bits():
    """More than 2^31 logits, apart by more than a row: the last rows are those of a call of their own."""
    n, V, ld = 8650, 248320, 248323
    buf = torch.empty(n * ld, dtype=torch.bfloat16, device=_dev())
    assert buf.numel() > 2 ** 31
    for i in range(0, buf.numel(), 1 << 28):
        buf[i:i + (1 << 28)].normal_(0, 4)
    x = buf.view(n, ld)[:, :V]
    par = _params(n, 21)
    tok, lp = _run(x, *par)
    for i in (0, 4321, n - 40):
        part = [v[i:i + 40] for v in par]
        t, l = _run(x[i:i + 40].contiguous(), *part)
        assert np.array_equal(tok[i:i + 40], t) and np.allclose(lp[i:i + 40], l, rtol=0, atol=1e-5, equal_nan=True)
        assert np.array_equal(t, _integer_definition(x[i:i + 40], *part))


@pytest.mark.parametrize("V", [11, 1025, 9000])
def test_draws_follow_the_distribution(V):
    """u over an even grid: each kept token is drawn in proportion to its mass, to within two grid steps."""
    n = 4096
    x = _logits(1, V, 2.0, V, torch.float32)
    p64 = np.exp(x[0].double().numpy() - float(x.max()))
    order = np.lexsort((np.arange(V), -p64))
    kept = order[:10]
    want = np.zeros(V)
    want[kept] = p64[kept] / p64[kept].sum()
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    one = np.ones(n, np.float32)
    tok, _ = _run(x.expand(n, V).contiguous().to(_dev()), one, np.full(n, 10, np.int32), one, one * 0, u)
    got = np.bincount(tok, minlength=V) / n
    assert np.abs(got - want).max() <= 2.0 / n
    assert (got[want == 0] == 0).all()


@pytest.mark.parametrize("V", [9, 1025, 40000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_cannot_be_drawn(V, dtype):
    """Empty rows, NaN, +inf and bad parameters: token -1, logprob NaN, the status bit, and no effect on the rest."""
    dev, n = _dev(), 12
    x = _logits(n, V, 2.0, 3, DT[dtype])
    ok = [0, 3, 5, 8, 10]
    x[1] = -math.inf
    one = lambda v: np.full(n, v, np.float32)  # noqa: E731
    tau, k, p, mp, u = one(1.0), np.zeros(n, np.int32), one(0.9), one(0.0), one(0.4)
    good, _ = _run(x.to(dev), tau, k, p, mp, u)

    def bits(x, *par):
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        tok, lp = _run(x.to(dev), *par, status=st)
        return tok, lp, int(st.item())

    tok, lp, st = bits(x, tau, k, p, mp, u)
    assert tok[1] == -1 and np.isnan(lp[1]) and st == 0
    for bad in (math.nan, math.inf):
        y = x.clone()
        y[2, V - 1] = bad
        y[4, 0] = bad
        y[6, :] = bad
        for t in (tau, one(0.0)):
            tok, lp, st = bits(y, t, k, p, mp, u)
            assert st == pkg.DS_DEV_ERR_LOGITS
            assert (tok[[2, 4, 6]] == -1).all() and np.isnan(lp[[2, 4, 6]]).all()
            if t is tau:
                assert np.array_equal(tok[ok], good[ok])
    for which, values in ((0, (-1.0, math.nan, math.inf)), (2, (0.0, 1.5, math.nan, -0.1)), (3, (-0.1, 1.1, math.nan)),
                          (4, (1.0, -0.1, math.nan))):
        for v in values:
            par = [tau.copy(), k, p.copy(), mp.copy(), u.copy()]
            par[which][7] = v
            tok, lp, st = bits(x, *par)
            assert st == pkg.DS_DEV_ERR_PARAM and tok[7] == -1 and np.isnan(lp[7])
            assert np.array_equal(tok[ok], good[ok])


def test_empty_call_and_other_stream():
    dev = _dev()
    e = torch.empty(0, dtype=torch.float32, device=dev)
    tok, lp = pkg.sample_filtered(torch.empty((0, 100), dtype=torch.bfloat16, device=dev), e, e)
    assert tok.numel() == 0 and lp.numel() == 0
    x = _logits(8, 4097, 2.0, 8, torch.bfloat16).to(dev)
    par = _params(8, 8)
    want, _ = _run(x, *par)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    up = [torch.from_numpy(v).to(dev) for v in par]
    torch.cuda.synchronize()
    tok, _ = pkg.sample_filtered(x, up[0], up[4], top_k=up[1], top_p=up[2], min_p=up[3], stream=s)
    s.synchronize()
    assert np.array_equal(tok.cpu().numpy(), want)
