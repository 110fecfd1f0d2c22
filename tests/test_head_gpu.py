"""ds_quantize_rows, ds_pack_i8 and ds_linear_i8 against 64-bit arithmetic, and the whole head."""
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


# ------------------------------------------------------------------ quantisation
def _check_quantised(x, gain, eps, q, scale):
    """fp32 error of y * 127 / amax: the sum of squares (a tree over K terms), the root, three products and a quotient
    stay below 16 roundings, so below 127 * 16 * 2^-24 = 1.3e-4 of a step; a q may be off its real value by half a step
    and that."""
    y = x.double()
    if gain is not None:
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + eps) * gain.double()
    amax = y.abs().amax(1, keepdim=True)
    real = torch.where(amax > 0, y * 127 / amax, torch.zeros_like(y))
    assert int(q.abs().max()) <= 127
    assert float((q.double() - real).abs().max()) <= 0.5 + 2e-4
    np.testing.assert_allclose(scale.double().cpu().numpy(), (amax[:, 0] / 127).cpu().numpy(), rtol=16 * 2.0 ** -24,
                               atol=0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,K", [(1, 1), (2, 3), (3, 31), (5, 64), (7, 257), (4, 1000), (33, 1024), (300, 2048), (3, 8191),
                                 (2, 20001)])
@pytest.mark.parametrize("norm", [False, True])
def test_quantize_rows(n, K, dtype, norm):
    dev = _dev()
    g = torch.Generator().manual_seed(n + K)
    x = (torch.randn((n, K), generator=g) * 3).to(DT[dtype]).to(dev)
    if n > 2:
        x[1] = 0
        x[2] *= 1e-6
    gain = (1 + 0.2 * torch.randn((K,), generator=g)).to(dev) if norm else None
    q, scale = pkg.quantize_rows(x, gain=gain, eps=1e-5)
    _check_quantised(x, gain, 1e-5, q, scale)
    if n > 2:
        assert float(scale[1]) == 0 and int(q[1].abs().max()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,pad,offset", [(64, 8, 0), (64, 3, 1), (1000, 1, 5), (1024, 0, 3)])
def test_quantize_strided(K, pad, offset, dtype):
    dev, n = _dev(), 9
    g = torch.Generator().manual_seed(K)
    buf = torch.randn((n * (K + pad) + offset,), generator=g).to(DT[dtype]).to(dev)
    x = buf[offset:].view(n, K + pad)[:, :K]
    q, scale = pkg.quantize_rows(x)
    _check_quantised(x, None, 0.0, q, scale)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("norm", [False, True])
def test_quantize_row_that_is_not_finite(bad, norm):
    dev = _dev()
    x = torch.randn((4, 500), generator=torch.Generator().manual_seed(1)).to(dev)
    gain = torch.ones(500, device=dev) if norm else None
    clean = pkg.quantize_rows(x, gain=gain)
    x[2, 499] = bad
    q, scale = pkg.quantize_rows(x, gain=gain)
    assert torch.isnan(scale[2]) and int(q[2].abs().max()) == 0
    for i in (0, 1, 3):
        assert torch.equal(q[i], clean[0][i]) and scale[i] == clean[1][i]


# ------------------------------------------------------------------ product
def _operands(n, N, K, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    if kind == "normal":
        a = torch.round(torch.randn((n, K), generator=g) * 36).clamp(-127, 127).to(torch.int8)
        w = torch.round(torch.randn((N, K), generator=g) * 32).clamp(-127, 127).to(torch.int8)
    elif kind == "all":  # every value of the type, -128 among them
        a = torch.randint(-128, 128, (n, K), generator=g).to(torch.int8)
        w = torch.randint(-128, 128, (N, K), generator=g).to(torch.int8)
    else:  # the largest sums there are
        a = torch.full((n, K), -128, dtype=torch.int8)
        w = torch.full((N, K), -128, dtype=torch.int8)
        w[1::2] = 127
    sa = torch.rand((n,), generator=g) + 0.5
    sw = (torch.rand((N,), generator=g) + 0.5) * 1e-3
    return [t.to(_dev()) for t in (a, sa, w, sw)]


def _exact(a, sa, w, sw):
    s = a.double() @ w.double().t()
    return s, s * sa.double()[:, None] * sw.double()[None]


def _check(out, a, sa, w, sw, K):
    """Sums are exact while their running value stays below 2^24; beyond, each of at most K additions rounds or
    truncates by 2^-23 of it. Two products and the conversion round once each (2^-24), bf16 once more (7 stored bits: 2^-8)."""
    s, want = _exact(a, sa, w, sw)
    run = (a.double().abs() @ w.double().abs().t())
    tol = torch.where(run < 2.0 ** 24, torch.zeros_like(run), run * K * 2.0 ** -23)
    tol = tol * sa.double()[:, None] * sw.double()[None] + want.abs() * 4 * 2.0 ** -24
    if out.dtype == torch.bfloat16:
        tol = tol + want.abs() * 2.0 ** -8 * (1 + 2.0 ** -20)
    off = (out.double() - want).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


SIZES = [(1, 1, 1), (1, 128, 128), (2, 3, 5), (3, 129, 127), (5, 1025, 64), (7, 1025, 1000), (8, 8200, 1024), (16, 257, 2048),
         (17, 300, 129), (33, 1025, 512), (64, 2000, 1024), (100, 513, 300), (128, 1025, 256), (129, 1025, 256),
         (255, 640, 384), (256, 1025, 1024), (257, 1025, 1024), (600, 700, 640), (1030, 1025, 96)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,N,K", SIZES)
def test_linear_i8(n, N, K, dtype):
    a, sa, w, sw = _operands(n, N, K, n + N + K)
    st = torch.zeros(1, dtype=torch.int32, device=_dev())
    out = pkg.linear_i8(a, sa, pkg.pack_i8(w, sw), dtype=DT[dtype], d_status=st)
    _check(out, a, sa, w, sw, K)
    assert int(st.item()) == 0


@pytest.mark.parametrize("n,N,K,kind", [(5, 300, 700, "all"), (40, 300, 1040, "all"), (200, 300, 4097, "all"),
                                        (5, 130, 1000, "largest"), (70, 130, 5000, "largest"),
                                        (300, 256, 1024, "largest")])
def test_linear_i8_extremes(n, N, K, kind):
    a, sa, w, sw = _operands(n, N, K, 3, kind)
    out = pkg.linear_i8(a, sa, pkg.pack_i8(w, sw), dtype=torch.float32)
    _check(out, a, sa, w, sw, K)


@pytest.mark.parametrize("n", [1, 6, 40, 150, 300])
def test_linear_i8_many_channel_blocks(n):
    """More channel blocks than the GPU has SMs, so that a CTA takes several."""
    a, sa, w, sw = _operands(n, 41000, 192, 11)
    out = pkg.linear_i8(a, sa, pkg.pack_i8(w, sw), dtype=torch.float32)
    _check(out, a, sa, w, sw, 192)


@pytest.mark.parametrize("n,N,K", [(24, 41000, 2048), (48, 41000, 2048), (200, 25000, 1500), (300, 25000, 1100),
                                   (9, 25000, 4224)])
def test_linear_i8_many_blocks_each_way(n, N, K):
    """Each ring of shared and tensor memory wraps many times, with few and many slots."""
    a, sa, w, sw = _operands(n, N, K, 12)
    out = pkg.linear_i8(a, sa, pkg.pack_i8(w, sw), dtype=torch.float32)
    _check(out, a, sa, w, sw, K)


@pytest.mark.parametrize("n,N,K", [(130, 25000, 640), (256, 41000, 300), (200, 20011, 1500), (777, 20100, 640),
                                   (1939, 8300, 256), (330, 129, 2100)])
def test_linear_i8_wide_tiles(n, N, K):
    """Row tiles above 128, bf16: several tiles for each pair of CTAs, an odd number of channel blocks, ragged ends."""
    a, sa, w, sw = _operands(n, N, K, 13)
    out = pkg.linear_i8(a, sa, pkg.pack_i8(w, sw))
    _check(out, a, sa, w, sw, K)


@pytest.mark.parametrize("n", [2, 140])
def test_linear_i8_longest_sum(n):
    a, sa, w, sw = _operands(n, 130, 131071, 14)
    out = pkg.linear_i8(a, sa, pkg.pack_i8(w, sw), dtype=torch.float32)
    _check(out, a, sa, w, sw, 131071)


def test_linear_i8_offsets_beyond_32_bits():
    """Results of more than 2^32 bytes and 2^31 elements: the last rows are those of a call of their own."""
    a, sa, w, sw = _operands(8800, 248320, 64, 15)
    weight = pkg.pack_i8(w, sw)
    out = pkg.linear_i8(a, sa, weight)
    assert out.numel() > 2 ** 31
    for i in (0, 4300, 8650):
        assert torch.equal(out[i:i + 150], pkg.linear_i8(a[i:i + 150], sa[i:i + 150], weight))
        _check(out[i:i + 150], a[i:i + 150], sa[i:i + 150], w, sw, 64)


@pytest.mark.parametrize("n,N,K,pa,pw,po", [(3, 200, 100, 1, 3, 5), (20, 200, 100, 28, 0, 1), (140, 333, 129, 7, 7, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_i8_strides(n, N, K, pa, pw, po, dtype):
    """Operands and results whose rows lie apart, at odd addresses; what lies between them is left alone."""
    dev = _dev()
    a, sa, w, sw = _operands(n, N, K, 5)
    ab = torch.full((n * (K + pa) + 1,), 77, dtype=torch.int8, device=dev)
    av = ab[1:].view(n, K + pa)[:, :K]
    av.copy_(a)
    wb = torch.full((N * (K + pw) + 3,), 77, dtype=torch.int8, device=dev)
    wv = wb[3:].view(N, K + pw)[:, :K]
    wv.copy_(w)
    ob = torch.full((n * (N + po) + 1,), 5.0, dtype=DT[dtype], device=dev)
    ov = ob[1:].view(n, N + po)
    out = pkg.linear_i8(av, sa, pkg.pack_i8(wv, sw), out=ov[:, :N])
    _check(out, a, sa, w, sw, K)
    assert bool((ov[:, N:] == 5.0).all()) and float(ob[0]) == 5.0


def test_linear_i8_repeats_and_streams():
    """One packed weight used from two streams at once; equal inputs give equal bits."""
    a, sa, w, sw = _operands(50, 3000, 768, 21)
    b, sb, _, _ = _operands(13, 3000, 768, 22)
    p = pkg.pack_i8(w, sw)
    want = pkg.linear_i8(a, sa, p), pkg.linear_i8(b, sb, p)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        got.append((pkg.linear_i8(a, sa, p, stream=s[0]), pkg.linear_i8(b, sb, p, stream=s[1])))
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


def test_linear_i8_scale_that_is_not_finite_stays_in_its_row():
    a, sa, w, sw = _operands(20, 300, 256, 31)
    p = pkg.pack_i8(w, sw)
    want = pkg.linear_i8(a, sa, p)
    sa[7] = math.nan
    out = pkg.linear_i8(a, sa, p)
    assert bool(torch.isnan(out[7]).all())
    assert torch.equal(out[:7], want[:7]) and torch.equal(out[8:], want[8:])


def test_empty_calls():
    dev = _dev()
    _, _, w, sw = _operands(1, 10, 20, 1)
    out = pkg.linear_i8(torch.empty((0, 20), dtype=torch.int8, device=dev), torch.empty(0, device=dev),
                        pkg.pack_i8(w, sw))
    assert tuple(out.shape) == (0, 10)
    q, s = pkg.quantize_rows(torch.empty((0, 20), device=dev))
    assert tuple(q.shape) == (0, 20) and s.numel() == 0


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("n,N,K", [(1, 1025, 512), (9, 4097, 768), (150, 1025, 1024)])
def test_head_close_to_the_unquantised_product(n, N, K):
    """Each operand is off by at most half a step of amax / 127 uniformly, so a logit's error is about
    sqrt(K) * (rms of the other operand) * step / sqrt(12) for each; eight times that covers the largest of them."""
    dev = _dev()
    g = torch.Generator().manual_seed(n)
    h = torch.randn((n, K), generator=g).to(torch.bfloat16).to(dev)
    W = (torch.randn((N, K), generator=g) / math.sqrt(K)).to(dev)
    gain = (1 + 0.1 * torch.randn((K,), generator=g)).to(dev)
    head = pkg.Int8Head.from_weight(W, gain=gain)
    out = head.logits(h, dtype=torch.float32).double()
    y = h.double()
    y = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6) * gain.double()
    want = y @ W.double().t()
    step_y = y.abs().amax(1, keepdim=True) / 127
    step_w = W.double().abs().amax(1)[None] / 127
    rms = lambda t: t.double().square().mean(1).sqrt()  # noqa: E731
    sd = math.sqrt(K / 12) * (step_y * rms(W)[None] + rms(y)[:, None] * step_w)
    assert float(((out - want).abs() / sd).max()) <= 8

    one = torch.ones(n, device=dev)
    tok, lp = head.sample(h, one * 0, one * 0)
    assert torch.equal(tok.long(), head.logits(h).float().argmax(1))
    want_lp = torch.log_softmax(head.logits(h).double(), 1).gather(1, tok.long()[:, None])[:, 0]
    assert float((lp.double() - want_lp).abs().max()) <= 1e-4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,N,K,norm", [(1, 1025, 512, True), (3, 300, 77, False), (17, 4097, 1000, True),
                                        (40, 700, 8200, True), (130, 1025, 2049, False), (300, 513, 9001, True)])
def test_head_is_quantise_then_product(n, N, K, norm, dtype):
    """One call, or quantised rows and then the product: the same bits, whatever the workspace held."""
    dev = _dev()
    g = torch.Generator().manual_seed(n + K)
    x = (torch.randn((n, K), generator=g) * 2).to(DT[dtype]).to(dev)
    if n > 2:
        x[1] = 0
        x[2, K // 2] = math.nan
    gain = (1 + 0.1 * torch.randn((K,), generator=g)).to(dev) if norm else None
    _, _, w, sw = _operands(1, N, K, 5)
    head = pkg.Int8Head(w, sw, gain=gain, eps=1e-5)
    q, scale = pkg.quantize_rows(x, gain=gain, eps=1e-5)
    want = pkg.linear_i8(q, scale, head.weight, dtype=torch.float32)
    junk = torch.full((pkg.head_i8_workspace(n, N, K) // 4 + 64,), math.nan, device=dev)
    del junk  # the next workspace is likely these bytes
    got = head.logits(x, dtype=torch.float32)
    assert torch.equal(torch.nan_to_num(got, nan=123.0), torch.nan_to_num(want, nan=123.0))
    assert bool(torch.isnan(got[2]).all()) if n > 2 else bool(torch.isfinite(got).all())


def test_head_strided_and_other_stream():
    dev = _dev()
    g = torch.Generator().manual_seed(8)
    buf = torch.randn((9, 131), generator=g).to(torch.bfloat16).to(dev)
    x = buf[:, 1:128]
    _, _, w, sw = _operands(1, 500, 127, 6)
    head = pkg.Int8Head(w, sw)
    want = head.logits(x.contiguous())
    assert torch.equal(head.logits(x), want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = head.logits(x, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_head_reports_a_bad_hidden_state():
    dev = _dev()
    g = torch.Generator().manual_seed(4)
    h = torch.randn((5, 256), generator=g).to(dev)
    head = pkg.Int8Head.from_weight(torch.randn((600, 256), generator=g).to(dev))
    h[3, 9] = math.nan
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    one = torch.ones(5, device=dev)
    tok, lp = head.sample(h, one, one * 0.5, d_status=st)
    assert int(st.item()) == pkg.DS_DEV_ERR_LOGITS
    assert int(tok[3]) == -1 and bool(torch.isnan(lp[3]))
    assert bool((tok[[0, 1, 2, 4]] >= 0).all())


def test_short_way_and_checked_way_agree():
    """Calls that make their outputs go past the interpreter, others through it: the same answers, the same refusals."""
    dev = _dev()
    n, N, K = 5, 700, 192
    a, sa, w, sw = _operands(n, N, K, 16)
    weight = pkg.pack_i8(w, sw)
    h = (torch.randn((n, K), generator=torch.Generator().manual_seed(1)) * 2).to(dev)
    head = pkg.Int8Head(w, sw, gain=torch.ones(K, device=dev))
    tau, u = torch.ones(n, device=dev), torch.arange(n, device=dev) / n
    k = torch.full((n,), 20, dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    for dtype in (torch.bfloat16, torch.float32):
        out = pkg.linear_i8(a, sa, weight, dtype=dtype)
        assert out.dtype == dtype and torch.equal(out, pkg.linear_i8(a, sa, weight, dtype=dtype, d_status=st))
        x = head.logits(h.to(dtype), dtype=dtype)
        assert x.dtype == dtype and torch.equal(x, head.logits(h.to(dtype), dtype=dtype, d_status=st))
        s = pkg.sample_filtered(x, tau, u, top_k=k)
        t = pkg.sample_filtered(x, tau, u, top_k=k, d_status=st)
        assert torch.equal(s[0], t[0]) and torch.equal(s[1], t[1]) and s[0].dtype == torch.int32
        for gain in (None, head.gain):
            q, s = pkg.quantize_rows(h.to(dtype), gain=gain, eps=1e-5)
            r = torch.empty_like(s)
            p, _ = pkg.quantize_rows(h.to(dtype), gain=gain, eps=1e-5, out_scale=r)
            assert torch.equal(q, p) and torch.equal(s, r) and q.dtype == torch.int8
    assert int(st.item()) == 0
    for bad in (dict(temperature=tau.double()), dict(temperature=tau[:4]), dict(temperature=None), dict(u=u.cpu()), dict(u=None),
                dict(u=torch.zeros((n, 2), device=dev)[:, 0]),
                dict(u=u.view(n, 1)), dict(top_k=k.long()), dict(top_p=k), dict(min_p=tau.half()), dict(logits=x.t()),
                dict(logits=x[0]), dict(logits=x.half()), dict(logits=x.cpu())):
        with pytest.raises(ValueError):
            pkg.sample_filtered(**dict(dict(logits=x, temperature=tau, u=u), **bad))
    for args in ((a.int(), sa, weight), (a[:, :100], sa, weight), (a, sa[:3], weight), (a, None, weight), (a, sa.double(), weight),
                 (a.cpu(), sa, weight)):
        with pytest.raises(ValueError):
            pkg.linear_i8(*args)
    for x in (h[:, :100], h.half(), h[0], h.cpu()):
        with pytest.raises(ValueError):
            head.logits(x)
    for x, gain in ((h.half(), None), (h[0], None), (h.t(), None), (h, sa), (h, torch.ones(K)), (h.cpu(), None)):
        with pytest.raises(ValueError):
            pkg.quantize_rows(x, gain=gain)
    with pytest.raises(ValueError):
        pkg.linear_i8(a, sa, weight, dtype=torch.float16)
