"""ds_add_adapters against the definition in 64 bits, and the serving head with adapters."""
import math
import os
import subprocess
import sys

import pytest
import torch

import vocab_wide_logit_gb300 as pkg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def _dev():
    assert torch.cuda.is_available(), "needs a GPU"
    return torch.device("cuda", 0)


def _inputs(n, N, K, R, L, dtype="f32", x_dtype="bf16", norm=False, seed=0, none=True):
    g = torch.Generator().manual_seed(seed + n + N + K + R + L)
    ids = torch.randint(-1 if none else 0, L, (n,), generator=g).to(torch.int32)
    base = (torch.randn((n, N), generator=g) * 0.01).to(DT[dtype])
    hidden = (torch.randn((n, K), generator=g) * 1.7).to(DT[x_dtype])
    gain = 1 + 0.2 * torch.randn((K,), generator=g) if norm else None
    a = (torch.randn((L, R, K), generator=g) * K ** -0.5).to(torch.bfloat16)
    b = torch.randn((L, N, R), generator=g).to(torch.bfloat16)
    scale = torch.rand((L,), generator=g) + 0.5
    to = lambda t: None if t is None else t.to(_dev())  # noqa: E731
    return to(base), to(hidden), pkg.Adapters(to(a), to(b), to(scale)), to(ids), to(gain)


def _reference(base, hidden, ad, ids, gain, eps=EPS):
    """(what is right, how far off it may be) in float64.

    t = A y: K products and their sum, K + 8 roundings of at most 2^-24 of the sum of sizes; the norm's root adds (K / 32 +
    16) / 2 of them and its products 3. As sums of bf16 parts, each off by 2^-8 of what the parts before it left, y and
    t lose 2^-16 each (two parts, bf16 logits) or 2^-24 (three, fp32 logits).
    B t: then R products, at most (3 R / 16 + 4) additions that
    each lose 2^-23 of the running size where a matrix instruction makes them and R of 2^-24 where not. The sum with base
    rounds once, and to bf16 once more (half a step, 2^-8)."""
    y = hidden.double()
    K = y.shape[1]
    down = K + 8
    if gain is not None:
        ss = (y * y).mean(1, keepdim=True) + eps
        y = torch.where(ss > 0, y / ss.clamp(min=1e-300).sqrt(), torch.zeros_like(y)) * gain.double()
        down += K / 64 + 11
    out = base.double().clone()
    size = torch.zeros_like(out)
    for i in range(ad.L):
        mine = torch.nonzero(ids == i).reshape(-1)
        if mine.numel():
            a, b, s = ad.a[i].double(), ad.b[i].double(), ad.scale[i].double()
            out[mine] += (y[mine] @ a.t() * s) @ b.t()
            size[mine] = (y[mine].abs() @ a.abs().t() * s.abs()) @ b.abs().t()
    tol = size * (down + 2 + 4 + 2 * (ad.R + 4)) * 2.0 ** -24 + out.abs() * 2.0 ** -23
    if base.dtype == torch.bfloat16:
        tol = tol + size * 2.0 ** -15 + out.abs() * 2.0 ** -8 * (1 + 2.0 ** -10)
    return out, tol


def _check(got, base, hidden, ad, ids, gain=None, eps=EPS):
    want, tol = _reference(base, hidden, ad, ids, gain, eps)
    assert got.dtype == base.dtype and got.shape == base.shape
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (int(bad.sum()), torch.nonzero(bad)[:4].tolist(), float((off / tol.clamp(min=1e-300)).max()))
    rest = ids < 0
    assert torch.equal(got[rest], base[rest])  # rows without an adapter are the base's bits


# sizes around a tile of rows, of channels, of ranks and of inputs
SIZES = [(1, 1, 1, 1, 1), (1, 1025, 64, 16, 1), (2, 3, 5, 2, 2), (3, 31, 33, 3, 2), (5, 64, 100, 4, 3), (7, 129, 127, 5, 3),
         (8, 256, 256, 8, 2), (9, 257, 1000, 7, 4), (15, 1000, 64, 16, 5), (16, 1025, 512, 16, 1), (17, 1025, 72, 17, 4),
         (24, 5003, 2048, 16, 8), (31, 640, 1024, 32, 40), (33, 513, 96, 33, 3), (64, 2000, 333, 64, 9), (65, 8200, 1024, 8, 5),
         (100, 300, 200, 100, 7), (128, 1024, 128, 128, 3), (37, 701, 1001, 13, 6), (257, 1025, 512, 24, 6), (600, 264, 160, 48, 2),
         (1939, 1025, 256, 8, 5), (40, 333, 5000, 127, 3), (1030, 77, 64, 1, 300), (4, 70001, 64, 16, 2),
         (32, 90, 40, 16, 3), (33, 90, 40, 16, 40), (8192, 33, 24, 5, 50), (8193, 33, 24, 5, 50), (20000, 17, 40, 16, 3), (30, 400, 64, 12, 3),
         (19, 1025, 64, 20, 3), (21, 600, 48, 36, 4), (18, 300, 64, 68, 3)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,N,K,R,L", SIZES)
def test_sizes(n, N, K, R, L, dtype):
    for x_dtype, norm in (("bf16", True), ("f32", False), ("bf16", False), ("f32", True)):
        base, hidden, ad, ids, gain = _inputs(n, N, K, R, L, dtype, x_dtype, norm)
        got = pkg.add_adapters(base, hidden, ad, ids, gain=gain, eps=EPS)
        _check(got, base, hidden, ad, ids, gain)


@pytest.mark.parametrize("R", [8, 16, 24, 64, 5])
def test_large_vocabulary(R):
    base, hidden, ad, ids, gain = _inputs(20, 248320, 256, R, 3, "bf16", norm=True)
    _check(pkg.add_adapters(base, hidden, ad, ids, gain=gain, eps=EPS), base, hidden, ad, ids, gain)


@pytest.mark.parametrize("kind", ["one", "none", "own", "runs", "last", "even"])
@pytest.mark.parametrize("n", [1, 16, 17, 50, 300])
def test_orders_of_ids(kind, n):
    L = 300 if kind == "own" else 4
    base, hidden, ad, ids, _ = _inputs(n, 530, 200, 16, L, none=False)
    row = torch.arange(n, device=_dev())
    ids.copy_({"one": row * 0 + 2, "none": row * 0 - 1, "own": row, "runs": row * 4 // n, "last": torch.where(row == n - 1, 3, -5),
               "even": torch.where(row % 2 == 0, 1, -1)}[kind])
    _check(pkg.add_adapters(base, hidden, ad, ids), base, hidden, ad, ids)


def test_most_adapters():
    L = pkg.DS_ADAPTERS_MAX
    base, hidden, ad, ids, _ = _inputs(700, 40, 24, 2, L)
    ids[:5] = torch.tensor([L - 1, 0, L - 1, -1, L - 2], dtype=torch.int32)
    want, tol = base.double(), None
    got = pkg.add_adapters(base, hidden, ad, ids)
    q = ids.long().clamp(min=0)
    t = (ad.a[q].double() @ hidden.double()[:, :, None])[:, :, 0] * ad.scale[q].double()[:, None]
    delta = (ad.b[q].double() @ t[:, :, None])[:, :, 0]
    size = (ad.b[q].double().abs() @ ((ad.a[q].double().abs() @ hidden.double().abs()[:, :, None])[:, :, 0] *
                                      ad.scale[q].double()[:, None])[:, :, None])[:, :, 0]
    want = base.double() + torch.where(ids[:, None] >= 0, delta, torch.zeros_like(delta))
    tol = size * (24 + 8 + 2 + 4 + 2 * 6) * 2.0 ** -24 + want.abs() * 2.0 ** -23  # as in _reference()
    assert bool(((got.double() - want).abs() <= tol).all())


def test_bad_ids_and_rows():
    base, hidden, ad, ids, _ = _inputs(40, 333, 64, 8, 5, none=False)
    ids[3], ids[20], ids[21] = 5, 2 ** 31 - 1, -(2 ** 31)
    hidden[7, 5], hidden[8, 63], hidden[9, 0] = math.nan, math.inf, -math.inf
    hidden[21, 1] = math.nan  # no adapter: not looked at
    status = torch.zeros(1, dtype=torch.int32, device=_dev())
    for gain in (None, torch.ones(64, device=_dev())):
        status.zero_()
        got = pkg.add_adapters(base, hidden, ad, ids, gain=gain, eps=EPS, d_status=status)
        assert int(status) == pkg.DS_DEV_ERR_PARAM
        bad = torch.tensor([3, 20, 7, 8, 9], device=_dev())
        assert bool(got[bad].isnan().all())
        good = torch.ones(40, dtype=torch.bool, device=_dev())
        good[bad] = False
        _check(got[good], base[good], torch.where(torch.isfinite(hidden), hidden, torch.zeros_like(hidden))[good], ad,
               ids[good], gain)


def test_values_that_are_not_finite_stay_where_they_are():
    """An infinite or NaN weight or logit reaches its own logits alone."""
    base, hidden, ad, ids, _ = _inputs(20, 200, 64, 8, 3, none=False)
    ids[:] = torch.arange(20, device=_dev()) % 3
    base[4, 7], base[5, 8] = -math.inf, math.nan
    clean = pkg.add_adapters(base, hidden, ad, ids)
    ad.b[1, 50, 3] = math.nan
    ad.b[1, 51, 7] = math.inf
    got = pkg.add_adapters(base, hidden, ad, ids)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[1::3, 50:52] = True
    assert bool((~torch.isfinite(got[hit])).all())
    same = (got == clean) | (got.isnan() & clean.isnan())
    assert bool(same[~hit].all())
    assert float(got[4, 7]) == -math.inf and bool(got[5, 8].isnan())


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e18, 1e30])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("x_dtype,n", [("f32", 20), ("bf16", 20), ("bf16", 50)])
def test_norm_of_small_and_large_rows(x_dtype, n, scale, eps):
    """Squares that leave fp32's range; a row of zeros."""
    base, hidden, ad, ids, gain = _inputs(n, 100, 128, 8, 2, x_dtype=x_dtype, norm=True, none=False)
    hidden *= scale
    hidden[3] = 0
    got = pkg.add_adapters(base, hidden, ad, ids, gain=gain, eps=eps)
    _check(got, base, hidden, ad, ids, gain, eps)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,pads,offset", [(1025, (0, 0, 0), 1), (1000, (8, 3, 16), 0), (1000, (1, 5, 3), 3), (264, (8, 8, 8), 8)])
def test_strides(N, pads, offset, dtype):
    n, K = 21, 96
    base, hidden, ad, ids, _ = _inputs(n, N, K, 16, 3, dtype)

    def spread(t, columns, pad):
        buf = torch.full((n * (columns + pad) + offset + 7,), 7.0, dtype=t.dtype, device=_dev())
        view = buf[offset:offset + n * (columns + pad)].view(n, columns + pad)[:, :columns]
        view.copy_(t)
        return buf, view

    _, b = spread(base, N, pads[0])
    _, h = spread(hidden, K, pads[1])
    obuf, out = spread(base, N, pads[2])
    assert pkg.add_adapters(b, h, ad, ids, out=out) is out
    _check(out.contiguous(), base, hidden, ad, ids)
    same = out.clone()
    out.zero_()
    assert float((obuf == 7.0).sum()) == offset + 7 + n * pads[2]
    bbuf, b = spread(base, N, pads[0])
    pkg.add_adapters(b, h, ad, ids, out=b)  # in place
    _check(b.contiguous(), base, hidden, ad, ids)
    assert torch.equal(b.contiguous(), same)
    b.zero_()
    assert float((bbuf == 7.0).sum()) == offset + 7 + n * pads[0]


@pytest.mark.parametrize("R", [5, 8, 16, 32, 40, 128])
@pytest.mark.parametrize("behind", [1, 2, 4])
def test_misaligned_adapters(R, behind):
    """Stacks that start 2, 4 or 8 bytes behind a 16-byte boundary."""
    base, hidden, ad, ids, _ = _inputs(20, 300, 72, R, 3)
    shifted = []
    for t in (ad.a, ad.b):
        buf = torch.empty(t.numel() + behind, dtype=t.dtype, device=_dev())
        shifted.append(buf[behind:].view(t.shape))
        shifted[-1].copy_(t)
    got = pkg.add_adapters(base, hidden, pkg.Adapters(*shifted, ad.scale), ids)
    _check(got, base, hidden, ad, ids)


def test_offsets_beyond_32_bits():
    n, N, ld = 3, 1000, 2 ** 31 - 9
    base, hidden, ad, ids, _ = _inputs(n, N, 64, 8, 2, "bf16", none=False)
    buf = torch.empty(2 * ld + N, dtype=torch.bfloat16, device=_dev())
    far = buf.as_strided((n, N), (ld, 1))
    far.copy_(base)
    pkg.add_adapters(far, hidden, ad, ids, out=far)
    _check(far.contiguous(), base, hidden, ad, ids)
    # a stack of more than 2^32 elements
    L, N, R = 70, 500000, 128
    b = torch.empty((L, N, R), dtype=torch.bfloat16, device=_dev())
    a = torch.randn((L, R, 16), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(_dev())
    b[L - 1].normal_(generator=torch.Generator(_dev()).manual_seed(2))
    base = torch.zeros((2, N), device=_dev())
    hidden = torch.randn((2, 16), device=_dev())
    ids = torch.tensor([-1, L - 1], dtype=torch.int32, device=_dev())
    got = pkg.add_adapters(base, hidden, pkg.Adapters(a, b, torch.ones(L, device=_dev())), ids)
    one = pkg.Adapters(a[L - 1:], b[L - 1:], torch.ones(1, device=_dev()))
    _check(got, base, hidden, one, torch.where(ids < 0, -1, 0).to(torch.int32))


def test_a_row_in_other_batches():
    """A row's result does not depend on the rows beside it, nor on the order of the call's work: bit for bit."""
    for R, dtype, norm in ((24, "f32", True), (16, "f32", True), (12, "bf16", True), (16, "bf16", False)):
        _other_batches(*_inputs(400, 2003, 320, R, 40, dtype, norm=norm))


def _other_batches(base, hidden, ad, ids, gain):
    whole = pkg.add_adapters(base, hidden, ad, ids, gain=gain, eps=EPS)
    for i, n in ((0, 1), (5, 20), (100, 33), (0, 300), (0, 400)):
        part = pkg.add_adapters(base[i:i + n], hidden[i:i + n], ad, ids[i:i + n], gain=gain, eps=EPS)
        assert torch.equal(part, whole[i:i + n])
    many = [t.repeat(21, 1) for t in (base, hidden)]  # more rows than the down kernel's CTAs plan for themselves
    got = pkg.add_adapters(*many, ad, ids.repeat(21), gain=gain, eps=EPS)
    assert torch.equal(got, whole.repeat(21, 1))


def test_slots_are_read_at_the_call():
    """A program rewrites a slot in place: nothing is kept of what was there."""
    base, hidden, ad, ids, _ = _inputs(10, 500, 64, 16, 2, none=False)
    pkg.add_adapters(base, hidden, ad, ids)
    ad.a[1].normal_()
    ad.b[1].normal_()
    ad.scale[1] = 3
    _check(pkg.add_adapters(base, hidden, ad, ids), base, hidden, ad, ids)


def test_streams_and_graphs():
    """Two captured graphs and an eager call at once, each with a workspace of its own; replayed on new inputs."""
    ad = _inputs(1, 3000, 128, 16, 6)[2]
    sides = []
    for seed in (1, 2):
        base, hidden, _, ids, gain = _inputs(40, 3000, 128, 16, 6, norm=True, seed=seed)
        pkg.add_adapters(base, hidden, ad, ids, gain=gain, eps=EPS)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = pkg.add_adapters(base, hidden, ad, ids, gain=gain, eps=EPS)
        sides.append((graph, base, hidden, ids, gain, out, torch.cuda.Stream()))
    for k, (_, base, hidden, ids, *_) in enumerate(sides):
        b, h, _, i, _ = _inputs(40, 3000, 128, 16, 6, norm=True, seed=20 + k)
        base.copy_(b)
        hidden.copy_(h)
        ids.copy_(i)
    torch.cuda.synchronize()
    eager = torch.cuda.Stream()
    for _ in range(4):
        for graph, *_, stream in sides:
            with torch.cuda.stream(stream):
                graph.replay()
        got = pkg.add_adapters(sides[0][1], sides[1][2], ad, sides[0][3], gain=sides[0][4], eps=EPS, stream=eager)
    torch.cuda.synchronize()
    for _, base, hidden, ids, gain, out, _ in sides:
        _check(out, base, hidden, ad, ids, gain)
    _check(got, sides[0][1], sides[1][2], ad, sides[0][3], sides[0][4])


def test_no_rows():
    ad = _inputs(1, 50, 16, 4, 2)[2]
    out = pkg.add_adapters(torch.empty((0, 50), device=_dev()), torch.empty((0, 16), device=_dev()), ad,
                           torch.empty(0, dtype=torch.int32, device=_dev()))
    assert out.shape == (0, 50)


def test_both_ways_of_a_call():
    status = torch.zeros(1, dtype=torch.int32, device=_dev())
    for dtype, x_dtype, norm in (("bf16", "bf16", True), ("f32", "f32", False)):
        base, hidden, ad, ids, gain = _inputs(9, 700, 64, 8, 3, dtype, x_dtype, norm)
        assert torch.equal(pkg.add_adapters(base, hidden, ad, ids, gain=gain, eps=EPS),
                           pkg.add_adapters(base, hidden, ad, ids, gain=gain, eps=EPS, d_status=status))
    for bad in (dict(ids=None), dict(ids=ids.long()), dict(ids=ids[:8]), dict(ids=ids.cpu()), dict(hidden=hidden[:, :63]),
                dict(hidden=hidden[:8]), dict(base=base[:, :699]), dict(base=base.half()), dict(gain=torch.ones(63, device=_dev()))):
        with pytest.raises(ValueError):
            pkg.add_adapters(**{**dict(base=base, hidden=hidden, adapters=ad, ids=ids), **bad})


def test_c_name():
    base, hidden, ad, ids, gain = _inputs(9, 700, 64, 8, 3, norm=True)
    out = torch.empty_like(base)
    ws = torch.empty(pkg.add_adapters_workspace(9, 3, 8), dtype=torch.uint8, device=_dev())
    pkg.ds_add_adapters(base, hidden, ad.a, ad.b, ad.scale, ids, out, ws, gain=gain, eps=EPS)
    assert torch.equal(out, pkg.add_adapters(base, hidden, ad, ids, gain=gain, eps=EPS))


# ------------------------------------------------------------------ together, as a serving head runs them
def _head(N, K, seed=3):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn((N, K), generator=g) * 3 * K ** -0.5).to(_dev())
    return pkg.Int8Head.from_weight(w, gain=(1 + 0.1 * torch.randn((K,), generator=g)).to(_dev()), eps=EPS)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_with_adapters(dtype):
    n, N, K = 24, 5003, 512
    head = _head(N, K)
    _, hidden, ad, ids, _ = _inputs(n, N, K, 16, 4)
    plain = head.logits(hidden, dtype=DT[dtype])
    got = head.logits(hidden, dtype=DT[dtype], adapters=ad, adapter_ids=ids)
    _check(got, plain, hidden, ad, ids, head.gain)
    out = torch.empty_like(got)
    assert head.logits(hidden, out=out, adapters=ad, adapter_ids=ids, stream=torch.cuda.current_stream()) is out
    assert torch.equal(out, got)
    assert torch.equal(head.logits(hidden, dtype=DT[dtype]), plain)


def test_head_samples_and_scores():
    """Hidden states through head and adapters to tokens, the tokens to scores, the scores to a gradient."""
    n, N, K = 16, 2000, 256
    head = _head(N, K)
    _, hidden, ad, ids, _ = _inputs(n, N, K, 8, 4)
    g = torch.Generator().manual_seed(2)
    u, tau = torch.rand((n,), generator=g).to(_dev()), torch.ones(n, device=_dev())
    status = torch.zeros(1, dtype=torch.int32, device=_dev())
    logits = head.logits(hidden, adapters=ad, adapter_ids=ids)
    tokens, logprobs = head.sample(hidden, tau, u, adapters=ad, adapter_ids=ids, d_status=status)
    want = pkg.sample_filtered(logits, tau, u)
    assert torch.equal(tokens, want[0]) and torch.equal(logprobs, want[1])
    r = head.score(hidden, tokens, top=3, adapters=ad, adapter_ids=ids, d_status=status)
    # two fp32 evaluations of one real number: each within 2000 / 256 + 300 roundings of it (see test_score_gpu.py)
    assert float((r.logprobs - logprobs).abs().max()) < 2 * 310 * 2.0 ** -24 + 4 * 12 * 2.0 ** -23
    for a, b in zip(r, pkg.score_tokens(logits, tokens, top=3)):
        assert torch.equal(a, b)
    dx = pkg.score_tokens_grad(logits, tokens, r.lse, g_logprobs=torch.ones(n, device=_dev()))
    # a row of one-hot minus p: its sum is 0 but for the bf16 rounding of each term, sizes adding up to 2 at most
    assert float(dx.double().sum(1).abs().max()) <= 2 * 2.0 ** -8
    assert int(status) == 0


def test_example_with_adapters_and_alternatives():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "next_token.py"), "--rows", "9", "--vocab", "3001",
                        "--hidden", "128", "--steps", "2", "--adapters", "3", "--alternatives", "4"], capture_output=True,
                       text=True, timeout=240)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("step ") == 2 and r.stdout.count("alternatives") == 2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [64, 333, 1001])
@pytest.mark.parametrize("R", [65, 72, 95, 96, 97])
def test_ranks_that_fill_up_to_128(R, K, dtype):
    """The last block of 32 ranks has none of R's (but of 97); the last adapter of the stack in use, stacks at a boundary of 16
    bytes and 2 bytes behind one. What lies behind the stack is in no result."""
    for n in (5, 40):
        base, hidden, ad, ids, gain = _inputs(n, 130, K, R, 2, dtype, norm=True, none=False)
        ids[0] = 1
        for behind in (0, 1):
            buf = torch.full((ad.a.numel() + behind + 64 * K,), math.nan, dtype=torch.bfloat16, device=_dev())
            a = buf[behind:behind + ad.a.numel()].view(ad.a.shape)
            a.copy_(ad.a)
            moved = pkg.Adapters(a, ad.b, ad.scale)
            _check(pkg.add_adapters(base, hidden, moved, ids, gain=gain, eps=EPS), base, hidden, moved, ids, gain)
