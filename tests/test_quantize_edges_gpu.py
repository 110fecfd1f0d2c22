"""ds_quantize_rows and the head where fp32's range ends: rows close to zero, squares that leave the range, no eps, and
rows of nearly 2^31 elements."""
import math

import pytest
import torch

import vocab_wide_logit_gb300 as pkg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
STEP = 2.0 ** -149  # the smallest fp32 number: what a scale below 2^-126 is rounded to a multiple of


def _check(x, gain, eps, q, scale):
    """The definition in 64 bits. fp32 arithmetic: 16 roundings of 2^-24 at most, so 127 * 16 * 2^-24 = 1.3e-4 of a step
    beside the half that rounding to an integer may take; a row whose y lies below 2^-126 has further errors of one STEP for each
    of three products, 127 * 3 of them in the largest."""
    y = x.double()
    if gain is not None:
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
        y = torch.where(x.double().abs().amax(1, keepdim=True) > 0, y, torch.zeros_like(y)) * gain.double()
    amax = y.abs().amax(1, keepdim=True)
    real = torch.where(amax > 0, y * 127 / amax, torch.zeros_like(y))
    room = torch.where(amax > 0, 0.5 + 2e-4 + (6 * 127 * STEP / amax if gain is not None else 0.0), torch.zeros_like(amax))
    assert int(q.abs().max()) <= 127
    assert bool(((q.double() - real).abs() <= room).all())
    want = amax[:, 0] / 127
    assert bool(((scale.double() - want).abs() <= want * 16 * 2.0 ** -24 + STEP * (4 if gain is not None else 0.5)).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [5, 64, 1000, 8192, 20001])
@pytest.mark.parametrize("norm", [False, True])
def test_rows_close_to_zero(K, dtype, norm):
    """127 / max|y| is beyond fp32 below 3.7e-37."""
    dev = torch.device("cuda", 0)
    sizes = [1e-36, 3.7e-37, 3e-37, 1e-37, 1e-38, 2e-39, 1e-41, 3e-44]
    x = torch.randn((len(sizes), K), generator=torch.Generator().manual_seed(K))
    x = x / x.abs().amax(1, keepdim=True) * torch.tensor(sizes, dtype=torch.float64)[:, None]
    x = x.to(DT[dtype]).to(dev)
    assert bool((x.abs().amax(1) > 0).all()) or dtype == "bf16"  # whose smallest number is 9e-41: the last two rows are zeros
    gain = (1 + 0.2 * torch.randn((K,), generator=torch.Generator().manual_seed(1))).to(dev) if norm else None
    eps = 1.0 if norm else 0.0  # y is then x times the gain
    q, scale = pkg.quantize_rows(x, gain=gain, eps=eps)
    _check(x, gain, eps, q, scale)
    head = pkg.Int8Head(torch.eye(K, dtype=torch.int8, device=dev)[:64].contiguous(), torch.ones(min(K, 64), device=dev),
                        gain=gain, eps=eps)
    assert torch.equal(head.logits(x, dtype=torch.float32), q[:, :64].float() * scale[:, None])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [5, 64, 1000, 8192, 20001])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-38, 9e-38, 1e-6, 3e38])
def test_norm_of_rows_whose_squares_leave_the_range(K, eps, dtype):
    """A row of zeros without eps, squares below 2^-126 and above 2^128, and a sum of them that passes 2^128 with eps."""
    dev = torch.device("cuda", 0)
    sizes = [0.0, 1e-44, 1e-40, 1e-38, 1e-30, 1e-22, 1e-19, 1e-18, 1.0, 1e18, 1.7e19, 3e19, 1e25, 1e38, 3e38]
    x = torch.randn((len(sizes), K), generator=torch.Generator().manual_seed(K))
    x = x / x.abs().amax(1, keepdim=True) * torch.tensor(sizes, dtype=torch.float64)[:, None]
    x[12, 1:] *= 1e-40  # one large value among small ones
    x = x.to(DT[dtype]).to(dev)
    gain = (1 + 0.2 * torch.randn((K,), generator=torch.Generator().manual_seed(1))).to(dev)
    q, scale = pkg.quantize_rows(x, gain=gain, eps=eps)
    _check(x, gain, float(torch.tensor(eps)), q, scale)  # the fp32 number that the call takes: 1e-44 is 9.8e-45
    assert float(scale[0]) == 0 and int(q[0].abs().max()) == 0
    w = torch.ones((3, K), dtype=torch.int8, device=dev)
    head = pkg.Int8Head(w, torch.ones(3, device=dev), gain=gain, eps=eps)
    assert torch.equal(head.logits(x, dtype=torch.float32),
                       pkg.linear_i8(q, scale, head.weight, dtype=torch.float32))
    x[3, K - 1], x[13, 0] = math.nan, math.inf
    q2, scale2 = pkg.quantize_rows(x, gain=gain, eps=eps)
    keep = [i for i in range(len(sizes)) if i not in (3, 13)]
    assert torch.equal(q2[keep], q[keep]) and torch.equal(scale2[keep], scale[keep])
    assert bool(torch.isnan(scale2[[3, 13]]).all()) and int(q2[[3, 13]].abs().max()) == 0


def test_the_longest_row():
    """2^31 - 1 elements: the chunk behind the last one starts at 2^31."""
    dev, K = torch.device("cuda", 0), 2 ** 31 - 1
    x = torch.empty((1, K), dtype=torch.bfloat16, device=dev)
    parts = [slice(i, min(i + (1 << 28), K)) for i in range(0, K, 1 << 28)]
    for i, p in enumerate(parts):
        x[0, p].normal_(0, 1 + i, generator=torch.Generator(device=dev).manual_seed(i))
    x[0, K - 1] = 100.0  # the largest, and the last
    q, scale = pkg.quantize_rows(x)
    assert int(q[0, K - 1]) == 127 and float(scale[0]) == float(torch.tensor(100.0) / 127)
    for p in parts:  # half a step, and the 16 roundings that _check allows
        assert float((q[0, p].float() * (100 / 127) - x[0, p].float()).abs().max()) <= (0.5 + 2e-4) * 100 / 127 * (1 + 1e-6)
    one = torch.ones(K, device=dev)
    qn, sn = pkg.quantize_rows(x, gain=one, eps=0.0)
    rms = (sum(float(x[0, p].double().square().sum()) for p in parts) / K) ** 0.5
    # a thread adds 2^23 squares in turn, each addition off by 2^-24 of its running sum at most, which is half of
    # the whole in the mean: 2^23 2^-24 / 2 = 1/4 of the sum at worst, 0.16 of its root
    assert abs(float(sn[0]) / (100.0 / 127 / rms) - 1) <= 0.16
    assert int(qn[0, K - 1]) == 127
