"""ds_linear_i8's sums: exact while the running sum stays below 2^24, however much its terms would add up to without their
signs, and beyond within a bound that zeros would not meet."""
import pytest
import torch

import vocab_wide_logit_gb300 as pkg

pytestmark = pytest.mark.gpu


def _dev():
    return torch.device("cuda", 0)


def _sums(a, w):
    """The sums, and the largest magnitude that the running sum of the first 16, 32, ... inputs takes: below 2^31, so
    exact in 64 bits."""
    a, w = a.double(), w.double()
    total = torch.zeros((a.shape[0], w.shape[0]), dtype=torch.float64, device=a.device)
    most = torch.zeros_like(total)
    for k in range(0, a.shape[1], 16):
        total += a[:, k:k + 16] @ w[:, k:k + 16].t()
        most = torch.maximum(most, total.abs())
    return total, most


def _product(a, w):
    n, N = a.shape[0], w.shape[0]
    one = torch.ones(n, device=a.device), torch.ones(N, device=a.device)
    return pkg.linear_i8(a, one[0], pkg.pack_i8(w, one[1]), dtype=torch.float32).double()


@pytest.mark.parametrize("n,N,K", [(2, 130, 131071), (140, 130, 131071), (5, 300, 5001), (200, 300, 4097),
                                   (40, 41000, 1040), (300, 256, 20000)])
def test_sums_that_stay_below_2_24_are_exact(n, N, K):
    """Signed operands of every size. A step adds the products of 16 inputs, so a running sum below 2^24 less 16 * 2^14
    is exact at every step in between too."""
    g = torch.Generator().manual_seed(K + n)
    a = torch.round(torch.randn((n, K), generator=g) * 36).clamp(-127, 127).to(torch.int8).to(_dev())
    w = torch.round(torch.randn((N, K), generator=g) * 32).clamp(-127, 127).to(torch.int8).to(_dev())
    want, most = _sums(a, w)
    exact = most < 2.0 ** 24 - 2.0 ** 18
    assert bool(exact.all())
    got = _product(a, w)
    assert torch.equal(got, want)
    assert float(want.abs().max()) > 1e4  # zeros would not do


@pytest.mark.parametrize("n", [2, 40, 140])
@pytest.mark.parametrize("K", [1040, 1041, 1056, 5000, 131071])
def test_sums_beyond_2_24(n, K):
    """Products of one sign, the largest there are. From 2^24 on each step of 16 inputs may drop what lies below the
    spacing of the running sum: less than 2^-23 of it, and not more often than K / 16 times."""
    a = torch.full((n, K), 127, dtype=torch.int8, device=_dev())
    w = torch.full((130, K), 127, dtype=torch.int8, device=_dev())
    a[1::2] = -128
    w[1::2] = 125
    w[2::3] = -128
    want, most = _sums(a, w)
    off = (_product(a, w) - want).abs()
    bound = torch.where(most < 2.0 ** 24, torch.zeros_like(most), most * (K / 16 + 1) * 2.0 ** -23)
    assert bool((off <= bound).all())
    assert float((bound / want.abs()).max()) <= 1e-3  # zeros would not do
