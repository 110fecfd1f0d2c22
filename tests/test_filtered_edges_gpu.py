"""ds_sample_filtered where a shortcut could go wrong: rows with a few allowed tokens, flat rows, very long ones."""
import math

import numpy as np
import pytest
import torch

import vocab_wide_logit_gb300 as pkg
from test_filtered_gpu import DT, _check_real, _dev, _integer_definition, _logits, _params, _run

pytestmark = pytest.mark.gpu


def _sparse(n, V, allowed, seed, dtype, low):
    """Rows with a few allowed tokens next to each other, at a place of each row's own, and the rest masked."""
    g = torch.Generator().manual_seed(seed)
    x = torch.full((n, V), low)
    at = torch.randint(0, V - allowed, (n, 1), generator=g) + torch.arange(allowed)[None]
    return x.scatter_(1, at, torch.randn((n, allowed), generator=g) * 2).to(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V", [(160, 20000), (160, 80000), (100, 200003)])
@pytest.mark.parametrize("allowed", [1, 5, 20])
def test_rows_whose_sample_holds_no_logit(n, V, allowed, dtype):
    """Enough long rows that each gets a CTA, which samples a part of its row first: most of the allowed tokens lie
    outside it, so that the row goes to the second pass without a cut. Every top-k up to and beyond its lists."""
    for low in (-math.inf, float(torch.finfo(DT[dtype]).min)):
        x = _sparse(n, V, allowed, V + allowed, DT[dtype], low).to(_dev())
        g = np.random.Generator(np.random.PCG64(allowed))
        tau = g.choice(np.array([0.0, 0.7, 1.0, 1.0], np.float32), n)
        k = g.choice(np.array([0, 1, 3, 50, 128, 129, 300], np.int32), n)
        p = g.choice(np.array([1.0, 0.9, 0.5], np.float32), n)
        mp = g.choice(np.array([0.0, 0.0, 0.05], np.float32), n)
        u = g.random(n, dtype=np.float32)
        tok, lp = _run(x, tau, k, p, mp, u)
        assert np.array_equal(tok, _integer_definition(x, tau, k, p, mp, u))
        want = torch.log_softmax(x.double(), 1).cpu().numpy()[np.arange(n), tok]
        assert np.abs(lp - want).max() <= 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,kind", [(1, "normal"), (3, "masked"), (2, "equal"), (80, "normal"), (80, "few")])
def test_the_largest_vocabulary(n, kind, dtype):
    """Rows of 2^21 logits: a cluster for each and a CTA for each, ties by the million, masses of up to 2^52."""
    V = pkg.DS_FILTERED_MAX_VOCAB
    x = _logits(n, V, 3.0, n, DT[dtype], kind)
    x[::5] *= 0.01  # flat rows: more logits at a boundary than the lists hold
    x = x.to(_dev())
    par = _params(n, n + 40)
    tok, lp = _run(x, *par)
    assert np.array_equal(tok, _integer_definition(x, *par))
    at = torch.from_numpy(tok).to(x.device).long()[:, None]
    want = torch.log_softmax(x.double(), 1).gather(1, at)[:, 0].cpu().numpy()
    assert np.abs(lp - want).max() <= 5e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,sigma", [(1300, 1025, 3.0), (700, 5003, 1.0), (160, 9001, 3.0), (100, 70001, 4.0),
                                       (100, 70001, 1.0), (200, 40000, 0.5), (80, 200003, 2.0)])
def test_batches_that_fill_the_gpu_against_real_numbers(n, V, sigma, dtype):
    """The launches for full batches, peaked to flat rows, against the distribution in 64 bits."""
    x = _logits(n, V, sigma, V + n, DT[dtype]).to(_dev())
    par = _params(n, V + 1)
    tok, lp = _run(x, *par)
    assert np.array_equal(tok, _integer_definition(x, *par))
    rows = np.arange(0, n, max(1, n // 60))
    _check_real(x[torch.from_numpy(rows).to(x.device)], tok[rows], lp[rows], *(v[rows] for v in par))
