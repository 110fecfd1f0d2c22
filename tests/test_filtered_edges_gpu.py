"""ds_sample_filtered where a shortcut could go wrong: grammar rows with a few allowed tokens, flat and very long rows."""
import math

import numpy as np
import pytest
import torch

from test_filtered_gpu import DT, _dev, _integer_definition, _params, _run

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
