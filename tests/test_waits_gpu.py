"""What is left when a wait inside a kernel runs out: the status bit, NaN for every result that is owed, and a GPU that
goes on. The waits are those of the kernels as they are, built so that they ask once instead of 2^20 times; copies and
instructions in flight are still waited for."""
import math
import os
import subprocess

import pytest
import torch

import vocab_wide_logit_gb300 as pkg
from vocab_wide_logit_gb300 import _lib, build

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    """The library with waits that ask once."""
    build.build()
    out = tmp_path_factory.mktemp("impatient")
    flags = build.ARCH + ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", build.INCLUDE, "-I", build.CSRC, "-I", build.OUT,
                          "--expt-relaxed-constexpr", "-DDS_WAIT_TRIES=0", '-DDS_WAIT_TRY="test_wait"']
    objs, jobs = [], []
    for src in build.SOURCES:
        own = src in ("k_linear_i8.cu", "k_sample_filtered.cu")
        obj = os.path.join(str(out) if own else build.OUT, src.replace(".cu", ".o"))
        objs.append(obj)
        if own:
            jobs.append(subprocess.Popen([build.nvcc()] + flags + ["-c", os.path.join(build.CSRC, src), "-o", obj]))
    assert [j.wait() for j in jobs] == [0] * len(jobs)
    path = str(out / "libdsample.so")
    subprocess.run([build.nvcc()] + build.ARCH + ["-shared", "-o", path] + objs + ["-lcudart"], check=True)
    return path


@pytest.fixture
def use(impatient):
    """Runs a call with the calls by C name bound to that library."""
    def run(call):
        saved, _lib._lib = _lib._lib, None
        try:
            _lib.load(impatient)
            call()
            torch.cuda.synchronize()
        finally:
            _lib._lib = saved
    _lib.load()
    return run


def _operands(n, N, K):
    dev, g = torch.device("cuda", 0), torch.Generator().manual_seed(n + K)
    a = torch.randint(-127, 128, (n, K), generator=g).to(torch.int8).to(dev)
    w = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8).to(dev)
    return a, torch.ones(n, device=dev), w, torch.ones(N, device=dev)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,N,K", [(1, 300, 128), (5, 41000, 192), (40, 1025, 5000), (140, 1025, 640), (256, 41000, 640),
                                   (300, 129, 2100)])
def test_product_that_gives_up(use, n, N, K, dtype):
    """Resident, streamed and paired row tiles, one tile a CTA and several."""
    a, sa, w, sw = _operands(n, N, K)
    p = pkg.pack_i8(w, sw)
    want = pkg.linear_i8(a, sa, p, dtype=DT[dtype])
    out = torch.full((n, N + 3), 5.0, dtype=DT[dtype], device=a.device)
    st = torch.zeros(1, dtype=torch.int32, device=a.device)
    ws = torch.empty(pkg.linear_i8_workspace(n, N, K), dtype=torch.uint8, device=a.device)
    use(lambda: pkg.ds_linear_i8(a, sa, p.packed, sw, out, N, K, workspace=ws, d_status=st))
    assert int(st.item()) == pkg.DS_DEV_ERR_TIMEOUT
    assert bool((out[:, N:] == 5.0).all())
    got = out[:, :N]
    lost = torch.isnan(got)
    assert bool(lost.any()) and bool((lost | (got == want)).all())
    assert torch.equal(pkg.linear_i8(a, sa, p, dtype=DT[dtype]), want)  # the next call is as before


@pytest.mark.parametrize("n", [3, 200])
def test_head_that_gives_up(use, n):
    N, K = 2000, 512
    _, _, w, sw = _operands(1, N, K)
    head = pkg.Int8Head(w, sw)
    x = torch.randn((n, K), generator=torch.Generator().manual_seed(n)).to(w.device)
    want = head.logits(x)
    out = torch.full((n, N), 5.0, dtype=torch.bfloat16, device=w.device)
    st = torch.zeros(1, dtype=torch.int32, device=w.device)
    ws = torch.empty(pkg.head_i8_workspace(n, N, K), dtype=torch.uint8, device=w.device)
    use(lambda: pkg.ds_head_i8(x, head.weight.packed, sw, out, ws, N, d_status=st))
    assert int(st.item()) == pkg.DS_DEV_ERR_TIMEOUT
    assert bool((torch.isnan(out) | (out == want)).all()) and bool(torch.isnan(out).any())
    tok, lp = pkg.sample_filtered(out, torch.ones(n, device=w.device), torch.full((n,), 0.5, device=w.device))
    hit = torch.isnan(out).any(1)  # the sampler reports such rows
    assert bool((tok[hit] == -1).all()) and all(math.isnan(v) for v in lp[hit].tolist())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sampler_that_gives_up(use, dtype):
    """Rows held in shared memory, by 128 threads each or by a warp each with a second launch behind it: a row whose copy
    was not waited for has token -1 and logprob NaN, and no row has another token than its own. A short row's copy is
    often there when it is asked for, so that a call may lose nothing, but not all of them together."""
    lost_rows = 0
    for n, V in [(1, 1025), (40, 1025), (15510, 1025), (1300, 2048), (3000, 5003), (160, 8001),
                 (20000, 8001)]:  # the last: more than L2 holds
        g = torch.Generator().manual_seed(n)
        dev = torch.device("cuda", 0)
        x = (torch.randn((n, V), generator=g) * 3).to(DT[dtype]).to(dev)
        tau = torch.where(torch.arange(n) % 3 == 0, 0.0, 0.8).to(dev)
        u, p = torch.rand((n,), generator=g).to(dev), torch.full((n,), 0.9, device=dev)
        k = torch.where(torch.arange(n) % 5 == 0, 200, 0).to(torch.int32).to(dev)
        want, want_lp = pkg.sample_filtered(x, tau, u, top_k=k, top_p=p)
        tok, lp = torch.full((n,), 7, dtype=torch.int32, device=dev), torch.full((n,), 7.0, device=dev)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        use(lambda: pkg.ds_sample_filtered(x, tau, u, tok, lp, top_k=k, top_p=p, d_status=st))
        lost = torch.isnan(lp)
        assert int(st.item()) == (pkg.DS_DEV_ERR_TIMEOUT if bool(lost.any()) else 0)
        assert bool((tok[lost] == -1).all())
        assert torch.equal(tok[~lost], want[~lost]) and torch.equal(lp[~lost], want_lp[~lost])
        again, _ = pkg.sample_filtered(x, tau, u, top_k=k, top_p=p)
        assert torch.equal(again, want)
        lost_rows += int(lost.sum())
    assert lost_rows
