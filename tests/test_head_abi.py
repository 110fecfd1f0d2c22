"""Refusals of the serving head's entry points: bad arguments are turned away on the host, before any CUDA call."""
import ctypes

import pytest
import torch

import vocab_wide_logit_gb300 as pkg
from vocab_wide_logit_gb300 import _lib

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x100001)
HALF = ctypes.c_void_p(0x100002)
OK, INVALID, UNSUPPORTED = _lib.DS_OK, _lib.DS_ERR_INVALID_ARG, _lib.DS_ERR_UNSUPPORTED
F32, BF16 = _lib.DS_DTYPE_F32, _lib.DS_DTYPE_BF16


@pytest.fixture(scope="module")
def lib():
    from vocab_wide_logit_gb300 import build
    build.build()
    return _lib.load()


def test_sample_filtered(lib):
    def call(x=FAKE, dtype=BF16, n=2, V=8, ld=8, tau=FAKE, k=None, p=None, mp=None, u=FAKE, tok=FAKE, lp=FAKE, st=None):
        return lib.ds_sample_filtered(x, dtype, n, V, ld, tau, k, p, mp, u, tok, lp, st, None)

    assert call(n=0) == OK
    for bad in (dict(n=-1), dict(V=0), dict(ld=7), dict(dtype=2), dict(x=None), dict(tau=None), dict(u=None),
                dict(tok=None), dict(lp=None), dict(x=ODD), dict(x=HALF, dtype=F32), dict(tau=HALF), dict(k=HALF),
                dict(p=ODD), dict(mp=ODD), dict(u=HALF), dict(tok=HALF), dict(lp=HALF), dict(st=HALF)):
        assert call(**bad) == INVALID, bad
    assert call(V=_lib.DS_FILTERED_MAX_VOCAB + 1, ld=1 << 30) == UNSUPPORTED
    assert call(ld=(1 << 40) + 1) == UNSUPPORTED


def test_quantize_rows(lib):
    def call(x=FAKE, dtype=BF16, n=2, K=8, ld=8, gain=None, eps=1e-6, q=FAKE, s=FAKE):
        return lib.ds_quantize_rows(x, dtype, n, K, ld, gain, eps, q, s, None)

    assert call(n=0) == OK
    for bad in (dict(n=-1), dict(K=0), dict(ld=7), dict(dtype=-1), dict(x=None), dict(q=None), dict(s=None), dict(x=ODD),
                dict(x=HALF, dtype=F32), dict(gain=HALF), dict(s=HALF), dict(gain=FAKE, eps=-1.0),
                dict(gain=FAKE, eps=float("nan")), dict(gain=FAKE, eps=float("inf"))):
        assert call(**bad) == INVALID, bad
    assert call(ld=(1 << 40) + 1) == UNSUPPORTED


def test_pack_and_linear(lib):
    def pack(w=FAKE, N=4, K=8, ld=8, p=FAKE):
        return lib.ds_pack_i8(w, N, K, ld, p, None)

    for bad in (dict(N=0), dict(K=0), dict(ld=7), dict(w=None), dict(p=None), dict(p=ctypes.c_void_p(0x100008))):
        assert pack(**bad) == INVALID, bad
    assert pack(K=_lib.DS_LINEAR_MAX_K + 1, ld=1 << 20) == UNSUPPORTED

    n, N, K = 300, 1000, 512
    need = lib.ds_linear_i8_workspace(n, N, K)

    def call(a=FAKE, lda=K, sa=FAKE, p=FAKE, sw=FAKE, n=n, N=N, K=K, out=FAKE, dtype=BF16, ldo=N, ws=FAKE, wb=1 << 40,
             st=None):
        return lib.ds_linear_i8(a, lda, sa, p, sw, n, N, K, out, dtype, ldo, ws, wb, st, None)

    assert call(n=0) == OK
    for bad in (dict(n=-1), dict(N=0), dict(K=0), dict(lda=K - 1), dict(ldo=N - 1), dict(dtype=3), dict(a=None),
                dict(sa=None), dict(p=None), dict(sw=None), dict(out=None), dict(sa=HALF), dict(sw=HALF), dict(st=HALF),
                dict(p=ctypes.c_void_p(0x100008)), dict(out=ODD), dict(out=HALF, dtype=F32)):
        assert call(**bad) == INVALID, bad
    if need:
        assert call(ws=None) == INVALID and call(wb=need - 1) == INVALID
        assert call(ws=ctypes.c_void_p(0x100010)) == INVALID
    assert call(K=_lib.DS_LINEAR_MAX_K + 1, lda=1 << 20) == UNSUPPORTED
    assert call(ldo=(1 << 40) + 1) == UNSUPPORTED


def test_head_i8(lib):
    n, N, K = 20, 1000, 512
    need = lib.ds_head_i8_workspace(n, N, K)
    assert need > lib.ds_linear_i8_workspace(n, N, K)

    def call(x=FAKE, dtype=BF16, n=n, K=K, ld=K, gain=None, eps=1e-6, p=FAKE, sw=FAKE, N=N, out=FAKE, out_dtype=BF16, ldo=N,
             ws=FAKE, wb=1 << 40, st=None):
        return lib.ds_head_i8(x, dtype, n, K, ld, gain, eps, p, sw, N, out, out_dtype, ldo, ws, wb, st, None)

    assert call(n=0) == OK
    for bad in (dict(n=-1), dict(N=0), dict(K=0), dict(ld=K - 1), dict(ldo=N - 1), dict(dtype=4), dict(out_dtype=-1),
                dict(x=None), dict(p=None), dict(sw=None), dict(out=None), dict(x=ODD), dict(x=HALF, dtype=F32),
                dict(gain=HALF), dict(gain=FAKE, eps=-1.0), dict(sw=HALF), dict(st=HALF), dict(out=ODD),
                dict(out=HALF, out_dtype=F32), dict(p=ctypes.c_void_p(0x100008)), dict(ws=None), dict(wb=need - 1),
                dict(ws=ctypes.c_void_p(0x100010))):
        assert call(**bad) == INVALID, bad
    assert call(K=_lib.DS_LINEAR_MAX_K + 1, ld=1 << 20) == UNSUPPORTED
    assert call(ld=(1 << 40) + 1) == UNSUPPORTED
    for bad in ((0, 5, 5), (5, 0, 5), (5, 5, 0), (5, 5, _lib.DS_LINEAR_MAX_K + 1)):
        assert pkg.head_i8_workspace(*bad) == 0


def test_sizes(lib):
    assert pkg.packed_i8_bytes(1, 1) == 128 * 128
    assert pkg.packed_i8_bytes(129, 300) == 256 * 384
    assert pkg.packed_i8_bytes(248320, 2048) == 248320 * 2048
    assert pkg.packed_i8_bytes(0, 5) == 0 and pkg.packed_i8_bytes(5, 0) == 0
    assert pkg.packed_i8_bytes(5, _lib.DS_LINEAR_MAX_K + 1) == 0
    for bad in ((0, 5, 5), (5, 0, 5), (5, 5, 0), (5, 5, _lib.DS_LINEAR_MAX_K + 1)):
        assert pkg.linear_i8_workspace(*bad) == 0


def test_wrappers_refuse_other_tensors():
    """Tensors that the library would misread: on the host, of another type or shape, or with strided elements."""
    x, v = torch.zeros((2, 8), dtype=torch.bfloat16), torch.zeros(2)
    with pytest.raises(ValueError):
        pkg.sample_filtered(x, v, v)  # not on the GPU
    with pytest.raises(ValueError):
        pkg.sample_filtered(x.double(), v, v)
    with pytest.raises(ValueError):
        pkg.quantize_rows(torch.zeros((2, 8)))
    with pytest.raises(ValueError):
        pkg.pack_i8(torch.zeros((2, 8)), v)


@pytest.mark.gpu
def test_wrappers_refuse_on_the_gpu():
    dev = torch.device("cuda", 0)
    x = torch.zeros((4, 16), dtype=torch.bfloat16, device=dev)
    v = torch.ones(4, device=dev)
    k = torch.ones(4, dtype=torch.int32, device=dev)
    for bad in (dict(logits=x.half()), dict(logits=x[:, ::2]), dict(logits=x[0]), dict(temperature=v[:3]),
                dict(temperature=v.double()), dict(temperature=None), dict(u=None), dict(u=v.cpu()), dict(top_k=k.long()),
                dict(top_k=v), dict(top_p=k), dict(min_p=torch.ones((8,), device=dev)[::2]),
                dict(out_tokens=k.long()), dict(out_logprobs=v.double()), dict(d_status=v[:1]), dict(d_status=k)):
        args = dict(logits=x, temperature=v, u=v * 0.5, top_k=k, top_p=v, min_p=v)
        args.update(bad)
        with pytest.raises(ValueError):
            pkg.sample_filtered(**args)
    w = torch.ones((6, 16), dtype=torch.int8, device=dev)
    sw = torch.ones(6, device=dev)
    for bad in (dict(w=w.int()), dict(w=w[:, ::2]), dict(scale=sw[:5]), dict(scale=None)):
        args = dict(w=w, scale=sw)
        args.update(bad)
        with pytest.raises(ValueError):
            pkg.pack_i8(**args)
    p = pkg.pack_i8(w, sw)
    a = torch.ones((4, 16), dtype=torch.int8, device=dev)
    for bad in (dict(a=a[:, :15]), dict(a=a.float()), dict(a_scale=v[:3]), dict(out=torch.empty((4, 5), device=dev)),
                dict(out=torch.empty((4, 6), dtype=torch.float16, device=dev)), dict(d_status=k)):
        args = dict(a=a, a_scale=v, weight=p)
        args.update(bad)
        with pytest.raises(ValueError):
            pkg.linear_i8(**args)
    with pytest.raises(ValueError):
        pkg.linear_i8(a, None, p)
    with pytest.raises(ValueError):
        pkg.linear_i8(a, v, p, dtype=torch.float16)
    head = pkg.Int8Head(w, sw)
    for bad in (x[:, :15], x.half(), x[:, ::2], x.cpu()):
        with pytest.raises(ValueError):
            head.logits(bad)
    with pytest.raises(ValueError):
        head.logits(x, out=torch.empty((4, 7), device=dev))
    with pytest.raises(ValueError):
        pkg.Int8Head(w, sw, gain=v)
    with pytest.raises(ValueError):
        pkg.quantize_rows(x, gain=v)
    with pytest.raises(ValueError):
        pkg.quantize_rows(x, out=torch.empty((4, 15), dtype=torch.int8, device=dev))
