"""Refusals of the scoring calls and of the adapters: bad arguments are turned away on the host, before any CUDA call."""
import ctypes
import types

import pytest
import torch

import vocab_wide_logit_gb300 as pkg
from vocab_wide_logit_gb300 import _lib

import test_head_devices
from test_head_devices import BF16, F32, I32, Tensor, _head

head_launched = test_head_devices.launched  # a fixture


@pytest.fixture
def launched(head_launched, monkeypatch):
    """The same, with a ds_calls module that hands every call back."""
    none = types.SimpleNamespace(**{name: lambda *a: None for name in ("sample", "quantize", "linear", "head", "score",
                                                                       "score_grad", "adapters")})
    monkeypatch.setattr(_lib, "calls", lambda: none)
    return head_launched


FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x100001)
HALF = ctypes.c_void_p(0x100002)
OK, INVALID, UNSUPPORTED = _lib.DS_OK, _lib.DS_ERR_INVALID_ARG, _lib.DS_ERR_UNSUPPORTED
C_F32, C_BF16 = _lib.DS_DTYPE_F32, _lib.DS_DTYPE_BF16


@pytest.fixture(scope="module")
def lib():
    from vocab_wide_logit_gb300 import build
    build.build()
    return _lib.load()


def test_score_tokens(lib):
    def call(x=FAKE, dtype=C_BF16, n=2, V=300, ld=300, tok=FAKE, top=3, lp=FAKE, z=None, h=None, rk=None, ti=FAKE, tl=FAKE,
             st=None):
        return lib.ds_score_tokens(x, dtype, n, V, ld, tok, top, lp, z, h, rk, ti, tl, st, None)

    assert call(n=0) == OK
    for bad in (dict(n=-1), dict(V=0), dict(ld=299), dict(dtype=2), dict(top=-1), dict(top=301), dict(x=None), dict(tok=None),
                dict(lp=None), dict(ti=None), dict(tl=None), dict(x=ODD), dict(x=HALF, dtype=C_F32), dict(tok=HALF), dict(lp=HALF),
                dict(z=HALF), dict(h=ODD), dict(rk=HALF), dict(ti=HALF), dict(tl=HALF), dict(st=HALF)):
        assert call(**bad) == INVALID, bad
    assert call(top=_lib.DS_SCORE_MAX_TOP + 1) == UNSUPPORTED
    assert call(ld=(1 << 40) + 1) == UNSUPPORTED


def test_score_tokens_grad(lib):
    def call(x=FAKE, dtype=C_BF16, n=2, V=8, ld=8, tok=FAKE, z=FAKE, h=FAKE, gl=FAKE, gh=FAKE, out=FAKE, ldo=8, st=None):
        return lib.ds_score_tokens_grad(x, dtype, n, V, ld, tok, z, h, gl, gh, out, ldo, st, None)

    assert call(n=0) == OK
    for bad in (dict(n=-1), dict(V=0), dict(ld=7), dict(ldo=7), dict(dtype=2), dict(x=None), dict(tok=None), dict(z=None),
                dict(out=None), dict(gl=None, gh=None), dict(h=None), dict(ld=9), dict(x=ODD), dict(out=ODD),
                dict(x=HALF, dtype=C_F32), dict(out=HALF, dtype=C_F32), dict(tok=HALF), dict(z=HALF), dict(h=HALF), dict(gl=HALF),
                dict(gh=HALF), dict(st=HALF)):
        assert call(**bad) == INVALID, bad
    assert call(ld=(1 << 40) + 1, ldo=(1 << 40) + 1) == UNSUPPORTED


def test_add_adapters(lib):
    n, N, K, L, R = 20, 1000, 512, 4, 16
    need = lib.ds_add_adapters_workspace(n, L, R)
    assert need > 0

    def call(base=FAKE, dtype=C_BF16, n=n, N=N, ldb=N, x=FAKE, xd=C_BF16, K=K, ldx=K, gain=None, eps=1e-6, a=FAKE, b=FAKE, s=FAKE,
             L=L, R=R, ids=FAKE, out=FAKE, ldo=N, ws=FAKE, wb=1 << 40, st=None):
        return lib.ds_add_adapters(base, dtype, n, N, ldb, x, xd, K, ldx, gain, eps, a, b, s, L, R, ids, out, ldo, ws, wb, st,
                                   None)

    assert call(n=0) == OK
    for bad in (dict(n=-1), dict(N=0), dict(K=0), dict(L=0), dict(R=0), dict(ldb=N - 1), dict(ldx=K - 1), dict(ldo=N - 1),
                dict(dtype=5), dict(xd=2), dict(base=None), dict(x=None), dict(a=None), dict(b=None), dict(s=None), dict(ids=None),
                dict(out=None), dict(ws=None), dict(wb=need - 1), dict(ws=ctypes.c_void_p(0x100010)), dict(base=ODD),
                dict(out=ODD), dict(base=HALF, dtype=C_F32), dict(out=HALF, dtype=C_F32), dict(x=ODD), dict(x=HALF, xd=C_F32),
                dict(a=ODD), dict(b=ODD), dict(s=HALF), dict(ids=HALF), dict(gain=HALF), dict(st=HALF), dict(gain=FAKE, eps=-1.0),
                dict(gain=FAKE, eps=float("nan")), dict(ldb=N + 1)):
        assert call(**bad) == INVALID, bad
    for big in (dict(N=(1 << 30) + 1, ldb=1 << 31, ldo=1 << 31), dict(K=(1 << 30) + 1, ldx=1 << 31),
                dict(L=_lib.DS_ADAPTERS_MAX + 1), dict(R=_lib.DS_ADAPTERS_MAX_RANK + 1), dict(ldb=(1 << 40) + 1, ldo=(1 << 40) + 1),
                dict(ldx=(1 << 40) + 1), dict(ldo=(1 << 40) + 1)):
        assert call(**big) == UNSUPPORTED, big
    for bad in ((0, 5, 5), (5, 0, 5), (5, 5, 0), (5, _lib.DS_ADAPTERS_MAX + 1, 5), (5, 5, _lib.DS_ADAPTERS_MAX_RANK + 1)):
        assert pkg.add_adapters_workspace(*bad) == 0
    big = 2 ** 31 - 1
    assert pkg.add_adapters_workspace(big, 8192, 128) >= big * 128 * 4


def _adapters(L, R, K, N, index):
    ad = object.__new__(pkg.Adapters)
    ad.L, ad.R, ad.K, ad.N = L, R, K, N
    ad.a, ad.b, ad.scale = Tensor((L, R, K), BF16, index), Tensor((L, N, R), BF16, index), Tensor((L,), F32, index)
    return ad


def _all_calls(index, n=4, V=16, K=32):
    def t(*shape, dtype=F32, address=0x100000):
        return Tensor(shape, dtype, index, address)
    v, ids = t(n), t(n, dtype=I32)
    ad = _adapters(3, 8, K, V, index)
    return {
        "score": lambda: pkg.score_tokens(t(n, V, dtype=BF16), ids, top=2),
        "score, status": lambda: pkg.score_tokens(t(n, V), ids, d_status=t(1, dtype=I32)),
        "grad": lambda: pkg.score_tokens_grad(t(n, V), ids, v, g_logprobs=v),
        "grad in place": lambda: pkg.score_tokens_grad(t(n, V), ids, v, v, v, v, out=t(n, V)),
        "adapters": lambda: pkg.add_adapters(t(n, V), t(n, K), ad, ids),
        "adapters in place": lambda: pkg.add_adapters(t(n, V), t(n, K), ad, ids, out=t(n, V)),
        "head": lambda: _head(V, K, index).logits(t(n, K), adapters=ad, adapter_ids=ids),
        "head, score": lambda: _head(V, K, index).score(t(n, K), ids, top=1, adapters=ad, adapter_ids=ids),
    }


@pytest.mark.parametrize("name", sorted(_all_calls(0)))
def test_tensors_of_the_current_device_are_launched(launched, name):
    _all_calls(0)[name]()
    assert launched


@pytest.mark.parametrize("name", sorted(_all_calls(0)))
def test_tensors_of_another_device_are_refused(launched, name):
    with pytest.raises(ValueError, match="current device"):
        _all_calls(1)[name]()
    assert not launched


@pytest.mark.parametrize("n,V", [(2 ** 32 + 5, 1), (2 ** 31, 2), (3, 2 ** 32 + 8)])
def test_sizes_beyond_32_bits_are_refused(launched, n, V):
    v, ids = Tensor((n,), F32), Tensor((n,), I32)
    for call in (lambda: pkg.score_tokens(Tensor((n, V), BF16), ids),
                 lambda: pkg.score_tokens_grad(Tensor((n, V), BF16), ids, v, g_logprobs=v),
                 lambda: pkg.add_adapters(Tensor((n, V), BF16), Tensor((n, 8), BF16), _adapters(2, 2, 8, V, 0), ids)):
        with pytest.raises(ValueError, match="2147483647"):
            call()
    assert not launched


def test_wrong_tensors_are_refused(launched):
    n, V, K = 4, 16, 32

    def t(*shape, dtype=F32, index=0, address=0x100000):
        return Tensor(shape, dtype, index, address)
    x, v, ids = t(n, V), t(n), t(n, dtype=I32)
    for bad in (dict(tokens=None), dict(tokens=v), dict(tokens=t(n, dtype=torch.int64)), dict(tokens=t(n - 1, dtype=I32)),
                dict(tokens=t(n, dtype=I32, index=1)), dict(top=-1), dict(top=V + 1), dict(top=129), dict(top=True),
                dict(top=2.0), dict(logits=t(n, V, dtype=torch.float16)), dict(logits=v), dict(d_status=v)):
        with pytest.raises(ValueError):
            pkg.score_tokens(**{**dict(logits=x, tokens=ids), **bad})
    for bad in (dict(tokens=None), dict(lse=None), dict(g_logprobs=None), dict(g_entropy=v), dict(lse=ids), dict(g_logprobs=t(n + 1)),
                dict(out=t(n, V, dtype=BF16)), dict(out=t(n, V - 1)), dict(out=t(n, V, index=1)),
                dict(out=t(n, V, address=0x100004)), dict(out=t(n, V, address=0x100000 - 4 * (n * V - 1)))):
        with pytest.raises(ValueError):
            pkg.score_tokens_grad(**{**dict(logits=x, tokens=ids, lse=v, g_logprobs=v), **bad})
    ad = _adapters(3, 8, K, V, 0)
    for bad in (dict(ids=None), dict(ids=v), dict(ids=t(n + 1, dtype=I32)), dict(hidden=t(n, K - 1)), dict(hidden=t(n - 1, K)),
                dict(base=t(n, V + 1)), dict(gain=t(K - 1)), dict(out=t(n, V, dtype=BF16)), dict(out=t(n, V, address=0x100040)),
                dict(adapters=_adapters(3, 8, K, V, 1))):
        with pytest.raises(ValueError):
            pkg.add_adapters(**{**dict(base=x, hidden=t(n, K), adapters=ad, ids=ids), **bad})
    head = _head(V, K, 0)
    for bad in (dict(adapter_ids=None), dict(adapters=None), dict(adapters=_adapters(3, 8, K, V + 1, 0)),
                dict(adapters=_adapters(3, 8, K + 1, V, 0)), dict(adapter_ids=t(n + 1, dtype=I32))):
        with pytest.raises(ValueError):
            head.logits(t(n, K), **{**dict(adapters=ad, adapter_ids=ids), **bad})
    assert not launched


def test_the_head_checks_adapters_before_the_projection(launched):
    """Stacks that were replaced by others than those that the Adapters were made of: the projection has not run, so that an
    `out` that was given is as it was."""
    n, V, K = 4, 16, 32

    def t(*shape, dtype=F32, index=0):
        return Tensor(shape, dtype, index)
    head, ids, hidden = _head(V, K, 0), t(n, dtype=I32), t(n, K)
    for name, stack in (("b", t(3, V, 9, dtype=BF16)), ("b", t(3, V + 1, 8, dtype=BF16)), ("b", t(3, V, 8, dtype=BF16, index=1)),
                        ("b", t(3, V, 8)), ("a", t(2, 8, K, dtype=BF16)), ("a", t(3, 8, K + 1, dtype=BF16)), ("scale", t(2)),
                        ("scale", None)):
        ad = _adapters(3, 8, K, V, 0)
        setattr(ad, name, stack)
        for call in (lambda: head.logits(hidden, out=t(n, V, dtype=BF16), adapters=ad, adapter_ids=ids),
                     lambda: head.sample(hidden, t(n), t(n), adapters=ad, adapter_ids=ids),
                     lambda: head.score(hidden, ids, adapters=ad, adapter_ids=ids)):
            with pytest.raises(ValueError):
                call()
            assert not launched, name


def test_stacks_larger_than_the_library_takes():
    """2^30 inputs and channels at most: refused when the stacks are put together, not at the first call."""
    big = (1 << 30) + 1
    for a, b in (((1, 1, big), (1, 4, 1)), ((1, 1, 4), (1, big, 1))):
        with pytest.raises(ValueError, match="1073741824"):
            pkg.Adapters(Tensor(a, BF16), Tensor(b, BF16), Tensor((1,), F32))


def test_results_beside_the_input_are_taken(launched):
    """Rows side by side in one buffer, and right behind the input."""
    n, V = 4, 16
    v, ids = Tensor((n,), F32), Tensor((n,), I32)

    class Half(Tensor):
        def stride(self, i=None):
            return (2 * V, 1) if i is None else (2 * V, 1)[i]

    pkg.score_tokens_grad(Half((n, V), F32), ids, v, g_logprobs=v, out=Half((n, V), F32, 0, 0x100000 + 4 * V))
    pkg.score_tokens_grad(Tensor((n, V), F32), ids, v, g_logprobs=v, out=Tensor((n, V), F32, 0, 0x100000 + 4 * n * V))
    with pytest.raises(ValueError):
        pkg.score_tokens_grad(Half((n, V), F32), ids, v, g_logprobs=v, out=Half((n, V), F32, 0, 0x100000 + 4 * V - 4))
    assert len(launched) == 2


def test_stacks_are_checked():
    def stack(a=(3, 8, 32), b=(3, 16, 8), s=(3,), da=BF16, db=BF16, ds_=F32, index=0):
        return pkg.Adapters(Tensor(a, da), Tensor(b, db, index), Tensor(s, ds_, index))

    stack()
    for bad in (dict(a=(3, 8)), dict(a=(3, 8, 0)), dict(a=(3, 7, 32)), dict(b=(2, 16, 8)), dict(s=(2,)), dict(da=F32), dict(db=F32),
                dict(ds_=BF16), dict(index=1), dict(a=(3, 129, 32), b=(3, 16, 129)), dict(a=(8193, 1, 1), b=(8193, 1, 1), s=(8193,))):
        with pytest.raises(ValueError):
            stack(**bad)
    with pytest.raises(ValueError):
        pkg.Adapters(torch.zeros((3, 8, 32), dtype=BF16), torch.zeros((3, 16, 8), dtype=BF16), torch.zeros(3))


def test_by_c_name_on_another_device(launched):
    """The address of another device's tensor on the current stream."""
    t = lambda *shape, dtype=F32: Tensor(shape, dtype, 1)  # noqa: E731
    ids = t(4, dtype=I32)
    for call in (lambda: pkg.ds_score_tokens(t(4, 16), ids, t(4)), lambda: pkg.ds_score_tokens_grad(t(4, 16), ids, t(4), t(4, 16)),
                 lambda: pkg.ds_add_adapters(t(4, 16), t(4, 8), t(2, 2, 8, dtype=BF16), t(2, 16, 2, dtype=BF16), t(2), ids, t(4, 16),
                                             t(999))):
        with pytest.raises(ValueError, match="cuda:1 for a stream of cuda:0"):
            call()
    assert not launched
