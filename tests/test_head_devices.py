"""Serving-head calls with tensors of another device, or of sizes that the library's 32-bit counts cannot hold: refused
on the host before anything is launched. Stand-ins for the tensors and for the library; no GPU is used."""
import types

import pytest
import torch

import vocab_wide_logit_gb300 as pkg
from vocab_wide_logit_gb300 import _lib, head


class Tensor:
    """What the wrappers ask of a device tensor."""

    def __init__(self, shape, dtype, index=0, address=0x100000):
        self.shape, self.dtype, self.index, self.address = tuple(shape), dtype, index, address
        self.is_cuda, self.device = True, torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def stride(self, i=None):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.address

    def element_size(self):
        return self.dtype.itemsize

    def is_floating_point(self):
        return self.dtype.is_floating_point


F32, BF16, I8, I32 = torch.float32, torch.bfloat16, torch.int8, torch.int32


@pytest.fixture
def launched(monkeypatch):
    """The names of the library's entry points that a call reached, with device 0 current."""
    names = []

    def entry(name):
        def call(*args):
            names.append(name)
            return 64 if name.endswith("workspace") or name.endswith("bytes") else _lib.DS_OK
        return call

    lib = types.SimpleNamespace(**{name: entry(name) for name in _lib.EXPORTED})
    none = types.SimpleNamespace(**{name: lambda *a: None for name in ("sample", "quantize", "linear", "head")})
    monkeypatch.setattr(_lib, "load", lambda *a: lib)
    monkeypatch.setattr(_lib, "calls", lambda: none)
    monkeypatch.setattr(_lib, "raw_stream", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0, device_index=0))
    make = lambda *shape, dtype=F32, device=None: Tensor(  # noqa: E731
        shape[0] if isinstance(shape[0], (tuple, list)) else shape, dtype, device.index)
    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(torch, "empty_like", lambda t: Tensor(t.shape, t.dtype, t.index))
    return names


def _weight(N, K, index):
    w = object.__new__(pkg.PackedI8)
    w.N, w.K, w.packed, w.scale = N, K, Tensor((N * K,), torch.uint8, index), Tensor((N,), F32, index)
    return w


def _head(N, K, index):
    h = object.__new__(pkg.Int8Head)
    h.weight, h.gain, h.eps = _weight(N, K, index), None, 1e-6
    return h


def _all_calls(index, n=4, V=16, K=32, N=24):
    t = lambda shape, dtype: Tensor(shape, dtype, index)  # noqa: E731
    v = t((n,), F32)
    return {
        "sample": lambda: pkg.sample_filtered(t((n, V), BF16), v, v),
        "sample, outputs given": lambda: pkg.sample_filtered(t((n, V), F32), v, v, out_tokens=t((n,), I32), out_logprobs=v),
        "sample, status": lambda: pkg.sample_filtered(t((n, V), F32), v, v, d_status=t((1,), I32)),
        "quantize": lambda: pkg.quantize_rows(t((n, K), BF16)),
        "quantize, outputs given": lambda: pkg.quantize_rows(t((n, K), BF16), out=t((n, K), I8), out_scale=v),
        "linear": lambda: pkg.linear_i8(t((n, K), I8), v, _weight(N, K, index)),
        "linear, output given": lambda: pkg.linear_i8(t((n, K), I8), v, _weight(N, K, index), out=t((n, N), BF16)),
        "logits": lambda: _head(N, K, index).logits(t((n, K), BF16)),
        "head": lambda: _head(N, K, index).sample(t((n, K), BF16), v, v),
        "pack": lambda: pkg.pack_i8(t((N, K), I8), t((N,), F32)),
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


@pytest.mark.parametrize("n,K", [(2 ** 32 + 5, 1), (2 ** 31, 2), (3, 2 ** 32 + 8)])
def test_sizes_beyond_32_bits_are_refused(launched, n, K):
    """The library counts rows and columns in 32 bits: 2^32 + 5 rows would be read as 5, the rest left unwritten."""
    v = Tensor((n,), F32)
    for call in (lambda: pkg.sample_filtered(Tensor((n, K), BF16), v, v), lambda: pkg.quantize_rows(Tensor((n, K), BF16)),
                 lambda: pkg.linear_i8(Tensor((n, K), I8), v, _weight(24, K, 0)),
                 lambda: pkg.pack_i8(Tensor((n, K), I8), v), lambda: _head(24, K, 0).logits(Tensor((n, K), BF16))):
        with pytest.raises(ValueError, match="2147483647"):
            call()
    assert not launched


def _named_calls(index, B=2, C=3, P=4, V=16, N=24, K=32):
    """The calls under the C names, which take the current stream when none is given."""
    t = lambda shape, dtype=F32: Tensor(shape, dtype, index)  # noqa: E731
    ids, per, cells, v = t((B,), I32), t((B,)), t((C, P)), t((P,))
    return {
        "sample": lambda **kw: pkg.ds_sample(ids, t((C, P, V), BF16), None, ids, per, per, 0.5, 0, 0, t((C, P), I32), cells,
                                             **kw),
        "sample_ex": lambda **kw: pkg.ds_sample(ids, t((C, P, V), BF16), None, ids, per, per, 0.5, 0, 0, t((C, P), I32),
                                                cells, top_ratios=per, **kw),
        "greedy": lambda **kw: pkg.ds_greedy_lse(t((P, V), BF16), v, v, t((P,), I32), **kw),
        "merge": lambda **kw: pkg.ds_merge_triples(t((P, 2, 3)), v, v, t((P,), I32), **kw),
        "log_softmax": lambda **kw: pkg.ds_log_softmax(t((P, V), BF16), t((P, V)), v, v, t((P,), I32), **kw),
        "reveal": lambda **kw: pkg.ds_reveal(cells, t((C, P), I32), ids, ids, t((C, P), I32), **kw),
        "filtered": lambda **kw: pkg.ds_sample_filtered(t((P, V)), v, v, t((P,), I32), v, **kw),
        "quantize": lambda **kw: pkg.ds_quantize_rows(t((P, K), BF16), t((P, K), I8), v, **kw),
        "pack": lambda **kw: pkg.ds_pack_i8(t((N, K), I8), t((N * K,), torch.uint8), **kw),
        "linear": lambda **kw: pkg.ds_linear_i8(t((P, K), I8), v, t((N * K,), torch.uint8), t((N,)), t((P, N)), N, K, **kw),
        "head": lambda **kw: pkg.ds_head_i8(t((P, K), BF16), t((N * K,), torch.uint8), t((N,)), t((P, N)),
                                            t((64,), torch.uint8), N, **kw),
    }


@pytest.mark.parametrize("name", sorted(_named_calls(0)))
def test_calls_by_c_name_keep_to_the_device_of_their_stream(launched, monkeypatch, name):
    def stream(i):
        return types.SimpleNamespace(cuda_stream=0, device_index=i)

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stream(0))
    with pytest.raises(ValueError, match="stream"):
        _named_calls(1)[name]()
    with pytest.raises(ValueError, match="stream"):
        _named_calls(0)[name](stream=stream(1))
    assert not launched
    _named_calls(0)[name]()
    _named_calls(0)[name](stream=stream(0))
    assert len(launched) == 2


@pytest.mark.parametrize("n", [1, 129, 10 ** 9, 2 ** 31 - 300, 2 ** 31 - 256, 2 ** 31 - 255, 2 ** 31 - 1])
def test_workspace_holds_every_row(n):
    """A row of up to 128 inputs takes 256 bytes there, and the last rows of a count close to 2^31 do too."""
    from vocab_wide_logit_gb300 import build
    build.build()
    for N in (1, 128, 2 ** 31 - 1):
        assert n * 256 <= pkg.linear_i8_workspace(n, N, 1) <= n * 256 + 256 * 256 * 2
        assert pkg.head_i8_workspace(n, N, 1) == pkg.linear_i8_workspace(n, N, 1) + 4 * n
        assert pkg.packed_i8_bytes(N, 1) == (N + 127) // 128 * 128 * 128


@pytest.mark.parametrize("name", sorted(_named_calls(0)))
def test_any_object_with_a_stream_handle_will_do(launched, name):
    """A stream of another library: a handle, and no word of its device."""
    _named_calls(0)[name](stream=types.SimpleNamespace(cuda_stream=7))
    assert launched
