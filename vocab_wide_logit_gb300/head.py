"""The serving head: hidden states to logits through an 8-bit vocabulary projection, and logits to tokens by
temperature, top-k, top-p and min-p.

Functions allocate their outputs and check their tensors (a tensor of another type or shape would be read as if it
were the expected one); the compute is in the library. Outputs and workspaces are allocated on the stream that the
call runs on.
"""
import torch

from . import _lib


class _On:
    """The stream context of a call: allocations inside belong to `stream` (None: the current one)."""

    def __init__(self, stream):
        self.ctx = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _rows(name, t, dtypes):
    """A device matrix whose rows are dense (any distance between rows)."""
    if t.dim() != 2 or t.dtype not in dtypes or not t.is_cuda:
        raise ValueError("%s: a 2-d cuda tensor of %s expected, got %s %s on %s" %
                         (name, "/".join(str(d) for d in dtypes), tuple(t.shape), t.dtype, t.device))
    if (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError("%s: rows must be dense and must not overlap, got strides %s" % (name, t.stride()))


def _vec(name, t, n, dtype, device):
    if t is None:
        return
    if t.dim() != 1 or t.shape[0] != n or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError("%s: a contiguous %s tensor [%d] on %s expected, got %s %s on %s" %
                         (name, dtype, n, device, tuple(t.shape), t.dtype, t.device))


def _status(t, device):
    if t is not None and (t.numel() != 1 or t.element_size() != 4 or t.is_floating_point() or t.device != device):
        raise ValueError("d_status: one 32-bit integer on %s expected" % device)


_LOGITS = (torch.bfloat16, torch.float32)
_INTS = (torch.int8,)


def sample_filtered(logits, temperature, u, top_k=None, top_p=None, min_p=None, out_tokens=None, out_logprobs=None,
                    d_status=None, stream=None):
    """One token per row of logits [n, V] (bfloat16 or float32, cuda, rows may lie apart) by temperature, top-k,
    top-p and min-p, drawn with the given uniform numbers u float32 [n] in [0, 1). temperature / top_p / min_p:
    float32 [n]; top_k: int32 [n]; None leaves a filter out. Returns (tokens int32 [n], logprobs float32 [n]); a row
    with nothing to draw, a bad parameter, a NaN or +inf gives (-1, NaN), the last two with a bit in d_status."""
    _rows("logits", logits, _LOGITS)
    n, dev = logits.shape[0], logits.device
    f32, i32 = torch.float32, torch.int32
    if temperature is None or u is None:
        raise ValueError("temperature and u are needed")
    _vec("temperature", temperature, n, f32, dev)
    _vec("u", u, n, f32, dev)
    _vec("top_k", top_k, n, i32, dev)
    _vec("top_p", top_p, n, f32, dev)
    _vec("min_p", min_p, n, f32, dev)
    _vec("out_tokens", out_tokens, n, i32, dev)
    _vec("out_logprobs", out_logprobs, n, f32, dev)
    _status(d_status, dev)
    with _On(stream):
        if out_tokens is None:
            out_tokens = torch.empty(n, dtype=i32, device=dev)
        if out_logprobs is None:
            out_logprobs = torch.empty(n, dtype=f32, device=dev)
        _lib.ds_sample_filtered(logits, temperature, u, out_tokens, out_logprobs, top_k=top_k, top_p=top_p,
                                min_p=min_p, d_status=d_status, stream=stream)
    return out_tokens, out_logprobs


def quantize_rows(x, gain=None, eps=1e-6, out=None, out_scale=None, stream=None):
    """Rows x [n, K] (bfloat16 or float32) to 8-bit integers with one scale each, after an RMS norm when gain
    (float32 [K]) is given. Returns (q int8 [n, K], scale float32 [n]) with q * scale close to the (normed) row."""
    _rows("x", x, _LOGITS)
    n, K = x.shape
    dev = x.device
    _vec("gain", gain, K, torch.float32, dev)
    _vec("out_scale", out_scale, n, torch.float32, dev)
    if out is not None and (out.shape != x.shape or out.dtype != torch.int8 or out.device != dev or
                            not out.is_contiguous()):
        raise ValueError("out: a contiguous int8 tensor %s on %s expected" % (tuple(x.shape), dev))
    with _On(stream):
        if out is None:
            out = torch.empty((n, K), dtype=torch.int8, device=dev)
        if out_scale is None:
            out_scale = torch.empty(n, dtype=torch.float32, device=dev)
        _lib.ds_quantize_rows(x, out, out_scale, gain=gain, eps=eps, stream=stream)
    return out, out_scale


class PackedI8:
    """An 8-bit weight [N, K] in the layout of ds_linear_i8, with its scale per channel. Holds no workspace, so
    calls on several streams may share it."""

    def __init__(self, w, scale, stream=None):
        _rows("w", w, _INTS)
        self.N, self.K = (int(d) for d in w.shape)
        _vec("scale", scale, self.N, torch.float32, w.device)
        if scale is None:
            raise ValueError("scale is needed")
        self.scale = scale
        with _On(stream):
            self.packed = torch.empty(_lib.packed_i8_bytes(self.N, self.K), dtype=torch.uint8, device=w.device)
            _lib.ds_pack_i8(w, self.packed, stream=stream)


def pack_i8(w, scale, stream=None):
    """Lay an int8 weight [N, K] with float32 scales [N] out for linear_i8 (once per weight)."""
    return PackedI8(w, scale, stream=stream)


def linear_i8(a, a_scale, weight, out=None, dtype=torch.bfloat16, d_status=None, stream=None):
    """out[i][j] = (sum_k a[i][k] w[j][k]) * a_scale[i] * w_scale[j] for a int8 [n, K], a_scale float32 [n] and a
    PackedI8 weight. out: bfloat16 or float32 [n, N] (rows may lie apart), allocated with dtype when None."""
    _rows("a", a, _INTS)
    n, dev = a.shape[0], a.device
    if a.shape[1] != weight.K or dev != weight.packed.device:
        raise ValueError("a: [n, %d] on %s expected, got %s on %s" % (weight.K, weight.packed.device,
                                                                      tuple(a.shape), dev))
    _vec("a_scale", a_scale, n, torch.float32, dev)
    _status(d_status, dev)
    if out is not None:
        _rows("out", out, _LOGITS)
        if tuple(out.shape) != (n, weight.N) or out.device != dev:
            raise ValueError("out: [%d, %d] on %s expected" % (n, weight.N, dev))
    with _On(stream):
        if out is None:
            out = torch.empty((n, weight.N), dtype=dtype, device=dev)
        need = _lib.linear_i8_workspace(n, weight.N, weight.K)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _lib.ds_linear_i8(a, a_scale, weight.packed, weight.scale, out, weight.N, weight.K, workspace=workspace,
                          d_status=d_status, n=n, stream=stream)
    return out


class Int8Head:
    """A model's output head in 8 bits: the final RMS norm (when gain is given), the vocabulary projection and the
    sampler. w int8 [N, K] with scale float32 [N]; from_weight() quantises a bfloat16 or float32 weight."""

    def __init__(self, w, scale, gain=None, eps=1e-6, stream=None):
        self.weight = pack_i8(w, scale, stream=stream)
        _vec("gain", gain, self.weight.K, torch.float32, w.device)
        self.gain, self.eps = gain, float(eps)

    @classmethod
    def from_weight(cls, w, gain=None, eps=1e-6):
        """Each channel of w [N, K] quantised with a scale of its own."""
        q, scale = quantize_rows(w)
        return cls(q, scale, gain=gain, eps=eps)

    def logits(self, hidden, out=None, dtype=torch.bfloat16, d_status=None, stream=None):
        """Logits [n, N] of hidden states [n, K] (bfloat16 or float32)."""
        q, scale = quantize_rows(hidden, gain=self.gain, eps=self.eps, stream=stream)
        return linear_i8(q, scale, self.weight, out=out, dtype=dtype, d_status=d_status, stream=stream)

    def sample(self, hidden, temperature, u, top_k=None, top_p=None, min_p=None, d_status=None, stream=None):
        """Hidden states [n, K] to (tokens, logprobs): logits() then sample_filtered()."""
        return sample_filtered(self.logits(hidden, d_status=d_status, stream=stream), temperature, u, top_k=top_k,
                               top_p=top_p, min_p=min_p, d_status=d_status, stream=stream)
