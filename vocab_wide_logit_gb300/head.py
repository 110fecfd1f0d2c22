"""The serving head: hidden states to logits through an 8-bit vocabulary projection, and logits to tokens by
temperature, top-k, top-p and min-p.

Functions allocate their outputs and check their tensors (a tensor of another type or shape would be read as if it
were the expected one); the compute is in the library. Outputs and workspaces are allocated on the stream that the
call runs on. At decoding sizes a call takes about as long to issue as to run, so the usual calls (outputs made here, no
status word) go through _lib.calls(), which checks and launches without the interpreter and hands everything else back;
here the checks are plain comparisons and the library is called with plain integers.
"""
import torch

from . import _lib

_F32, _I32, _I8, _U8, _BF16 = torch.float32, torch.int32, torch.int8, torch.uint8, torch.bfloat16
_INT_MAX = 2 ** 31 - 1
_CODE = {_F32: _lib.DS_DTYPE_F32, _BF16: _lib.DS_DTYPE_BF16}


def _bad(name, want, t):
    got = "None" if t is None else "%s %s strides %s on %s" % (tuple(t.shape), t.dtype, t.stride(), t.device)
    raise ValueError("%s: %s expected, got %s" % (name, want, got))


def _rows(name, t, codes):
    """(rows, columns, elements between rows, device index) of a matrix on the current device whose rows are dense. The
    launch goes to that device's stream, where the addresses of another device's tensors would fault or race."""
    if t.dim() != 2 or t.dtype not in codes or not t.is_cuda:
        _bad(name, "a 2-d cuda tensor of %s" % "/".join(str(d) for d in codes), t)
    if t.get_device() != torch.cuda.current_device():
        _bad(name, "a tensor on the current device (cuda:%d, or that of the given stream)" % torch.cuda.current_device(), t)
    n, k = t.shape
    if n > _INT_MAX or k > _INT_MAX:  # would lose their upper bits on the way into the library
        _bad(name, "at most %d rows and columns" % _INT_MAX, t)
    ld, step = t.stride()
    if n <= 1:
        ld = k
    if (k > 1 and step != 1) or ld < k:
        _bad(name, "a tensor with dense rows that do not overlap", t)
    return n, k, ld, t.get_device()


def _vec(name, t, n, dtype, index):
    """The address of a contiguous device vector, None for None."""
    if t is None:
        return None
    if t.dim() != 1 or t.numel() != n or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        _bad(name, "a contiguous %s tensor [%d] on cuda:%d" % (dtype, n, index), t)
    return t.data_ptr()


def _status(t, index):
    if t is None:
        return None
    if t.numel() != 1 or t.element_size() != 4 or t.is_floating_point() or t.get_device() != index:
        _bad("d_status", "one 32-bit integer on cuda:%d" % index, t)
    return t.data_ptr()


def _check(name, rc):
    if rc != _lib.DS_OK:
        raise _lib.DsError(name, rc)


def sample_filtered(logits, temperature, u, top_k=None, top_p=None, min_p=None, out_tokens=None, out_logprobs=None,
                    d_status=None, stream=None):
    """One token per row of logits [n, V] (bfloat16 or float32, cuda, rows may lie apart) by temperature, top-k,
    top-p and min-p, drawn with the given uniform numbers u float32 [n] in [0, 1). temperature / top_p / min_p:
    float32 [n]; top_k: int32 [n]; None leaves a filter out. Returns (tokens int32 [n], logprobs float32 [n]); a row
    with nothing to draw, a bad parameter, a NaN or +inf gives (-1, NaN), the last two with a bit in d_status."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return sample_filtered(logits, temperature, u, top_k, top_p, min_p, out_tokens, out_logprobs, d_status)
    if out_tokens is None and out_logprobs is None and d_status is None:
        r = _lib.calls().sample(logits, temperature, u, top_k, top_p, min_p)
        if r is not None:
            return r if type(r) is tuple else _check("ds_sample_filtered", r)
    n, V, ld, index = _rows("logits", logits, _CODE)
    if temperature is None or u is None:
        raise ValueError("temperature and u are needed")
    tau = _vec("temperature", temperature, n, _F32, index)
    up = _vec("u", u, n, _F32, index)
    k = _vec("top_k", top_k, n, _I32, index)
    p = _vec("top_p", top_p, n, _F32, index)
    mp = _vec("min_p", min_p, n, _F32, index)
    st = _status(d_status, index)
    if out_tokens is None:
        out_tokens = torch.empty(n, dtype=_I32, device=logits.device)
        tok = out_tokens.data_ptr()
    else:
        tok = _vec("out_tokens", out_tokens, n, _I32, index)
    if out_logprobs is None:
        out_logprobs = torch.empty_like(temperature)
        lp = out_logprobs.data_ptr()
    else:
        lp = _vec("out_logprobs", out_logprobs, n, _F32, index)
    _check("ds_sample_filtered", _lib.load().ds_sample_filtered(
        logits.data_ptr(), _CODE[logits.dtype], n, V, ld, tau, k, p, mp, up, tok, lp, st, _lib.raw_stream()))
    return out_tokens, out_logprobs


def quantize_rows(x, gain=None, eps=1e-6, out=None, out_scale=None, stream=None):
    """Rows x [n, K] (bfloat16 or float32) to 8-bit integers with one scale each, after an RMS norm when gain
    (float32 [K]) is given. Returns (q int8 [n, K], scale float32 [n]) with q * scale close to the (normed) row."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return quantize_rows(x, gain, eps, out, out_scale)
    if out is None and out_scale is None:
        r = _lib.calls().quantize(x, gain, eps)
        if r is not None:
            return r if type(r) is tuple else _check("ds_quantize_rows", r)
    n, K, ld, index = _rows("x", x, _CODE)
    gp = _vec("gain", gain, K, _F32, index)
    if out is None:
        out = torch.empty((n, K), dtype=_I8, device=x.device)
    elif out.shape != x.shape or out.dtype != _I8 or out.get_device() != index or not out.is_contiguous():
        _bad("out", "a contiguous int8 tensor [%d, %d] on cuda:%d" % (n, K, index), out)
    if out_scale is None:
        out_scale = torch.empty(n, dtype=_F32, device=x.device)
        sp = out_scale.data_ptr()
    else:
        sp = _vec("out_scale", out_scale, n, _F32, index)
    _check("ds_quantize_rows", _lib.load().ds_quantize_rows(x.data_ptr(), _CODE[x.dtype], n, K, ld, gp, eps,
                                                            out.data_ptr(), sp, _lib.raw_stream()))
    return out, out_scale


class PackedI8:
    """An 8-bit weight [N, K] in the layout of ds_linear_i8, with its scale per channel. Holds no workspace, so
    calls on several streams may share it."""

    def __init__(self, w, scale, stream=None):
        if scale is None:
            raise ValueError("scale is needed")
        with torch.cuda.stream(stream):
            N, K, ld, index = _rows("w", w, (_I8,))
            _vec("scale", scale, N, _F32, index)
            self.N, self.K, self.scale = N, K, scale
            self.packed = torch.empty(_lib.packed_i8_bytes(N, K), dtype=_U8, device=w.device)
            _lib.ds_pack_i8(w, self.packed, N, K, ld)


def pack_i8(w, scale, stream=None):
    """Lay an int8 weight [N, K] with float32 scales [N] out for linear_i8 (once per weight)."""
    return PackedI8(w, scale, stream=stream)


def _out(out, n, N, dtype, device, index):
    """(tensor, address, type code, elements between rows) of a result [n, N]."""
    if out is None:
        if dtype not in _CODE:
            raise ValueError("dtype: torch.bfloat16 or torch.float32 expected, got %s" % dtype)
        out = torch.empty((n, N), dtype=dtype, device=device)
        return out, out.data_ptr(), _CODE[dtype], N
    rows, columns, ldo, at = _rows("out", out, _CODE)
    if rows != n or columns != N or at != index:
        _bad("out", "[%d, %d] on cuda:%d" % (n, N, index), out)
    return out, out.data_ptr(), _CODE[out.dtype], ldo


def linear_i8(a, a_scale, weight, out=None, dtype=torch.bfloat16, d_status=None, stream=None):
    """out[i][j] = (sum_k a[i][k] w[j][k]) * a_scale[i] * w_scale[j] for a int8 [n, K], a_scale float32 [n] and a
    PackedI8 weight. out: bfloat16 or float32 [n, N] (rows may lie apart), allocated with dtype when None."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_i8(a, a_scale, weight, out, dtype, d_status)
    if out is None and d_status is None and dtype in _CODE:
        r = _lib.calls().linear(a, a_scale, weight.packed, weight.scale, weight.N, weight.K, _CODE[dtype])
        if r is not None:
            return _check("ds_linear_i8", r) if type(r) is int else r
    n, K, lda, index = _rows("a", a, (_I8,))
    N = weight.N
    if K != weight.K or index != weight.packed.get_device():
        _bad("a", "[n, %d] on %s" % (weight.K, weight.packed.device), a)
    if a_scale is None:
        raise ValueError("a_scale is needed")
    sp = _vec("a_scale", a_scale, n, _F32, index)
    st = _status(d_status, index)
    out, op, code, ldo = _out(out, n, N, dtype, a.device, index)
    lib = _lib.load()
    need = lib.ds_linear_i8_workspace(n, N, K)
    ws = torch.empty(need, dtype=_U8, device=a.device) if need else None
    _check("ds_linear_i8", lib.ds_linear_i8(a.data_ptr(), lda, sp, weight.packed.data_ptr(), weight.scale.data_ptr(), n,
                                            N, K, op, code, ldo, None if ws is None else ws.data_ptr(), need, st,
                                            _lib.raw_stream()))
    return out


class Int8Head:
    """A model's output head in 8 bits: the final RMS norm (when gain is given), the vocabulary projection and the
    sampler. w int8 [N, K] with scale float32 [N]; from_weight() quantises a bfloat16 or float32 weight."""

    def __init__(self, w, scale, gain=None, eps=1e-6, stream=None):
        self.weight = pack_i8(w, scale, stream=stream)
        _vec("gain", gain, self.weight.K, _F32, w.get_device())
        self.gain, self.eps = gain, float(eps)

    @classmethod
    def from_weight(cls, w, gain=None, eps=1e-6):
        """Each channel of w [N, K] quantised with a scale of its own."""
        q, scale = quantize_rows(w)
        return cls(q, scale, gain=gain, eps=eps)

    def logits(self, hidden, out=None, dtype=torch.bfloat16, d_status=None, stream=None):
        """Logits [n, N] of hidden states [n, K] (bfloat16 or float32): quantize_rows() and linear_i8() in one call."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.logits(hidden, out, dtype, d_status)
        if out is None and d_status is None and dtype in _CODE:
            w = self.weight
            r = _lib.calls().head(hidden, self.gain, w.packed, w.scale, w.N, w.K, _CODE[dtype], self.eps)
            if r is not None:
                return _check("ds_head_i8", r) if type(r) is int else r
        n, K, ld, index = _rows("hidden", hidden, _CODE)
        weight, gain = self.weight, self.gain
        if K != weight.K or index != weight.packed.get_device():
            _bad("hidden", "[n, %d] on %s" % (weight.K, weight.packed.device), hidden)
        st = _status(d_status, index)
        out, op, code, ldo = _out(out, n, weight.N, dtype, hidden.device, index)
        lib = _lib.load()
        need = lib.ds_head_i8_workspace(n, weight.N, K)
        ws = torch.empty(need, dtype=_U8, device=hidden.device)
        _check("ds_head_i8", lib.ds_head_i8(hidden.data_ptr(), _CODE[hidden.dtype], n, K, ld,
                                            None if gain is None else gain.data_ptr(), self.eps,
                                            weight.packed.data_ptr(), weight.scale.data_ptr(), weight.N, op, code, ldo,
                                            ws.data_ptr(), need, st, _lib.raw_stream()))
        return out

    def sample(self, hidden, temperature, u, top_k=None, top_p=None, min_p=None, d_status=None, stream=None):
        """Hidden states [n, K] to (tokens, logprobs): logits() then sample_filtered()."""
        return sample_filtered(self.logits(hidden, d_status=d_status, stream=stream), temperature, u, top_k=top_k,
                               top_p=top_p, min_p=min_p, d_status=d_status, stream=stream)
