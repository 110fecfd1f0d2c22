"""The serving head: hidden states to logits through an 8-bit vocabulary projection and each request's low-rank adapter,
and logits to tokens by temperature, top-k, top-p and min-p.

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
_ADAPTERS_MAX_SIZE = 2 ** 30
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


def _meet(given, ld, out, ldo):
    """Whether two matrices of one shape and type share memory."""
    n, columns = given.shape
    size = given.element_size()
    apart = (out.data_ptr() - given.data_ptr()) // size
    if apart >= (n - 1) * ld + columns or -apart >= (n - 1) * ldo + columns:
        return False
    # rows of one buffer side by side
    return not (n > 1 and ld == ldo and columns <= apart % ld <= ld - columns)


def _like(out, given, ld, index):
    """(tensor, elements between rows) of a result of the shape and type of `given`, whose rows are ld apart: a new one, or
    one that is `given` or shares no memory with it."""
    n, columns = given.shape
    if out is None:
        return torch.empty((n, columns), dtype=given.dtype, device=given.device), columns
    rows, width, ldo, at = _rows("out", out, (given.dtype,))
    if rows != n or width != columns or at != index:
        _bad("out", "[%d, %d] on cuda:%d" % (n, columns, index), out)
    if n and out.data_ptr() == given.data_ptr():
        if ldo != ld:
            _bad("out", "rows %d elements apart, as those of the tensor that it overwrites" % ld, out)
    elif n and _meet(given, ld, out, ldo):
        _bad("out", "the input itself or memory of its own", out)
    return out, ldo


def _stacks(a, b, scale):
    """(L, R, K, N) of the stacks of Adapters."""
    for name, t, what in (("a", a, "[L, R, K]"), ("b", b, "[L, N, R]")):
        if t.dim() != 3 or t.dtype != _BF16 or not t.is_cuda or not t.is_contiguous() or not t.numel():
            _bad(name, "a contiguous cuda bfloat16 tensor %s" % what, t)
    L, R, K = a.shape
    N = b.shape[1]
    if b.shape[0] != L or b.shape[2] != R or b.get_device() != a.get_device():
        _bad("b", "[%d, N, %d] on %s" % (L, R, a.device), b)
    if scale is None:
        raise ValueError("scale is needed")
    _vec("scale", scale, L, _F32, a.get_device())
    if L > _lib.DS_ADAPTERS_MAX or R > _lib.DS_ADAPTERS_MAX_RANK or max(N, K) > _ADAPTERS_MAX_SIZE:
        raise ValueError("at most %d adapters of rank %d at most on at most %d inputs and channels, got %d of rank %d on %d and %d" % (
            _lib.DS_ADAPTERS_MAX, _lib.DS_ADAPTERS_MAX_RANK, _ADAPTERS_MAX_SIZE, L, R, K, N))
    return L, R, K, N


class Adapters:
    """Low-rank adapters of one projection, in stacks: a bfloat16 [L, R, K], b bfloat16 [L, N, R], scale float32 [L], all
    contiguous on one device. Adapter i adds scale[i] * b[i] @ (a[i] @ y) to the projection of y. The tensors are used as
    they are, so that a program may rewrite the adapter in a slot between calls; one of a lower rank is filled up with
    zeros. Holds no workspace: calls on several streams may share it."""

    def __init__(self, a, b, scale):
        self.L, self.R, self.K, self.N = _stacks(a, b, scale)
        self.a, self.b, self.scale = a, b, scale


def _adapter_inputs(n, N, index, hidden, adapters, ids, gain, d_status):
    """Checks what goes with a base [n, N] on a device: (elements between hidden's rows, L, R, and the addresses of ids, gain and
    status)."""
    rows, K, ldx, at = _rows("hidden", hidden, _CODE)
    L, R, inputs, channels = _stacks(adapters.a, adapters.b, adapters.scale)  # as they are now
    if rows != n or K != inputs or at != index:
        _bad("hidden", "[%d, %d] on cuda:%d" % (n, inputs, index), hidden)
    if N != channels or adapters.a.get_device() != index:
        _bad("adapters", "of a projection [%d, %d] on cuda:%d" % (N, K, index), adapters.b)
    if ids is None:
        raise ValueError("ids are needed")
    return (ldx, L, R, _vec("ids", ids, n, _I32, index), _vec("gain", gain, K, _F32, index), _status(d_status, index))


def _add_adapters(base, ldb, hidden, adapters, inputs, eps, out, ldo):
    """The launch, of checked tensors; inputs: what _adapter_inputs() returned."""
    ldx, L, R, ids, gain, status = inputs
    n, N = base.shape
    lib = _lib.load()
    need = lib.ds_add_adapters_workspace(n, L, R)
    ws = torch.empty(need, dtype=_U8, device=base.device)
    _check("ds_add_adapters", lib.ds_add_adapters(
        base.data_ptr(), _CODE[base.dtype], n, N, ldb, hidden.data_ptr(), _CODE[hidden.dtype], hidden.shape[1], ldx, gain, eps,
        adapters.a.data_ptr(), adapters.b.data_ptr(), adapters.scale.data_ptr(), L, R, ids,
        out.data_ptr(), ldo, ws.data_ptr(), need, status, _lib.raw_stream()))
    return out


def add_adapters(base, hidden, adapters, ids, gain=None, eps=1e-6, out=None, d_status=None, stream=None):
    """Each row's low-rank adapter added to the logits of a projection that all rows share: base [n, N] (bfloat16 or
    float32) + scale B (A y) with the Adapters entry ids[row] (int32 [n], any order, -1 for none), y the hidden states
    [n, K] (bfloat16 or float32), RMS-normed with gain (float32 [K]) and eps when that is given. Sums are float32, rounded once
    to base's type; y and A y meet the adapters' bfloat16 as sums of bfloat16 parts that lose 2^-24 of them for float32 base
    and 2^-16 for bfloat16. out: such a tensor (rows may lie apart), base itself to add in place; allocated when None, up to
    an eighth of it more in memory than it shows (the workspace lies behind it). An id beyond the stack gives a row of NaN and
    a bit in d_status. Not recorded by autograd."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return add_adapters(base, hidden, adapters, ids, gain, eps, out, d_status)
    if out is None and d_status is None:
        r = _lib.calls().adapters(base, hidden, adapters.a, adapters.b, adapters.scale, ids, gain, eps)
        if r is not None:
            return _check("ds_add_adapters", r) if type(r) is int else r
    n, N, ldb, index = _rows("base", base, _CODE)
    inputs = _adapter_inputs(n, N, index, hidden, adapters, ids, gain, d_status)
    out, ldo = _like(out, base, ldb, index)
    return _add_adapters(base, ldb, hidden, adapters, inputs, eps, out, ldo)


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

    def logits(self, hidden, out=None, dtype=torch.bfloat16, d_status=None, stream=None, adapters=None, adapter_ids=None):
        """Logits [n, N] of hidden states [n, K] (bfloat16 or float32): quantize_rows() and linear_i8() in one call. With
        Adapters and an id per row (int32 [n], -1 for none) add_adapters() adds to them in place; bfloat16 logits are
        then rounded twice, before the sum and after it (float32 ones in effect once)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.logits(hidden, out, dtype, d_status, None, adapters, adapter_ids)
        if adapters is not None:
            # checked before the projection runs: a refused call leaves out as it was
            if adapter_ids is None:
                raise ValueError("adapter_ids are needed")
            n, _, _, index = _rows("hidden", hidden, _CODE)
            inputs = _adapter_inputs(n, self.weight.N, index, hidden, adapters, adapter_ids, self.gain, d_status)
            out = self.logits(hidden, out, dtype, d_status)
            ldo = out.stride(0) if n > 1 else self.weight.N
            return _add_adapters(out, ldo, hidden, adapters, inputs, self.eps, out, ldo)
        if adapter_ids is not None:
            raise ValueError("adapter_ids without adapters")
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

    def sample(self, hidden, temperature, u, top_k=None, top_p=None, min_p=None, d_status=None, stream=None, adapters=None,
               adapter_ids=None):
        """Hidden states [n, K] to (tokens, logprobs): logits() then sample_filtered()."""
        logits = self.logits(hidden, d_status=d_status, stream=stream, adapters=adapters, adapter_ids=adapter_ids)
        return sample_filtered(logits, temperature, u, top_k=top_k, top_p=top_p, min_p=min_p, d_status=d_status,
                               stream=stream)

    def score(self, hidden, tokens, top=0, d_status=None, stream=None, adapters=None, adapter_ids=None):
        """Hidden states [n, K] and a given token per row (int32 [n], -1 for none) to TokenScores: logits() then
        score_tokens()."""
        from .score import score_tokens
        logits = self.logits(hidden, d_status=d_status, stream=stream, adapters=adapters, adapter_ids=adapter_ids)
        return score_tokens(logits, tokens, top=top, d_status=d_status, stream=stream)
