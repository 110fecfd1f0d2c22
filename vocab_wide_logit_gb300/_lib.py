"""ctypes binding of libdsample (argument marshalling only).

Every step of the sampling and greedy passes runs in the CUDA library; this
module only turns torch tensors into device pointers and the current CUDA
stream into a handle. There is no fallback: if the library is missing the
import of a call raises.
"""
import ctypes
import importlib.util
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_build", "libdsample.so")

DS_OK = 0
DS_ERR_INVALID_ARG = 1
DS_ERR_UNSUPPORTED = 2
DS_ERR_CUDA = 3
DS_DEV_ERR_LAYOUT = 1
DS_DEV_ERR_NO_UNCOND = 2
DS_DEV_ERR_PARAM = 4
DS_DEV_ERR_LOGITS = 8
DS_DEV_ERR_TIMEOUT = 16
DS_MAX_VOCAB = 524281
DS_FILTERED_MAX_VOCAB = 2097152
DS_LINEAR_MAX_K = 131071
DS_SCORE_MAX_TOP = 128
DS_ADAPTERS_MAX = 8192
DS_ADAPTERS_MAX_RANK = 128

EXPORTED = ("ds_sample", "ds_greedy_lse", "ds_status_string", "ds_top_k", "ds_merge_triples", "ds_log_softmax",
            "ds_reveal", "ds_sample_ex", "ds_launch_count", "ds_sample_filtered", "ds_quantize_rows",
            "ds_packed_i8_bytes", "ds_pack_i8", "ds_linear_i8_workspace", "ds_linear_i8", "ds_head_i8_workspace",
            "ds_head_i8", "ds_score_tokens", "ds_score_tokens_grad", "ds_add_adapters_workspace", "ds_add_adapters")
DS_FLAG_KEEP_TIES = 1
DS_FLAG_SKIP_EXACT_PASS = 2
DS_MARKED = -2
DS_DTYPE_F32 = 0
DS_DTYPE_BF16 = 1

_lib = None
_calls = None


class DsError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (fn, status_string(code), code))


def load(path: str = LIB_PATH):
    """Load libdsample.so (raises OSError when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError("libdsample.so not built at %s: run __graft_entry__.build() or "
                      "python vocab_wide_logit_gb300/build.py" % path)
    L = ctypes.CDLL(path)
    vp, i32, u32, u64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float
    L.ds_sample.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, f32, u64, u32, vp, vp, vp, vp]
    L.ds_sample.restype = ctypes.c_int
    L.ds_greedy_lse.argtypes = [vp, i32, i32, vp, vp, vp, vp]
    L.ds_greedy_lse.restype = ctypes.c_int
    L.ds_status_string.argtypes = [ctypes.c_int]
    L.ds_status_string.restype = ctypes.c_char_p
    L.ds_top_k.argtypes = [f32, i32]
    L.ds_top_k.restype = i32
    L.ds_launch_count.argtypes = []
    L.ds_launch_count.restype = ctypes.c_uint64
    L.ds_merge_triples.argtypes = [vp, i32, i32, vp, vp, vp, vp]
    L.ds_merge_triples.restype = ctypes.c_int
    L.ds_log_softmax.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp, vp]
    L.ds_log_softmax.restype = ctypes.c_int
    L.ds_reveal.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp]
    L.ds_reveal.restype = ctypes.c_int
    L.ds_sample_ex.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, f32, u64, vp, u32, u32, vp, vp, vp,
                               vp]
    L.ds_sample_ex.restype = ctypes.c_int
    i64 = ctypes.c_int64
    L.ds_sample_filtered.argtypes = [vp, i32, i32, i32, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.ds_sample_filtered.restype = ctypes.c_int
    L.ds_quantize_rows.argtypes = [vp, i32, i32, i32, i64, vp, f32, vp, vp, vp]
    L.ds_quantize_rows.restype = ctypes.c_int
    L.ds_packed_i8_bytes.argtypes = [i32, i32]
    L.ds_packed_i8_bytes.restype = i64
    L.ds_pack_i8.argtypes = [vp, i32, i32, i64, vp, vp]
    L.ds_pack_i8.restype = ctypes.c_int
    L.ds_linear_i8_workspace.argtypes = [i32, i32, i32]
    L.ds_linear_i8_workspace.restype = i64
    L.ds_linear_i8.argtypes = [vp, i64, vp, vp, vp, i32, i32, i32, vp, i32, i64, vp, i64, vp, vp]
    L.ds_linear_i8.restype = ctypes.c_int
    L.ds_head_i8_workspace.argtypes = [i32, i32, i32]
    L.ds_head_i8_workspace.restype = i64
    L.ds_head_i8.argtypes = [vp, i32, i32, i32, i64, vp, f32, vp, vp, i32, vp, i32, i64, vp, i64, vp, vp]
    L.ds_head_i8.restype = ctypes.c_int
    L.ds_score_tokens.argtypes = [vp, i32, i32, i32, i64, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    L.ds_score_tokens.restype = ctypes.c_int
    L.ds_score_tokens_grad.argtypes = [vp, i32, i32, i32, i64, vp, vp, vp, vp, vp, vp, i64, vp, vp]
    L.ds_score_tokens_grad.restype = ctypes.c_int
    L.ds_add_adapters_workspace.argtypes = [i32, i32, i32]
    L.ds_add_adapters_workspace.restype = i64
    L.ds_add_adapters.argtypes = [vp, i32, i32, i32, i64, vp, i32, i32, i64, vp, f32, vp, vp, vp, i32, i32, vp, vp, i64,
                                  vp, i64, vp, vp]
    L.ds_add_adapters.restype = ctypes.c_int
    _lib = L
    return L


def status_string(code: int) -> str:
    return load().ds_status_string(int(code)).decode()


def top_k(top_ratio: float, V: int) -> int:
    return int(load().ds_top_k(float(top_ratio), int(V)))


def launch_count() -> int:
    """Kernels the library has launched in this process so far (ds_launch_count)."""
    return int(load().ds_launch_count())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, t):
    """Handle of the stream (None: the current one) that a call on t is launched on. The addresses of another device's
    tensors would fault or race there."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    index = getattr(stream, "device_index", None)  # another library's stream may not say
    if t is not None and index is not None and t.is_cuda and t.get_device() != index:
        raise ValueError("a tensor on cuda:%d for a stream of cuda:%d (the current stream unless one is given)"
                         % (t.get_device(), index))
    return ctypes.c_void_p(stream.cuda_stream)


def ds_sample(request_ids, c_logits, u_logits, seq_lens, guidance, temperature, top_ratio, seed,
              iteration, out_tokens, out_logprobs, d_status=None, B=None, C=None, P=None, V=None,
              stream=None, check=True, top_ratios=None, iterations=None, keep_ties=False, flags=0):
    """Call ds_sample (ds_sample_ex when per-request top_ratios / iterations are given) on device
    tensors. Shapes: c_logits [C, P, V] bf16, u_logits [C, P_u, V] bf16 or None,
    request_ids/seq_lens int32 [B], guidance/temperature float32 [B], top_ratios float32 [B] or
    None, iterations int32/uint32 [B] or None, out_tokens int32 [C, P], out_logprobs float32
    [C, P], d_status uint32/int32 [1] or None. flags: extra DS_FLAG_* bits (keep_ties sets
    DS_FLAG_KEEP_TIES)."""
    if C is None:
        C, P, V = c_logits.shape
    if B is None:
        B = seq_lens.shape[0]
    flags = int(flags) | (DS_FLAG_KEEP_TIES if keep_ties else 0)
    if top_ratios is None and iterations is None and flags == 0:
        rc = load().ds_sample(_ptr(request_ids), _ptr(c_logits), _ptr(u_logits), _ptr(seq_lens), int(B),
                              int(C), int(P), int(V), _ptr(guidance), _ptr(temperature), float(top_ratio),
                              int(seed) & (2 ** 64 - 1), int(iteration), _ptr(out_tokens), _ptr(out_logprobs),
                              _ptr(d_status), _stream(stream, c_logits))
        name = "ds_sample"
    else:
        rc = load().ds_sample_ex(_ptr(request_ids), _ptr(c_logits), _ptr(u_logits), _ptr(seq_lens), int(B),
                                 int(C), int(P), int(V), _ptr(guidance), _ptr(temperature), _ptr(top_ratios),
                                 float(top_ratio), int(seed) & (2 ** 64 - 1), _ptr(iterations), int(iteration),
                                 flags, _ptr(out_tokens), _ptr(out_logprobs),
                                 _ptr(d_status), _stream(stream, c_logits))
        name = "ds_sample_ex"
    if check and rc != DS_OK:
        raise DsError(name, rc)
    return rc


def ds_greedy_lse(logits, out_max, out_lse, out_argmax, n=None, V=None, stream=None, check=True):
    """Call ds_greedy_lse on device tensors: logits [n, V] bf16, outputs [n] float32/float32/int32."""
    if n is None:
        n, V = logits.shape
    rc = load().ds_greedy_lse(_ptr(logits), int(n), int(V), _ptr(out_max), _ptr(out_lse), _ptr(out_argmax),
                              _stream(stream, logits))
    if check and rc != DS_OK:
        raise DsError("ds_greedy_lse", rc)
    return rc


def ds_merge_triples(triples, out_max, out_lse, out_argmax, n=None, shards=None, stream=None, check=True):
    """Call ds_merge_triples: triples float32 [n, shards, 3] (max, lse, global argmax bits)."""
    if n is None:
        n, shards = triples.shape[0], triples.shape[1]
    rc = load().ds_merge_triples(_ptr(triples), int(n), int(shards), _ptr(out_max), _ptr(out_lse),
                                 _ptr(out_argmax), _stream(stream, triples))
    if check and rc != DS_OK:
        raise DsError("ds_merge_triples", rc)
    return rc


def ds_log_softmax(logits, out, out_max, out_lse, out_argmax, out_dtype=None, n=None, V=None, stream=None,
                   check=True):
    """Call ds_log_softmax: logits [n, V] bf16; out [n, V] float32 or bfloat16."""
    import torch
    if n is None:
        n, V = logits.shape
    if out_dtype is None:
        out_dtype = DS_DTYPE_BF16 if out.dtype == torch.bfloat16 else DS_DTYPE_F32
    rc = load().ds_log_softmax(_ptr(logits), int(n), int(V), _ptr(out), int(out_dtype), _ptr(out_max),
                               _ptr(out_lse), _ptr(out_argmax), _stream(stream, logits))
    if check and rc != DS_OK:
        raise DsError("ds_log_softmax", rc)
    return rc


def ds_reveal(scores, tokens, seq_lens, reveal_counts, canvas, revealed=None, d_status=None, B=None, C=None,
              P=None, stream=None, check=True):
    """Call ds_reveal: scores float32 [C, P], tokens/canvas int32 [C, P], seq_lens/reveal_counts int32 [B],
    revealed uint8 [C, P] or None."""
    if C is None:
        C, P = scores.shape
    if B is None:
        B = seq_lens.shape[0]
    rc = load().ds_reveal(_ptr(scores), _ptr(tokens), _ptr(seq_lens), _ptr(reveal_counts), int(B), int(C),
                          int(P), _ptr(canvas), _ptr(revealed), _ptr(d_status), _stream(stream, scores))
    if check and rc != DS_OK:
        raise DsError("ds_reveal", rc)
    return rc


def calls():
    """The module that runs the serving head's calls on torch tensors (csrc/py_calls.cpp), bound to the library."""
    global _calls
    if _calls is None:
        L, path = load(), os.path.join(os.path.dirname(LIB_PATH), "ds_calls.so")
        if not os.path.exists(path):
            raise OSError("ds_calls.so not built at %s: run __graft_entry__.build() or "
                          "python vocab_wide_logit_gb300/build.py" % path)
        import torch  # noqa: F401  (its libraries are what the module links to)
        from .build import torch_identity
        try:
            with open(os.path.splitext(path)[0] + ".torch") as f:
                built_with = f.read()
        except OSError:
            built_with = None
        if built_with != torch_identity():
            raise OSError("%s was built for another torch: run __graft_entry__.build() or "
                          "python vocab_wide_logit_gb300/build.py" % path)
        spec = importlib.util.spec_from_file_location("ds_calls", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.ds_sample_filtered, L.ds_linear_i8_workspace, L.ds_linear_i8, L.ds_head_i8_workspace, L.ds_head_i8,
            L.ds_quantize_rows, L.ds_score_tokens, L.ds_score_tokens_grad, L.ds_add_adapters_workspace,
            L.ds_add_adapters)))
        _calls = module
    return _calls


def raw_stream():
    """Handle of the current stream of the current device, without making a stream object for it."""
    import torch
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return DS_DTYPE_BF16
    if t.dtype == torch.float32:
        return DS_DTYPE_F32
    raise TypeError("bfloat16 or float32 expected, got %s" % t.dtype)


def ds_sample_filtered(logits, temperature, u, out_tokens, out_logprobs, top_k=None, top_p=None, min_p=None,
                       d_status=None, n=None, V=None, ld=None, stream=None, check=True):
    """Call ds_sample_filtered: logits [n, V] bfloat16 or float32 (rows ld elements apart), temperature / u / top_p /
    min_p float32 [n], top_k int32 [n], out_tokens int32 [n], out_logprobs float32 [n]."""
    if n is None:
        n, V = logits.shape
    if ld is None:
        ld = logits.stride(0) if n > 1 else V
    rc = load().ds_sample_filtered(logits.data_ptr(), _dtype_code(logits), n, V, ld, _ptr(temperature), _ptr(top_k),
                                   _ptr(top_p), _ptr(min_p), _ptr(u), _ptr(out_tokens), _ptr(out_logprobs),
                                   _ptr(d_status), _stream(stream, logits))
    if check and rc != DS_OK:
        raise DsError("ds_sample_filtered", rc)
    return rc


def ds_quantize_rows(x, out_q, out_scale, gain=None, eps=1e-6, n=None, K=None, ld=None, stream=None, check=True):
    """Call ds_quantize_rows: x [n, K] bfloat16 or float32, gain float32 [K] or None, out_q int8 [n, K] dense,
    out_scale float32 [n]."""
    if n is None:
        n, K = x.shape
    if ld is None:
        ld = x.stride(0) if n > 1 else K
    rc = load().ds_quantize_rows(x.data_ptr(), _dtype_code(x), n, K, ld, _ptr(gain), float(eps), _ptr(out_q),
                                 _ptr(out_scale), _stream(stream, x))
    if check and rc != DS_OK:
        raise DsError("ds_quantize_rows", rc)
    return rc


def packed_i8_bytes(N: int, K: int) -> int:
    return int(load().ds_packed_i8_bytes(int(N), int(K)))


def linear_i8_workspace(n: int, N: int, K: int) -> int:
    return int(load().ds_linear_i8_workspace(int(n), int(N), int(K)))


def head_i8_workspace(n: int, N: int, K: int) -> int:
    return int(load().ds_head_i8_workspace(int(n), int(N), int(K)))


def ds_head_i8(x, packed, w_scale, out, workspace, N, gain=None, eps=1e-6, d_status=None, n=None, K=None, ld=None,
               ldo=None, out_dtype=None, workspace_bytes=None, stream=None, check=True):
    """Call ds_head_i8: x [n, K] bfloat16 or float32, packed / w_scale of an [N, K] weight, out [n, N] bfloat16 or
    float32, workspace uint8 of ds_head_i8_workspace(n, N, K) bytes."""
    if n is None:
        n, K = x.shape
    if ld is None:
        ld = x.stride(0) if n > 1 else K
    if ldo is None:
        ldo = out.stride(0) if n > 1 else N
    if out_dtype is None:
        out_dtype = _dtype_code(out)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = load().ds_head_i8(x.data_ptr(), _dtype_code(x), n, K, ld, _ptr(gain), float(eps), _ptr(packed), _ptr(w_scale),
                           N, _ptr(out), out_dtype, ldo, _ptr(workspace), workspace_bytes, _ptr(d_status),
                           _stream(stream, x))
    if check and rc != DS_OK:
        raise DsError("ds_head_i8", rc)
    return rc


def ds_pack_i8(w, packed, N=None, K=None, ldw=None, stream=None, check=True):
    """Call ds_pack_i8: w int8 [N, K], packed uint8 [ds_packed_i8_bytes(N, K)]."""
    if N is None:
        N, K = w.shape
    if ldw is None:
        ldw = w.stride(0) if N > 1 else K
    rc = load().ds_pack_i8(_ptr(w), N, K, ldw, _ptr(packed), _stream(stream, w))
    if check and rc != DS_OK:
        raise DsError("ds_pack_i8", rc)
    return rc


def ds_linear_i8(a, a_scale, packed, w_scale, out, N, K, workspace=None, d_status=None, n=None, lda=None, ldo=None,
                 out_dtype=None, workspace_bytes=None, stream=None, check=True):
    """Call ds_linear_i8: a int8 [n, K], a_scale float32 [n], packed uint8 (ds_pack_i8), w_scale float32 [N], out
    [n, N] bfloat16 or float32, workspace uint8 of ds_linear_i8_workspace(n, N, K) bytes or None."""
    if n is None:
        n = a.shape[0]
    if lda is None:
        lda = a.stride(0) if n > 1 else K
    if ldo is None:
        ldo = out.stride(0) if n > 1 else N
    if out_dtype is None:
        out_dtype = _dtype_code(out)
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ds_linear_i8(a.data_ptr(), lda, _ptr(a_scale), _ptr(packed), _ptr(w_scale), n, N, K, _ptr(out),
                             out_dtype, ldo, _ptr(workspace), workspace_bytes, _ptr(d_status), _stream(stream, a))
    if check and rc != DS_OK:
        raise DsError("ds_linear_i8", rc)
    return rc


def ds_score_tokens(logits, tokens, out_logprobs, out_lse=None, out_entropy=None, out_ranks=None, out_top_ids=None,
                    out_top_logprobs=None, top=None, d_status=None, n=None, V=None, ld=None, stream=None, check=True):
    """Call ds_score_tokens: logits [n, V] bfloat16 or float32 (rows ld elements apart), tokens int32 [n], out_logprobs /
    out_lse / out_entropy float32 [n], out_ranks int32 [n], out_top_ids int32 and out_top_logprobs float32 [n, top]."""
    if n is None:
        n, V = logits.shape
    if ld is None:
        ld = logits.stride(0) if n > 1 else V
    if top is None:
        top = 0 if out_top_ids is None else out_top_ids.shape[1]
    rc = load().ds_score_tokens(logits.data_ptr(), _dtype_code(logits), n, V, ld, _ptr(tokens), top, _ptr(out_logprobs),
                                _ptr(out_lse), _ptr(out_entropy), _ptr(out_ranks), _ptr(out_top_ids),
                                _ptr(out_top_logprobs), _ptr(d_status), _stream(stream, logits))
    if check and rc != DS_OK:
        raise DsError("ds_score_tokens", rc)
    return rc


def ds_score_tokens_grad(logits, tokens, lse, out, entropy=None, g_logprobs=None, g_entropy=None, d_status=None, n=None,
                         V=None, ld=None, ldo=None, stream=None, check=True):
    """Call ds_score_tokens_grad: logits and out [n, V] of one type, tokens int32 [n], lse / entropy / g_logprobs /
    g_entropy float32 [n]."""
    if n is None:
        n, V = logits.shape
    if ld is None:
        ld = logits.stride(0) if n > 1 else V
    if ldo is None:
        ldo = out.stride(0) if n > 1 else V
    rc = load().ds_score_tokens_grad(logits.data_ptr(), _dtype_code(logits), n, V, ld, _ptr(tokens), _ptr(lse),
                                     _ptr(entropy), _ptr(g_logprobs), _ptr(g_entropy), _ptr(out), ldo, _ptr(d_status),
                                     _stream(stream, logits))
    if check and rc != DS_OK:
        raise DsError("ds_score_tokens_grad", rc)
    return rc


def add_adapters_workspace(n: int, L: int, R: int) -> int:
    return int(load().ds_add_adapters_workspace(int(n), int(L), int(R)))


def ds_add_adapters(base, x, a, b, scale, ids, out, workspace, gain=None, eps=1e-6, d_status=None, n=None, N=None,
                    K=None, L=None, R=None, ldb=None, ldx=None, ldo=None, workspace_bytes=None, stream=None, check=True):
    """Call ds_add_adapters: base and out [n, N] of one type, x [n, K], a bfloat16 [L, R, K], b bfloat16 [L, N, R], scale
    float32 [L], ids int32 [n], gain float32 [K] or None, workspace uint8 of ds_add_adapters_workspace(n, L, R) bytes."""
    if n is None:
        n, N = base.shape
    if K is None:
        K = x.shape[1]
    if L is None:
        L, R = a.shape[:2]
    if ldb is None:
        ldb = base.stride(0) if n > 1 else N
    if ldx is None:
        ldx = x.stride(0) if n > 1 else K
    if ldo is None:
        ldo = out.stride(0) if n > 1 else N
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = load().ds_add_adapters(base.data_ptr(), _dtype_code(base), n, N, ldb, x.data_ptr(), _dtype_code(x), K, ldx,
                                _ptr(gain), float(eps), _ptr(a), _ptr(b), _ptr(scale), L, R, _ptr(ids), _ptr(out), ldo,
                                _ptr(workspace), workspace_bytes, _ptr(d_status), _stream(stream, base))
    if check and rc != DS_OK:
        raise DsError("ds_add_adapters", rc)
    return rc
