"""libdsample: the GB300 vocab-wide sampling pass (CFG combine, max/logsumexp/argmax,
exact top-ratio filter, Gumbel-max) and the large-vocab greedy max/LSE/argmax pass.

The compute lives in the CUDA library (csrc/, built by build.py); the Python
side only marshals arguments through the C ABI declared in include/dsample.h.
"""
from ._lib import (DS_DEV_ERR_LAYOUT, DS_DEV_ERR_NO_UNCOND, DS_DEV_ERR_PARAM, DS_DTYPE_BF16, DS_DTYPE_F32,
                   DS_FLAG_KEEP_TIES, DS_FLAG_SKIP_EXACT_PASS, DS_MARKED, DS_MAX_VOCAB, DsError, ds_greedy_lse, ds_log_softmax, ds_merge_triples, ds_reveal, ds_sample, load,
                   launch_count, status_string, top_k)
from ._lib import (DS_DEV_ERR_LOGITS, DS_DEV_ERR_TIMEOUT, DS_FILTERED_MAX_VOCAB, DS_LINEAR_MAX_K, ds_head_i8,
                   ds_linear_i8, ds_pack_i8, ds_quantize_rows, ds_sample_filtered, head_i8_workspace, linear_i8_workspace,
                   packed_i8_bytes)
from ._lib import (DS_ADAPTERS_MAX, DS_ADAPTERS_MAX_RANK, DS_SCORE_MAX_TOP, add_adapters_workspace, ds_add_adapters,
                   ds_score_tokens, ds_score_tokens_grad)
from .api import greedy_lse, log_softmax, merge_triples, reveal, sample, sample_host
from .head import Adapters, Int8Head, PackedI8, add_adapters, linear_i8, pack_i8, quantize_rows, sample_filtered
from .score import TokenScores, score_tokens, score_tokens_grad

__all__ = ["ds_sample", "ds_greedy_lse", "ds_merge_triples", "ds_log_softmax", "ds_reveal", "sample",
           "sample_host", "greedy_lse", "merge_triples", "log_softmax", "reveal", "load", "top_k", "launch_count", "DS_DTYPE_F32", "DS_DTYPE_BF16",
           "status_string", "DsError", "DS_MAX_VOCAB", "DS_DEV_ERR_LAYOUT", "DS_DEV_ERR_NO_UNCOND",
           "ds_sample_filtered", "ds_quantize_rows", "ds_pack_i8", "ds_linear_i8", "sample_filtered", "quantize_rows",
           "pack_i8", "linear_i8", "ds_head_i8", "head_i8_workspace", "PackedI8", "Int8Head", "packed_i8_bytes", "linear_i8_workspace",
           "DS_DEV_ERR_LOGITS", "DS_DEV_ERR_TIMEOUT", "DS_FILTERED_MAX_VOCAB", "DS_LINEAR_MAX_K",
           "Adapters", "TokenScores", "add_adapters", "score_tokens", "score_tokens_grad", "ds_add_adapters",
           "ds_score_tokens", "ds_score_tokens_grad", "add_adapters_workspace", "DS_ADAPTERS_MAX", "DS_ADAPTERS_MAX_RANK",
           "DS_SCORE_MAX_TOP", "DS_DEV_ERR_PARAM", "DS_FLAG_KEEP_TIES", "DS_FLAG_SKIP_EXACT_PASS", "DS_MARKED"]
