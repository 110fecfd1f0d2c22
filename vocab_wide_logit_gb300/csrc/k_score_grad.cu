// k_score_grad.cu -- gradient of log-probabilities and entropies with respect to
// the logits.
//
// With p = exp(x - lse), the forward pass's lse and entropy H, and the loss's
// gradient gl by the row's log-probability and gh by its entropy:
//   dx_j = gl (1[j = token] - p_j) - gh p_j (x_j - lse + H)
//        = gl 1[j = token] - p_j (gl + gh (x_j - lse + H)),
// in fp32, rounded once to the type of the logits. Every logit is read once and
// written once and nothing is shared between them but five numbers a row, so HBM
// bounds it: the 16-byte chunks of all rows are one list, each thread takes four of
// them 256 apart, which is the same for one long row and for many short ones.
// A row whose lse is -inf (nothing in it) gets zeros; a logit of probability zero
// gets exactly zero from the entropy, -inf among them.
#include "ds_device.cuh"
#include "ds_launch.h"

namespace ds {

namespace {

constexpr int kThreads = 256;
constexpr int kChunks = 4;  // 16-byte chunks a thread

// Not through the read-only path: the result may stand where the logits are.
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void st16(void* p, uint4 v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Two floats to a word of two bf16, the first in the low half, to nearest even.
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) k_score_grad(const ScoreGradArgs a, int nq) {
  constexpr int E = F32 ? 4 : 8;             // elements of a chunk
  constexpr int kSize = F32 ? 4 : 2;
  pdl_release();
  pdl_wait();
  const long long first = (long long)blockIdx.x * (kThreads * kChunks);
  const long long row0 = first / nq;
  const uint32_t rem = (uint32_t)(first - row0 * nq);
  uint4 v[kChunks];
  const char* row_at[kChunks];
  int row[kChunks], q[kChunks];
#pragma unroll
  for (int u = 0; u < kChunks; ++u) {
    const uint32_t i = rem + threadIdx.x + u * kThreads;
    const uint32_t down = i < (uint32_t)nq ? 0u : i / (uint32_t)nq;
    const long long r = row0 + down;
    row[u] = r < a.n ? (int)r : -1;
    q[u] = (int)(i - down * (uint32_t)nq);
    if (row[u] < 0) continue;
    row_at[u] = static_cast<const char*>(a.x) + r * a.ld * kSize;
    const uintptr_t at = reinterpret_cast<uintptr_t>(row_at[u]);
    const int dc = (int)(at & 15) / kSize;
    if ((long long)q[u] * E - dc >= a.V)
      row[u] = -1;  // the chunk that only rows starting further into a chunk have
    else
      v[u] = ld16(reinterpret_cast<const char*>(at & ~(uintptr_t)15) + 16LL * q[u]);
  }
#pragma unroll
  for (int u = 0; u < kChunks; ++u) {
    if (row[u] < 0) continue;
    const int r = row[u];
    const int token = a.tokens[r];
    const float lse = a.lse[r];
    const bool given = token >= 0 && token < a.V;
    if (q[u] == 0 && token >= a.V) report(a.d_status, DS_DEV_ERR_PARAM);
    const float gl = given && a.g_logprobs ? a.g_logprobs[r] : 0.f;
    const float gh = a.g_entropy ? a.g_entropy[r] : 0.f;
    const float shift = a.g_entropy ? a.entropy[r] : 0.f;
    const bool dead = lse == -kInf;
    const int dc = (int)(reinterpret_cast<uintptr_t>(row_at[u]) & 15) / kSize;
    const int id0 = q[u] * E - dc;
    float f[E];
    if constexpr (F32) {
      f[0] = __uint_as_float(v[u].x);
      f[1] = __uint_as_float(v[u].y);
      f[2] = __uint_as_float(v[u].z);
      f[3] = __uint_as_float(v[u].w);
    } else {
      unpack8(v[u], f);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float d = f[i] - lse;
      const float p = ex2_approx(d * kLog2e);
      // p = 0 has no part in the entropy; its d may be -inf
      const float w = p == 0.f ? 0.f : p * __fmaf_rn(gh, d + shift, gl);
      f[i] = dead ? 0.f : (id0 + i == token ? gl - w : -w);
    }
    char* out = static_cast<char*>(a.out) + (r * a.ldo + id0) * kSize;
    if (id0 >= 0 && (long long)id0 + E <= a.V && (reinterpret_cast<uintptr_t>(out) & 15) == 0) {
      if constexpr (F32)
        st16(out, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
      else
        st16(out, make_uint4(pack_bf(f[0], f[1]), pack_bf(f[2], f[3]), pack_bf(f[4], f[5]), pack_bf(f[6], f[7])));
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const long long id = (long long)id0 + i;
        if (id < 0 || id >= a.V) continue;
        if constexpr (F32)
          reinterpret_cast<float*>(out)[i] = f[i];
        else
          reinterpret_cast<uint16_t*>(out)[i] = (uint16_t)pack_bf(f[i], 0.f);
      }
    }
  }
}

}  // namespace

cudaError_t launch_score_grad(const ScoreGradArgs& a, bool f32, cudaStream_t st) {
  const int E = f32 ? 4 : 8;
  const int nq = (int)(((long long)a.V + 2 * E - 2) / E);
  const long long blocks = ((long long)a.n * nq + kThreads * kChunks - 1) / (kThreads * kChunks);
  if (blocks > 2147483647LL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = f32 ? cudaLaunchKernelEx(&cfg, k_score_grad<true>, a, nq)
                            : cudaLaunchKernelEx(&cfg, k_score_grad<false>, a, nq);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace ds
