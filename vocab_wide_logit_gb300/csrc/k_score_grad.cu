// k_score_grad.cu -- gradient of log-probabilities and entropies with respect to
// the logits.
//
// With p = exp(x - lse), the forward pass's lse and entropy H, and the loss's
// gradient gl by the row's log-probability and gh by its entropy:
//   dx_j = gl (1[j = token] - p_j) - gh p_j (x_j - lse + H)
//        = gl 1[j = token] - p_j (gl + gh (x_j - lse + H)),
// in fp32, rounded once to the type of the logits. Every logit is read once and
// written once and nothing is shared between them but five numbers a row, so HBM
// bounds it, as long as a bf16 logit costs fewer than about ten instructions: packed
// fp32 differences and products, the entropy's guard as one packed maximum (a logit
// 256 below lse counts as that; its p is 0, and -inf stays out of a product with it),
// the given token apart. The 16-byte chunks of all rows are one list, each thread takes
// four of them 256 apart, which is the same for one long row and for many short ones;
// a CTA whose chunks are one row's reads the row's numbers once. 256 x 248320 bf16: 38 us,
// 6.7 TB/s; 300 x 70001 fp32 with the entropy: 26 us, 6.5 TB/s (55 and 33 us with 28
// instructions a logit).
// A row whose lse is -inf (nothing in it) gets zeros; a logit of probability zero
// gets exactly zero from the entropy, -inf among them.
#include "ds_device.cuh"
#include "ds_index.h"
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

// What a row's logits share.
struct RowGrad {
  float lse, gl, c, h;  // the gradient is -p (c + h (x - lse)), c = gl + gh H, h = gh
  uint32_t low2;        // bf16: what x may not fall below, twice
  int token;            // -1: none
  bool dead, low;       // nothing in the row; lse so low that nothing finite lies 256 below it
};
template <bool ENT>
__device__ __forceinline__ RowGrad row_grad(const ScoreGradArgs& a, int r) {
  RowGrad g;
  const int token = a.tokens[r];
  g.token = token < a.V ? token : -1;
  g.lse = a.lse[r];
  g.gl = g.token >= 0 && a.g_logprobs ? a.g_logprobs[r] : 0.f;
  g.c = g.gl;
  g.h = 0.f;
  g.dead = g.lse == -kInf;
  g.low = g.lse < -1e38f;
  if constexpr (ENT) {
    g.h = a.g_entropy[r];
    g.c = __fmaf_rn(g.h, a.entropy[r], g.gl);
    // 192 below lse or more whatever the rounding to bf16 (up to 2^-8 of it, a quarter of the distance for large lse): the
    // exponential is 0 there
    const float low = g.lse - fmaxf(256.f, fabsf(g.lse) * 0.015625f);
    g.low2 = pack_bf(low, low);
  }
  return g;
}

template <bool F32, bool ENT>
__device__ __forceinline__ uint4 chunk_grad(const uint4& v, const RowGrad& g, int first) {
  constexpr int E = F32 ? 4 : 8;
  if (g.dead) return make_uint4(0, 0, 0, 0);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const float2 nl = make_float2(-g.lse, -g.lse), l2e = make_float2(kLog2e, kLog2e);
  const float2 nc = make_float2(-g.c, -g.c), nh = make_float2(-g.h, -g.h);
  float2 f[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    float2 x;
    if constexpr (F32) {
      x = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
      uint32_t c = w[i];
      if constexpr (ENT)
        if (!g.low) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(c), "r"(g.low2));
      x = make_float2(bf_lo(c), bf_hi(c));
    }
    float2 d = __fadd2_rn(x, nl);
    const float2 t = __fmul2_rn(d, l2e);
    const float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
    if constexpr (ENT) {
      if (F32 || g.low) d = make_float2(fmaxf(d.x, -256.f), fmaxf(d.y, -256.f));
      f[i] = __fmul2_rn(p, __ffma2_rn(nh, d, nc));
    } else {
      f[i] = __fmul2_rn(p, nc);
    }
  }
  const unsigned at = place_of(g.token, first);  // the given token's own part
  if (g.token >= 0 && at < E) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      if (at == 2 * i) f[i].x += g.gl;
      if (at == 2 * i + 1) f[i].y += g.gl;
    }
  }
  if constexpr (F32)
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
  else
    return make_uint4(pack_bf(f[0].x, f[0].y), pack_bf(f[1].x, f[1].y), pack_bf(f[2].x, f[2].y), pack_bf(f[3].x, f[3].y));
}

template <bool F32, bool ENT>
__global__ void __launch_bounds__(kThreads) k_score_grad(const ScoreGradArgs a, int nq) {
  constexpr int E = F32 ? 4 : 8;  // elements of a chunk
  constexpr int kSize = F32 ? 4 : 2;
  pdl_release();
  pdl_wait();
  const long long first = (long long)blockIdx.x * (kThreads * kChunks);
  const long long row0 = first / nq;
  const uint32_t rem = (uint32_t)(first - row0 * nq);
  auto write = [&](char* out, int id0, const uint4& z) {
    if (all_in_row(id0, E, a.V) && (reinterpret_cast<uintptr_t>(out) & 15) == 0) {
      st16(out, z);
    } else {
      const uint32_t w[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (!in_row(id0, i, a.V)) continue;
        if constexpr (F32)
          reinterpret_cast<uint32_t*>(out)[i] = w[i];
        else
          reinterpret_cast<uint16_t*>(out)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
      }
    }
  };
  if (rem + kThreads * kChunks <= (uint32_t)nq) {
    // one row
    const char* x = static_cast<const char*>(a.x) + row0 * a.ld * kSize;
    const int dc = (int)(reinterpret_cast<uintptr_t>(x) & 15) / kSize;
    const uint32_t q = rem + threadIdx.x, chunks = chunks_of(a.V, E, dc);
    const int id0 = first_of_chunk(q, E, dc);
    x += (long long)id0 * kSize;
    uint4 v[kChunks];
#pragma unroll
    for (int u = 0; u < kChunks; ++u)
      if (q + u * kThreads < chunks) v[u] = ld16(x + u * kThreads * 16);
    const RowGrad g = row_grad<ENT>(a, (int)row0);
    char* out = static_cast<char*>(a.out) + (row0 * a.ldo + id0) * kSize;
#pragma unroll
    for (int u = 0; u < kChunks; ++u)
      if (q + u * kThreads < chunks)
        write(out + u * kThreads * 16, id0 + u * kThreads * E, chunk_grad<F32, ENT>(v[u], g, id0 + u * kThreads * E));
    if (rem == 0 && threadIdx.x == 0 && a.tokens[row0] >= a.V) report(a.d_status, DS_DEV_ERR_PARAM);
    return;
  }
  uint4 v[kChunks];
  int row[kChunks], at[kChunks];
#pragma unroll
  for (int u = 0; u < kChunks; ++u) {
    const uint32_t i = rem + threadIdx.x + u * kThreads;
    const uint32_t down = i < (uint32_t)nq ? 0u : i / (uint32_t)nq, q = i - down * (uint32_t)nq;
    const long long r = row0 + down;
    row[u] = -1;
    if (r >= a.n) continue;
    const char* x = static_cast<const char*>(a.x) + r * a.ld * kSize;
    const long long id0 = (long long)q * E - (int)(reinterpret_cast<uintptr_t>(x) & 15) / kSize;
    if (id0 >= a.V) continue;  // the chunk that only rows starting further into a chunk have
    row[u] = (int)r;
    at[u] = (int)id0;
    v[u] = ld16(x + id0 * kSize);
    if (q == 0 && a.tokens[r] >= a.V) report(a.d_status, DS_DEV_ERR_PARAM);
  }
#pragma unroll
  for (int u = 0; u < kChunks; ++u) {
    if (row[u] < 0) continue;
    const RowGrad g = row_grad<ENT>(a, row[u]);
    write(static_cast<char*>(a.out) + (row[u] * a.ldo + at[u]) * kSize, at[u], chunk_grad<F32, ENT>(v[u], g, at[u]));
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
  const auto kern = a.g_entropy ? (f32 ? k_score_grad<true, true> : k_score_grad<false, true>)
                                : (f32 ? k_score_grad<true, false> : k_score_grad<false, false>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, nq);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace ds
