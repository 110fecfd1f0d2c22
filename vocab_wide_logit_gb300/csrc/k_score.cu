// k_score.cu -- log-probabilities of given tokens, with log-sum-exp, entropy, rank
// and the most likely alternatives.
//
// Per row, with m = max x, e_j = exp(x_j - m) and s = sum e:
//   lse = m + log s,  logprob = x_token - lse,  H = log s - (sum e_j (x_j - m)) / s,
//   rank = how many come before the token by (x descending, id ascending),
// and the first `top` of that order. One CTA per row, the row read once for m, once
// for the sums and once for each alternative.
#include "ds_device.cuh"
#include "ds_launch.h"

namespace ds {

namespace {

constexpr int kThreads = 256;

template <bool F32>
__device__ __forceinline__ float load(const void* row, long long i) {
  if constexpr (F32)
    return static_cast<const float*>(row)[i];
  else
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(row)[i] << 16);
}

// The order (x descending, id ascending; -0 and +0 tie) as an integer.
__device__ __forceinline__ unsigned long long order_of(float x, int id) {
  return ((unsigned long long)order_key(x + 0.f) << 32) | (uint32_t)~id;
}

struct Sum {
  __device__ float operator()(float p, float q) const { return p + q; }
};
struct Max {
  template <typename T>
  __device__ T operator()(T p, T q) const {
    return p > q ? p : q;
  }
};

template <typename T, typename F>
__device__ T cta_reduce(T v, F f) {
  __shared__ T part[kThreads / 32];
  __syncthreads();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
  for (int i = 1; i < kThreads / 32; ++i) v = f(v, part[i]);
  return v;
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) k_score(const ScoreArgs a) {
  pdl_release();
  pdl_wait();
  const float nan = __int_as_float(0x7fffffff);
  for (int row = blockIdx.x; row < a.n; row += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + (long long)row * a.ld * (F32 ? 4 : 2);
    const int token = a.tokens[row];
    const bool given = token >= 0 && token < a.V;
    const float at = given ? load<F32>(x, token) : 0.f;
    float m = -kInf;
    int bad = 0;
    for (long long i = threadIdx.x; i < a.V; i += kThreads) {
      const float v = load<F32>(x, i);
      bad |= !(v < kInf);
      m = fmaxf(m, v);
    }
    m = cta_reduce(m, Max());
    bad = __syncthreads_or(bad);
    float s = 0.f, t = 0.f;
    int before = 0;
    for (long long i = threadIdx.x; i < a.V; i += kThreads) {
      const float v = load<F32>(x, i), d = v - m, e = __expf(d);
      s += e;
      t += e > 0.f ? e * d : 0.f;
      before += v > at || (v == at && i < token);
    }
    s = cta_reduce(s, Sum());
    t = cta_reduce(t, Sum());
    const int rank = (int)cta_reduce((float)(before >> 12), Sum()) * 4096 + (int)cta_reduce((float)(before & 4095), Sum());
    const bool none = bad || m == -kInf;
    const float lse = bad ? nan : none ? -kInf : m + logf(s);
    if (threadIdx.x == 0) {
      a.out_logprobs[row] = none || !given ? nan : at - lse;
      if (a.out_lse) a.out_lse[row] = lse;
      if (a.out_entropy) a.out_entropy[row] = none ? nan : logf(s) - t / s;
      if (a.out_ranks) a.out_ranks[row] = none || !given ? -1 : rank;
      const uint32_t bits = (token >= a.V ? DS_DEV_ERR_PARAM : 0u) | (bad ? DS_DEV_ERR_LOGITS : 0u);
      if (bits) report(a.d_status, bits);
    }
    unsigned long long last = ~0ull;
    for (int j = 0; j < a.top; ++j) {
      unsigned long long best = 0;
      if (!none)
        for (long long i = threadIdx.x; i < a.V; i += kThreads) {
          const unsigned long long o = order_of(load<F32>(x, i), (int)i);
          if (o < last && o > best) best = o;
        }
      best = cta_reduce(best, Max());
      last = best;
      if (threadIdx.x == 0) {
        const int id = none ? -1 : (int)~(uint32_t)best;
        a.out_top_ids[(long long)row * a.top + j] = id;
        a.out_top_logprobs[(long long)row * a.top + j] = none ? nan : load<F32>(x, id) - lse;
      }
    }
  }
}

}  // namespace

cudaError_t launch_score(const ScoreArgs& a, bool f32, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.n, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      f32 ? cudaLaunchKernelEx(&cfg, k_score<true>, a) : cudaLaunchKernelEx(&cfg, k_score<false>, a);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace ds
