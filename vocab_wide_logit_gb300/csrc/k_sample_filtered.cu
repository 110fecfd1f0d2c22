// k_sample_filtered.cu -- temperature, top-k, top-p and min-p sampling of rows
// of logits from one given uniform number per row.
//
// The mathematics. With m the row's maximum and r = 1 / tau, a logit's weight is
// the integer w = rint(2^31 exp((x - m) r)), the exponential in fp32. Integers,
// so that every sum is exact: the mass of a set does not depend on how the row
// was split or in which order it was added, and a draw that lands on a boundary
// is the same draw on every batch, split and device. In the order (x
// descending, id ascending) each filter keeps a prefix:
//   top-k   the first k                                   T  = its mass
//   top-p   the elements with less than top_p T before them, of mass Tp
//   min-p   the elements with w >= min_p 2^31, of mass M
// so the kept set is the prefix of mass T' = min(Tp, M), and the token is the
// first element whose running mass passes floor(u T'). All three are one
// question, "which element is the first whose running count (or mass) passes
// t", asked of the whole row.
#include <climits>

#include "ds_device.cuh"
#include "ds_launch.h"

namespace ds {

namespace {

using u64 = unsigned long long;

constexpr int kSfNT = 512;
constexpr float kSfOne = 2147483648.f;  // 2^31, the weight of the row's maximum

// A logit's value, and its order key: larger logit, larger key, -0 folded onto
// +0. bf16 keys are the upper half of the fp32 ones.
template <typename T>
struct Logit;
template <>
struct Logit<uint16_t> {
  static __device__ __forceinline__ float get(const uint16_t* p, long long i) {
    return __uint_as_float((uint32_t)__ldg(p + i) << 16);
  }
  static __device__ __forceinline__ uint32_t key(float x) { return order_key(x == 0.f ? 0.f : x) >> 16; }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float(((k & 0x8000u) ? k ^ 0x8000u : ~k) << 16);
  }
};
template <>
struct Logit<float> {
  static __device__ __forceinline__ float get(const float* p, long long i) { return __ldg(p + i); }
  static __device__ __forceinline__ uint32_t key(float x) { return order_key(x == 0.f ? 0.f : x); }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
  }
};

// The expression is spelt with rounding intrinsics so that no contraction
// changes a weight: it is part of the result.
__device__ __forceinline__ uint32_t sf_weight(float x, float m, float r) {
  return __float2uint_rn(__fmul_rn(expf(__fmul_rn(__fsub_rn(x, m), r)), kSfOne));
}

// Where a running measure passes its target.
struct Cut {
  uint32_t key;
  u64 before;  // measure of the elements above `key`
  u64 each;    // measure of one element at `key`
};

template <int NT>
__device__ __forceinline__ u64 block_sum(u64 v, u64* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // red is free
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 s = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) s += red[i];
  return s;
}

// What is summed: 1 for each element (its rank), or its weight.
enum Measure { kCount, kMass };

// Measure of the row's elements with key >= lo.
template <typename T, int NT>
__device__ u64 row_measure(const T* row, int V, Measure what, uint32_t lo, float m, float r, u64* red) {
  u64 s = 0;
  for (int i = threadIdx.x; i < V; i += NT) {
    const float x = Logit<T>::get(row, i);
    if (Logit<T>::key(x) >= lo) s += (what == kCount) ? 1ull : (u64)sf_weight(x, m, r);
  }
  return block_sum<NT>(s, red);
}

// The first element whose running measure passes t (t < the whole row's
// measure), by bisection on its key: the largest key whose inclusive measure is
// above t.
template <typename T, int NT>
__device__ Cut row_select(const T* row, int V, Measure what, u64 t, float m, float r, u64* red) {
  uint32_t lo = Logit<T>::key(-kInf), hi = Logit<T>::key(m);  // measure(lo) > t; the answer lies in [lo, hi]
  u64 above = 0;                                              // measure of the keys above hi
  while (lo < hi) {
    const uint32_t mid = hi - (hi - lo) / 2;  // in (lo, hi]
    const u64 s = row_measure<T, NT>(row, V, what, mid, m, r, red);
    if (s > t) {
      lo = mid;
    } else {
      above = s;
      hi = mid - 1;
    }
  }
  Cut c;
  c.key = lo;
  c.before = above;
  c.each = what == kCount ? 1ull : (u64)sf_weight(Logit<T>::value(lo), m, r);
  return c;
}

// Id of the j-th (from 0) element with the given key, in id order.
template <typename T, int NT>
__device__ int row_nth(const T* row, int V, uint32_t key, u64 j, u64* red, int* slot) {
  const int per = (V + NT - 1) / NT;
  const int b = min(V, (int)threadIdx.x * per), e = min(V, b + per);
  int c = 0;
  for (int i = b; i < e; ++i) c += Logit<T>::key(Logit<T>::get(row, i)) == key;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int in_warp = warp_excl_scan(c, lane);
  __syncthreads();
  if (lane == 31) red[wid] = (u64)(in_warp + c);
  if (threadIdx.x == 0) *slot = 0;
  __syncthreads();
  u64 before = (u64)in_warp;
  for (int w = 0; w < wid; ++w) before += red[w];
  if (j >= before && j < before + (u64)c) {
    u64 left = j - before;
    for (int i = b; i < e; ++i)
      if (Logit<T>::key(Logit<T>::get(row, i)) == key && left-- == 0) {
        *slot = i;
        break;
      }
  }
  __syncthreads();
  return *slot;
}

// Mass of the prefix that ends with the first element whose running measure passes t.
__device__ __forceinline__ u64 cut_mass_through(const Cut& c, u64 t) {
  const u64 j = (t - c.before) / c.each;
  return c.before + (j + 1) * c.each;
}

}  // namespace

// One CTA per row; every question by bisection over the row, re-read from L2.
template <typename T>
__global__ void __launch_bounds__(kSfNT) k_sample_filtered_rows(FilteredArgs a) {
  pdl_wait();
  pdl_release();
  __shared__ u64 red[kSfNT / 32];
  __shared__ float fred[kSfNT / 32];
  __shared__ int slot;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  for (long long n = blockIdx.x; n < a.n; n += gridDim.x) {
    const T* row = static_cast<const T*>(a.x) + n * a.ld;
    const int V = a.V;
    float m = -kInf;
    for (int i = tid; i < V; i += kSfNT) m = fmaxf(m, Logit<T>::get(row, i));
    m = warp_max(m);
    __syncthreads();
    if (lane == 0) fred[wid] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSfNT / 32; ++i) m = fmaxf(m, fred[i]);
    // The sum is NaN when the row holds a NaN or +inf (inf - inf), or nothing but -inf.
    float s = 0.f;
    for (int i = tid; i < V; i += kSfNT) s += expf(Logit<T>::get(row, i) - m);
    s = warp_sum(s);
    __syncthreads();
    if (lane == 0) fred[wid] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSfNT / 32; ++i) s += fred[i];
    const float lse = m + logf(s);

    const float tau = a.temperature[n], u = a.u[n];
    const float p = a.top_p ? a.top_p[n] : 1.f, mp = a.min_p ? a.min_p[n] : 0.f;
    const int k = a.top_k ? a.top_k[n] : 0;
    const bool bad_param = !(tau >= 0.f && tau < kInf) || !(u >= 0.f && u < 1.f) || !(p > 0.f && p <= 1.f) ||
                           !(mp >= 0.f && mp <= 1.f);
    int token = -1;
    float lp = __int_as_float(0x7fffffff);
    if (bad_param) {
      if (tid == 0) report(a.d_status, DS_DEV_ERR_PARAM);
    } else if (!(s < kInf)) {
      // all -inf: nothing to draw. Otherwise NaN or +inf somewhere; a row of NaN alone has m = -inf too.
      float nan = 0.f;
      for (int i = tid; i < V; i += kSfNT) {
        const float x = Logit<T>::get(row, i);
        if (x != x || x == kInf) nan = 1.f;
      }
      if (__syncthreads_or(nan != 0.f) && tid == 0) report(a.d_status, DS_DEV_ERR_LOGITS);
    } else if (tau == 0.f) {
      token = row_nth<T, kSfNT>(row, V, Logit<T>::key(m), 0, red, &slot);
      lp = m - lse;
    } else {
      const float r = fminf(__frcp_rn(tau), 3.402823466e38f);
      u64 total = row_measure<T, kSfNT>(row, V, kMass, 0u, m, r, red);
      if (k > 0 && k < V) {
        const Cut c = row_select<T, kSfNT>(row, V, kCount, (u64)k - 1, m, r, red);
        const u64 above = row_measure<T, kSfNT>(row, V, kMass, c.key + 1u, m, r, red);
        total = above + ((u64)k - c.before) * sf_weight(Logit<T>::value(c.key), m, r);
      }
      if (p < 1.f) {
        // kept while the mass before is below p * total: through the first whose running mass reaches it
        const u64 need = (u64)ceil((double)p * (double)total);
        if (need < total)
          total = cut_mass_through(row_select<T, kSfNT>(row, V, kMass, need - 1, m, r, red), need - 1);
      }
      if (mp > 0.f) {
        const double floor_w = (double)mp * 2147483648.0;
        u64 sum = 0;
        for (int i = tid; i < V; i += kSfNT) {
          const uint32_t w = sf_weight(Logit<T>::get(row, i), m, r);
          if ((double)w >= floor_w) sum += w;
        }
        sum = block_sum<kSfNT>(sum, red);
        total = sum < total ? sum : total;
      }
      const u64 t = (u64)floor((double)u * (double)total);
      const Cut c = row_select<T, kSfNT>(row, V, kMass, t, m, r, red);
      token = row_nth<T, kSfNT>(row, V, c.key, (t - c.before) / c.each, red, &slot);
      lp = Logit<T>::get(row, token) - lse;
    }
    if (tid == 0) {
      a.out_tokens[n] = token;
      a.out_logprobs[n] = lp;
    }
    __syncthreads();
  }
}

cudaError_t launch_sample_filtered(const FilteredArgs& a, bool f32, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorUnknown;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)min((long long)a.n, (long long)sms * 4));
  cfg.blockDim = dim3(kSfNT);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = f32 ? cudaLaunchKernelEx(&cfg, k_sample_filtered_rows<float>, a)
                            : cudaLaunchKernelEx(&cfg, k_sample_filtered_rows<uint16_t>, a);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace ds
