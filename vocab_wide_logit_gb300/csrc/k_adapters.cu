// k_adapters.cu -- low-rank adapters of many requests added to shared logits.
//
//   out_i = base_i + scale_a B_a (A_a y_i),  a = ids[i],
//   y = x, or x rsqrt(mean x^2 + eps) gain
// First t_i = scale_a A_a y_i, R numbers a row, one CTA per row; then a thread per
// logit.
#include "ds_device.cuh"
#include "ds_launch.h"

namespace ds {

namespace {

constexpr int kThreads = 256;

template <bool F32>
__device__ __forceinline__ float load(const void* p, long long i) {
  if constexpr (F32)
    return static_cast<const float*>(p)[i];
  else
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) k_adapters_down(const AdapterArgs g) {
  pdl_release();
  pdl_wait();
  __shared__ double part[kThreads / 32];
  const int row = blockIdx.x, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int a = g.ids[row];
  if (a < 0) return;
  if (a >= g.L) {
    if (threadIdx.x == 0) report(g.d_status, DS_DEV_ERR_PARAM);
    return;
  }
  const char* x = static_cast<const char*>(g.x) + row * g.ldx * (F32 ? 4 : 2);
  float rs = 1.f;
  int bad = 0;
  for (int k = threadIdx.x; k < g.K; k += kThreads) bad |= !(fabsf(load<F32>(x, k)) < kInf);
  if (__syncthreads_or(bad)) rs = __int_as_float(0x7fffffff);
  if (g.gain) {
    double ss = 0;
    for (int k = threadIdx.x; k < g.K; k += kThreads) ss += (double)load<F32>(x, k) * load<F32>(x, k);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) part[wid] = ss;
    __syncthreads();
    ss = 0;
    for (int i = 0; i < kThreads / 32; ++i) ss += part[i];
    rs *= ss == 0 ? 0.f : (float)(1.0 / sqrt(ss / g.K + g.eps));
  }
  float* t = static_cast<float*>(g.workspace) + (long long)row * g.R;
  for (int r = wid; r < g.R; r += kThreads / 32) {
    const uint16_t* w = g.a + ((long long)a * g.R + r) * g.K;
    float sum = 0.f;
    for (int k = lane; k < g.K; k += 32) sum = __fmaf_rn(load<false>(w, k), load<F32>(x, k) * rs * (g.gain ? g.gain[k] : 1.f), sum);
    sum = warp_sum(sum);
    if (lane == 0) t[r] = sum * g.scale[a];
  }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) k_adapters_up(const AdapterArgs g) {
  pdl_release();
  pdl_wait();
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= g.N) return;
  for (int row = blockIdx.y; row < g.n; row += gridDim.y) {
    const int a = g.ids[row];
    float v = load<F32>(g.base, row * g.ldb + j);
    if (a >= g.L) v = __int_as_float(0x7fffffff);
    if (a >= 0 && a < g.L) {
      const float* t = static_cast<const float*>(g.workspace) + (long long)row * g.R;
      const uint16_t* w = g.b + ((long long)a * g.N + j) * g.R;
      float sum = 0.f;
      for (int r = 0; r < g.R; ++r) sum = __fmaf_rn(load<false>(w, r), t[r], sum);
      v += sum;
    }
    if constexpr (F32) {
      static_cast<float*>(g.out)[row * g.ldo + j] = v;
    } else {
      uint32_t w;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(0.f), "f"(v));
      static_cast<uint16_t*>(g.out)[row * g.ldo + j] = (uint16_t)w;
    }
  }
}

}  // namespace

long long adapters_workspace(int n, int L, int R) { return (long long)n * R * 4; }

cudaError_t launch_add_adapters(const AdapterArgs& g, bool x_f32, bool f32, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)g.n, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e =
      x_f32 ? cudaLaunchKernelEx(&cfg, k_adapters_down<true>, g) : cudaLaunchKernelEx(&cfg, k_adapters_down<false>, g);
  if (e != cudaSuccess) return e;
  note_launch();
  cfg.gridDim = dim3((unsigned)((g.N + (kThreads - 1LL)) / kThreads), (unsigned)(g.n < 65535 ? g.n : 65535), 1);
  e = f32 ? cudaLaunchKernelEx(&cfg, k_adapters_up<true>, g) : cudaLaunchKernelEx(&cfg, k_adapters_up<false>, g);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace ds
