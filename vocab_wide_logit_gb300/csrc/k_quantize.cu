// k_quantize.cu -- rows to 8-bit integers with one scale each, after an optional
// RMS norm.
//
// y = x, or x * rsqrt(mean(x^2) + eps) * gain; scale = max|y| / 127 and
// q = rint(y * (127 / max|y|)). The norm's factor is one number per row, so the
// row is read for its sum of squares, for max|y| and for q.
#include "ds_device.cuh"
#include "ds_launch.h"

namespace ds {

namespace {

constexpr int kQrNT = 256;

__device__ __forceinline__ float qr_get(const uint16_t* p, long long i) {
  return __uint_as_float((uint32_t)__ldg(p + i) << 16);
}
__device__ __forceinline__ float qr_get(const float* p, long long i) { return __ldg(p + i); }

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kQrNT) k_quantize_rows(const void* x, int n, int K, long long ld, const float* gain,
                                                         float eps, int8_t* q, float* scale) {
  pdl_wait();
  pdl_release();
  __shared__ float red[kQrNT / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  for (long long i = blockIdx.x; i < n; i += gridDim.x) {
    const T* row = static_cast<const T*>(x) + i * ld;
    float f = 1.f;
    int bad = 0;
    if (gain) {
      float s = 0.f;
      for (int k = tid; k < K; k += kQrNT) {
        const float v = qr_get(row, k);
        s = __fmaf_rn(v, v, s);
      }
      s = warp_sum(s);
      __syncthreads();
      if (lane == 0) red[wid] = s;
      __syncthreads();
      s = 0.f;
#pragma unroll
      for (int w = 0; w < kQrNT / 32; ++w) s += red[w];
      f = rsqrtf(s / (float)K + eps);
      bad = !(s < kInf);  // a NaN, an infinity, or squares that overflow
    }
    float amax = 0.f;
    for (int k = tid; k < K; k += kQrNT) {
      float y = qr_get(row, k);
      if (gain) y = y * f * gain[k];
      bad |= !(fabsf(y) < kInf);
      amax = fmaxf(amax, fabsf(y));
    }
    amax = warp_max(amax);
    bad = __syncthreads_or(bad);
    if (lane == 0) red[wid] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQrNT / 32; ++w) amax = fmaxf(amax, red[w]);
    const float inv = (bad || amax == 0.f) ? 0.f : fminf(127.f / amax, 3.402823466e38f);
    for (int k = tid; k < K; k += kQrNT) {
      float y = qr_get(row, k);
      if (gain) y = y * f * gain[k];
      q[i * K + k] = bad ? (int8_t)0 : (int8_t)__float2int_rn(fminf(fmaxf(y * inv, -127.f), 127.f));
    }
    if (tid == 0) scale[i] = bad ? __int_as_float(0x7fffffff) : amax / 127.f;
    __syncthreads();
  }
}

cudaError_t launch_quantize_rows(const void* x, bool f32, int n, int K, int64_t ld, const float* gain, float eps,
                                 int8_t* q, float* scale, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorUnknown;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n < sms * 8 ? n : sms * 8));
  cfg.blockDim = dim3(kQrNT);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      f32 ? cudaLaunchKernelEx(&cfg, k_quantize_rows<float>, x, n, K, (long long)ld, gain, eps, q, scale)
          : cudaLaunchKernelEx(&cfg, k_quantize_rows<uint16_t>, x, n, K, (long long)ld, gain, eps, q, scale);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace ds
