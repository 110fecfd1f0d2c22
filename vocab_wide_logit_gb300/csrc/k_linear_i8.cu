// k_linear_i8.cu -- product of 8-bit integers scaled by row and channel:
// out[i][j] = (sum_k a[i][k] w[j][k]) * a_scale[i] * w_scale[j].
#include <cuda_bf16.h>

#include "ds_device.cuh"
#include "ds_launch.h"

namespace ds {

namespace {

constexpr int kLiRows = 8;  // rows of a per CTA

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

}  // namespace

// One thread per 16-byte chunk of a packed block.
__global__ void __launch_bounds__(256) k_pack_i8(const int8_t* w, int N, int K, long long ldw, uint8_t* packed) {
  pdl_wait();
  pdl_release();
  const int kb = (K + kPackK - 1) / kPackK;
  const long long chunks = (long long)((N + kPackRows - 1) / kPackRows) * kb * (kPackRows * kPackK / 16);
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < chunks; i += (long long)gridDim.x * 256) {
    const int c = (int)(i & 7), r = (int)((i >> 3) & (kPackRows - 1));
    const long long b = i >> 10;
    const long long row = b / kb * kPackRows + r;
    const int k0 = (int)(b % kb) * kPackK + ((c ^ (r & 7)) << 4);
    uint32_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t x = 0;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int k = k0 + 4 * j + t;
        const uint32_t byte = (row < N && k < K) ? (uint32_t)(uint8_t)w[row * ldw + k] ^ 0x80u : 0x80u;
        x |= byte << (8 * t);
      }
      v[j] = x;
    }
    reinterpret_cast<uint4*>(packed)[i] = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// One thread per channel, kLiRows rows of a: exact sums by four-way integer dot products.
template <typename OUT>
__global__ void __launch_bounds__(kPackRows) k_linear_i8(LinearArgs g) {
  pdl_wait();
  pdl_release();
  __shared__ int as[kLiRows][kPackK / 4];
  const int kb = (g.K + kPackK - 1) / kPackK;
  const int r = threadIdx.x;
  const long long j = (long long)blockIdx.x * kPackRows + r;
  for (int i0 = blockIdx.y * kLiRows; i0 < g.n; i0 += gridDim.y * kLiRows) {
    int acc[kLiRows] = {};
    for (int b = 0; b < kb; ++b) {
      __syncthreads();
      for (int e = r; e < kLiRows * kPackK; e += kPackRows) {
        const int i = i0 + e / kPackK, k = b * kPackK + e % kPackK;
        reinterpret_cast<int8_t*>(as)[e] = (i < g.n && k < g.K) ? g.a[(long long)i * g.lda + k] : (int8_t)0;
      }
      __syncthreads();
      const uint4* blk =
          reinterpret_cast<const uint4*>(g.packed + ((long long)blockIdx.x * kb + b) * (kPackRows * kPackK)) + r * 8;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 v = blk[c ^ (r & 7)];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < kLiRows; ++i) acc[i] = __dp4a((int)(w[q] ^ 0x80808080u), as[i][c * 4 + q], acc[i]);
      }
    }
    if (j < g.N) {
      const float sw = g.w_scale[j];
#pragma unroll
      for (int i = 0; i < kLiRows; ++i)
        if (i0 + i < g.n)
          store_out(static_cast<OUT*>(g.out) + (long long)(i0 + i) * g.ldo + j,
                    (float)acc[i] * g.a_scale[i0 + i] * sw);
    }
  }
}

long long linear_i8_workspace(int, int, int) { return 0; }

cudaError_t launch_pack_i8(const int8_t* w, int N, int K, int64_t ldw, uint8_t* packed, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorUnknown;
  const long long chunks = (long long)((N + kPackRows - 1) / kPackRows) * ((K + kPackK - 1) / kPackK) * 1024;
  const long long want = (chunks + 255) / 256;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(want < sms * 16LL ? want : sms * 16LL));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_pack_i8, w, N, K, (long long)ldw, packed);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_linear_i8(const LinearArgs& g, bool bf16_out, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  const int by = (g.n + kLiRows - 1) / kLiRows;
  cfg.gridDim = dim3((unsigned)((g.N + kPackRows - 1LL) / kPackRows), (unsigned)(by < 65535 ? by : 65535));
  cfg.blockDim = dim3(kPackRows);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = bf16_out ? cudaLaunchKernelEx(&cfg, k_linear_i8<__nv_bfloat16>, g)
                                 : cudaLaunchKernelEx(&cfg, k_linear_i8<float>, g);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace ds
