// k_quantize.cu -- rows to 8-bit integers with one scale each, after an optional
// RMS norm.
//
// y = x, or x * f * gain with f = rsqrt(mean(x^2) + eps); scale = max|y| / 127 and
// q = rint(y * (127 / max|y|)). A CTA has a row, a thread its chunks of 8, and
// a row of up to 8192 stays in registers between the three walks (sum of squares,
// max|y|, q); a longer one is read again from L1 and L2. Written as int8 rows, or
// as the fp16 tiles that the product of 8-bit integers reads (launch_linear_i8),
// which saves that call its own pass over them.
//
// Bound by latency at decoding sizes, a load, two block reductions and a store:
// 1.8 us for a row of 1024, 1.9 us for 24 rows of 2048, 2.1 us for 256 (bf16, with a
// gain). Wide batches: 8192 rows of 4096 take 35 us, 2.9 TB/s. 24 instructions an
// input fill 61% of the issue slots, and a CTA has none of the next row's loads in
// flight across a row's two reductions, which the profile shows as the longest
// stall. A thread keeps 1, 2 or 4 chunks by K: with 4 throughout, 8192 x 4096 took
// 90 us for the registers it held.
#include <cuda_fp16.h>

#include <type_traits>

#include "ds_device.cuh"
#include "ds_launch.h"

namespace ds {

namespace {

constexpr int kQrNT = 256;

__device__ __forceinline__ float qr_get(const uint16_t* p, long long i) {
  return __uint_as_float((uint32_t)__ldg(p + i) << 16);
}
__device__ __forceinline__ float qr_get(const float* p, long long i) { return __ldg(p + i); }

// 8 elements from chunk c on, zero past K.
__device__ __forceinline__ void qr_chunk(const uint16_t* row, int c, int K, bool wide, float (&f)[8]) {
  if (wide && c < K / 8) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(row) + c), f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 8 * c + i < K ? qr_get(row, 8 * c + i) : 0.f;
  }
}
__device__ __forceinline__ void qr_chunk(const float* row, int c, int K, bool wide, float (&f)[8]) {
  if (wide && c < K / 8) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(row) + 2 * c);
    const float4 b = __ldg(reinterpret_cast<const float4*>(row) + 2 * c + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 8 * c + i < K ? qr_get(row, 8 * c + i) : 0.f;
  }
}

}  // namespace

// TILES: rows of fp16 tiles, grid rows up to the last tile's end (zero past n, zero past K).
// HELD: chunks of a row that a thread keeps.
template <typename T, bool TILES, int HELD>
__global__ void __launch_bounds__(kQrNT, HELD == 4 ? 3 : HELD == 2 ? 4 : 5) k_quantize_rows(const void* x, int n, int K, long long ld, const float* gain,
                                                         float eps, int8_t* q, float* scale, I8Tiles tiles) {
  pdl_wait();
  pdl_release();
  __shared__ float red[2][kQrNT / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int parts = (int)((K + 7LL) / 8);  // chunks of 8 inputs: counted, as 8 c passes 32 bits behind a row of 2^31 - 1
  const int chunks = TILES ? tiles.kb * 8 : parts;  // a tile's row goes on to its last block's end
  const long long rows = TILES ? (long long)tiles.rows * tiles.tiles : n;
  for (long long i = blockIdx.x; i < rows; i += gridDim.x) {
    const T* row = static_cast<const T*>(x) + i * ld;
    const bool live = i < n;
    const bool wide = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
    const bool wide_gain = (reinterpret_cast<uintptr_t>(gain) & 15) == 0;
    float held[HELD][8];
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      const int c = tid + h * kQrNT;
      if (live && c < parts) {
        qr_chunk(row, c, K, wide, held[h]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) held[h][e] = 0.f;
      }
    }
    float f = 1.f, pre = 1.f;  // pre: a power of two that x is taken times, in `held` already
    auto rest = [&](int c, float (&v)[8]) {
      qr_chunk(row, c, K, wide, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= pre;
    };
    auto squares = [&] {
      float s = 0.f;
#pragma unroll
      for (int h = 0; h < HELD; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = __fmaf_rn(held[h][e], held[h][e], s);
      if (live)
        for (int c = tid + HELD * kQrNT; c < parts; c += kQrNT) {
          float v[8];
          rest(c, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) s = __fmaf_rn(v[e], v[e], s);
        }
      s = warp_sum(s);
      if (lane == 0) red[0][wid] = s;
      __syncthreads();
      s = 0.f;
#pragma unroll
      for (int w = 0; w < kQrNT / 32; ++w) s += red[0][w];
      return s;
    };
    if (gain) {
      const float v = squares() / (float)K + eps;
      f = rsqrtf(v);
      // Squares lose bits below 2^-126, which matters where their mean is that small,
      // and overflow from 1.8e19 on: the row is then taken times a power of two that
      // brings the larger of max|x| and sqrt(eps) to between 1 and 4.
      if (!(v >= 1e-37f && v < kInf)) {
        uint32_t top = 0;
#pragma unroll
        for (int h = 0; h < HELD; ++h)
#pragma unroll
          for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(held[h][e]) & 0x7fffffffu);
        if (live)
          for (int c = tid + HELD * kQrNT; c < parts; c += kQrNT) {
            float w[8];
            rest(c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(w[e]) & 0x7fffffffu);
          }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) red[1][wid] = __uint_as_float(top);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kQrNT / 32; ++w) top = max(top, __float_as_uint(red[1][w]));
        const float most = fmaxf(__uint_as_float(top), sqrtf(eps));
        if (top >= 0x7f800000u) {
          f = 1.f;  // a NaN or an infinity, which y has then too
        } else if (most == 0.f) {
          f = 0.f;  // zeros, without eps
        } else {
          pre = __uint_as_float((uint32_t)max(1, 254 - max(1, (int)(__float_as_uint(most) >> 23))) << 23);
#pragma unroll
          for (int h = 0; h < HELD; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) held[h][e] *= pre;
          f = rsqrtf(squares() / (float)K + eps * pre * pre);
        }
      }
    }
    auto normed = [&](int c, float (&v)[8]) {
      if (gain) {
        float w[8];
        qr_chunk(gain, c, K, wide_gain, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * f * w[e];
      }
    };
    // max |y| as bits: of numbers without sign they are in the numbers' order, infinities and NaN last
    uint32_t top = 0;
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      const int c = tid + h * kQrNT;
      if (c < parts) normed(c, held[h]);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(held[h][e]) & 0x7fffffffu);
    }
    if (live)
      for (int c = tid + HELD * kQrNT; c < parts; c += kQrNT) {
        float v[8];
        rest(c, v);
        normed(c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
      }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) red[1][wid] = __uint_as_float(top);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQrNT / 32; ++w) top = max(top, __float_as_uint(red[1][w]));
    const float amax = __uint_as_float(top);
    const bool bad = top >= 0x7f800000u;
    // 127 / max|y| is beyond fp32 below 3.7e-37: such a row is taken 2^64 times as large, exactly
    const bool small = amax < 4e-37f;
    const float lift = small ? 18446744073709551616.f : 1.f;
    const float inv = (bad || top == 0u) ? 0.f : 127.f / (amax * lift);
    if (small) {
#pragma unroll
      for (int h = 0; h < HELD; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e) held[h][e] *= lift;
    }
    auto put = [&](int c, const float (&v)[8]) {
      // |y inv| <= 127 (1 + 2^-23): added to 1.5 2^23 it is rounded to the nearest integer, which the low
      // bits then hold
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = bad ? 12582912.f : __fadd_rn(__fmul_rn(v[e], inv), 12582912.f);
      if (TILES) {
        const int r = (int)(i % tiles.rows);
        const long long block = (i / tiles.rows) * tiles.kb + (c >> 3);
        __half2 h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = __floats2half2_rn(w[2 * e] - 12582912.f, w[2 * e + 1] - 12582912.f);
        reinterpret_cast<uint4*>(tiles.out)[(block * tiles.rows + r) * 8 + ((c & 7) ^ (r & 7))] =
            *reinterpret_cast<const uint4*>(h);
      } else if ((K & 7) == 0 && (reinterpret_cast<uintptr_t>(q) & 7) == 0) {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo |= (__float_as_uint(w[e]) & 0xffu) << (8 * e);
          hi |= (__float_as_uint(w[4 + e]) & 0xffu) << (8 * e);
        }
        *reinterpret_cast<uint2*>(q + i * K + 8 * c) = make_uint2(lo, hi);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (8 * c + e < K) q[i * K + 8 * c + e] = (int8_t)(__float_as_uint(w[e]) & 0xffu);
      }
    };
#pragma unroll
    for (int h = 0; h < HELD; ++h)
      if (tid + h * kQrNT < chunks) put(tid + h * kQrNT, held[h]);
    for (int c = tid + HELD * kQrNT; c < chunks; c += kQrNT) {
      float v[8] = {};
      if (live && c < parts) {
        rest(c, v);
        normed(c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= lift;
      }
      put(c, v);
    }
    if (tid == 0 && live) scale[i] = bad ? __int_as_float(0x7fffffff) : amax / 127.f;
    __syncthreads();  // red is free
  }
}

cudaError_t launch_quantize_rows(const void* x, bool f32, int n, int K, int64_t ld, const float* gain, float eps,
                                 int8_t* q, float* scale, const I8Tiles* tiles, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorUnknown;
  const long long rows = tiles ? (long long)tiles->rows * tiles->tiles : n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows < sms * 8LL ? rows : sms * 8LL));
  cfg.blockDim = dim3(kQrNT);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto pick = [&](auto held) {
    constexpr int H = decltype(held)::value;
    return tiles ? (f32 ? k_quantize_rows<float, true, H> : k_quantize_rows<uint16_t, true, H>)
                 : (f32 ? k_quantize_rows<float, false, H> : k_quantize_rows<uint16_t, false, H>);
  };
  auto kern = K <= 8 * kQrNT ? pick(std::integral_constant<int, 1>{})
                             : K <= 16 * kQrNT ? pick(std::integral_constant<int, 2>{}) : pick(std::integral_constant<int, 4>{});
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, x, n, K, (long long)ld, gain, eps, q, scale,
                                           tiles ? *tiles : I8Tiles{nullptr, 0, 0, 0});
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace ds
