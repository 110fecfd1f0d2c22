// k_adapters.cu -- low-rank adapters of many requests added to shared logits.
//
//   out_i = base_i + scale_a B_a (A_a y_i),  a = ids[i],
//   y = x, or x rsqrt(mean x^2 + eps) gain
//
// Rows are gathered into tiles of up to 16 that have the same adapter, so that an
// adapter's weights are read once for 16 rows in whatever order the rows come.
//   k_adapters_plan  (more than 256 rows) one CTA counts the rows of each adapter and
//                    deals them out to tiles; up to 256 rows the next kernel's CTAs
//                    each find their own tile.
//   k_adapters_down  a CTA per tile and 32 ranks: t = scale A y by matrix instructions
//                    (16 rows x 8 ranks x 16 inputs), the inputs split over 16 warps.
//   k_adapters_up    a warp per tile and 256 bytes of each row's logits: t B^T by
//                    matrix instructions (16 rows x 8 channels x 16 ranks), then base
//                    and result in whole 16-byte chunks a row.
// The adapters' bf16 goes into the instructions as it is. The fp32 operand goes in as a
// sum of bf16 parts, each the rest that the parts before it left: three of them (2^-27
// of it is lost) for fp32 logits, two (2^-18) for bf16 logits, whose own rounding is
// 2^-9. Sums are fp32.
//
// What bounds it is HBM: base, result and the weights once. The weights' bytes go
// from memory to the registers that the instructions read, 8 or 16 bytes a lane, each
// lane taking the ranks that lie together there as "its" four of an instruction's 16
// (any order of the ranks is right that both operands share). Rows start at any
// element: a tile of channels starts for each row at that row's own 16-byte boundary,
// for which eight channels in front of the tile are computed twice.
#include <cuda_bf16.h>

#include "ds_device.cuh"
#include "ds_launch.h"

namespace ds {

namespace {

constexpr int kRows = 16;          // rows of a tile
constexpr int kSelfPlan = 256;     // rows up to which k_adapters_down plans for itself
constexpr int kDownThreads = 512;
constexpr int kDownWarps = kDownThreads / 32;
constexpr int kDownRanks = 32;     // ranks of a CTA
constexpr int kPlanThreads = 1024;
constexpr int kUpWarps = 8;
constexpr int kNone = -1, kBad = -2;  // a tile of rows without an adapter, of ids beyond the stack

// Rows of one adapter; count 0: no tile.
struct Tile {
  int32_t adapter, count;
  int32_t rows[kRows];
  int32_t pad[14];
};
static_assert(sizeof(Tile) == 128, "tiles keep what follows them aligned");

// Ranks filled up with zeros: 16, or a power of two from 32.
__host__ __device__ constexpr int padded(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128; }
// Tiles that n rows can make: one for every 16 rows and a partial one for each kind.
__host__ __device__ constexpr long long tiles_of(int n, int L) {
  const long long kinds = n < L + 2 ? n : L + 2, most = n / kRows + kinds;
  return most < n ? most : n;
}
// Bytes of t of a tile, in the order of the instructions' first operand:
// [step of 16 ranks][part][lane][8 bf16].
__host__ __device__ constexpr long long t_bytes(int R) { return (long long)padded(R) / 16 * 3 * 32 * 16; }

__device__ __forceinline__ int kind_of(int id, int L) { return id < 0 ? kNone : id < L ? id : kBad; }

// d (16 x 8, fp32) += a (16 x 16, bf16) b (16 x 8, bf16).
__device__ __forceinline__ void mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool F32>
__device__ __forceinline__ float load(const void* p, long long i) {
  if constexpr (F32)
    return __ldg(static_cast<const float*>(p) + i);
  else
    return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << 16);
}

// Eight inputs from k on, zeros from K on. VEC: at a 16-byte boundary, K a multiple of 8.
template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* row, int k, int K, float (&f)[8]) {
  if constexpr (VEC) {
    if (k >= K) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.f;
    } else if constexpr (F32) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(row) + k));
      const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(row) + k) + 1);
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
      unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + k)), f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = k + i < K ? load<F32>(row, k + i) : 0.f;
  }
}
// `count` (4 or 8) weights as they are, from i on, zeros from `end` on.
template <int COUNT, bool VEC>
__device__ __forceinline__ void load_weights(const uint16_t* row, int i, int end, uint32_t (&w)[COUNT / 2]) {
  if constexpr (VEC) {
    if (i >= end) {
#pragma unroll
      for (int j = 0; j < COUNT / 2; ++j) w[j] = 0;
    } else if constexpr (COUNT == 8) {
      const uint4 v = ld_stream16(row + i);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + i));
      w[0] = v.x, w[1] = v.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < COUNT / 2; ++j) {
      const uint32_t lo = i + 2 * j < end ? __ldg(row + i + 2 * j) : 0u;
      const uint32_t hi = i + 2 * j + 1 < end ? __ldg(row + i + 2 * j + 1) : 0u;
      w[j] = lo | (hi << 16);
    }
  }
}

// ---------------------------------------------------------------- tiles
// More than 256 rows: counted, then dealt out. Which rows share a tile may differ from
// run to run; a row's result does not depend on it.
__global__ void __launch_bounds__(kPlanThreads) k_adapters_plan(const AdapterArgs g, Tile* tiles, int most) {
  extern __shared__ uint32_t counts[];  // rows of each kind (adapters, none, bad), then its first tile
  __shared__ int warp_sums[kPlanThreads / 32];
  pdl_release();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, kinds = g.L + 2;
  for (int i = tid; i < kinds; i += kPlanThreads) counts[i] = 0;
  __syncthreads();
  for (long long i = tid; i < g.n; i += kPlanThreads) {
    const int a = kind_of(g.ids[i], g.L);
    if (a == kBad) report(g.d_status, DS_DEV_ERR_PARAM);
    atomicAdd(&counts[a >= 0 ? a : g.L - 1 - a], 1u);
  }
  __syncthreads();
  // first tiles: a running sum over each thread's share of the kinds
  const int per = (kinds + kPlanThreads - 1) / kPlanThreads, lo = tid * per, hi = min(lo + per, kinds);
  int mine = 0;
  for (int i = lo; i < hi; ++i) mine += (int)((counts[i] + kRows - 1) / kRows);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[wid] = incl;
  __syncthreads();
  int at = incl - mine;
  for (int i = 0; i < wid; ++i) at += warp_sums[i];
  int all = 0;
  for (int i = 0; i < kPlanThreads / 32; ++i) all += warp_sums[i];
  for (int i = lo; i < hi; ++i) {
    int c = (int)counts[i];
    counts[i] = (uint32_t)at * kRows;  // where the kind's next row goes
    for (; c > 0; c -= kRows, ++at) {
      tiles[at].adapter = i < g.L ? i : g.L - 1 - i;
      tiles[at].count = min(c, kRows);
    }
  }
  __syncthreads();
  for (long long i = tid; i < g.n; i += kPlanThreads) {
    const int a = kind_of(g.ids[i], g.L);
    const uint32_t slot = atomicAdd(&counts[a >= 0 ? a : g.L - 1 - a], 1u);
    tiles[slot / kRows].rows[slot % kRows] = (int)i;
  }
  for (int i = all + tid; i < most; i += kPlanThreads) tiles[i].count = 0;
}

// Up to 256 rows: tile number `want` of those that the rows' order makes, found by a CTA.
struct SelfPlan {
  int kinds[kSelfPlan];
  int leaders[kDownWarps];
  int at;  // the row that opens the tile
  int count;
};
__device__ __forceinline__ void self_plan(const AdapterArgs& g, int want, SelfPlan& s, Tile& tile) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid < kSelfPlan) s.kinds[tid] = tid < g.n ? kind_of(g.ids[tid], g.L) : kBad - 1;
  if (tid == 0) s.at = -1;
  __syncthreads();
  const int kind = tid < g.n ? s.kinds[tid] : kBad - 1;
  int before = 0;  // rows of this kind in front of this one
  if (wid * 32 < g.n) {
    const int4* four = reinterpret_cast<const int4*>(s.kinds);
    for (int j = 0; j < wid * 8; ++j) {
      const int4 v = four[j];
      before += (v.x == kind) + (v.y == kind) + (v.z == kind) + (v.w == kind);
    }
    before += __popc(__match_any_sync(0xffffffffu, kind) & ((1u << lane) - 1));
  }
  const bool leads = tid < g.n && before % kRows == 0;
  const unsigned who = __ballot_sync(0xffffffffu, leads);
  if (lane == 0) s.leaders[wid] = __popc(who);
  __syncthreads();
  int number = __popc(who & ((1u << lane) - 1));
  for (int i = 0; i < wid; ++i) number += s.leaders[i];
  if (leads && number == want) {
    s.at = tid;
    s.count = before;
    tile.adapter = kind;
  }
  __syncthreads();
  const int at = s.at;
  const bool in = at >= 0 && kind == s.kinds[max(at, 0)] && tid < g.n && before / kRows == s.count / kRows;
  if (in) tile.rows[before % kRows] = tid;
  const int c = __syncthreads_count(in);
  if (tid == 0) tile.count = c;
  if (tid < kRows && tid >= c) tile.rows[tid] = 0;
  __syncthreads();
}

// ---------------------------------------------------------------- t = scale A y
struct Down {
  Tile tile;
  SelfPlan plan;
  float t[kDownWarps][kRows][kDownRanks + 1];
  float squares[kDownWarps][kRows];
  float odd[kDownWarps][kRows];  // 0, or NaN where a row's input is not finite
  double wide[kDownWarps];
  float factor[kRows];
};

// PARTS: bf16 parts of an input. VEC: 16-byte loads.
template <bool XF32, int PARTS, bool VEC>
__global__ void __launch_bounds__(kDownThreads) k_adapters_down(const AdapterArgs g, Tile* tiles, uint8_t* t_out, int parts_out) {
  extern __shared__ __align__(16) unsigned char raw[];
  Down& sh = *reinterpret_cast<Down*>(raw);
  pdl_release();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, gq = lane >> 2, q = lane & 3;
  if (g.n <= kSelfPlan) {
    self_plan(g, blockIdx.x, sh.plan, sh.tile);
    if (blockIdx.y == 0 && tid < 2 + kRows)
      reinterpret_cast<int32_t*>(&tiles[blockIdx.x])[tid] = reinterpret_cast<const int32_t*>(&sh.tile)[tid];
  } else {
    if (tid < 2 + kRows)
      reinterpret_cast<int32_t*>(&sh.tile)[tid] = reinterpret_cast<const int32_t*>(&tiles[blockIdx.x])[tid];
    __syncthreads();
  }
  const int count = sh.tile.count, a = sh.tile.adapter;
  if (count <= 0) return;
  if (a < 0) {
    if (a == kBad && g.n <= kSelfPlan && blockIdx.y == 0 && tid == 0) report(g.d_status, DS_DEV_ERR_PARAM);
    return;
  }
  constexpr int kSize = XF32 ? 4 : 2;
  const char* x = static_cast<const char*>(g.x);
  const bool has0 = gq < count, has1 = gq + 8 < count;
  const char* x0 = x + (has0 ? sh.tile.rows[gq] : 0) * g.ldx * kSize;
  const char* x1 = x + (has1 ? sh.tile.rows[gq + 8] : 0) * g.ldx * kSize;
  const int rank0 = blockIdx.y * kDownRanks;
  const int groups = min(kDownRanks, padded(g.R) - rank0) / 8;  // of 8 ranks: 2 or 4
  const uint16_t* w = g.a + ((long long)a * g.R + rank0) * g.K;

  float d[4][4] = {};
  float ss0 = 0.f, ss1 = 0.f, odd0 = 0.f, odd1 = 0.f;
  // 32 inputs a step: lane q of a row's four takes 8 that lie together, four of them
  // for each of two instructions
#pragma unroll 2
  for (int k0 = wid * 32; k0 < g.K; k0 += kDownWarps * 32) {
    const int k = k0 + 8 * q;
    float f0[8], f1[8];
    load8<XF32, VEC>(x0, k, has0 ? g.K : 0, f0);
    load8<XF32, VEC>(x1, k, has1 ? g.K : 0, f1);
    uint32_t b[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 8 * j + gq;
      const bool there = j < groups && rank0 + r < g.R;
      load_weights<8, VEC>(w + (there ? (long long)r * g.K : 0), k, there ? g.K : 0, b[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      odd0 = __fmaf_rn(f0[i], 0.f, odd0);
      odd1 = __fmaf_rn(f1[i], 0.f, odd1);
    }
    if (g.gain) {
      float n8[8];
      load8<true, VEC>(g.gain, k, g.K, n8);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss0 = __fmaf_rn(f0[i], f0[i], ss0);
        ss1 = __fmaf_rn(f1[i], f1[i], ss1);
        f0[i] *= n8[i];
        f1[i] *= n8[i];
      }
    }
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      uint32_t h0[4], h1[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h0[i] = pack_bf(f0[2 * i], f0[2 * i + 1]);
        h1[i] = pack_bf(f1[2 * i], f1[2 * i + 1]);
        if (p + 1 < PARTS) {
          f0[2 * i] -= bf_lo(h0[i]);
          f0[2 * i + 1] -= bf_hi(h0[i]);
          f1[2 * i] -= bf_lo(h1[i]);
          f1[2 * i + 1] -= bf_hi(h1[i]);
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint4 av = make_uint4(h0[2 * s], h1[2 * s], h0[2 * s + 1], h1[2 * s + 1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma(d[j], av, b[j][2 * s], b[j][2 * s + 1]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sh.t[wid][gq][8 * j + 2 * q] = d[j][0];
    sh.t[wid][gq][8 * j + 2 * q + 1] = d[j][1];
    sh.t[wid][gq + 8][8 * j + 2 * q] = d[j][2];
    sh.t[wid][gq + 8][8 * j + 2 * q + 1] = d[j][3];
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    ss0 += __shfl_xor_sync(0xffffffffu, ss0, o);
    ss1 += __shfl_xor_sync(0xffffffffu, ss1, o);
    odd0 += __shfl_xor_sync(0xffffffffu, odd0, o);
    odd1 += __shfl_xor_sync(0xffffffffu, odd1, o);
  }
  if (q == 0) {
    sh.squares[wid][gq] = ss0;
    sh.squares[wid][gq + 8] = ss1;
    sh.odd[wid][gq] = odd0;
    sh.odd[wid][gq + 8] = odd1;
  }
  __syncthreads();
  // each row's factor: scale, the norm's root, NaN for a row that is not finite
  if (tid < kRows) {
    float ss = 0.f, odd = 0.f;
    for (int i = 0; i < kDownWarps; ++i) {
      ss += sh.squares[i][tid];
      odd += sh.odd[i][tid];
    }
    float f = 1.f;
    if (g.gain) f = ss > 1e-25f && ss < 1e37f ? rsqrtf(ss / (float)g.K + g.eps) : -1.f;  // -1: below
    sh.factor[tid] = odd != 0.f || odd != odd ? __int_as_float(0x7fffffff) : f;
  }
  __syncthreads();
  if (g.gain) {
    // squares that leave fp32's range, rows of zeros: the sum in 64 bits
    for (int r = 0; r < count; ++r) {
      if (sh.factor[r] != -1.f) continue;
      const char* row = x + sh.tile.rows[r] * g.ldx * kSize;
      double ss = 0;
      for (int k = tid; k < g.K; k += kDownThreads) {
        const double v = load<XF32>(row, k);
        ss += v * v;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (lane == 0) sh.wide[wid] = ss;
      __syncthreads();
      ss = 0;
      for (int i = 0; i < kDownWarps; ++i) ss += sh.wide[i];
      __syncthreads();
      if (tid == 0) sh.factor[r] = ss == 0 ? 0.f : (float)(1.0 / sqrt(ss / g.K + g.eps));
    }
    __syncthreads();
  }
  // a thread per row and rank
  const int row = tid / kDownRanks, r = tid % kDownRanks, rank = rank0 + r;
  if (r < groups * 8) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kDownWarps; ++i) t += sh.t[i][row][r];
    t = row < count ? t * (sh.factor[row] * g.scale[a]) : 0.f;
    // which step, lane and place holds this rank
    const int rp = padded(g.R);
    const int step = rp == 16 ? 0 : 2 * (rank / 32) + (rank >> 2) % 2, qt = rp == 16 ? rank / 4 : (rank % 32) / 8, e = rank % 4;
    uint16_t* out = reinterpret_cast<uint16_t*>(t_out + blockIdx.x * t_bytes(g.R)) + ((step * 3 * 32) + (row % 8) * 4 + qt) * 8 +
                    (e >> 1) * 4 + (row / 8) * 2 + (e & 1);
    for (int p = 0; p < parts_out; ++p) {
      const uint32_t h = pack_bf(t, 0.f) & 0xffffu;
      out[p * 32 * 8] = (uint16_t)h;
      t -= __uint_as_float(h << 16);
    }
  }
}

// ---------------------------------------------------------------- base + t B^T
// Logits that a warp makes of each row, 16 chunks of 16 bytes, and the pitch of its
// results in shared memory (rows 8 banks apart).
template <bool F32>
struct Up {
  static constexpr int E = F32 ? 4 : 8;
  static constexpr int kChannels = 16 * E;
  static constexpr int kPitch = kChannels + 8;
  static constexpr int kSmem = kUpWarps * kRows * kPitch * 4;
};

// Not through the read-only path: base may be the result.
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

// RP: padded ranks. VEC: weights in one load a lane and step. NEAR: base and result
// rows lie the same way to 16 bytes. SHIFT: some row starts between two chunks.
template <bool F32, int RP, bool VEC, bool NEAR, bool SHIFT>
__global__ void __launch_bounds__(kUpWarps * 32, RP <= 64 ? 2 : 1)
    k_adapters_up(const AdapterArgs g, const Tile* tiles, const uint8_t* t_in) {
  using U = Up<F32>;
  constexpr int E = U::E, kSize = F32 ? 4 : 2, PARTS = F32 ? 3 : 2, STEPS = RP / 16;
  constexpr int kLoad = RP == 16 ? 4 : 8;  // weights of a lane and load: one instruction's, or two's
  extern __shared__ __align__(16) float results[];
  pdl_release();
  pdl_wait();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, gq = lane >> 2, q = lane & 3;
  const Tile& tile = tiles[blockIdx.y];
  const int count = tile.count, a = tile.adapter;
  const long long block = (long long)blockIdx.x * kUpWarps + wid;  // of 16 chunks
  const long long c0 = block * U::kChannels;
  if (count <= 0 || c0 >= (long long)g.N + (SHIFT ? E - 1 : 0)) return;
  if (a == kNone && g.out == g.base) return;
  float* mine = results + wid * kRows * U::kPitch;
  const int my_row = lane < count ? tile.rows[lane] : 0;
  char* out = static_cast<char*>(g.out);
  const char* base = static_cast<const char*>(g.base);
  // how many logits of a row's first chunk are before it
  auto shift_of = [&](long long row) {
    return SHIFT ? (int)(reinterpret_cast<uintptr_t>(out + row * g.ldo * kSize) & 15) / kSize : 0;
  };

  // lane l, turn i: chunk l % 16 of the tile's row 2 i + l / 16
  uint4 v[8];
  if (a != kBad) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (2 * i >= count) break;
      const int r = 2 * i + (lane >> 4);
      const long long row = __shfl_sync(0xffffffffu, my_row, r);
      const long long id = c0 + (lane & 15) * E - shift_of(row);
      if (r >= count || id >= g.N) continue;
      const char* p = base + (row * g.ldb + id) * kSize;
      if constexpr (NEAR) {
        v[i] = ld16(p);  // its edges may be other rows' bytes, of the same 16
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (id + e < 0 || id + e >= g.N) continue;
          if constexpr (F32)
            w[e] = reinterpret_cast<const volatile uint32_t*>(p)[e];
          else
            w[e >> 1] |= (uint32_t) reinterpret_cast<const volatile uint16_t*>(p)[e] << (16 * (e & 1));
        }
        v[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }

  if (a >= 0) {
    const uint4* t4 = reinterpret_cast<const uint4*>(t_in + blockIdx.y * t_bytes(g.R)) + lane;
    uint4 t[RP <= 64 ? STEPS : 1][PARTS];
    if constexpr (RP <= 64) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int p = 0; p < PARTS; ++p) t[s][p] = t4[(s * 3 + p) * 32];
    }
    const int dc0 = shift_of(__shfl_sync(0xffffffffu, my_row, gq)), dc1 = shift_of(__shfl_sync(0xffffffffu, my_row, gq + 8));
    // this lane's two sums of a group of 8 channels go here, the group's place added
    float* to0 = mine + gq * U::kPitch + 2 * q + dc0;
    float* to1 = mine + (gq + 8) * U::kPitch + 2 * q + dc1;
    const uint16_t* w = g.b + (long long)a * g.N * g.R;
    auto weights = [&](int n, uint32_t (&b)[RP / 8]) {  // of channels c0 + 8 n + gq
      const long long ch = c0 + 8 * n + gq;
      const bool there = (!SHIFT || ch >= 0) && ch < g.N;
      const uint16_t* row = w + (there ? ch * g.R : 0);
#pragma unroll
      for (int h = 0; h < RP / (4 * kLoad); ++h) {
        uint32_t part[kLoad / 2];
        load_weights<kLoad, VEC>(row, 4 * kLoad * h + kLoad * q, there ? g.R : 0, part);
#pragma unroll
        for (int i = 0; i < kLoad / 2; ++i) b[h * (kLoad / 2) + i] = part[i];
      }
    };
    auto multiply = [&](const uint32_t (&b)[RP / 8], float (&d)[4]) {
      d[0] = d[1] = d[2] = d[3] = 0.f;
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int p = PARTS - 1; p >= 0; --p) {
          if constexpr (RP <= 64)
            mma(d, t[s][p], b[2 * s], b[2 * s + 1]);
          else
            mma(d, t4[(s * 3 + p) * 32], b[2 * s], b[2 * s + 1]);
        }
    };
    constexpr int kTurn = RP <= 64 ? 4 : 2;  // groups of 8 channels with their loads in flight
#pragma unroll 1
    for (int n0 = 0; n0 < U::kChannels / 8; n0 += kTurn) {
      uint32_t b[kTurn][RP / 8];
#pragma unroll
      for (int j = 0; j < kTurn; ++j) weights(n0 + j, b[j]);
#pragma unroll
      for (int j = 0; j < kTurn; ++j) {
        float d[4];
        multiply(b[j], d);
        // up to 7 places behind the last chunk: the pitch has room, nobody reads them
        const int at = 8 * (n0 + j);
        if constexpr (SHIFT) {
          to0[at] = d[0];
          to0[at + 1] = d[1];
        } else {
          *reinterpret_cast<float2*>(to0 + at) = make_float2(d[0], d[1]);
        }
        if (count > 8) {
          if constexpr (SHIFT) {
            to1[at] = d[2];
            to1[at + 1] = d[3];
          } else {
            *reinterpret_cast<float2*>(to1 + at) = make_float2(d[2], d[3]);
          }
        }
      }
    }
    if constexpr (SHIFT) {  // the last channels in front of the block, where a row's chunks start earlier
      uint32_t b[RP / 8];
      float d[4];
      weights(-1, b);
      multiply(b, d);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (2 * q + e + dc0 >= 8) to0[e - 8] = d[e];
        if (2 * q + e + dc1 >= 8) to1[e - 8] = d[2 + e];
      }
    }
    __syncwarp();
  }

#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (2 * i >= count) break;
    const int r = 2 * i + (lane >> 4);
    const long long row = __shfl_sync(0xffffffffu, my_row, r);
    const long long id = c0 + (lane & 15) * E - shift_of(row);
    if (r >= count || id >= g.N) continue;
    char* o = out + (row * g.ldo + id) * kSize;
    uint4 z = v[i];
    if (a == kBad) {
      const uint32_t nan = F32 ? 0x7fffffffu : 0x7fff7fffu;
      z = make_uint4(nan, nan, nan, nan);
    } else if (a >= 0) {
      const float4* s = reinterpret_cast<const float4*>(mine + r * U::kPitch + (lane & 15) * E);
      if constexpr (F32) {
        const float4 f = s[0];
        z = make_uint4(__float_as_uint(__uint_as_float(z.x) + f.x), __float_as_uint(__uint_as_float(z.y) + f.y),
                       __float_as_uint(__uint_as_float(z.z) + f.z), __float_as_uint(__uint_as_float(z.w) + f.w));
      } else {
        const float4 f = s[0], h = s[1];
        z = make_uint4(pack_bf(bf_lo(z.x) + f.x, bf_hi(z.x) + f.y), pack_bf(bf_lo(z.y) + f.z, bf_hi(z.y) + f.w),
                       pack_bf(bf_lo(z.z) + h.x, bf_hi(z.z) + h.y), pack_bf(bf_lo(z.w) + h.z, bf_hi(z.w) + h.w));
      }
    }
    if ((!SHIFT || id >= 0) && id + E <= g.N) {
      st16(o, z);
    } else {  // the ends of a row
      const uint32_t w[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (id + e < 0 || id + e >= g.N) continue;
        if constexpr (F32)
          reinterpret_cast<uint32_t*>(o)[e] = w[e];
        else
          reinterpret_cast<uint16_t*>(o)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

cudaLaunchConfig_t config(dim3 grid, int threads, size_t smem, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}
// Opts a kernel into its shared memory, once per device.
template <typename K>
bool allow_smem(K kern, int bytes) {
  return cached(reinterpret_cast<const void*>(kern), bytes, [&](int) {
           return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess ? 1 : -1;
         }) == 1;
}

template <bool XF32, int PARTS, bool VEC>
cudaError_t launch_down(const AdapterArgs& g, long long most, Tile* tiles, uint8_t* t, int parts, cudaStream_t st) {
  auto kern = k_adapters_down<XF32, PARTS, VEC>;
  if (!allow_smem(kern, (int)sizeof(Down))) return cudaErrorUnknown;
  cudaLaunchAttribute attr;
  const dim3 grid((unsigned)most, (unsigned)((padded(g.R) + kDownRanks - 1) / kDownRanks), 1);
  const cudaLaunchConfig_t cfg = config(grid, kDownThreads, sizeof(Down), st, &attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, g, tiles, t, parts);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <bool F32, int RP, bool VEC, bool NEAR, bool SHIFT>
cudaError_t launch_up(const AdapterArgs& g, unsigned most, const Tile* tiles, const uint8_t* t, cudaStream_t st) {
  using U = Up<F32>;
  auto kern = k_adapters_up<F32, RP, VEC, NEAR, SHIFT>;
  if (!allow_smem(kern, U::kSmem)) return cudaErrorUnknown;
  cudaLaunchAttribute attr;
  const long long blocks = ((long long)g.N + (SHIFT ? U::E - 1 : 0) + U::kChannels - 1) / U::kChannels;
  const dim3 grid((unsigned)((blocks + kUpWarps - 1) / kUpWarps), most, 1);
  const cudaLaunchConfig_t cfg = config(grid, kUpWarps * 32, U::kSmem, st, &attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, g, tiles, t);
  if (e == cudaSuccess) note_launch();
  return e;
}
template <bool F32, int RP, bool VEC>
cudaError_t launch_up_as(const AdapterArgs& g, bool near, bool shift, unsigned most, const Tile* tiles, const uint8_t* t,
                         cudaStream_t st) {
  if (!near) return launch_up<F32, RP, VEC, false, true>(g, most, tiles, t, st);
  return shift ? launch_up<F32, RP, VEC, true, true>(g, most, tiles, t, st)
               : launch_up<F32, RP, VEC, true, false>(g, most, tiles, t, st);
}
template <bool F32>
cudaError_t launch_up_ranks(const AdapterArgs& g, bool vec, bool near, bool shift, unsigned most, const Tile* tiles,
                            const uint8_t* t, cudaStream_t st) {
#define DS_UP(RP)                                                            \
  return vec ? launch_up_as<F32, RP, true>(g, near, shift, most, tiles, t, st) \
             : launch_up_as<F32, RP, false>(g, near, shift, most, tiles, t, st)
  switch (padded(g.R)) {
    case 16: DS_UP(16);
    case 32: DS_UP(32);
    case 64: DS_UP(64);
    default: DS_UP(128);
  }
#undef DS_UP
}

}  // namespace

long long adapters_workspace(int n, int L, int R) { return tiles_of(n, L) * ((long long)sizeof(Tile) + t_bytes(R)); }

cudaError_t launch_add_adapters(const AdapterArgs& g, bool x_f32, bool f32, cudaStream_t st) {
  const long long most = tiles_of(g.n, g.L);
  Tile* tiles = static_cast<Tile*>(g.workspace);
  uint8_t* t = reinterpret_cast<uint8_t*>(tiles + most);
  cudaLaunchAttribute attr;
  cudaError_t e = cudaSuccess;
  if (g.n > kSelfPlan) {
    const int smem = (g.L + 2) * 4;
    const cudaLaunchConfig_t cfg = config(dim3(1, 1, 1), kPlanThreads, (size_t)smem, st, &attr);
    e = cudaLaunchKernelEx(&cfg, k_adapters_plan, g, tiles, (int)most);
    if (e != cudaSuccess) return e;
    note_launch();
  }
  const auto at16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const int xs = x_f32 ? 4 : 2, s = f32 ? 4 : 2, parts = f32 ? 3 : 2;
  const bool x_vec = at16(g.x) && at16(g.a) && at16(g.gain) && g.K % 8 == 0 && g.ldx * xs % 16 == 0;
  if (!x_f32 && !g.gain)  // the inputs are bf16 themselves
    e = x_vec ? launch_down<false, 1, true>(g, most, tiles, t, parts, st) : launch_down<false, 1, false>(g, most, tiles, t, parts, st);
  else if (x_f32 && f32)
    e = x_vec ? launch_down<true, 3, true>(g, most, tiles, t, parts, st) : launch_down<true, 3, false>(g, most, tiles, t, parts, st);
  else if (x_f32)
    e = x_vec ? launch_down<true, 2, true>(g, most, tiles, t, parts, st) : launch_down<true, 2, false>(g, most, tiles, t, parts, st);
  else if (f32)
    e = x_vec ? launch_down<false, 3, true>(g, most, tiles, t, parts, st) : launch_down<false, 3, false>(g, most, tiles, t, parts, st);
  else
    e = x_vec ? launch_down<false, 2, true>(g, most, tiles, t, parts, st) : launch_down<false, 2, false>(g, most, tiles, t, parts, st);
  if (e != cudaSuccess) return e;
  const bool vec = padded(g.R) == 16 ? g.R % 4 == 0 && (reinterpret_cast<uintptr_t>(g.b) & 7) == 0 : g.R % 8 == 0 && at16(g.b);
  const bool near = ((reinterpret_cast<uintptr_t>(g.base) ^ reinterpret_cast<uintptr_t>(g.out)) & 15) == 0 &&
                    (g.ldb - g.ldo) * s % 16 == 0;
  const bool shift = !at16(g.out) || g.ldo * s % 16 != 0;
  // the grid's second dimension ends at 65535
  for (long long first = 0; first < most && e == cudaSuccess; first += 65535) {
    const unsigned some = (unsigned)(most - first < 65535 ? most - first : 65535);
    const uint8_t* ts = t + first * t_bytes(g.R);
    e = f32 ? launch_up_ranks<true>(g, vec, near, shift, some, tiles + first, ts, st)
            : launch_up_ranks<false>(g, vec, near, shift, some, tiles + first, ts, st);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace ds
