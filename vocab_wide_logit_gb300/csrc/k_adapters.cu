// k_adapters.cu -- low-rank adapters of many requests added to shared logits.
//
//   out_i = base_i + scale_a B_a (A_a y_i),  a = ids[i],
//   y = x, or x rsqrt(mean x^2 + eps) gain
//
// Rows are gathered into tiles of up to 16 that have the same adapter, so that an
// adapter's weights are read once for 16 rows in whatever order the rows come.
//   k_adapters_plan  (more than 8192 rows) one CTA counts the rows of each adapter and
//                    deals them out to tiles; up to 8192 rows the next kernel's CTAs each
//                    find their own tile, which saves a launch (4 us).
//   k_adapters_down  a CTA per tile and 32 ranks: t = scale A y by matrix instructions
//                    (16 rows x 8 ranks x 16 inputs), the inputs split over 16 warps.
//   k_adapters_up    CTAs that stay, each with an equal share of (tile, block of channels)
//                    pairs: t B^T by matrix instructions (16 rows x 8 channels x 16
//                    ranks), then base and result in whole 16-byte chunks a row.
// The adapters' bf16 goes into the instructions as it is. The fp32 operand goes in as a
// sum of bf16 parts, each the rest that the parts before it left, off by 2^-8 of it at
// most: three of them (2^-24 is lost) for fp32 logits, two (2^-16) for bf16 logits, whose
// own rounding is 2^-8. Sums are fp32.
//
// What bounds it is HBM: base, result and the weights once. The weights of a block of
// channels are one run of bytes whatever the rank, and come to shared memory with the
// base's chunks by asynchronous copies of 16 bytes, two or three blocks ahead: with the
// loads of a block in registers instead, 16 warps of 100 registers an SM left the memory
// idle two thirds of the time. 256 rows x 248320 of rank 64 and 32 adapters: 200 us,
// 6.4 TB/s; 24 rows of rank 16 and 8 adapters: 26 us, 6 of them for t. A lane takes the
// ranks that lie together, 8 or 16 bytes, as "its" four of an instruction's 16 (any order
// of the ranks is right that both operands share). Rows start at any element: a block of
// channels starts for each row at that row's own 16-byte boundary, for which eight
// channels in front of the block are computed twice.
#include "ds_device.cuh"
#include "ds_index.h"
#include "ds_launch.h"

namespace ds {

namespace {

constexpr int kRows = 16;          // rows of a tile
constexpr int kSelfPlan = 8192;    // rows up to which k_adapters_down plans for itself
constexpr int kDownThreads = 512;
constexpr int kDownWarps = kDownThreads / 32;
constexpr int kDownRanks = 32;     // ranks of a CTA
constexpr int kPlanThreads = 1024;
constexpr int kUpThreads = 256;
constexpr int kWideShare = 10;     // blocks a CTA from which they are wide
constexpr int kNone = -1, kBad = -2;  // a tile of rows without an adapter, of ids beyond the stack

// Rows of one adapter; count 0: no tile.
struct Tile {
  int32_t adapter, count;
  int32_t rows[kRows];
  int32_t pad[14];
};
static_assert(sizeof(Tile) == 128, "tiles keep what follows them aligned");

// What stands in front of the tiles.
struct Head {
  int32_t tiles;
  int32_t pad[31];
};

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

// Eight fp32 from k on that start at any 4 bytes, zeros from K on.
__device__ __forceinline__ void load8(const void* row, int k, int K, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = k + i < K ? load<true>(row, k + i) : 0.f;
}
// Eight weights of 16 bytes as they are, zeros from `end` on.
__device__ __forceinline__ void load_weights(const uint16_t* row, int i, int end, uint32_t (&w)[4]) {
  const uint4 v = i < end ? ld_stream16(row + i) : make_uint4(0, 0, 0, 0);
  w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
}

// ---------------------------------------------------------------- tiles
// More than 8192 rows: counted, then dealt out. Which rows share a tile may differ from
// run to run; a row's result does not depend on it.
__global__ void __launch_bounds__(kPlanThreads) k_adapters_plan(const AdapterArgs g, Head* head, Tile* tiles, int most) {
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
  if (tid == 0) head->tiles = all;
}

// Up to 32 rows: tile number `want` of those that the rows' order makes, found by a warp
// alone, to rows[]. Returns how many there are.
__device__ __forceinline__ int warp_plan(const AdapterArgs& g, int want, int32_t* rows, int& adapter, int& count) {
  const int lane = threadIdx.x & 31;
  const bool there = lane < g.n;
  const int kind = there ? kind_of(g.ids[lane], g.L) : kBad - 1;
  const int before = __popc(__match_any_sync(0xffffffffu, kind) & ((1u << lane) - 1));  // rows of the kind in front
  unsigned leaders = __ballot_sync(0xffffffffu, there && before % kRows == 0);
  const int all = __popc(leaders);
  for (int i = 0; i < want; ++i) leaders &= leaders - 1;
  const int leader = leaders ? __ffs(leaders) - 1 : 0;
  adapter = __shfl_sync(0xffffffffu, kind, leader);
  const int first = __shfl_sync(0xffffffffu, before, leader);
  const bool in = leaders && there && kind == adapter && before / kRows == first / kRows;
  if (lane < kRows) rows[lane] = 0;
  __syncwarp();
  if (in) rows[before % kRows] = lane;
  count = __popc(__ballot_sync(0xffffffffu, in));
  return all;
}

// Up to 8192 rows: the same by a CTA, the tiles in the order of the adapters, then those
// without one, then the bad ones.
constexpr int kFewKinds = 32;  // a lane each
struct SelfPlan {
  int sums[kDownWarps];
  int adapter, part, count;
  int few[kDownWarps][kFewKinds];  // rows of each kind in each warp's stretch
};
__device__ __forceinline__ int block_plan(const AdapterArgs& g, int want, SelfPlan& s, uint32_t* counts, int32_t* rows, int& adapter,
                                          int& count) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, kinds = g.L + 2;
  // a stretch of rows to each warp, 32 at a time
  constexpr int kTimes = kSelfPlan / kDownThreads;
  const int times = (g.n + kDownThreads - 1) / kDownThreads, i0 = wid * times * 32 + lane;
  int kind[kTimes];
#pragma unroll
  for (int i = 0; i < kTimes; ++i) kind[i] = i < times && i0 + 32 * i < g.n ? g.ids[i0 + 32 * i] : 0;
  if (tid < kRows) rows[tid] = 0;
  auto index_of = [&](int kind) { return kind >= 0 ? kind : g.L - 1 - kind; };
#pragma unroll
  for (int i = 0; i < kTimes; ++i)
    if (i < times) kind[i] = i0 + 32 * i < g.n ? kind_of(kind[i], g.L) : kBad - 1;
  int all = 0, slot;  // slot: the place in the tile of the warp's first row of the kind
  if (kinds <= kFewKinds) {
    s.few[wid][lane] = 0;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      if (i >= times) break;
      const unsigned same = __match_any_sync(0xffffffffu, kind[i]);
      if (kind[i] >= kBad && (same & ((1u << lane) - 1)) == 0) s.few[wid][index_of(kind[i])] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    // every warp finds the tile for itself, a kind a lane
    int rows_of = 0, before = 0;
#pragma unroll
    for (int i = 0; i < kDownWarps; ++i) {
      const int c = s.few[i][lane];
      rows_of += c;
      before += i < wid ? c : 0;
    }
    const int mine = (rows_of + kRows - 1) / kRows;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    all = __shfl_sync(0xffffffffu, incl, 31);
    const unsigned who = __ballot_sync(0xffffffffu, want >= incl - mine && want < incl);
    if (!who) {
      count = 0;
      adapter = kNone;
      return all;
    }
    const int owner = __ffs(who) - 1;
    const int part = want - __shfl_sync(0xffffffffu, incl - mine, owner);
    adapter = owner < g.L ? owner : g.L - 1 - owner;
    count = min(kRows, __shfl_sync(0xffffffffu, rows_of, owner) - part * kRows);
    slot = __shfl_sync(0xffffffffu, before, owner) - part * kRows;
  } else {
    for (int i = tid; i < kinds; i += kDownThreads) counts[i] = 0;
    if (tid == 0) s.count = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      if (i >= times) break;
      const unsigned same = __match_any_sync(0xffffffffu, kind[i]);
      if (kind[i] >= kBad && (same & ((1u << lane) - 1)) == 0) atomicAdd(&counts[index_of(kind[i])], (uint32_t)__popc(same));
    }
    __syncthreads();
    const int per = (kinds + kDownThreads - 1) / kDownThreads, lo = tid * per, hi = min(lo + per, kinds);
    int mine = 0;
    for (int i = lo; i < hi; ++i) mine += (int)((counts[i] + kRows - 1) / kRows);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s.sums[wid] = incl;
    __syncthreads();
    int at = incl - mine;
    for (int i = 0; i < kDownWarps; ++i) {
      at += i < wid ? s.sums[i] : 0;
      all += s.sums[i];
    }
    if (want >= at && want < at + mine)
      for (int i = lo; i < hi; ++i) {
        const int t = (int)((counts[i] + kRows - 1) / kRows);
        if (want >= at && want < at + t) {
          s.adapter = i < g.L ? i : g.L - 1 - i;
          s.part = want - at;
          s.count = min(kRows, (int)counts[i] - s.part * kRows);
        }
        at += t;
      }
    __syncthreads();
    adapter = s.adapter;
    count = s.count;
    if (count == 0) return all;
    int found = 0;
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      if (i >= times) break;
      found += __popc(__ballot_sync(0xffffffffu, kind[i] == adapter));
    }
    if (lane == 0) s.sums[wid] = found;
    __syncthreads();
    slot = -s.part * kRows;
    for (int i = 0; i < wid; ++i) slot += s.sums[i];
  }
  __syncthreads();  // rows[] is zero
#pragma unroll
  for (int i = 0; i < kTimes; ++i) {
    if (i >= times) break;
    const bool in = kind[i] == adapter;
    const unsigned who = __ballot_sync(0xffffffffu, in);
    const int to = slot + __popc(who & ((1u << lane) - 1));
    if (in && to >= 0 && to < kRows) rows[to] = i0 + 32 * i;
    slot += __popc(who);
  }
  __syncthreads();
  return all;
}

// ---------------------------------------------------------------- t = scale A y
struct Down {
  SelfPlan plan;
  int32_t rows[kDownWarps][kRows];  // the tile's, a copy for each warp that finds it alone
  float t[kDownWarps][kRows][kDownRanks + 1];
  float squares[kDownWarps][kRows];
  double wide[kDownWarps];
  float factor[kRows];
};

// Eight inputs as they come from memory.
template <bool F32>
struct Raw {
  uint4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const char* row, int k, int K) {
    const uint4* p = reinterpret_cast<const uint4*>(row + (long long)k * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = k < K ? __ldg(p + i) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(v[i].x), f[4 * i + 1] = __uint_as_float(v[i].y);
        f[4 * i + 2] = __uint_as_float(v[i].z), f[4 * i + 3] = __uint_as_float(v[i].w);
      }
    } else {
      unpack8(v[0], f);
    }
  }
};

// Eight bf16 from i on that start at any 2 bytes, as they are; zeros from `end` on: words
// of 4 bytes, each of which has one of those in front of `end`.
__device__ __forceinline__ void load_any(const uint16_t* row, int i, int end, uint32_t (&w)[4]) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + i);
  const int odd = (int)(at >> 1) & 1;
  const uint32_t* p = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
  uint32_t f[5];
#pragma unroll
  for (int j = 0; j < 5; ++j) f[j] = word_wanted(i, j, odd, end) ? __ldg(p + j) : 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = odd ? __funnelshift_r(f[j], f[j + 1], 16) : f[j];
  if (i + 8 > end) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + 2 * j >= end) w[j] = 0;
      if (i + 2 * j + 1 >= end) w[j] &= 0xffffu;
    }
  }
}

// PARTS: bf16 parts of an input. VEC: 16-byte loads. GROUPS: of 8 ranks, 2 or 4.
template <bool XF32, int PARTS, bool VEC, int GROUPS>
__global__ void __launch_bounds__(kDownThreads) k_adapters_down(const AdapterArgs g, Head* head, Tile* tiles, uint8_t* t_out,
                                                                int parts_out) {
  extern __shared__ __align__(16) unsigned char raw[];
  Down& sh = *reinterpret_cast<Down*>(raw);
  pdl_release();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, gq = lane >> 2, q = lane & 3;
  const int32_t* rows = sh.rows[0];
  int count, a, all = -1;
  if (g.n <= 32) {
    all = warp_plan(g, blockIdx.x, sh.rows[wid], a, count);
    rows = sh.rows[wid];
    __syncwarp();
  } else if (g.n <= kSelfPlan) {
    all = block_plan(g, blockIdx.x, sh.plan, reinterpret_cast<uint32_t*>(raw + sizeof(Down)), sh.rows[0], a, count);
  } else {
    const Tile& tile = tiles[blockIdx.x];
    count = tile.count;
    a = tile.adapter;
    if (tid < kRows) sh.rows[0][tid] = tid < count ? tile.rows[tid] : 0;
    __syncthreads();
  }
  if (all >= 0 && blockIdx.y == 0 && wid == 0) {
    Tile& tile = tiles[blockIdx.x];
    if (lane < kRows) tile.rows[lane] = rows[lane];
    if (lane == 0) {
      tile.adapter = a;
      tile.count = count;
      if (blockIdx.x == 0) head->tiles = all;
      if (count > 0 && a == kBad) report(g.d_status, DS_DEV_ERR_PARAM);
    }
  }
  if (count <= 0 || a < 0) return;
  constexpr int kSize = XF32 ? 4 : 2;
  const char* x = static_cast<const char*>(g.x);
  const bool has0 = gq < count, has1 = gq + 8 < count;
  const char* x0 = x + rows[gq] * g.ldx * kSize;
  const char* x1 = x + rows[gq + 8] * g.ldx * kSize;
  const int K0 = has0 ? g.K : 0, K1 = has1 ? g.K : 0;
  const int rank0 = blockIdx.y * kDownRanks;
  const uint16_t* wr[GROUPS];
  int Kw[GROUPS];
#pragma unroll
  for (int j = 0; j < GROUPS; ++j) {
    const int r = rank0 + 8 * j + gq;
    Kw[j] = r < g.R ? g.K : 0;  // (of 65 to 96 ranks filled up to 128 the last block has none)
    wr[j] = g.a + rank_at(a, r, g.R, g.K);
  }

  float d[GROUPS][4] = {};
  float ss0 = 0.f, ss1 = 0.f;
  const bool half = count <= 8;
  auto take = [&](float (&f0)[8], float (&f1)[8], const float (&n8)[8], const uint32_t (&b)[GROUPS][4]) {
    if (g.gain) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss0 = __fmaf_rn(f0[i], f0[i], ss0);
        f0[i] *= n8[i];
      }
      if (!half) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss1 = __fmaf_rn(f1[i], f1[i], ss1);
          f1[i] *= n8[i];
        }
      }
    }
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      uint32_t h0[4], h1[4] = {0, 0, 0, 0};
      auto part = [&](float (&f)[8], uint32_t (&h)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[i] = pack_bf(f[2 * i], f[2 * i + 1]);
          if (p + 1 < PARTS) {
            f[2 * i] -= bf_lo(h[i]);
            f[2 * i + 1] -= bf_hi(h[i]);
          }
        }
      };
      part(f0, h0);
      if (!half) part(f1, h1);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint4 av = make_uint4(h0[2 * s], h1[2 * s], h0[2 * s + 1], h1[2 * s + 1]);
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) mma(d[j], av, b[j][2 * s], b[j][2 * s + 1]);
      }
    }
  };
  // 32 inputs a step: lane q of a row's four takes 8 that lie together, four of them
  // for each of two instructions
  constexpr int kStep = kDownWarps * 32;
  if constexpr (VEC) {
    constexpr int kDepth = GROUPS == 2 && !XF32 ? 4 : 2;  // steps in flight
    for (int k0 = wid * 32; k0 < g.K; k0 += kDepth * kStep) {
      Raw<XF32> r0[kDepth], r1[kDepth];
      Raw<true> rn[kDepth];
      uint32_t b[kDepth][GROUPS][4];
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        const int k = k0 + i * kStep + 8 * q;
        r0[i].load(x0, k, K0);
        r1[i].load(x1, k, K1);
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) load_weights(wr[j], k, Kw[j], b[i][j]);
        if (g.gain) rn[i].load(reinterpret_cast<const char*>(g.gain), k, g.K);
      }
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        if (k0 + i * kStep >= g.K) break;
        float f0[8], f1[8], n8[8];
        r0[i].floats(f0);
        r1[i].floats(f1);
        rn[i].floats(n8);
        take(f0, f1, n8, b[i]);
      }
    }
  } else {
#pragma unroll 2
    for (int k0 = wid * 32; k0 < g.K; k0 += kStep) {
      const int k = k0 + 8 * q;
      float f0[8], f1[8], n8[8];
      uint32_t b[GROUPS][4];
      if constexpr (XF32) {
        load8(x0, k, K0, f0);
        load8(x1, k, K1, f1);
      } else {
        uint32_t w0[4], w1[4];
        load_any(reinterpret_cast<const uint16_t*>(x0), k, K0, w0);
        load_any(reinterpret_cast<const uint16_t*>(x1), k, K1, w1);
        unpack8(make_uint4(w0[0], w0[1], w0[2], w0[3]), f0);
        unpack8(make_uint4(w1[0], w1[1], w1[2], w1[3]), f1);
      }
#pragma unroll
      for (int j = 0; j < GROUPS; ++j) load_any(wr[j], k, Kw[j], b[j]);
      load8(g.gain, k, g.gain ? g.K : 0, n8);
      take(f0, f1, n8, b);
    }
  }
#pragma unroll
  for (int j = 0; j < GROUPS; ++j) {
    sh.t[wid][gq][8 * j + 2 * q] = d[j][0];
    sh.t[wid][gq][8 * j + 2 * q + 1] = d[j][1];
    sh.t[wid][gq + 8][8 * j + 2 * q] = d[j][2];
    sh.t[wid][gq + 8][8 * j + 2 * q + 1] = d[j][3];
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    ss0 += __shfl_xor_sync(0xffffffffu, ss0, o);
    ss1 += __shfl_xor_sync(0xffffffffu, ss1, o);
  }
  if (q == 0) {
    sh.squares[wid][gq] = ss0;
    sh.squares[wid][gq + 8] = ss1;
  }
  __syncthreads();
  // a thread per row and rank; the row's factor is scale and the norm's root
  const int row = tid / kDownRanks, r = tid % kDownRanks, rank = rank0 + r;
  float t = 0.f, factor = 1.f;
  if (r < GROUPS * 8)
#pragma unroll
    for (int i = 0; i < kDownWarps; ++i) t += sh.t[i][row][r];
  if (g.gain) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kDownWarps; ++i) ss += sh.squares[i][row];
    const bool usual = ss > 1e-25f && ss < 1e37f;
    factor = rsqrtf(ss / (float)g.K + g.eps);
    // squares that leave fp32's range, rows of zeros: the sum in 64 bits
    if (__syncthreads_or(row < count && !usual)) {
      if (r == 0) sh.factor[row] = row < count && !usual ? -1.f : factor;
      __syncthreads();
      for (int i = 0; i < count; ++i) {
        if (sh.factor[i] != -1.f) continue;
        const char* p = x + rows[i] * g.ldx * kSize;
        double sum = 0;
        for (int k = tid; k < g.K; k += kDownThreads) {
          const double v = load<XF32>(p, k);
          sum += v * v;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) sh.wide[wid] = sum;
        __syncthreads();
        sum = 0;
        for (int j = 0; j < kDownWarps; ++j) sum += sh.wide[j];
        __syncthreads();
        if (tid == 0) sh.factor[i] = sum == 0 ? 0.f : (float)(1.0 / sqrt(sum / g.K + g.eps));
      }
      __syncthreads();
      factor = sh.factor[row];
    }
  }
  if (r < GROUPS * 8) {
    // an infinity or NaN in x is in every t of its row, whatever the weights
    if (!(fabsf(t) < kInf)) t = __int_as_float(0x7fffffff);
    t = row < count ? t * (factor * g.scale[a]) : 0.f;
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
// The kernel's sizes. RP: padded ranks. WIDE: blocks of 64 chunks of a row instead of 32,
// with 16 ranks.
template <bool F32, int RP, bool SHIFT, bool WIDE>
struct Up {
  static constexpr int E = F32 ? 4 : 8;                          // logits of a chunk
  static constexpr int kChunks = WIDE ? 64 : (F32 ? RP <= 64 : RP <= 32) ? 32 : F32 || RP <= 64 ? 16 : 8;  // of a row and block
  static constexpr int kChannels = kChunks * E;                  // of a block
  static constexpr int kGroups = kChannels / 8;                  // of 8 channels
  static constexpr int kFront = SHIFT ? 8 : 0;                   // channels in front of the block
  // Channels of a warp and block: 8 columns of as many instructions. Where two of each
  // make whole chunks a lane and rows start on chunks, sums go straight from the lane that
  // has them to the result; else through shared memory.
  // With 128 ranks half of the warps take half of the ranks each: t stays in registers.
  static constexpr int kHalves = RP == 128 ? 2 : 1, kWarps = 8 / kHalves;
  static constexpr int kMine = kGroups / kWarps;
  static constexpr int kPieces = 2 * kMine / E;                  // chunks of a lane
  static constexpr bool kDirect = !SHIFT && kPieces > 0 && kHalves == 1;
  static constexpr int kPitch = kChannels + 8;                   // rows of results lie 8 banks apart
  // weights that may start at any 2 bytes, and base
  static constexpr int kWeights = (kChannels + kFront) * RP * 2 + 32;
  static constexpr int kStage = kWeights + kRows * kChunks * 16;
  static constexpr int kResults = kDirect ? 0 : kHalves * kRows * kPitch * 4;
  static constexpr int kCtas = RP == 16 && kChunks == 32 ? 3 : 2;  // of an SM
  static constexpr int kStages = kCtas * (4 * kStage + kResults) <= 220 * 1024 ? 4 : 3;
  static constexpr int kSmem = kStages * kStage + kResults;
};

__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void st16(void* p, uint4 v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// `COUNT` (4 or 8) weights in shared memory from rank i on, zeros from `end` on, PIECE (8, 4
// or 1) of them a load.
template <int COUNT, int PIECE>
__device__ __forceinline__ void shared_weights(const unsigned char* row, int i, int end, uint32_t* w) {
  if constexpr (PIECE == 8 && COUNT == 8) {
    const uint4 v = i < end ? *reinterpret_cast<const uint4*>(row + 2 * i) : make_uint4(0, 0, 0, 0);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (PIECE >= 4) {
#pragma unroll
    for (int j = 0; j < COUNT / 4; ++j) {
      const uint2 v = i + 4 * j < end ? *reinterpret_cast<const uint2*>(row + 2 * i + 8 * j) : make_uint2(0, 0);
      w[2 * j] = v.x, w[2 * j + 1] = v.y;
    }
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
    for (int j = 0; j < COUNT / 2; ++j) {
      const uint32_t lo = i + 2 * j < end ? p[i + 2 * j] : 0u, hi = i + 2 * j + 1 < end ? p[i + 2 * j + 1] : 0u;
      w[j] = lo | (hi << 16);
    }
  }
}

// PIECE: weights of a load. NEAR: base and result rows lie the same way to
// 16 bytes. SHIFT: some row starts between two chunks.
template <bool F32, int RP, int PIECE, bool NEAR, bool SHIFT, bool WIDE>
__global__ void __launch_bounds__(kUpThreads, (Up<F32, RP, SHIFT, WIDE>::kCtas))
    k_adapters_up(const AdapterArgs g, const Head* head, const Tile* tiles, const uint8_t* t_in, int blocks) {
  using U = Up<F32, RP, SHIFT, WIDE>;
  constexpr int E = U::E, kSize = F32 ? 4 : 2, PARTS = F32 ? 3 : 2, STEPS = RP / 16 / U::kHalves, S = U::kStages, W = U::kChunks;
  constexpr int kLoad = RP == 16 ? 4 : 8;  // weights of a lane and load: one instruction's, or two's
  constexpr int kTurns = (kRows * W + kUpThreads - 1) / kUpThreads;
  extern __shared__ __align__(16) unsigned char smem[];
  float* results = reinterpret_cast<float*>(smem + S * U::kStage);  // without kDirect
  const uint32_t smem_at = (uint32_t)__cvta_generic_to_shared(smem);
  pdl_release();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, gq = lane >> 2, q = lane & 3;
  // this CTA's share: total / grid blocks, one more for the first ones
  const long long total = (long long)head->tiles * blocks;
  const bool few = total <= 0x7fffffffLL;  // 64-bit quotients take 100 ns each
  const long long share = few ? (uint32_t)total / gridDim.x : total / gridDim.x;
  const int more = (int)(total - share * gridDim.x);
  const long long lo = share * blockIdx.x + min((int)blockIdx.x, more), hi = lo + share + ((int)blockIdx.x < more);
  const int first_tile = few ? (int)((uint32_t)lo / (uint32_t)blocks) : (int)(lo / blocks);
  const int first_block = (int)(lo - (long long)first_tile * blocks);
  char* out = static_cast<char*>(g.out);
  const char* base = static_cast<const char*>(g.base);
  // how many logits of a row's first chunk are before it
  auto shift_of = [&](long long row) {
    return SHIFT ? (int)(reinterpret_cast<uintptr_t>(out + row * g.ldo * kSize) & 15) / kSize : 0;
  };
  // turn k of a thread: chunk tid % W of the tile's row tid / W + kPerTurn k
  constexpr int kPerTurn = kUpThreads / W;
  const int my_chunk = (tid % W) * E, my_row = tid / W;
  const int row_bytes = g.R * 2;
  // a block's first copied channel: with SHIFT those in front of it too
  auto front = [&](int b) { return SHIFT && b > 0 ? 8 : 0; };

  // Asks for blocks one after the other, on its own way through the tiles.
  struct Ask {
    int tile, block, count, adapter;
    const char* weights;           // the adapter's, of channel 0
    const char* base[kTurns];      // this thread's chunks of block 0
    int shift[kTurns];
  } ask;
  ask.tile = -1;
  int ask_at = first_tile;
  ask.block = first_block;
  long long asked = lo;
  auto issue = [&](int stage) {
    if (asked < hi) {
      if (ask.tile != ask_at) {
        ask.tile = ask_at;
        const Tile& tile = tiles[ask_at];
        ask.count = tile.count;
        ask.adapter = tile.adapter;
        ask.weights = reinterpret_cast<const char*>(g.b) + (long long)max(ask.adapter, 0) * g.N * row_bytes;
        if (!NEAR || ask.adapter == kBad || (ask.adapter == kNone && g.out == g.base)) ask.count = 0;  // no base
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
          const int r = my_row + kPerTurn * k;
          const long long row = r < ask.count ? tile.rows[r] : 0;
          ask.shift[k] = shift_of(row);
          ask.base[k] = base + (row * g.ldb + my_chunk - ask.shift[k]) * kSize;
        }
      }
      const int c0 = ask.block * U::kChannels;
      const uint32_t to = smem_at + stage * U::kStage + 16 * tid;
      if (ask.adapter >= 0) {
        const int f = front(ask.block), c1 = min(U::kChannels, g.N - c0);
        const char* from = ask.weights + (long long)(c0 - f) * row_bytes;
        const int off = (int)(reinterpret_cast<uintptr_t>(from) & 15);
        const int bytes = off + (c1 + f) * row_bytes;
        from += 16 * tid - off;
#pragma unroll
        for (int i = 0; i < (U::kWeights / 16 + kUpThreads - 1) / kUpThreads; ++i)
          if (16 * (tid + i * kUpThreads) < bytes) copy16(to + 16 * i * kUpThreads, from + 16 * i * kUpThreads);
      }
#pragma unroll
      for (int k = 0; k < kTurns; ++k) {
        if (my_row + kPerTurn * k >= ask.count) break;
        // the ends may be other rows' bytes, of the same 16
        if (c0 + my_chunk - ask.shift[k] < g.N)
          copy16(to + U::kWeights + 16 * k * kUpThreads, ask.base[k] + (long long)c0 * kSize);
      }
      if (++ask.block == blocks) ask.block = 0, ++ask_at;
      ++asked;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);

  int at = first_tile, block = first_block, stage = 0, ready = -1;
  int count = 0, a = kNone, dc0 = 0, dc1 = 0;
  bool idle = true;
  const char* weights = nullptr;
  constexpr int kMine = U::kMine;
  char* to_direct[2];  // kDirect: this lane's channels of block 0 in its two rows
  char* to_out[kTurns];
  const char* from_base[kTurns];  // without NEAR
  int shift[kTurns];
  const uint4* t4 = nullptr;
  uint4 t[STEPS][PARTS];
  const int strand = wid % U::kWarps, half = wid / U::kWarps;  // of the warp's channels, of its ranks
  for (long long item = lo; item < hi; ++item) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    __syncthreads();
    issue(stage == 0 ? S - 1 : stage - 1);
    if (ready != at) {
      ready = at;
      const Tile& tile = tiles[at];
      count = tile.count;
      a = tile.adapter;
      idle = a == kNone && g.out == g.base;
      weights = reinterpret_cast<const char*>(g.b) + (long long)max(a, 0) * g.N * row_bytes;
      t4 = reinterpret_cast<const uint4*>(t_in + at * t_bytes(g.R)) + lane;
      if constexpr (U::kDirect) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const long long row = gq + 8 * k < count ? tile.rows[gq + 8 * k] : 0;
          to_direct[k] = out + (row * g.ldo + 8 * kMine * wid + 2 * kMine * q) * kSize;
        }
      }
#pragma unroll
      for (int k = 0; !U::kDirect && k < kTurns; ++k) {
        const int r = my_row + kPerTurn * k;
        const long long row = r < count ? tile.rows[r] : 0;
        shift[k] = shift_of(row);
        to_out[k] = out + (row * g.ldo + my_chunk - shift[k]) * kSize;
        from_base[k] = base + (row * g.ldb + my_chunk - shift[k]) * kSize;
      }
      if (a >= 0) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
          for (int p = 0; p < PARTS; ++p) t[s][p] = t4[((half * STEPS + s) * 3 + p) * 32];
        dc0 = gq < count ? shift_of(tile.rows[gq]) : 0;
        dc1 = gq + 8 < count ? shift_of(tile.rows[gq + 8]) : 0;
      }
    }
    const int c0 = block * U::kChannels, left = g.N - c0;  // channels from here on
    const unsigned char* here = smem + stage * U::kStage;
    if constexpr (U::kDirect) {
      if (!idle) {
        // instruction j's column n is channel 2 kMine (n / 2) + 2 j + n % 2 of the warp's: a lane's
        // two columns of all of them lie together
        float d[kMine][4] = {};
        if (a >= 0) {
          const int first = 8 * kMine * wid + 2 * kMine * (gq >> 1) + (gq & 1);
          const unsigned char* w = here + (int)((reinterpret_cast<uintptr_t>(weights) + (long long)c0 * row_bytes) & 15) +
                                   first * row_bytes;
#pragma unroll
          for (int j = 0; j < kMine; ++j) {
            const bool there = left >= U::kChannels || first + 2 * j < left;
            const unsigned char* row = w + (there ? 2 * j * row_bytes : 0);
#pragma unroll
            for (int h = 0; h < RP / (4 * kLoad); ++h) {
              uint32_t b[kLoad / 2];
              shared_weights<kLoad, PIECE>(row, 4 * kLoad * h + kLoad * q, there ? g.R : 0, b);
#pragma unroll
              for (int i = 0; i < kLoad / 4; ++i)
#pragma unroll
                for (int p = PARTS - 1; p >= 0; --p) mma(d[j], t[h * (kLoad / 4) + i][p], b[2 * i], b[2 * i + 1]);
            }
          }
        }
        const int id0 = c0 + 8 * kMine * wid + 2 * kMine * q;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (gq + 8 * k >= count) break;
          const unsigned char* from = here + U::kWeights + 16 * ((gq + 8 * k) * W + U::kPieces * (4 * wid + q));
          char* o = to_direct[k] + (long long)c0 * kSize;
#pragma unroll
          for (int c = 0; c < U::kPieces; ++c) {
            const int id = id0 + c * E;
            if (id >= g.N) break;
            uint4 z = *reinterpret_cast<const uint4*>(from + 16 * c);
            if (a == kBad) {
              const uint32_t nan = F32 ? 0x7fffffffu : 0x7fff7fffu;
              z = make_uint4(nan, nan, nan, nan);
            } else if (a >= 0) {
              uint32_t f[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
              for (int j = 0; j < E / 2; ++j) {
                const float* s = &d[c * (E / 2) + j][2 * k];
                if constexpr (F32) {
                  f[2 * j] = __float_as_uint(__uint_as_float(f[2 * j]) + s[0]);
                  f[2 * j + 1] = __float_as_uint(__uint_as_float(f[2 * j + 1]) + s[1]);
                } else {
                  f[j] = pack_bf(bf_lo(f[j]) + s[0], bf_hi(f[j]) + s[1]);
                }
              }
              z = make_uint4(f[0], f[1], f[2], f[3]);
            }
            if (g.N - id >= E) {
              st16(o + 16 * c, z);
            } else {  // the end of a row
              const uint32_t w4[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
              for (int e = 0; e < E; ++e) {
                if (e >= g.N - id) break;
                if constexpr (F32)
                  reinterpret_cast<uint32_t*>(o + 16 * c)[e] = w4[e];
                else
                  reinterpret_cast<uint16_t*>(o + 16 * c)[e] = (uint16_t)(w4[e >> 1] >> (16 * (e & 1)));
              }
            }
          }
        }
      }
      if (++block == blocks) block = 0, ++at;
      if (++stage == S) stage = 0;
      continue;
    }
    if (a >= 0) {
      const int f = front(block);
      const unsigned char* w = here + (int)((reinterpret_cast<uintptr_t>(weights) + (long long)(c0 - f) * row_bytes) & 15) +
                               (f + gq) * row_bytes;
      auto multiply = [&](int n, bool there, float (&d)[4]) {  // of channels c0 + 8 n + gq
        const unsigned char* row = w + (there ? n * 8 * row_bytes : 0);
        d[0] = d[1] = d[2] = d[3] = 0.f;
#pragma unroll
        for (int h = 0; h < STEPS * 4 / kLoad; ++h) {
          uint32_t b[kLoad / 2];
          shared_weights<kLoad, PIECE>(row, 16 * STEPS * half + 4 * kLoad * h + kLoad * q, there ? g.R : 0, b);
#pragma unroll
          for (int i = 0; i < kLoad / 4; ++i)
#pragma unroll
            for (int p = PARTS - 1; p >= 0; --p) mma(d, t[h * (kLoad / 4) + i][p], b[2 * i], b[2 * i + 1]);
        }
      };
      // this lane's two sums of a group of 8 channels go here, the group's place added
      float* to0 = results + (half * kRows + gq) * U::kPitch + 2 * q + dc0;
      float* to1 = results + (half * kRows + gq + 8) * U::kPitch + 2 * q + dc1;
      auto put = [&](int n, const float (&d)[4]) {
        // up to 7 places behind the last chunk: the pitch has room, nobody reads them
        if constexpr (SHIFT) {
          to0[8 * n] = d[0];
          to0[8 * n + 1] = d[1];
        } else {
          *reinterpret_cast<float2*>(to0 + 8 * n) = make_float2(d[0], d[1]);
        }
        if (count > 8) {
          if constexpr (SHIFT) {
            to1[8 * n] = d[2];
            to1[8 * n + 1] = d[3];
          } else {
            *reinterpret_cast<float2*>(to1 + 8 * n) = make_float2(d[2], d[3]);
          }
        }
      };
      static_assert(U::kGroups % U::kWarps == 0, "the same number for each");
      float d[kMine][4];
      if (left >= U::kChannels) {
#pragma unroll
        for (int j = 0; j < kMine; ++j) multiply(strand + U::kWarps * j, true, d[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kMine; ++j) multiply(strand + U::kWarps * j, 8 * (strand + U::kWarps * j) + gq < left, d[j]);
      }
#pragma unroll
      for (int j = 0; j < kMine; ++j) put(strand + U::kWarps * j, d[j]);
      if (SHIFT && strand == U::kWarps - 1) {  // the last channels in front of the block, where a row's chunks start earlier
        multiply(-1, f > 0 && gq - 8 < left, d[0]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (2 * q + e + dc0 >= 8) to0[e - 8] = d[0][e];
          if (2 * q + e + dc1 >= 8) to1[e - 8] = d[0][2 + e];
        }
      }
      __syncthreads();
    }
    if (!idle) {
#pragma unroll
      for (int k = 0; k < kTurns; ++k) {
        if (my_row + kPerTurn * k >= count) break;
        const int id = c0 + my_chunk - shift[k];
        if (id >= g.N) continue;
        uint4 z = make_uint4(0, 0, 0, 0);
        if constexpr (NEAR) {
          z = *reinterpret_cast<const uint4*>(here + U::kWeights + 16 * (tid + k * kUpThreads));
        } else {
          const char* p = from_base[k] + (long long)c0 * kSize;
          uint32_t w4[4] = {0, 0, 0, 0};
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (id + e < 0 || id + e >= g.N) continue;
            if constexpr (F32)
              w4[e] = reinterpret_cast<const volatile uint32_t*>(p)[e];
            else
              w4[e >> 1] |= (uint32_t) reinterpret_cast<const volatile uint16_t*>(p)[e] << (16 * (e & 1));
          }
          z = make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
        if (a == kBad) {
          const uint32_t nan = F32 ? 0x7fffffffu : 0x7fff7fffu;
          z = make_uint4(nan, nan, nan, nan);
        } else if (a >= 0) {
          const float4* s = reinterpret_cast<const float4*>(results + (my_row + kPerTurn * k) * U::kPitch + my_chunk);
          if constexpr (F32) {
            float4 f = s[0];
            if constexpr (U::kHalves == 2) f = add4(f, s[kRows * U::kPitch / 4]);
            z = make_uint4(__float_as_uint(__uint_as_float(z.x) + f.x), __float_as_uint(__uint_as_float(z.y) + f.y),
                           __float_as_uint(__uint_as_float(z.z) + f.z), __float_as_uint(__uint_as_float(z.w) + f.w));
          } else {
            float4 f = s[0], h = s[1];
            if constexpr (U::kHalves == 2) f = add4(f, s[kRows * U::kPitch / 4]), h = add4(h, s[kRows * U::kPitch / 4 + 1]);
            z = make_uint4(pack_bf(bf_lo(z.x) + f.x, bf_hi(z.x) + f.y), pack_bf(bf_lo(z.y) + f.z, bf_hi(z.y) + f.w),
                           pack_bf(bf_lo(z.z) + h.x, bf_hi(z.z) + h.y), pack_bf(bf_lo(z.w) + h.z, bf_hi(z.w) + h.w));
          }
        }
        char* o = to_out[k] + (long long)c0 * kSize;
        if ((!SHIFT || id >= 0) && g.N - id >= E) {
          st16(o, z);
        } else {  // the ends of a row
          const uint32_t w4[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (id + e < 0 || id + e >= g.N) continue;
            if constexpr (F32)
              reinterpret_cast<uint32_t*>(o)[e] = w4[e];
            else
              reinterpret_cast<uint16_t*>(o)[e] = (uint16_t)(w4[e >> 1] >> (16 * (e & 1)));
          }
        }
      }
    }
    if (++block == blocks) block = 0, ++at;
    if (++stage == S) stage = 0;
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

template <bool XF32, int PARTS, bool VEC, int GROUPS>
cudaError_t launch_down(const AdapterArgs& g, long long most, Head* head, Tile* tiles, uint8_t* t, int parts, cudaStream_t st) {
  auto kern = k_adapters_down<XF32, PARTS, VEC, GROUPS>;
  if (!allow_smem(kern, (int)sizeof(Down) + (DS_ADAPTERS_MAX + 2) * 4)) return cudaErrorUnknown;
  cudaLaunchAttribute attr;
  const dim3 grid((unsigned)most, (unsigned)((padded(g.R) + kDownRanks - 1) / kDownRanks), 1);
  const size_t smem = sizeof(Down) + (g.n > 32 && g.n <= kSelfPlan ? (g.L + 2) * 4 : 0);
  const cudaLaunchConfig_t cfg = config(grid, kDownThreads, smem, st, &attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, g, head, tiles, t, parts);
  if (e == cudaSuccess) note_launch();
  return e;
}
template <bool XF32, int PARTS>
cudaError_t launch_down_as(const AdapterArgs& g, bool vec, long long most, Head* head, Tile* tiles, uint8_t* t, int parts,
                           cudaStream_t st) {
  if (g.R <= 16)
    return vec ? launch_down<XF32, PARTS, true, 2>(g, most, head, tiles, t, parts, st)
               : launch_down<XF32, PARTS, false, 2>(g, most, head, tiles, t, parts, st);
  return vec ? launch_down<XF32, PARTS, true, 4>(g, most, head, tiles, t, parts, st)
             : launch_down<XF32, PARTS, false, 4>(g, most, head, tiles, t, parts, st);
}

template <bool F32, int RP, int PIECE, bool NEAR, bool SHIFT, bool WIDE>
cudaError_t launch_up(const AdapterArgs& g, long long most, const Head* head, const Tile* tiles, const uint8_t* t,
                      cudaStream_t st) {
  using U = Up<F32, RP, SHIFT, WIDE>;
  static_assert(U::kCtas * (U::kSmem + 1024) <= 228 * 1024, "CTAs an SM");
  auto kern = k_adapters_up<F32, RP, PIECE, NEAR, SHIFT, WIDE>;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorUnknown;
  const long long blocks = ((long long)g.N + (SHIFT ? U::E - 1 : 0) + U::kChannels - 1) / U::kChannels;
  const long long items = most * blocks, ctas = (long long)U::kCtas * sms;
  // wide blocks halve what each costs beside its bytes, and leave CTAs with a few of them
  // in unequal shares: 24 x 248320 (14 a CTA) 25.6 us for 28.2, 1939 x 8200 (7) 22.9 for 22.2
  if constexpr (WIDE && !F32)
    if (items < kWideShare * ctas) return launch_up<F32, RP, PIECE, NEAR, SHIFT, false>(g, most, head, tiles, t, st);
  if (!allow_smem(kern, U::kSmem)) return cudaErrorUnknown;
  cudaLaunchAttribute attr;
  const dim3 grid((unsigned)(items < ctas ? items : ctas), 1, 1);
  const cudaLaunchConfig_t cfg = config(grid, kUpThreads, U::kSmem, st, &attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, g, head, tiles, t, (int)blocks);
  if (e == cudaSuccess) note_launch();
  return e;
}
template <bool F32, int RP, int PIECE>
cudaError_t launch_up_as(const AdapterArgs& g, bool near, bool shift, long long most, const Head* head, const Tile* tiles,
                         const uint8_t* t, cudaStream_t st) {
  constexpr bool kWide = RP == 16;  // (rows between chunks have their sums in shared memory: fp32's fit it)
  if (!near) return launch_up<F32, RP, PIECE, false, true, kWide && F32>(g, most, head, tiles, t, st);
  return shift ? launch_up<F32, RP, PIECE, true, true, kWide && F32>(g, most, head, tiles, t, st)
               : launch_up<F32, RP, PIECE, true, false, kWide>(g, most, head, tiles, t, st);
}
template <bool F32>
cudaError_t launch_up_ranks(const AdapterArgs& g, int piece, bool near, bool shift, long long most, const Head* head,
                            const Tile* tiles, const uint8_t* t, cudaStream_t st) {
#define DS_UP(RP, PIECE) return launch_up_as<F32, RP, PIECE>(g, near, shift, most, head, tiles, t, st)
  switch (padded(g.R)) {
    case 16:
      if (piece == 1) DS_UP(16, 1);
      DS_UP(16, 4);
    case 32:
      if (piece == 1) DS_UP(32, 1);
      if (piece == 4) DS_UP(32, 4);
      DS_UP(32, 8);
    case 64:
      if (piece == 1) DS_UP(64, 1);
      if (piece == 4) DS_UP(64, 4);
      DS_UP(64, 8);
    default:
      if (piece == 1) DS_UP(128, 1);
      if (piece == 4) DS_UP(128, 4);
      DS_UP(128, 8);
  }
#undef DS_UP
}

}  // namespace

long long adapters_workspace(int n, int L, int R) {
  return (long long)sizeof(Head) + tiles_of(n, L) * ((long long)sizeof(Tile) + t_bytes(R));
}

cudaError_t launch_add_adapters(const AdapterArgs& g, bool x_f32, bool f32, cudaStream_t st) {
  const long long most = tiles_of(g.n, g.L);
  Head* head = static_cast<Head*>(g.workspace);
  Tile* tiles = reinterpret_cast<Tile*>(head + 1);
  uint8_t* t = reinterpret_cast<uint8_t*>(tiles + most);
  cudaLaunchAttribute attr;
  cudaError_t e = cudaSuccess;
  if (g.n > kSelfPlan) {
    const int smem = (g.L + 2) * 4;
    const cudaLaunchConfig_t cfg = config(dim3(1, 1, 1), kPlanThreads, (size_t)smem, st, &attr);
    e = cudaLaunchKernelEx(&cfg, k_adapters_plan, g, head, tiles, (int)most);
    if (e != cudaSuccess) return e;
    note_launch();
  }
  const auto at16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const int xs = x_f32 ? 4 : 2, s = f32 ? 4 : 2, parts = f32 ? 3 : 2;
  const bool x_vec = at16(g.x) && at16(g.a) && at16(g.gain) && g.K % 8 == 0 && g.ldx * xs % 16 == 0;
#define DS_DOWN(XF32, PARTS) launch_down_as<XF32, PARTS>(g, x_vec, most, head, tiles, t, parts, st)
  if (!x_f32 && !g.gain)  // the inputs are bf16 themselves
    e = DS_DOWN(false, 1);
  else if (x_f32)
    e = f32 ? DS_DOWN(true, 3) : DS_DOWN(true, 2);
  else
    e = f32 ? DS_DOWN(false, 3) : DS_DOWN(false, 2);
#undef DS_DOWN
  if (e != cudaSuccess) return e;
  // weights that lie together at 16 or 8 bytes in every row of every stack
  const uintptr_t b = reinterpret_cast<uintptr_t>(g.b);
  const int piece = g.R % 8 == 0 && (b & 15) == 0 ? 8 : g.R % 4 == 0 && (b & 7) == 0 ? 4 : 1;
  const bool near = ((reinterpret_cast<uintptr_t>(g.base) ^ reinterpret_cast<uintptr_t>(g.out)) & 15) == 0 &&
                    (g.ldb - g.ldo) * s % 16 == 0;
  const bool shift = !at16(g.out) || g.ldo * s % 16 != 0;
  e = f32 ? launch_up_ranks<true>(g, piece, near, shift, most, head, tiles, t, st)
          : launch_up_ranks<false>(g, piece, near, shift, most, head, tiles, t, st);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace ds
