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
#include <cooperative_groups.h>

#include "ds_device.cuh"
#include "ds_launch.h"

namespace cg = cooperative_groups;

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

// A row's filter parameters, and what its kernels share of it.
struct RowParams {
  float tau, p, mp, u, r;
  int k;  // 0: no top-k
  bool bad;
};

__device__ __forceinline__ RowParams row_params(const FilteredArgs& a, long long n) {
  RowParams q;
  q.tau = a.temperature[n];
  q.u = a.u[n];
  q.p = a.top_p ? a.top_p[n] : 1.f;
  q.mp = a.min_p ? a.min_p[n] : 0.f;
  const int k = a.top_k ? a.top_k[n] : 0;
  q.k = (k > 0 && k < a.V) ? k : 0;
  q.bad = !(q.tau >= 0.f && q.tau < kInf) || !(q.u >= 0.f && q.u < 1.f) || !(q.p > 0.f && q.p <= 1.f) ||
          !(q.mp >= 0.f && q.mp <= 1.f);
  q.r = fminf(__frcp_rn(q.tau), 3.402823466e38f);
  return q;
}

// The smallest integer mass at which top-p is met, and the draw's target.
__device__ __forceinline__ u64 need_of(float p, u64 total) { return (u64)ceil((double)p * (double)total); }
__device__ __forceinline__ u64 target_of(float u, u64 total) { return (u64)floor((double)u * (double)total); }

// The row's token by bisection on the keys, one CTA re-reading the row for every
// question. Slow (some 50 passes) and without any assumption on the row: it
// finishes the rows whose ties are too many for the lists of the fast kernel.
template <typename T, int NT>
__device__ __noinline__ int row_exact(const T* row, int V, const RowParams& q, float m, u64* red, int* slot) {
  const float r = q.r;
  u64 total = row_measure<T, NT>(row, V, kMass, 0u, m, r, red);
  if (q.k) {
    const Cut c = row_select<T, NT>(row, V, kCount, (u64)q.k - 1, m, r, red);
    const u64 above = row_measure<T, NT>(row, V, kMass, c.key + 1u, m, r, red);
    total = above + ((u64)q.k - c.before) * sf_weight(Logit<T>::value(c.key), m, r);
  }
  if (q.p < 1.f) {
    // kept while the mass before is below p * total: through the first whose running mass reaches it
    const u64 need = need_of(q.p, total);
    if (need < total) total = cut_mass_through(row_select<T, NT>(row, V, kMass, need - 1, m, r, red), need - 1);
  }
  if (q.mp > 0.f) {
    const double floor_w = (double)q.mp * (double)kSfOne;
    u64 sum = 0;
    for (int i = threadIdx.x; i < V; i += NT) {
      const uint32_t w = sf_weight(Logit<T>::get(row, i), m, r);
      if ((double)w >= floor_w) sum += w;
    }
    sum = block_sum<NT>(sum, red);
    total = sum < total ? sum : total;
  }
  const u64 t = target_of(q.u, total);
  const Cut c = row_select<T, NT>(row, V, kMass, t, m, r, red);
  return row_nth<T, NT>(row, V, c.key, (t - c.before) / c.each, red, slot);
}

}  // namespace

// One CTA per row, re-read from global memory: rows too long for a cluster's shared memory.
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
    int odd = 0;  // a NaN or +inf
    for (int i = tid; i < V; i += kSfNT) {
      const float x = Logit<T>::get(row, i);
      odd |= !(x < kInf);
      s += expf(x - m);
    }
    s = warp_sum(s);
    odd = __syncthreads_or(odd);
    if (lane == 0) fred[wid] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSfNT / 32; ++i) s += fred[i];
    const float lse = m + logf(s);

    const RowParams q = row_params(a, n);
    int token = -1;
    float lp = __int_as_float(0x7fffffff);
    if (q.bad || odd || m == -kInf) {
      if (tid == 0 && (q.bad || odd)) report(a.d_status, q.bad ? DS_DEV_ERR_PARAM : DS_DEV_ERR_LOGITS);
    } else {
      token = q.tau == 0.f ? row_nth<T, kSfNT>(row, V, Logit<T>::key(m), 0, red, &slot)
                           : row_exact<T, kSfNT>(row, V, q, m, red, &slot);
      lp = Logit<T>::get(row, token) - lse;
    }
    if (tid == 0) {
      a.out_tokens[n] = token;
      a.out_logprobs[n] = lp;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- the row on chip
//
// A cluster of cs CTAs holds a row in shared memory, a contiguous slice each, and
// answers the three questions from histograms over bins of x:
//   max     m, the smallest logit that is no mask, and a cut x1 below which about
//           half of the threads' maxima lie, so that some thousand logits at most
//           are above it while NT / 4 at least are
//   weigh   sum exp(x - m); the mass of the row (unless a small top-k makes it
//           needless); and for the logits >= x1, the ones that decide nearly
//           every row, count and mass in bins linear in x
//   decide  the CTA of rank 0 sums up the bins and finds those where the top-k,
//           top-p and draw boundaries can lie. If one lies below x1, the rest of
//           the row gets bins too.
//   gather  the logits of those bins, a few dozen, come to rank 0, which sorts
//           them and answers exactly.
// A row whose boundary bins hold more than CAP logits (ties) is finished by
// row_exact. So a logit costs two exponentials and its share of three walks over
// shared memory, an atomic only above x1.
namespace {

template <int NT, int NB, int CAP>
struct SfShared {
  uint32_t cnt[NB], lo[NB], hi[NB];  // this CTA's bins: count, and mass as two sums of 16-bit halves
  u64 pm[NB];                        // rank 0: mass through each bin
  uint32_t pc[NB];                   // rank 0: count through each bin
  u64 list[CAP];                     // rank 0: gathered (key, ~id)
  u64 incl[CAP];                     // rank 0: running mass through each of them
  u64 red[NT / 32];
  float fred[3][NT / 32];
  uint32_t marks[NB / 32];
  u64 part_total, part_floor;  // read by rank 0
  float part_max, part_min, part_cut, part_sum;
  float row[4];
  int part_odd;
  int command, gate, n_list, first_id;
  u64 known_total, known_floor;
  float known_sum;
  int known_odd;
  int kb;
  int slot;
};

enum Command { kDone, kGather, kTail, kExact };

// v of the lane of rank `want` (0: largest) among the first `lanes` lanes.
__device__ __forceinline__ float warp_nth_largest(float v, int lane, int lanes, int want) {
  int rank = 0;
  for (int j = 0; j < lanes; ++j) {
    const float o = __shfl_sync(0xffffffffu, v, j);
    rank += (o > v) || (o == v && j < lane);
  }
  const unsigned at = __ballot_sync(0xffffffffu, lane < lanes && rank == want);
  return __shfl_sync(0xffffffffu, v, at ? __ffs(at) - 1 : 0);
}

// Index of the first element of the ascending array that is >= t (n if none), by one warp.
template <typename U>
__device__ __forceinline__ int warp_lower_bound(const U* v, int n, U t, int lane) {
  const int step = n / 32;
  const int seg = __popc(__ballot_sync(0xffffffffu, v[(lane + 1) * step - 1] < t));
  if (seg == 32) return n;
  int at = seg * step;
  for (int o = 0; o < step; o += 32) {
    const unsigned below = __ballot_sync(0xffffffffu, o + lane < step && v[seg * step + o + lane] < t);
    at += __popc(below);
  }
  return at;
}

template <typename T>
struct Chunk;  // 16 bytes of logits as fp32
template <>
struct Chunk<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[8]) { unpack8(v, f); }
};
template <>
struct Chunk<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
};

__device__ __forceinline__ void sf_cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

}  // namespace

template <typename T, int NT, int NB, int CAP>
__global__ void __launch_bounds__(NT, 1024 / NT) k_sample_filtered(FilteredArgs a) {
  constexpr int EPC = Chunk<T>::N, NBT = NB / 2, NW = NT / 32;
  using Shared = SfShared<NT, NB, CAP>;
  extern __shared__ uint4 slice[];
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int cs = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const long long n_clusters = (long long)gridDim.x / cs, cid = (long long)blockIdx.x / cs;
  Shared* lead = cl.map_shared_rank(&sh, 0);
  auto sync = [&] {
    if (cs == 1)
      __syncthreads();
    else
      cl.sync();
  };
  pdl_wait();
  pdl_release();

  // This CTA's slice of a row: chunks [q_lo, q_hi) of the row's 16-byte chunks
  // (chunk 0 starts at the row's first element rounded down to 16 bytes; the
  // copies stay inside the 16-byte blocks that hold the row).
  struct Slice {
    const uint4* base;
    int dc, nq, q_lo, q_hi;
  };
  auto slice_of = [&](long long n) {
    Slice g;
    const uintptr_t ad = reinterpret_cast<uintptr_t>(static_cast<const T*>(a.x) + n * a.ld);
    g.base = reinterpret_cast<const uint4*>(ad & ~(uintptr_t)15);
    g.dc = (int)((ad & 15) / sizeof(T));
    g.nq = (g.dc + a.V + EPC - 1) / EPC;
    g.q_lo = (int)((long long)rank * g.nq / cs);
    g.q_hi = (int)((long long)(rank + 1) * g.nq / cs);
    return g;
  };
  auto start_copy = [&](long long n) {
    if (n < a.n) {
      const Slice g = slice_of(n);
      for (int q = g.q_lo + tid; q < g.q_hi; q += NT) sf_cp_async16(&slice[q - g.q_lo], g.base + q);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  start_copy(cid);

  for (long long n = cid; n < a.n; n += n_clusters) {
    const Slice g = slice_of(n);
    const RowParams q = row_params(a, n);
    // the logits of chunk j of this thread's walk; ids outside the row read as -inf
    auto values = [&](int j, float (&f)[EPC]) {
      Chunk<T>::get(slice[j - g.q_lo], f);
      if (j == 0 || j == g.nq - 1) {
#pragma unroll
        for (int i = 0; i < EPC; ++i) {
          const int e = EPC * j - g.dc + i;
          if (e < 0 || e >= a.V) f[i] = -kInf;
        }
      }
    };
    for (int i = tid; i < NB; i += NT) sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
    if (tid == 0) {
      sh.n_list = 0;
      sh.first_id = INT_MAX;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // a thread reads only the chunks that it copied

    // ---- max
    float mx = -kInf, mn = kInf;
    for (int j = g.q_lo + tid; j < g.q_hi; j += NT) {
      float f[EPC];
      values(j, f);
#pragma unroll
      for (int i = 0; i < EPC; ++i) {
        mx = fmaxf(mx, f[i]);
        if (f[i] > -3e37f) mn = fminf(mn, f[i]);
      }
    }
    {
      const float wm = warp_max(mx), wn = -warp_max(-mn), wc = warp_nth_largest(mx, lane, 32, 15);
      if (lane == 0) {
        sh.fred[0][wid] = wm;
        sh.fred[1][wid] = wn;
        sh.fred[2][wid] = wc;
      }
      __syncthreads();
      if (wid == 0) {
        const float bm = warp_max(lane < NW ? sh.fred[0][lane] : -kInf);
        const float bn = -warp_max(lane < NW ? -sh.fred[1][lane] : -kInf);
        const float bc = warp_nth_largest(lane < NW ? sh.fred[2][lane] : -kInf, lane, NW, NW / 2 - 1);
        if (lane == 0) {
          sh.part_max = bm;
          sh.part_min = bn;
          sh.part_cut = bc;
        }
      }
      sync();
      if (wid == 0) {
        const Shared* o = lane < cs ? cl.map_shared_rank(&sh, lane) : &sh;
        const float m = warp_max(o->part_max), lo = -warp_max(-o->part_min), cut = warp_max(o->part_cut);
        if (lane == 0) {
          sh.row[0] = m;
          sh.row[1] = fminf(lo, m);
          sh.row[2] = cut;
        }
      }
      __syncthreads();
    }
    const float m = sh.row[0];
    // No logit below x_low has a weight: w > 0 needs (x - m) r > -22.2, and the
    // rest is room for the rounding of x_low. Masks are told from logits by
    // their size, which needs a range that ends above them.
    const float lowest = (m - 24.f * q.tau) - fabsf(m) * 2.4e-7f;
    const float x_low = lowest > -3e37f ? fmaxf(sh.row[1], lowest) : fmaxf(lowest, -3.402823466e38f);
    const float x1 = fmaxf(sh.row[2], x_low);  // splits the rest
    const float sc1 = fminf((float)NBT / (m - x1), 3.402823466e38f);
    const float sc2 = fminf((float)(NB - NBT) / (x1 - x_low), 3.402823466e38f);
    auto bin_of = [&](float x) {  // for x_low <= x <= m
      return x >= x1 ? min(NBT - 1, __float2int_rz((m - x) * sc1))
                     : min(NB - 1, NBT + min(NB, __float2int_rz((x1 - x) * sc2)));
    };
    const bool drawn = !q.bad && q.tau > 0.f && m > -kInf && m < kInf;
    const bool greedy = !q.bad && q.tau == 0.f && m > -kInf && m < kInf;
    // A top-k of at most NT / 4 ends above x1: the mass below is then not asked for.
    const bool whole = drawn && !(q.k && q.k <= NT / 4);
    const double floor_w = (double)q.mp * (double)kSfOne;
    const uint32_t floor_i = (uint32_t)ceil(floor_w);

    // ---- weigh
    float s = 0.f;
    u64 total = 0, above_floor = 0;
    int odd = 0, first = INT_MAX;
    for (int j = g.q_lo + tid; j < g.q_hi; j += NT) {
      float f[EPC];
      values(j, f);
#pragma unroll
      for (int i = 0; i < EPC; ++i) {
        const float x = f[i];
        odd |= !(x < kInf);
        s += ex2_approx((x - m) * kLog2e);
        if (greedy && x == m) first = min(first, EPC * j - g.dc + i);
        if (drawn && x >= (whole ? x_low : x1)) {
          const uint32_t w = sf_weight(x, m, q.r);
          total += w;
          if (w >= floor_i) above_floor += w;
          if (x >= x1 && w) {
            const int b = bin_of(x);
            atomicAdd(&sh.cnt[b], 1u);
            atomicAdd(&sh.lo[b], w & 0xffffu);
            atomicAdd(&sh.hi[b], w >> 16);
          }
        }
      }
    }
    s = warp_sum(s);
    total = block_sum<NT>(total, sh.red);
    above_floor = block_sum<NT>(above_floor, sh.red);
    odd = __syncthreads_or(odd);
    if (lane == 0) sh.fred[0][wid] = s;
    if (greedy) {
      first = warp_min_i(first);
      if (lane == 0 && first != INT_MAX) atomicMin(&lead->first_id, first);
    }
    __syncthreads();
    if (tid == 0) {
      s = 0.f;
      for (int i = 0; i < NW; ++i) s += sh.fred[0][i];
      sh.part_sum = s;
      sh.part_total = total;
      sh.part_floor = above_floor;
      sh.part_odd = odd;
    }
    sync();

    // Sums the cluster's bins [b0, b0 + NB / 2) into rank 0's pm and pc, a share of them per CTA.
    auto merge_bins = [&](int b0) {
      for (int i = rank * NT + tid; i < NB / 2; i += cs * NT) {
        const int b = b0 + i;
        uint32_t c = 0;
        u64 mass = 0;
        for (int o = 0; o < cs; ++o) {
          const Shared* peer = cl.map_shared_rank(&sh, o);
          c += peer->cnt[b];
          mass += (u64)peer->lo[b] + ((u64)peer->hi[b] << 16);
        }
        lead->pc[b] = c;
        lead->pm[b] = mass;
      }
    };
    // Rank 0: running sums of those bins, continuing from (m0, c0).
    auto scan_bins = [&](int b0, u64 m0, uint32_t c0) {
      constexpr int PER = (NBT + NT - 1) / NT;
      u64 mass[PER], sm = 0;
      uint32_t c[PER], sc = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        mass[i] = b < NBT ? sh.pm[b0 + b] : 0;
        c[i] = b < NBT ? sh.pc[b0 + b] : 0;
        sm += mass[i];
        sc += c[i];
      }
      u64 im = sm;
      uint32_t ic = sc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 um = __shfl_up_sync(0xffffffffu, im, o);
        const uint32_t uc = __shfl_up_sync(0xffffffffu, ic, o);
        if (lane >= o) {
          im += um;
          ic += uc;
        }
      }
      __syncthreads();
      if (lane == 31) {
        sh.red[wid] = im;
        sh.fred[0][wid] = __uint_as_float(ic);
      }
      __syncthreads();
      u64 bm = m0 + im - sm;
      uint32_t bc = c0 + ic - sc;
      for (int w = 0; w < wid; ++w) {
        bm += sh.red[w];
        bc += __float_as_uint(sh.fred[0][w]);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        bm += mass[i];
        bc += c[i];
        if (b < NBT) {
          sh.pm[b0 + b] = bm;
          sh.pc[b0 + b] = bc;
        }
      }
      __syncthreads();
    };
    // Rank 0, warp 0: which bins the boundaries can lie in (see the kernel's comment).
    auto decide = [&](bool tail) {
      const int nb = tail ? NB : NBT;
      const u64 known = sh.pm[nb - 1], all = sh.known_total, fl = sh.known_floor;
      const uint32_t count = sh.pc[nb - 1];
      const bool complete = tail || !whole || known == all;
      uint32_t mark = 0;  // lane l: bins [32 l, 32 l + 32)
      auto mark_range = [&](int b0, int b1) {
        for (int wd = lane; wd < NB / 32; wd += 32) {
          const int lo = max(b0 - 32 * wd, 0), hi = min(b1 - 32 * wd, 31);
          if (lo <= hi) mark |= (0xffffffffu << lo) & (0xffffffffu >> (31 - hi));
        }
      };
      u64 t_lo, t_hi;  // bounds of the kept mass
      int kb = -1;
      if (q.k && (uint32_t)q.k <= count) {
        kb = warp_lower_bound<uint32_t>(sh.pc, nb, (uint32_t)q.k, lane);
        t_hi = sh.pm[kb];
        t_lo = t_hi;
        if (sh.pc[kb] != (uint32_t)q.k) {
          t_lo = kb ? sh.pm[kb - 1] : 0;
          mark_range(kb, kb);
        }
      } else if (q.k && !complete) {
        return (int)kTail;
      } else {
        t_lo = t_hi = whole ? all : known;
      }
      if (q.p < 1.f) {
        const u64 n_lo = need_of(q.p, t_lo), n_hi = need_of(q.p, t_hi);
        if (n_hi > known) return complete ? (int)kExact : (int)kTail;
        const int b0 = warp_lower_bound<u64>(sh.pm, nb, n_lo > 0 ? n_lo : 1, lane);
        const int b1 = warp_lower_bound<u64>(sh.pm, nb, n_hi, lane);
        mark_range(b0, b1);
        t_lo = b0 ? sh.pm[b0 - 1] : 0;
        t_hi = sh.pm[b1];
      }
      if (q.mp > 0.f) {
        t_lo = fl < t_lo ? fl : t_lo;
        t_hi = fl < t_hi ? fl : t_hi;
      }
      const u64 d_lo = target_of(q.u, t_lo), d_hi = target_of(q.u, t_hi);
      if (d_hi >= known) return complete ? (int)kExact : (int)kTail;
      mark_range(warp_lower_bound<u64>(sh.pm, nb, d_lo + 1, lane), warp_lower_bound<u64>(sh.pm, nb, d_hi + 1, lane));
      int listed = 0;
      for (uint32_t w = lane < NB / 32 ? mark : 0u; w; w &= w - 1) {
        const int b = 32 * lane + __ffs(w) - 1;
        listed += (int)(sh.pc[b] - (b ? sh.pc[b - 1] : 0u));
      }
      if (warp_sum_i(listed) > CAP) return (int)kExact;
      if (lane < NB / 32) sh.marks[lane] = mark;
      if (lane == 0) {
        sh.kb = kb;
      }
      const bool low = __any_sync(0xffffffffu, lane >= NBT / 32 && lane < NB / 32 && mark);
      if (lane == 0) sh.gate = low;
      return (int)kGather;
    };

    if (!drawn) {
      start_copy(n + n_clusters);
      if (rank == 0 && tid == 0) {
        int bits = 0;
        float sum = 0.f;
        for (int o = 0; o < cs; ++o) {
          const Shared* peer = cl.map_shared_rank(&sh, o);
          bits |= peer->part_odd;
          sum += peer->part_sum;
        }
        const bool ok = greedy && !bits;
        if (q.bad || bits) report(a.d_status, q.bad ? DS_DEV_ERR_PARAM : DS_DEV_ERR_LOGITS);
        a.out_tokens[n] = ok ? sh.first_id : -1;
        a.out_logprobs[n] = ok ? m - (m + logf(sum)) : __int_as_float(0x7fffffff);
      }
      sync();  // the partials are read before the next row writes them
      continue;
    }

    merge_bins(0);
    if (rank == 0 && wid == 0) {
      const Shared* peer = lane < cs ? cl.map_shared_rank(&sh, lane) : nullptr;
      u64 t = peer ? peer->part_total : 0, fl = peer ? peer->part_floor : 0;
      float sum = peer ? peer->part_sum : 0.f;
      int bits = peer ? peer->part_odd : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        t += __shfl_xor_sync(0xffffffffu, t, o);
        fl += __shfl_xor_sync(0xffffffffu, fl, o);
        bits |= __shfl_xor_sync(0xffffffffu, bits, o);
      }
      sum = warp_sum(sum);
      if (lane == 0) {
        sh.known_total = t;
        sh.known_floor = fl;
        sh.known_sum = sum;
        sh.known_odd = bits;
      }
    }
    sync();
    int command;
    for (bool tail = false;; tail = true) {
      if (rank == 0) {
        if (tail)
          scan_bins(NBT, sh.pm[NBT - 1], sh.pc[NBT - 1]);
        else
          scan_bins(0, 0, 0);
        if (wid == 0) {
          const int c = sh.known_odd ? (int)kDone : decide(tail);
          __syncwarp();
          for (int o = 0; o < cs; ++o) {
            Shared* peer = cl.map_shared_rank(&sh, o);
            if (o && lane < NB / 32) peer->marks[lane] = sh.marks[lane];
            if (lane == 0) {
              peer->gate = sh.gate;
              peer->command = c;
            }
          }
        }
      }
      sync();
      command = sh.command;
      if (command != kTail) break;
      for (int j = g.q_lo + tid; j < g.q_hi; j += NT) {
        float f[EPC];
        values(j, f);
#pragma unroll
        for (int i = 0; i < EPC; ++i) {
          const float x = f[i];
          if (x >= x_low && x < x1) {
            const uint32_t w = sf_weight(x, m, q.r);
            if (w) {
              const int b = bin_of(x);
              atomicAdd(&sh.cnt[b], 1u);
              atomicAdd(&sh.lo[b], w & 0xffffu);
              atomicAdd(&sh.hi[b], w >> 16);
            }
          }
        }
      }
      sync();
      merge_bins(NBT);
      sync();
    }
    if (command == kGather) {
      const float gate = sh.gate ? x_low : x1;
      for (int j = g.q_lo + tid; j < g.q_hi; j += NT) {
        float f[EPC];
        values(j, f);
#pragma unroll
        for (int i = 0; i < EPC; ++i) {
          const float x = f[i];
          if (x >= gate) {
            const int b = bin_of(x);
            if ((sh.marks[b >> 5] >> (b & 31)) & 1u) {
              if (sf_weight(x, m, q.r)) {
                const int at = atomicAdd(&lead->n_list, 1);
                if (at < CAP)
                  lead->list[at] =
                      ((u64)Logit<T>::key(x) << 32) | (u64)(0xffffffffu - (uint32_t)(EPC * j - g.dc + i));
              }
            }
          }
        }
      }
      sync();
    }
    start_copy(n + n_clusters);
    if (rank != 0) continue;

    // ---- rank 0 answers
    const float lse = m + logf(sh.known_sum);
    if (command == kDone) {
      if (tid == 0) {
        report(a.d_status, DS_DEV_ERR_LOGITS);
        a.out_tokens[n] = -1;
        a.out_logprobs[n] = __int_as_float(0x7fffffff);
      }
    } else if (command == kExact) {
      const T* row = static_cast<const T*>(a.x) + n * a.ld;
      const int token = row_exact<T, NT>(row, a.V, q, m, sh.red, &sh.slot);
      if (tid == 0) {
        a.out_tokens[n] = token;
        a.out_logprobs[n] = Logit<T>::get(row, token) - lse;
      }
    } else {
      const int len = sh.n_list;
      int pow2 = 32;
      while (pow2 < len) pow2 *= 2;
      for (int i = len + tid; i < pow2; i += NT) sh.list[i] = 0;
      __syncthreads();
      // bitonic sort, descending
      for (int size = 2; size <= pow2; size *= 2)
        for (int d = size / 2; d > 0; d /= 2) {
          for (int i = tid; i < pow2 / 2; i += NT) {
            const int x = 2 * i - (i & (d - 1)), y = x + d;
            const u64 u = sh.list[x], v = sh.list[y];
            if ((u < v) == ((x & size) == 0)) {
              sh.list[x] = v;
              sh.list[y] = u;
            }
          }
          __syncthreads();
        }
      if (wid == 0) {
        // running mass through each listed logit: through its bin's predecessor, plus the listed ones of its bin
        u64 sum = 0, off = 0, kept = 0;
        int off_at = 0, off_count = 0, last_bin = -1;
        for (int j = 0; j < len; j += 32) {
          const bool in = j + lane < len;
          const float x = in ? Logit<T>::value((uint32_t)(sh.list[j + lane] >> 32)) : 0.f;
          const u64 w = in ? (u64)sf_weight(x, m, q.r) : 0;
          const int b = in ? bin_of(x) : NB;
          u64 run = w;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const u64 up = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += up;
          }
          run += sum;
          int before = __shfl_up_sync(0xffffffffu, b, 1);
          if (lane == 0) before = last_bin;
          const bool head = in && b != before;
          const u64 my_off = head ? (b ? sh.pm[b - 1] : 0) - (run - w) : 0;  // wraps: added back below
          const int my_count = head && b ? (int)sh.pc[b - 1] : 0;
          const unsigned heads = __ballot_sync(0xffffffffu, head) & (0xffffffffu >> (31 - lane));
          const int src = heads ? 31 - __clz(heads) : 0;
          const u64 so = __shfl_sync(0xffffffffu, my_off, src);
          const int sc = __shfl_sync(0xffffffffu, my_count, src);
          const u64 o_use = heads ? so : off;
          const int c_use = heads ? sc : off_count, at_use = heads ? j + src : off_at;
          if (in) sh.incl[j + lane] = run + o_use;
          const bool at_k = in && sh.kb >= 0 && c_use + (j + lane - at_use) + 1 == q.k;
          const unsigned ks = __ballot_sync(0xffffffffu, at_k);
          if (ks) kept = __shfl_sync(0xffffffffu, run + o_use, __ffs(ks) - 1);
          sum = __shfl_sync(0xffffffffu, run, 31);
          off = __shfl_sync(0xffffffffu, o_use, 31);
          off_count = __shfl_sync(0xffffffffu, c_use, 31);
          off_at = __shfl_sync(0xffffffffu, at_use, 31);
          last_bin = __shfl_sync(0xffffffffu, b, 31);
        }
        __syncwarp();
        auto first_at_least = [&](u64 t) {
          for (int j = 0; j < len; j += 32) {
            const unsigned hit = __ballot_sync(0xffffffffu, j + lane < len && sh.incl[j + lane] >= t);
            if (hit) return j + __ffs(hit) - 1;
          }
          return len - 1;  // not reached: the boundary's bin is listed
        };
        u64 all;
        if (sh.kb >= 0)
          all = sh.pc[sh.kb] == (uint32_t)q.k ? sh.pm[sh.kb] : kept;
        else
          all = whole ? sh.known_total : sh.pm[NBT - 1];
        if (q.p < 1.f) all = sh.incl[first_at_least(need_of(q.p, all))];
        if (q.mp > 0.f) all = sh.known_floor < all ? sh.known_floor : all;
        const int at = first_at_least(target_of(q.u, all) + 1);
        if (lane == 0) {
          const u64 e = sh.list[at];
          a.out_tokens[n] = (int)(0xffffffffu - (uint32_t)e);
          a.out_logprobs[n] = Logit<T>::value((uint32_t)(e >> 32)) - lse;
        }
      }
    }
    __syncthreads();  // the lists are free
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  sync();  // no CTA leaves while a peer may still use its shared memory
}

namespace {

constexpr int kSfSmallV = 4096;             // rows up to here: 128-thread CTAs
constexpr long long kSfSlice = 64 << 10;    // bytes of a row per CTA, two CTAs per SM
constexpr long long kSfSliceMax = 128 << 10;  // one CTA per SM; at most 65536 logits, which the bins' 32-bit sums allow
constexpr long long kSfSliceMin = 8 << 10;

// Launches the cluster kernel; *refused when no cluster of that shape fits.
template <typename T, int NT, int NB, int CAP>
cudaError_t launch_on_chip(const FilteredArgs& a, int cs, size_t smem, cudaStream_t st, bool* refused) {
  auto kern = k_sample_filtered<T, NT, NB, CAP>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.gridDim = dim3((unsigned)cs);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const void* site = reinterpret_cast<const void*>(kern);
  const int ok = cached(site, -1, [&](int) {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSfSliceMax + 32);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (r != cudaSuccess) (void)cudaGetLastError();
    return r == cudaSuccess ? 1 : 0;
  });
  const int fit = ok <= 0 ? 0 : cached(site, (long long)smem * 32 + cs, [&](int) {
    int v = 0;
    const cudaError_t r = cudaOccupancyMaxActiveClusters(&v, kern, &cfg);
    if (r != cudaSuccess) {
      (void)cudaGetLastError();
      return 0;
    }
    return v;
  });
  if (fit < 1) {
    *refused = true;
    return cudaSuccess;
  }
  const long long clusters = a.n < fit ? a.n : fit;
  cfg.gridDim = dim3((unsigned)(clusters * cs));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

template <typename T>
static cudaError_t launch_filtered(const FilteredArgs& a, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorUnknown;
  const long long bytes = (long long)a.V * sizeof(T) + 16;
  bool refused = false;
  if (a.V <= kSfSmallV) {
    const cudaError_t e = launch_on_chip<T, 128, 128, 256>(a, 1, (size_t)(bytes + 15) / 16 * 16, st, &refused);
    if (!refused) return e;
  } else {
    int cs = 1;
    while (cs < 16 && bytes > cs * kSfSlice) cs *= 2;
    // few rows: more CTAs per row, down to 8 KB each
    while (cs < 8 && (long long)a.n * cs * 2 <= sms && bytes > cs * 2 * kSfSliceMin) cs *= 2;
    const long long slice = (bytes / 16 + cs) / cs * 16 + 16;
    if (slice <= kSfSliceMax) {
      const cudaError_t e = launch_on_chip<T, 512, 1024, 1024>(a, cs, (size_t)slice, st, &refused);
      if (!refused) return e;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.n < sms * 4LL ? a.n : sms * 4LL));
  cfg.blockDim = dim3(kSfNT);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_sample_filtered_rows<T>, a);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_sample_filtered(const FilteredArgs& a, bool f32, cudaStream_t st) {
  return f32 ? launch_filtered<float>(a, st) : launch_filtered<uint16_t>(a, st);
}

}  // namespace ds
