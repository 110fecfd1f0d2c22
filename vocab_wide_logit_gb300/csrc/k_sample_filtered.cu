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
  static __device__ __forceinline__ float load(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
  static __device__ __forceinline__ uint32_t key(float x) { return order_key(x == 0.f ? 0.f : x) >> 16; }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float(((k & 0x8000u) ? k ^ 0x8000u : ~k) << 16);
  }
};
template <>
struct Logit<float> {
  static __device__ __forceinline__ float get(const float* p, long long i) { return __ldg(p + i); }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
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
//   max     m, the smallest logit that is no mask, and a cut x1: the least of
//           GROUPS groups' maxima, so that GROUPS logits at least are above it
//           and, of independent ones, about ln(GROUPS) times as many
//   weigh   sum exp(x - m); the mass of the row (unless a small top-k makes it
//           needless); and for the logits >= x1, the ones that decide nearly
//           every row, count and mass in bins linear in x
//   decide  the CTA of rank 0 sums up the bins and finds those where the top-k,
//           top-p and draw boundaries can lie. If one lies below x1, the rest of
//           the row gets bins too.
//   gather  the logits of those bins, a few dozen, come to rank 0, which sorts
//           them and answers exactly.
// A row whose boundary bins hold more than CAP logits (ties) is finished by
// row_exact. So a logit costs two exponentials and its share of two walks over
// shared memory, an atomic only above x1.
namespace {

template <int NT, int NB, int CAP>
struct SfShared {
  uint32_t cnt[NB], lo[NB], hi[NB];  // this CTA's bins: count, and mass as two sums of 16-bit halves
  u64 pm[NB];                        // rank 0: mass through each bin
  uint32_t pc[NB];                   // rank 0: count through each bin
  u64 list[CAP];                     // rank 0: gathered (key, ~id)
  u64 incl[CAP];                     // rank 0: running mass through each of them
  u64 full;                          // the slice's copy is done
  u64 red[NT / 32], red2[NT / 32];
  float fred[3][NT / 32], sred[2][NT / 32];
  uint32_t marks[NB / 32];
  // each CTA's partials, pushed by it to everyone (max) or to rank 0 (weigh)
  float part_max[16], part_min[16], part_cut[16], part_sum[16];
  u64 part_total[16], part_floor[16];
  int part_odd[16];
  int command, gate, n_list, first_id;
  u64 known_total, known_floor;
  float known_sum;
  int known_odd;
  int kb;
  int slot;
};

enum Command { kDone, kGather, kTail, kExact };

// Index of the first element of the ascending array that is >= t (n if none), by one warp.
template <typename U>
__device__ __forceinline__ int warp_lower_bound(const U* v, int n, U t, int lane) {
  const int step = n / 32;
  const int seg = __popc(__ballot_sync(0xffffffffu, v[(lane + 1) * step - 1] < t));
  if (seg == 32) return n;
  return seg * step + __popc(__ballot_sync(0xffffffffu, lane < step && v[seg * step + lane] < t));
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

template <int N>
__device__ __forceinline__ float max_of(const float (&f)[N]) {
  float c = f[0];
#pragma unroll
  for (int i = 1; i < N; ++i) c = fmaxf(c, f[i]);
  return c;
}

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_min_r(float v) { return -warp_max_r(-v); }

__device__ __forceinline__ uint32_t sf_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Waits for the slice's copy; gives up after a while (false).
__device__ __forceinline__ bool sf_wait(u64* bar, uint32_t parity) {
  for (int i = 0; i < (1 << 20); ++i) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(sf_smem(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}

}  // namespace

template <typename T, int NT, int NB, int CAP, int GROUPS>
__global__ void __launch_bounds__(NT, 1024 / NT)
    k_sample_filtered(FilteredArgs a, int slice_chunks) {
  constexpr int EPC = Chunk<T>::N, NBT = NB / 2, NW = NT / 32;
  using Shared = SfShared<NT, NB, CAP>;
  extern __shared__ uint4 slice[];
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int cs = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const long long n_clusters = (long long)gridDim.x / cs, cid = (long long)blockIdx.x / cs;
  Shared* lead = cl.map_shared_rank(&sh, 0);
  // behind the slice: each warp's queue of its chunks that hold a logit >= x1, room for all of them
  const int walk = ((slice_chunks + NT - 1) / NT) * 32;
  uint16_t* queue = reinterpret_cast<uint16_t*>(slice + slice_chunks) + wid * walk;
  auto cta_sync = [&] {
    if (NT == 32)
      __syncwarp();
    else
      __syncthreads();
  };
  auto sync = [&] {
    if (NT == 32 || cs == 1)
      cta_sync();
    else
      cl.sync();
  };
  if (tid == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(sf_smem(&sh.full)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  sync();  // every CTA of the cluster runs before any writes into another's shared memory
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
  // One bulk copy of the row's slice, started when nobody reads the last one any more.
  auto start_copy = [&](long long n) {
    if (tid == 0 && n < a.n) {
      const Slice g = slice_of(n);
      const uint32_t bytes = (uint32_t)(g.q_hi - g.q_lo) * 16u;
      asm volatile("{\n.reg .b64 t;\nmbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n}" ::"r"(sf_smem(&sh.full)),
                   "r"(bytes)
                   : "memory");
      if (bytes)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                sf_smem(slice)),
            "l"(g.base + g.q_lo), "r"(bytes), "r"(sf_smem(&sh.full))
            : "memory");
    }
  };
  start_copy(cid);

  uint32_t parity = 0;
  for (long long n = cid; n < a.n; n += n_clusters, parity ^= 1u) {
    const Slice g = slice_of(n);
    const RowParams q = row_params(a, n);
    // the logits of chunk j; ids outside the row read as -inf
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
    if (!sf_wait(&sh.full, parity)) report(a.d_status, DS_DEV_ERR_TIMEOUT);

    // ---- max
    float mx = -kInf, mn = kInf;
    for (int j = g.q_lo + tid; j < g.q_hi; j += NT) {
      float f[EPC];
      values(j, f);
      mx = fmaxf(mx, max_of(f));
#pragma unroll
      for (int i = 0; i < EPC; ++i) mn = fminf(mn, f[i] > -3e37f ? f[i] : kInf);
    }
    float m, lo, cut;
    {
      float grp = mx;
#pragma unroll
      for (int o = 1; o < NT / GROUPS; o <<= 1) grp = fmaxf(grp, __shfl_xor_sync(0xffffffffu, grp, o));
      m = warp_max_r(mx);
      lo = warp_min_r(mn);
      cut = warp_min_r(grp);
      if (NW > 1) {
        if (lane == 0) {
          sh.fred[0][wid] = m;
          sh.fred[1][wid] = lo;
          sh.fred[2][wid] = cut;
        }
        cta_sync();
        if (cs == 1) {
          m = warp_max_r(sh.fred[0][lane % NW]);
          lo = warp_min_r(sh.fred[1][lane % NW]);
          cut = warp_min_r(sh.fred[2][lane % NW]);
        } else {
          if (wid == 0) {
            m = warp_max_r(sh.fred[0][lane % NW]);
            lo = warp_min_r(sh.fred[1][lane % NW]);
            cut = warp_min_r(sh.fred[2][lane % NW]);
            if (lane < cs) {
              Shared* peer = cl.map_shared_rank(&sh, lane);
              peer->part_max[rank] = m;
              peer->part_min[rank] = lo;
              peer->part_cut[rank] = cut;
            }
          }
          sync();
          m = warp_max_r(sh.part_max[lane % cs]);
          lo = warp_min_r(sh.part_min[lane % cs]);
          cut = warp_max_r(sh.part_cut[lane % cs]);
        }
      }
    }
    // No logit below x_low has a weight: w > 0 needs (x - m) r > -22.2, and the
    // rest is room for the rounding of x_low. Masks are told from logits by
    // their size, which needs a range that ends above them.
    const float lowest = (m - 24.f * q.tau) - fabsf(m) * 2.4e-7f;
    const float x_low = lowest > -3e37f ? fmaxf(fminf(lo, m), lowest) : fmaxf(lowest, -3.402823466e38f);
    const float x1 = fmaxf(cut, x_low);  // splits the rest
    const float sc1 = fminf((float)NBT / (m - x1), 3.402823466e38f);
    const float sc2 = fminf((float)(NB - NBT) / (x1 - x_low), 3.402823466e38f);
    auto bin_of = [&](float x) {  // for x_low <= x <= m
      return x >= x1 ? min(NBT - 1, __float2int_rz((m - x) * sc1))
                     : min(NB - 1, NBT + min(NB, __float2int_rz((x1 - x) * sc2)));
    };
    const bool finite = m > -kInf && m < kInf;
    const bool drawn = !q.bad && q.tau > 0.f && finite;
    const bool greedy = !q.bad && q.tau == 0.f && finite;
    // A top-k of at most GROUPS ends above x1: the mass below is then not asked for.
    const bool whole = drawn && !(q.k && q.k <= GROUPS);
    const bool floored = q.mp > 0.f;
    const uint32_t floor_i = (uint32_t)ceil((double)q.mp * (double)kSfOne);
    // one logit of chunk j
    auto value = [&](int j, int i) {
      const int e = EPC * j - g.dc + i;
      const float x = Logit<T>::load(reinterpret_cast<const T*>(slice) + (EPC * (j - g.q_lo) + i));
      return e >= 0 && e < a.V ? x : -kInf;
    };
    auto add_bins = [&](float x, uint32_t w) {
      if (w) {
        const int b = bin_of(x);
        atomicAdd(&sh.cnt[b], 1u);
        atomicAdd(&sh.lo[b], w & 0xffffu);
        if (w >> 16) atomicAdd(&sh.hi[b], w >> 16);
      }
    };

    // ---- weigh
    float s = 0.f;
    u64 total = 0, above_floor = 0;
    int first = INT_MAX, odd = 0;
    int queued = 0;
    for (int j0 = g.q_lo + wid * 32; j0 < g.q_hi; j0 += NT) {
      const int j = j0 + lane;
      float f[EPC];
      if (j < g.q_hi) {
        values(j, f);
      } else {
#pragma unroll
        for (int i = 0; i < EPC; ++i) f[i] = -kInf;
      }
      const float c = max_of(f);
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < EPC; ++i) part += ex2_approx((f[i] - m) * kLog2e);
      s += part;
      if (whole) {
#pragma unroll
        for (int i = 0; i < EPC; ++i) {
          const uint32_t w = sf_weight(f[i], m, q.r);
          total += w;
          if (floored) above_floor += w >= floor_i ? w : 0u;
        }
      }
      const unsigned high = __ballot_sync(0xffffffffu, drawn && c >= x1);
      if (drawn && c >= x1) queue[queued + __popc(high & ((1u << lane) - 1u))] = (uint16_t)(j - g.q_lo);
      queued += __popc(high);
      if (greedy && c == m) {
#pragma unroll
        for (int i = 0; i < EPC; ++i)
          if (f[i] == m) first = min(first, EPC * j - g.dc + i);
      }
      if (!finite) {
#pragma unroll
        for (int i = 0; i < EPC; ++i) odd |= !(f[i] < kInf);
      }
    }
    // The queued chunks, a logit per lane: in the walk itself a few lanes at a
    // time would weigh while the others wait.
    __syncwarp();
    // Four logits of the queued chunks per lane, -inf past their end.
    auto four_queued = [&](int i0, float (&x)[4], int (&j)[4]) {
#pragma unroll
      for (int u = 0; u < 4; ++u) j[u] = g.q_lo + queue[min(i0 + lane / EPC + u * (32 / EPC), queued - 1)];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        x[u] = value(j[u], lane % EPC);
        if (i0 + lane / EPC + u * (32 / EPC) >= queued) x[u] = -kInf;
      }
    };
    for (int i0 = 0; i0 < queued; i0 += 128 / EPC) {
      float x[4];
      int j[4];
      four_queued(i0, x, j);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (x[u] >= x1) {
          const uint32_t w = sf_weight(x[u], m, q.r);
          add_bins(x[u], w);
          if (!whole && floored) above_floor += w >= floor_i ? w : 0u;
        }
    }
    __syncwarp();
    // A NaN, or +inf under a finite maximum, makes the sum NaN.
    s = warp_sum(s);
    odd |= finite && !(s < kInf);
    odd = __any_sync(0xffffffffu, odd);
    if (whole) total = warp_sum_u64(total);
    if (floored) above_floor = warp_sum_u64(above_floor);
    if (greedy) {
      first = warp_min_i(first);
      if (lane == 0 && first != INT_MAX) atomicMin(&lead->first_id, first);
    }
    if (lane == 0) {
      sh.red[wid] = total;
      sh.red2[wid] = above_floor;
      sh.sred[0][wid] = s;
      sh.sred[1][wid] = __int_as_float(odd);
    }
    cta_sync();
    if (wid == 0) {
      const bool in = lane < NW;
      total = warp_sum_u64(in ? sh.red[lane] : 0);
      above_floor = warp_sum_u64(in ? sh.red2[lane] : 0);
      s = warp_sum(in ? sh.sred[0][lane] : 0.f);
      odd = __any_sync(0xffffffffu, in && __float_as_int(sh.sred[1][lane]));
      if (lane == 0) {
        lead->part_total[rank] = total;
        lead->part_floor[rank] = above_floor;
        lead->part_sum[rank] = s;
        lead->part_odd[rank] = odd;
      }
    }
    sync();

    if (!drawn) {
      start_copy(n + n_clusters);
      if (rank == 0 && tid == 0) {
        int bits = 0;
        float sum = 0.f;
        for (int o = 0; o < cs; ++o) {
          bits |= sh.part_odd[o];
          sum += sh.part_sum[o];
        }
        const bool ok = greedy && !bits;
        if (q.bad || bits) report(a.d_status, q.bad ? DS_DEV_ERR_PARAM : DS_DEV_ERR_LOGITS);
        a.out_tokens[n] = ok ? sh.first_id : -1;
        a.out_logprobs[n] = ok ? m - (m + logf(sum)) : __int_as_float(0x7fffffff);
      }
      continue;  // the partials are read before this CTA meets the others again
    }

    // Sums the cluster's bins [b0, b0 + NB / 2) into rank 0's pm and pc: a share
    // of the bins per CTA, a thread per bin and peer, so that the reads of other
    // CTAs' memory are one round trip.
    auto merge_bins = [&](int b0) {
      for (int i = tid; i < NBT; i += NT) {
        const int b = b0 + rank * (NBT / cs) + i / cs;
        const Shared* peer = cl.map_shared_rank(&sh, i % cs);
        uint32_t c = peer->cnt[b];
        u64 mass = (u64)peer->lo[b] + ((u64)peer->hi[b] << 16);
        for (int o = 1; o < cs; o <<= 1) {
          c += __shfl_xor_sync(0xffffffffu, c, o);
          mass += __shfl_xor_sync(0xffffffffu, mass, o);
        }
        if (i % cs == 0) {
          lead->pc[b] = c;
          lead->pm[b] = mass;
        }
      }
    };
    // Rank 0: running sums of those bins, continuing from (m0, c0). Alone in its
    // cluster, it takes them as they are.
    auto scan_bins = [&](int b0, u64 m0, uint32_t c0) {
      constexpr int PER = (NBT + NT - 1) / NT;
      u64 mass[PER], sm = 0;
      uint32_t c[PER], sc = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        mass[i] = 0;
        c[i] = 0;
        if (b < NBT) {
          mass[i] = cs == 1 ? (u64)sh.lo[b0 + b] + ((u64)sh.hi[b0 + b] << 16) : sh.pm[b0 + b];
          c[i] = cs == 1 ? sh.cnt[b0 + b] : sh.pc[b0 + b];
        }
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
      u64 bm = m0 + im - sm;
      uint32_t bc = c0 + ic - sc;
      if (NW > 1) {
        if (lane == 31) {
          sh.red[wid] = im;
          sh.fred[0][wid] = __uint_as_float(ic);
        }
        cta_sync();
#pragma unroll
        for (int w = 0; w < NW; ++w)
          if (w < wid) {
            bm += sh.red[w];
            bc += __float_as_uint(sh.fred[0][w]);
          }
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
      cta_sync();
    };
    // Rank 0, warp 0: which bins the boundaries can lie in (see the kernel's comment).
    auto decide = [&](bool tail) {
      const int nb = tail ? NB : NBT;
      const u64 known = sh.pm[nb - 1], all = sh.known_total, fl = sh.known_floor;
      const uint32_t count = sh.pc[nb - 1];
      const bool complete = tail || !whole || known == all;
      uint32_t mark = 0;  // lane l: bins [32 l, 32 l + 32)
      auto mark_range = [&](int b0, int b1) {
        const int from = max(b0 - 32 * lane, 0), to = min(b1 - 32 * lane, 31);
        if (lane < NB / 32 && from <= to) mark |= (0xffffffffu << from) & (0xffffffffu >> (31 - to));
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
        const u64 n_hi = need_of(q.p, t_hi), n_lo = t_lo == t_hi ? n_hi : need_of(q.p, t_lo);
        if (n_hi > known) return complete ? (int)kExact : (int)kTail;
        const int b0 = warp_lower_bound<u64>(sh.pm, nb, n_lo > 0 ? n_lo : 1, lane);
        const int b1 = n_lo == n_hi ? b0 : warp_lower_bound<u64>(sh.pm, nb, n_hi, lane);
        mark_range(b0, b1);
        t_lo = b0 ? sh.pm[b0 - 1] : 0;
        t_hi = sh.pm[b1];
      }
      if (floored) {
        t_lo = fl < t_lo ? fl : t_lo;
        t_hi = fl < t_hi ? fl : t_hi;
      }
      const u64 d_hi = target_of(q.u, t_hi), d_lo = t_lo == t_hi ? d_hi : target_of(q.u, t_lo);
      if (d_hi >= known) return complete ? (int)kExact : (int)kTail;
      const int b0 = warp_lower_bound<u64>(sh.pm, nb, d_lo + 1, lane);
      mark_range(b0, d_lo == d_hi ? b0 : warp_lower_bound<u64>(sh.pm, nb, d_hi + 1, lane));
      int listed = 0;
      for (uint32_t w = mark; w; w &= w - 1) {
        const int b = 32 * lane + __ffs(w) - 1;
        listed += (int)(sh.pc[b] - (b ? sh.pc[b - 1] : 0u));
      }
      if (warp_sum_i(listed) > CAP) return (int)kExact;
      if (lane < NB / 32) sh.marks[lane] = mark;
      const bool low = __any_sync(0xffffffffu, lane >= NBT / 32 && mark);
      if (lane == 0) {
        sh.kb = kb;
        sh.gate = low;
      }
      return (int)kGather;
    };

    if (cs > 1) merge_bins(0);
    if (rank == 0 && wid == 0) {
      if (cs > 1) {
        const bool in = lane < cs;
        total = warp_sum_u64(in ? sh.part_total[lane] : 0);
        above_floor = warp_sum_u64(in ? sh.part_floor[lane] : 0);
        s = warp_sum(in ? sh.part_sum[lane] : 0.f);
        odd = __any_sync(0xffffffffu, in && sh.part_odd[lane]);
      }
      if (lane == 0) {
        sh.known_total = total;
        sh.known_floor = above_floor;
        sh.known_sum = s;
        sh.known_odd = odd;
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
          for (int o = 1; o < cs; ++o) {
            Shared* peer = cl.map_shared_rank(&sh, o);
            if (lane < NB / 32) peer->marks[lane] = sh.marks[lane];
            if (lane == 0) {
              peer->gate = sh.gate;
              peer->command = c;
            }
          }
          if (lane == 0) sh.command = c;
        }
      }
      sync();
      command = sh.command;
      if (command != kTail) break;
      const int logits = (g.q_hi - g.q_lo) * EPC;
      for (int e0 = tid; e0 < logits; e0 += 4 * NT) {
        float x[4];
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = e0 + u * NT;
          x[u] = e < logits ? value(g.q_lo + e / EPC, e % EPC) : -kInf;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = sf_weight(x[u], m, q.r);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (x[u] >= x_low && x[u] < x1) add_bins(x[u], w[u]);
      }
      sync();
      if (cs > 1) {
        merge_bins(NBT);
        sync();
      }
    }
    if (command == kGather) {
      auto take = [&](float x, int j, int i) {
        const int b = bin_of(x);
        if (((sh.marks[b >> 5] >> (b & 31)) & 1u) && sf_weight(x, m, q.r)) {
          const int at = atomicAdd(&lead->n_list, 1);
          if (at < CAP)
            lead->list[at] = ((u64)Logit<T>::key(x) << 32) | (u64)(0xffffffffu - (uint32_t)(EPC * j - g.dc + i));
        }
      };
      if (!sh.gate) {
        for (int i0 = 0; i0 < queued; i0 += 128 / EPC) {
          float x[4];
          int j[4];
          four_queued(i0, x, j);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (x[u] >= x1) take(x[u], j[u], lane % EPC);
        }
      } else {
        const int logits = (g.q_hi - g.q_lo) * EPC;
        for (int e0 = tid; e0 < logits; e0 += 4 * NT) {
          float x[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int e = e0 + u * NT;
            x[u] = e < logits ? value(g.q_lo + e / EPC, e % EPC) : -kInf;
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int e = e0 + u * NT;
            if (x[u] >= x_low) take(x[u], g.q_lo + e / EPC, e % EPC);
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
      if (len <= 32) {
        if (wid == 0) {
          // bitonic sort in registers, descending
          u64 e = lane < len ? sh.list[lane] : 0;
#pragma unroll
          for (int size = 2; size <= 32; size *= 2)
#pragma unroll
            for (int d = size / 2; d > 0; d /= 2) {
              const u64 o = __shfl_xor_sync(0xffffffffu, e, d);
              const bool keep_max = ((lane & d) == 0) == ((lane & size) == 0);
              e = (e > o) == keep_max ? e : o;
            }
          if (lane < len) sh.list[lane] = e;
          __syncwarp();
        }
      } else {
        // each entry to the place that the number of larger ones gives; all differ
        for (int i = tid; i < len; i += NT) {
          const u64 e = sh.list[i];
          int place = 0;
#pragma unroll 8
          for (int o = 0; o < len; ++o) place += sh.list[o] > e;
          sh.incl[place] = e;
        }
        cta_sync();
        for (int i = tid; i < len; i += NT) sh.list[i] = sh.incl[i];
        cta_sync();
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
          return max(len - 1, 0);  // not reached: the boundary's bin is listed
        };
        u64 all;
        if (sh.kb >= 0)
          all = sh.pc[sh.kb] == (uint32_t)q.k ? sh.pm[sh.kb] : kept;
        else
          all = whole ? sh.known_total : sh.pm[NBT - 1];
        if (q.p < 1.f) all = sh.incl[first_at_least(need_of(q.p, all))];
        if (floored) all = sh.known_floor < all ? sh.known_floor : all;
        const int at = first_at_least(target_of(q.u, all) + 1);
        if (lane == 0) {
          const u64 e = sh.list[at];
          a.out_tokens[n] = (int)(0xffffffffu - (uint32_t)e);
          a.out_logprobs[n] = Logit<T>::value((uint32_t)(e >> 32)) - lse;
        }
      }
    }
    cta_sync();  // the lists are free
  }
  sync();  // no CTA leaves while a peer may still use its shared memory
}

namespace {

constexpr int kSfSmallV = 2048;   // rows up to here, when there are enough to fill the GPU: a warp each
constexpr int kSfMediumV = 8192;  // rows up to here: 128-thread CTAs
constexpr long long kSfSlice = 64 << 10;    // bytes of a row per CTA, two CTAs per SM
constexpr long long kSfSliceMax = 128 << 10;  // one CTA per SM; at most 65536 logits, which the bins' 32-bit sums allow
constexpr long long kSfSliceMin = 8 << 10;

// Launches the cluster kernel; *refused when no cluster of that shape fits.
template <typename T, int NT, int NB, int CAP, int GROUPS>
cudaError_t launch_on_chip(const FilteredArgs& a, int cs, int chunks, cudaStream_t st, bool* refused) {
  const size_t smem = (size_t)chunks * 16 + (size_t)((chunks + NT - 1) / NT * NT) * 2;  // a slice and its queues
  auto kern = k_sample_filtered<T, NT, NB, CAP, GROUPS>;
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
  // A CTA alone is launched without a cluster: as clusters of one, only eight of them run on an SM.
  if (cs == 1) attr[0] = attr[1];
  cfg.attrs = attr;
  cfg.numAttrs = cs == 1 ? 1 : 2;
  const void* site = reinterpret_cast<const void*>(kern);
  const int ok = cached(site, -1, [&](int) {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kSfSliceMax + kSfSliceMax / 8 + 2048));
    if (r == cudaSuccess) r = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (r != cudaSuccess) (void)cudaGetLastError();
    return r == cudaSuccess ? 1 : 0;
  });
  const int fit = ok <= 0 ? 0 : cached(site, (long long)smem * 32 + cs, [&](int) {
    int v = 0;
    const cudaError_t r = cs == 1 ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kern, NT, smem)
                                  : cudaOccupancyMaxActiveClusters(&v, kern, &cfg);
    if (r != cudaSuccess) {
      (void)cudaGetLastError();
      return 0;
    }
    return cs == 1 ? v * device_sms() : v;
  });
  if (fit < 1) {
    *refused = true;
    return cudaSuccess;
  }
  const long long clusters = a.n < fit ? a.n : fit;
  cfg.gridDim = dim3((unsigned)(clusters * cs));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, chunks);
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
  if (a.V <= kSfSmallV && a.n >= sms * 8LL) {
    const cudaError_t e = launch_on_chip<T, 32, 128, 128, 32>(a, 1, (int)((bytes + 15) / 16), st, &refused);
    if (!refused) return e;
  } else if (a.V <= kSfMediumV) {
    const cudaError_t e = launch_on_chip<T, 128, 256, 256, 32>(a, 1, (int)((bytes + 15) / 16), st, &refused);
    if (!refused) return e;
  } else {
    int cs = 1;
    while (cs < 16 && bytes > cs * kSfSlice) cs *= 2;
    // few rows: more CTAs per row, down to 8 KB each
    while (cs < 8 && (long long)a.n * cs * 2 <= sms && bytes > cs * 2 * kSfSliceMin) cs *= 2;
    const long long slice = (bytes / 16 + cs) / cs * 16 + 16;
    if (slice <= kSfSliceMax) {
      const cudaError_t e = launch_on_chip<T, 512, 1024, 1024, 128>(a, cs, (int)(slice / 16), st, &refused);
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
