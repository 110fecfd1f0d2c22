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

// 16 bytes of logits as fp32.
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
  static constexpr int N = 8;
  static constexpr uint32_t NEG_INF = 0xff80ff80u;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[8]) { unpack8(v, f); }
};
template <>
struct Chunk<float> {
  static constexpr int N = 4;
  static constexpr uint32_t NEG_INF = 0xff800000u;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
};

// A row as 16-byte chunks: chunk 0 starts at the row's first element rounded down
// to 16 bytes, so that loads stay inside the 16-byte blocks that hold the row.
template <typename T>
struct Row {
  static constexpr int EPC = Chunk<T>::N;
  const uint4* base;
  int dc, nq, V;  // elements before the row in chunk 0, chunks, length
  __device__ __forceinline__ Row(const T* row, int V_) : V(V_) {
    const uintptr_t ad = reinterpret_cast<uintptr_t>(row);
    base = reinterpret_cast<const uint4*>(ad & ~(uintptr_t)15);
    dc = (int)((ad & 15) / sizeof(T));
    nq = (dc + V + EPC - 1) / EPC;
  }
  __device__ __forceinline__ int id(int j, int i) const { return EPC * j - dc + i; }
  // the logits of chunk j; ids outside the row read as -inf
  __device__ __forceinline__ void values(const uint4& raw, int j, float (&f)[EPC]) const {
    Chunk<T>::get(raw, f);
    if (j == 0 || j == nq - 1) {
#pragma unroll
      for (int i = 0; i < EPC; ++i)
        if (id(j, i) < 0 || id(j, i) >= V) f[i] = -kInf;
    }
  }
  // Calls body(j, chunk) for the chunks of [from, to) that this lane has, U loads
  // at a time; all lanes of the warp together, with -inf past the end. BACK: from
  // the end.
  template <int NT, int U, bool BACK, typename Load, typename Body>
  __device__ __forceinline__ void walk(int from, int to, Load load, Body body) const {
    const int rounds = (to - from + U * NT - 1) / (U * NT);
#pragma unroll 1
    for (int it = 0; it < rounds; ++it) {
      const int j0 = from + (BACK ? rounds - 1 - it : it) * (U * NT) + (int)(threadIdx.x & ~31u);
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * NT + (int)(threadIdx.x & 31u);
        raw[u] = make_uint4(Chunk<T>::NEG_INF, Chunk<T>::NEG_INF, Chunk<T>::NEG_INF, Chunk<T>::NEG_INF);
        if (j < to) raw[u] = load(j);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) body(j0 + u * NT + (int)(threadIdx.x & 31u), raw[u]);
    }
  }
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

// The mass of a row's logits with weight >= floor_w.
template <typename T, int NT>
__device__ u64 row_mass(const Row<T>& row, uint32_t floor_w, float m, float r, u64* red) {
  u64 s = 0;
  row.template walk<NT, 2, false>(
      0, row.nq, [&](int j) { return __ldg(row.base + j); },
      [&](int j, const uint4& raw) {
        float f[Chunk<T>::N];
        row.values(raw, j, f);
#pragma unroll
        for (int i = 0; i < Chunk<T>::N; ++i) {
          const uint32_t w = sf_weight(f[i], m, r);
          s += w >= floor_w ? w : 0u;
        }
      });
  return block_sum<NT>(s, red);
}

// Where a running measure passes its target.
struct Cut {
  uint32_t key;
  u64 before;        // mass of the logits above `key`
  u64 count_before;  // and their number
  u64 each;          // weight of a logit at `key`
};

// Scratch of a search: counts, and masses as three sums of 11, 10 and 11 bits of
// the weights, which 2^21 logits cannot overflow.
template <int NB>
struct Bins {
  uint32_t *cnt, *w0, *w1, *w2;  // [NB]
  u64* red;                      // [NT / 32]
  u64* out;                      // [4]
};

// The first logit with a weight whose running count (by_count) or mass passes t,
// t below the row's: a radix search on the key, NB ways a pass. One CTA.
template <typename T, int NT, int NB>
__device__ __noinline__ Cut row_select(const Row<T> row, bool by_count, u64 t, float m, float r, const Bins<NB> b) {
  constexpr int NW = NT / 32, PER = NB / NT > 0 ? NB / NT : 1;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  uint32_t lo = Logit<T>::key(-kInf), hi = Logit<T>::key(m);
  u64 mass0 = 0, count0 = 0;  // of the logits above hi
  for (;;) {
    int s = 0;
    while (((hi - lo) >> s) >= (uint32_t)NB) ++s;
    __syncthreads();
    for (int i = tid; i < NB; i += NT) b.cnt[i] = b.w0[i] = b.w1[i] = b.w2[i] = 0;
    __syncthreads();
    row.template walk<NT, 2, false>(
        0, row.nq, [&](int j) { return __ldg(row.base + j); },
        [&](int j, const uint4& raw) {
          float f[Chunk<T>::N];
          row.values(raw, j, f);
#pragma unroll
          for (int i = 0; i < Chunk<T>::N; ++i) {
            const uint32_t key = Logit<T>::key(f[i]);
            const uint32_t w = sf_weight(f[i], m, r);
            const bool in = key >= lo && key <= hi && w;
            // a warp whose logits all fall on one bin adds them up first: ties are one thing this search is for
            const unsigned who = __ballot_sync(0xffffffffu, in);
            if (!who) continue;
            const int bin = in ? (int)((hi - key) >> s) : -1;
            const int first = __shfl_sync(0xffffffffu, bin, __ffs(who) - 1);
            if (__all_sync(0xffffffffu, !in || bin == first)) {
              const uint32_t a = __reduce_add_sync(0xffffffffu, in ? w & 0x7ffu : 0u);
              const uint32_t c = __reduce_add_sync(0xffffffffu, in ? w >> 11 & 0x3ffu : 0u);
              const uint32_t d = __reduce_add_sync(0xffffffffu, in ? w >> 21 : 0u);
              if (lane == 0) {
                atomicAdd(&b.cnt[first], (uint32_t)__popc(who));
                atomicAdd(&b.w0[first], a);
                atomicAdd(&b.w1[first], c);
                atomicAdd(&b.w2[first], d);
              }
            } else if (in) {
              atomicAdd(&b.cnt[bin], 1u);
              atomicAdd(&b.w0[bin], w & 0x7ffu);
              atomicAdd(&b.w1[bin], w >> 11 & 0x3ffu);
              atomicAdd(&b.w2[bin], w >> 21);
            }
          }
        });
    __syncthreads();
    // running sums; the thread that meets t writes what it found
    u64 sc = 0, sm = 0;
    for (int i = 0; i < PER; ++i) {
      const int k = tid * PER + i;
      if (k < NB) {
        sc += b.cnt[k];
        sm += (u64)b.w0[k] + ((u64)b.w1[k] << 11) + ((u64)b.w2[k] << 21);
      }
    }
    u64 ic = sc, im = sm;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 uc = __shfl_up_sync(0xffffffffu, ic, o), um = __shfl_up_sync(0xffffffffu, im, o);
      if (lane >= o) {
        ic += uc;
        im += um;
      }
    }
    u64 bc = count0 + ic - sc, bm = mass0 + im - sm;
    if (lane == 31) b.red[wid] = ic;
    __syncthreads();
    for (int w = 0; w < wid && w < NW; ++w) bc += b.red[w];
    __syncthreads();
    if (lane == 31) b.red[wid] = im;
    if (tid == 0) b.out[3] = 0;
    __syncthreads();
    for (int w = 0; w < wid && w < NW; ++w) bm += b.red[w];
    for (int i = 0; i < PER; ++i) {
      const int k = tid * PER + i;
      if (k >= NB) break;
      const u64 c = b.cnt[k], mass = (u64)b.w0[k] + ((u64)b.w1[k] << 11) + ((u64)b.w2[k] << 21);
      const u64 at = by_count ? bc : bm, step = by_count ? c : mass;
      if (at <= t && t < at + step) {
        b.out[0] = (u64)k;
        b.out[1] = bc;
        b.out[2] = bm;
        b.out[3] = 1;
      }
      bc += c;
      bm += mass;
    }
    __syncthreads();
    Cut c = {hi, mass0, count0, 1};
    if (!b.out[3]) return c;  // not reached: t is below the row's measure
    hi -= (uint32_t)b.out[0] << s;
    if (hi - lo > (1u << s) - 1u) lo = hi - ((1u << s) - 1u);
    count0 = b.out[1];
    mass0 = b.out[2];
    if (s == 0) {
      c.key = hi;
      c.before = mass0;
      c.count_before = count0;
      c.each = (u64)sf_weight(Logit<T>::value(hi), m, r);
      return c;
    }
  }
}

// Id of the j-th (from 0) logit with the given key, in id order. One CTA.
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

// A row's filter parameters, and what its kernels share of it.
struct RowParams {
  float tau, p, mp, u, r;
  int k;             // 0: no top-k
  uint32_t floor_w;  // min-p keeps the weights from here
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
  q.floor_w = (uint32_t)ceil((double)q.mp * (double)kSfOne);
  return q;
}

// The smallest integer mass at which top-p is met, and the draw's target.
__device__ __forceinline__ u64 need_of(float p, u64 total) { return (u64)ceil((double)p * (double)total); }
__device__ __forceinline__ u64 target_of(float u, u64 total) { return (u64)floor((double)u * (double)total); }

// Integers around f * total (0 <= f <= 1, total < 2^53): both functions above lie
// between them. FP64 runs at a sixty-fourth of FP32's rate, and where a boundary
// may lie is asked up to eight times a row.
__device__ __forceinline__ u64 fraction_low(float f, u64 total) {
  const u64 bits = (u64)(f * 4294967296.f);  // f has 24 bits: exact from 2^-8 on, less by under 2^-32 below
  const u64 x = bits >> 32 ? total : __umul64hi(total, bits << 32);
  return x > 2 ? x - 2 : 0;
}
__device__ __forceinline__ u64 fraction_high(float f, u64 total) {
  const u64 bits = (u64)(f * 4294967296.f) + 1;
  const u64 x = bits >> 32 ? total : __umul64hi(total, bits << 32);
  return x + 3 < total ? x + 3 : total;
}

// The row's token, each question by a search over the row, which one CTA re-reads
// some ten times. It assumes nothing of the row: it finishes those whose boundaries
// meet too many logits for the lists of the fast kernel, by ties or in a flat row.
template <typename T, int NT, int NB>
__device__ __noinline__ int row_exact(const T* p, int V, const RowParams& q, float m, const Bins<NB>& b, int* slot) {
  const Row<T> row(p, V);
  const float r = q.r;
  u64 total = row_mass<T, NT>(row, 0u, m, r, b.red);
  if (q.k) {
    // a top-k that reaches the logits without a weight leaves the mass as it is
    const Cut c = row_select<T, NT, NB>(row, true, (u64)q.k - 1, m, r, b);
    if (b.out[3]) total = c.before + ((u64)q.k - c.count_before) * c.each;
  }
  auto through = [&](const Cut& c, u64 t) { return c.before + ((t - c.before) / c.each + 1) * c.each; };
  if (q.p < 1.f) {
    // kept while the mass before is below p * total: through the first whose running mass reaches it
    const u64 need = need_of(q.p, total);
    if (need < total) total = through(row_select<T, NT, NB>(row, false, need - 1, m, r, b), need - 1);
  }
  if (q.mp > 0.f) {
    const u64 sum = row_mass<T, NT>(row, q.floor_w, m, r, b.red);
    total = sum < total ? sum : total;
  }
  const u64 t = target_of(q.u, total);
  const Cut c = row_select<T, NT, NB>(row, false, t, m, r, b);
  return row_nth<T, NT>(p, V, c.key, (t - c.before) / c.each, b.red, slot);
}

}  // namespace

// ---------------------------------------------------------------- the fast kernel
//
// A cluster of cs CTAs takes a row, a contiguous slice each, and answers the
// three questions from histograms over bins of x. A short row is held in shared
// memory (RESIDENT), the next one copied there while this one is answered.
//   max     m, the smallest logit that is no mask, and a cut x1: the least of
//           GROUPS groups' maxima, so that GROUPS logits at least are above it
//           and, of independent ones, about ln(GROUPS) times as many
//   weigh   sum exp(x - m), and (unless a small top-k makes it needless) the
//           tempered sum, both in fp32; and for the logits >= x1, the ones that
//           decide nearly every row, exact count and mass in bins linear in x
//   decide  the CTA of rank 0 sums up the bins and finds those where the top-k,
//           top-p, min-p and draw boundaries can lie, given what the tempered
//           sum says of the row's mass. If one lies below x1, the cut is lowered
//           and the bins are made again.
//   gather  the logits of those bins, a few dozen, come to rank 0, which sorts
//           them and answers exactly.
// The row's mass is used through "which logit does top_p T (or u T) fall on", so
// bounds on it nearly always do: a_i = ex2(fl(y log2 e)) on the weight's own
// y = fl(fl(x - m) r) is off by |y| 7.3e-8 <= 1.6e-6 for the rounding of the
// product, 2.4e-7 for ex2.approx and 1.2e-7 for expf, relatively (kSfSlack); the
// sum, a tree over 8 logits, a thread's chunks in turn and a tree over threads and
// CTAs, by 2^-24 for each of these steps (kSfRounding); and each weight's rounding
// to an integer by half a unit. Where the boundary's logits are too light for
// that, the cluster weighs the rest of the row exactly (kWeigh), and where it
// falls between two listed logits all the same, rank 0 does.
// A row whose boundary bins hold more than CAP logits is finished by row_exact, in
// one CTA: rows of ties, and flat rows, whose nucleus or draw reaches so far down
// that a bin of x there holds that many. Every other row's logit costs two ex2 and
// its share of two walks over the row; an exact weight and an atomic only above x1.
//
// Batches that fill the GPU take a warp (short rows) or a CTA (long ones) per row
// and leave the few rows that need more to a second launch (kFirst, kMarked): the
// first kernel then has none of that code, and a slow row holds nobody up. A long
// row's CTA reads it once (ONE_WALK): the cut and a reference for the sums come
// from a sixteenth of the row, and the logits that turn out high are read again
// singly. Splitting every row over a cluster instead took 203 us where this takes
// 80 (256 rows x 248320, top-p: each cluster barrier waits for the slowest CTA of
// a row's latency-bound steps); two walks per CTA 96 us, the second from HBM again
// because 256 rows do not fit L2.
//
// What bounds it: long rows HBM first, then the latency of the steps behind the
// walk (51 us for 256 x 248320 with a top-k, 19 of them at the copy rate); short
// rows instructions and their fetch (3100 per row of 1025 at 56% of the issue
// rate, 110 us for 15510 rows of 1025); single rows the barriers (9 us for 1025,
// 19 us for 248320). Flat rows row_exact, a CTA a row: 256 x 248320, top-p 0.9 of
// normal logits of spread 4, 3, 2, 1: 0.27, 1.1, 4.7, 6.3 ms (bf16), 0.29, 0.39, 4.2,
// 10.0 ms (fp32).
namespace {

template <int NT, int NB, int CAP, int QCAP, int CS>  // QCAP 0: no queue; CS: most CTAs of a cluster
struct SfShared {
  uint32_t cnt[NB], lo[NB], hi[NB];  // this CTA's bins: count, and mass as two sums of 16-bit halves
  u64 pm[NB];                        // rank 0: mass through each bin
  uint32_t pc[NB];                   // rank 0: count through each bin
  u64 list[CAP];                     // rank 0: gathered (key, ~id)
  u64 incl[CAP];                     // this CTA's gathered ones; rank 0: running mass through each listed one
  uint16_t queue[NT / 32][QCAP > 0 ? QCAP : 1];  // each warp's chunks that hold a logit >= x1, by their place in its walk
  u64 full;                          // the slice's copy is done
  u64 red[NT / 32];
  float fred[3][NT / 32], sred[2][NT / 32], groups[32];
  int ired[3][NT / 32];
  uint32_t marks[NB / 32];
  // each CTA's partials, pushed by it to everyone (max) or to rank 0 (weigh)
  float part_max[CS], part_min[CS], part_cut[CS], part_sum[CS];
  float part_tempered[CS];
  u64 part_total[CS];
  int part_odd[CS], part_floor[CS], part_below[CS];
  int gave_up;  // a warp's wait for the slice ran out
  int command, n_list, n_mine, mine_at, first_id;
  u64 t_lo, t_hi;  // bounds of the row's mass
  float known_sum;
  int known_odd, known_floor, known_below;
  int kb, again, crowded;
  float hint;  // a lower cut that the boundary most likely lies above
  u64 found[4];
  int slot;
};

// kOnce does every row. kFirst, a kernel of its own without the code for them,
// leaves the rows whose boundaries lie below the first cut, need the row's mass
// exactly or overflow a list marked; kMarked does those.
enum Pass { kOnce, kFirst, kMarked };

enum Command { kDone, kGather, kWeigh, kLower, kExact, kMark };

constexpr float kSfSlack = 2.2e-6f, kSfRounding = 6e-8f;

// Index of the first element of the ascending array that is >= t (n if none), by one warp.
template <typename U>
__device__ __forceinline__ int warp_lower_bound(const U* v, int n, U t, int lane) {
  const int step = n / 32;
  const int seg = __popc(__ballot_sync(0xffffffffu, v[(lane + 1) * step - 1] < t));
  if (seg == 32) return n;
  return seg * step + __popc(__ballot_sync(0xffffffffu, lane < step && v[seg * step + lane] < t));
}

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
__device__ __forceinline__ bool sf_wait(u64* bar, uint32_t parity, int tries = DS_WAIT_TRIES) {
  for (int i = 0; i <= tries; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier." DS_WAIT_TRY ".parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(sf_smem(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}

}  // namespace

template <typename T, int NT, int NB, int CAP, int GROUPS, int QCAP, int ECAP, bool RESIDENT, Pass PASS>
__global__ void __launch_bounds__(NT, NT == 32 ? 28 : NT == 128 ? 6 : 1024 / NT) k_sample_filtered(FilteredArgs a, int slice_chunks) {
  constexpr int EPC = Chunk<T>::N, NW = NT / 32, U = RESIDENT ? 1 : 4;
  constexpr bool ONE_WALK = PASS == kFirst && !RESIDENT;  // one CTA a row
  static_assert(!ONE_WALK || GROUPS == 32, "a warp picks among the groups' maxima");
  using Shared = SfShared<NT, NB, CAP, QCAP, RESIDENT || ONE_WALK ? 1 : 8>;
  extern __shared__ uint4 slice[];
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int cs = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const long long n_clusters = (long long)gridDim.x / cs, cid = (long long)blockIdx.x / cs;
  Shared* lead = cl.map_shared_rank(&sh, 0);
  uint16_t* queue = sh.queue[wid];
  // behind the slice: the logits >= x1 of each warp's walk, and their places in the row's chunks
  // (of a slice in shared memory the places alone, room for every logit of the walk)
  float* high_x = reinterpret_cast<float*>(slice + slice_chunks) + wid * 2 * ECAP;
  int* high_at = reinterpret_cast<int*>(high_x + ECAP);
  uint16_t* high_place =
      reinterpret_cast<uint16_t*>(slice + slice_chunks) + wid * ((slice_chunks + NT - 1) / NT * 32 * EPC);
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
  pdl_wait();
  pdl_release();
  // The first row from n on that this cluster has to do: 32 are looked at at a time.
  auto row_from = [&](long long n) {
    if constexpr (PASS == kMarked) {
      for (; n < a.n; n += 32 * n_clusters) {
        const long long i = n + lane * n_clusters;
        const unsigned marked = __ballot_sync(0xffffffffu, i < a.n && a.out_tokens[i] == kStreamMark);
        if (marked) return n + (__ffs(marked) - 1) * n_clusters;
      }
    }
    return n;
  };
  long long next = row_from(cid);
  if (PASS == kMarked && next >= a.n) return;  // nothing marked among this cluster's rows: all of its CTAs leave
  if (tid == 0) {
    sh.gave_up = 0;
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(sf_smem(&sh.full)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  sync();  // every CTA of the cluster runs before any writes into another's shared memory

  // This CTA's slice of a row: chunks [q_lo, q_hi).
  auto row_of = [&](long long n) { return Row<T>(static_cast<const T*>(a.x) + n * a.ld, a.V); };
  auto from_of = [&](const Row<T>& g, int r) { return (int)((long long)r * g.nq / cs); };
  // One bulk copy of the row's slice, started when nobody reads the last one any more.
  auto start_copy = [&](long long n) {
    if (RESIDENT && tid == 0 && n < a.n) {
      const Row<T> g = row_of(n);
      const int from = from_of(g, rank);
      const uint32_t bytes = (uint32_t)(from_of(g, rank + 1) - from) * 16u;
      asm volatile("{\n.reg .b64 t;\nmbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n}" ::"r"(sf_smem(&sh.full)),
                   "r"(bytes)
                   : "memory");
      if (bytes)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                sf_smem(slice)),
            "l"(g.base + from), "r"(bytes), "r"(sf_smem(&sh.full))
            : "memory");
    }
  };
  start_copy(next);

  uint32_t parity = 0;
  for (long long n; (n = next) < a.n; parity ^= 1u) {
    next = row_from(n + n_clusters);
    const Row<T> g = row_of(n);
    const int q_lo = from_of(g, rank), q_hi = from_of(g, rank + 1);
    const RowParams q = row_params(a, n);
    auto load = [&](int j) { return RESIDENT ? slice[j - q_lo] : __ldg(g.base + j); };
    auto walk = [&](auto body) { g.template walk<NT, U, false>(q_lo, q_hi, load, body); };
    // The second walk goes back: of a batch of rows larger than L2, what was read last is still there.
    auto walk_back = [&](auto body) { g.template walk<NT, U, !RESIDENT>(q_lo, q_hi, load, body); };
    for (int i = tid; i < NB; i += NT) sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
    if (tid == 0) {
      sh.n_list = sh.n_mine = 0;
      sh.first_id = INT_MAX;
      sh.crowded = 0;
    }
    bool gave_up = RESIDENT && !sf_wait(&sh.full, parity);

    // ---- the sums of a chunk and its largest logit, relative to `ref`
    float s = 0.f, st = 0.f;
    const float2 l2e = make_float2(kLog2e, kLog2e), rr = make_float2(q.r, q.r);
    auto sum_chunk = [&](const float (&f)[EPC], float ref, bool also_tempered) {
      const float2 neg = make_float2(-ref, -ref);
      float2 d[EPC / 2], e[EPC / 2];
#pragma unroll
      for (int i = 0; i < EPC / 2; ++i) d[i] = __fadd2_rn(make_float2(f[2 * i], f[2 * i + 1]), neg);
      auto sum_of_ex2 = [&]() {
#pragma unroll
        for (int i = 0; i < EPC / 2; ++i) {
          e[i] = __fmul2_rn(e[i], l2e);
          e[i] = make_float2(ex2_approx(e[i].x), ex2_approx(e[i].y));
        }
#pragma unroll
        for (int o = 1; o < EPC / 2; o *= 2)
#pragma unroll
          for (int i = 0; i + o < EPC / 2; i += 2 * o) e[i] = __fadd2_rn(e[i], e[i + o]);
        return e[0].x + e[0].y;
      };
#pragma unroll
      for (int i = 0; i < EPC / 2; ++i) e[i] = d[i];
      s += sum_of_ex2();
      if (also_tempered) {
#pragma unroll
        for (int i = 0; i < EPC / 2; ++i) e[i] = __fmul2_rn(d[i], rr);
        st += sum_of_ex2();
      }
    };

    // ---- the logits above the cut
    float x1 = 0.f;
    int queued = 0;
    int have = 0;  // logits >= x1 of this warp's walk; more than fit: the walk itself is repeated for them
    // ONE_WALK: a warp has 32-chunk blocks in a row, from this chunk on
    const int warp_from = q_lo + (int)((long long)wid * ((q_hi - q_lo + 31) / 32) / NW) * 32;
    const int warp_to = min(q_hi, q_lo + (int)((long long)(wid + 1) * ((q_hi - q_lo + 31) / 32) / NW) * 32);
    auto keep = [&](bool high, float x, int at) {
      const unsigned who = __ballot_sync(0xffffffffu, high);
      const int slot = have + __popc(who & ((1u << lane) - 1u));
      if (RESIDENT) {
        if (high) high_place[slot] = (uint16_t)(at - EPC * q_lo);
      } else if (high && slot < ECAP) {
        high_x[slot] = x;
        high_at[slot] = at;
      }
      have += __popc(who);
    };
    auto kept_place = [&](int i) { return RESIDENT ? EPC * q_lo + (int)high_place[i] : high_at[i]; };
    auto kept_value = [&](int i) {
      return RESIDENT ? Logit<T>::load(reinterpret_cast<const T*>(slice) + high_place[i]) : high_x[i];
    };
    // Of a short row every logit is looked at in the walk; of a long one, chunks
    // with a high logit are queued, so that the walk pays a ballot a chunk.
    auto collect = [&](int j, const float (&f)[EPC], bool high) {
      const unsigned who = __ballot_sync(0xffffffffu, high);
      if (RESIDENT) {
        if (who) {
#pragma unroll
          for (int i = 0; i < EPC; ++i) keep(high && f[i] >= x1, f[i], EPC * j + i);
        }
      } else {
        const int at = queued + __popc(who & ((1u << lane) - 1u));
        if (high && at < QCAP) queue[at] = (uint16_t)(ONE_WALK ? j - warp_from : (j - q_lo) / NT * 32 + lane);
        queued += __popc(who);
      }
    };
    auto collect_queued = [&] {
      __syncwarp();
      if (RESIDENT) return;
      have = queued <= QCAP ? 0 : ECAP + 1;
      if (have) return;
      constexpr int B = 4;  // loads in flight
      for (int i0 = 0; i0 < queued; i0 += 32 * B / EPC) {
        float x[B];
        int at[B];
#pragma unroll
        for (int u = 0; u < B; ++u) {
          const int k = queue[min(i0 + lane / EPC + u * (32 / EPC), queued - 1)];
          at[u] = EPC * (ONE_WALK ? warp_from + k : q_lo + wid * 32 + k / 32 * NT + k % 32) + lane % EPC;
          x[u] = Logit<T>::get(reinterpret_cast<const T*>(g.base), at[u]);
        }
#pragma unroll
        for (int u = 0; u < B; ++u) {
          const int id = at[u] - g.dc;
          keep(x[u] >= x1 && i0 + lane / EPC + u * (32 / EPC) < queued && id >= 0 && id < a.V, x[u], at[u]);
        }
      }
      __syncwarp();
    };

    // ---- max (ONE_WALK: of a sample, the first blocks of every warp's share)
    float mx = -kInf, mn = kInf;
    uint4 sample[ONE_WALK ? U : 1];
    if constexpr (ONE_WALK) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = warp_from + 32 * u + lane;
        sample[u] = make_uint4(Chunk<T>::NEG_INF, Chunk<T>::NEG_INF, Chunk<T>::NEG_INF, Chunk<T>::NEG_INF);
        if (j < warp_to) sample[u] = load(j);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[EPC];
        g.values(sample[u], warp_from + 32 * u + lane, f);
        mx = fmaxf(mx, max_of(f));
      }
    } else {
      walk([&](int j, const uint4& raw) {
        float f[EPC];
        g.values(raw, j, f);
        mx = fmaxf(mx, max_of(f));
#pragma unroll
        for (int i = 0; i < EPC; ++i) mn = fminf(mn, f[i] > -3e37f ? f[i] : kInf);
      });
    }
    float m, lo, cut, grp;
    {
      grp = mx;
#pragma unroll
      for (int o = 1; o < NT / GROUPS; o <<= 1) grp = fmaxf(grp, __shfl_xor_sync(0xffffffffu, grp, o));
      m = warp_max_r(mx);
      lo = warp_min_r(mn);
      cut = warp_min_r(grp);
      if (RESIDENT) {
        gave_up = __any_sync(0xffffffffu, gave_up);
        if (NW > 1 && gave_up && lane == 0) sh.gave_up = 1;
      }
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
    if (RESIDENT && (NW > 1 ? sh.gave_up : (int)gave_up)) {
      // The copy of this row never came: neither it nor this CTA's further rows are
      // answered. A later launch has nothing to do for them.
      if (tid == 0) {
        report(a.d_status, DS_DEV_ERR_TIMEOUT);
        (void)sf_wait(&sh.full, parity, kDrainTries);  // not while it is still to be written
      }
      for (long long i = n; i < a.n; i = row_from(i + n_clusters)) {
        if (tid == 0) {
          a.out_tokens[i] = -1;
          a.out_logprobs[i] = __int_as_float(0x7fffffff);
        }
      }
      break;
    }
    // ---- ONE_WALK: the sums relative to the sample's maximum, the queue, and the maximum itself
    const float ref = m;
    if constexpr (ONE_WALK) {
      // The cut is the third least of the groups' maxima: the least scatters so much
      // that one row in sixty had more logits above it than the lists hold.
      if (lane % (NT / GROUPS) == 0) sh.groups[tid / (NT / GROUPS)] = grp;
      cta_sync();
      float v = sh.groups[lane];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        cut = warp_min_r(v);
        if (__ffs(__ballot_sync(0xffffffffu, v == cut)) - 1 == lane) v = kInf;
      }
      // Where the sample is much of the row, few logits of it lie above its cut.
      x1 = cut > -kInf && 4 * 32 * U * NW > q_hi - q_lo ? cut - 0.27f * (m - cut) : cut;
      cut = x1;
      const bool may_temper = q.r != 1.f && !(q.k && q.k <= 8 * GROUPS);
      auto body = [&](int j, const uint4& raw) {
        float f[EPC];
        g.values(raw, j, f);
        const float c = max_of(f);
        mx = fmaxf(mx, c);
        sum_chunk(f, ref, may_temper);
        collect(j, f, c >= x1 && c > -kInf);
      };
#pragma unroll
      for (int u = 0; u < U; ++u) body(warp_from + 32 * u + lane, sample[u]);
#pragma unroll 1
      for (int j0 = warp_from + 32 * U; j0 < warp_to; j0 += 32 * U) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + 32 * u + lane;
          raw[u] = make_uint4(Chunk<T>::NEG_INF, Chunk<T>::NEG_INF, Chunk<T>::NEG_INF, Chunk<T>::NEG_INF);
          if (j < warp_to) raw[u] = load(j);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) body(j0 + 32 * u + lane, raw[u]);
      }
      m = warp_max_r(mx);
      cta_sync();  // the sample's maxima are read
      if (lane == 0) sh.fred[0][wid] = m;
      cta_sync();
      m = warp_max_r(sh.fred[0][lane % NW]);
      lo = -3.402823466e38f;  // not looked for: a row that needs it goes to the second pass
    }
    // No logit below x_low has a weight: w > 0 needs (x - m) r > -22.2, and the
    // rest is room for the rounding of x_low. Masks are told from logits by
    // their size, which needs a range that ends above them.
    const float lowest = (m - 24.f * q.tau) - fabsf(m) * 2.4e-7f;
    const float x_low = lowest > -3e37f ? fmaxf(fminf(lo, m), lowest) : fmaxf(lowest, -3.402823466e38f);
    // The first cut; none for a short row of the second pass.
    // A warp's own row starts a little lower, and lower still for a top-k that
    // would end below (15510 x 1025, 12% of the rows with k = 200: 148 -> 129 us).
    // These shares, like the other steps of the cut, were fitted to normal logits of
    // spread 3 and 4. They decide how many walks a row takes, never its answer.
    const float further = PASS == kMarked ? (RESIDENT ? 1e30f : 0.f) : NT == 32 ? (q.k > 64 ? .35f : .15f) : 0.f;
    // Without a cut (in each CTA a group without a logit) all of the row is above it.
    x1 = ONE_WALK || !(cut > -kInf) ? cut : cut - further * (m - cut);
    if (PASS == kMarked && !RESIDENT) x1 = fminf(x1, a.out_logprobs[n]);  // the first pass's hint, +inf for none
    x1 = fmaxf(x1, x_low);  // never above m: the bins hold the maximum at least
    float per_x = fminf((float)NB / (m - x1), 3.402823466e38f);
    auto bin_of = [&](float x) { return min(NB - 1, __float2int_rz((m - x) * per_x)); };  // for x1 <= x <= m
    const bool finite = m > -kInf && m < kInf;
    const bool drawn = !q.bad && q.tau > 0.f && finite;
    const bool greedy = !q.bad && q.tau == 0.f && finite;
    // A top-k of at most GROUPS ends above x1: the mass below is then not asked
    // for. A longer one most likely does: its row is left to the second pass if not.
    const bool sure = q.k && q.k <= (ONE_WALK ? GROUPS - 2 : GROUPS);
    const bool whole = drawn && !(q.k && q.k <= (ONE_WALK ? 8 * GROUPS : GROUPS));
    // A row of the second pass is weighed exactly at once: bounds did not do, or will not that far down.
    const bool exact = PASS == kMarked && whole && x1 > x_low;
    const bool tempered = PASS != kMarked && whole && (ONE_WALK || x1 > x_low) && q.r != 1.f;
    u64 mass = 0;
    const bool floored = q.mp > 0.f;
    auto add_bins = [&](float x, uint32_t w) {
      if (w) {
        const int b = bin_of(x);
        atomicAdd(&sh.cnt[b], 1u);
        atomicAdd(&sh.lo[b], w & 0xffffu);
        if (w >> 16) atomicAdd(&sh.hi[b], w >> 16);
      }
    };

    // ---- weigh
    int first = INT_MAX, odd = 0;
    if constexpr (!ONE_WALK) {
      walk_back([&](int j, const uint4& raw) {
        float f[EPC];
        g.values(raw, j, f);
        const float c = max_of(f);
        sum_chunk(f, ref, tempered);
        if (exact) {
#pragma unroll
          for (int i = 0; i < EPC; ++i) mass += sf_weight(f[i], m, q.r);
        }
        collect(j, f, drawn && c >= x1);
        if (greedy && c == m) {
#pragma unroll
          for (int i = 0; i < EPC; ++i)
            if (f[i] == m) first = min(first, g.id(j, i));
        }
        if (!finite) {
#pragma unroll
          for (int i = 0; i < EPC; ++i) odd |= !(f[i] < kInf);
        }
      });
    } else {
      odd = m == kInf;
    }
    // min-p: the last bin with a logit that stays, and whether one above x1 does not
    int floor_bin = -1, below = 0;
    auto bin_high = [&] {
      collect_queued();
      floor_bin = -1;
      below = 0;
      auto add = [&](float x, uint32_t w) {
        if (x >= x1) {
          add_bins(x, w);
          if (floored) {
            if (w >= q.floor_w)
              floor_bin = max(floor_bin, bin_of(x));
            else
              below = 1;
          }
        }
      };
      if (RESIDENT || have <= ECAP) {
        for (int i = lane; i < have; i += 32) add(kept_value(i), sf_weight(kept_value(i), m, q.r));
      } else if constexpr (PASS == kFirst) {
        if (lane == 0) lead->crowded = 1;
      } else {
        walk([&](int j, const uint4& raw) {
          float f[EPC];
          uint32_t w[EPC];
          g.values(raw, j, f);
#pragma unroll
          for (int i = 0; i < EPC; ++i) w[i] = sf_weight(f[i], m, q.r);
#pragma unroll
          for (int i = 0; i < EPC; ++i) add(f[i], w[i]);
        });
      }
      __syncwarp();
      if (floored) {
        floor_bin = __reduce_max_sync(0xffffffffu, floor_bin);
        below = __any_sync(0xffffffffu, below);
      }
      if (lane == 0) {
        sh.ired[1][wid] = floor_bin;
        sh.ired[2][wid] = below;
      }
    };
    if (!ONE_WALK || drawn) {
      bin_high();
    } else {
      collect_queued();
      if (greedy) {
        if (have > ECAP && lane == 0) sh.crowded = 1;
        for (int i = lane; i < min(have, ECAP); i += 32)
          if (high_x[i] == m) first = min(first, high_at[i] - g.dc);
      }
    }
    // A NaN, or +inf under a finite maximum, makes the sum NaN.
    s = warp_sum(s);
    odd |= finite && !(s < kInf);
    if (tempered) st = warp_sum(st);
    // What one walk cannot settle: a sample without a logit, a maximum so far
    // above the sample's that the sums overflow.
    if (ONE_WALK && lane == 0 && (!(ref > -kInf) || s == kInf || (tempered && !(st < kInf)))) sh.crowded = 1;
    odd = __any_sync(0xffffffffu, odd);
    if (greedy) {
      first = warp_min_i(first);
      if (lane == 0 && first != INT_MAX) atomicMin(&lead->first_id, first);
    }
    // this CTA's share of what rank 0 needs to know, pushed there
    auto push_bins_info = [&] {
      if (NW > 1) {
        floor_bin = __reduce_max_sync(0xffffffffu, lane < NW ? sh.ired[1][lane] : -1);
        below = __any_sync(0xffffffffu, lane < NW && sh.ired[2][lane]);
      }
      if (lane == 0) {
        lead->part_floor[rank] = floor_bin;
        lead->part_below[rank] = below;
      }
    };
    if (exact) mass = warp_sum_u64(mass);
    if (NW > 1) {
      if (lane == 0) {
        sh.sred[0][wid] = s;
        sh.sred[1][wid] = st;
        sh.ired[0][wid] = odd;
        if (PASS == kMarked) sh.red[wid] = mass;
      }
      cta_sync();
    }
    if (wid == 0) {
      if (NW > 1) {
        const bool in = lane < NW;
        s = warp_sum(in ? sh.sred[0][lane] : 0.f);
        st = warp_sum(in ? sh.sred[1][lane] : 0.f);
        odd = __any_sync(0xffffffffu, in && sh.ired[0][lane]);
        if (exact) mass = warp_sum_u64(in ? sh.red[lane] : 0);
        if (ONE_WALK && lane == 0 && (s == kInf || (tempered && !(st < kInf)))) sh.crowded = 1;
      }
      if (lane == 0) {
        if (PASS == kMarked) lead->part_total[rank] = mass;
        lead->part_sum[rank] = s;
        lead->part_tempered[rank] = st;
        lead->part_odd[rank] = odd;
      }
      push_bins_info();
    }
    sync();

    if (!drawn) {
      start_copy(next);
      if (rank == 0 && tid == 0) {
        int bits = 0;
        float sum = 0.f;
        for (int o = 0; o < cs; ++o) {
          bits |= sh.part_odd[o];
          sum += sh.part_sum[o];
        }
        const bool ok = greedy && !bits;
        if (ONE_WALK && !q.bad && sh.crowded) {
          a.out_tokens[n] = kStreamMark;
          a.out_logprobs[n] = kInf;
        } else {
          if (q.bad || bits) report(a.d_status, q.bad ? DS_DEV_ERR_PARAM : DS_DEV_ERR_LOGITS);
          a.out_tokens[n] = ok ? sh.first_id : -1;
          a.out_logprobs[n] = ok ? m - (ref + logf(sum)) : __int_as_float(0x7fffffff);
        }
      }
      continue;  // the partials are read before this CTA meets the others again
    }

    // Sums the cluster's bins into rank 0's pm and pc: a share of the bins per CTA,
    // a thread per bin and peer, so that the reads of other CTAs' memory are one
    // round trip. A CTA's bin of more than 2^16 logits may have overflowed.
    auto merge_bins = [&] {
      for (int i = tid; i < NB; i += NT) {
        const int b = rank * (NB / cs) + i / cs;
        const Shared* peer = cl.map_shared_rank(&sh, i % cs);
        uint32_t c = peer->cnt[b];
        u64 mass = (u64)peer->lo[b] + ((u64)peer->hi[b] << 16);
        if (c > 65536u) lead->crowded = 1;
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
    // Rank 0: running sums of the bins. Alone in its cluster, it takes them as they are.
    auto scan_bins = [&] {
      constexpr int PER = (NB + NT - 1) / NT;
      u64 mass[PER], sm = 0;
      uint32_t c[PER], sc = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        mass[i] = 0;
        c[i] = 0;
        if (b < NB) {
          mass[i] = cs == 1 ? (u64)sh.lo[b] + ((u64)sh.hi[b] << 16) : sh.pm[b];
          c[i] = cs == 1 ? sh.cnt[b] : sh.pc[b];
          if (cs == 1 && c[i] > 65536u) sh.crowded = 1;
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
      u64 bm = im - sm;
      uint32_t bc = ic - sc;
      if (NW > 1) {
        if (lane == 31) {
          sh.red[wid] = im;
          sh.fred[0][wid] = __uint_as_float(ic);
        }
        cta_sync();
        const u64 wm = lane < wid ? sh.red[lane] : 0;
        const uint32_t wc = lane < wid ? __float_as_uint(sh.fred[0][lane]) : 0u;
        bm += warp_sum_u64(wm);
        bc += __reduce_add_sync(0xffffffffu, wc);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        bm += mass[i];
        bc += c[i];
        if (b < NB) {
          sh.pm[b] = bm;
          sh.pc[b] = bc;
        }
      }
      cta_sync();
    };
    // Rank 0, warp 0: which bins the boundaries can lie in (see the kernel's comment).
    // `weighed`: t_lo = t_hi is the row's mass.
    auto decide = [&](bool weighed) {
      const int nb = NB;
      const u64 known = sh.pm[nb - 1];
      const uint32_t count = sh.pc[nb - 1];
      const bool complete = sure || x1 <= x_low;  // nothing that is asked for lies below x1
      if (PASS == kFirst && lane == 0) sh.hint = kInf;  // none
      if (sh.crowded || !known) return (int)kExact;  // a search among empty bins would end behind the last
      uint32_t mark = 0;  // lane l: bins [32 l, 32 l + 32)
      auto mark_range = [&](int b0, int b1) {
        const int from = max(b0 - 32 * lane, 0), to = min(b1 - 32 * lane, 31);
        if (lane < NB / 32 && from <= to) mark |= (0xffffffffu << from) & (0xffffffffu >> (31 - to));
      };
      // a width that the logits of the bin are too light for
      auto light = [&](int b, u64 width) {
        const u64 mass = sh.pm[b] - (b ? sh.pm[b - 1] : 0);
        const uint32_t c = sh.pc[b] - (b ? sh.pc[b - 1] : 0u);
        return width > 0 && width * 4 * c > mass;
      };
      if (complete) {
        if (lane == 0) sh.t_lo = sh.t_hi = known;
        weighed = true;
        __syncwarp();
      }
      // Goes on below x1: with what mass missing, by the fall of the mass from one
      // quarter of the bins to the next.
      auto lower = [&](u64 target) {
        if (PASS == kFirst && !RESIDENT) {
          const float q3 = (float)(sh.pm[NB * 3 / 4 - 1] - sh.pm[NB / 2 - 1]), q4 = (float)(known - sh.pm[NB * 3 / 4 - 1]);
          const float fall = fminf(q4 / q3, 0.98f);
          float missing = 1.2f * (float)(target - known), step = q4;
          int quarters = 1;
          for (; quarters < 24 && missing > 0.f; ++quarters) {
            step *= fall;
            missing -= step;
          }
          if (lane == 0) sh.hint = missing > 0.f ? -kInf : x1 - 0.25f * (float)quarters * (m - x1);
        }
        return (int)kLower;
      };
      u64 t_lo = sh.t_lo, t_hi = sh.t_hi;  // bounds of the kept mass
      bool loose = !weighed;               // they differ by what is not known of the row's mass
      int kb = -1;
      if (q.k && (uint32_t)q.k <= count) {
        kb = warp_lower_bound<uint32_t>(sh.pc, nb, (uint32_t)q.k, lane);
        t_lo = t_hi = sh.pm[kb];
        loose = false;
        if (sh.pc[kb] != (uint32_t)q.k) {
          t_lo = kb ? sh.pm[kb - 1] : 0;
          mark_range(kb, kb);
        }
      } else if (q.k && !complete) {
        return (int)kLower;
      }
      if (q.p < 1.f) {
        const u64 n_hi = fraction_high(q.p, t_hi), n_lo = fraction_low(q.p, t_lo);
        if (n_hi > known) return complete ? (int)kExact : lower(n_hi);
        const int b0 = warp_lower_bound<u64>(sh.pm, nb, n_lo > 0 ? n_lo : 1, lane);
        const int b1 = n_hi <= sh.pm[b0] ? b0 : warp_lower_bound<u64>(sh.pm, nb, n_hi, lane);
        if (loose && light(b1, n_hi - n_lo)) return (int)kWeigh;
        loose = false;
        mark_range(b0, b1);
        t_lo = b0 ? sh.pm[b0 - 1] : 0;
        t_hi = sh.pm[b1];
      }
      if (floored) {
        // the mass of what min-p keeps ends in floor_bin, or beyond what is known
        const int fb = sh.known_floor;
        const bool ends = complete || sh.known_below;
        const u64 f_lo = !ends ? known : fb > 0 ? sh.pm[fb - 1] : 0, f_hi = ends ? sh.pm[max(fb, 0)] : t_hi;
        if (f_lo < t_hi) {
          if (!ends) return (int)kLower;
          mark_range(fb, fb);
          if (f_hi <= t_lo) loose = false;
          t_lo = f_lo < t_lo ? f_lo : t_lo;
          t_hi = f_hi < t_hi ? f_hi : t_hi;
        }
      }
      // the draw's target is below the kept mass
      u64 d_hi = fraction_high(q.u, t_hi), d_lo = fraction_low(q.u, t_lo);
      if (d_hi >= t_hi && t_hi) d_hi = t_hi - 1;
      if (d_lo > d_hi) d_lo = d_hi;
      if (d_hi >= known) return complete ? (int)kExact : lower(d_hi + 1);
      const int b0 = warp_lower_bound<u64>(sh.pm, nb, d_lo + 1, lane);
      const int b1 = d_hi < sh.pm[b0] ? b0 : warp_lower_bound<u64>(sh.pm, nb, d_hi + 1, lane);
      if (loose && light(b1, d_hi - d_lo)) return (int)kWeigh;
      mark_range(b0, b1);
      int listed = 0;
      for (uint32_t w = mark; w; w &= w - 1) {
        const int b = 32 * lane + __ffs(w) - 1;
        listed += (int)(sh.pc[b] - (b ? sh.pc[b - 1] : 0u));
      }
      if (warp_sum_i(listed) > CAP) return (int)kExact;
      if (lane < NB / 32) sh.marks[lane] = mark;
      if (lane == 0) sh.kb = kb;
      return (int)kGather;
    };

    if (cs > 1) merge_bins();
    if (rank == 0 && wid == 0) {
      if (cs > 1) {
        const bool in = lane < cs;
        s = warp_sum(in ? sh.part_sum[lane] : 0.f);
        st = warp_sum(in ? sh.part_tempered[lane] : 0.f);
        odd = __any_sync(0xffffffffu, in && sh.part_odd[lane]);
        if (exact) mass = warp_sum_u64(in ? sh.part_total[lane] : 0);
      }
      if (lane == 0) {
        float t = (tempered ? st : s) * kSfOne, rel = kSfSlack;
        if (ONE_WALK) {
          // The exponents are taken from ref, the sample's maximum: three roundings of (x - ref) r beside two of
          // (x - m) r, both 15 at most in the mean (ln V), (m - ref) r further off here; and the factor's own.
          const float off = (m - ref) * q.r;
          t *= expf(-off);
          rel += kSfRounding * (2.f * 15.f + 3.f * (15.f + off) + off + 4.f);
        }
        rel += kSfRounding * (float)(25 + (q_hi - q_lo + NT - 1) / NT);
        const u64 mid = (u64)t, slack = (u64)(t * rel) + (u64)(a.V / 2) + 2;
        sh.t_lo = mid > slack ? mid - slack : 0;
        sh.t_hi = mid + slack;
        if (exact) sh.t_lo = sh.t_hi = mass;
        sh.known_sum = s;
        sh.known_odd = odd;
      }
    }
    sync();
    int command;
    bool weighed = exact, fresh = true;
    for (int lowered = 0;;) {
      if (rank == 0) {
        if (fresh) scan_bins();
        if (wid == 0) {
          const int fb = __reduce_max_sync(0xffffffffu, lane < cs ? sh.part_floor[lane] : -1);
          const bool be = __any_sync(0xffffffffu, lane < cs && sh.part_below[lane]);
          if (lane == 0) {
            sh.known_floor = fb;
            sh.known_below = be;
          }
          __syncwarp();
          int c = sh.known_odd && !(ONE_WALK && sh.crowded) ? (int)kDone : decide(weighed);
          if (PASS == kFirst && c != kDone && c != kGather) c = kMark;
          __syncwarp();
          for (int o = 1; o < cs; ++o) {
            Shared* peer = cl.map_shared_rank(&sh, o);
            if (lane < NB / 32) peer->marks[lane] = sh.marks[lane];
            if (lane == 0) peer->command = c;
          }
          if (lane == 0) sh.command = c;
        }
      }
      sync();
      command = sh.command;
      if (PASS == kFirst || (command != kLower && command != kWeigh)) break;
      if (command == kLower) {
        // A lower cut: a quarter further from the maximum each time, which in the
        // tail of normal logits holds some four times as many, and at last all.
        x1 = lowered < 4 ? fmaxf(x_low, x1 - 0.27f * (m - x1)) : x_low;
        ++lowered;
        per_x = fminf((float)NB / (m - x1), 3.402823466e38f);
        for (int i = tid; i < NB; i += NT) sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
        cta_sync();
        queued = have = 0;
        walk([&](int j, const uint4& raw) {
          float f[EPC];
          g.values(raw, j, f);
          collect(j, f, max_of(f) >= x1);
        });
        bin_high();
        cta_sync();
        if (wid == 0) push_bins_info();
        sync();
        if (cs > 1) {
          merge_bins();
          sync();
        }
        fresh = true;
      } else {
        // the mass of the rest of the row, exactly
        u64 total = 0;
        walk([&](int j, const uint4& raw) {
          float f[EPC];
          g.values(raw, j, f);
#pragma unroll
          for (int i = 0; i < EPC; ++i) {
            const uint32_t w = sf_weight(f[i], m, q.r);
            total += f[i] < x1 ? w : 0u;
          }
        });
        total = warp_sum_u64(total);
        if (lane == 0) sh.red[wid] = total;
        cta_sync();
        if (wid == 0) {
          total = warp_sum_u64(lane < NW ? sh.red[lane] : 0);
          if (lane == 0) lead->part_total[rank] = total;
        }
        sync();
        if (rank == 0 && wid == 0) {
          total = warp_sum_u64(lane < cs ? sh.part_total[lane] : 0);
          if (lane == 0) sh.t_lo = sh.t_hi = sh.pm[NB - 1] + total;
          __syncwarp();
        }
        weighed = true;
        fresh = false;
      }
    }
    if (command == kGather) {
      auto take = [&](float x, int at) {
        const int b = bin_of(x);
        if (((sh.marks[b >> 5] >> (b & 31)) & 1u) && sf_weight(x, m, q.r)) {
          const int slot = atomicAdd(&sh.n_mine, 1);
          if (slot < CAP)
            sh.incl[slot] = ((u64)Logit<T>::key(x) << 32) | (u64)(0xffffffffu - (uint32_t)(at - g.dc));
        }
      };
      if (RESIDENT || have <= ECAP) {
        for (int i = lane; i < have; i += 32) take(kept_value(i), kept_place(i));
      } else if constexpr (PASS != kFirst) {
        walk([&](int j, const uint4& raw) {
          float f[EPC];
          g.values(raw, j, f);
#pragma unroll
          for (int i = 0; i < EPC; ++i)
            if (f[i] >= x1) take(f[i], EPC * j + i);
        });
      }
      // to rank 0's list, in one piece
      cta_sync();
      const int mine = min(sh.n_mine, CAP);
      if (cs == 1) {
        if (tid == 0) sh.n_list = mine;
        for (int i = tid; i < mine; i += NT) sh.list[i] = sh.incl[i];
      } else if (mine) {
        if (tid == 0) sh.mine_at = atomicAdd(&lead->n_list, mine);
        cta_sync();
        for (int i = tid; i < mine; i += NT)
          if (sh.mine_at + i < CAP) lead->list[sh.mine_at + i] = sh.incl[i];
      }
      sync();
    }
    start_copy(next);
    if (rank != 0) continue;

    // ---- rank 0 answers
    const float lse = ref + logf(sh.known_sum);
    if (PASS == kFirst && command == kMark) {
      if (tid == 0) {
        a.out_tokens[n] = kStreamMark;
        a.out_logprobs[n] = sh.hint;
      }
    } else if (command == kDone) {
      if (tid == 0) {
        report(a.d_status, DS_DEV_ERR_LOGITS);
        a.out_tokens[n] = -1;
        a.out_logprobs[n] = __int_as_float(0x7fffffff);
      }
    } else if (PASS != kFirst && command == kExact) {
      const T* row = static_cast<const T*>(a.x) + n * a.ld;
      const Bins<NB> bins = {sh.cnt, sh.lo, sh.hi, sh.pc, sh.red, sh.found};
      const int token = row_exact<T, NT, NB>(row, a.V, q, m, bins, &sh.slot);
      if (tid == 0) {
        a.out_tokens[n] = token;
        a.out_logprobs[n] = Logit<T>::get(row, token) - lse;
      }
    } else {
      const int len = sh.n_list;
      if (len == 1) {
        // every boundary falls on it
        if (tid == 0) {
          const u64 e = sh.list[0];
          a.out_tokens[n] = (int)(0xffffffffu - (uint32_t)e);
          a.out_logprobs[n] = Logit<T>::value((uint32_t)(e >> 32)) - lse;
        }
        cta_sync();
        continue;
      }
      if (len <= 32) {
        if (wid == 0) {
          // each entry to the place that the number of larger ones gives; all differ
          const u64 v = lane < len ? sh.list[lane] : 0;
          int place = 0;
          for (int o = 0; o < len; ++o) place += sh.list[o] > v;
          __syncwarp();
          if (lane < len) sh.list[place] = v;
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
      u64 kept = 0;  // mass through the last of the top-k
      if (wid == 0) {
        // running mass through each listed logit: through its bin's predecessor, plus the listed ones of its bin
        u64 sum = 0, off = 0;
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
      }
      for (;;) {
        if (wid == 0) {
          auto first_at_least = [&](u64 t) {
            for (int j = 0; j < len; j += 32) {
              const unsigned hit = __ballot_sync(0xffffffffu, j + lane < len && sh.incl[j + lane] >= t);
              if (hit) return j + __ffs(hit) - 1;
            }
            return max(len - 1, 0);  // not reached: the boundary's bin is listed
          };
          u64 lo_t = sh.t_lo, hi_t = sh.t_hi;
          if (sh.kb >= 0) lo_t = hi_t = sh.pc[sh.kb] == (uint32_t)q.k ? sh.pm[sh.kb] : kept;
          if (q.p < 1.f) {
            const int hi_at = first_at_least(need_of(q.p, hi_t));
            const int lo_at = lo_t == hi_t ? hi_at : first_at_least(need_of(q.p, lo_t));
            hi_t = sh.incl[hi_at];
            lo_t = sh.incl[lo_at];
          }
          if (floored) {
            // through the last listed logit that min-p keeps
            u64 f = ~0ull;
            const int fb = sh.known_floor;
            if ((sh.marks[max(fb, 0) >> 5] >> (max(fb, 0) & 31)) & 1u) {
              for (int j = 0; j < len; j += 32) {
                bool stays = false;
                if (j + lane < len) {
                  const float x = Logit<T>::value((uint32_t)(sh.list[j + lane] >> 32));
                  stays = bin_of(x) == fb && sf_weight(x, m, q.r) >= q.floor_w;
                }
                const unsigned st_ = __ballot_sync(0xffffffffu, stays);
                if (st_) f = sh.incl[j + 31 - __clz(st_)];
              }
            }
            lo_t = f < lo_t ? f : lo_t;
            hi_t = f < hi_t ? f : hi_t;
          }
          const int at = first_at_least(target_of(q.u, hi_t) + 1);
          const int lo_at = lo_t == hi_t ? at : first_at_least(target_of(q.u, lo_t) + 1);
          if (lane == 0) {
            sh.again = at != lo_at;
            const u64 e = sh.list[at];
            a.out_tokens[n] = PASS == kFirst && RESIDENT && at != lo_at ? kStreamMark : (int)(0xffffffffu - (uint32_t)e);
            a.out_logprobs[n] = Logit<T>::value((uint32_t)(e >> 32)) - lse;
          }
        }
        if (PASS == kFirst && RESIDENT) break;
        cta_sync();
        if (!sh.again) break;
        // the bounds fall on two logits: weigh the whole row here
        const u64 sum = row_mass<T, NT>(g, 0u, m, q.r, sh.red);
        cta_sync();
        if (tid == 0) sh.t_lo = sh.t_hi = sum;
        cta_sync();
      }
    }
    cta_sync();  // the lists are free
  }
  sync();  // no CTA leaves while a peer may still use its shared memory
}

namespace {

// Which kernel a call runs. Measured (us, rows x V of bf16, mixed parameters):
//   a warp per row          8000 x 2048    95    2000 x 4000  68   8000 x 4000 181
//   128 threads, resident                        2000 x 4000  50   8000 x 4000 156   600 x 16000  62   4 x 16000 21
//   512 threads, streamed   600 x 16000   107    2000 x 32000 233  300 x 64000  58   1000 x 64000 163
//   256 threads, streamed   100 x 32000 29 (41)  2000 x 32000 149  300 x 64000  66   1000 x 64000 136
constexpr int kSfSmallV = 2048;   // rows up to here, when there are enough to fill the GPU: a warp each
constexpr int kSfMediumV = 8192;  // rows up to here: 128-thread CTAs, held in shared memory
constexpr long long kSfMediumBytes = 32 << 10;  // and, when there are enough to fill the GPU, up to here
constexpr long long kSfLongBytes = 128 << 10;   // streamed rows up to here: 256 threads, two CTAs in a second pass
constexpr long long kSfSliceMin = 8 << 10;

// Launches the fast kernel with cs CTAs per row; *refused when no cluster of that shape fits.
template <typename T, int NT, int NB, int CAP, int GROUPS, int QCAP, int ECAP, bool RESIDENT, Pass PASS>
cudaError_t launch_fast(const FilteredArgs& a, int cs, cudaStream_t st, bool* refused) {
  auto kern = k_sample_filtered<T, NT, NB, CAP, GROUPS, QCAP, ECAP, RESIDENT, PASS>;
  // a resident slice: the most chunks that a row's 16-byte blocks can make, shared out
  const int chunks = RESIDENT ? (int)((((long long)a.V * sizeof(T) + 46 - 2 * sizeof(T)) / 16 + cs - 1) / cs) : 0;
  const size_t smem = RESIDENT ? (size_t)chunks * 16 + (size_t)((chunks + NT - 1) / NT) * NT * (16 / sizeof(T)) * 2
                               : (size_t)(NT / 32) * ECAP * 8;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.gridDim = dim3((unsigned)cs);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cs;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  // A CTA alone is launched without a cluster: as clusters of one, only eight of them run on an SM.
  cfg.numAttrs = cs == 1 ? 1 : 2;
  const void* site = reinterpret_cast<const void*>(kern);
  const int ok = cached(site, -1, [&](int) {
    const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 << 10);
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
  // Marked rows are few and fall anywhere: short shares, handed out as clusters
  // come free (15510 x 1025: one, two, four or eight shares per resident CTA 133,
  // 126, 126, 128 us). Empty CTAs of long rows cost more: 256 x 248320, none / an
  // eighth marked, 49 / 144 us with three shares per cluster, 52 / 123 us with eight.
  const long long most = PASS != kMarked ? fit : RESIDENT ? 4ll * fit : 8ll * fit;
  const long long clusters = a.n < most ? a.n : most;
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
  bool refused = false;
  cudaError_t e;
  if (a.V <= kSfSmallV && a.n >= sms * 8LL) {
    e = launch_fast<T, 32, 64, 64, 32, 0, 0, true, kFirst>(a, 1, st, &refused);
    if (!refused && e == cudaSuccess) e = launch_fast<T, 128, 256, 256, 32, 0, 0, true, kMarked>(a, 1, st, &refused);
  } else if (a.V <= kSfMediumV || (a.n >= sms && (long long)a.V * sizeof(T) <= kSfMediumBytes)) {
    e = launch_fast<T, 128, 256, 256, 32, 0, 0, true, kOnce>(a, 1, st, &refused);
  } else {
    // A CTA per row, or as many as the SMs that the rows leave, down to 8 KB of a
    // row each. A CTA alone would hold the call up with a row that takes several
    // more walks: such rows get two or eight CTAs each in a second pass.
    const long long bytes = (long long)a.V * sizeof(T);
    int cs = 1;
    while (cs < 8 && a.n * cs * 2LL <= sms && bytes >= cs * 2 * kSfSliceMin) cs *= 2;
    if (cs == 1) {
      e = bytes <= kSfLongBytes ? launch_fast<T, 256, 512, 512, 32, 384, 256, false, kFirst>(a, 1, st, &refused)
                                : launch_fast<T, 512, 1024, 512, 32, 384, 256, false, kFirst>(a, 1, st, &refused);
      if (refused || e != cudaSuccess) return refused ? cudaErrorLaunchOutOfResources : e;
      e = launch_fast<T, 512, 1024, 512, 128, 384, 512, false, kMarked>(a, bytes <= kSfLongBytes ? 2 : 8, st, &refused);
    } else {
      e = launch_fast<T, 512, 1024, 512, 128, 384, 512, false, kOnce>(a, cs, st, &refused);
    }
    if (refused) {
      // no cluster of that size fits beside another program's work: a CTA per row does
      refused = false;
      e = cs == 1 ? launch_fast<T, 512, 1024, 512, 128, 384, 512, false, kMarked>(a, 1, st, &refused)
                  : launch_fast<T, 512, 1024, 512, 128, 384, 512, false, kOnce>(a, 1, st, &refused);
    }
  }
  return refused ? cudaErrorLaunchOutOfResources : e;
}

cudaError_t launch_sample_filtered(const FilteredArgs& a, bool f32, cudaStream_t st) {
  return f32 ? launch_filtered<float>(a, st) : launch_filtered<uint16_t>(a, st);
}

}  // namespace ds
