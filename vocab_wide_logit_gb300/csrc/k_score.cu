// k_score.cu -- log-probabilities of given tokens, with log-sum-exp, entropy, rank
// and the most likely alternatives.
//
// Per row, with m = max x, e_j = exp(x_j - m), s = sum e_j and t = sum e_j (x_j - m):
//   lse = m + log s,  logprob = x_token - lse,  H = log s - t / s,
//   rank = how many come before the token by (x descending, id ascending),
// and the first `top` of that order, all from one read of the row.
//
// Sums: m is a running maximum, s and t are rescaled when it moves. Two bf16 logits
// cost one packed maximum, one packed clamp (which keeps -inf out of the product in t:
// at 256 below m an exponential is 0 already), two exponentials, four packed fp32
// instructions and, for the rank, a packed comparison and a packed sum.
//
// Alternatives: a logit is among the first `top` only if its thread's own maximum
// is: of the groups of threads (a warp's lanes, or 64 or more groups of a block)
// the maxima are ranked, and the top-th of them bounds the top-th logit from below.
// What reaches the bound, a few more than `top` for rows in any usual order, is
// listed, from the registers or a second look at those threads' shares, and ranked by
// counting who comes before whom. The bound is a pair (logit, chunk of 16 bytes), so
// that ties (a masked row's -inf above all) list a few chunks and not the row. A list that
// is long all the same is cut at its exact top-th entry, found bit by bit.
#include <climits>
#include <cooperative_groups.h>

#include "ds_device.cuh"
#include "ds_index.h"
#include "ds_launch.h"

namespace cg = cooperative_groups;

namespace ds {

namespace {

typedef unsigned long long u64;
constexpr uint32_t kMinusInf2 = 0xff80ff80u;  // two bf16 of -inf
constexpr uint32_t kMinusInf = 0xff800000u;

// ---------------------------------------------------------------- packed bf16
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {  // a NaN stays
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t gt2(uint32_t a, uint32_t b) {  // 1 or 0, as bf16
  uint32_t r;
  asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t ge2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("set.ge.bf16x2.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf2(float f) {  // f rounded, in both halves
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(r) : "f"(f));
  return r;
}

// ---------------------------------------------------------------- a row's logits
template <bool F32>
struct Row {
  static constexpr int E = F32 ? 4 : 8;     // logits of a 16-byte chunk
  static constexpr int kSize = F32 ? 4 : 2;
  const char* at;    // the row
  const char* base;  // its first chunk
  int dc;            // logits of the first chunk that are before the row
  int nq;            // chunks
  __device__ __forceinline__ Row(const ScoreArgs& a, int row) {
    at = static_cast<const char*>(a.x) + (long long)row * a.ld * kSize;
    const uintptr_t p = reinterpret_cast<uintptr_t>(at);
    base = reinterpret_cast<const char*>(p & ~(uintptr_t)15);
    dc = (int)(p & 15) / kSize;
    nq = (int)(((long long)dc + a.V + E - 1) / E);
  }
  __device__ __forceinline__ uint4 chunk(int q) const { return ld_stream16(base + 16LL * q); }
  __device__ __forceinline__ float logit(int id) const {
    if constexpr (F32)
      return __ldg(reinterpret_cast<const float*>(at) + id);
    else
      return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(at) + id) << 16);
  }
};

template <bool F32>
__device__ __forceinline__ float logit_of(const uint4& v, int i) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (F32)
    return __uint_as_float(w[i]);
  else
    return (i & 1) ? bf_hi(w[i >> 1]) : bf_lo(w[i >> 1]);
}

template <bool F32>
__device__ __forceinline__ uint4 nothing() {
  const uint32_t w = F32 ? kMinusInf : kMinusInf2;
  return make_uint4(w, w, w, w);
}

// The logits of a chunk that are not the row's become -inf.
template <bool F32>
__device__ __forceinline__ void mask_edges(uint4& v, int q, int dc, int V) {
  constexpr int E = Row<F32>::E;
  // a bit for each logit of the row
  const long long first = (long long)q * E - dc;
  const int lo = first < 0 ? (int)-first : 0, hi = V - first < E ? (int)(V - first) : E;
  const uint32_t keep = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      w[i] = (keep >> i & 1u) ? w[i] : kMinusInf;
    } else {
      const uint32_t m = (0u - (keep >> (2 * i) & 1u)) & 0x0000ffffu | (0u - (keep >> (2 * i + 1) & 1u)) & 0xffff0000u;
      w[i] = (w[i] & m) | (kMinusInf2 & ~m);
    }
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F32>
__device__ __forceinline__ float chunk_max(const uint4& v) {
  if constexpr (F32) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else {
    const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
    return fmaxf(bf_lo(m), bf_hi(m));
  }
}

template <bool F32, int U>
__device__ __forceinline__ float chunks_max(const uint4 (&v)[U]) {
  if constexpr (F32) {
    float m = chunk_max<F32>(v[0]);
#pragma unroll
    for (int u = 1; u < U; ++u) m = fmaxf(m, chunk_max<F32>(v[u]));
    return m;
  } else {
    uint32_t m = max2(max2(v[0].x, v[0].y), max2(v[0].z, v[0].w));
#pragma unroll
    for (int u = 1; u < U; ++u) m = max2(m, max2(max2(v[u].x, v[u].y), max2(v[u].z, v[u].w)));
    return fmaxf(bf_lo(m), bf_hi(m));
  }
}

// Adds exp(x - m) and exp(x - m) (x - m) of a chunk to s and t; m is finite and not
// below any x. A NaN shows in s.
template <bool F32>
__device__ __forceinline__ void add_sums(const uint4& v, float m, uint32_t low2, float2& s, float2& t) {
  const float2 nm = make_float2(-m, -m), l2e = make_float2(kLog2e, kLog2e);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 d = __fadd2_rn(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), nm);
      const float2 a = __fmul2_rn(d, l2e);
      const float2 e = make_float2(ex2_approx(a.x), ex2_approx(a.y));
      s = __fadd2_rn(s, e);
      d = make_float2(fmaxf(d.x, -256.f), fmaxf(d.y, -256.f));
      t = __ffma2_rn(e, d, t);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = max2_nan(w[i], low2);
      const float2 d = __fadd2_rn(make_float2(bf_lo(c), bf_hi(c)), nm);
      const float2 a = __fmul2_rn(d, l2e);
      const float2 e = make_float2(ex2_approx(a.x), ex2_approx(a.y));
      s = __fadd2_rn(s, e);
      t = __ffma2_rn(e, d, t);
    }
  }
}
// The same where m is so low that nothing finite lies 256 below it: logits are 1e31 apart
// there, each exponential is 0 or 1 and the sums are counts, exact up to 2^24.
template <bool F32>
__device__ __noinline__ void add_sums_low(uint4 v, float m, float2& s, float2& t) {
  for (int i = 0; i < Row<F32>::E; ++i) {
    const float d = logit_of<F32>(v, i) - m, e = ex2_approx(d * kLog2e);
    s.x += e;
    t.x += e > 0.f ? e * d : 0.f;
  }
}
// NaN when one of a chunk is, else 0.
template <bool F32>
__device__ __noinline__ float nan_of(uint4 v) {
  float n = 0.f;
  for (int i = 0; i < Row<F32>::E; ++i) {
    const float f = logit_of<F32>(v, i);
    if (f != f) n = f;
  }
  return n;
}
// What the clamp of bf16 logits may not fall below: 192 under m or more, whatever the
// rounding to bf16 (up to 2^-8 of it, a quarter of the distance for large m). The
// exponential of -104 is 0 already.
__device__ __forceinline__ uint32_t low_of(float m) { return bf2(m - fmaxf(256.f, fabsf(m) * 0.015625f)); }
__device__ __forceinline__ bool is_low(float m) { return m < -1e38f; }

// How many logits of a chunk come before the token: those above x_token, and in
// chunks in front of the token's those equal to it. (In the token's own chunk those
// are counted apart, once a row.)
template <bool F32>
__device__ __forceinline__ int count_before(const uint4& v, bool front, float xt) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  int n = 0;
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) n += front ? __uint_as_float(w[i]) >= xt : __uint_as_float(w[i]) > xt;
  } else {
    const uint32_t x2 = bf2(xt);
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c = add2(c, front ? ge2(w[i], x2) : gt2(w[i], x2));
    n = (int)(bf_lo(c) + bf_hi(c));
  }
  return n;
}
// The same for chunks none of which is in front of the token's.
template <bool F32, int U>
__device__ __forceinline__ int count_all(const uint4 (&v)[U], float xt) {
  int n = 0;
  if constexpr (F32) {
#pragma unroll
    for (int u = 0; u < U; ++u) n += count_before<F32>(v[u], false, xt);
  } else {
    static_assert(U * 4 <= 128, "sums of ones in bf16 are exact up to 256");
    const uint32_t x2 = bf2(xt);
    uint32_t c = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      c = add2(c, add2(add2(gt2(v[u].x, x2), gt2(v[u].y, x2)), add2(gt2(v[u].z, x2), gt2(v[u].w, x2))));
    n = (int)(bf_lo(c) + bf_hi(c));
  }
  return n;
}

// The order (x descending, id or chunk ascending; -0 and +0 tie) as an integer. No
// logit gives 0.
__device__ __forceinline__ u64 order_of(float x, int id) {
  return ((u64)order_key(x + 0.f) << 32) | (uint32_t)~id;
}
__device__ __forceinline__ int id_of(u64 key) { return (int)~(uint32_t)key; }
__device__ __forceinline__ float logit_of_key(u64 key) {
  const uint32_t k = (uint32_t)(key >> 32);
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// ---------------------------------------------------------------- a row's results
struct Sums {
  float m, s, t;
  int before;
};

struct Given {
  int token;  // -1: none
  float x;    // its logit; +inf without one (nothing counts as before)
  int chunk;  // its chunk; 0 without one
};
template <bool F32>
__device__ __forceinline__ Given given_token(const ScoreArgs& a, int row, const Row<F32>& x) {
  const int tok = a.tokens[row];
  Given g{-1, kInf, 0};
  if (tok >= 0 && tok < a.V) {
    g.token = tok;
    g.x = x.logit(tok);
    g.chunk = chunk_of(tok, Row<F32>::E, x.dc);
  }
  return g;
}
// Lane i: logit i of the token's chunk when that is in front of the token, else NaN.
template <bool F32>
__device__ __forceinline__ float in_front(const Row<F32>& x, const Given& g) {
  const int first = first_in_chunk(g.chunk, Row<F32>::E, x.dc), place = (int)(threadIdx.x & 31);
  return in_front_of(g.token, first, place) ? x.logit(first + place) : __int_as_float(0x7fffffff);
}
// What `before` lacks or has too much: ties in front of the token in its own chunk;
// the padding in front of the row, which ties with a token of -inf. For a whole warp.
__device__ __forceinline__ int rank_mend(const Given& g, float near, int dc) {
  const int n = __popc(__ballot_sync(0xffffffffu, near == g.x));
  return n - (g.x == -kInf && g.chunk > 0 ? dc : 0);
}

// Writes the row's four numbers.
__device__ __forceinline__ void write_row(const ScoreArgs& a, int row, const Sums& r, const Given& g, float log_s) {
  const float nan = __int_as_float(0x7fffffff);
  const bool bad = !(r.s < kInf) || r.m == kInf;  // a NaN or +inf among the logits
  const bool none = bad || r.m == -kInf;
  const float lse = bad ? nan : none ? -kInf : r.m + log_s;
  a.out_logprobs[row] = none || g.token < 0 ? nan : (g.x - r.m) - log_s;
  if (a.out_lse) a.out_lse[row] = lse;
  if (a.out_entropy) a.out_entropy[row] = none ? nan : log_s - r.t / r.s;
  if (a.out_ranks) a.out_ranks[row] = none || g.token < 0 ? -1 : r.before;
  const uint32_t bits = (a.tokens[row] >= a.V ? DS_DEV_ERR_PARAM : 0u) | (bad ? DS_DEV_ERR_LOGITS : 0u);
  if (bits) report(a.d_status, bits);
}
// Alternative number r; key 0 for none.
__device__ __forceinline__ void write_top(const ScoreArgs& a, int row, int r, u64 key, float m, float log_s, bool none) {
  const long long at = (long long)row * a.top + r;
  a.out_top_ids[at] = none ? -1 : id_of(key);
  a.out_top_logprobs[at] = none ? __int_as_float(0x7fffffff) : (logit_of_key(key) - m) - log_s;
}
__device__ __forceinline__ bool is_none(const Sums& r) { return !(r.s < kInf) || r.m == kInf || r.m == -kInf; }

// ---------------------------------------------------------------- a warp per row
// Rows of up to 32 C chunks, held in registers, so that the maximum is known before the
// one walk that makes the sums. Bounded by instructions: 1107 for 1025 bf16 logits and 8
// alternatives; 15510 such rows take 19.8 us (11.1 us without alternatives), 1.7 TB/s.
constexpr int kWarps = 4;
// Alternatives that are bounded by a lane's maximum each, more by a chunk's: the 20th of 32
// maxima lists 31 logits in the mean, the 32nd 130.
constexpr int kWarpTop = 24;
// Candidates a row may list: as many chunks of 8 as alternatives or lanes.
__host__ __device__ constexpr int warp_list(bool many) { return 8 * (many ? DS_SCORE_MAX_TOP : 32); }
constexpr int kLongList = 128;  // entries from which the exact cut is cheaper than ranking all

// The top-th largest of n unique keys.
__device__ __noinline__ u64 warp_cut(const u64* list, int n, int top) {
  const int lane = threadIdx.x & 31;
  const u64 any = list[0];
  u64 d = 1;
  for (int i = lane; i < n; i += 32) d |= list[i] ^ any;
  d = ((u64)__reduce_or_sync(0xffffffffu, (uint32_t)(d >> 32)) << 32) | __reduce_or_sync(0xffffffffu, (uint32_t)d);
  const int from = 63 - __clzll((long long)d);  // above it all of them agree
  u64 cut = from == 63 ? 0 : any >> (from + 1) << (from + 1);
  for (int bit = from; bit >= 0; --bit) {
    const u64 trial = cut | (1ull << bit);
    int c = 0;
    for (int i = lane; i < n; i += 32) c += list[i] >= trial;
    c = warp_sum_i(c);
    if (c >= top) cut = trial;
    if (c == top) break;
  }
  return cut;
}

// Which logits of a chunk are at or above f, a bit each.
template <bool F32>
__device__ __forceinline__ uint32_t reaching(const uint4& v, float f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t bits = 0;
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) bits |= (uint32_t)(__uint_as_float(w[i]) >= f) << i;
  } else {
    const uint32_t f2 = bf2(f);
    uint32_t c = 0;  // a one is 0x3f80: its bit 7
#pragma unroll
    for (int i = 0; i < 4; ++i) c |= (ge2(w[i], f2) & 0x00800080u) >> (7 - 2 * i);
    bits = (c | (c >> 15)) & 0xffu;
  }
  return bits;
}
// Logit i of a chunk in registers.
template <bool F32>
__device__ __forceinline__ float pick(const uint4& v, int i) {
  const int k = F32 ? i : i >> 1;
  const uint32_t lo = (k & 1) ? v.y : v.x, hi = (k & 1) ? v.w : v.z, w = (k & 2) ? hi : lo;
  if constexpr (F32)
    return __uint_as_float(w);
  else
    return (i & 1) ? bf_hi(w) : bf_lo(w);
}

// The first `top` of a row, listed in no order, when its order puts the largest
// into few lanes: the exact cut, then the list, from memory. Returns how many.
template <bool F32>
__device__ __noinline__ int warp_list_exact(const Row<F32> x, int V, int top, u64* list, int size) {
  const int lane = threadIdx.x & 31;
  u64 cut = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const u64 trial = cut | (1ull << bit);
    int c = 0;
    for (int id = lane; id < V; id += 32) c += order_of(x.logit(id), id) >= trial;
    c = warp_sum_i(c);
    if (c >= top) cut = trial;
    if (c == top) break;
  }
  int listed = 0;
  for (int id0 = 0; id0 < V; id0 += 32) {
    const u64 o = id0 + lane < V ? order_of(x.logit(id0 + lane), id0 + lane) : 0;
    const bool in = o != 0 && o >= cut;
    const unsigned who = __ballot_sync(0xffffffffu, in);
    const int pos = listed + __popc(who & ((1u << lane) - 1));
    if (in && pos < size) list[pos] = o;
    listed += __popc(who);
  }
  __syncwarp();
  return min(listed, size);
}

// Leaves of n listed keys those at or above the cut, in their order. Returns how many.
__device__ __forceinline__ int warp_keep(u64* list, int n, u64 cut) {
  const int lane = threadIdx.x & 31;
  int kept = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const u64 key = i0 + lane < n ? list[i0 + lane] : 0;
    const bool in = key != 0 && key >= cut;
    const unsigned who = __ballot_sync(0xffffffffu, in);
    if (in) list[kept + __popc(who & ((1u << lane) - 1))] = key;
    kept += __popc(who);
    __syncwarp();
  }
  return kept;
}

// MANY: more than kWarpTop alternatives. TAIL: up to 32 logits behind the 32 C chunks, one a
// lane, where lengths just above 32 C chunks would have a turn of chunks for a few of them.
// Launched for bf16 rows of 762 to 1049 logits (C = 4) and fp32 rows of 382 to 541 (C = 4) and
// 894 to 1053 (C = 8); other lengths take the next C that holds them. It needs the loop
// over a lane's bits (C > 2) and a bit of the 64 beside theirs (C E < 64): there is none for
// 513 bf16 logits, nor for 2049.
template <bool F32, int C, bool MANY, bool TAIL>
__global__ void __launch_bounds__(kWarps * 32) k_score_warp(const ScoreArgs a) {
  constexpr int E = Row<F32>::E, kWarpList = warp_list(MANY);
  static_assert(!TAIL || (!MANY && C > 2 && C * E < 64), "a bit for the logit behind the chunks");
  __shared__ u64 lists[kWarps][kWarpList];
  pdl_release();
  pdl_wait();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const long long row_l = (long long)blockIdx.x * kWarps + wid;
  if (row_l >= a.n) return;
  const int row = (int)row_l;
  const Row<F32> x(a, row);
  uint4 v[C];
#pragma unroll
  for (int u = 0; u < C; ++u) {
    const int q = lane + 32 * u;
    v[u] = q < x.nq ? x.chunk(q) : nothing<F32>();
  }
  const int tail_id = 32 * C * E - x.dc + lane, tail_chunk = 32 * C + lane / E;
  const bool has_tail = TAIL && tail_id < a.V;
  const float tail = has_tail ? x.logit(tail_id) : -kInf;
  const Given g = given_token(a, row, x);
  const float near = in_front(x, g);
  // the row's first and last chunk reach beyond it
  if (lane == 0) mask_edges<F32>(v[0], 0, x.dc, a.V);
#pragma unroll
  for (int u = 0; u < C; ++u)
    if (lane + 32 * u == x.nq - 1) mask_edges<F32>(v[u], lane + 32 * u, x.dc, a.V);

  float best = -kInf;  // the lane's maximum and its first chunk
  int at = lane;
  Sums r{-kInf, 0.f, 0.f, 0};
#pragma unroll
  for (int u = 0; u < C; ++u) {
    const float c = chunk_max<F32>(v[u]);
    if (c > best) {
      best = c;
      at = lane + 32 * u;
    }
    const int q = lane + 32 * u;
    if (q < x.nq) r.before += count_before<F32>(v[u], q < g.chunk, g.x);
  }
  if (TAIL && tail > best) {
    best = tail;
    at = tail_chunk;
  }
  if (has_tail) r.before += tail_chunk < g.chunk ? tail >= g.x : tail > g.x;
  r.m = warp_max_r(best);
  float2 s = make_float2(0.f, 0.f), t = s;
  if (is_low(r.m)) {
    if (r.m != -kInf)
#pragma unroll
      for (int u = 0; u < C; ++u) add_sums_low<F32>(v[u], r.m, s, t);
  } else {
    const uint32_t low2 = low_of(r.m);
#pragma unroll
    for (int u = 0; u < C; ++u) add_sums<F32>(v[u], r.m, low2, s, t);
  }
  if (TAIL && r.m != -kInf) {
    const float d = tail - r.m, e = ex2_approx(d * kLog2e);
    s.x += e;
    t.x += e > 0.f ? e * d : 0.f;
  }
  r.s = warp_sum(s.x + s.y);
  r.t = warp_sum(t.x + t.y);
  if (r.m == -kInf) {  // a row of NaN and -inf alone: s shows the NaN
    float seen = 0.f;
#pragma unroll
    for (int u = 0; u < C; ++u) seen += nan_of<F32>(v[u]);
    if (tail != tail) seen = tail;
    r.s = warp_sum(seen);
  }
  r.before = warp_sum_i(r.before);
  r.before += rank_mend(g, near, x.dc);
  const float log_s = logf(r.s);
  if (lane == 0) write_row(a, row, r, g, log_s);
  if (a.top == 0) return;
  const bool none = is_none(r);
  if (none) {
    for (int i = lane; i < a.top; i += 32) write_top(a, row, i, 0, 0.f, 0.f, true);
    return;
  }

  // the bound: the top-th of the lanes' maxima, or of the chunks', by (logit, chunk)
  uint32_t key = lane < x.nq ? order_key(best + 0.f) : 0u, bound = 0;
  int bound_at = INT_MAX;
  const bool all = x.nq < a.top;
  if constexpr (MANY) {
    uint32_t keys[C];
#pragma unroll
    for (int u = 0; u < C; ++u) keys[u] = lane + 32 * u < x.nq ? order_key(chunk_max<F32>(v[u]) + 0.f) : 0u;
    auto count = [&](auto f) {
      int c = 0;
#pragma unroll
      for (int u = 0; u < C; ++u) c += f(keys[u], lane + 32 * u);
      return warp_sum_i(c);
    };
    if (!all) {
      // bit by bit; of a bf16's key the upper half says it
      for (int bit = 31; bit >= (F32 ? 0 : 16); --bit) {
        const uint32_t trial = bound | (1u << bit);
        if (count([&](uint32_t k, int) { return k >= trial; }) >= a.top) bound = trial;
      }
      if (!F32 && bound < 0x80000000u) bound |= 0xffffu;
      // of those that tie, the chunks up to the one that makes them enough
      const int left = a.top - count([&](uint32_t k, int) { return k > bound; });
      int below = 0;  // the largest number such that fewer tie in front of it
      for (int bit = 1 << 9; bit > 0; bit >>= 1)
        if (count([&](uint32_t k, int q) { return k == bound && q < (below | bit); }) < left) below |= bit;
      bound_at = below;
    }
  } else if (!all) {
    int left = a.top;
    uint32_t rest = key;
    while (true) {
      bound = __reduce_max_sync(0xffffffffu, rest);
      const bool mine = rest == bound;
      const int c = __popc(__ballot_sync(0xffffffffu, mine));
      if (c >= left) {
        // of those that tie, the left-th chunk
        unsigned chunk = mine ? (unsigned)at : UINT_MAX;
        for (; left > 0; --left) {
          bound_at = (int)__reduce_min_sync(0xffffffffu, chunk);
          if (chunk == (unsigned)bound_at) chunk = UINT_MAX;
        }
        break;
      }
      left -= c;
      if (mine) rest = 0;
    }
  }
  // list what reaches it
  u64* list = lists[wid];
  int listed = 0;
  const u64 cut = ((u64)bound << 32) | (uint32_t)~bound_at;
  const float bound_x = logit_of_key(cut);
  const bool any = lane < x.nq && (MANY || (((u64)key << 32) | (uint32_t)~at) >= cut);
  if (all) {  // fewer chunks than alternatives
    for (int id = lane; id < a.V; id += 32) list[id] = order_of(x.logit(id), id);
    listed = a.V;
  } else if constexpr (C > 2 && C * E <= 64) {
    // a bit for each logit of the lane that reaches the bound; the logits from memory again
    u64 reach = 0;
#pragma unroll
    for (int u = 0; u < C; ++u) reach |= (u64)reaching<F32>(v[u], bound_x) << (E * u);
    if (TAIL && tail >= bound_x) reach |= 1ull << (C * E & 63);
    if (!any) reach = 0;
    const int first = lane * E - x.dc;
    while (__any_sync(0xffffffffu, reach != 0)) {
      const int i = reach ? __ffsll((long long)reach) - 1 : 0;
      int q = lane + 32 * (i / E), id = first + 32 * E * (i / E) + i % E;
      if (TAIL && i == C * E) q = tail_chunk, id = tail_id;
      const bool in_row = reach && id >= 0 && id < a.V;
      const uint32_t k = order_key((in_row ? x.logit(id) : 0.f) + 0.f);
      const bool in = in_row && (((u64)k << 32) | (uint32_t)~q) >= cut;
      const unsigned who = __ballot_sync(0xffffffffu, in);
      const int pos = listed + __popc(who & ((1u << lane) - 1));
      if (in && pos < kWarpList) list[pos] = ((u64)k << 32) | (uint32_t)~id;
      listed += __popc(who);
      reach &= reach - 1;
    }
  } else {
#pragma unroll
    for (int u = 0; u < C; ++u) {
      const int q = lane + 32 * u;
      const bool here = any && q < x.nq && chunk_max<F32>(v[u]) >= bound_x;
      if (!__any_sync(0xffffffffu, here)) continue;
      uint32_t reach = here ? reaching<F32>(v[u], bound_x) : 0;
      while (__any_sync(0xffffffffu, reach != 0)) {
        const int i = reach ? __ffs(reach) - 1 : 0, id = q * E - x.dc + i;
        const uint32_t k = order_key(pick<F32>(v[u], i) + 0.f);
        const bool in = reach && id >= 0 && id < a.V && (((u64)k << 32) | (uint32_t)~q) >= cut;
        const unsigned who = __ballot_sync(0xffffffffu, in);
        const int pos = listed + __popc(who & ((1u << lane) - 1));
        if (in && pos < kWarpList) list[pos] = ((u64)k << 32) | (uint32_t)~id;
        listed += __popc(who);
        reach &= reach - 1;
      }
    }
  }
  __syncwarp();
  if (listed > kWarpList)
    listed = warp_list_exact<F32>(x, a.V, a.top, list, kWarpList);
  else if (listed > kLongList && listed > a.top)
    listed = warp_keep(list, listed, warp_cut(list, listed, a.top));
  for (int i = lane; i < listed; i += 32) {
    const u64 mine = list[i];
    int before = 0;
    for (int j = 0; j < listed; ++j) before += list[j] > mine;
    if (before < a.top) write_top(a, row, before, mine, r.m, log_s, false);
  }
}

// ---------------------------------------------------------------- blocks per row
// A row over a cluster of CTAs, each with a slice of it; one of them joins. One CTA a row
// where there are rows for all SMs: clusters of 2 to 8 pay their barriers and the steps
// behind the last chunk as often (44 to 90 us for 35). 256 x 248320 bf16 take 35 us with
// 20 alternatives (3.6 TB/s): 22.5 us are loads and maxima, 3 the exponentials, up to 4
// the rank of unlikely tokens, 5.5 the alternatives. 37 x 70001 fp32, four CTAs a row:
// 12 us, latency.
constexpr int kMaxCluster = 8;
// Candidates a slice may list: `top` chunks of 8 logits for each thread of a group.
__host__ __device__ constexpr int list_size(int threads) { return threads >= 512 ? 2048 : 1024; }
constexpr int kLong = 160;     // entries from which the exact cut is cheaper than ranking all
constexpr int kUnroll = 4;     // chunks a thread has in flight, twice
constexpr int kFewTop = 32;    // alternatives for which 64 groups of threads are enough

template <int NT>
struct Shared {
  u64 list[list_size(NT)];  // candidates; in the joining CTA then the survivors of all slices
  u64 sorted[(NT >= 512 ? kMaxCluster : 1) * DS_SCORE_MAX_TOP];  // each slice's alternatives in order
  u64 keys[64];             // groups' maxima
  Sums warps[NT / 32];
  Sums slices[kMaxCluster];
  Sums total;
  u64 bound, differ;
  int count;
  int bits[64];
};

__device__ __forceinline__ Sums join(const Sums& p, const Sums& q) {
  Sums r;
  r.m = fmaxf(p.m, q.m);
  r.before = p.before + q.before;
  // an empty side has s = t = 0 and m = -inf: no product with that difference
  const float dp = p.m == -kInf ? 0.f : p.m - r.m, dq = q.m == -kInf ? 0.f : q.m - r.m;
  const float fp = ex2_approx(dp * kLog2e), fq = ex2_approx(dq * kLog2e);
  r.s = p.s * fp + q.s * fq;
  // far below the other's maximum a part counts nothing, whatever the distance
  r.t = (fp > 0.f ? (p.t + p.s * dp) * fp : 0.f) + (fq > 0.f ? (q.t + q.s * dq) * fq : 0.f);
  return r;
}
__device__ __forceinline__ Sums warp_join(Sums p, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) {
    Sums q;
    q.m = __shfl_xor_sync(0xffffffffu, p.m, o);
    q.s = __shfl_xor_sync(0xffffffffu, p.s, o);
    q.t = __shfl_xor_sync(0xffffffffu, p.t, o);
    q.before = __shfl_xor_sync(0xffffffffu, p.before, o);
    p = join(p, q);
  }
  return p;
}

// The top-th largest of what count(trial) counts at or above trial, for a block; bits
// are 64 zeros and stay used. All of them agree with `any` above bit `from`.
template <typename F>
__device__ __forceinline__ u64 block_cut(int* bits, int top, u64 any, int from, F count) {
  u64 cut = from == 63 ? 0 : any >> (from + 1) << (from + 1);
  for (int bit = from; bit >= 0; --bit) {
    const u64 trial = cut | (1ull << bit);
    const int c = warp_sum_i(count(trial));
    if ((threadIdx.x & 31) == 0 && c) atomicAdd(&bits[bit], c);
    __syncthreads();
    const int all = bits[bit];
    if (all >= top) cut = trial;
    if (all == top) break;
  }
  return cut;
}
// The same for n listed keys; *differ is 0 and stays used.
template <int NT>
__device__ __forceinline__ u64 list_cut(const u64* list, int n, int* bits, u64* differ, int top) {
  const u64 any = list[0];
  u64 d = 0;
  for (int i = threadIdx.x; i < n; i += NT) d |= list[i] ^ any;
  const uint32_t hi = __reduce_or_sync(0xffffffffu, (uint32_t)(d >> 32)), lo = __reduce_or_sync(0xffffffffu, (uint32_t)d);
  if ((threadIdx.x & 31) == 0) atomicOr(differ, ((u64)hi << 32) | lo);
  __syncthreads();
  return block_cut(bits, top, any, 63 - __clzll((long long)(*differ | 1)), [&](u64 trial) {
    int c = 0;
    for (int i = threadIdx.x; i < n; i += NT) c += list[i] >= trial;
    return c;
  });
}

// f(key, how many of the list are above it) for each of n keys, 16 threads a key.
template <int NT, typename F>
__device__ __forceinline__ void rank_list(const u64* list, int n, u64 cut, F f) {
  const int half = threadIdx.x >> 4, part = threadIdx.x & 15;
  for (int i = half; (i & ~1) < n; i += NT / 16) {  // both halves of a warp, or neither
    const u64 mine = i < n ? list[i] : 0;
    int above = 0;
    if (mine >= cut)
      for (int j = part; j < n; j += 16) above += list[j] > mine;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
    if (part == 0 && i < n && mine >= cut) f(mine, above);
  }
}

template <bool F32, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) k_score_block(const ScoreArgs a) {
  constexpr int E = Row<F32>::E, U = kUnroll, kList = list_size(NT);
  __shared__ Shared<NT> sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (cs > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_release();
  pdl_wait();
  const int row = (int)(blockIdx.x / (unsigned)cs);
  const Row<F32> x(a, row);
  const int q_lo = (int)((long long)rank * x.nq / cs), q_hi = (int)((long long)(rank + 1) * x.nq / cs);
  const int q_in = min(q_hi, x.nq - 1);  // chunks below it (but the row's first) lie within the row

  auto load_edge = [&](uint4 (&v)[U], int q) {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = q + u * NT < q_hi ? x.chunk(q + u * NT) : nothing<F32>();
    // the row's first and last chunk reach beyond it
    if (q == 0) mask_edges<F32>(v[0], 0, x.dc, a.V);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (q + u * NT == x.nq - 1) mask_edges<F32>(v[u], q + u * NT, x.dc, a.V);
  };

  uint4 v[U], w[U];
  int q = q_lo + tid;
  load_edge(v, q);
  if (tid < 64) sh.bits[tid] = 0;
  if (tid == 0) sh.count = 0, sh.differ = 0;
  const Given g = given_token(a, row, x);
  float m = -kInf, second = -kInf;  // second: the largest of the other batches
  uint32_t low2 = 0;
  int at = q, before = 0;
  bool usual = false;
  float2 s = make_float2(0.f, 0.f), t = s;
  // takes a batch while the next one is on its way; false behind the last
  auto step = [&](const uint4 (&v)[U], uint4 (&next)[U]) {
    const int qn = q + U * NT;
    if (qn + (U - 1) * NT < q_in) {
      const char* p = x.base + 16LL * qn;
#pragma unroll
      for (int u = 0; u < U; ++u) next[u] = ld_stream16(p + u * NT * 16);
    } else if (qn < q_hi) {
      load_edge(next, qn);
    }
    // the running maximum and the first chunk that has it
    const float c = chunks_max<F32, U>(v);
    second = fmaxf(second, fminf(c, m));
    if (c > m) {
#pragma unroll
      for (int u = U - 1; u >= 0; --u)
        if (chunk_max<F32>(v[u]) == c) at = q + u * NT;
      const float d = m - c, f = ex2_approx(d * kLog2e);
      // nothing yet, or nothing that counts beside c: no product with an infinite distance
      t = f > 0.f ? make_float2((t.x + s.x * d) * f, (t.y + s.y * d) * f) : make_float2(0.f, 0.f);
      s = make_float2(s.x * f, s.y * f);
      m = c;
      low2 = low_of(m);
      usual = !is_low(m);
    }
    if (c >= g.x) {  // few batches reach a likely token
      if (q >= g.chunk)
        before += count_all<F32, U>(v, g.x);
      else
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (q + u * NT < q_hi) before += count_before<F32>(v[u], q + u * NT < g.chunk, g.x);
    }
    if (usual) {
      // a batch's sums apart: a thread's chain of additions is as long as its batches, for fp32
      // half as long (a batch has half the logits, and its two sums go to one of s.x and s.y in turn)
      float2 bs = make_float2(0.f, 0.f), bt = bs;
#pragma unroll
      for (int u = 0; u < U; ++u) add_sums<F32>(v[u], m, low2, bs, bt);
      if constexpr (F32) {
        s = make_float2(s.y, s.x + (bs.x + bs.y));
        t = make_float2(t.y, t.x + (bt.x + bt.y));
      } else {
        s = __fadd2_rn(s, bs);
        t = __fadd2_rn(t, bt);
      }
    } else if (m != -kInf) {
      for (int u = 0; u < U; ++u) add_sums_low<F32>(v[u], m, s, t);
    } else {  // -inf and NaN alone: s shows the NaN
      for (int u = 0; u < U; ++u) s.x += nan_of<F32>(v[u]);
    }
    q = qn;
    return qn < q_hi;
  };
  // (two turns with the batches' roles exchanged instead of moved: 31.5 us for 28.5 at 256 x
  // 248320 without alternatives)
  if (q < q_hi)
#pragma unroll 1
    while (step(v, w)) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = w[u];
    }

  const float near = wid == 0 ? in_front(x, g) : 0.f;
  // join the block's sums
  {
    Sums p{m, s.x + s.y, t.x + t.y, before};
    p = warp_join(p, 32);
    if (lane == 0) sh.warps[wid] = p;
  }
  const int top = a.top;
  const u64 own = q_lo + tid < q_hi ? ((u64)order_key(m + 0.f) << 32) | (uint32_t)~at : 0;
  constexpr int kWidth = NT / 64;  // threads of a group
  const bool few = top <= kFewTop;
  if (top > 0 && few) {
    u64 k = own;
#pragma unroll
    for (int o = kWidth >> 1; o > 0; o >>= 1) {
      const u64 other = __shfl_xor_sync(0xffffffffu, k, o);
      k = k > other ? k : other;
    }
    if ((tid & (kWidth - 1)) == 0) sh.keys[tid / kWidth] = k;
  }
  __syncthreads();
  if (wid == NT / 32 - 1) {
    Sums p = lane < NT / 32 ? sh.warps[lane] : Sums{-kInf, 0.f, 0.f, 0};
    p = warp_join(p, 32);
    if (lane == 0) sh.total = p;
  }
  // The top-th of the groups' maxima bounds the slice's top-th logit from below; the
  // threads of a group share the comparisons. For more alternatives the top-th of the
  // threads' maxima, bit by bit (ranking 256 groups took 1.5 us more).
  u64 bound = 0;
  if (top > 0 && few) {
    const int group = tid / kWidth;
    const u64 k = sh.keys[group];
    int above = 0;
#pragma unroll 8
    for (int j = tid & (kWidth - 1); j < 64; j += kWidth) above += sh.keys[j] > k || (sh.keys[j] == k && j < group);
#pragma unroll
    for (int o = kWidth >> 1; o > 0; o >>= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
    if (above == top - 1) sh.bound = k;
  } else if (top > 0 && __syncthreads_count(own != 0) >= top) {
    for (int bit = 63; bit >= 0; --bit) {
      if (!F32 && bit == 47) {  // of a bf16's key the upper half says it
        if (!(bound >> 63)) bound |= 0xffffull << 32;
        bit = 31;
      }
      const u64 trial = bound | (1ull << bit);
      const int c = __syncthreads_count(own >= trial);
      if (c >= top) bound = trial;
      if (c == top) break;
    }
  }
  __syncthreads();
  if (cs == 1) {
    Sums r = sh.total;
    if (wid == 0) {
      r.before += rank_mend(g, near, x.dc);
      if (tid == 0) write_row(a, row, r, g, logf(r.s));
    }
    if (is_none(r)) {  // nothing to list
      for (int i = tid; i < top; i += NT) write_top(a, row, i, 0, 0.f, 0.f, true);
      return;
    }
    if (top == 0) return;
  }
  int listed = 0;
  u64 cut = 0;
  const bool dead = sh.total.m == -kInf;  // a slice of -inf alone: its first ones, without a look
  if (top > 0 && !dead) {
    if (few) bound = sh.bound;
    const float bound_x = bound == 0 ? -kInf : logit_of_key(bound);
    // The logits that reach the bound: in the best batch of each thread whose maximum does,
    // and in all of the thread's share, taken by its whole warp, when another batch has any.
    const int at_batch = q_lo + tid + (at - q_lo - tid) / (U * NT) * (U * NT);
    const bool has = own != 0 && own >= bound;
    // (a tie with the maximum comes after its batch)
    const uint32_t earliest = second == m ? (uint32_t)~(at_batch + U * NT) : 0xffffffffu;
    const bool one = (((u64)order_key(second + 0.f) << 32) | earliest) < bound;
    auto visit = [&](const uint4& b, int q1, auto f) {
      if ((((u64)order_key(chunk_max<F32>(b) + 0.f) << 32) | (uint32_t)~q1) < bound) return;
      for (uint32_t reach = reaching<F32>(b, bound_x); reach; reach &= reach - 1) {
        const int i = __ffs(reach) - 1;
        const long long id = (long long)q1 * E - x.dc + i;
        const uint32_t l = order_key(pick<F32>(b, i) + 0.f);
        if (id >= 0 && id < a.V && (((u64)l << 32) | (uint32_t)~q1) >= bound) f(((u64)l << 32) | (uint32_t)~(int)id);
      }
    };
    auto scan = [&](auto f) {
      if (has && one) {
        uint4 b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) b[u] = at_batch + u * NT < q_hi ? x.chunk(at_batch + u * NT) : nothing<F32>();
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (at_batch + u * NT < q_hi) visit(b[u], at_batch + u * NT, f);
      }
      for (unsigned all = __ballot_sync(0xffffffffu, has && !one); all; all &= all - 1)
        for (long long p = q_lo + (tid & ~31) + __ffs(all) - 1 + (long long)lane * NT; p < q_hi; p += 32 * NT)
          visit(x.chunk((int)p), (int)p, f);
      __syncwarp();
    };
    auto put = [&](u64 key) {
      const int pos = atomicAdd(&sh.count, 1);
      if (pos < kList) sh.list[pos] = key;
    };
    scan(put);
    __syncthreads();
    listed = sh.count;
    if (listed > kList) {
      // the largest logits met in few threads: the exact cut, then the list again
      cut = block_cut(sh.bits, top, 0, 63, [&](u64 trial) {
        int c = 0;
        scan([&](u64 key) { c += key >= trial; });
        return c;
      });
      __syncthreads();
      if (tid == 0) sh.count = 0;
      __syncthreads();
      scan([&](u64 key) {
        if (key >= cut) put(key);
      });
      __syncthreads();
      listed = min(sh.count, kList);
    } else if (listed > kLong) {
      cut = list_cut<NT>(sh.list, listed, sh.bits, &sh.differ, top);
    }
  }
  if (cs == 1) {
    const float m_row = sh.total.m, log_s = logf(sh.total.s);
    rank_list<NT>(sh.list, listed, cut, [&](u64 key, int above) {
      if (above < top) write_top(a, row, above, key, m_row, log_s, false);
    });
    return;
  }

  // in order to the joining CTA, zeros behind the last
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  {
    u64* sorted = cluster.map_shared_rank(sh.sorted, 0) + rank * top;
    rank_list<NT>(sh.list, listed, cut, [&](u64 key, int above) {
      if (above < top) sorted[above] = key;
    });
    const long long first = max(0LL, (long long)q_lo * E - x.dc), end = min((long long)a.V, (long long)q_hi * E - x.dc);
    for (int i = listed + tid; i < top; i += NT) sorted[i] = dead && first + i < end ? order_of(-kInf, (int)(first + i)) : 0;
  }
  if (tid == 0) *cluster.map_shared_rank(&sh.slices[rank], 0) = sh.total;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (rank != 0) return;  // what it wrote is the joining CTA's, which is still there
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

  // every warp joins the slices' sums for itself
  Sums r = lane < cs ? sh.slices[lane] : Sums{-kInf, 0.f, 0.f, 0};
  r = warp_join(r, 32);
  if (wid == 0) {
    Sums all = r;
    all.before += rank_mend(g, near, x.dc);
    if (tid == 0) write_row(a, row, all, g, logf(r.s));
  }
  if (top == 0) return;
  if (is_none(r)) {
    for (int i = tid; i < top; i += NT) write_top(a, row, i, 0, 0.f, 0.f, true);
    return;
  }
  // Bounds of the row's top-th: the largest of the slices' top-th entries, and, with
  // c slices that have d entries at or above a key, c d >= top, that key
  {
    const int d = (top + (cs >> 1) - 1) / (cs >> 1), c = (top + d - 1) / d;
    const u64 kd = lane < cs ? sh.sorted[lane * top + d - 1] : 0, kt = lane < cs ? sh.sorted[lane * top + top - 1] : 0;
    int above = 0;
    u64 most = 0;
    for (int j = 0; j < cs; ++j) {
      const u64 other = __shfl_sync(0xffffffffu, kd, j), last = __shfl_sync(0xffffffffu, kt, j);
      above += other > kd || (other == kd && j < lane);
      most = most > last ? most : last;
    }
    const unsigned who = __ballot_sync(0xffffffffu, lane < cs && above == c - 1);
    const u64 second_bound = __shfl_sync(0xffffffffu, kd, __ffs(who) - 1);
    bound = most > second_bound ? most : second_bound;
  }
  if (tid == 0) sh.count = 0, sh.differ = 0;
  if (tid < 64) sh.bits[tid] = 0;
  __syncthreads();
  for (int i = tid; i < cs * top; i += NT) {
    const u64 key = sh.sorted[i];
    if (key == 0 || key < bound) continue;
    sh.list[atomicAdd(&sh.count, 1)] = key;  // at most cs top, which it holds
  }
  __syncthreads();
  listed = sh.count;
  cut = listed > kLong ? list_cut<NT>(sh.list, listed, sh.bits, &sh.differ, top) : 0;
  const float log_s = logf(r.s);
  rank_list<NT>(sh.list, listed, cut, [&](u64 key, int above) {
    if (above < top) write_top(a, row, above, key, r.m, log_s, false);
  });
}
static_assert(kMaxCluster * DS_SCORE_MAX_TOP <= list_size(512), "the survivors of all slices fit the list");

template <typename K>
cudaError_t launch(K kern, const ScoreArgs& a, long long blocks, int threads, int cs, cudaStream_t st) {
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cs;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cs > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

template <bool F32>
cudaError_t launch_rows(const ScoreArgs& a, cudaStream_t st) {
  const int E = F32 ? 4 : 8;
  const long long nq = ((long long)a.V + 2 * E - 2) / E;  // the most chunks a row has
  if (nq <= 32 * 16) {
    const long long blocks = ((long long)a.n + kWarps - 1) / kWarps;
    const int c = (int)((nq + 31) / 32);
#define DS_WARP(C, MANY) return launch(k_score_warp<F32, C, MANY, false>, a, blocks, kWarps * 32, 1, st)
#define DS_TAIL(C)                                                                         \
  if (c >= C && (long long)a.V + E - 1 <= 32 * C * E + 32 && a.top <= kWarpTop)             \
    return launch(k_score_warp<F32, C, false, true>, a, blocks, kWarps * 32, 1, st)
    if (a.top > kWarpTop) {
      if (c <= 5) DS_WARP(5, true);
      if (c <= 9) DS_WARP(9, true);
      DS_WARP(16, true);
    }
    DS_TAIL(4);
    if constexpr (F32) DS_TAIL(8);
    if (c <= 1) DS_WARP(1, false);
    if (c <= 2) DS_WARP(2, false);
    if (c <= 3) DS_WARP(3, false);
    if (c <= 5) DS_WARP(5, false);
    if (c <= 7) DS_WARP(7, false);
    if (c <= 9) DS_WARP(9, false);
    if (c <= 12) DS_WARP(12, false);
    DS_WARP(16, false);
#undef DS_TAIL
#undef DS_WARP
  }
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorUnknown;
  // (128 alternatives from the maxima of 128 threads would list half the row)
  if (a.top <= kFewTop) {
    if (nq <= 2048) return launch(k_score_block<F32, 128>, a, a.n, 128, 1, st);
    // (rows of 5001 chunks: 1000 of them 30 us with 256 threads, 38 with 512)
    if (nq <= 4096 || (nq <= 8192 && a.n > 2 * sms)) return launch(k_score_block<F32, 256>, a, a.n, 256, 1, st);
  }
  // slices of at least 4.5 chunks a thread while all CTAs run at once
  int cs = 1;
  while (cs < kMaxCluster && nq / (2 * cs) >= 2304 && 2LL * a.n * cs <= 2LL * sms) cs *= 2;
  return launch(k_score_block<F32, 512>, a, (long long)a.n * cs, 512, cs, st);
}

}  // namespace

cudaError_t launch_score(const ScoreArgs& a, bool f32, cudaStream_t st) {
  return f32 ? launch_rows<true>(a, st) : launch_rows<false>(a, st);
}

}  // namespace ds
