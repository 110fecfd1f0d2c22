// k_linear_i8.cu -- product of 8-bit integers scaled by row and channel:
// out[i][j] = (sum_k a[i][k] w[j][k]) * a_scale[i] * w_scale[j].
//
// The mathematics. Integers of 8 bits are exact in fp16 and their products (at most
// 2^14) in fp32, so the tensor cores' fp16 products with fp32 sums are the integer
// product as long as a running sum stays below 2^24. Beyond, an instruction (16
// inputs) truncates: with operands of one sign and the largest size, 1.8e-4 of the
// sum is lost at K = 131071, 1.1e-4 at 16384 and one unit at 1041. The 8-bit integer
// rate of this GPU is far below its fp16 rate; rows and weights of a model have both
// signs, and their sums stay below 2^24 at any K allowed.
//
// The layout. The weight is the large operand and is read once, as 8 bits. It is
// packed once into blocks of 128 channels x 128 inputs (16 KB, consecutive in memory),
// which bulk copies bring into a ring in shared memory. Warps widen a block (a byte
// permutation and a subtraction for two values) and write it to tensor memory as the
// instruction's first operand, which costs no shared memory and no second pass. The
// rows of a are the second operand: a short kernel before this one writes them as
// fp16 tiles in the swizzled order that the instruction reads, or ds_quantize_rows
// does so itself. So one instruction has 128 channels x `rows` rows x 16 inputs.
// Each of loads, widening, instructions and results has warps of its own, joined by
// mbarriers, and the weight loads start before the row tiles are there.
//   rows <= 128  a CTA per 128 channels. Two accumulators, so that results go out
//                beside the next tile's instructions. A row tile that fits stays in
//                shared memory for all channel blocks.
//   rows > 128   a pair of CTAs per 256 channels, one instruction for both, each with
//                half of the row tile: 96 KB instead of 160 KB through shared memory
//                per block of 128 inputs. One CTA alone took 1150-1190 cycles per block
//                of 1024 of instructions and 172 us where the pair takes 150 (256 rows
//                x 248320 x 2048; 777 x 20011 x 4096: 122 and 94 us).
//
// What bounds it (bf16 out, K and the rest as stated):
//   24 x 248320 x 2048    82 us with its ds_quantize_rows, 522 MB at 6.4 TB/s: HBM
//   256 x 248320 x 2048   150 us, 260 GFLOP at 1.74 PFLOP/s, tensor pipe 79% busy; the
//                         rest is reading the accumulator, 128 KB in 2300-2600 cycles
//                         per tile, and the handing over to the next tile. A warp has
//                         one load of 2 KB in flight and waits for it, so that this may
//                         be latency as well as tensor memory's rate: not told apart
//   777 x 20011 x 4096    94 us, 1.35 PFLOP/s: the same, and 316 tiles on 76 pairs
//   1939 x 8200 x 1024    32 us: tiles of 8 blocks, a third of the time between them
//   one row x 8200 x 1024 8.5 us with its ds_quantize_rows: latency, 65 tiles on 152 SMs
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ds_device.cuh"
#include "ds_launch.h"

namespace ds {

namespace {

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

}  // namespace

// One thread per 16-byte chunk of a packed block.
__global__ void __launch_bounds__(256) k_pack_i8(const int8_t* w, int N, int K, long long ldw, uint8_t* packed) {
  pdl_wait();
  pdl_release();
  const int kb = (K + kPackK - 1) / kPackK;
  const long long chunks = (long long)channel_blocks(N) * kb * (kPackRows * kPackK / 16);
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

// The rows of a as the fp16 tiles that the product reads.
__global__ void __launch_bounds__(256) k_expand_i8(const int8_t* a, long long lda, int n, int K, I8Tiles t) {
  pdl_wait();
  pdl_release();
  const int rows = t.rows, tiles = t.tiles, kb64 = t.kb;
  uint4* out = static_cast<uint4*>(t.out);
  const long long chunks = (long long)tiles * kb64 * rows * 8;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < chunks; i += (long long)gridDim.x * 256) {
    const int c = (int)(i & 7);
    const long long q = i >> 3;
    const int r = (int)(q % rows);
    const int b = (int)(q / rows % kb64);
    const long long row = q / rows / kb64 * rows + r;
    const int k0 = b * 64 + ((c ^ (r & 7)) << 3);
    __half h[8];
    const int8_t* src = a + row * lda + k0;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = __int2half_rn((row < n && k0 + j < K) ? (int)src[j] : 0);
    out[i] = *reinterpret_cast<const uint4*>(h);
  }
}

namespace {

// ------------------------------------------------------------ tensor-core helpers
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("{\n.reg .b64 t;\nmbarrier.arrive.shared::cta.b64 t, [%0];\n}" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("{\n.reg .b64 t;\nmbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n}" ::"r"(smem_u32(b)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier." DS_WAIT_TRY ".parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Arrives at the barrier of the pair's first CTA. What it reports are finished
// bulk copies and tensor-memory accesses (the tcgen05 fences order those), never
// this thread's own writes, so nothing is released to the cluster: that would
// wait for every result this CTA has on its way to memory (1600 cycles and more
// per arrival, 248 us where this takes 160 for 256 rows x 248320 x 2048).
__device__ __forceinline__ void mbar_arrive_first(uint64_t* b) {
  asm volatile(
      "{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %0, 0;\nmbarrier.arrive.shared::cluster.b64 _, [a];\n}" ::"r"(
          smem_u32(b))
      : "memory");
}
// Raises the stop flag of the pair's other CTA as well.
__device__ __forceinline__ void tell_peer(int* flag, uint32_t peer) {
  asm volatile("{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %0, %1;\nst.shared::cluster.u32 [a], %2;\n}" ::"r"(
                   smem_u32(flag)),
               "r"(peer), "r"(1)
               : "memory");
}
// Every wait gives up after a while: it raises the CTA's stop flag, which ends
// the other waits too, and the caller leaves its loop. What the CTA has started is
// then still waited for (mbar_drain), and the results that it owes become NaN.
__device__ __noinline__ bool mbar_wait_slow(uint64_t* b, uint32_t parity, volatile int* stop) {
  for (int i = 0; i < DS_WAIT_TRIES; ++i) {
    if (mbar_try(b, parity)) return true;
    if (*stop) return false;
  }
  *stop = 1;
  return false;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity, volatile int* stop) {
  return mbar_try(b, parity) || mbar_wait_slow(b, parity, stop);
}
// No copy or matrix instruction may be in flight when the CTA leaves its shared
// and tensor memory.
__device__ __forceinline__ void mbar_drain(uint64_t* b, uint32_t parity) {
  for (int i = 0; i < kDrainTries && !mbar_try(b, parity); ++i) {
  }
}
// The same for the last uses of a ring that was used n times.
__device__ __noinline__ void ring_drain(uint64_t* full, uint32_t slots, uint32_t n) {
  for (uint32_t i = n > slots ? n - slots : 0; i < n; ++i) mbar_drain(&full[i % slots], (i / slots) & 1u);
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// True in one thread of the (converged) warp. The compiler knows the branch to be
// taken by one thread, which keeps the operands of the matrix instructions in
// uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// The tiles of a CTA (or pair): channel blocks (or pairs of them) outermost, row
// tiles innermost, one tile in `step`. Without a division between tiles.
struct Walk {
  long long t;
  const uint32_t step, tiles;
  const int d_block, d_tile;
  int block, tile;
  __device__ __forceinline__ Walk(uint32_t first, uint32_t step_, uint32_t tiles_)
      : t(first), step(step_), tiles(tiles_), d_block((int)(step_ / tiles_)), d_tile((int)(step_ % tiles_)),
        block((int)(first / tiles_)), tile((int)(first % tiles_)) {}
  __device__ __forceinline__ void next() {
    t += step;
    block += d_block;
    tile += d_tile;
    if (tile >= (int)tiles) {
      tile -= (int)tiles;
      ++block;
    }
  }
};

// A slot of a ring and the parity of its current use.
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t slots) {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// The barrier (of both CTAs of a pair) hears of the instructions so far when they are done.
template <bool PAIR>
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((unsigned short)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D[128][N] (+)= A[128][16] B[N][16]^T: A in tensor memory, B in shared memory. A
// pair: D[256][N], each CTA with its 128 rows of D and A and its half of B.
template <bool PAIR>
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
// 16 columns of this thread's lane, and the wait for them. The wait names the
// registers, so that no use of them moves above it.
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tc_ld16_wait(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}
// The next 32 columns, `columns` of them read (16 or 32).
__device__ __forceinline__ void tc_ld32(uint32_t addr, int columns, float (&f)[32]) {
  uint32_t v[32];
  tc_ld16(addr, v);
  if (columns > 16) {
    tc_ld16(addr + 16, v + 16);
  } else {
#pragma unroll
    for (int i = 16; i < 32; ++i) v[i] = 0u;
  }
  tc_ld16_wait(v);
  tc_ld16_wait(v + 16);
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
}

// Two results, scaled and rounded to bf16.
__device__ __forceinline__ __nv_bfloat162 scaled2(uint32_t x, uint32_t y, float sx, float sy, float sw) {
  uint32_t r;
  asm("{\n.reg .b64 v, s, w;\n.reg .f32 a, b;\n"
      "mov.b64 v, {%1, %2};\nmov.b64 s, {%3, %4};\nmov.b64 w, {%5, %5};\n"
      "mul.rn.f32x2 v, v, s;\nmul.rn.f32x2 v, v, w;\n"
      "mov.b64 {a, b}, v;\ncvt.rn.bf16x2.f32 %0, b, a;\n}"
      : "=r"(r)
      : "r"(x), "r"(y), "f"(sx), "f"(sy), "f"(sw));
  return *reinterpret_cast<const __nv_bfloat162*>(&r);
}

// Matrix descriptor of a K-major tile with 128-byte swizzle: 8-row groups 1024
// bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Four biased bytes b = w + 128 to four fp16 values w: 0x6400 | b is 1024 + b,
// and 1024 + b - 1152 is exact.
__device__ __forceinline__ void widen4(uint32_t b, uint32_t& lo, uint32_t& hi) {
  const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));
  uint32_t l, h;
  asm("prmt.b32 %0, %1, %2, 0x4140;" : "=r"(l) : "r"(b), "r"(0x64646464u));
  asm("prmt.b32 %0, %1, %2, 0x4342;" : "=r"(h) : "r"(b), "r"(0x64646464u));
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&l), bias), y = __hsub2(*reinterpret_cast<__half2*>(&h), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

constexpr int kTcEpi = 8;   // warps 0-7: results out of tensor memory, two per lane quarter
constexpr int kTcCvt = 8;   // warps 8-15: int8 weights to fp16, two groups of four
constexpr int kTcWarps = kTcEpi + kTcCvt + 3;  // then: weight loads, row loads, matrix instructions
constexpr int kTcNT = kTcWarps * 32;
constexpr int kTcBlock = kPackRows * kPackK;  // bytes of a weight block
constexpr int kTcWSlots = 12;                 // most weight slots
constexpr int kTcBSlots = 32;                 // most row-tile slots
constexpr int kTcASlots = 4;                  // fp16 weight blocks in tensor memory, 64 columns each
constexpr int kTcACol = 256;                  // their first column; accumulators are below
constexpr int kTcPairRows = 128;  // row tiles above this: a pair of CTAs
constexpr int kTcSms = 152;  // SMs that calls are cut for
constexpr size_t kTcSmem = 232448 - 2048;     // dynamic shared memory of a CTA, barriers apart

// The warps that read results: all of them meet, and whether one of their threads says so.
__device__ __forceinline__ void epi_sync() { asm volatile("barrier.sync 1, %0;" ::"n"(kTcEpi * 32) : "memory"); }
__device__ __forceinline__ bool epi_any(bool p) {
  uint32_t any;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.red.or.pred q, 1, %2, p;\nselp.u32 %0, 1, 0, q;\n}"
      : "=r"(any)
      : "r"((uint32_t)p), "n"(kTcEpi * 32)
      : "memory");
  return any != 0;
}

// The CTA's threads, or the pair's, meet.
template <bool PAIR>
__device__ __forceinline__ void all_sync() {
  if (PAIR) {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  } else {
    __syncthreads();
  }
}

// How a call of n rows is cut: row tiles of `rows` (a multiple of 16, at most
// 256), their slots in shared memory, and whether all of a tile's slots stay
// there for every channel block.
struct TcPlan {
  int rows, tiles, kb, b_slots, w_slots, resident, pair;
};

}  // namespace

// Estimated cycles of a call cut into `tiles` row tiles. Measured: an instruction
// takes rows / 2 cycles, but 100 at least (its 4 KB of weights come from tensor
// memory); between tiles lie 1500 cycles and 10 a row, beside the next tile's
// instructions only where two accumulators fit (rows <= 128). The choices that it
// makes and the next ones: 1939 x 8200 x 1024 in 9, 8, 11 tiles 33.4, 35.3, 37.4 us;
// 777 x 20011 x 4096 in 4, 5, 7 tiles 97, 111, 135 us; 256 x 248320 x 2048 in 1, 2
// tiles 151, 220 us.
static long long tc_cycles(int n, int N, int kb, int tiles, int rows) {
  const long long ctas = (long long)channel_blocks(N) * tiles, waves = (ctas + kTcSms - 1) / kTcSms;
  const long long mma = 8LL * kb * (rows > 200 ? rows / 2 : 100), out = 1500 + 10LL * rows;
  return waves * (rows > 128 ? mma + out : mma > out ? mma : out);
}

static TcPlan tc_plan(int n, int N, int K) {
  TcPlan p;
  p.kb = (K + kPackK - 1) / kPackK;
  // as few row tiles as fit, or a few more where that fills the last wave better
  const int least = (int)((n + 255LL) / 256);
  long long best = 0;
  for (int tiles = least; tiles <= least + 8; ++tiles) {
    const int each = (int)(((long long)n + tiles - 1) / tiles), pair = each > kTcPairRows, step = pair ? 32 : 16;
    const int rows = (each + step - 1) / step * step;
    if ((long long)rows * (tiles - 1) >= n) continue;  // its last tile would be empty
    const long long c = tc_cycles(n, N, p.kb, tiles, rows);
    if (tiles == least || c < best) {
      best = c;
      p.tiles = tiles;
      p.rows = rows;
      p.pair = pair;
    }
  }
  const long long room = (long long)kTcSmem - 1024;  // the tiles start on 1024 bytes
  const long long slot = (long long)p.rows * (p.pair ? 64 : 128), all = slot * 2 * p.kb;
  p.resident = !p.pair && p.tiles == 1 && 2 * p.kb <= kTcBSlots && all + 6 * kTcBlock <= room;
  p.b_slots = p.resident ? 2 * p.kb : p.pair ? 8 : 4;
  // An even number: the two converting groups take blocks in turn, and each has
  // to meet every use of the slots it waits on, or a parity of two uses ago
  // would look like the current one.
  const long long w = (room - slot * p.b_slots) / kTcBlock & ~1ll;
  p.w_slots = (int)(w < kTcWSlots ? w : kTcWSlots);
  return p;
}

static_assert(kTcWSlots % 2 == 0 && kTcASlots % 2 == 0, "each converting group keeps its slots");

// One CTA per SM, or one pair of CTAs per two, walks tiles of 128 or 256 channels x
// `rows` rows of a.
template <typename OUT, bool PAIR>
__global__ void __launch_bounds__(kTcNT, 1) k_linear_i8_tc(LinearArgs g, TcPlan p) {
  extern __shared__ uint8_t dyn[];
  __shared__ uint64_t w_full[kTcWSlots], w_empty[kTcWSlots], b_full[kTcBSlots], b_empty[kTcBSlots];
  __shared__ uint64_t a_full[kTcASlots], a_empty[kTcASlots], peer_full[kTcASlots], d_full[2], d_empty[2], drained;
  __shared__ uint32_t tmem_base;
  __shared__ __align__(16) float a_scale[256];
  __shared__ int stop_flag;
  __shared__ uint32_t started[3];  // weight blocks, blocks of row tiles, tiles handed on, once their warp is done
  volatile int* stop = &stop_flag;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint8_t* bs = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
  const uint32_t rank = PAIR ? blockIdx.x & 1u : 0u;
  const uint32_t b_bytes = (uint32_t)p.rows * (PAIR ? 64u : 128u);  // this CTA's rows of a tile's 64 inputs
  uint8_t* ws = bs + (size_t)b_bytes * p.b_slots;
  const int d_bufs = p.rows <= 128 ? 2 : 1;

  if (threadIdx.x == 0) {
    stop_flag = 0;
    for (int i = 0; i < kTcWSlots; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], 4);
    }
    for (int i = 0; i < kTcBSlots; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    for (int i = 0; i < kTcASlots; ++i) {
      mbar_init(&a_full[i], 4);
      mbar_init(&a_empty[i], 1);
      mbar_init(&peer_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], PAIR ? 2 * kTcEpi : kTcEpi);
    }
    mbar_init(&drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    if (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base))
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base))
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  tc_fence_before();
  all_sync<PAIR>();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  // Launched while the kernel that makes the row tiles runs, which in turn started
  // after everything before it on the stream was done: the weights are there, and
  // only what that kernel writes is waited for.
  pdl_release();

  const int kb = p.kb;
  const int blocks = channel_blocks(g.N);
  const long long n_tiles = (long long)(PAIR ? (blocks + 1) / 2 : blocks) * p.tiles;
  const uint32_t t0 = PAIR ? blockIdx.x >> 1 : blockIdx.x, t_step = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (warp == kTcEpi + kTcCvt) {
    // ---- weight blocks, in the order they are used
    if (lane == 0) {
      uint32_t it = 0;
      Ring rw;
      bool ok = true;
      for (Walk at(t0, t_step, p.tiles); ok && at.t < n_tiles; at.next()) {
        // the second CTA of the last pair may have no channels of its own: it reads the first's
        const int own = PAIR ? min(2 * at.block + (int)rank, blocks - 1) : at.block;
        const uint8_t* src = g.packed + (long long)own * kb * kTcBlock;
        for (int b = 0; b < kb; ++b, ++it, rw.next(p.w_slots)) {
          if (it >= (uint32_t)p.w_slots && !mbar_wait(&w_empty[rw.slot], rw.phase ^ 1u, stop)) {
            ok = false;
            break;
          }
          mbar_expect(&w_full[rw.slot], kTcBlock);
          bulk_load(ws + rw.slot * kTcBlock, src + (long long)b * kTcBlock, kTcBlock, &w_full[rw.slot]);
        }
      }
      started[0] = it;
    }
  } else if (warp == kTcEpi + kTcCvt + 1) {
    // ---- row tiles
    if (lane == 0) {
      pdl_wait();
      uint32_t it = 0;
      Ring rb;
      bool ok = true;
      const uint8_t* base = static_cast<const uint8_t*>(g.workspace);
      for (Walk at(t0, t_step, p.tiles); ok && at.t < n_tiles; at.next()) {
        if (p.resident && it > 0) break;
        const uint32_t tile_bytes = (uint32_t)p.rows * 128u;
        const uint8_t* src = base + (long long)at.tile * (2 * kb) * tile_bytes + rank * b_bytes;
        for (int b = 0; b < 2 * kb; ++b, ++it, rb.next(p.b_slots)) {
          if (it >= (uint32_t)p.b_slots && !mbar_wait(&b_empty[rb.slot], rb.phase ^ 1u, stop)) {
            ok = false;
            break;
          }
          mbar_expect(&b_full[rb.slot], b_bytes);
          bulk_load(bs + rb.slot * b_bytes, src + (long long)b * tile_bytes, b_bytes, &b_full[rb.slot]);
        }
      }
      started[1] = it;
    }
  } else if (warp == kTcEpi + kTcCvt + 2) {
    // ---- matrix instructions, by one thread
    if (PAIR && rank == 1) {
      // the pair's first CTA issues them; this one says when its operands are there
      if (elect_one()) {
        Ring ra, rb;
        bool ok = true;
        started[2] = 0;
        for (Walk at(t0, t_step, p.tiles); ok && at.t < n_tiles; at.next())
          for (int b = 0; ok && b < kb; ++b) {
            ok = mbar_wait(&a_full[ra.slot], ra.phase, stop);
            tc_fence_after();
            for (int h = 0; ok && h < 2; ++h) {
              ok = mbar_wait(&b_full[rb.slot], rb.phase, stop);
              rb.next(p.b_slots);
            }
            tc_fence_before();
            if (ok) mbar_arrive_first(&peer_full[ra.slot]);
            ra.next(kTcASlots);
          }
      }
    } else if (elect_one()) {
      // fp32 accumulators, fp16 operands, M = 128 or 256, N = rows
      const uint32_t idesc =
          (1u << 4) | ((uint32_t)(p.rows >> 3) << 17) | ((uint32_t)((PAIR ? 2 : 1) * kPackRows >> 4) << 24);
      const uint64_t b_desc = sw128_desc(smem_u32(bs));
      const uint32_t b_step = b_bytes >> 4;
      Ring ra, rb, rd;
      uint32_t handed = 0;  // tiles
      bool ok = true, loaded = false;
      for (Walk at(t0, t_step, p.tiles); ok && at.t < n_tiles; at.next()) {
        ok = mbar_wait(&d_empty[rd.slot], rd.phase ^ 1u, stop);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + rd.slot * 128u;
        uint32_t accumulate = 0;
        for (int b = 0; ok && b < kb; ++b) {
          ok = mbar_wait(&a_full[ra.slot], ra.phase, stop) &&
               (!PAIR || mbar_wait(&peer_full[ra.slot], ra.phase, stop));
          if (!ok) break;
          tc_fence_after();
          const uint32_t acol = tmem + kTcACol + ra.slot * 64u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!loaded) {
              ok = mbar_wait(&b_full[rb.slot], rb.phase, stop);
              if (!ok) break;
            }
            const uint64_t bd = b_desc + (uint64_t)(rb.slot * b_step);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              tc_mma<PAIR>(d, acol + (uint32_t)(h * 32 + k * 8), bd + (uint64_t)(k * 2), idesc, accumulate);
              accumulate = 1;
            }
            if (!p.resident) tc_commit<PAIR>(&b_empty[rb.slot]);
            rb.next(p.b_slots);
          }
          if (ok) tc_commit<PAIR>(&a_empty[ra.slot]);
          ra.next(kTcASlots);
        }
        if (ok) {
          tc_commit<PAIR>(&d_full[rd.slot]);
          ++handed;
        }
        rd.next(d_bufs);
        loaded = p.resident;  // a resident row tile has a slot for each of its blocks: the ring is back at the first
      }
      started[2] = handed;
      if (!ok) {
        tc_commit<PAIR>(&drained);  // of a tile that was not handed on
        mbar_drain(&drained, 0);
      }
    }
  } else if (warp >= kTcEpi) {
    // ---- weights to fp16: a group of four warps takes every second block, a
    // thread one channel of it
    const int group = (warp - kTcEpi) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    uint32_t it = 0, s = group, s_phase = 0;  // s: the slot of this group's block, every second of the even ring
    bool ok = true;
    for (Walk at(t0, t_step, p.tiles); ok && at.t < n_tiles; at.next()) {
      for (int b = 0; b < kb; ++b, ++it) {
        if ((int)(it & 1) != group) continue;
        const uint32_t sa = it % kTcASlots, use = it / kTcASlots;
        ok = __all_sync(0xffffffffu, mbar_wait(&w_full[s], s_phase, stop));
        if (!ok) break;
        const uint8_t* src = ws + (size_t)s * kTcBlock + row * 128;
        uint32_t v[2][32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + ((c ^ (row & 7)) << 4));
          uint32_t* o = &v[c >> 2][(c & 3) * 8];
          widen4(x.x, o[0], o[1]);
          widen4(x.y, o[2], o[3]);
          widen4(x.z, o[4], o[5]);
          widen4(x.w, o[6], o[7]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&w_empty[s]);
        s += 2;
        if (s >= (uint32_t)p.w_slots) {
          s -= p.w_slots;
          s_phase ^= 1u;
        }
        if (use > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(&a_empty[sa], (use - 1) & 1, stop));
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t dst = tmem + ((uint32_t)(quad * 32) << 16) + kTcACol + sa * 64u;
        tc_st32(dst, v[0]);
        tc_st32(dst + 32, v[1]);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&a_full[sa]);
      }
    }
  } else {
    // ---- results: a thread has one channel, a column of tensor memory is one row of a
    const int quad = warp & 3, half = warp >> 2;
    Ring rd;
    int scales = -1;  // row tile whose scales are in shared memory
    pdl_wait();
    Walk at(t0, t_step, p.tiles);
    auto channel = [&] { return (PAIR ? 2LL * at.block + rank : (long long)at.block) * kPackRows + quad * 32 + lane; };
    for (; at.t < n_tiles; at.next()) {
      const long long j = channel();
      const long long i0 = (long long)at.tile * p.rows;
      const float sw = j < g.N ? g.w_scale[j] : 0.f;
      const bool gone = !mbar_wait(&d_full[rd.slot], rd.phase, stop) || *stop;
      if (epi_any(gone)) break;  // all of these warps or none: they meet at barriers below
      tc_fence_after();
      if (at.tile != scales) {
        for (int i = threadIdx.x; i < p.rows; i += kTcEpi * 32) a_scale[i] = i0 + i < g.n ? g.a_scale[i0 + i] : 0.f;
        epi_sync();
        scales = at.tile;
      }
      const uint32_t src = tmem + ((uint32_t)(quad * 32) << 16) + rd.slot * 128u;
      const int rows = (int)(g.n - i0 < p.rows ? g.n - i0 : p.rows);  // of this tile
      // the two warps of a quarter take 32 columns in turn
      OUT* out = static_cast<OUT*>(g.out) + (i0 + 32 * half) * g.ldo + j;
      auto freed = [&] {  // the accumulator may be written again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_first(&d_empty[rd.slot]);
          else
            mbar_arrive(&d_empty[rd.slot]);
        }
      };
      if constexpr (PAIR && sizeof(OUT) == 2) {
        // There is one accumulator: all of it into registers first, rounded, and to
        // memory beside the next tile's instructions.
        __nv_bfloat162 held[4][16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = 32 * half + 64 * q + 16 * h;
            if (c < p.rows) {
              uint32_t v[16];
              tc_ld16(src + c, v);
              tc_ld16_wait(v);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 sa = reinterpret_cast<const float4*>(a_scale + c)[i];
                held[q][8 * h + 2 * i] = scaled2(v[4 * i], v[4 * i + 1], sa.x, sa.y, sw);
                held[q][8 * h + 2 * i + 1] = scaled2(v[4 * i + 2], v[4 * i + 3], sa.z, sa.w, sw);
              }
            }
          }
        }
        freed();
        if (j < g.N) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int left = rows - (32 * half + 64 * q);
            OUT* o = out + 64 * q * g.ldo;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (2 * i < left) *o = held[q][i].x;
              o += g.ldo;
              if (2 * i + 1 < left) *o = held[q][i].y;
              o += g.ldo;
              asm volatile("" : "+l"(o));  // stepped, not 32 row offsets kept in registers
            }
          }
        }
      } else {
        for (int c = 32 * half; c < p.rows; c += 64, out += 64 * g.ldo) {
          float f[32];
          tc_ld32(src + c, p.rows - c, f);
          const int left = rows - c;
          if (j < g.N) {
            if (left >= 32) {
#pragma unroll
              for (int i = 0; i < 32; ++i) store_out(out + i * g.ldo, f[i] * a_scale[c + i] * sw);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i < left) store_out(out + i * g.ldo, f[i] * a_scale[c + i] * sw);
            }
          }
        }
        freed();
      }
      rd.next(d_bufs);
    }
    // given up: the rest of this CTA's results
    for (; at.t < n_tiles; at.next()) {
      const long long j = channel(), i0 = (long long)at.tile * p.rows;
      if (j < g.N)
        for (long long i = i0 + half; i < g.n && i < i0 + p.rows; i += 2)
          store_out(static_cast<OUT*>(g.out) + i * g.ldo + j, __int_as_float(0x7fffffff));
    }
  }

  tc_fence_before();
  if (PAIR && *stop) tell_peer(&stop_flag, rank ^ 1u);
  all_sync<PAIR>();  // of a pair, neither leaves while the other may still use its memory
  if (*stop) {
    // Given up, and whoever did may have left the others' work in flight.
    if (threadIdx.x == 0) ring_drain(w_full, p.w_slots, started[0]);
    if (threadIdx.x == 32) ring_drain(b_full, p.b_slots, started[1]);
    if (threadIdx.x == 64) ring_drain(d_full, d_bufs, started[2]);
    all_sync<PAIR>();
  }
  tc_fence_after();
  if (warp == 0) {
    if (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
  if (threadIdx.x == 0 && stop_flag) report(g.d_status, DS_DEV_ERR_TIMEOUT);
}

long long linear_i8_workspace(int n, int N, int K) {
  const TcPlan p = tc_plan(n, N, K);
  return (long long)p.tiles * p.rows * p.kb * kPackK * 2;
}

I8Tiles linear_i8_tiles(int n, int N, int K, void* workspace) {
  const TcPlan p = tc_plan(n, N, K);
  return {workspace, p.rows, p.tiles, 2 * p.kb};
}

cudaError_t launch_pack_i8(const int8_t* w, int N, int K, int64_t ldw, uint8_t* packed, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorUnknown;
  const long long chunks = (long long)channel_blocks(N) * ((K + kPackK - 1) / kPackK) * 1024;
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
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorUnknown;
  const TcPlan p = tc_plan(g.n, g.N, g.K);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;

  cudaError_t e;
  if (g.a) {
    const long long chunks = (long long)p.tiles * 2 * p.kb * p.rows * 8, want = (chunks + 255) / 256;
    cfg.gridDim = dim3((unsigned)(want < sms * 8LL ? want : sms * 8LL));
    cfg.blockDim = dim3(256);
    e = cudaLaunchKernelEx(&cfg, k_expand_i8, g.a, (long long)g.lda, g.n, g.K,
                           linear_i8_tiles(g.n, g.N, g.K, g.workspace));
    if (e != cudaSuccess) return e;
    note_launch();
  }

  auto kern = p.pair ? (bf16_out ? k_linear_i8_tc<__nv_bfloat16, true> : k_linear_i8_tc<float, true>)
                     : (bf16_out ? k_linear_i8_tc<__nv_bfloat16, false> : k_linear_i8_tc<float, false>);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = p.pair ? 2 : 1;
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kTcNT);
  cfg.dynamicSmemBytes = kTcSmem;
  const int fit = cached(reinterpret_cast<const void*>(kern), -1, [&](int) {
    int v = 0;
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmem);
    if (r == cudaSuccess && p.pair) r = cudaOccupancyMaxActiveClusters(&v, kern, &cfg);
    if (r != cudaSuccess) (void)cudaGetLastError();
    return r != cudaSuccess ? 0 : p.pair ? v : sms;
  });
  if (fit <= 0) return cudaErrorUnknown;
  const long long blocks = channel_blocks(g.N);
  const long long tiles = (p.pair ? (blocks + 1) / 2 : blocks) * p.tiles, ctas = tiles < fit ? tiles : fit;
  cfg.gridDim = dim3((unsigned)(p.pair ? 2 * ctas : ctas));
  e = cudaLaunchKernelEx(&cfg, kern, g, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace ds
