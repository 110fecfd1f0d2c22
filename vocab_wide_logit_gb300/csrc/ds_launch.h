// ds_launch.h -- internal launch entry points of the libdsample kernels.
#pragma once

#include <cuda_runtime.h>

#include "dsample.h"
#include "ds_device.cuh"

namespace ds {

// Counts every kernel the library launches (read by ds_launch_count).
void note_launch();

// Launch-time queries (a kernel's occupancy, its shared-memory attribute, the
// SM count) cost microseconds of host time each; their answers depend only on
// the device, the kernel and its shared memory. cached(site, param, init) runs
// init(device) the first time a (site, current device, param) key is seen and
// returns its positive result from then on (a result <= 0 is an error and is
// not kept). Thread-safe.
bool cache_lookup(const void* site, int dev, long long param, int* value);
void cache_store(const void* site, int dev, long long param, int value);
template <typename F>
int cached(const void* site, long long param, F init) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  int v = 0;
  if (cache_lookup(site, dev, param, &v)) return v;
  v = init(dev);
  if (v > 0) cache_store(site, dev, param, v);
  return v;
}
// SM count of the current device (cached).
int device_sms();

// How often a wait inside a serving-head kernel asks before it gives up, and the
// instruction that asks. Another build (no second time, and without the suspension
// that try_wait may add) makes waits run out, to test what is left then.
#ifndef DS_WAIT_TRIES
#define DS_WAIT_TRIES (1 << 20)
#define DS_WAIT_TRY "try_wait"
#endif
// A kernel that has given up asks this often for its own copies and instructions
// in flight before it leaves.
constexpr int kDrainTries = 1 << 20;

constexpr int kWarpKernelThreads = 128;
constexpr int kStreamMark = DS_MARKED_TOKEN;  // out_tokens marker left by a fast pass for the exact one

// Largest V of the one-warp-per-cell kernel and of the cluster kernel.
int warp_kernel_max_vocab();
int cluster_kernel_max_vocab();

// One warp per cell: a lean pass that marks the cells it cannot settle on its
// common path (too few or too many candidates for its balanced list), then
// (exact_pass) the full kernel over the marked cells only.
cudaError_t launch_sample_warp(const SampleArgs& a, cudaStream_t st, int num_sms, bool exact_pass);

// Staged cluster kernel (z kept in shared memory); with only_marked it finishes
// just the cells the streaming kernel marked with kStreamMark.
cudaError_t launch_sample_cluster(const SampleArgs& a, cudaStream_t st, int only_marked);
// Streaming cluster kernel (candidates only in shared memory) for k well below V.
cudaError_t launch_sample_stream(const SampleArgs& a, cudaStream_t st);
cudaError_t launch_greedy(const uint16_t* x, int n, int V, float* out_max, float* out_lse, int* out_argmax,
                          cudaStream_t st);
cudaError_t launch_merge_triples(const float* triples, int n, int shards, float* out_max, float* out_lse,
                                 int* out_argmax, cudaStream_t st);
cudaError_t launch_reveal(const float* scores, const int32_t* tokens, const int32_t* seq_lens,
                          const int32_t* reveal_counts, int B, int C, int P, int32_t* canvas, uint8_t* revealed,
                          uint32_t* d_status, cudaStream_t st);
cudaError_t launch_log_softmax_write(const uint16_t* x, int n, int V, const float* lse, void* out, bool bf16_out,
                                     cudaStream_t st);

// Dense log-softmax with each row held in a cluster's shared memory (one read of
// the logits); fits when a row splits into at most 8 slices of 64 KB. When no
// cluster of the needed shape fits the device, *refused is set, nothing is
// launched and cudaSuccess is returned.
bool log_softmax_fused_fits(int V);
cudaError_t launch_log_softmax_fused(const uint16_t* x, int n, int V, float* out_max, float* out_lse,
                                     int* out_argmax, void* out, bool bf16_out, cudaStream_t st, bool* refused);

// Filtered sampling of n rows of V logits, ld elements apart.
struct FilteredArgs {
  const void* x;  // bf16 or fp32
  int64_t ld;
  int32_t n, V;
  const float* temperature;
  const int32_t* top_k;  // or null
  const float* top_p;    // or null
  const float* min_p;    // or null
  const float* u;
  int32_t* out_tokens;
  float* out_logprobs;
  uint32_t* d_status;
};
cudaError_t launch_sample_filtered(const FilteredArgs& a, bool f32, cudaStream_t st);

// The left operand of the product of 8-bit integers as fp16: [row tile][block of
// 64 inputs][row][128 bytes], 16-byte chunk c of row i at chunk c ^ (i & 7) (the
// 128-byte swizzle of the matrix descriptors). Rows and inputs past the end are
// zero: a zero weight does not cancel a NaN left in the workspace.
struct I8Tiles {
  void* out;
  int rows, tiles, kb;  // rows of a tile, tiles, blocks of 64 inputs
};

// Rows of x (optionally RMS-normalised) to int8 with one scale per row: to q, or
// as such tiles when given.
cudaError_t launch_quantize_rows(const void* x, bool f32, int n, int K, int64_t ld, const float* gain, float eps,
                                 int8_t* q, float* scale, const I8Tiles* tiles, cudaStream_t st);

// The packed form of an int8 weight [N][K]: blocks of kPackRows channels x
// kPackK inputs, 16 KB each, block (channels / kPackRows, inputs / kPackK) at
// index (channel block) * (input blocks) + (input block). In a block, channel r
// has 128 bytes at r * 128; its 16-byte chunk c stands at chunk c ^ (r & 7), so
// that eight threads reading the same chunk of eight channels meet no bank
// twice. Bytes hold w + 128, channels and inputs beyond N and K hold 128 (zero).
constexpr int kPackRows = 128;
constexpr int kPackK = 128;
__host__ __device__ constexpr int channel_blocks(int N) { return (int)((N + (kPackRows - 1LL)) / kPackRows); }
static_assert(channel_blocks(2147483647) == 16777216, "counted beyond 32 bits");
cudaError_t launch_pack_i8(const int8_t* w, int N, int K, int64_t ldw, uint8_t* packed, cudaStream_t st);

struct LinearArgs {
  const int8_t* a;
  int64_t lda;
  const float* a_scale;
  const uint8_t* packed;
  const float* w_scale;
  int32_t n, N, K;
  void* out;
  int64_t ldo;
  void* workspace;
  uint32_t* d_status;
};
long long linear_i8_workspace(int n, int N, int K);
I8Tiles linear_i8_tiles(int n, int N, int K, void* workspace);
// With g.a null the workspace holds the tiles already.
cudaError_t launch_linear_i8(const LinearArgs& a, bool bf16_out, cudaStream_t st);

// Scores of given tokens in n rows of V logits, ld elements apart.
struct ScoreArgs {
  const void* x;  // bf16 or fp32
  int64_t ld;
  int32_t n, V, top;
  const int32_t* tokens;
  float* out_logprobs;
  float* out_lse;      // or null
  float* out_entropy;  // or null
  int32_t* out_ranks;  // or null
  int32_t* out_top_ids;     // null without alternatives
  float* out_top_logprobs;  // the same
  uint32_t* d_status;
};
cudaError_t launch_score(const ScoreArgs& a, bool f32, cudaStream_t st);

struct ScoreGradArgs {
  const void* x;  // bf16 or fp32, as the result
  int64_t ld;
  int32_t n, V;
  const int32_t* tokens;
  const float* lse;
  const float* entropy;     // null without g_entropy
  const float* g_logprobs;  // or null
  const float* g_entropy;   // or null
  void* out;
  int64_t ldo;
  uint32_t* d_status;
};
cudaError_t launch_score_grad(const ScoreGradArgs& a, bool f32, cudaStream_t st);

// Low-rank adapters added to n rows of N logits.
struct AdapterArgs {
  const void* base;  // bf16 or fp32, as the result
  int64_t ldb;
  const void* x;  // bf16 or fp32
  int64_t ldx;
  const float* gain;  // or null
  float eps;
  const uint16_t* a;  // [L][R][K]
  const uint16_t* b;  // [L][N][R]
  const float* scale;
  const int32_t* ids;
  int32_t n, N, K, L, R;
  void* out;
  int64_t ldo;
  void* workspace;
  uint32_t* d_status;
};
long long adapters_workspace(int n, int L, int R);
cudaError_t launch_add_adapters(const AdapterArgs& a, bool x_f32, bool f32, cudaStream_t st);

}  // namespace ds
