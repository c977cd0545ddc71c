// Internal interface of the head operators (log-probabilities of given tokens with entropy, top
// alternatives, the 8-bit product): the kernels of cce_head.cu and their host side in cce_head_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <stdint.h>

#include "cce_internal.h"

namespace cce {

constexpr int kHeadBM = 128;       // rows of a logit tile
constexpr int kHeadBN = 256;       // vocabulary columns of a logit tile
constexpr int kHeadUnit = 64;      // smallest unit of the split
constexpr int kHeadGroup = 32;     // row blocks that walk the vocabulary together (their E stays in L2)
constexpr int kHeadMaxTokens = 32; // given tokens a row
constexpr int kHeadMaxTop = 24;    // alternatives a row
constexpr int kHeadParts = 4;      // epilogue warps of a row: partial statistics of a segment
constexpr int kHeadPick = 16;      // columns of a pick: the unit whose largest logit is kept for the alternatives
constexpr int kHeadDotRows = 64;   // rows of a work item of head_dots_kernel
constexpr int kHeadSlab = 4096;    // rows whose alternatives are found at a time: bounds their workspace

constexpr int kHeadMaxGrid = 148;  // SMs of a B200

// How the logit tiles are split over the blocks of the grid. Row blocks are taken in `ngroups` groups of
// nearly equal size. A group's work is the list of its units (`unit` vocabulary columns of one row
// block), row block by row block; part c of the P = min(grid, units) parts gets the units
// [c U / P, (c + 1) U / P), and one block walks it. What a block gets of one row block is a segment: it
// keeps the softmax statistics of the segment on chip and writes them once.
struct HeadSplit {
  int nb;       // row blocks
  int nu;       // units of a row block
  int unit;     // columns of a unit: a multiple of 64
  int ngroups;
  int grid;     // at most kHeadMaxGrid
  // Which part a block takes, for the smaller groups and for those with one row block more: by where in the
  // vocabulary the part starts. Neighbouring blocks (two SMs that share a path to L2) then walk the same columns of
  // C on different row blocks, and what both load at a time crosses from L2 once (2048 x 2048 x 128256: 256
  // million sectors, against 334 million in the parts' own order, where neighbours share rows of E instead).
  uint8_t order[2][kHeadMaxGrid];

  __host__ __device__ int group_begin(int g) const {
    return static_cast<int>(static_cast<long long>(nb) * g / ngroups);
  }
  __host__ __device__ int units(int rows) const { return rows * nu; }
  __host__ __device__ int parts(int total) const { return total < grid ? total : grid; }
  __host__ __device__ static int part_begin(int c, int total, int P) {
    return static_cast<int>(static_cast<long long>(total) * c / P);
  }
  // The part that holds unit x: the largest c with part_begin(c) <= x.
  __host__ __device__ static int owner(int x, int total, int P) {
    return static_cast<int>(((static_cast<long long>(x) + 1) * P - 1) / total);
  }
  // At most this many segments a row block.
  __host__ __device__ int max_segments() const {
    const int rows = nb / ngroups < 1 ? 1 : nb / ngroups;  // the smallest group
    return (grid + rows - 1) / rows + 1;
  }
};

struct HeadArgs {
  HeadSplit split;
  int N, D, V;
  int num_kb;    // K-blocks of 128 bytes
  int kb_chunk;  // K-blocks summed in one tensor-memory accumulator
  int e_rows;    // rows of E a TMA box
  const __nv_bfloat16* bias;  // [V] or null
  const float* e_scale;       // [N], [V]: scales of 8-bit operands
  const float* c_scale;
  const int64_t* tokens;      // [N, K]
  const int* tok_t;           // [K, N]: each row's tokens in ascending order, kNoToken for none (K > 1)
  int64_t ignore_index;
  int K;
  float* zt;        // [K, N]: logits of the given tokens, in the order of tok_t
  float* tile_max;  // [ceil(V / 64), max_pitch]: largest y of each 64 columns, or null
  int64_t max_pitch;
  float* pick_max;  // [N, picks]: largest logit of each pick, or null
  int picks;        // a multiple of 4, at least the number of picks
  float inv_t;      // 1 / temperature
  float* part_m;    // [4 segments, N]: largest logit, sum of 2^d, sum of d 2^d, see cce_head.cu
  float* part_s;
  float* part_w;
  void* out;        // [N, V] logits (8-bit product)
  int out_fp32;
  int out_tma;      // rows of out start on 16-byte boundaries
  int* err;
  int* failed;      // set when a bounded wait ran out
  int clear;        // the first head kernel of a call clears both
  uint64_t timeout_ns;
  int inject_stall;
};

// The picks of every row, their rows and logits (cce_head.cu: alternatives).
struct HeadPicks {
  int N, D, V;
  const void* E;  // bf16 or 8-bit rows
  const void* C;
  const float* e_scale;
  const float* c_scale;
  const __nv_bfloat16* bias;
  const float* pick_max;  // [N, picks]
  int picks;
  int wanted;       // picks a row, at most 32
  int grouped;      // whether equal picks of several rows are brought together
  int* done;        // [2]: blocks done (zero before), work items
  int* count;       // [picks], zero before: rows that want the pick
  int* base;        // [picks]: their place in rows
  int* pick;        // [N, 32]: the rows' picks, -1 for none
  int* slot;        // [N, 32]: place among the pick's rows
  int* rows;        // [32 N]: 32 row + j
  int3* items;      // [32 N]: pick, first of its rows, how many
  float* logits;    // [N, 32, 16]
  float* norm;      // [N, 32]: largest norm of the pick's rows of C (bf16)
};

struct HeadMaps {
  CUtensorMap E;    // box of e_rows rows x 128 bytes
  CUtensorMap C;    // box of 256 rows
  CUtensorMap C64;  // box of 64 rows
  CUtensorMap out;  // logits, box of 16 rows x 128 bytes (HeadArgs.out_tma)
};

struct HeadFinish {
  HeadSplit split;
  int N, D, V;
  const __nv_bfloat16* E;  // for the order of close alternatives: bf16 operands, or the 8-bit ones
  const __nv_bfloat16* C;
  const int8_t* E8;
  const int8_t* C8;
  const float* e_scale;
  const float* c_scale;
  const __nv_bfloat16* bias;
  const int64_t* tokens;
  int64_t ignore_index;
  int K;
  const float* zt;
  float inv_t;
  const float* part_m;
  const float* part_s;
  const float* part_w;
  const int* pick;
  const float* logits;  // of the picks
  const float* norm;    // HeadPicks.norm
  int wanted;
  int top_k;
  int after_dots;    // it follows head_dots_kernel, and may read what the head kernel wrote before that has ended
  float* logprobs;   // [N, K]
  float* entropy;    // [N]
  float* lse;        // [N]
  float* row_max;    // [N] or null: largest logit, and ln of the sum of exp(y - y_max)
  float* row_ln_s;
  float* top_logprobs;  // [N, top_k]
  int64_t* top_ids;
  int* err;
  const int* failed;
};

cudaError_t launch_head(const HeadMaps& M, const HeadArgs& A, bool int8, bool after_kernel, cudaStream_t s);
// Up to this many rows every pick is computed for its row alone: the rows' picks are then nearly all different, and
// bringing equal ones together costs more (a launch, and a chain of atomics in the one before) than it saves. Alone
// and together, 20 alternatives, us: 16 x 4096 x 128256: 211, 222; 96 x 1024 x 50257: 63, 68; 128 x 2048 x 128256:
// 162, 166; 160 x 2048 x 128256: 211, 211; 200 x 2048 x 50257: 149, 128.
constexpr int kUngroupedRows = 128;
inline bool picks_grouped(int64_t rows) { return rows > kUngroupedRows; }
// These two follow a kernel of the same call on s. With picks_grouped the counters are zero before.
// The first also launches the finish.
cudaError_t launch_head_picks(HeadPicks P, const HeadFinish& F, bool int8, int sms, cudaStream_t s);
cudaError_t launch_head_finish(HeadFinish F, cudaStream_t s);
cudaError_t launch_head_tokens(const int64_t* tokens, int N, int K, int V, int64_t ignore_index, int* tok_t,
                               cudaStream_t s);
// Rows of 8-bit integers: scale = max |x| / 127, q = x / scale to the nearest integer.
cudaError_t launch_quantize_rows(const __nv_bfloat16* x, int64_t rows, int64_t D, int8_t* q, float* scale,
                                 cudaStream_t s);

}  // namespace cce
