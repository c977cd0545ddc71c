// Host-side helpers shared by the files that implement the C ABI (defined in cce_api.cu). Not installed.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "cce.h"

namespace cce {

constexpr size_t kHeaderBytes = 256;  // start of every workspace: WsHeader
constexpr size_t kAlign = 256;        // of every array in a workspace

// Layout of the area at the start of every workspace (zeroed by every call).
struct WsHeader {
  int err;   // device error word
  int done;  // blocks of the forward's finish kernel that are done
  int bar;   // grid barrier counter of the backward's planning launch
  int failed;  // set by the head kernel when a bounded wait ran out
};

// Sets the message of cce_last_error_message() and returns s.
cce_status fail(cce_status s, const char* fmt, ...);
cce_status cuda_fail(cudaError_t e, const char* what);
void clear_last_error();

// Compute capability and the number of SMs of the current device; the tensor-map encoder of the driver.
cce_status check_device(int* num_sms);
cce_status get_encoder();

// 2-D row-major tensor [rows, cols] with contiguous rows, box [box_rows, box_cols], 128B swizzle.
cce_status make_map(CUtensorMap* map, CUtensorMapDataType dtype, size_t elem, const void* ptr, int64_t rows,
                    int64_t cols, uint32_t box_cols, uint32_t box_rows);

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

// What the backward of the log-probabilities differs in from the loss's (cce_logprobs_backward): the gradient
// of a row's logits comes from the gradients of its log-probabilities and its entropy.
struct LogprobGrads {
  const int64_t* tokens;      // [N, K]
  int64_t ignore_index;
  int K;
  float temperature;
  const float* lse;           // [N] of the logits over the temperature
  const float* row_stats;     // [2, N], see cce_logprobs_stats(), or null
  const float* entropy;       // [N]
  const float* logprobs;      // [N, K]
  const float* g_logprobs;    // [N, K] or null (zeros)
  const float* g_entropy;     // [N] or null
  int dbias_fp32;             // dbias in fp32 whatever the other outputs' type
};
size_t logprobs_backward_bytes(const cce_problem* p, int K, int32_t out_fp32);
cce_status logprobs_backward(const cce_problem* p, const LogprobGrads& g, const void* E, const void* C,
                             const void* bias, const float* tile_max, float filter_eps, void* dE, void* dC, void* dbias,
                             int32_t out_fp32, int64_t* filtered_tiles, void* workspace, size_t workspace_bytes,
                             cudaStream_t s);

}  // namespace cce

#define CCE_TRY(expr)                                        \
  do {                                                       \
    cudaError_t e_ = (expr);                                 \
    if (e_ != cudaSuccess) return cce::cuda_fail(e_, #expr); \
  } while (0)

#define CCE_CHECK(expr)          \
  do {                           \
    cce_status s_ = (expr);      \
    if (s_ != CCE_OK) return s_; \
  } while (0)
