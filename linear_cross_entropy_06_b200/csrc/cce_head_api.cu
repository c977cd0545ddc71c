// C ABI of the head operators (declared in include/cce.h): log-probabilities of given tokens with
// entropy and top alternatives, their backward, and the product with a classifier of 8-bit integers.
// Argument checks, workspace carving, tensor maps and the launches. Host code only.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "cce.h"
#include "cce_head.h"
#include "cce_host.h"
#include "cce_internal.h"

namespace {

using cce::aligned16;
using cce::align_up;
using cce::ceil_div;
using cce::fail;

// Largest width of 8-bit operands: 127 * 127 * D stays below 2^31.
constexpr int64_t kInt8MaxD = 131072;
bool sizes_ok(int64_t N, int64_t D, int64_t V, bool int8, bool set_error) {
  auto bad = [&](const char* msg) {
    if (set_error) fail(CCE_ERR_INVALID_ARG, "%s", msg);
    return false;
  };
  if (N < 0) return bad("N must be >= 0");
  if (V < 1) return bad("V must be >= 1");
  if (int8 && (D < 16 || D % 16 != 0)) return bad("D must be a positive multiple of 16 for 8-bit operands");
  if (int8 && D > kInt8MaxD) return bad("D too large for 8-bit operands");
  if (D < 8 || D % 8 != 0) return bad("D must be a positive multiple of 8");
  if (N >= (int64_t(1) << 31) - 256 || V >= (int64_t(1) << 31) - 256 || D >= (int64_t(1) << 24))
    return bad("N, V or D too large");
  return true;
}

bool logprobs_ok(const cce_logprob_problem* p, bool set_error) {
  auto bad = [&](const char* msg) {
    if (set_error) fail(CCE_ERR_INVALID_ARG, "%s", msg);
    return false;
  };
  if (p == nullptr) return bad("problem is NULL");
  if (!sizes_ok(p->N, p->D, p->V, p->int8 != 0, set_error)) return false;
  if (p->int8 != 0 && p->int8 != 1) return bad("int8 must be 0 or 1");
  if (p->num_tokens < 0 || p->num_tokens > cce::kHeadMaxTokens) return bad("num_tokens must be in [0, 32]");
  if (p->top_k < 0 || p->top_k > cce::kHeadMaxTop) return bad("top_k must be in [0, 24]");
  if (p->top_k > p->V) return bad("top_k must not exceed V");
  if (p->num_tokens == 0 && p->top_k == 0) return bad("num_tokens and top_k are both 0: nothing to compute");
  // (beyond these, differences of logits over the temperature leave the range of fp32)
  if (!(p->temperature >= 1e-6f && p->temperature <= 1e6f)) return bad("temperature must be in [1e-6, 1e6]");
  if (p->reserved != 0) return bad("reserved must be 0");
  return true;
}

// The split of the logit tiles over `sms` blocks. With at least kWideTiles tiles a block, units of a whole tile: a
// block's share is uneven by at most one tile in that many, and the walk can be aligned. With fewer, units of 64
// columns, so that the blocks' shares stay even. Whole tiles and 64 columns, us: 4.3 tiles a block (513 x 1032 x
// 32003) 66, 62; 16 (1500 x 1024 x 50257) 157, 163; 54 (2048 x 2048 x 128256, 8-bit logits) 512, 576; between 6 and
// 16 tiles of 2048-long rows nothing within the noise of 3 %.
constexpr int64_t kWideTiles = 12;

cce::HeadSplit make_split(int64_t N, int64_t V, int sms) {
  cce::HeadSplit S;
  S.nb = static_cast<int>(ceil_div(N, cce::kHeadBM));
  S.ngroups = static_cast<int>(ceil_div(S.nb, cce::kHeadGroup));
  S.grid = sms;
  const int64_t rows = std::max<int64_t>(S.nb / std::max(S.ngroups, 1), 1);
  const bool wide = rows * ceil_div(V, cce::kHeadBN) >= kWideTiles * sms;
  S.unit = wide ? cce::kHeadBN : cce::kHeadUnit;
  S.nu = static_cast<int>(ceil_div(V, S.unit));
  // Small problems: the same number of parts for every row block. The row blocks' parts then start at the same
  // columns, and each column of C is read from HBM once (777 x 1288 x 50257: 138 us against 173 with even shares for
  // all SMs; with 15 row blocks, which leave the most SMs idle, 13 of 148: 1920 x 1024 x 16000 62 against 66). With
  // wide units the walk itself is aligned (for_tiles), and idle SMs cost more than that leaves to gain (2048 x 2048 x
  // 128256: 906 us against 889 on the same machine).
  if (!wide && S.ngroups == 1 && sms >= S.nb) S.grid = sms / S.nb * S.nb;
  return S;
}

// Parts by where they start in the vocabulary: counted into 256 equal stretches of it (nearer than that their order
// does not matter).
void order_parts(cce::HeadSplit* S) {
  for (int k = 0; k < 2; ++k) {
    const int total = S->units(S->nb / S->ngroups + k), P = S->parts(total);
    uint8_t stretch[cce::kHeadMaxGrid];
    int place[257] = {};
    for (int i = 0; i < P; ++i) {
      const int64_t start = cce::HeadSplit::part_begin(i, total, P) % S->nu;
      stretch[i] = static_cast<uint8_t>(start * 256 / S->nu);
      ++place[stretch[i] + 1];
    }
    for (int i = 0; i < 256; ++i) place[i + 1] += place[i];
    for (int i = 0; i < P; ++i) S->order[k][place[stretch[i]]++] = static_cast<uint8_t>(i);
    if (S->nb % S->ngroups == 0) break;  // every group has the same number of row blocks
  }
}

constexpr int kMaxSms = cce::kHeadMaxGrid;  // the workspace is sized for it; a device with fewer SMs needs no more

int picks_pitch(int64_t V) { return static_cast<int>(ceil_div(ceil_div(V, cce::kHeadPick), 4) * 4); }
int picks_wanted(int top_k) { return top_k + 8; }

struct HeadWs {
  cce::WsHeader* hdr;
  int* counters;   // HeadPicks.done and .count, directly behind the header
  size_t counter_bytes;
  int* tok_t;      // [K, N] (K > 1), see HeadArgs
  float* zt;       // [K, N]
  float* part_m;   // [4 segments, N] each
  float* part_s;
  float* part_w;
  float* pick_max; // alternatives, for a slab of rows: see HeadPicks
  int* base;
  int* pick;
  int* slot;
  int* rows;
  int3* items;
  float* logits;
  float* norm;
  int8_t* e8;      // [N, D]
  float* e_scale;  // [N]
  size_t bytes;
};

// The statistics are those of a slab of rows where alternatives are wanted, of all rows where not.
int64_t slab_rows(int64_t N, int top_k) { return top_k > 0 ? std::min<int64_t>(N, cce::kHeadSlab) : N; }

HeadWs carve(int64_t N, int64_t D, int64_t V, int K, int top_k, bool int8, bool stats, void* base) {
  HeadWs w{};
  char* b = static_cast<char*>(base);
  size_t off = cce::kHeaderBytes;
  auto take = [&](size_t bytes) {
    char* ptr = b + off;
    off = align_up(off + bytes);
    return ptr;
  };
  w.hdr = reinterpret_cast<cce::WsHeader*>(b);
  const int64_t slab = slab_rows(N, top_k);
  const size_t n = static_cast<size_t>(slab), k = static_cast<size_t>(K);
  if (top_k > 0) {
    const size_t picks = static_cast<size_t>(picks_pitch(V));
    w.counter_bytes = sizeof(int) * (4 + picks);
    w.counters = reinterpret_cast<int*>(take(w.counter_bytes));
    w.base = reinterpret_cast<int*>(take(sizeof(int) * picks));
    w.pick_max = reinterpret_cast<float*>(take(sizeof(float) * n * picks));
    w.pick = reinterpret_cast<int*>(take(sizeof(int) * n * 32));
    w.slot = reinterpret_cast<int*>(take(sizeof(int) * n * 32));
    w.rows = reinterpret_cast<int*>(take(sizeof(int) * n * 32));
    w.items = reinterpret_cast<int3*>(take(sizeof(int3) * n * 32));
    w.logits = reinterpret_cast<float*>(take(sizeof(float) * n * 32 * cce::kHeadPick));
    w.norm = reinterpret_cast<float*>(take(sizeof(float) * n * 32));
  }
  if (stats && N > 0) {
    // the largest of the slabs' splits: a slab with fewer row blocks has more segments a row block
    size_t parts = 0;
    for (int64_t rows : {slab, N % slab}) {
      if (rows == 0) continue;
      const size_t segments = static_cast<size_t>(make_split(rows, V, kMaxSms).max_segments());
      parts = std::max(parts, cce::kHeadParts * segments * static_cast<size_t>(rows));
    }
    if (K > 1) w.tok_t = reinterpret_cast<int*>(take(sizeof(int) * n * k));
    w.zt = reinterpret_cast<float*>(take(sizeof(float) * n * k));
    w.part_m = reinterpret_cast<float*>(take(sizeof(float) * parts));
    w.part_s = reinterpret_cast<float*>(take(sizeof(float) * parts));
    w.part_w = reinterpret_cast<float*>(take(sizeof(float) * parts));
  }
  if (int8) {
    w.e8 = reinterpret_cast<int8_t*>(take(static_cast<size_t>(N) * static_cast<size_t>(D)));
    w.e_scale = reinterpret_cast<float*>(take(sizeof(float) * static_cast<size_t>(N)));
  }
  w.bytes = off;
  return w;
}

// The arguments and tensor maps that every head launch shares; E and e_scale: the operand's own rows.
cce_status head_args(int64_t N, int64_t D, int64_t V, bool int8, const void* E, const float* e_scale, const void* C,
                     const void* bias, const float* c_scale, const HeadWs& w, int sms, cce::HeadArgs* A,
                     cce::HeadMaps* M) {
  A->split = make_split(N, V, std::min(sms, kMaxSms));
  order_parts(&A->split);
  A->N = static_cast<int>(N);
  A->D = static_cast<int>(D);
  A->V = static_cast<int>(V);
  const int per_block = int8 ? 128 : 64;  // values of a 128-byte K-block
  A->num_kb = static_cast<int>(ceil_div(D, per_block));
  A->kb_chunk = int8 ? A->num_kb : cce::logit_kb_chunk(D);
  A->e_rows = static_cast<int>(std::min<int64_t>(cce::kHeadBM, (N + 7) / 8 * 8));
  A->bias = static_cast<const __nv_bfloat16*>(bias);
  A->e_scale = e_scale;
  A->c_scale = c_scale;
  A->err = &w.hdr->err;
  A->failed = &w.hdr->failed;
  A->timeout_ns = cce::wait_timeout_ns();
  // Failure-detection test hook: CCE_TEST_INJECT_STALL=4 makes the first bounded wait of the head kernel run out
  // (reported as CCE_ERR_DEVICE_TIMEOUT by cce_check_device_error).
  const char* stall = std::getenv("CCE_TEST_INJECT_STALL");
  A->inject_stall = (stall != nullptr && stall[0] == '4') ? 1 : 0;
  const auto type = int8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const size_t size = int8 ? 1 : 2;
  CCE_CHECK(cce::make_map(&M->E, type, size, E, N, D, per_block, static_cast<uint32_t>(A->e_rows)));
  CCE_CHECK(cce::make_map(&M->C, type, size, C, V, D, per_block, cce::kHeadBN));
  CCE_CHECK(cce::make_map(&M->C64, type, size, C, V, D, per_block, cce::kHeadUnit));
  return CCE_OK;
}

cce_problem backward_problem(const cce_logprob_problem* p) {
  cce_problem q{};
  q.N = p->N;
  q.D = p->D;
  q.V = p->V;
  q.ignore_index = -100;
  q.reduction = CCE_REDUCTION_SUM;
  q.vocab_start = 0;
  q.vocab_total = p->V + 1;  // id V: a row that is scored but has no target of its own
  return q;
}

}  // namespace

extern "C" {

size_t cce_logprobs_workspace_size(const cce_logprob_problem* p) {
  if (!logprobs_ok(p, false)) return 0;
  return carve(p->N, p->D, p->V, p->num_tokens, p->top_k, p->int8 != 0, true, nullptr).bytes;
}

cce_status cce_logprobs(const cce_logprob_problem* p, const void* E, const void* C, const float* c_scale,
                        const void* bias, const int64_t* tokens, float* logprobs, float* entropy, float* lse,
                        float* tile_max, float* top_logprobs, int64_t* top_ids, void* workspace, size_t workspace_bytes,
                        cce_stream_t stream) {
  return cce_logprobs_stats(p, E, C, c_scale, bias, tokens, logprobs, entropy, lse, nullptr, tile_max, top_logprobs,
                            top_ids, workspace, workspace_bytes, stream);
}

cce_status cce_logprobs_stats(const cce_logprob_problem* p, const void* E, const void* C, const float* c_scale,
                              const void* bias, const int64_t* tokens, float* logprobs, float* entropy, float* lse,
                              float* row_stats, float* tile_max, float* top_logprobs, int64_t* top_ids, void* workspace,
                              size_t workspace_bytes, cce_stream_t stream) {
  cce::clear_last_error();
  if (!logprobs_ok(p, true)) return CCE_ERR_INVALID_ARG;
  const bool int8 = p->int8 != 0;
  const bool has_rows = p->N > 0;
  if (C == nullptr || workspace == nullptr || (int8 && c_scale == nullptr) ||
      (has_rows && (E == nullptr ||
                    (p->num_tokens > 0 &&
                     (tokens == nullptr || logprobs == nullptr || entropy == nullptr || lse == nullptr)) ||
                    (p->top_k > 0 && (top_logprobs == nullptr || top_ids == nullptr)))))
    return fail(CCE_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(E) || !aligned16(C) || !aligned16(c_scale) || !aligned16(bias) || !aligned16(workspace))
    return fail(CCE_ERR_INVALID_ARG, "E, C, c_scale, bias and workspace must be 16-byte aligned");
  const HeadWs w = carve(p->N, p->D, p->V, p->num_tokens, p->top_k, int8, true, workspace);
  if (workspace_bytes < w.bytes)
    return fail(CCE_ERR_WORKSPACE, "workspace is %zu bytes, needs %zu", workspace_bytes, w.bytes);
  int sms = 0;
  CCE_CHECK(cce::check_device(&sms));
  CCE_CHECK(cce::get_encoder());
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int K = p->num_tokens, top_k = p->top_k;
  if (!has_rows) {
    CCE_TRY(cudaMemsetAsync(w.hdr, 0, sizeof(cce::WsHeader), s));
    return CCE_OK;
  }
  if (int8)
    CCE_TRY(cce::launch_quantize_rows(static_cast<const __nv_bfloat16*>(E), p->N, p->D, w.e8, w.e_scale, s));

  const int64_t slab = slab_rows(p->N, top_k);
  for (int64_t r0 = 0; r0 < p->N; r0 += slab) {
    const int64_t n = std::min(slab, p->N - r0);
    const auto* Eb = static_cast<const __nv_bfloat16*>(E) + r0 * p->D;
    const void* operand = int8 ? static_cast<const void*>(w.e8 + r0 * p->D) : Eb;
    const float* e_scale = int8 ? w.e_scale + r0 : nullptr;
    const int64_t* tok = K > 0 ? tokens + r0 * K : nullptr;
    // the header is cleared by the head kernel
    if (top_k > 0 && cce::picks_grouped(n)) CCE_TRY(cudaMemsetAsync(w.counters, 0, w.counter_bytes, s));
    if (K > 1) CCE_TRY(cce::launch_head_tokens(tok, static_cast<int>(n), K, static_cast<int>(p->V), p->ignore_index,
                                               w.tok_t, s));
    cce::HeadArgs A{};
    cce::HeadMaps M{};
    CCE_CHECK(head_args(n, p->D, p->V, int8, operand, e_scale, C, bias, c_scale, w, sms, &A, &M));
    A.clear = r0 == 0;
    A.tokens = tok;
    A.tok_t = w.tok_t;
    A.ignore_index = p->ignore_index;
    A.K = K;
    A.zt = w.zt;
    A.tile_max = tile_max == nullptr ? nullptr : tile_max + r0;
    A.max_pitch = p->N;
    A.pick_max = top_k > 0 ? w.pick_max : nullptr;
    A.picks = top_k > 0 ? picks_pitch(p->V) : 0;
    A.inv_t = 1.f / p->temperature;
    A.part_m = w.part_m;
    A.part_s = w.part_s;
    A.part_w = w.part_w;
    // it follows a kernel directly where the tokens, or the operands and no counters, were prepared on the stream
    const bool cleared = top_k > 0 && cce::picks_grouped(n);
    CCE_TRY(cce::launch_head(M, A, int8, K > 1 || (int8 && r0 == 0 && !cleared), s));

    cce::HeadFinish F{};
    F.split = A.split;
    F.N = A.N;
    F.D = A.D;
    F.V = A.V;
    F.E = Eb;
    F.C = int8 ? nullptr : static_cast<const __nv_bfloat16*>(C);
    F.E8 = int8 ? w.e8 + r0 * p->D : nullptr;
    F.C8 = int8 ? static_cast<const int8_t*>(C) : nullptr;
    F.e_scale = e_scale;
    F.c_scale = c_scale;
    F.bias = A.bias;
    F.tokens = tok;
    F.ignore_index = p->ignore_index;
    F.K = K;
    F.zt = w.zt;
    F.inv_t = A.inv_t;
    F.part_m = w.part_m;
    F.part_s = w.part_s;
    F.part_w = w.part_w;
    F.pick = w.pick;
    F.logits = w.logits;
    F.norm = w.norm;
    F.wanted = picks_wanted(top_k);
    F.top_k = top_k;
    F.logprobs = K > 0 ? logprobs + r0 * K : nullptr;
    F.entropy = K > 0 ? entropy + r0 : nullptr;
    F.lse = K > 0 ? lse + r0 : nullptr;
    F.row_max = K > 0 && row_stats != nullptr ? row_stats + r0 : nullptr;
    F.row_ln_s = F.row_max != nullptr ? F.row_max + p->N : nullptr;
    F.top_logprobs = top_k > 0 ? top_logprobs + r0 * top_k : nullptr;
    F.top_ids = top_k > 0 ? top_ids + r0 * top_k : nullptr;
    F.err = A.err;
    F.failed = A.failed;
    if (top_k == 0) {
      CCE_TRY(cce::launch_head_finish(F, s));
      continue;
    }
    cce::HeadPicks P{};
    P.N = A.N;
    P.D = A.D;
    P.V = A.V;
    P.E = operand;
    P.C = C;
    P.e_scale = e_scale;
    P.c_scale = c_scale;
    P.bias = A.bias;
    P.pick_max = w.pick_max;
    P.picks = A.picks;
    P.wanted = picks_wanted(top_k);
    P.done = w.counters;
    P.count = w.counters + 4;
    P.base = w.base;
    P.pick = w.pick;
    P.slot = w.slot;
    P.rows = w.rows;
    P.items = w.items;
    P.logits = w.logits;
    P.norm = w.norm;
    CCE_TRY(cce::launch_head_picks(P, F, int8, sms, s));
  }
  return CCE_OK;
}

size_t cce_logprobs_backward_workspace_size(const cce_logprob_problem* p, int32_t out_fp32) {
  if (!logprobs_ok(p, false) || p->int8 != 0 || p->num_tokens == 0 || out_fp32 < CCE_OUT_BF16 ||
      out_fp32 > CCE_OUT_DE_FP32)
    return 0;
  const cce_problem q = backward_problem(p);
  return cce::logprobs_backward_bytes(&q, p->num_tokens, out_fp32);
}

cce_status cce_logprobs_backward(const cce_logprob_problem* p, const void* E, const void* C, const void* bias,
                                 const int64_t* tokens, const float* logprobs, const float* lse, const float* entropy,
                                 const float* tile_max,
                                 const float* grad_logprobs, const float* grad_entropy, float filter_eps, void* dE,
                                 void* dC, void* dbias, int32_t out_fp32, int64_t* filtered_tiles, void* workspace,
                                 size_t workspace_bytes, cce_stream_t stream) {
  return cce_logprobs_stats_backward(p, E, C, bias, tokens, logprobs, lse, nullptr, entropy, tile_max, grad_logprobs,
                                     grad_entropy, filter_eps, dE, dC, dbias, out_fp32, 0, filtered_tiles, workspace,
                                     workspace_bytes, stream);
}

cce_status cce_logprobs_stats_backward(const cce_logprob_problem* p, const void* E, const void* C, const void* bias,
                                       const int64_t* tokens, const float* logprobs, const float* lse,
                                       const float* row_stats, const float* entropy, const float* tile_max,
                                       const float* grad_logprobs, const float* grad_entropy, float filter_eps,
                                       void* dE, void* dC, void* dbias, int32_t out_fp32, int32_t dbias_fp32,
                                       int64_t* filtered_tiles, void* workspace, size_t workspace_bytes,
                                       cce_stream_t stream) {
  cce::clear_last_error();
  if (!logprobs_ok(p, true)) return CCE_ERR_INVALID_ARG;
  if (p->int8 != 0) return fail(CCE_ERR_INVALID_ARG, "a classifier of 8-bit integers has no gradient");
  if (p->num_tokens == 0) return fail(CCE_ERR_INVALID_ARG, "without given tokens there is nothing to differentiate");
  const bool has_rows = p->N > 0;
  if (C == nullptr || dC == nullptr || filtered_tiles == nullptr || workspace == nullptr ||
      (has_rows && (E == nullptr || tokens == nullptr || logprobs == nullptr || lse == nullptr || entropy == nullptr ||
                    dE == nullptr ||
                    (filter_eps > 0.f && tile_max == nullptr))))
    return fail(CCE_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(E) || !aligned16(C) || !aligned16(bias) || !aligned16(dE) || !aligned16(dC) || !aligned16(dbias) ||
      !aligned16(workspace))
    return fail(CCE_ERR_INVALID_ARG, "E, C, bias, dE, dC, dbias and workspace must be 16-byte aligned");
  if (std::isnan(filter_eps)) return fail(CCE_ERR_INVALID_ARG, "filter_eps is NaN");
  if (out_fp32 < CCE_OUT_BF16 || out_fp32 > CCE_OUT_DE_FP32)
    return fail(CCE_ERR_INVALID_ARG, "out_fp32 must be CCE_OUT_BF16, CCE_OUT_FP32 or CCE_OUT_DE_FP32");
  if (dbias_fp32 != 0 && dbias_fp32 != 1) return fail(CCE_ERR_INVALID_ARG, "dbias_fp32 must be 0 or 1");
  const cce_problem q = backward_problem(p);
  cce::LogprobGrads g{};
  g.dbias_fp32 = dbias_fp32;
  g.tokens = tokens;
  g.ignore_index = p->ignore_index;
  g.K = p->num_tokens;
  g.temperature = p->temperature;
  g.lse = lse;
  g.row_stats = row_stats;
  g.entropy = entropy;
  g.logprobs = logprobs;
  g.g_logprobs = grad_logprobs;
  g.g_entropy = grad_entropy;
  return cce::logprobs_backward(&q, g, E, C, bias, tile_max, filter_eps, dE, dC, dbias, out_fp32, filtered_tiles,
                                workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

cce_status cce_quantize_int8(const void* x, int64_t rows, int64_t D, int8_t* q, float* scale, cce_stream_t stream) {
  cce::clear_last_error();
  if (!sizes_ok(rows, D, 1, true, true)) return CCE_ERR_INVALID_ARG;
  if (rows > 0 && (x == nullptr || q == nullptr || scale == nullptr))
    return fail(CCE_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(x) || !aligned16(q)) return fail(CCE_ERR_INVALID_ARG, "x and q must be 16-byte aligned");
  int sms = 0;
  CCE_CHECK(cce::check_device(&sms));
  CCE_TRY(cce::launch_quantize_rows(static_cast<const __nv_bfloat16*>(x), rows, D, q, scale,
                                    reinterpret_cast<cudaStream_t>(stream)));
  return CCE_OK;
}

size_t cce_int8_linear_workspace_size(int64_t N, int64_t D, int64_t V) {
  if (!sizes_ok(N, D, V, true, false)) return 0;
  return carve(N, D, V, 0, 0, true, false, nullptr).bytes;
}

cce_status cce_int8_linear(int64_t N, int64_t D, int64_t V, const void* E, const int8_t* C, const float* c_scale,
                           const void* bias, void* out, int32_t out_fp32, void* workspace, size_t workspace_bytes,
                           cce_stream_t stream) {
  cce::clear_last_error();
  if (!sizes_ok(N, D, V, true, true)) return CCE_ERR_INVALID_ARG;
  if (C == nullptr || c_scale == nullptr || workspace == nullptr || (N > 0 && (E == nullptr || out == nullptr)))
    return fail(CCE_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(E) || !aligned16(C) || !aligned16(c_scale) || !aligned16(bias) || !aligned16(out) ||
      !aligned16(workspace))
    return fail(CCE_ERR_INVALID_ARG, "E, C, c_scale, bias, out and workspace must be 16-byte aligned");
  if (out_fp32 != 0 && out_fp32 != 1) return fail(CCE_ERR_INVALID_ARG, "out_fp32 must be 0 or 1");
  const HeadWs w = carve(N, D, V, 0, 0, true, false, workspace);
  if (workspace_bytes < w.bytes)
    return fail(CCE_ERR_WORKSPACE, "workspace is %zu bytes, needs %zu", workspace_bytes, w.bytes);
  int sms = 0;
  CCE_CHECK(cce::check_device(&sms));
  CCE_CHECK(cce::get_encoder());
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) {
    CCE_TRY(cudaMemsetAsync(w.hdr, 0, sizeof(cce::WsHeader), s));
    return CCE_OK;
  }
  CCE_TRY(cce::launch_quantize_rows(static_cast<const __nv_bfloat16*>(E), N, D, w.e8, w.e_scale, s));
  cce::HeadArgs A{};
  cce::HeadMaps M{};
  CCE_CHECK(head_args(N, D, V, true, w.e8, w.e_scale, C, bias, c_scale, w, sms, &A, &M));
  A.clear = 1;
  A.inv_t = 1.f;
  A.out = out;
  A.out_fp32 = out_fp32;
  const int64_t out_size = out_fp32 ? 4 : 2;
  A.out_tma = V * out_size % 16 == 0;
  if (A.out_tma)
    CCE_CHECK(cce::make_map(&M.out, out_fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                            static_cast<size_t>(out_size), out, N, V, static_cast<uint32_t>(128 / out_size), 16));
  CCE_TRY(cce::launch_head(M, A, true, true, s));
  return CCE_OK;
}

}  // extern "C"
