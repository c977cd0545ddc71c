// The head operators on sm_100a: logit tiles z = E_b C_t^T (+ bias) of a classifier on the tcgen05 tensor
// cores, reduced on the fly to what the caller asked for. With y = z / temperature, per row:
//   lse = ln sum_v exp(y_v)       entropy H = lse - sum_v p_v y_v, p = softmax(y)
//   log-probability of a given token t: y_t - lse
//   the k tokens with the largest y
// or the logits themselves, for operands of 8-bit integers (z = (sum_d qe qc) se sc + bias).
//
// One pass over the columns keeps, per row, the largest logit m, S = sum 2^d and W = sum d 2^d with
// d = (z - m) log2(e) / temperature <= 0; then lse = m / temperature + ln S and H = ln S - ln2 W / S. Neither
// loses anything for large |z|: only differences to the maximum are exponentiated. A new maximum m' takes
// S to S f and W to f (W + S d'), f = 2^d', d' = (m - m') log2(e) / temperature.
//
// Design (B200): one persistent block per SM, 20 warps.
//   warp 0       producer: E and C K-blocks of 128 bytes (128B swizzle) by TMA into a 4-stage ring.
//   warp 1       tensor memory owner; one lane issues tcgen05.mma, M = 128 rows, N = up to 256 columns.
//   warps 4..19  epilogue, four warps for each 32 rows (one for each 64 columns of the tile): a thread owns
//                64 logits of one row, in registers. Four warps a scheduler hide the latency of tensor memory
//                and of the exponentials; eight warps with 128 logits each were bound by it (2048 x 2048 x
//                128256: 844 us against 785).
// What bounds it: the delivery of operands from L2, 48 KB a step of 128 x 256 x 64 (2048 x 2048 x 128256: tensor pipe
// 79 % busy at 1.53 GHz, 770 us, 1397 TFLOP/s); with few rows reading C (one row of D = 4096: 6.1 TB/s).
// Sums over K: the tensor cores add into their fp32 accumulator without rounding to nearest, so a long sum
// drifts towards zero (D = 4096, logits of 11: -5e-5, sixteen times what fp32 sums lose). The accumulator is
// therefore handed over every kb_chunk K-blocks (512 or 256 values of K) and the parts are added in registers,
// rounded to nearest: two tensor-memory buffers alternate by parts, and the drift falls with the parts' number.
// 8-bit products are exact in 32-bit integers, so they keep one part.
#include <algorithm>
#include <type_traits>

#include "cce_device.cuh"
#include "cce_head.h"
#include "cce_internal.h"

namespace cce {
namespace {

constexpr int BM = kHeadBM;
constexpr int BN = kHeadBN;
constexpr int STAGES = 4;
constexpr int KB_BYTES = 128;  // one swizzle row: 64 bf16 or 128 8-bit values of K
constexpr int A_BYTES = BM * KB_BYTES;
constexpr int B_BYTES = BN * KB_BYTES;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 16;
constexpr int NUM_THREADS = 128 + 32 * EPI_WARPS;
constexpr int COLS = BN / (EPI_WARPS / 4);  // columns of a thread
constexpr int TMEM_COLS = 512;
constexpr int NUM_BARRIERS = 2 * STAGES + 4 + 1;
constexpr int SCRATCH_WARP = 2048;  // of each epilogue warp: a piece of the logits going out (16 rows of 128 bytes)
constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_WARPS * SCRATCH_WARP + NUM_BARRIERS * 8 + 16;
static_assert(SMEM_BYTES <= 232448, "fits the 227 KB opt-in shared memory of an SM");
static_assert(COLS == kSubTile && COLS == 4 * kHeadPick, "a thread's columns are one saved maximum, and four picks");

// Registers a thread: 640 threads are launched with 96 each; the first warpgroup hands 32 of its own to the four that
// hold logits in registers.
constexpr int REGS_FEW = 64, REGS_MANY = 104;
static_assert(REGS_FEW * 128 + REGS_MANY * 512 <= 96 * 640, "setmaxnreg draws on the launch's registers");

__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor without N: kind::f16 with bf16 operands and an fp32 accumulator, or kind::i8 with signed
// operands (format 1) and a 32-bit integer accumulator (format 2).
__device__ __forceinline__ uint32_t idesc_n(bool int8, int n) {
  const uint32_t base = int8 ? (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(BM >> 4) << 24)
                             : idesc_bf16(BM, 0, false, false);
  return base | (static_cast<uint32_t>(n >> 3) << 17);
}

// The larger of two numbers, NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Keys order (logit, column) pairs: a larger key is a larger logit, or the lower column of two equal ones. 0 is below
// every key.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 is 0
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t o) {
  return __uint_as_float(o ^ ((o & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ unsigned long long make_key(float v, uint32_t col) {
  return (static_cast<unsigned long long>(order_bits(v)) << 32) | (0xffffffffu - col);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  return k == 0 ? -INFINITY : from_order_bits(static_cast<uint32_t>(k >> 32));
}
__device__ __forceinline__ int key_column(unsigned long long k) {
  return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
}

__device__ __forceinline__ int token_or_none(int64_t id, int64_t ignore_index, int V) {
  return id != ignore_index && id >= 0 && id < V ? static_cast<int>(id) : kNoToken;
}

// One tile of a block's walk.
struct HeadTile {
  int b;           // row block
  int seg;         // segment of the row block
  int col, ncol;   // its first column, and how many
  bool first, last;  // of the segment
};

// Rows of C that a tile loads and multiplies: all 256 in one box, or those it needs 64 at a time (one box a stage
// instead of four: 896 x 2048 x 50257: 161 us against 182).
__device__ __forceinline__ int tile_rows(const HeadTile& t) {
  return (t.ncol + kHeadUnit - 1) / kHeadUnit * kHeadUnit;
}

// Calls f(tile) for every tile of this block, in the order that all roles share; f returns false to stop. Within a
// segment the walk starts at the tile whose position is 0 modulo the length of a block's share: the blocks on
// different row blocks then pass the same columns of C at about the same time, and C is read from HBM about once
// a group.
template <typename F>
__device__ __forceinline__ void for_tiles(const HeadSplit& S, int V, F&& f) {
  for (int g = 0; g < S.ngroups; ++g) {
    int x, hi, c;
    {
      const int gb = S.group_begin(g + 1) - S.group_begin(g), total = S.units(gb), P = S.parts(total);
      if (static_cast<int>(blockIdx.x) >= P) continue;
      c = S.order[gb == S.nb / S.ngroups ? 0 : 1][blockIdx.x];
      x = HeadSplit::part_begin(c, total, P);
      hi = HeadSplit::part_begin(c + 1, total, P);
    }
    while (x < hi) {
      HeadTile t;
      const int bi = x / S.nu, u0 = x - bi * S.nu, u1 = min(S.nu, u0 + hi - x);
      const int c0 = u0 * S.unit, n = (min(V, u1 * S.unit) - c0 + BN - 1) / BN;
      int at = 0;
      {
        const int b0 = S.group_begin(g), total = S.units(S.group_begin(g + 1) - b0), P = S.parts(total);
        t.b = b0 + bi;
        t.seg = c - HeadSplit::owner(bi * S.nu, total, P);
        if (S.unit == BN) {
          const int share = total / P;
          at = u0 % share;
          at = at == 0 ? 0 : share - at;
          if (at >= n) at = 0;
        }
      }
      for (int i = 0; i < n; ++i) {
        t.col = c0 + at * BN;
        t.ncol = min(BN, min(V, u1 * S.unit) - t.col);
        t.first = i == 0;
        t.last = i == n - 1;
        if (!f(t)) return;
        if (++at == n) at = 0;
      }
      x += u1 - u0;
    }
  }
}

// Adds sum 2^d and sum d 2^d, d = (a - m) sc, of a thread's columns. MASKED: some a may be -inf; its power is 0, and
// with d held above -1e4 (where the power is 0 too) so is its product with d.
template <bool MASKED>
__device__ __forceinline__ void add_powers(const float (&a)[COLS], float m, float sc, float& s, float& w) {
  const uint64_t mm = pack2(-m, -m), cc = pack2(sc, sc);
  uint64_t s2 = 0, w2 = 0;
#pragma unroll
  for (int i = 0; i < COLS; i += 2) {
    const uint64_t d2 = mul2(add2(pack2(a[i], a[i + 1]), mm), cc);
    float d0, d1;
    unpack2(d2, d0, d1);
    if (MASKED) {
      d0 = max_nan(d0, -1e4f);
      d1 = max_nan(d1, -1e4f);
    }
    const uint64_t e2 = pack2(ex2(d0), ex2(d1));
    s2 = add2(s2, e2);
    w2 = fma2(MASKED ? pack2(d0, d1) : d2, e2, w2);
  }
  float x, y;
  unpack2(s2, x, y);
  s += x + y;
  unpack2(w2, x, y);
  w += x + y;
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(src),
               "r"(x), "r"(y)
               : "memory");
}

// Writes a warp's 32 rows x COLS columns of logits through its scratch. Where rows start on 16-byte boundaries, by
// TMA, 16 rows of 128 bytes at a time, which clips them to the tensor; else the warp writes 32 words of a row at a
// time (1000 x 1024 x 50257: 154 us, 178 by single elements of two rows).
// 2048 x 2048 x 128256 in bf16: 460 us; 510 by 32-byte stores of each thread's own row, or with 32 rows at a time and
// one stage of the ring less to make room for them; 401 without writing anything.
template <bool F32>
__device__ __forceinline__ void write_logits(const HeadArgs& A, const CUtensorMap& tmOut, const float (&a)[COLS],
                                             int row0, int col0, int ncol, int lane, uint8_t* scratch) {
  const uint32_t buf = smem_u32(scratch);
  if (A.out_tma) {
    const uint32_t mine = buf + static_cast<uint32_t>(lane & 15) * 128u;
    const uint32_t x = static_cast<uint32_t>(lane & 7);
#pragma unroll
    for (int h = 0; h < (F32 ? 2 : 1); ++h) {  // 64 columns of bf16, or 32 of fp32
      if (32 * h >= ncol) break;
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // 16 rows
        if (row0 + 16 * u >= A.N) break;
        if (lane == 0) bulk_wait_group_read0();
        __syncwarp();
        if ((lane >> 4) == u) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t dst = mine + ((static_cast<uint32_t>(c) ^ x) << 4);
            if (F32) {
              const int i = 32 * h + 4 * c;
              st_shared_v4(dst, __float_as_uint(a[i]), __float_as_uint(a[i + 1]), __float_as_uint(a[i + 2]),
                           __float_as_uint(a[i + 3]));
            } else {
              st_shared_v4(dst, pack_bf16x2(a[8 * c], a[8 * c + 1]), pack_bf16x2(a[8 * c + 2], a[8 * c + 3]),
                           pack_bf16x2(a[8 * c + 4], a[8 * c + 5]), pack_bf16x2(a[8 * c + 6], a[8 * c + 7]));
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tmOut, buf, col0 + 32 * h, row0 + 16 * u);
          bulk_commit_group();
        }
      }
    }
    return;
  }
  // 16 rows x 32 words at a time, word w of row k at 32 k + (w + k) % 32: no bank meets twice, in or out
  uint32_t* st = reinterpret_cast<uint32_t*>(scratch);
#pragma unroll
  for (int h = 0; h < (F32 ? 2 : 1); ++h) {
    const int j = 32 * h, n = min(F32 ? 32 : 64, ncol - j);  // columns from j
    if (n <= 0) break;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int n_rows = min(16, A.N - row0 - 16 * u);
      if (n_rows <= 0) break;
      __syncwarp();
      if ((lane >> 4) == u) {
        const int k = lane & 15;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          st[k * 32 + ((i + k) & 31)] = F32 ? __float_as_uint(a[j + i]) : pack_bf16x2(a[2 * i], a[2 * i + 1]);
      }
      __syncwarp();
#pragma unroll 4
      for (int k = 0; k < n_rows; ++k) {
        const int64_t o = static_cast<int64_t>(row0 + 16 * u + k) * A.V + col0 + j;
        const uint32_t x = st[k * 32 + ((lane + k) & 31)];
        if (F32) {
          if (lane < n) static_cast<uint32_t*>(A.out)[o + lane] = x;
        } else {
          // whole words of the output: columns 2 w and 2 w + 1 of the piece, or 2 w + 1 and 2 w + 2, and the single
          // columns left at its ends
          uint16_t* out = static_cast<uint16_t*>(A.out) + o;
          const int odd = static_cast<int>(o & 1);
          const uint32_t next = __shfl_down_sync(0xffffffffu, x, 1);
          const uint32_t pair = odd ? (x >> 16) | (next << 16) : x;
          const int c = 2 * lane + odd;
          if (c + 1 < n) *reinterpret_cast<uint32_t*>(out + c) = pair;
          else if (c < n) out[c] = static_cast<uint16_t>(pair & 0xffffu);
          if (odd && lane == 0) out[0] = static_cast<uint16_t>(x & 0xffffu);
        }
      }
    }
  }
}

// OUT: the logits are written out, in bf16 (1) or fp32 (2), instead of reduced.
template <bool I8, int OUT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    head_kernel(const __grid_constant__ CUtensorMap tmE, const __grid_constant__ CUtensorMap tmC,
                const __grid_constant__ CUtensorMap tmC64, const __grid_constant__ CUtensorMap tmOut,
                const __grid_constant__ HeadArgs A) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* scratch = base + STAGES * STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(scratch + EPI_WARPS * SCRATCH_WARP);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + NUM_BARRIERS);
  int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  if (A.clear && blockIdx.x == 0 && threadIdx.x == 0) {  // nothing is reported before the waits below
    *A.err = 0;
    *A.failed = 0;
  }
  const WaitCtl wc{abort_flag, A.err, A.timeout_ns};
  const int num_kb = A.num_kb;
  constexpr int KE = I8 ? KB_BYTES : KB_BYTES / 2;  // values of K a block

  if (warp < 4) regs_dec<REGS_FEW>();
  else regs_inc<REGS_MANY>();
  if (warp >= 4) {
    // ---------------- epilogue ----------------
    wait_for_previous_grid();  // the scales of E or the transposed tokens, when a kernel of this call made them
    const int q = warp & 3;             // tensor-memory lanes of this warp
    const int part = (warp - 4) >> 2;   // columns COLS part .. COLS part + COLS - 1 of a tile
    const uint32_t tmine = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(part * COLS);
    int acc = 0;
    uint32_t acc_phase = 0;
    const float sc = A.inv_t * kLog2e;
    float m = -INFINITY, s = 0.f, w = 0.f;
    // The row's given tokens are met in ascending order: `id` is the next one, the row's `at_id`-th.
    int id = kNoToken, at_id = 0, walked = 0;
    for_tiles(A.split, A.V, [&](const HeadTile& t) {
      const int row0 = t.b * BM + q * 32, r = row0 + lane;
      const bool rows = row0 < A.N;                // any row of this warp
      const int ncol = min(COLS, t.ncol - part * COLS);  // columns of this warp (none if <= 0)
      const int col0 = t.col + part * COLS;
      if (OUT == 0 && t.first) {
        m = -INFINITY;
        s = w = 0.f;
      }
      if (OUT == 0 && A.K > 0 && (t.first || t.col < walked)) {  // a segment begins, or its walk turns round
        at_id = 0;
        id = kNoToken;
        if (r < A.N) {
          if (A.K == 1) {
            const int64_t tok = A.tokens[r];
            if (tok >= col0) id = token_or_none(tok, A.ignore_index, A.V);
          } else {
            for (int k = 0; k < A.K; ++k) at_id += A.tok_t[static_cast<int64_t>(k) * A.N + r] < col0 ? 1 : 0;
            if (at_id < A.K) id = A.tok_t[static_cast<int64_t>(at_id) * A.N + r];
          }
        }
      }
      walked = t.col;
      float a[COLS];
      // columns past ncol hold what an earlier tile left; they are masked below
      for (int k0 = 0; k0 < num_kb; k0 += A.kb_chunk) {
        const bool got = mbar_wait(tfull_bar(acc), acc_phase, wc);
        if (!__all_sync(0xffffffffu, got ? 1 : 0)) return false;
        tc_fence_after();
        const uint32_t src = tmine + static_cast<uint32_t>(acc * BN);
        if (k0 == 0) {
#pragma unroll
          for (int j = 0; j < COLS; j += 16) tmem_ld16(src + j, a + j);
        } else {
#pragma unroll
          for (int j = 0; j < COLS; j += 16) {
            float v[16];
            tmem_ld16(src + j, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) a[j + i] += v[i];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!rows) return true;
      if (ncol > 0) {
        if (I8) {
          const float es = r < A.N ? A.e_scale[r] : 0.f;
#pragma unroll
          for (int j = 0; j < COLS; ++j) a[j] = static_cast<float>(__float_as_int(a[j]));
#pragma unroll
          for (int j = 0; j < COLS; j += 4) {
            float4 c = make_float4(0.f, 0.f, 0.f, 0.f);  // the scales' tail is read one by one
            if (col0 + j + 4 <= A.V) {
              c = *reinterpret_cast<const float4*>(A.c_scale + col0 + j);
            } else {
              if (col0 + j < A.V) c.x = A.c_scale[col0 + j];
              if (col0 + j + 1 < A.V) c.y = A.c_scale[col0 + j + 1];
              if (col0 + j + 2 < A.V) c.z = A.c_scale[col0 + j + 2];
            }
            a[j] *= es * c.x;
            a[j + 1] *= es * c.y;
            a[j + 2] *= es * c.z;
            a[j + 3] *= es * c.w;
          }
        }
        if (A.bias != nullptr) {
#pragma unroll
          for (int j = 0; j < COLS; j += 8) {
            if (col0 + j + 8 <= A.V) {
              const uint4 u = ld_global_nc_v4(A.bias + col0 + j);
              const uint32_t us[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                a[j + 2 * k] += __uint_as_float(us[k] << 16);
                a[j + 2 * k + 1] += __uint_as_float(us[k] & 0xffff0000u);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (col0 + j + k < A.V) a[j + k] += __bfloat162float(A.bias[col0 + j + k]);
            }
          }
        }
        if constexpr (OUT != 0) {
          write_logits<OUT == 2>(A, tmOut, a, row0, col0, ncol, lane, scratch + (warp - 4) * SCRATCH_WARP);
        } else {
          const bool cut = ncol < COLS;
          if (cut) {
#pragma unroll
            for (int i = 0; i < COLS; ++i) a[i] = i < ncol ? a[i] : -INFINITY;
          }
          // The given tokens of the row among these columns, and those that other warps' columns hold, in the order
          // of tok_t: a tile costs as many steps as its fullest row has tokens in it, not one for each of K (777 x
          // 1288 x 50257, K = 20: 143 us against 162 with every token looked for in every tile).
          while (__any_sync(0xffffffffu, id < col0 + ncol)) {
            const int at = id - col0;
            if (__any_sync(0xffffffffu, at >= 0 && at < ncol)) {
              float z = 0.f;
#pragma unroll
              for (int i = 0; i < COLS; ++i) z = i == at ? a[i] : z;
              if (at >= 0 && at < ncol) A.zt[static_cast<int64_t>(at_id) * A.N + r] = z;
            }
            if (at < ncol) {
              ++at_id;
              id = at_id < A.K ? A.tok_t[static_cast<int64_t>(at_id) * A.N + r] : kNoToken;
            }
          }
          float cm[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x = a[kHeadPick * j];
#pragma unroll
            for (int i = 1; i < kHeadPick; ++i) x = fmaxf(x, a[kHeadPick * j + i]);
            cm[j] = x;
          }
          const float mt = fmaxf(fmaxf(cm[0], cm[1]), fmaxf(cm[2], cm[3]));
          if (r < A.N) {
            if (A.tile_max != nullptr) A.tile_max[col0 / kSubTile * A.max_pitch + r] = mt * A.inv_t;
            if (A.pick_max != nullptr)
              *reinterpret_cast<float4*>(A.pick_max + static_cast<int64_t>(r) * A.picks + col0 / kHeadPick) =
                  make_float4(cm[0], cm[1], cm[2], cm[3]);
          }
          const float mn = fmaxf(m, mt);
          if (mn == -INFINITY) {  // nothing but -inf (masked columns) so far; a NaN among them still counts
#pragma unroll
            for (int i = 0; i < COLS; ++i)
              if (a[i] != a[i]) s = a[i];
          } else {
            if (m != mn && m != -INFINITY) {
              const float d = (m - mn) * sc, f = ex2(d);
              w = f * fmaf(s, fmaxf(d, -1e30f), w);
              s *= f;
            }
            m = mn;
            if (cut || A.bias != nullptr) add_powers<true>(a, m, sc, s, w);
            else add_powers<false>(a, m, sc, s, w);
          }
        }
      }
      if (OUT == 0 && t.last && r < A.N) {
        const int64_t o = static_cast<int64_t>(kHeadParts * t.seg + part) * A.N + r;
        A.part_m[o] = m;
        A.part_s[o] = s;
        A.part_w[o] = w;
      }
      return true;
    });
  } else if (warp == 0) {
    // ---------------- producer ----------------
    // inject_stall (test hook): nothing is loaded, so the bounded wait of the next role runs out.
    if (lane == 0 && !A.inject_stall) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued[STAGES] = {};
      bool ok = true, first = true;
      const uint32_t e_bytes = static_cast<uint32_t>(A.e_rows) * KB_BYTES;
      for_tiles(A.split, A.V, [&](const HeadTile& t) {
        const int rows_c = tile_rows(t);
        const uint32_t bytes = e_bytes + static_cast<uint32_t>(rows_c) * KB_BYTES;
        auto load_c = [&](int st, int kb) {
          const uint32_t dst = smem_u32(base + st * STAGE_BYTES) + A_BYTES;
          mbar_arrive_expect_tx(full_bar(st), bytes);
          if (rows_c == BN) {
            tma_load_2d(dst, &tmC, full_bar(st), kb * KE, t.col);
          } else {
            for (int j = 0; j < rows_c; j += kHeadUnit)
              tma_load_2d(dst + static_cast<uint32_t>(j) * KB_BYTES, &tmC64, full_bar(st), kb * KE, t.col + j);
          }
        };
        // The first stages' rows of C are on their way before the kernel that makes the 8-bit rows of E has ended.
        int ahead = 0;
        if (first) {
          ahead = min(STAGES, num_kb);
          for (int kb = 0; kb < ahead; ++kb) load_c(kb, kb);
          wait_for_previous_grid();
          first = false;
        }
        for (int kb = 0; kb < num_kb; ++kb) {
          if (kb >= ahead) {
            if (!mbar_wait(empty_bar(stage), phase ^ 1u, wc)) return ok = false;
            load_c(stage, kb);
          }
          tma_load_2d(smem_u32(base + stage * STAGE_BYTES), &tmE, full_bar(stage), kb * KE, t.b * BM);
          ++issued[stage];
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        return true;
      });
      if (!ok) {  // every load already issued lands before the block can exit
        for (int s = 0; s < STAGES; ++s)
          if (issued[s]) mbar_wait_drain(full_bar(s), (issued[s] - 1u) & 1u, 200000000ull);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, issued_any = false;
      for_tiles(A.split, A.V, [&](const HeadTile& t) {
        const uint32_t idesc = idesc_n(I8, tile_rows(t));
        for (int k0 = 0; k0 < num_kb; k0 += A.kb_chunk) {
          if (!mbar_wait(tempty_bar(acc), acc_phase ^ 1u, wc)) return ok = false;
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
          const int k1 = min(num_kb, k0 + A.kb_chunk);
          for (int kb = k0; kb < k1; ++kb) {
            if (!mbar_wait(full_bar(stage), phase, wc)) return ok = false;
            tc_fence_after();
            const uint32_t a0 = smem_u32(base + stage * STAGE_BYTES);
#pragma unroll
            for (int k = 0; k < KB_BYTES / 32; ++k) {  // 32 bytes of K an instruction
              const uint64_t da = sdesc_sw128(a0 + 32u * k, 16, 1024);
              const uint64_t db = sdesc_sw128(a0 + A_BYTES + 32u * k, 16, 1024);
              const uint32_t add = kb != k0 || k != 0 ? 1u : 0u;
              if (I8) tc_mma_i8(d, da, db, idesc, add);
              else tc_mma_bf16(d, da, db, idesc, add);
            }
            issued_any = true;
            tc_commit(empty_bar(stage));
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          tc_commit(tfull_bar(acc));
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
        return true;
      });
      if (!ok && issued_any) {  // no MMA may still write tensor memory when it is released
        tc_commit(drain_bar);
        mbar_wait_drain(drain_bar, 0, 200000000ull);
      }
    }
  }

  if (OUT != 0 && warp >= 4) {  // every store of the logits is complete before the kernel ends
    if (lane == 0) bulk_wait_group0();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) *A.failed = 1;  // what follows then writes NaN
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

__device__ __forceinline__ float sum_squares(const uint4& u) {
  const uint32_t us[4] = {u.x, u.y, u.z, u.w};
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float lo = __uint_as_float(us[k] << 16), hi = __uint_as_float(us[k] & 0xffff0000u);
    s = fmaf(lo, lo, s);
    s = fmaf(hi, hi, s);
  }
  return s;
}

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The logit of row r at column `col` in 64 bits, by the whole warp: products of bf16 pairs and of 8-bit pairs are
// exact, and the order of the sum depends on D alone.
__device__ double exact_logit(const HeadFinish& F, int64_t r, int col, int lane) {
  double z;
  if (F.C8 != nullptr) {
    long long acc = 0;
    const int8_t* e = F.E8 + r * F.D;
    const int8_t* c = F.C8 + static_cast<int64_t>(col) * F.D;
#pragma unroll 4
    for (int d = lane * 16; d < F.D; d += 512) {  // D is a multiple of 16
      const uint4 x = *reinterpret_cast<const uint4*>(e + d), y = *reinterpret_cast<const uint4*>(c + d);
      int p = __dp4a(static_cast<int>(x.x), static_cast<int>(y.x), 0);
      p = __dp4a(static_cast<int>(x.y), static_cast<int>(y.y), p);
      p = __dp4a(static_cast<int>(x.z), static_cast<int>(y.z), p);
      p = __dp4a(static_cast<int>(x.w), static_cast<int>(y.w), p);
      acc += p;
    }
    z = warp_sum_f64(static_cast<double>(acc)) * static_cast<double>(F.e_scale[r]) *
        static_cast<double>(F.c_scale[col]);
  } else {
    double acc = 0.0;
    const __nv_bfloat16* e = F.E + r * F.D;
    const __nv_bfloat16* c = F.C + static_cast<int64_t>(col) * F.D;
#pragma unroll 8
    for (int d = lane * 8; d < F.D; d += 256) {  // D is a multiple of 8
      const uint4 x = *reinterpret_cast<const uint4*>(e + d), y = *reinterpret_cast<const uint4*>(c + d);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc = fma(static_cast<double>(__uint_as_float(xs[k] << 16)), static_cast<double>(__uint_as_float(ys[k] << 16)),
                  acc);
        acc = fma(static_cast<double>(__uint_as_float(xs[k] & 0xffff0000u)),
                  static_cast<double>(__uint_as_float(ys[k] & 0xffff0000u)), acc);
      }
    }
    z = warp_sum_f64(acc);
  }
  if (F.bias != nullptr) z += static_cast<double>(__bfloat162float(F.bias[col]));
  return z;
}

// ---------------------------------------------------------------------------------------------
// Alternatives. The head kernel leaves, per row, the largest logit of every pick (16 columns). The best W
// logits of a row lie in the W picks with the largest maxima (each pick ahead of theirs holds a better one),
// so W = top_k + 8 picks a row are computed again, and the best of their 16 W logits are the row's. Keeping
// sorted lists in the head kernel instead costs it more than the products: 2048 x 2048 x 128256, 20
// alternatives: 1566 us with lists of 28 in registers, against 844 us without.
//   head_pick_kernel     the W picks of each row; how many rows want each pick
//   head_scatter_kernel  the rows of each pick, side by side
//   head_dots_kernel     the logits of each pick for its rows: a pick's 16 rows of C are read once for up to
//                        64 rows of E
//   head_finish_kernel   the best of a row's 16 W logits, in order
// ---------------------------------------------------------------------------------------------

// A bound that `want` to `most` of a warp's 32 R keys reach (R in each lane's registers; 0 is below every key), or the
// smallest of them that is not 0 where there are fewer: bisection on the keys' bits, stopped as soon as there is one
// (at the want-th largest at the latest). Each step is R comparisons and one sum over the warp, independent of the
// data's order (inserting into a sorted list across the lanes takes a chain of shuffles for every key that passes).
template <int R>
__device__ __forceinline__ unsigned long long warp_bound(const unsigned long long (&key)[R], int want, int most) {
  uint32_t hi = 0, lo = 0xffffffffu;  // upper words: of the largest key, and of the smallest that is not 0
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const uint32_t u = static_cast<uint32_t>(key[i] >> 32);
    hi = max(hi, u);
    if (key[i] != 0) lo = min(lo, u);
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (hi == 0) return 1;  // no key at all
  // upper words first: at least `want` keys are >= lo << 32 (or all that there are), fewer are >= (hi + 1) << 32
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2 + 1;
    int n = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) n += static_cast<uint32_t>(key[i] >> 32) >= mid ? 1 : 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (n >= want && n <= most) return static_cast<unsigned long long>(mid) << 32;
    if (n > want) lo = mid;
    else hi = mid - 1;
  }
  // equal upper words around the bound: the lower ones decide
  int above = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) above += static_cast<uint32_t>(key[i] >> 32) > lo ? 1 : 0;
  above = __reduce_add_sync(0xffffffffu, above);
  uint32_t l = 0, h = 0xffffffffu;
  while (l < h) {
    const uint32_t mid = l + (h - l) / 2 + 1;
    int n = 0;
#pragma unroll
    for (int i = 0; i < R; ++i)
      n += static_cast<uint32_t>(key[i] >> 32) == lo && static_cast<uint32_t>(key[i]) >= mid ? 1 : 0;
    n = above + __reduce_add_sync(0xffffffffu, n);
    if (n == want) {
      l = mid;
      break;
    }
    if (n > want) l = mid;
    else h = mid - 1;
  }
  return (static_cast<unsigned long long>(lo) << 32) | l;
}

// Writes the warp's keys >= bound (and not 0) to out[0 ..], at most 32; returns how many.
template <int R>
__device__ __forceinline__ int warp_collect(const unsigned long long (&key)[R], unsigned long long bound, int lane,
                                            unsigned long long* out) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const bool in = key[i] != 0 && key[i] >= bound;
    const unsigned mask = __ballot_sync(0xffffffffu, in);
    const int at = n + __popc(mask & ((1u << lane) - 1u));
    if (in && at < 32) out[at] = key[i];
    n += __popc(mask);
  }
  return min(n, 32);
}

// Sorts a key of each lane: lane 0 gets the largest.
__device__ __forceinline__ unsigned long long warp_sort(unsigned long long key, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, j);
      const bool keep_max = ((lane & k) == 0) == ((lane & j) == 0);
      key = (key > other) == keep_max ? key : other;
    }
  }
  return key;
}

constexpr int kPickGroups = 256; // groups of maxima of a row in the sieve
constexpr int kPickHeld = 16;    // maxima a lane holds at a time
constexpr int kPickSifted = 512; // candidates kept by the sieve

// The W best of `count` keys in shared memory, to out[0 ..] (which may be the same memory), by one warp that holds
// R in each lane; returns how many.
template <int R>
__device__ __forceinline__ int warp_best(const unsigned long long* keys, int count, int W, int lane,
                                         unsigned long long* out) {
  unsigned long long key[R];
#pragma unroll
  for (int i = 0; i < R; ++i) key[i] = 32 * i + lane < count ? keys[32 * i + lane] : 0ull;
  __syncwarp();
  const int m = warp_collect(key, warp_bound(key, W, W), lane, out);
  __syncwarp();
  return min(m, W);
}

// One block per row. A sieve first: the maxima are dealt to 256 groups, and a value that W of the groups' largest
// reach, or up to a quarter more (which ends the bisection early), is a bound that at least W maxima reach, and few
// more, as the best W sit in almost as many groups. What reaches it is collected, and the best W of that are the row's
// picks. The row is read 16 bytes a load (V = 128256, one row: 5.4 us, by words 7.5; 2048 rows: 54 and 60).
// Where more than kPickSifted reach the bound (equal logits), every warp bisects over its share, 512 maxima at a
// time together with what it kept before, and the best W of what the warps kept are the picks.
// P.grouped: the last block to finish lays out the picks' rows: every pick that some row wants gets its place in
// `rows` and one work item for each 64 of its rows (in any order: nothing depends on it).
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 5 : 1)
    head_pick_kernel(const __grid_constant__ HeadPicks P) {
  constexpr int kKeys = WARPS * 32 > kPickSifted ? WARPS * 32 : kPickSifted;
  static_assert(kPickGroups <= kKeys && WARPS * 32 % kPickGroups == 0, "groups share the keys' memory");
  __shared__ unsigned long long keys[kKeys];
  __shared__ unsigned long long bound_s;
  __shared__ int sifted;
  __shared__ int last;
  __shared__ int placed[2];  // rows and work items so far
  if (threadIdx.x < 2) placed[threadIdx.x] = 0;
  if (threadIdx.x == 0) sifted = 0;
  wait_for_previous_grid();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int r = blockIdx.x, W = P.wanted;
  const int n = (P.V + kHeadPick - 1) / kHeadPick;
  const float* mx = P.pick_max + static_cast<int64_t>(r) * P.picks;
  unsigned long long best = 0;
  const float4* mx4 = reinterpret_cast<const float4*>(mx);  // P.picks is a multiple of 4
  const int n4 = (n + 3) / 4;
#pragma unroll 4
  for (int u4 = threadIdx.x; u4 < n4; u4 += WARPS * 32) {
    const float4 x4 = mx4[u4];
    const float xs[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int u = 4 * u4 + j;
      const unsigned long long x = u < n ? make_key(xs[j], static_cast<uint32_t>(u)) : 0ull;
      best = x > best ? x : best;
    }
  }
  constexpr int lanes = WARPS * 32 / kPickGroups;  // of a group: neighbours
#pragma unroll
  for (int o = 1; o < lanes; o <<= 1) {
    const unsigned long long x = __shfl_xor_sync(0xffffffffu, best, o);
    best = x > best ? x : best;
  }
  if (threadIdx.x % lanes == 0) keys[threadIdx.x / lanes] = best;
  __syncthreads();
  if (w == 0) {
    unsigned long long key[kPickGroups / 32];
#pragma unroll
    for (int i = 0; i < kPickGroups / 32; ++i) key[i] = keys[32 * i + lane];
    int groups = 0;  // that hold anything: with fewer than W of them (a few dozen maxima) all maxima go on
#pragma unroll
    for (int i = 0; i < kPickGroups / 32; ++i) groups += key[i] != 0 ? 1 : 0;
    groups = __reduce_add_sync(0xffffffffu, groups);
    const unsigned long long bound = groups < W ? 1 : warp_bound(key, W, W + W / 4);
    if (lane == 0) bound_s = bound;
  }
  __syncthreads();
  const unsigned long long bound = bound_s;
#pragma unroll 4
  for (int u4 = threadIdx.x; u4 < n4; u4 += WARPS * 32) {
    const float4 x4 = mx4[u4];
    const float xs[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int u = 4 * u4 + j;
      const unsigned long long x = make_key(xs[j], static_cast<uint32_t>(u));
      if (x >= bound && u < n) {
        const int at = atomicAdd(&sifted, 1);
        if (at < kPickSifted) keys[at] = x;
      }
    }
  }
  __syncthreads();
  const bool sieve = sifted <= kPickSifted;
  if (!sieve) {
    const int share = (n + WARPS * 32 - 1) / (WARPS * 32) * 32;
    const int u1 = min(n, (w + 1) * share);
    unsigned long long* kept = keys + 32 * w;
    unsigned long long mine = 0;  // lane i: a key that the warp has kept
    for (int u0 = w * share; u0 < u1; u0 += 32 * kPickHeld) {
      unsigned long long key[kPickHeld + 1];
#pragma unroll
      for (int j = 0; j < kPickHeld; ++j) {
        const int u = u0 + 32 * j + lane;
        key[j] = u < u1 ? make_key(mx[u], static_cast<uint32_t>(u)) : 0ull;
      }
      key[kPickHeld] = mine;
      const int m = warp_collect(key, warp_bound(key, W, W), lane, kept);
      __syncwarp();
      mine = lane < min(m, W) ? kept[lane] : 0ull;
      __syncwarp();
    }
    kept[lane] = mine;
    __syncthreads();
  }
  if (w == 0) {
    const int count = sieve ? sifted : 32 * WARPS;
    const int m = count <= 64 ? warp_best<2>(keys, count, W, lane, keys)
                              : warp_best<kKeys / 32>(keys, count, W, lane, keys);
    const int unit = lane < m ? key_column(keys[lane]) : -1;
    if (P.grouped) {
      const int slot = unit >= 0 ? atomicAdd(P.count + unit, 1) : 0;
      __threadfence();
      __syncwarp();
      if (lane == 0) last = atomicAdd(P.done, 1) == static_cast<int>(gridDim.x) - 1;
      P.slot[static_cast<int64_t>(r) * 32 + lane] = slot;
    }
    P.pick[static_cast<int64_t>(r) * 32 + lane] = unit;
  }
  if (!P.grouped) return;
  __syncthreads();
  if (!last) return;
  __threadfence();
  constexpr int kAhead = 8;
  for (int first = 0; first < n; first += WARPS * 32 * kAhead) {
    const int u0 = first + threadIdx.x;
    int c[kAhead], mine[2] = {0, 0};  // rows and items of the thread's picks, of which a warp takes its places at once
#pragma unroll
    for (int i = 0; i < kAhead; ++i) c[i] = u0 + WARPS * 32 * i < n ? __ldcg(P.count + u0 + WARPS * 32 * i) : 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      mine[0] += c[i];
      mine[1] += (c[i] + kHeadDotRows - 1) / kHeadDotRows;
    }
    int to[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      int sum = mine[j];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      int before = 0;
      if (lane == 31) before = atomicAdd(&placed[j], sum);
      to[j] = __shfl_sync(0xffffffffu, before, 31) + sum - mine[j];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (c[i] == 0) continue;
      const int u = u0 + WARPS * 32 * i, items = (c[i] + kHeadDotRows - 1) / kHeadDotRows;
      const int at = to[0], it = to[1];
      to[0] += c[i];
      to[1] += items;
      P.base[u] = at;
      for (int k = 0; k < items; ++k)
        P.items[it + k] = make_int3(u, at + k * kHeadDotRows, min(kHeadDotRows, c[i] - k * kHeadDotRows));
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) P.done[1] = placed[1];
}

__global__ void __launch_bounds__(256) head_scatter_kernel(const __grid_constant__ HeadPicks P) {
  wait_for_previous_grid();
  const int p = blockIdx.x * 256 + threadIdx.x;
  if (p >= P.N * 32) return;
  const int u = P.pick[p];
  if (u >= 0) P.rows[P.base[u] + P.slot[p]] = p;
}

constexpr int kDotStep = 64;  // bytes of a row a step

// Bound on the error of a logit of head_dots_kernel (bf16), in units of |e| |c|, which bounds sum |e_d c_d|: an
// instruction adds 16 products and the running sum, each cut at 2^-24 of the largest, two of them a step; the steps and
// the warps' sums are added rounded to nearest, at most D / 128 + 10 additions.
__device__ __forceinline__ float dot_error(int D) {
  return (2.f * 17.f + 10.f + static_cast<float>(D) / 128.f) * 0x1p-24f;
}

// The row's softmax statistics from those of its segments: (m, s, w) and (m2, s2, w2) -> (m, s, w) of both.
__device__ __forceinline__ void join_stats(float& m, float& s, float& w, float m2, float s2, float w2, float sc) {
  const float mn = fmaxf(m, m2);
  if (mn == -INFINITY) {  // nothing but masked columns in either: the sums are 0, or NaN
    s += s2;
    return;
  }
  // a side without a maximum has the sums 0 (or NaN); below -1e4 the power is 0 and so is its product with d
  const float d = fmaxf((m - mn) * sc, -1e4f), d2 = fmaxf((m2 - mn) * sc, -1e4f);
  const float f = ex2(d), f2 = ex2(d2);
  w = f * fmaf(s, d, w) + f2 * fmaf(s2, d2, w2);
  s = f * s + f2 * s2;
  m = mn;
}

// WARPS warps per row, ROWS rows a block: the segments' statistics joined, then the row's outputs.
// Alternatives: the best 32 of the picks' logits, sorted. They carry the rounding of 32-bit sums, so where two
// neighbours are closer than that, their order (and which of them is the top_k-th) is not known yet: every run
// of such neighbours is computed again in 64 bits, a warp for each logit, and ordered by that, the lower id first among
// equal ones. What a sum loses grows with the magnitudes that it adds, not with what is left of them (two large
// features of opposite sign, a bias that takes most of the product away), so the bound is on |e| |c|, and for 8 bits,
// whose products are exact, on the product and the bias by themselves. Runs are short and few of the neighbours are in
// one, so this reads little (the call with 20 alternatives against a bound of 2^-15 of the logit, which misses those
// cases: 2048 x 2048 x 128256 997 us and 981, 1 x 4096 x 128256 194 and 191, 128 x 2048 x 128256 171 and 163).
// What it cannot see: a token that nine or more others displace, all of which are below it by less than the rounding,
// is not among the picks or the 32.
template <int WARPS, int ROWS>
__global__ void __launch_bounds__(WARPS * ROWS * 32) head_finish_kernel(const __grid_constant__ HeadFinish F) {
  __shared__ float stats[WARPS][3];
  __shared__ unsigned long long best[32];
  __shared__ double exact[32];
  __shared__ unsigned run_mask;
  if (!F.after_dots) wait_for_previous_grid();
  const int64_t r = static_cast<int64_t>(blockIdx.x) * ROWS + (threadIdx.x >> 5) / WARPS;
  if (r >= F.N) return;  // ROWS > 1 only: there nothing below waits for other warps
  const int lane = threadIdx.x & 31, wi = (threadIdx.x >> 5) % WARPS;
  const HeadSplit& S = F.split;
  const int b = static_cast<int>(r / kHeadBM);
  int g = static_cast<int>(static_cast<long long>(b) * S.ngroups / S.nb);  // the group of row block b, or one off
  while (S.group_begin(g) > b) --g;
  while (S.group_begin(g + 1) <= b) ++g;
  const int b0 = S.group_begin(g), gb = S.group_begin(g + 1) - b0;
  const int total = S.units(gb), P = S.parts(total);
  const int nseg = kHeadParts * (HeadSplit::owner(S.units(b - b0 + 1) - 1, total, P) -
                                 HeadSplit::owner(S.units(b - b0), total, P) + 1);
  const bool failed = *F.failed != 0;
  const float sc = F.inv_t * kLog2e;

  float m = -INFINITY, s = 0.f, w = 0.f;
#pragma unroll 4
  for (int i = wi * 32 + lane; i < nseg; i += 32 * WARPS) {
    const int64_t o = static_cast<int64_t>(i) * F.N + r;
    join_stats(m, s, w, F.part_m[o], F.part_s[o], F.part_w[o], sc);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o),
                w2 = __shfl_xor_sync(0xffffffffu, w, o);
    join_stats(m, s, w, m2, s2, w2, sc);
  }
  if (WARPS > 1) {
    if (lane == 0) {
      stats[wi][0] = m;
      stats[wi][1] = s;
      stats[wi][2] = w;
    }
    __syncthreads();
    m = stats[0][0];
    s = stats[0][1];
    w = stats[0][2];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) join_stats(m, s, w, stats[i][0], stats[i][1], stats[i][2], sc);
  } else {
    // one lane's sums for all: two lanes joined the same pair from either side, with the last bit theirs
    m = __shfl_sync(0xffffffffu, m, 0);
    s = __shfl_sync(0xffffffffu, s, 0);
    w = __shfl_sync(0xffffffffu, w, 0);
  }
  const float ln_s = logf(s);
  const float nan = __int_as_float(0x7fffffff);
  const bool none = m == -INFINITY && s == 0.f;  // every logit of the row is -inf
  if (F.K > 0 && wi == 0) {
    bool any = false;
    int place = 0;  // of the lane's token among the row's, see head_tokens_kernel
    if (F.K > 1) {
      const int mine = lane < F.K ? token_or_none(F.tokens[r * F.K + lane], F.ignore_index, F.V) : kNoToken;
      for (int k = 0; k < F.K; ++k) {
        const int other = __shfl_sync(0xffffffffu, mine, k);
        place += other < mine || (other == mine && k < lane) ? 1 : 0;
      }
    }
    if (lane < F.K) {
      const int64_t id = F.tokens[r * F.K + lane];
      float lp = 0.f;
      if (id != F.ignore_index) {
        any = true;
        if (id < 0 || id >= F.V) {
          record_error(F.err, kErrTargetRange);
          lp = nan;
        } else {
          lp = none ? -INFINITY : (F.zt[static_cast<int64_t>(place) * F.N + r] - m) * F.inv_t - ln_s;
        }
      }
      F.logprobs[r * F.K + lane] = failed ? nan : lp;
    }
    any = __any_sync(0xffffffffu, any);
    if (lane == 0) {
      const float h = none || !any ? 0.f : ln_s - 0.6931471805599453f * (w / s);
      F.entropy[r] = failed ? nan : h;
      F.lse[r] = failed ? nan : (none ? -INFINITY : fmaf(m, F.inv_t, ln_s));
      if (F.row_max != nullptr) {
        F.row_max[r] = failed ? nan : m;
        F.row_ln_s[r] = failed ? nan : ln_s;
      }
    }
  }
  if (ROWS > 1 || F.top_k == 0) return;
  if (failed) {
    if (threadIdx.x < F.top_k) {
      F.top_logprobs[r * F.top_k + threadIdx.x] = nan;
      F.top_ids[r * F.top_k + threadIdx.x] = -1;
    }
    return;
  }

  float e_norm = 0.f;  // of the row of E, while the picks' logits are still being formed
  if (wi == 0 && F.C8 == nullptr) {
    const __nv_bfloat16* e = F.E + r * F.D;
#pragma unroll 4
    for (int d = lane * 8; d < F.D; d += 256) e_norm += sum_squares(ld_global_nc_v4(e + d));
    e_norm = sqrtf(warp_sum(e_norm));
  }
  wait_for_previous_grid();  // the picks' logits
  if (wi == 0) {
    unsigned long long key[kHeadPick];
#pragma unroll
    for (int i = 0; i < kHeadPick; ++i) {
      const int j = 2 * i + (lane >> 4);  // two picks a step
      const int unit = j < F.wanted ? F.pick[r * 32 + j] : -1;
      const int c = unit * kHeadPick + (lane & 15);
      key[i] = unit >= 0 && c < F.V
                   ? make_key(F.logits[(r * 32 + j) * kHeadPick + (lane & 15)], static_cast<uint32_t>(c))
                   : 0ull;
    }
    const unsigned long long bound = warp_bound(key, 32, 32);
    best[lane] = 0;
    __syncwarp();
    warp_collect(key, bound, lane, best);
    __syncwarp();
    const unsigned long long mine = warp_sort(best[lane], lane);
    best[lane] = mine;
    const float v = key_value(mine);
    // What the two of a pair may be off: the sum of products, and the rounding of z (or for 8 bits, with |product| <=
    // |z| + |bias|, three roundings of the product and that of z).
    float off = 0x1p-24f * fabsf(v);
    if (F.C8 != nullptr) {
      const float b = F.bias != nullptr && mine != 0 ? fabsf(__bfloat162float(F.bias[key_column(mine)])) : 0.f;
      off += 0x1.8p-23f * (fabsf(v) + b);
    } else {
      float c_norm = lane < F.wanted && F.pick[r * 32 + lane] >= 0 ? F.norm[r * 32 + lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) c_norm = max_nan(c_norm, __shfl_xor_sync(0xffffffffu, c_norm, o));
      off += dot_error(F.D) * 1.01f * e_norm * c_norm;
    }
    const float tol = off + __shfl_up_sync(0xffffffffu, off, 1);
    const float before = __shfl_up_sync(0xffffffffu, v, 1);
    const bool close = lane > 0 && mine != 0 && isfinite(v) && isfinite(before) && before - v <= tol;
    unsigned joins = __ballot_sync(0xffffffffu, close);  // bit i: i is close to i - 1
    if (F.top_k < 32) {  // runs that start behind the last alternative do not matter
      const unsigned behind = joins >> F.top_k;
      const unsigned reach = ~behind == 0 ? 32u : static_cast<unsigned>(__ffs(static_cast<int>(~behind)) - 1);
      const unsigned end = F.top_k + reach;
      if (end < 32) joins &= (1u << end) - 1u;
    }
    exact[lane] = static_cast<double>(v);
    if (lane == 0) run_mask = joins;
  }
  __syncthreads();
  const unsigned joins = run_mask, runs = joins | (joins >> 1);  // members of a run
  int turn = 0;
  for (unsigned todo = runs; todo != 0; todo &= todo - 1, ++turn) {
    if (turn % WARPS != wi) continue;
    const int i = __ffs(todo) - 1;
    const double z = exact_logit(F, r, key_column(best[i]), lane);
    if (lane == 0) exact[i] = z;
  }
  __syncthreads();
  if (wi != 0) return;
  const bool in = best[lane] != 0;
  const int col = in ? key_column(best[lane]) : -1;
  const double zx = exact[lane];
  int place = lane;
  if ((runs >> lane) & 1u) {
    const unsigned starts = ~joins;  // bit i: a run (or a single one) starts at i
    place = 31 - __clz(static_cast<int>(starts & (0xffffffffu >> (31 - lane))));
    const int first = place;
    for (int i = first; i < 32 && (i == first || ((joins >> i) & 1u)); ++i) {
      const double zi = exact[i];
      if (i != lane && (zi > zx || (zi == zx && key_column(best[i]) < col))) ++place;
    }
  }
  if (place < F.top_k && in) {
    const float lp = m == -INFINITY ? -INFINITY
                                    : static_cast<float>((zx - static_cast<double>(m)) *
                                                         static_cast<double>(F.inv_t)) - ln_s;
    F.top_logprobs[r * F.top_k + place] = s != s ? nan : lp;
    F.top_ids[r * F.top_k + place] = col;
  }
}

__device__ __forceinline__ void mma_16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16x8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A work item: 16 columns x up to 64 gathered rows. The operands are the rows themselves, read 64 bytes a row and
// step: the WARPS warps take the steps in turn and their sums are added through shared memory. Four warps, and four
// blocks an SM, where there are many items (2048 rows of D = 2048: 116 us, 120 with eight warps and two blocks),
// eight where there are few and each should be done soon. A lane's 16 bytes of a row feed two instructions whose K
// positions are the same bytes of both operands, so nothing is rearranged.
// Rows picked by index suit neither a TMA box nor an M = 128 tile (a pick has 7 rows of 2048 on average); the warp
// instruction's 16-row tile wastes little, and the kernel is bound by reading C once.
// sq (bf16): sums of squares of the pick's rows of C, from the same loads.
template <bool I8, int WARPS, int TILES, int UNROLL, typename Acc>
__device__ __forceinline__ void dot_item(const HeadPicks& P, int pick, int n, const int* ids,
                                         Acc* red, float* sq, int64_t pitch, int lane, int w) {
  const int g = lane >> 2, t = lane & 3;
  const int steps = static_cast<int>((pitch + kDotStep - 1) / kDotStep);
  const char* er[TILES][2];
#pragma unroll
  for (int mt = 0; mt < TILES; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      er[mt][h] = static_cast<const char*>(P.E) + (ids[min(16 * mt + 8 * h + g, n - 1)] >> 5) * pitch + t * 16;
  const char* cr[2];
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
    cr[nt] = static_cast<const char*>(P.C) + min(pick * kHeadPick + 8 * nt + g, P.V - 1) * pitch + t * 16;
  Acc sum[TILES][2][4] = {};
  float squares[2][4] = {};
#pragma unroll 1
  for (int s = w; s < steps; s += WARPS * UNROLL) {
    uint4 b[UNROLL][2], a[UNROLL][TILES][2];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t off = static_cast<int64_t>(s + u * WARPS) * kDotStep;
      const bool in = s + u * WARPS < steps && off + t * 16 < pitch;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) b[u][nt] = in ? ld_global_nc_v4(cr[nt] + off) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int mt = 0; mt < TILES; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          a[u][mt][h] = in ? ld_global_nc_v4(er[mt][h] + off) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
        for (int mt = 0; mt < TILES; ++mt) {
          const uint4 x = a[u][mt][0], y = a[u][mt][1];
          if constexpr (I8) {
            mma_16x8(sum[mt][nt], x.x, y.x, x.y, y.y, b[u][nt].x, b[u][nt].y);
            mma_16x8(sum[mt][nt], x.z, y.z, x.w, y.w, b[u][nt].z, b[u][nt].w);
          } else {  // a step by itself, so that little is cut (dot_error)
            float acc[4] = {};
            mma_16x8(acc, x.x, y.x, x.y, y.y, b[u][nt].x, b[u][nt].y);
            mma_16x8(acc, x.z, y.z, x.w, y.w, b[u][nt].z, b[u][nt].w);
#pragma unroll
            for (int i = 0; i < 4; i += 2)
              unpack2(add2(pack2(sum[mt][nt][i], sum[mt][nt][i + 1]), pack2(acc[i], acc[i + 1])), sum[mt][nt][i],
                      sum[mt][nt][i + 1]);
          }
        }
        if constexpr (!I8) {  // the pick's rows by themselves: their squares are on the diagonal
          const uint4 x = b[u][0], y = b[u][1];
          mma_16x8(squares[nt], x.x, y.x, x.y, y.y, b[u][nt].x, b[u][nt].y);
          mma_16x8(squares[nt], x.z, y.z, x.w, y.w, b[u][nt].z, b[u][nt].w);
        }
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < TILES; ++mt)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[(16 * mt + g + 8 * (i >> 1)) * kHeadPick + 8 * nt + 2 * t + (i & 1)] = sum[mt][nt][i];
  if (!I8 && g >> 1 == t) {  // rows 8 nt + g, columns 8 nt + 2 t and the next
    sq[g] = (g & 1) ? squares[0][1] : squares[0][0];
    sq[8 + g] = (g & 1) ? squares[1][3] : squares[1][2];
  }
}

// Ungrouped (ROWS = 16) every row has its own items.
template <bool I8, int WARPS, int ROWS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS)
    head_dots_kernel(const __grid_constant__ HeadPicks P) {
  constexpr bool kGrouped = ROWS > 16;
  using Acc = typename std::conditional<I8, int, float>::type;
  __shared__ Acc red[WARPS][ROWS * kHeadPick];
  __shared__ float sq[WARPS][kHeadPick];
  __shared__ int ids[kHeadDotRows];
  wait_for_previous_grid();
  let_next_grid_start();  // the head kernel has ended: the finish may join its statistics meanwhile
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t pitch = static_cast<int64_t>(P.D) * (I8 ? 1 : 2);  // a multiple of 16 bytes
  const int nitems = kGrouped ? P.done[1] : P.N * P.wanted;
  for (int it = blockIdx.x; it < nitems; it += gridDim.x) {
    const int pair = it / P.wanted * 32 + it % P.wanted;  // ungrouped: the row's pick
    const int3 item = kGrouped ? P.items[it] : make_int3(P.pick[pair], 0, 1);
    __syncthreads();  // the previous item's sums and ids have been read
    if (threadIdx.x < item.z) ids[threadIdx.x] = kGrouped ? P.rows[item.y + threadIdx.x] : pair;
    __syncthreads();
    if (kGrouped || item.x >= 0) {
      if (ROWS <= 16 || item.z <= 16) dot_item<I8, WARPS, 1, 4>(P, item.x, item.z, ids, red[w], sq[w], pitch, lane, w);
      else dot_item<I8, WARPS, ROWS / 16, 1>(P, item.x, item.z, ids, red[w], sq[w], pitch, lane, w);
      __syncthreads();
      for (int i = threadIdx.x; i < item.z * kHeadPick; i += WARPS * 32) {
        Acc z = 0;
  #pragma unroll
        for (int k = 0; k < WARPS; ++k) z += red[k][i];
        const int p = ids[i / kHeadPick], col = item.x * kHeadPick + i % kHeadPick;
        if (col < P.V) {
          float v = static_cast<float>(z);
          if (I8) v *= P.e_scale[p >> 5] * P.c_scale[col];
          if (P.bias != nullptr) v += __bfloat162float(P.bias[col]);
          P.logits[static_cast<int64_t>(p) * kHeadPick + i % kHeadPick] = v;
        }
        if (!I8) {  // the largest norm of the pick's rows of C, by the 16 threads of a row
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < WARPS; ++k) s += sq[k][i % kHeadPick];
#pragma unroll
          for (int o = kHeadPick / 2; o > 0; o >>= 1)
            s = max_nan(s, __shfl_xor_sync(0xffffu << (lane & 16), s, o));
          if (i % kHeadPick == 0) P.norm[p] = sqrtf(s);
        }
      }
    }
  }
}

// tokens [N, K] -> tok_t [K, N], each row's in ascending order, equal ones in the order given, and those that ask for
// nothing behind the others: the head kernel's warps read the next token of 32 rows at once.
__global__ void __launch_bounds__(256) head_tokens_kernel(const int64_t* __restrict__ tokens, int N, int K, int V,
                                                          int64_t ignore_index, int* __restrict__ tok_t) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  let_next_grid_start();
  if (i >= static_cast<int64_t>(N) * K) return;
  const int64_t r = i / K;
  const int mine_at = static_cast<int>(i - r * K), mine = token_or_none(tokens[i], ignore_index, V);
  int place = 0;
  for (int k = 0; k < K; ++k) {
    const int other = token_or_none(tokens[r * K + k], ignore_index, V);
    place += other < mine || (other == mine && k < mine_at) ? 1 : 0;
  }
  tok_t[place * static_cast<int64_t>(N) + r] = mine;
}

// One block per row: the largest magnitude, then the integers. scale = max |x| / 127, rounded to nearest; q is the
// integer nearest to x / scale, the even one of two equally near. A 32-bit quotient that falls on a half may have
// been rounded there: the sign of x - quotient * scale, exact in one fused operation, says on which side it was.
// A row that holds an infinity or a NaN gets the scale NaN.
constexpr int kQuantThreads = 256;

__device__ __forceinline__ int quantized(float x, float scale) {
  const float t = __fdiv_rn(x, scale);
  float q = rintf(t);
  if (fabsf(t - truncf(t)) == 0.5f) {
    const float rest = fmaf(-t, scale, x);
    if (rest > 0.f) q = ceilf(t);
    else if (rest < 0.f) q = floorf(t);
  }
  return static_cast<int>(q);
}

__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const __nv_bfloat16* __restrict__ x, int64_t rows,
                                                                      int64_t D, int8_t* __restrict__ q,
                                                                      float* __restrict__ scale) {
  __shared__ float wmax[kQuantThreads / 32];
  let_next_grid_start();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const __nv_bfloat16* src = x + r * D;
    float m = 0.f;
    for (int64_t d = threadIdx.x * 8; d < D; d += kQuantThreads * 8) {
      const uint4 u = ld_global_nc_v4(src + d);
      const uint32_t us[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m = max_nan(m, fabsf(__uint_as_float(us[k] << 16)));
        m = max_nan(m, fabsf(__uint_as_float(us[k] & 0xffff0000u)));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();  // the previous row's maxima have been read
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kQuantThreads / 32; ++k) m = max_nan(m, wmax[k]);
    const bool fine = m <= 3.4028234e38f;
    const float sc = fine ? __fdiv_rn(m, 127.f) : __int_as_float(0x7fffffff);
    if (threadIdx.x == 0) scale[r] = sc;
    const bool zero = !fine || sc == 0.f;
    for (int64_t d = threadIdx.x * 8; d < D; d += kQuantThreads * 8) {
      const uint4 u = ld_global_nc_v4(src + d);
      const uint32_t us[4] = {u.x, u.y, u.z, u.w};
      uint32_t o[2] = {0, 0};
      if (!zero) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int lo = quantized(__uint_as_float(us[k] << 16), sc);
          const int hi = quantized(__uint_as_float(us[k] & 0xffff0000u), sc);
          o[k >> 1] |= (static_cast<uint32_t>(lo & 0xff) | (static_cast<uint32_t>(hi & 0xff) << 8)) << (16 * (k & 1));
        }
      }
      *reinterpret_cast<uint2*>(q + r * D + d) = make_uint2(o[0], o[1]);
    }
  }
}

template <bool I8, int OUT>
cudaError_t launch_one(const HeadMaps& M, const HeadArgs& A, bool after_kernel, cudaStream_t s) {
  auto kernel = head_kernel<I8, OUT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  if (after_kernel) {
    e = launch_after_previous(kernel, dim3(A.split.grid), dim3(NUM_THREADS), SMEM_BYTES, s, M.E, M.C, M.C64, M.out, A);
    if (e != cudaSuccess) return e;
  } else {
    kernel<<<A.split.grid, NUM_THREADS, SMEM_BYTES, s>>>(M.E, M.C, M.C64, M.out, A);
  }
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_head(const HeadMaps& M, const HeadArgs& A, bool int8, bool after_kernel, cudaStream_t s) {
  if (A.out != nullptr) {
    return A.out_fp32 ? launch_one<true, 2>(M, A, after_kernel, s) : launch_one<true, 1>(M, A, after_kernel, s);
  }
  if (int8) return launch_one<true, 0>(M, A, after_kernel, s);
  return launch_one<false, 0>(M, A, after_kernel, s);
}

cudaError_t launch_head_picks(HeadPicks P, const HeadFinish& F, bool int8, int sms, cudaStream_t s) {
  P.grouped = picks_grouped(P.N) ? 1 : 0;
  // with few rows each gets more warps, as the machine is not full
  cudaError_t e = P.N < 2 * sms ? launch_after_previous(head_pick_kernel<32>, dim3(P.N), dim3(1024), 0, s, P)
                                : launch_after_previous(head_pick_kernel<8>, dim3(P.N), dim3(256), 0, s, P);
  if (e != cudaSuccess) return e;
  if (!P.grouped) {
    const dim3 grid(std::min(P.N * P.wanted, 2 * sms));
    e = int8 ? launch_after_previous(head_dots_kernel<true, 8, 16>, grid, dim3(256), 0, s, P)
             : launch_after_previous(head_dots_kernel<false, 8, 16>, grid, dim3(256), 0, s, P);
    if (e != cudaSuccess) return e;
    note_launches(2);
    return launch_head_finish(F, s);
  }
  e = launch_after_previous(head_scatter_kernel, dim3((P.N * 32 + 255) / 256), dim3(256), 0, s, P);
  if (e != cudaSuccess) return e;
  const dim3 grid(std::min(P.N * 32, 4 * sms));
  e = int8 ? launch_after_previous(head_dots_kernel<true, 4, kHeadDotRows>, grid, dim3(128), 0, s, P)
           : launch_after_previous(head_dots_kernel<false, 4, kHeadDotRows>, grid, dim3(128), 0, s, P);
  if (e != cudaSuccess) return e;
  note_launches(3);
  return launch_head_finish(F, s);
}

cudaError_t launch_head_finish(HeadFinish F, cudaStream_t s) {
  F.after_dots = F.top_k > 0 ? 1 : 0;
  // A block of eight warps per row where a row has very many segments (one or two row blocks share the machine), so
  // that they are read at once; else two where alternatives are to be ordered; else a warp per row, four rows a block.
  cudaError_t e;
  if (F.split.max_segments() > 64) {
    e = launch_after_previous(head_finish_kernel<8, 1>, dim3(F.N), dim3(256), 0, s, F);
  } else if (F.top_k > 0) {
    e = launch_after_previous(head_finish_kernel<2, 1>, dim3(F.N), dim3(64), 0, s, F);
  } else {
    e = launch_after_previous(head_finish_kernel<1, 4>, dim3((F.N + 3) / 4), dim3(128), 0, s, F);
  }
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_head_tokens(const int64_t* tokens, int N, int K, int V, int64_t ignore_index, int* tok_t,
                               cudaStream_t s) {
  const int64_t n = static_cast<int64_t>(N) * K;
  head_tokens_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(tokens, N, K, V, ignore_index, tok_t);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_quantize_rows(const __nv_bfloat16* x, int64_t rows, int64_t D, int8_t* q, float* scale,
                                 cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  quantize_rows_kernel<<<static_cast<unsigned>(std::min<int64_t>(rows, 148 * 8)), kQuantThreads, 0, s>>>(x, rows, D, q,
                                                                                                       scale);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace cce
