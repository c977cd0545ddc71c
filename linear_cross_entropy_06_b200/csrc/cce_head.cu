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
// Design (B200): one persistent block per SM, 12 warps.
//   warp 0       producer: E and C K-blocks of 128 bytes (128B swizzle) by TMA into a 4-stage ring.
//   warp 1       tensor memory owner; one lane issues tcgen05.mma, M = 128 rows, N = up to 256 columns.
//   warps 4..11  epilogue, two warps for each 32 rows (one for each 128 columns of the tile): a thread owns
//                128 logits of one row, in registers.
// Sums over K: the tensor cores add into their fp32 accumulator without rounding to nearest, so a long sum
// drifts towards zero (D = 4096, logits of 11: -5e-5, sixteen times what fp32 sums lose). The accumulator is
// therefore handed over every kb_chunk K-blocks (512 values of K) and the parts are added in registers, rounded
// to nearest: two tensor-memory buffers alternate by parts, and the drift falls with the parts' number.
// 8-bit products are exact in 32-bit integers, so they keep one part.
#include <algorithm>

#include "cce_device.cuh"
#include "cce_head.h"
#include "cce_internal.h"

namespace cce {
namespace {

constexpr int BM = kHeadBM;
constexpr int BN = kHeadBN;
constexpr int KB_BYTES = 128;  // one swizzle row: 64 bf16 or 128 8-bit values of K
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * KB_BYTES;
constexpr int B_BYTES = BN * KB_BYTES;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int NUM_THREADS = 384;
constexpr int EPI_THREADS = 256;
constexpr int TMEM_COLS = 512;
constexpr int NUM_BARRIERS = 2 * STAGES + 4 + 1;
constexpr int SCRATCH_WARP = 4096;  // of each epilogue warp: its rows' tokens, or a piece of the logits on its way out
constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + 8 * SCRATCH_WARP + NUM_BARRIERS * 8 + 16;
static_assert(SMEM_BYTES <= 232448, "fits the 227 KB opt-in shared memory of an SM");
static_assert(kHeadMaxTokens * 32 * 4 <= SCRATCH_WARP, "the tokens of a warp's 32 rows fit its scratch");

// Registers a thread: 384 threads are launched with 168 each; the first warpgroup hands 128 of its own to the two
// that hold logits and lists in registers (56 x 128 + 224 x 256 = 168 x 384).
constexpr int REGS_FEW = 40, REGS_MANY = 232;
static_assert(REGS_FEW * 128 + REGS_MANY * 256 <= 168 * 384, "setmaxnreg draws on the launch's registers");

template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

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

// 32 lanes x 16 consecutive columns of tensor memory.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// The larger of two numbers, NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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

// One tile of a block's walk.
struct HeadTile {
  int b;           // row block
  int seg;         // segment of the row block
  int col, ncol;   // its first column, and how many
  bool first, last;  // of the segment
};

// Calls f(tile) for every tile of block c, in the order that all roles share; f returns false to stop. Within a
// segment the walk starts at the tile whose position is 0 modulo the length of a block's share: the blocks on
// different row blocks then pass the same columns of C at about the same time, and C is read from HBM about once
// a group.
template <typename F>
__device__ __forceinline__ void for_tiles(const HeadSplit& S, int V, int c, F&& f) {
  for (int g = 0; g < S.ngroups; ++g) {
    int x, hi;
    {
      const int total = S.units(S.group_begin(g + 1) - S.group_begin(g)), P = S.parts(total);
      if (c >= P) continue;
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

// v[i] = c_scale[col0 + i] (columns from `limit` on: 0), 32 columns from a multiple of 32.
__device__ __forceinline__ void load_scale32(float (&v)[32], const float* scale, int col0, int limit) {
  if (col0 + 32 <= limit) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint4 u = ld_global_nc_v4(scale + col0 + 4 * q);
      v[4 * q] = __uint_as_float(u.x);
      v[4 * q + 1] = __uint_as_float(u.y);
      v[4 * q + 2] = __uint_as_float(u.z);
      v[4 * q + 3] = __uint_as_float(u.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = col0 + i < limit ? scale[col0 + i] : 0.f;
  }
}

// a[i] of 32 registers, i in the lane's own register: five levels of selection.
__device__ __forceinline__ float pick32(const float* a, int i) {
  float t16[16], t8[8], t4[4], t2[2];
#pragma unroll
  for (int k = 0; k < 16; ++k) t16[k] = (i & 16) ? a[k + 16] : a[k];
#pragma unroll
  for (int k = 0; k < 8; ++k) t8[k] = (i & 8) ? t16[k + 8] : t16[k];
#pragma unroll
  for (int k = 0; k < 4; ++k) t4[k] = (i & 4) ? t8[k + 4] : t8[k];
#pragma unroll
  for (int k = 0; k < 2; ++k) t2[k] = (i & 2) ? t4[k + 2] : t4[k];
  return (i & 1) ? t2[1] : t2[0];
}

// L: entries of a thread's list of best keys (0: none). OUT: the logits are written out instead of reduced.
template <bool I8, int L, bool OUT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    head_kernel(const __grid_constant__ CUtensorMap tmE, const __grid_constant__ CUtensorMap tmC,
                const __grid_constant__ HeadArgs A) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* scratch = base + STAGES * STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(scratch + 8 * SCRATCH_WARP);
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
      mbar_init(tempty_bar(a), EPI_THREADS);
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
  wait_for_previous_grid();  // the 8-bit rows of E, when a kernel of this call made them
  const WaitCtl wc{abort_flag, A.err, A.timeout_ns};
  const int num_kb = A.num_kb;
  constexpr int KE = I8 ? KB_BYTES : KB_BYTES / 2;  // values of K a block

  if (warp < 4) {
    regs_dec<REGS_FEW>();
    if (warp == 0) {
      // ---------------- producer ----------------
      // inject_stall (test hook): nothing is loaded, so the bounded wait of the next role runs out.
      if (lane == 0 && !A.inject_stall) {
        int stage = 0;
        uint32_t phase = 0;
        uint32_t issued[STAGES] = {0, 0, 0, 0};
        bool ok = true;
        const uint32_t e_bytes = static_cast<uint32_t>(A.e_rows) * KB_BYTES;
        const uint32_t box_bytes = static_cast<uint32_t>(A.box_c) * KB_BYTES;
        for_tiles(A.split, A.V, blockIdx.x, [&](const HeadTile& t) {
          const int nbox = (t.ncol + A.box_c - 1) / A.box_c;
          for (int kb = 0; kb < num_kb; ++kb) {
            if (!mbar_wait(empty_bar(stage), phase ^ 1u, wc)) return ok = false;
            const uint32_t dst = smem_u32(base + stage * STAGE_BYTES);
            mbar_arrive_expect_tx(full_bar(stage), e_bytes + static_cast<uint32_t>(nbox) * box_bytes);
            tma_load_2d(dst, &tmE, full_bar(stage), kb * KE, t.b * BM);
            for (int j = 0; j < nbox; ++j)
              tma_load_2d(dst + A_BYTES + static_cast<uint32_t>(j) * box_bytes, &tmC, full_bar(stage), kb * KE,
                          t.col + j * A.box_c);
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
        for_tiles(A.split, A.V, blockIdx.x, [&](const HeadTile& t) {
          const uint32_t idesc = idesc_n(I8, (t.ncol + A.box_c - 1) / A.box_c * A.box_c);
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
  } else {
    // ---------------- epilogue ----------------
    regs_inc<REGS_MANY>();
    const int q = warp & 3;            // tensor-memory lanes of this warp
    const int half = (warp - 4) >> 2;  // columns 128 half .. 128 half + 127 of a tile
    const uint32_t tquarter = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * 128);
    uint8_t* mine = scratch + (warp - 4) * SCRATCH_WARP;
    int* tok_s = reinterpret_cast<int*>(mine);  // [K][32]: the tokens of this warp's rows, -1 for none
    int acc = 0;
    uint32_t acc_phase = 0;
    const float sc = A.inv_t * kLog2e;
    float m = -INFINITY, s = 0.f, w = 0.f;
    unsigned long long list[L > 0 ? L : 1];
    float a[128];
    for_tiles(A.split, A.V, blockIdx.x, [&](const HeadTile& t) {
      const int r = t.b * BM + q * 32 + lane;
      const bool rows = t.b * BM + q * 32 < A.N;  // any row of this warp
      const int ncol = min(128, t.ncol - half * 128);  // columns of this warp (none if <= 0)
      const int col0 = t.col + half * 128;
      if (!OUT && t.first) {
        m = -INFINITY;
        s = w = 0.f;
        if constexpr (L > 0) {
#pragma unroll
          for (int j = 0; j < L; ++j) list[j] = 0;
        }
        __syncwarp();
        for (int k = 0; k < A.K; ++k) {
          const int64_t id = r < A.N ? A.tokens[static_cast<int64_t>(r) * A.K + k] : -1;
          tok_s[k * 32 + lane] = id != A.ignore_index && id >= 0 && id < A.V ? static_cast<int>(id) : -1;
        }
        __syncwarp();
      }
      for (int k0 = 0; k0 < num_kb; k0 += A.kb_chunk) {
        const bool got = mbar_wait(tfull_bar(acc), acc_phase, wc);
        if (!__all_sync(0xffffffffu, got ? 1 : 0)) return false;
        tc_fence_after();
        if (rows && ncol > 0) {
          const uint32_t src = tquarter + static_cast<uint32_t>(acc * BN);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (32 * j < ncol) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float v[16];
                tmem_ld16(src + 32u * j + 16u * h, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const int n = 32 * j + 16 * h + i;
                  if (I8) a[n] = static_cast<float>(__float_as_int(v[i]));
                  else a[n] = k0 == 0 ? v[i] : a[n] + v[i];
                }
              }
            }
          }
        }
        tc_fence_before();
        mbar_arrive(tempty_bar(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!rows) return true;
      if (ncol > 0) {
        const float es = I8 && r < A.N ? A.e_scale[r] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (32 * j >= ncol) {
#pragma unroll
            for (int i = 0; i < 32; ++i) a[32 * j + i] = -INFINITY;
            continue;
          }
          float v[32];
          if (I8) {
            load_scale32(v, A.c_scale, col0 + 32 * j, A.V);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = a[32 * j + i] * (es * v[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = a[32 * j + i];
          }
          if (A.bias != nullptr) add_bias32(v, A.bias, col0 + 32 * j, A.V);
#pragma unroll
          for (int i = 0; i < 32; ++i) a[32 * j + i] = 32 * j + i < ncol ? v[i] : -INFINITY;
        }
        if constexpr (OUT) {
          // 32 rows x 32 columns at a time through the warp's scratch, then whole rows of it: 32 lanes write one
          // row's 32 columns, whatever the alignment of V.
          float* st = reinterpret_cast<float*>(mine);
          const int n_rows = min(32, A.N - (t.b * BM + q * 32));
          const int64_t row0 = static_cast<int64_t>(t.b) * BM + q * 32;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (32 * j >= ncol) break;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 32; ++i) st[lane * 32 + ((i + lane) & 31)] = a[32 * j + i];
            __syncwarp();
            const bool in = 32 * j + lane < ncol;
            for (int k = 0; k < n_rows; ++k) {
              const float v = st[k * 32 + ((lane + k) & 31)];
              const int64_t o = (row0 + k) * A.V + col0 + 32 * j + lane;
              if (in) {
                if (A.out_fp32) static_cast<float*>(A.out)[o] = v;
                else static_cast<__nv_bfloat16*>(A.out)[o] = __float2bfloat16_rn(v);
              }
            }
          }
        } else {
          // the given tokens of the row among these columns
          for (int k = 0; k < A.K; ++k) {
            const int id = tok_s[k * 32 + lane];
            const int at = id - col0;
            const bool hit = id >= 0 && at >= 0 && at < ncol;
            if (!__any_sync(0xffffffffu, hit)) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool here = hit && (at >> 5) == j;
              if (__any_sync(0xffffffffu, here)) {
                const float z = pick32(a + 32 * j, at & 31);
                if (here) A.zt[static_cast<int64_t>(k) * A.N + r] = z;
              }
            }
          }
          float cm[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x = a[32 * j];
#pragma unroll
            for (int i = 1; i < 32; ++i) x = fmaxf(x, a[32 * j + i]);
            cm[j] = x;
          }
          if (A.tile_max != nullptr && r < A.N) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (64 * j < ncol)
                A.tile_max[static_cast<int64_t>((col0 >> 6) + j) * A.N + r] = fmaxf(cm[2 * j], cm[2 * j + 1]) * A.inv_t;
            }
          }
          const float mt = fmaxf(fmaxf(cm[0], cm[1]), fmaxf(cm[2], cm[3]));
          const float mn = fmaxf(m, mt);
          if (mn == -INFINITY) {  // nothing but -inf (masked columns) so far; a NaN among them still counts
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (a[i] != a[i]) s = a[i];
          } else {
            if (m != mn && m != -INFINITY) {
              const float d = (m - mn) * sc, f = ex2(d);
              w = f * fmaf(s, fmaxf(d, -1e30f), w);
              s *= f;
            }
            m = mn;
            float s0 = 0.f, s1 = 0.f, w0 = 0.f, w1 = 0.f;
#pragma unroll
            for (int i = 0; i < 128; i += 2) {
              // below -1e4 (a masked column: -inf) the power is 0, and so is its product with d
              const float d0 = max_nan((a[i] - mn) * sc, -1e4f), d1 = max_nan((a[i + 1] - mn) * sc, -1e4f);
              const float e0 = ex2(d0), e1 = ex2(d1);
              s0 += e0;
              s1 += e1;
              w0 = fmaf(d0, e0, w0);
              w1 = fmaf(d1, e1, w1);
            }
            s += s0 + s1;
            w += w0 + w1;
          }
          if constexpr (L > 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // no key of these 32 columns is above that of their largest logit at their first column
              const uint32_t cj = static_cast<uint32_t>(col0 + 32 * j);
              if (32 * j >= ncol || !__any_sync(0xffffffffu, make_key(cm[j], cj) > list[L - 1])) continue;
              const float low = key_value(list[L - 1]);
              uint32_t bits = 0;
#pragma unroll
              for (int i = 0; i < 32; ++i) bits |= (a[32 * j + i] >= low ? 1u : 0u) << i;
              const int left = ncol - 32 * j;
              if (left < 32) bits &= (1u << left) - 1u;
              while (__any_sync(0xffffffffu, bits != 0)) {
                const int i = __ffs(bits) - 1;  // -1 where this lane has none left
                unsigned long long x = 0;
                if (i >= 0) x = make_key(pick32(a + 32 * j, i), cj + static_cast<uint32_t>(i));
                bits &= bits - 1;
                if (!__any_sync(0xffffffffu, x > list[L - 1])) continue;
#pragma unroll
                for (int k = 0; k < L; ++k) {  // the list stays sorted; what falls out at the end is dropped
                  const unsigned long long y = list[k];
                  const bool up = x > y;
                  list[k] = up ? x : y;
                  x = up ? y : x;
                }
              }
            }
          }
        }
      }
      if (!OUT && t.last && r < A.N) {
        const int64_t o = static_cast<int64_t>(2 * t.seg + half) * A.N + r;
        A.part_m[o] = m;
        A.part_s[o] = s;
        A.part_w[o] = w;
        if constexpr (L > 0) {
          ulonglong2* dst = reinterpret_cast<ulonglong2*>(A.lists + o * L);
#pragma unroll
          for (int k = 0; k < L; k += 2) dst[k / 2] = make_ulonglong2(list[k], list[k + 1]);
        }
      }
      return true;
    });
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long u = __shfl_xor_sync(0xffffffffu, v, o);
    v = u > v ? u : v;
  }
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
    for (int d = lane * 16; d < F.D; d += 512) {  // D is a multiple of 16
      const uint4 x = *reinterpret_cast<const uint4*>(e + d), y = *reinterpret_cast<const uint4*>(c + d);
      int p = __dp4a(static_cast<int>(x.x), static_cast<int>(y.x), 0);
      p = __dp4a(static_cast<int>(x.y), static_cast<int>(y.y), p);
      p = __dp4a(static_cast<int>(x.z), static_cast<int>(y.z), p);
      p = __dp4a(static_cast<int>(x.w), static_cast<int>(y.w), p);
      acc += p;
    }
    z = warp_sum_f64(static_cast<double>(acc)) * static_cast<double>(F.e_scale[r]) * static_cast<double>(F.c_scale[col]);
  } else {
    double acc = 0.0;
    const __nv_bfloat16* e = F.E + r * F.D;
    const __nv_bfloat16* c = F.C + static_cast<int64_t>(col) * F.D;
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

constexpr int kFinishWarps = 4;
constexpr int kListsLane = 10;  // lists of a row a lane follows: 32 x 10 >= 2 x (148 + 1)

// One warp per row: the segments' statistics joined, then the row's outputs. The alternatives: the heads of the
// segments' sorted lists are merged, largest key first, into the L > top_k best. The logits behind their
// keys carry the rounding of 32-bit sums, so where two neighbours are closer than that, their order (and which of
// them is the top_k-th) is not known yet: every run of such neighbours is computed again in 64 bits and ordered by
// that, the lower id first among equal ones. Runs are short and rare (a few percent of the neighbours), so this
// reads little.
__global__ void __launch_bounds__(kFinishWarps * 32) head_finish_kernel(const __grid_constant__ HeadFinish F) {
  wait_for_previous_grid();
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kFinishWarps + (threadIdx.x >> 5);
  if (r >= F.N) return;
  const HeadSplit& S = F.split;
  const int b = static_cast<int>(r / kHeadBM);
  int g = static_cast<int>(static_cast<long long>(b) * S.ngroups / S.nb);  // the group of row block b, or one off
  while (S.group_begin(g) > b) --g;
  while (S.group_begin(g + 1) <= b) ++g;
  const int b0 = S.group_begin(g), gb = S.group_begin(g + 1) - b0;
  const int total = S.units(gb), P = S.parts(total);
  const int nlist =
      2 * (HeadSplit::owner(S.units(b - b0 + 1) - 1, total, P) - HeadSplit::owner(S.units(b - b0), total, P) + 1);
  const bool failed = *F.err != 0;
  const float sc = F.inv_t * kLog2e;

  float m = -INFINITY;
  for (int i = lane; i < nlist; i += 32) m = fmaxf(m, F.part_m[static_cast<int64_t>(i) * F.N + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = 0.f, w = 0.f;
  for (int i = lane; i < nlist; i += 32) {
    const int64_t o = static_cast<int64_t>(i) * F.N + r;
    const float mi = F.part_m[o], si = F.part_s[o];
    if (mi == -INFINITY) {
      s += si;  // 0, or NaN
    } else {
      const float d = (mi - m) * sc, f = ex2(d);
      s = fmaf(f, si, s);
      w += f * fmaf(si, fmaxf(d, -1e30f), F.part_w[o]);
    }
  }
  s = warp_sum(s);
  w = warp_sum(w);
  const float ln_s = logf(s);
  const float nan = __int_as_float(0x7fffffff);
  const bool none = m == -INFINITY && s == 0.f;  // every logit of the row is -inf
  if (F.K > 0) {
    bool any = false;
    for (int k = lane; k < F.K; k += 32) {
      const int64_t id = F.tokens[r * F.K + k];
      float lp = 0.f;
      if (id != F.ignore_index) {
        any = true;
        if (id < 0 || id >= F.V) {
          record_error(F.err, kErrTargetRange);
          lp = nan;
        } else {
          lp = none ? -INFINITY : (F.zt[static_cast<int64_t>(k) * F.N + r] - m) * F.inv_t - ln_s;
        }
      }
      F.logprobs[r * F.K + k] = failed ? nan : lp;
    }
    any = __any_sync(0xffffffffu, any);
    if (lane == 0) {
      const float h = none || !any ? 0.f : ln_s - 0.6931471805599453f * (w / s);
      F.entropy[r] = failed ? nan : h;
      F.lse[r] = failed ? nan : (none ? -INFINITY : fmaf(m, F.inv_t, ln_s));
    }
  }
  if (F.L == 0) return;

  // merge: lane l follows lists l, l + 32, ...
  unsigned long long head[kListsLane];
  int pos[kListsLane];
  const int64_t step = static_cast<int64_t>(F.N) * F.L;
#pragma unroll
  for (int i = 0; i < kListsLane; ++i) {
    const int li = lane + 32 * i;
    pos[i] = 0;
    head[i] = li < nlist ? F.lists[li * step + r * F.L] : 0;
  }
  const int want = F.L;
  unsigned long long mykey = 0;  // lane i: the i-th best
  for (int j = 0; j < want; ++j) {
    unsigned long long best = 0;
#pragma unroll
    for (int i = 0; i < kListsLane; ++i) best = head[i] > best ? head[i] : best;
    const unsigned long long top = warp_max_u64(best);
    if (lane == j) mykey = top;
    if (top == 0) break;
    if (best == top) {
#pragma unroll
      for (int i = 0; i < kListsLane; ++i) {
        if (head[i] == top) {
          ++pos[i];
          head[i] = pos[i] < F.L ? F.lists[(lane + 32 * i) * step + r * F.L + pos[i]] : 0;
        }
      }
    }
  }
  const float v = key_value(mykey);
  const int col = mykey == 0 ? -1 : key_column(mykey);
  // Neighbours closer than what a 32-bit sum loses: the sums of 512 products carry up to a few 2^-24 of their
  // largest part each (2^-15 of the logits leaves room); 8-bit products are exact but for three roundings.
  const float scale = fmaxf(fabsf(__shfl_sync(0xffffffffu, v, 0)), fabsf(v));
  const float tol = (F.C8 != nullptr ? 0x1p-21f : 0x1p-15f) * (scale < 3e38f ? scale : 0.f);
  const float before = __shfl_up_sync(0xffffffffu, v, 1);
  const bool close = lane > 0 && col >= 0 && isfinite(v) && isfinite(before) && before - v <= tol;
  const unsigned joins = __ballot_sync(0xffffffffu, close);  // bit i: i is close to i - 1
  const unsigned runs = joins | (joins >> 1);                // members of a run
  double zx = static_cast<double>(v);
  for (unsigned todo = runs; todo != 0; todo &= todo - 1) {
    const int i = __ffs(todo) - 1;
    const double z = exact_logit(F, r, __shfl_sync(0xffffffffu, col, i), lane);
    if (lane == i) zx = z;
  }
  int place = lane;
  if ((runs >> lane) & 1u) {
    const unsigned starts = ~joins;  // bit i: a run (or a single one) starts at i
    place = 31 - __clz(static_cast<int>(starts & (0xffffffffu >> (31 - lane))));
  }
  const int first = place;  // start of this lane's run
  for (int i = 0; i < 32; ++i) {
    const int fi = __shfl_sync(0xffffffffu, first, i), ci = __shfl_sync(0xffffffffu, col, i);
    const double zi = __shfl_sync(0xffffffffu, zx, i);
    if (((runs >> lane) & 1u) && i != lane && ((runs >> i) & 1u) && fi == first && (zi > zx || (zi == zx && ci < col)))
      ++place;
  }
  if (place < F.top_k && col >= 0) {
    const float lp = m == -INFINITY ? -INFINITY
                                    : static_cast<float>((zx - static_cast<double>(m)) * static_cast<double>(F.inv_t)) - ln_s;
    F.top_logprobs[r * F.top_k + place] = failed || s != s ? nan : lp;
    F.top_ids[r * F.top_k + place] = failed ? -1 : col;
  } else if (col < 0 && lane < F.top_k) {  // NaN logits leave the lists short
    F.top_logprobs[r * F.top_k + lane] = nan;
    F.top_ids[r * F.top_k + lane] = -1;
  }
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

template <bool I8, int L, bool OUT>
cudaError_t launch_one(const CUtensorMap& tmE, const CUtensorMap& tmC, const HeadArgs& A, bool after_kernel,
                       cudaStream_t s) {
  auto kernel = head_kernel<I8, L, OUT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  if (after_kernel) {
    e = launch_after_previous(kernel, dim3(A.split.grid), dim3(NUM_THREADS), SMEM_BYTES, s, tmE, tmC, A);
    if (e != cudaSuccess) return e;
  } else {
    kernel<<<A.split.grid, NUM_THREADS, SMEM_BYTES, s>>>(tmE, tmC, A);
  }
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_head(const CUtensorMap& tmE, const CUtensorMap& tmC, const HeadArgs& A, bool int8, int list_len,
                        bool after_kernel, cudaStream_t s) {
  if (A.out != nullptr) return launch_one<true, 0, true>(tmE, tmC, A, after_kernel, s);
  if (int8) {
    if (list_len == 0) return launch_one<true, 0, false>(tmE, tmC, A, after_kernel, s);
    if (list_len == kHeadShortList) return launch_one<true, kHeadShortList, false>(tmE, tmC, A, after_kernel, s);
    return launch_one<true, kHeadLongList, false>(tmE, tmC, A, after_kernel, s);
  }
  if (list_len == 0) return launch_one<false, 0, false>(tmE, tmC, A, after_kernel, s);
  if (list_len == kHeadShortList) return launch_one<false, kHeadShortList, false>(tmE, tmC, A, after_kernel, s);
  return launch_one<false, kHeadLongList, false>(tmE, tmC, A, after_kernel, s);
}

cudaError_t launch_head_finish(const HeadFinish& F, bool after_kernel, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((F.N + kFinishWarps - 1) / kFinishWarps)), block(kFinishWarps * 32);
  if (after_kernel) {
    const cudaError_t e = launch_after_previous(head_finish_kernel, grid, block, 0, s, F);
    if (e != cudaSuccess) return e;
  } else {
    head_finish_kernel<<<grid, block, 0, s>>>(F);
  }
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
