// tc_linear_attn.cuh - tensor-core (tcgen05) pass of linear attention with a decay for each head,
// bf16 roles x, y, w (q, k, v in the forward), d = 64; the rule and the roles are those of
// linear_attn.cuh, with chunks of 128 tokens:
//   P     = x y^T                         128 x 128 x 64
//   out   = a (P o m) w + c diag(f) x C   128 x 64 x (128 + 64)
//   C^T  <- gamma^n C^T + w^T (e diag(h) y)   64 x (3 x 64) x 128
//
// One CTA of 20 warps takes a unit's segment; its roles run apart and meet at mbarriers:
//   warp 0        TMA: x, y, w tiles of a chunk, three stages ahead
//   warp 1        issues every product: w^T y', x C, P w, the next chunk's x y^T
//   warps 4-7     P: row t of 128 columns out of tensor memory, masked and decayed, back
//                 as the bf16 A operand of P w
//   warps 8-11    y' = e h_s y_s as three bf16 tiles
//   warps 12-15   state: C^T in 32 fp32 registers a thread, rewritten as the operand of x C
//   warps 16-19   outputs: a P w + c f_t x C, through shared memory and a TMA store
// Nothing of a chunk waits for the previous chunk's outputs; only the state is a chain, and its
// step (one product, one scaling) is shorter than a chunk's products.
//
// What bounds it: shared memory.  A product of N = 64 reads its operands longer than it
// computes (128 bytes a cycle: M128 N64 K16 takes 48 cycles for 16 of arithmetic), and a
// chunk moves about 310 KB through it, 2400 of the 2860 cycles that its 64 KB of HBM
// traffic take; hence the state's product with M = 64 and all three parts of y' as one N = 192.
//
// Precision: x, y, w are exact in bf16 and every product accumulates in fp32.  Each summand of
// an output passes one operand rounded to bf16, P o m or C (2^-8 of it, as coarse as the
// output's own rounding).  The state is an fp32 result that is carried on: it stays in fp32
// registers, and the decayed rows y' that enter it are three bf16 numbers, all of fp32 (two
// would leave 2.5e-6 of the state).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_status.cuh"
#include "linear_attn.cuh"
#include "sm100.cuh"

namespace ttt {
namespace tclattn {

using namespace ::ttt::sm100;
using lattn::D;
using lattn::decay_pow;
using lattn::Params;

constexpr int CHUNK = 128;
constexpr int THREADS = 640;
constexpr int STAGES = 3;
constexpr uint32_t TILE = CHUNK * D * 2;  // 16 KB: one role's tile, 128-byte swizzled rows

// Shared-memory map (bytes from a 1024-byte aligned base).
constexpr uint32_t OFF_STAGE = 0;                            // stages of {x, y, w}
constexpr uint32_t STAGE_BYTES = 3 * TILE;
constexpr uint32_t OFF_YS = STAGES * STAGE_BYTES;            // y' in three parts
constexpr uint32_t OFF_C = OFF_YS + 3 * TILE;                // 2 buffers of C^T [64][64] bf16
constexpr uint32_t C_BYTES = D * D * 2;
constexpr uint32_t OFF_OUT = OFF_C + 2 * C_BYTES;            // output tile
constexpr uint32_t OFF_PW = OFF_OUT + TILE;                  // gamma^0 .. gamma^128
constexpr uint32_t OFF_CT = OFF_PW + (CHUNK + 4) * 4;        // gamma^31 .. gamma^0 (reverse: gamma^0 ..)
constexpr uint32_t OFF_BAR = OFF_CT + 32 * 4;
constexpr uint32_t OFF_TSLOT = OFF_BAR + 20 * 8;
constexpr uint32_t OFF_ABORT = OFF_TSLOT + 4;
constexpr uint32_t SMEM_USED = OFF_ABORT + 4;
constexpr uint32_t SMEM_BYTES = SMEM_USED + 1024;  // + alignment slack
static_assert(SMEM_BYTES <= 227 * 1024, "one CTA's shared memory");

// Tensor memory columns: P in fp32, P in bf16, x C, P w, the state's product (three parts).
constexpr uint32_t T_P = 0, T_PB = 128, T_XC = 192, T_PW = 256, T_M = 320, TMEM_COLS = 512;

enum {
  FULL = 0, EMPTY = 3, PFULL = 6, PREADY = 7, YREADY = 8, CREADY = 9, MFULL = 10, OFULL = 11, OFREE = 12, NEVER = 13,
  DRAIN = 14, NUM_BARS = 15
};
constexpr long long WAIT_LIMIT = 1ll << 32;            // SM cycles, ~2 s
constexpr long long INJECTED_WAIT_LIMIT = 1ll << 20;
constexpr uint32_t NB_OUT = 1;                         // named barrier of the output warps

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 3-D tiled store of a box out of shared memory (rows past the tensor's end are left out).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *smem_src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(smem_src))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// The part of a wait that is not the common case, kept out of the roles' code.
__device__ __noinline__ bool wait_longer(uint64_t *bar, uint32_t parity, volatile int *abort, long long limit) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (clock64() - t0 > limit) {
      *abort = 1;
      record_device_error(-5 /* TTT_ERR_TIMEOUT */);
      return false;
    }
  }
  return true;
}

// False once a wait of this CTA has run out: the caller leaves its loop.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                     long long limit = WAIT_LIMIT) {
  return mbar_try_wait(bar, parity) || wait_longer(bar, parity, abort, limit);
}

// The same for a whole warp, one answer for all lanes.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, wait(bar, parity, abort));
}

// After tmem_wait_ld: registers that a tensor memory load filled, not to be used before this place.
template <int N>
__device__ __forceinline__ void loaded(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// A product of N steps along its inner axis, whose operands advance by these bytes a step.  (The
// loop stays rolled: twenty warps in five roles share the SM's instruction cache, see below.)
template <int N>
__device__ __forceinline__ void issue(uint32_t d, uint64_t a, uint32_t step_a, uint64_t b, uint32_t step_b, uint32_t id) {
#pragma unroll 1
  for (int k = 0; k < N; ++k, a += step_a >> 4, b += step_b >> 4) umma_ss_w(d, a, b, id, k > 0);
}

// STATE_ONLY: the segments' own states (y and w alone).
template <bool REVERSE, bool STATE_ONLY>
__global__ void __launch_bounds__(THREADS, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmY,
                   const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmOut, const Params p,
                   const int inject_timeout) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = blockIdx.x / p.nseg, seg = blockIdx.x % p.nseg;
  const bool first = REVERSE ? seg == p.nseg - 1 : seg == 0;
  const bool last = REVERSE ? seg == 0 : seg == p.nseg - 1;
  if (STATE_ONLY && last) return;  // no segment follows it: its own state has no reader
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + OFF_TSLOT);
  volatile int *abort = reinterpret_cast<volatile int *>(sm + OFF_ABORT);
  float *pw = reinterpret_cast<float *>(sm + OFF_PW);
  float *ct = reinterpret_cast<float *>(sm + OFF_CT);

  if (tid == 0) {
    for (int i = 0; i < NUM_BARS; ++i) {
      const bool warps4 = i == PREADY || i == YREADY || i == CREADY || i == OFREE;
      mbar_init(&bars[i], warps4 ? 4 : 1);
    }
    *abort = 0;
    fence_mbarrier_init();
    if (!STATE_ONLY) {
      prefetch_tensormap(&tmX);
      prefetch_tensormap(&tmOut);
    }
    prefetch_tensormap(&tmY);
    prefetch_tensormap(&tmW);
  }
  if (warp == 2) {
    tmem_alloc(tslot, TMEM_COLS);
    tmem_relinquish();
  }
  const float g = p.log_decay[unit % p.H];
  if (tid <= CHUNK) pw[tid] = decay_pow(g, tid);
  if (tid < 32) ct[tid] = decay_pow(g, REVERSE ? tid : 31 - tid);
  const int len = lattn::sequence_length(p.lengths, unit / p.H, p.T);
  const int t_lo = seg * p.seg_len;
  const int t_hi = min(t_lo + p.seg_len, p.T);
  const int n_seg = min(max(len - t_lo, 0), t_hi - t_lo);
  const int nchunks = (n_seg + CHUNK - 1) / CHUNK;
  auto chunk_start = [&](int ci) { return (REVERSE ? nchunks - 1 - ci : ci) * CHUNK; };
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tb = *tslot;

  bool ok = true;
  if (inject_timeout) ok = wait(&bars[NEVER], 0, abort, INJECTED_WAIT_LIMIT);

  if (warp == 0) {
    // ---- loads -------------------------------------------------------------------
    if (lane == 0) {
      int c = 0;
      for (; ok && c < nchunks; ++c) {
        const int st = c % STAGES;
        if (c >= STAGES && !wait(&bars[EMPTY + st], (uint32_t)(c / STAGES - 1) & 1u, abort)) break;
        uint8_t *s = sm + OFF_STAGE + st * STAGE_BYTES;
        const int t0 = t_lo + chunk_start(c);
        mbar_arrive_expect_tx(&bars[FULL + st], STATE_ONLY ? 2 * TILE : 3 * TILE);
        tma_load_3d(s + TILE, &tmY, 0, t0, unit, &bars[FULL + st]);
        if (!STATE_ONLY) tma_load_3d(s, &tmX, 0, t0, unit, &bars[FULL + st]);
        tma_load_3d(s + 2 * TILE, &tmW, 0, t0, unit, &bars[FULL + st]);
      }
      // A CTA that gave up waits for its loads in flight (at most one a stage).
      if (*abort)
        for (int k = max(0, c - STAGES); k < c; ++k) mbar_wait(&bars[FULL + k % STAGES], (uint32_t)(k / STAGES) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- products (the whole warp, converged; one lane elected to issue) ---------------
    constexpr uint32_t ID_P = idesc_bf16_f32(128, 128, false, false, false);
    constexpr uint32_t ID_XC = idesc_bf16_f32(128, 64, false, false, false);
    constexpr uint32_t ID_PW = idesc_bf16_f32(128, 64, false, true, false);
    constexpr uint32_t ID_M = idesc_bf16_f32(64, 192, true, true, false);
    auto stage = [&](int c) { return sbase + OFF_STAGE + (c % STAGES) * STAGE_BYTES; };
    auto scores = [&](int c) {  // P of chunk c, once its tiles are in
      if (!wait_warp(&bars[FULL + c % STAGES], (uint32_t)(c / STAGES) & 1u, abort)) return false;
      tc_fence_after_sync();
      const uint32_t x = stage(c), y = x + TILE;
      issue<4>(tb + T_P, smem_desc_sw128(x, 16, 1024), 32, smem_desc_sw128(y, 16, 1024), 32, ID_P);
      umma_commit_w(&bars[PFULL]);
      return true;
    };
    if (!STATE_ONLY && ok && nchunks > 0) ok = scores(0);
    for (int c = 0; ok && c < nchunks; ++c) {
      const uint32_t par = (uint32_t)c & 1u;
      const uint32_t x = stage(c), w = x + 2 * TILE;
      // w^T y', once y' is written, the last product read and C's operand written.  (The warps of a
      // barrier arrive once a phase: none can be a chunk ahead of another, since its next arrival
      // follows a product that waited for all of them.)
      if (!(ok = wait_warp(&bars[YREADY], par, abort))) break;
      if (!(ok = wait_warp(&bars[CREADY], par, abort))) break;
      tc_fence_after_sync();
      issue<8>(tb + T_M, smem_desc_sw128(w, 8192, 1024), 2048, smem_desc_sw128(sbase + OFF_YS, TILE, 1024), 2048, ID_M);
      umma_commit_w(&bars[MFULL]);
      if (STATE_ONLY) {
        if (c + STAGES < nchunks) umma_commit_w(&bars[EMPTY + c % STAGES]);
        continue;
      }
      // x C, once the outputs of the last chunk are read.
      if (c > 0 && !(ok = wait_warp(&bars[OFREE], par ^ 1u, abort))) break;
      tc_fence_after_sync();
      const uint32_t cop = sbase + OFF_C + (c & 1) * C_BYTES;
      issue<4>(tb + T_XC, smem_desc_sw128(x, 16, 1024), 32, smem_desc_sw128(cop, 16, 1024), 32, ID_XC);
      // P w; then the next chunk's P, whose fp32 columns are read by now and whose bf16 ones are
      // free when P w is done, which PFULL of the next chunk says too.
      if (!(ok = wait_warp(&bars[PREADY], par, abort))) break;
      tc_fence_after_sync();
      {
        uint64_t b = smem_desc_sw128(w, 8192, 1024);
#pragma unroll 1
        for (int k = 0; k < 8; ++k, b += 2048 >> 4) umma_ts_w(tb + T_PW, tb + T_PB + 8 * k, b, ID_PW, k > 0);
      }
      umma_commit_w(&bars[OFULL]);
      if (c + STAGES < nchunks) umma_commit_w(&bars[EMPTY + c % STAGES]);
      if (c + 1 < nchunks && !(ok = scores(c + 1))) break;
    }
    __syncwarp();
    if (*abort) {  // products in flight end before the tensor memory is freed
      umma_commit_w(&bars[DRAIN]);
      mbar_wait(&bars[DRAIN], 0, WAIT_LIMIT);
    }
  } else if (!STATE_ONLY && warp >= 4 && warp < 8) {
    // ---- P: mask and decay, to bf16 ------------------------------------------------------
    // Row t = 32 w4 + lane.  In a block of 32 columns off the diagonal the power of gamma is the
    // product of one of the row's (base) and one of the column's (ct), both at most 1.
    const int w4 = warp & 3;
    const uint32_t row = tmem_addr(tb, 32 * w4, T_P), dst = tmem_addr(tb, 32 * w4, T_PB);
    for (int c = 0; ok && c < nchunks; ++c) {
      const int n = min(CHUNK, n_seg - chunk_start(c));
      if (!(ok = wait_warp(&bars[PFULL], (uint32_t)c & 1u, abort))) break;
      tc_fence_after_sync();
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        const int d = REVERSE ? j - w4 : w4 - j;
        uint32_t pk[16];
        if (d < 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0u;
        } else {
          uint32_t r[32];
          tmem_ld_32x32b_x32(row + 32 * j, r);
          const int end = REVERSE ? n - 32 * j : 32;  // columns that hold tokens (forward: s <= t decides)
          if (d == 0 || end < 32) {
            const float *f = pw + (REVERSE ? 32 * d - lane : 32 * d + lane);
            const int most = REVERSE ? end : 32 * d + lane + 1, least = REVERSE ? lane - 32 * d : 0;
            tmem_wait_ld();
            loaded(r);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float v[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int s = 2 * e + i;
                const bool in = s < most && s >= least;
                v[i] = in ? __uint_as_float(r[s]) * (p.a * f[REVERSE ? s : -s]) : 0.f;
              }
              pk[e] = pack_bf16x2(v[0], v[1]);
            }
          } else {
            const float b = p.a * pw[REVERSE ? 32 * d - lane : lane + 32 * d - 31];
            const float2 b2 = make_float2(b, b);
            tmem_wait_ld();
            loaded(r);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float4 t4 = *reinterpret_cast<const float4 *>(ct + 4 * q);
              const float2 u = __fmul2_rn(__fmul2_rn(b2, make_float2(t4.x, t4.y)),
                                          make_float2(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1])));
              const float2 v = __fmul2_rn(__fmul2_rn(b2, make_float2(t4.z, t4.w)),
                                          make_float2(__uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3])));
              pk[2 * q] = pack_bf16x2(u.x, u.y);
              pk[2 * q + 1] = pack_bf16x2(v.x, v.y);
            }
          }
        }
        tmem_st_32x32b_x16(dst + 16 * j, pk);
      }
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[PREADY]);
    }
  } else if (warp >= 8 && warp < 12) {
    // ---- y' (zeros past the end), and zeros over w's rows past the end: what lies there is any
    // value, and enters the products ---------------------------------------------------------
    const int s = 32 * (warp & 3) + lane;
    for (int c = 0; ok && c < nchunks; ++c) {
      const int n = min(CHUNK, n_seg - chunk_start(c));
      if (!(ok = wait_warp(&bars[FULL + c % STAGES], (uint32_t)(c / STAGES) & 1u, abort))) break;
      uint8_t *st = sm + OFF_STAGE + (c % STAGES) * STAGE_BYTES;
      const float h1 = s < n ? p.e * pw[REVERSE ? s + 1 : n - 1 - s] : 0.f;
      const float2 h = make_float2(h1, h1);
      // The tiles are free when the last chunk's product is done.
      if (c > 0 && !(ok = wait_warp(&bars[MFULL], (uint32_t)(c - 1) & 1u, abort))) break;
      uint32_t off = sw128_offset(s, 0);
      uint4 y = *reinterpret_cast<const uint4 *>(st + TILE + off);
#pragma unroll 1
      for (int q = 0; q < 8; ++q) {
        if (s >= n) {
          y = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4 *>(st + 2 * TILE + off) = y;
        }
        const uint32_t u[4] = {y.x, y.y, y.z, y.w};
        const uint32_t next = sw128_offset(s, 8 * (q + 1 & 7));
        y = *reinterpret_cast<const uint4 *>(st + TILE + next);
        uint32_t part[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 r = __fmul2_rn(h, unpack_bf16x2(u[e]));
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            part[k][e] = pack_bf16x2(r.x, r.y);
            if (k < 2) {
              const float2 f = unpack_bf16x2(part[k][e]);
              r = __fadd2_rn(r, make_float2(-f.x, -f.y));
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *reinterpret_cast<uint4 *>(sm + OFF_YS + k * TILE + off) = make_uint4(part[k][0], part[k][1], part[k][2], part[k][3]);
        off = next;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[YREADY]);
    }
  } else if (warp >= 12 && warp < 16) {
    // ---- state ----------------------------------------------------------------------
    // A product of M = 64 lies in the lower 16 of each warp's 32 lanes; the 16x256b load gives
    // this thread rows row and row + 8 of C^T at columns 8 j + col + {0, 1}: C[4 j + {0, 1}] and
    // C[4 j + {2, 3}].
    const int w4 = warp & 3;
    const int row = 16 * w4 + (lane >> 2), col = 2 * (lane & 3);
    float C[32];
    {
      const float *C0 = nullptr;
      if (p.C0 && (p.c0_segments || first))
        C0 = p.C0 + (long long)unit * p.c0_stride + (p.c0_segments ? (long long)seg * D * D : 0);
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int r = row + 8 * ((e >> 1) & 1), cc = 8 * (e >> 2) + col + (e & 1);
        C[e] = C0 ? (p.c0_transposed ? C0[r * D + cc] : C0[cc * D + r]) : 0.f;
      }
    }
    auto write_operand = [&](int buf) {
      if (!STATE_ONLY) {
        uint8_t *to = sm + OFF_C + buf * C_BYTES;
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          *reinterpret_cast<uint32_t *>(to + sw128_offset(row + 8 * ((e >> 1) & 1), 8 * (e >> 2) + col)) =
              pack_bf16x2(C[e], C[e + 1]);
        fence_proxy_async_smem();
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[CREADY]);
    };
    if (ok && nchunks > 0) write_operand(0);
    for (int c = 0; ok && c < nchunks; ++c) {
      const int n = min(CHUNK, n_seg - chunk_start(c));
      const float dn = pw[n];
      if (!(ok = wait_warp(&bars[MFULL], (uint32_t)c & 1u, abort))) break;
      tc_fence_after_sync();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t m[3][16];
#pragma unroll
        for (int k = 0; k < 3; ++k) tmem_ld_16x256b_x4(tmem_addr(tb, 32 * w4, T_M + 64 * k + 32 * h), m[k]);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 3; ++k) loaded(m[k]);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          auto pair = [&](int k) { return make_float2(__uint_as_float(m[k][e]), __uint_as_float(m[k][e + 1])); };
          const float2 v = __ffma2_rn(make_float2(dn, dn), make_float2(C[16 * h + e], C[16 * h + e + 1]),
                                      __fadd2_rn(pair(0), __fadd2_rn(pair(1), pair(2))));
          C[16 * h + e] = v.x;
          C[16 * h + e + 1] = v.y;
        }
      }
      // The other buffer's reader, x C of the last chunk, was issued before this chunk's w^T y'
      // and is done with it.
      if (c + 1 < nchunks) write_operand((c + 1) & 1);
    }
    if (p.C_out && (p.c_out_segments || last)) {
      float *Co = p.C_out + (p.c_out_segments ? ((long long)unit * p.nseg + seg) : unit) * (long long)(D * D);
#pragma unroll
      for (int e = 0; e < 32; ++e) Co[(8 * (e >> 2) + col + (e & 1)) * D + row + 8 * ((e >> 1) & 1)] = C[e];
    }
  } else if (!STATE_ONLY && warp >= 16) {
    // ---- outputs --------------------------------------------------------------------
    const int w4 = warp & 3, t = 32 * w4 + lane;
    // (These warps meet at a named barrier, so none leaves the loop alone: after a wait that ran
    // out the rest of the loop runs on whatever the tensor memory holds.)
    for (int c = 0; c < nchunks; ++c) {
      const int c0 = chunk_start(c), n = min(CHUNK, n_seg - c0);
      const float f1 = t < n ? p.c * pw[REVERSE ? n - 1 - t : t + 1] : 0.f;
      const float2 f = make_float2(f1, f1);
      if (ok) ok = wait_warp(&bars[OFULL], (uint32_t)c & 1u, abort);
      tc_fence_after_sync();
      // The tile is free once the last store has read it.
      if (warp == 16 && lane == 0) tma_store_wait_read();
      named_barrier_sync(NB_OUT, 128);
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {
        uint32_t xc[16], pv[16], o[8];
        tmem_ld_32x32b_x16(tmem_addr(tb, 32 * w4, T_XC + 16 * h), xc);
        tmem_ld_32x32b_x16(tmem_addr(tb, 32 * w4, T_PW + 16 * h), pv);
        tmem_wait_ld();
        loaded(xc);
        loaded(pv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 v =
              __ffma2_rn(f, make_float2(__uint_as_float(xc[2 * e]), __uint_as_float(xc[2 * e + 1])),
                         make_float2(__uint_as_float(pv[2 * e]), __uint_as_float(pv[2 * e + 1])));
          o[e] = t < n ? pack_bf16x2(v.x, v.y) : 0u;
        }
        *reinterpret_cast<uint4 *>(sm + OFF_OUT + sw128_offset(t, 16 * h)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(sm + OFF_OUT + sw128_offset(t, 16 * h + 8)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      tc_fence_before_sync();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[OFREE]);
      named_barrier_sync(NB_OUT, 128);
      if (warp == 16 && lane == 0) tma_store_3d(&tmOut, sm + OFF_OUT, 0, t_lo + c0, unit);
    }
    // Rows of chunks wholly behind the end (those of the last chunk are in its tile).
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + ((long long)unit * p.T + t_lo) * D;
    const int x0 = min(nchunks * CHUNK, t_hi - t_lo) * (D / 8), x1 = (t_hi - t_lo) * (D / 8);
    for (int x = x0 + (tid & 127); x < x1; x += 128)
      reinterpret_cast<uint4 *>(out)[x] = make_uint4(0u, 0u, 0u, 0u);
    if (warp == 16 && lane == 0) tma_store_wait_read();
    __syncwarp();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after_sync();
    tmem_dealloc(tb, TMEM_COLS);
  }
}

}  // namespace tclattn
}  // namespace ttt
