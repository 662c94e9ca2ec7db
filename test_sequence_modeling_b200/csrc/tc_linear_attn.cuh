// tc_linear_attn.cuh - tensor-core (tcgen05) pass of linear attention with a decay for each head,
// bf16 roles x, y, w (q, k, v in the forward), d = 64; the rule and the roles are those of
// linear_attn.cuh, with chunks of 128 tokens:
//   P     = x y^T                         128 x 128 x 64
//   out   = a (P o m) w + c diag(f) x C   128 x 64 x (128 + 64, C as two bf16 operands)
//   C^T  <- gamma^n C^T + w^T (e diag(h) y)
//
// One CTA of 16 warps takes a unit's segment; its roles run apart and meet at mbarriers:
//   warp 0        TMA: x, y, w tiles of a chunk, three stages ahead
//   warp 1        issues every product, in the order w^T y', x C, the next chunk's x y^T, P w
//   warps 4-7     P: row t of 128 columns out of tensor memory, masked and decayed, back in
//                 place as the bf16 A operand of P w
//   warps 8-11    state: y' = e h_s y_s as two bf16 tiles, and C^T in 32 fp32 registers a
//                 thread (rows: w's features; the products' M = 128 holds them twice, so that
//                 each warp pair takes half of the columns), rewritten as the operand of x C
//   warps 12-15   outputs: a P w + c f_t x C, through shared memory and a TMA store
// Nothing of a chunk waits for the previous chunk's outputs; only the state is a chain, and its
// step (y' of the next chunk, one product, one scaling) is shorter than a chunk's products.
//
// Precision: x, y, w are exact in bf16 and every product accumulates in fp32.  P o m is
// rounded to bf16 (2^-8 of each summand, as coarse as the output's own rounding).  The
// state is fp32 in registers; as an operand it, and the decayed rows y', are two bf16 numbers
// (2^-16), because the state is an fp32 result that is carried on.
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
constexpr int THREADS = 512;
constexpr int STAGES = 3;
constexpr uint32_t TILE = CHUNK * D * 2;  // 16 KB: one role's tile, 128-byte swizzled rows

// Shared-memory map (bytes from a 1024-byte aligned base).
constexpr uint32_t OFF_STAGE = 0;                            // stages of {x, y, w}
constexpr uint32_t STAGE_BYTES = 3 * TILE;
constexpr uint32_t OFF_YS = STAGES * STAGE_BYTES;            // y' hi, lo
constexpr uint32_t OFF_C = OFF_YS + 2 * TILE;                // 2 buffers of C^T {hi, lo} [64][64] bf16
constexpr uint32_t C_BYTES = 2 * D * D * 2;
constexpr uint32_t OFF_OUT = OFF_C + 2 * C_BYTES;            // output tile
constexpr uint32_t OFF_PW = OFF_OUT + TILE;                  // gamma^0 .. gamma^128
constexpr uint32_t OFF_BAR = OFF_PW + (CHUNK + 4) * 4;
constexpr uint32_t OFF_TSLOT = OFF_BAR + 20 * 8;
constexpr uint32_t OFF_ABORT = OFF_TSLOT + 4;
constexpr uint32_t SMEM_USED = OFF_ABORT + 4;
constexpr uint32_t SMEM_BYTES = SMEM_USED + 1024;  // + alignment slack
static_assert(SMEM_BYTES <= 227 * 1024, "one CTA's shared memory");

// Tensor memory columns: P twice, x C, P w, the state's product (hi | lo).
constexpr uint32_t T_P = 0, T_XC = 256, T_PW = 320, T_M = 384, TMEM_COLS = 512;

enum {
  FULL = 0, EMPTY = 3, PFULL = 6, PREADY = 8, YREADY = 10, CREADY = 11, MFULL = 12, OFULL = 13, OFREE = 14,
  NEVER = 15, DRAIN = 16, NUM_BARS = 17
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

// False once a wait of this CTA has run out: the caller leaves its loop.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                     long long limit = WAIT_LIMIT) {
  if (mbar_try_wait(bar, parity)) return true;
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

// The same for a whole warp, one answer for all lanes.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, wait(bar, parity, abort));
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

  if (tid == 0) {
    for (int i = 0; i < NUM_BARS; ++i) {
      const bool warps4 = i == PREADY || i == PREADY + 1 || i == YREADY || i == CREADY || i == OFREE;
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
    constexpr uint32_t ID_M = idesc_bf16_f32(128, 128, true, true, false);
    auto stage = [&](int c) { return sbase + OFF_STAGE + (c % STAGES) * STAGE_BYTES; };
    auto scores = [&](int c) {  // P of chunk c, once its tiles are in
      if (!wait_warp(&bars[FULL + c % STAGES], (uint32_t)(c / STAGES) & 1u, abort)) return false;
      tc_fence_after_sync();
      const uint32_t x = stage(c), y = x + TILE;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        umma_ss_w(tb + T_P + 128 * (c & 1), smem_desc_sw128(x + 32 * k, 16, 1024), smem_desc_sw128(y + 32 * k, 16, 1024),
                  ID_P, k > 0);
      umma_commit_w(&bars[PFULL + (c & 1)]);
      return true;
    };
    if (!STATE_ONLY && ok && nchunks > 0) ok = scores(0);
    for (int c = 0; ok && c < nchunks; ++c) {
      const uint32_t par = (uint32_t)c & 1u;
      const uint32_t x = stage(c), w = x + 2 * TILE;
      // w^T y': the state warps have written y' of this chunk and read the last product.
      if (!(ok = wait_warp(&bars[YREADY], par, abort))) break;
      tc_fence_after_sync();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_ss_w(tb + T_M, smem_desc_sw128(w + 2048 * k, 0, 1024),
                  smem_desc_sw128(sbase + OFF_YS + 2048 * k, TILE, 1024), ID_M, k > 0);
      umma_commit_w(&bars[MFULL]);
      if (STATE_ONLY) {
        if (c + STAGES < nchunks) umma_commit_w(&bars[EMPTY + c % STAGES]);
        continue;
      }
      // x C, once the operand is written and the outputs of the last chunk are read (which also
      // means that its P w is done: the other half of P may be overwritten).
      if (!(ok = wait_warp(&bars[CREADY], par, abort))) break;
      if (c > 0 && !(ok = wait_warp(&bars[OFREE], (uint32_t)(c - 1) & 1u, abort))) break;
      tc_fence_after_sync();
      const uint32_t cop = sbase + OFF_C + (c & 1) * C_BYTES;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_ss_w(tb + T_XC, smem_desc_sw128(x + 32 * k, 16, 1024),
                    smem_desc_sw128(cop + h * (D * D * 2) + 32 * k, 16, 1024), ID_XC, h + k > 0);
      if (c + 1 < nchunks && !(ok = scores(c + 1))) break;
      // P w
      if (!(ok = wait_warp(&bars[PREADY + (c & 1)], (uint32_t)(c >> 1) & 1u, abort))) break;
      tc_fence_after_sync();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_ts_w(tb + T_PW, tb + T_P + 128 * (c & 1) + 8 * k, smem_desc_sw128(w + 2048 * k, 8192, 1024), ID_PW, k > 0);
      umma_commit_w(&bars[OFULL]);
      if (c + STAGES < nchunks) umma_commit_w(&bars[EMPTY + c % STAGES]);
    }
    __syncwarp();
    if (*abort) {  // products in flight end before the tensor memory is freed
      umma_commit_w(&bars[DRAIN]);
      mbar_wait(&bars[DRAIN], 0, WAIT_LIMIT);
    }
  } else if (!STATE_ONLY && warp >= 4 && warp < 8) {
    // ---- P: mask and decay, to bf16 in place --------------------------------------------
    const int w4 = warp & 3, t = 32 * w4 + lane;
    for (int c = 0; ok && c < nchunks; ++c) {
      const int n = min(CHUNK, n_seg - chunk_start(c));
      if (!(ok = wait_warp(&bars[PFULL + (c & 1)], (uint32_t)(c >> 1) & 1u, abort))) break;
      tc_fence_after_sync();
      const uint32_t row = tmem_addr(tb, 32 * w4, T_P + 128 * (c & 1));
      // Columns in ascending blocks of 32: a block's 16 columns of bf16 pairs lie below every
      // column that is still to be read.
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t pk[16];
        if (REVERSE ? j >= w4 : j <= w4) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(row + 32 * j, r);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int s = 32 * j + 2 * e + i;
              const int gap = REVERSE ? s - t : t - s;
              const bool in = REVERSE ? gap >= 0 && s < n : gap >= 0;
              v[i] = in ? __uint_as_float(r[2 * e + i]) * pw[max(gap, 0)] : 0.f;
            }
            pk[e] = pack_bf16x2(v[0], v[1]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0u;
        }
        tmem_st_32x32b_x16(row + 16 * j, pk);
      }
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[PREADY + (c & 1)]);
    }
  } else if (warp >= 8 && warp < 12) {
    // ---- state ----------------------------------------------------------------------
    const int w4 = warp & 3;
    const int row = 32 * (w4 & 1) + lane, col0 = 32 * (w4 >> 1);  // this thread's C^T[row][col0 ..]
    const int s = 32 * w4 + lane;                                 // and its token of y'
    float C[32];
    {
      const float *C0 = nullptr;
      if (p.C0 && (p.c0_segments || first))
        C0 = p.C0 + (long long)unit * p.c0_stride + (p.c0_segments ? (long long)seg * D * D : 0);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        C[e] = C0 ? (p.c0_transposed ? C0[row * D + col0 + e] : C0[(col0 + e) * D + row]) : 0.f;
    }
    auto write_operand = [&](int buf) {
      if (STATE_ONLY) return;
      uint8_t *dst = sm + OFF_C + buf * C_BYTES;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16x2(C[8 * q + 2 * e], C[8 * q + 2 * e + 1], hi[e], lo[e]);
        const uint32_t off = sw128_offset(row, col0 + 8 * q);
        *reinterpret_cast<uint4 *>(dst + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(dst + D * D * 2 + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[CREADY]);
    };
    // y' of chunk c (zeros past the end), and zeros over w's rows past the end: what lies there
    // is any value, and enters the products.
    auto decayed_rows = [&](int c) {
      const int n = min(CHUNK, n_seg - chunk_start(c));
      if (!wait_warp(&bars[FULL + c % STAGES], (uint32_t)(c / STAGES) & 1u, abort)) return false;
      uint8_t *st = sm + OFF_STAGE + (c % STAGES) * STAGE_BYTES;
      const float h = s < n ? p.e * pw[REVERSE ? s + 1 : n - 1 - s] : 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t off = sw128_offset(s, 8 * q);
        uint32_t hi[4] = {}, lo[4] = {};
        if (s < n) {
          const uint4 y = *reinterpret_cast<const uint4 *>(st + TILE + off);
          const uint32_t u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack_bf16x2(u[e]);
            split_bf16x2(h * f.x, h * f.y, hi[e], lo[e]);
          }
        } else {
          *reinterpret_cast<uint4 *>(st + 2 * TILE + off) = make_uint4(0u, 0u, 0u, 0u);
        }
        *reinterpret_cast<uint4 *>(sm + OFF_YS + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(sm + OFF_YS + TILE + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();  // the last product's columns are read
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[YREADY]);
      return true;
    };
    if (ok && nchunks > 0) {
      ok = decayed_rows(0);
      write_operand(0);
    }
    for (int c = 0; ok && c < nchunks; ++c) {
      const int n = min(CHUNK, n_seg - chunk_start(c));
      if (!(ok = wait_warp(&bars[MFULL], (uint32_t)c & 1u, abort))) break;
      tc_fence_after_sync();
      const float dn = pw[n];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t m0[16], m1[16];
        tmem_ld_32x32b_x16(tmem_addr(tb, 32 * w4, T_M + col0 + 16 * h), m0);
        tmem_ld_32x32b_x16(tmem_addr(tb, 32 * w4, T_M + 64 + col0 + 16 * h), m1);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          C[16 * h + e] = fmaf(dn, C[16 * h + e], __uint_as_float(m0[e]) + __uint_as_float(m1[e]));
      }
      if (c + 1 < nchunks) {
        // (The product is complete, so y' may be overwritten; so is every product issued before
        // it, x C of the last chunk among them, whose operand buffer is written next.)
        if (!(ok = decayed_rows(c + 1))) break;
        write_operand((c + 1) & 1);
      }
    }
    if (p.C_out && (p.c_out_segments || last)) {
      float *Co = p.C_out + (p.c_out_segments ? ((long long)unit * p.nseg + seg) : unit) * (long long)(D * D);
#pragma unroll
      for (int e = 0; e < 32; ++e) Co[(col0 + e) * D + row] = C[e];
    }
  } else if (!STATE_ONLY && warp >= 12) {
    // ---- outputs --------------------------------------------------------------------
    const int w4 = warp & 3, t = 32 * w4 + lane;
    // (These warps meet at a named barrier, so none leaves the loop alone: after a wait that ran
    // out the rest of the loop runs on whatever the tensor memory holds.)
    for (int c = 0; c < nchunks; ++c) {
      const int c0 = chunk_start(c), n = min(CHUNK, n_seg - c0);
      if (ok) ok = wait_warp(&bars[OFULL], (uint32_t)c & 1u, abort);
      tc_fence_after_sync();
      const float f = t < n ? p.c * pw[REVERSE ? n - 1 - t : t + 1] : 0.f;
      uint32_t o[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t xc[32], pv[32];
        tmem_ld_32x32b_x32(tmem_addr(tb, 32 * w4, T_XC + 32 * h), xc);
        tmem_ld_32x32b_x32(tmem_addr(tb, 32 * w4, T_PW + 32 * h), pv);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float v[2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            v[i] = t < n ? fmaf(f, __uint_as_float(xc[2 * e + i]), p.a * __uint_as_float(pv[2 * e + i])) : 0.f;
          o[16 * h + e] = pack_bf16x2(v[0], v[1]);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[OFREE]);
      // The tile is free once the last store has read it.
      if (warp == 12 && lane == 0) tma_store_wait_read();
      named_barrier_sync(NB_OUT, 128);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *reinterpret_cast<uint4 *>(sm + OFF_OUT + sw128_offset(t, 8 * q)) =
            make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      fence_proxy_async_smem();
      named_barrier_sync(NB_OUT, 128);
      if (warp == 12 && lane == 0) tma_store_3d(&tmOut, sm + OFF_OUT, 0, t_lo + c0, unit);
    }
    // Rows of chunks wholly behind the end (those of the last chunk are in its tile).
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + ((long long)unit * p.T + t_lo) * D;
    const int x0 = min(nchunks * CHUNK, t_hi - t_lo) * (D / 8), x1 = (t_hi - t_lo) * (D / 8);
    for (int x = x0 + (tid & 127); x < x1; x += 128)
      reinterpret_cast<uint4 *>(out)[x] = make_uint4(0u, 0u, 0u, 0u);
    if (warp == 12 && lane == 0) tma_store_wait_read();
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
