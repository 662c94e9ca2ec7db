// tc_linear_attn.cuh - tensor-core (tcgen05) pass of linear attention with a decay for each head,
// bf16 roles x, y, w (q, k, v in the forward), d = 64; the rule and the roles are those of
// linear_attn.cuh, with chunks of 128 tokens:
//   P     = x y^T                         128 x 128 x 64
//   out   = a (P o m) w + c diag(f) x C   128 x 64 x (128 + 64)
//   C^T  <- gamma^n C^T + w^T (e diag(h) y)   64 x (3 x 64) x 128
//
// One CTA of 24 warps an SM takes segments of units in turn (a CTA's roles run on into its next
// segment without a stop); the roles run apart and meet at mbarriers:
//   warp 0        TMA: x, y, w tiles of a chunk, two slots each, refilled one by one
//   warp 1        issues every product: w^T y', x C, P w, the next chunk's x y^T
//   warp 3        says ahead which segments there are, with their powers of gamma
//   warps 4-11    P: row t of 128 columns out of tensor memory (two warps a row), masked and
//                 decayed, back as the bf16 A operand of P w
//   warps 12-15   y' = e h_s y_s as three bf16 tiles, two buffers
//   warps 16-19   state: C^T in 32 fp32 registers a thread, rewritten as the operand of x C
//   warps 20-23   outputs: a P w + c f_t x C, through shared memory and a TMA store
// Nothing of a chunk waits for the previous chunk's outputs; only the state is a chain, and its
// step (one product, one scaling) is shorter than a chunk's products.
//
// Where there are more units than SMs the CTAs share the chunks of all of them evenly, each a range of
// consecutive ones, whose ends may lie inside a unit.  A CTA begins with the head of the unit that its
// range ends in and hands the state on through memory; the tail of the unit that its range begins in
// comes last, when the CTA before it has handed its state on long ago.  A CTA's number is a ticket
// taken at its start, so the one before it has started, and what it waits for waits for nothing.
//
// Why so: a chunk's 64 KB of HBM traffic take an SM 2920 cycles at the measured copy rate.  The
// products take 1580 of them: measured back to back, a product with K = 16 takes N / 2 cycles for
// N >= 128 whatever M is, and for N = 64 37 cycles with M = 64 or A in tensor memory, 52 else.  The
// rest is the warps' work on what is between the products, so every part of it has warps of its
// own.  Their loops are kept short: with the loops unrolled the five roles missed the instruction
// cache and the same kernel took 1.5 times as long.
//
// Measured on one B200 at 1965 MHz: forward B16 H32 T8192 408 us (2.16 GB: 5.3 TB/s, 81 % of the
// measured copy), B16 H12 T2048 55 us (3.7 TB/s), B1 H32 T32768, which is cut, 182 us (0.54 GB, and
// 0.24 GB again for the segments' states: 4.3 TB/s); backward of the latter two 135 us (three passes of
// four tensors, 0.6 GB: 4.5 TB/s) and 407 us (cut in three; 1.6 GB, and 0.36 GB again: 4.8 TB/s).  A
// launch's start and end cost about 10 us.  Called without a pause for seconds the kernel reaches the
// board's power limit (1000 W; a plain copy takes 550), the clock falls to 1.5 GHz, and the first takes
// 480 to 500 us.  A chunk takes 3620 cycles: the products one after the other with what they wait for.
// What did not help, all measured:
// three slots for the tiles at the price of one buffer for y' (444 us, 425 then), a second P in tensor
// memory, so that the next chunk's is there early, at the price of a state product in 64 columns (457), 28
// warps with two that issue, a prefetch of the next tiles to L2, y' unrolled.
//
// Precision: x, y, w are exact in bf16 and every product accumulates in fp32.  Each summand of
// an output passes one operand rounded to bf16, P o m or C (2^-8 of it, as coarse as the
// output's own rounding): an output's error is 2.35e-3 of its size against 1.66e-3 for its own
// rounding alone.  P o m in two parts (the second over P's columns) left 1.88e-3 and took 478 us
// where this takes 413, timed in turn; for a second part of C there is no shared memory.  The state is an fp32 result that is carried on: it stays in fp32
// registers, and the decayed rows y' that enter it are three bf16 numbers, all of fp32 (two
// would leave 2.5e-6 of the state), cut off rather than rounded, so that an infinity's parts agree.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>

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
constexpr int THREADS = 768;
constexpr uint32_t TILE = CHUNK * D * 2;  // 16 KB: one role's tile, 128-byte swizzled rows

// Shared-memory map (bytes from a 1024-byte aligned base); the slots and buffers in twos are taken in turn.
constexpr uint32_t OFF_X = 0;
constexpr uint32_t OFF_Y = 2 * TILE;
constexpr uint32_t OFF_W = 4 * TILE;
constexpr uint32_t OFF_YS = 6 * TILE;            // y' in three parts
constexpr uint32_t OFF_C = OFF_YS + 6 * TILE;    // C^T [64][64] bf16
constexpr uint32_t C_BYTES = D * D * 2;
constexpr uint32_t OFF_OUT = OFF_C + 2 * C_BYTES;  // output tile (one)
constexpr uint32_t OFF_SEG = OFF_OUT + TILE;       // 2 segments said ahead
struct Said {
  int valid;           // 0: there are no more
  int pass, reverse;
  int unit, t_lo, rows, n, nchunks;  // its place, its rows and tokens, their chunks
  int last, slot;      // as in lattn::Segment
  int hand_to;         // the slot of the state that it hands on, or -1
  float full;          // gamma^128
  // Powers of gamma, laid out so that either way their users count down in the columns:
  float ct[32];        // gamma^31 .. gamma^0; reverse: gamma^0 .. gamma^31
  float pw[CHUNK];     // gamma^0 .. gamma^127; reverse: gamma^127 .. gamma^0
  float pad[32];       // (read for columns that the mask leaves out)
  // gamma^x in pw.
  __device__ __forceinline__ int at(int x) const { return reverse ? CHUNK - 1 - x : x; }
};
constexpr uint32_t OFF_BAR = OFF_SEG + 2 * sizeof(Said);
constexpr uint32_t OFF_TSLOT = OFF_BAR + 28 * 8;
constexpr uint32_t OFF_ABORT = OFF_TSLOT + 4;
constexpr uint32_t OFF_TOTAL = OFF_ABORT + 4;
constexpr uint32_t OFF_NUMBER = OFF_TOTAL + 4;
constexpr uint32_t SMEM_USED = OFF_NUMBER + 4;
constexpr uint32_t SMEM_BYTES = SMEM_USED + 1024;  // + alignment slack
static_assert(SMEM_BYTES <= 227 * 1024, "one CTA's shared memory");

// Tensor memory columns: P in fp32, P in bf16, x C, P w, the state's product (three parts).
constexpr uint32_t T_P = 0, T_PB = 128, T_XC = 192, T_PW = 256, T_M = 320, TMEM_COLS = 512;

// mbarriers.  Chunks are numbered through over a CTA's segments; of barriers in twos chunk i takes
// number i % 2, and no warp can arrive at one a second time before the others' first: its next arrival
// there follows a product that waited for all.
enum {
  FX = 0, FY = 2, FW = 4,        // a slot's tile is loaded
  EX = 6, EY = 8, EW = 10,       // and read
  PFULL = 12, PREADY = 13, YREADY = 14, CREADY = 16, MFULL = 17, OFULL = 19, OFREE = 20, NEVER = 21, DRAIN = 22,
  SAID = 23, HEARD = 25, SUM = 27,  // a segment is said, and done with; the number of chunks is known
  NUM_BARS = 28
};
constexpr long long WAIT_LIMIT = 1ll << 32;            // SM cycles, ~2 s
constexpr long long INJECTED_WAIT_LIMIT = 1ll << 20;
constexpr int OUT_ROWS = 32;                           // rows of an output store: one warp's

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// tmem_ld_16x256b_x8 over 2 groups of 8 columns (16 columns).
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(taddr));
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
  for (;;) {
    // (A waiting warp shares its scheduler with working ones: few instructions a try.)
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > limit) {
      *abort = 1;
      record_device_error(-5 /* TTT_ERR_TIMEOUT */);
      return false;
    }
  }
}

// False once a wait of this CTA has run out: the caller leaves its loop.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                     long long limit = WAIT_LIMIT) {
  return mbar_try_wait(bar, parity) || wait_longer(bar, parity, abort, limit);
}

// The same for a whole warp, one answer for all lanes.  (Mostly the turn is over: one try and one vote.)
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_longer(bar, parity, abort, WAIT_LIMIT));
}

// A pair's leading bits as bf16, cut off: three such parts hold all 24 bits, and all have the value's sign.
__device__ __forceinline__ uint32_t leading_bf16x2(float2 x) {
  return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}
// x less a pair of bf16 numbers, exact for x's leading bits.
__device__ __forceinline__ float2 minus_bf16x2(float2 x, uint32_t b) {
  float2 d;
  asm("{\n\t.reg .b16 lo, hi, m;\n\tmov.b32 {lo, hi}, %2;\n\tmov.b16 m, 0xBF80;\n\t"
      "fma.rn.f32.bf16 %0, lo, m, %3;\n\tfma.rn.f32.bf16 %1, hi, m, %4;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "r"(b), "f"(x.x), "f"(x.y));
  return d;
}

// After tmem_wait_ld: registers that a tensor memory load filled, not to be used before this place.
template <int N>
__device__ __forceinline__ void loaded(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// A product of N steps along its inner axis, whose operands advance by these bytes a step.
template <int N>
__device__ __forceinline__ void issue(uint32_t d, uint64_t a, uint32_t step_a, uint64_t b, uint32_t step_b, uint32_t id) {
#pragma unroll
  for (int k = 0; k < N; ++k) umma_ss_w(d, a + k * (step_a >> 4), b + k * (step_b >> 4), id, k > 0);
}

// A state handed from CTA j - 1 to CTA j: each of the four state warps counts in once it has written.
__device__ __forceinline__ void hand_on(int *flag) {
  __threadfence();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    __threadfence();
    atomicAdd(flag, 1);
  }
}
__device__ __forceinline__ bool wait_handed(const int *flag, volatile int *abort) {
  const long long t0 = clock64();
  for (;;) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    if (__all_sync(0xffffffffu, v == 4)) return true;
    const bool late = clock64() - t0 > WAIT_LIMIT;
    if (__any_sync(0xffffffffu, late || *abort)) {
      if (late && !*abort) {
        *abort = 1;
        record_device_error(-5 /* TTT_ERR_TIMEOUT */);
      }
      return false;
    }
    __nanosleep(200);
  }
}

// The tiles' maps of a pass.
struct Maps {
  CUtensorMap x, y, w, out;
};
struct AllMaps {
  Maps pass[lattn::MOST_PASSES];
};
// What a launch's CTAs take: `passes` passes over `units` units, the first one forward, the others in
// reverse.  Where steps > 0 they share `steps` chunks of each unit of each pass evenly: ticket[0] counts the
// CTAs, ticket[1 + j] the state that CTA j hands on in slot j; all zero before the launch.
struct Work {
  int passes, units, steps;
  int *ticket;
};

// STATE_ONLY: the segments' own states (y and w alone).  Only with BACKWARD are there passes in reverse (a
// forward kernel that could go either way took 5 % longer).
template <bool STATE_ONLY, bool BACKWARD>
__global__ void __launch_bounds__(THREADS, 1)
    attn_tc_kernel(const __grid_constant__ AllMaps maps, const __grid_constant__ lattn::Passes ps,
                   const __grid_constant__ Work work, const int inject_timeout) {
  const Params &p = ps.p[0];  // but for tensors, states and factors the passes are alike
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, w4 = warp & 3;
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + OFF_TSLOT);
  volatile int *abort = reinterpret_cast<volatile int *>(sm + OFF_ABORT);

  if (tid == 0) {
    for (int i = 0; i < NUM_BARS; ++i) {
      const bool warps4 = i == YREADY || i == YREADY + 1 || i == CREADY || i == OFREE;
      // A y slot is read by the four warps that decay it and by the product P.
      const bool y_slot = i == EY || i == EY + 1;
      const bool heard = i == HEARD || i == HEARD + 1;  // by the warps of loads, P, y', state and outputs
      mbar_init(&bars[i], heard ? (STATE_ONLY ? 9 : 21) : i == PREADY ? 8 : y_slot ? (STATE_ONLY ? 4 : 5) : warps4 ? 4 : 1);
    }
    *abort = 0;
    fence_mbarrier_init();
    for (int i = 0; i < work.passes; ++i) {
      if (!STATE_ONLY) {
        prefetch_tensormap(&maps.pass[i].x);
        prefetch_tensormap(&maps.pass[i].out);
      }
      prefetch_tensormap(&maps.pass[i].y);
      prefetch_tensormap(&maps.pass[i].w);
    }
  }
  if (warp == 2) {
    tmem_alloc(tslot, TMEM_COLS);
    tmem_relinquish();
  }
  int *number = reinterpret_cast<int *>(sm + OFF_NUMBER);
  if (tid == 0) *number = work.steps ? atomicAdd(work.ticket, 1) : (int)blockIdx.x;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tb = *tslot;  // all columns are this CTA's: the base is 0, which the roles take as a constant

  const int cta = *number;
  auto chunk_start = [](const Said &g, int nchunks, int c) { return (BACKWARD && g.reverse ? nchunks - 1 - c : c) * CHUNK; };
  Said *segments = reinterpret_cast<Said *>(sm + OFF_SEG);
  // Segment k, as warp 3 says it; false: there is none, or a wait ran out.
  auto hear = [&](int k, bool &ok) {
    if (ok) ok = wait_warp(&bars[SAID + (k & 1)], (uint32_t)(k >> 1) & 1u, abort);
    return ok && segments[k & 1].valid;
  };
  auto heard = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[HEARD + (k & 1)]);
  };

  bool ok = true;
  if (inject_timeout) ok = wait(&bars[NEVER], 0, abort, INJECTED_WAIT_LIMIT);

  if (warp == 0) {
    // ---- loads -------------------------------------------------------------------
    int i = 0;
    for (int k = 0; hear(k, ok); ++k) {
      const Said &g = segments[k & 1];
      const int nchunks = g.nchunks;
      const Maps &map = maps.pass[g.pass];
      if (lane == 0) {
        for (int c = 0; ok && c < nchunks; ++c, ++i) {
          const int slot = i & 1, t0 = g.t_lo + chunk_start(g, nchunks, c);
          const uint32_t par = (uint32_t)(i / 2 - 1) & 1u;
          auto load = [&](int full, int empty, uint32_t off, const CUtensorMap *map) {
            if (i > 1 && !wait(&bars[empty + slot], par, abort)) return false;
            mbar_arrive_expect_tx(&bars[full + slot], TILE);
            tma_load_3d(sm + off + slot * TILE, map, 0, t0, g.unit, &bars[full + slot]);
            return true;
          };
          // (In the order in which a chunk's slots get free.)
          ok = load(FY, EY, OFF_Y, &map.y) && (STATE_ONLY || load(FX, EX, OFF_X, &map.x)) && load(FW, EW, OFF_W, &map.w);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      heard(k);
    }
    // A CTA that gave up lets its loads in flight land: the tiles of the last chunks, of which the
    // very last may lack some (a wait for those runs out soon: they count as never armed).
    if (lane == 0 && *abort) {
      for (int j = max(0, i - 3); j < i; ++j) {
        const uint32_t par = (uint32_t)(j / 2) & 1u;
        mbar_wait(&bars[FY + (j & 1)], par, INJECTED_WAIT_LIMIT);
        if (!STATE_ONLY) mbar_wait(&bars[FX + (j & 1)], par, INJECTED_WAIT_LIMIT);
        mbar_wait(&bars[FW + (j & 1)], par, INJECTED_WAIT_LIMIT);
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---- segments -----------------------------------------------------------------------
    // One after the other, a segment ahead of the warps that take them: what leads from one segment to
    // the next is long, rarely run code, which would stand in the way of five roles.
    // (A unit of pass i counts as unit i * units + unit here.)
    int unit_a = 0, step_a = 0, unit_b = 0, step_b = 0;  // the ends of a shared range
    if (work.steps) {
      const long long all = (long long)work.passes * work.units * work.steps;
      const long long a = all * cta / gridDim.x, b = all * (cta + 1) / gridDim.x;
      unit_a = (int)(a / work.steps), step_a = (int)(a - (long long)unit_a * work.steps);
      unit_b = (int)(b / work.steps), step_b = (int)(b - (long long)unit_b * work.steps);
    }
    auto segment = [&](int idx, Said &g) {
      g.hand_to = -1;
      if (!work.steps) {
        int k = cta + idx * (int)gridDim.x;
        if (k >= work.passes * p.segments) return false;
        g.pass = k / p.segments;
        g.reverse = BACKWARD && g.pass > 0;
        k -= g.pass * p.segments;
        const lattn::Segment o = lattn::segment_of<STATE_ONLY>(p, k, g.reverse);
        g.unit = o.unit, g.t_lo = o.t_lo, g.rows = o.rows, g.last = o.last, g.slot = o.slot;
      } else {
        const int whole0 = step_a ? unit_a + 1 : unit_a;
        const int k = idx - (step_b ? 1 : 0) + whole0;
        int lo = 0, hi = work.steps;
        if (step_b && idx == 0) {
          g.unit = unit_b;
          hi = step_b;
          g.hand_to = cta;
        } else if (k < unit_b) {
          g.unit = k;
        } else if (k == unit_b && step_a) {
          g.unit = unit_a;
          lo = step_a;
        } else {
          return false;
        }
        g.pass = g.unit / work.units;
        g.reverse = BACKWARD && g.pass > 0;
        g.unit -= g.pass * work.units;
        g.t_lo = (g.reverse ? work.steps - hi : lo) * CHUNK;
        g.rows = min((g.reverse ? work.steps - lo : hi) * CHUNK, p.T) - g.t_lo;
        g.last = hi == work.steps;
        g.slot = lo ? cta - 1 : -1;
      }
      g.n = min(max(lattn::sequence_length(p.lengths, g.unit / p.H, p.T) - g.t_lo, 0), g.rows);
      g.nchunks = (g.n + CHUNK - 1) / CHUNK;
      return true;
    };
    Said g;
    int total = 0;  // (a lane every 32nd segment: there may be thousands of a chunk each)
    for (int k = lane; segment(k, g); k += 32) total += g.nchunks;
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) {
      *reinterpret_cast<int *>(sm + OFF_TOTAL) = total;
      mbar_arrive(&bars[SUM]);
    }
    for (int k = 0; ok; ++k) {
      if (k > 1 && !(ok = wait_warp(&bars[HEARD + (k & 1)], (uint32_t)(k / 2 - 1) & 1u, abort))) break;
      Said &to = segments[k & 1];
      const bool valid = segment(k, g);
      if (valid) {
        const float ld = p.log_decay[g.unit % p.H];
        g.full = decay_pow(ld, CHUNK);
        for (int n = lane; n < CHUNK; n += 32) to.pw[g.at(n)] = decay_pow(ld, n);
        to.ct[lane] = decay_pow(ld, g.reverse ? lane : 31 - lane);
      }
      if (lane == 0) {
        to.valid = valid;
        if (valid) {
          to.pass = g.pass, to.reverse = g.reverse, to.unit = g.unit, to.t_lo = g.t_lo, to.rows = g.rows, to.n = g.n, to.nchunks = g.nchunks;
          to.last = g.last, to.slot = g.slot, to.hand_to = g.hand_to, to.full = g.full;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[SAID + (k & 1)]);
      if (!valid) break;
    }
  } else if (warp == 1) {
    // ---- products (the whole warp, converged; one lane elected to issue).  They do not depend on
    // where a segment ends. -----------------------------------------------------------------
    constexpr uint32_t ID_P = idesc_bf16_f32(128, 128, false, false, false);
    constexpr uint32_t ID_XC = idesc_bf16_f32(128, 64, false, false, false);
    constexpr uint32_t ID_PW = idesc_bf16_f32(128, 64, false, true, false);
    constexpr uint32_t ID_M = idesc_bf16_f32(64, 192, true, true, false);
    if (ok) ok = wait_warp(&bars[SUM], 0, abort);
    const int total = ok ? *reinterpret_cast<const int *>(sm + OFF_TOTAL) : 0;
    auto scores = [&](int i) {  // P of chunk i, once its tiles are in
      const uint32_t slot = i & 1, par = (uint32_t)(i >> 1) & 1u;
      if (!wait_warp(&bars[FX + slot], par, abort) || !wait_warp(&bars[FY + slot], par, abort)) return false;
      tc_fence_after_sync();
      issue<4>(T_P, smem_desc_sw128(sbase + OFF_X + slot * TILE, 16, 1024), 32,
               smem_desc_sw128(sbase + OFF_Y + slot * TILE, 16, 1024), 32, ID_P);
      umma_commit_w(&bars[PFULL]);
      if (i + 2 < total) umma_commit_w(&bars[EY + slot]);  // (a commit that nothing waits for could outlive the CTA)
      return true;
    };
    if (!STATE_ONLY && ok && total > 0) ok = scores(0);
    for (int i = 0; ok && i < total; ++i) {
      const uint32_t slot = i & 1, par = (uint32_t)i & 1u, par2 = (uint32_t)(i >> 1) & 1u;
      const uint32_t w = sbase + OFF_W + slot * TILE;
      // w^T y', once y' is written, the last product read and C's operand written.
      if (!(ok = wait_warp(&bars[YREADY + slot], par2, abort))) break;
      if (!(ok = wait_warp(&bars[CREADY], par, abort))) break;
      if (!(ok = wait_warp(&bars[FW + slot], par2, abort))) break;
      tc_fence_after_sync();
      issue<8>(T_M, smem_desc_sw128(w, 8192, 1024), 2048,
               smem_desc_sw128(sbase + OFF_YS + slot * (3 * TILE), TILE, 1024), 2048, ID_M);
      umma_commit_w(&bars[MFULL + slot]);
      if (STATE_ONLY) {
        if (i + 2 < total) umma_commit_w(&bars[EW + slot]);
        continue;
      }
      // x C, once the outputs of the last chunk are read.
      if (i > 0 && !(ok = wait_warp(&bars[OFREE], par ^ 1u, abort))) break;
      tc_fence_after_sync();
      issue<4>(T_XC, smem_desc_sw128(sbase + OFF_X + slot * TILE, 16, 1024), 32,
               smem_desc_sw128(sbase + OFF_C + slot * C_BYTES, 16, 1024), 32, ID_XC);
      if (i + 2 < total) umma_commit_w(&bars[EX + slot]);
      // P is read and its bf16 form written: P w, then the next chunk's P.  (In this order: where the next
      // chunk lies behind empty segments, its tiles come only when every warp is done with this one's
      // segment, the output warps among them.)
      if (!(ok = wait_warp(&bars[PREADY], par, abort))) break;
      tc_fence_after_sync();
      {
        const uint64_t b = smem_desc_sw128(w, 8192, 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k) umma_ts_w(T_PW, T_PB + 8 * k, b + k * (2048 >> 4), ID_PW, k > 0);
      }
      umma_commit_w(&bars[OFULL]);
      if (i + 2 < total) umma_commit_w(&bars[EW + slot]);
      if (i + 1 < total && !(ok = scores(i + 1))) break;
    }
    __syncwarp();
    if (*abort) {  // products in flight end before the tensor memory is freed
      umma_commit_w(&bars[DRAIN]);
      mbar_wait(&bars[DRAIN], 0, WAIT_LIMIT);
    }
  } else if (!STATE_ONLY && warp >= 4 && warp < 12) {
    // ---- P: mask and decay, to bf16 ------------------------------------------------------
    // Row t = 32 w4 + lane, blocks 2 half and 2 half + 1 of 32 columns.  Off the diagonal block the
    // power of gamma is the product of one of the row's and one of the column's (ct), both at most 1.
    const int half = (warp - 4) >> 2;
    const uint32_t row = tmem_addr(0, 32 * w4, T_P), dst = tmem_addr(0, 32 * w4, T_PB);
    int i = 0;
    for (int k = 0; hear(k, ok); ++k) {
      const Said &g = segments[k & 1];
      const int nchunks = g.nchunks, ntok = g.n;
      auto reverse = [&]() { return BACKWARD && g.reverse; };  // (not kept: a register is worth more than a read)
      const float a = ps.p[BACKWARD ? g.pass : 0].a;
      const float *pw = g.pw, *ct = g.ct;
      for (int c = 0; c < nchunks; ++c, ++i) {
        const int n = min(CHUNK, ntok - chunk_start(g, nchunks, c));
        if (!(ok = wait_warp(&bars[PFULL], (uint32_t)i & 1u, abort))) break;
        tc_fence_after_sync();
#pragma unroll 1
        for (int j = 2 * half; j < 2 * half + 2; ++j) {
          const int d = reverse() ? j - w4 : w4 - j;
          uint32_t pk[16];
          if (d < 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = 0u;
          } else {
            uint32_t r[32];
            tmem_ld_32x32b_x32(row + 32 * j, r);
            // The columns that count: s <= t, or, in reverse, s >= t and of a token.
            const int least = reverse() ? lane - 32 * d : 0, most = reverse() ? n - 32 * j : 32 * d + lane + 1;
            if (d == 0 || (reverse() && most < 32)) {
              // gamma^(t - s), or gamma^(s - t): in pw, backwards from here.
              const float *f = pw + (reverse() ? CHUNK - 1 - 32 * d : 32 * d) + lane;
              const float2 a2 = make_float2(a, a);
              tmem_wait_ld();
              loaded(r);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float v[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int s = 2 * e + h;
                  v[h] = s < most && s >= least ? __uint_as_float(r[s]) * f[-s] : 0.f;
                }
                const float2 u = __fmul2_rn(a2, make_float2(v[0], v[1]));
                pk[e] = pack_bf16x2(u.x, u.y);
              }
            } else {
              const float b = a * pw[reverse() ? CHUNK - 1 - 32 * d + lane : lane + 32 * d - 31];
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
          // The last chunk's P w has read what this overwrites: it was issued before this chunk's P, and the
          // barrier of that stands for all products issued before.
          tmem_st_32x32b_x16(dst + 16 * j, pk);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[PREADY]);
      }
      heard(k);
    }
  } else if (warp >= 12 && warp < 16) {
    // ---- y' (zeros past the end), and zeros over w's rows past the end: what lies there is any
    // value, and enters the products ---------------------------------------------------------
    const int s = 32 * w4 + lane;
    const uint32_t row = sw128_offset(s, 0);  // piece q of the row is at row ^ (16 q)
    int i = 0;
    for (int k = 0; hear(k, ok); ++k) {
      const Said &g = segments[k & 1];
      const int nchunks = g.nchunks, ntok = g.n;
      auto reverse = [&]() { return BACKWARD && g.reverse; };  // (not kept: a register is worth more than a read)
      const float e = ps.p[BACKWARD ? g.pass : 0].e;
      // (gamma^(s + 1) of the last row in reverse is gamma^128, which has a place of its own.)
      const float h_full = e * (!reverse() ? g.pw[CHUNK - 1 - s] : s == CHUNK - 1 ? g.full : g.pw[g.at(s + 1)]);
      for (int c = 0; ok && c < nchunks; ++c, ++i) {
        const int n = min(CHUNK, ntok - chunk_start(g, nchunks, c));
        const uint32_t slot = i & 1, par2 = (uint32_t)(i >> 1) & 1u;
        uint8_t *ty = sm + OFF_Y + slot * TILE;
        uint8_t *ys = sm + OFF_YS + slot * (3 * TILE);
        if (!(ok = wait_warp(&bars[FY + slot], par2, abort))) break;
        // The buffer is free when the product that read it, two chunks ago, is done.
        if (i > 1 && !(ok = wait_warp(&bars[MFULL + slot], par2 ^ 1u, abort))) break;
        float h1 = h_full;
        if (n < CHUNK) {
          if (!reverse()) h1 = e * g.pw[max(n - 1 - s, 0)];
          if (!(ok = wait_warp(&bars[FW + slot], par2, abort))) break;
          if (s >= n) {
#pragma unroll 1
            for (uint32_t q = 0; q < 128; q += 16) {
              *reinterpret_cast<uint4 *>(ty + (row ^ q)) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4 *>(sm + OFF_W + slot * TILE + (row ^ q)) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        const float2 h = make_float2(h1, h1);
        uint4 y = *reinterpret_cast<const uint4 *>(ty + row);
#pragma unroll 1
        for (uint32_t q = 0; q < 128; q += 16) {
          const uint32_t u[4] = {y.x, y.y, y.z, y.w};
          y = *reinterpret_cast<const uint4 *>(ty + (row ^ ((q + 16) & 127)));
          uint32_t part[3][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 r = __fmul2_rn(h, unpack_bf16x2(u[e]));
#pragma unroll
            for (int m = 0; m < 3; ++m) {
              part[m][e] = leading_bf16x2(r);
              if (m < 2) r = minus_bf16x2(r, part[m][e]);
            }
          }
#pragma unroll
          for (int m = 0; m < 3; ++m)
            *reinterpret_cast<uint4 *>(ys + m * TILE + (row ^ q)) =
                make_uint4(part[m][0], part[m][1], part[m][2], part[m][3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[EY + slot]);
          mbar_arrive(&bars[YREADY + slot]);
        }
      }
      heard(k);
    }
  } else if (warp >= 16 && warp < 20) {
    // ---- state ----------------------------------------------------------------------
    // A product of M = 64 lies in the lower 16 of each warp's 32 lanes; the 16x256b load gives
    // this thread rows row and row + 8 of C^T at columns 8 j + col + {0, 1}: C[4 j + {0, 1}] and
    // C[4 j + {2, 3}].
    const int row = 16 * w4 + (lane >> 2), col = 2 * (lane & 3);
    int i = 0;
    for (int k = 0; hear(k, ok); ++k) {
      const Said &g = segments[k & 1];
      const int nchunks = g.nchunks, ntok = g.n;
      float C[32];
      {
        // (A state handed on lies as this kernel carries it, C^T.)
        const bool handed = work.steps && g.slot >= 0;
        if (handed && !(ok = wait_handed(work.ticket + 1 + g.slot, abort))) break;
        const float *C0 = lattn::start_state(ps.p[g.pass], g.unit, g.slot);
        const bool as_is = ps.p[g.pass].transposed || handed;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int r = row + 8 * ((e >> 1) & 1), cc = 8 * (e >> 2) + col + (e & 1);
          C[e] = C0 ? __ldcg(C0 + (as_is ? r * D + cc : cc * D + r)) : 0.f;
        }
      }
      for (int c = 0; c < nchunks; ++c, ++i) {
        // The operand of x C, in the buffer whose last reader, x C two chunks ago, was issued before
        // the last chunk's w^T y', whose end these warps have seen.
        if (!STATE_ONLY) {
          uint8_t *to = sm + OFF_C + (i & 1) * C_BYTES;
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            *reinterpret_cast<uint32_t *>(to + sw128_offset(row + 8 * ((e >> 1) & 1), 8 * (e >> 2) + col)) =
                pack_bf16x2(C[e], C[e + 1]);
          fence_proxy_async_smem();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[CREADY]);
        const int n = min(CHUNK, ntok - chunk_start(g, nchunks, c));
        const float dn = n == CHUNK ? g.full : g.pw[BACKWARD ? g.at(n) : n];
        if (!(ok = wait_warp(&bars[MFULL + (i & 1)], (uint32_t)(i >> 1) & 1u, abort))) break;
        tc_fence_after_sync();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t m[3][8];
#pragma unroll
          for (int q = 0; q < 3; ++q) tmem_ld_16x256b_x2(tmem_addr(0, 32 * w4, T_M + 64 * q + 16 * h), m[q]);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 3; ++q) loaded(m[q]);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            auto pair = [&](int q) { return make_float2(__uint_as_float(m[q][e]), __uint_as_float(m[q][e + 1])); };
            // Where an infinity of y or w makes the first part's sum infinite, the others' are infinities of its
            // sign or NaN (inf - inf, 0 inf): min makes a finite number of both but for -inf, which agrees.  (A
            // select of the finite ones instead: 1 to 2 % of the kernel's time, against 0.3 to 1 %.)
            float2 rest = __fadd2_rn(pair(1), pair(2));
            rest.x = fminf(rest.x, FLT_MAX);
            rest.y = fminf(rest.y, FLT_MAX);
            const float2 v = __ffma2_rn(make_float2(dn, dn), make_float2(C[8 * h + e], C[8 * h + e + 1]),
                                        __fadd2_rn(pair(0), rest));
            C[8 * h + e] = v.x;
            C[8 * h + e + 1] = v.y;
          }
        }
      }
      if (g.hand_to >= 0) {
        float *Co = p.slots + (long long)(g.hand_to) * (D * D);
#pragma unroll
        for (int e = 0; e < 32; ++e) Co[(row + 8 * ((e >> 1) & 1)) * D + 8 * (e >> 2) + col + (e & 1)] = C[e];
        hand_on(work.ticket + 1 + g.hand_to);
      } else if (float *Co = lattn::end_state(ps.p[g.pass], g.unit, g.slot, g.last)) {
#pragma unroll
        for (int e = 0; e < 32; ++e) Co[(8 * (e >> 2) + col + (e & 1)) * D + row + 8 * ((e >> 1) & 1)] = C[e];
      }
      heard(k);
    }
  } else if (!STATE_ONLY && warp >= 20) {
    // ---- outputs: each warp its own 32 rows ---------------------------------------------
    const int t = 32 * w4 + lane;
    int i = 0;
    for (int k = 0; hear(k, ok); ++k) {
      const Said &g = segments[k & 1];
      const int nchunks = g.nchunks, ntok = g.n;
      for (int c = 0; c < nchunks; ++c, ++i) {
        const int c0 = chunk_start(g, nchunks, c), n = min(CHUNK, ntok - c0);
        const int x = BACKWARD && g.reverse ? max(n - 1 - t, 0) : t + 1;
        const float f1 = ps.p[BACKWARD ? g.pass : 0].c * (x == CHUNK ? g.full : g.pw[BACKWARD ? g.at(x) : x]);
        const float2 f = make_float2(f1, f1);
        if (!(ok = wait_warp(&bars[OFULL], (uint32_t)i & 1u, abort))) break;
        tc_fence_after_sync();
        if (lane == 0) tma_store_wait_read();  // the warp's last store has read the tile
        __syncwarp();
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {
          uint32_t xc[16], pv[16], o[8];
          tmem_ld_32x32b_x16(tmem_addr(0, 32 * w4, T_XC + 16 * h), xc);
          tmem_ld_32x32b_x16(tmem_addr(0, 32 * w4, T_PW + 16 * h), pv);
          tmem_wait_ld();
          loaded(xc);
          loaded(pv);
          if (h == 3) {  // the products' places are free
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[OFREE]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 v =
                __ffma2_rn(f, make_float2(__uint_as_float(xc[2 * e]), __uint_as_float(xc[2 * e + 1])),
                           make_float2(__uint_as_float(pv[2 * e]), __uint_as_float(pv[2 * e + 1])));
            o[e] = pack_bf16x2(v.x, v.y);
          }
          if (t >= n) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 0u;
          }
          *reinterpret_cast<uint4 *>(sm + OFF_OUT + sw128_offset(t, 16 * h)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4 *>(sm + OFF_OUT + sw128_offset(t, 16 * h + 8)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          const int t0 = g.t_lo + c0 + 32 * w4;
          if (t0 < p.T) tma_store_3d(&maps.pass[g.pass].out, sm + OFF_OUT + 32 * w4 * 128, 0, t0, g.unit);
        }
      }
      // Rows of chunks wholly behind the end (those of the last chunk are in its tile).
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(ps.p[g.pass].out) + ((long long)g.unit * p.T + g.t_lo) * D;
      const int x0 = min(nchunks * CHUNK, g.rows) * (D / 8), x1 = g.rows * (D / 8);
      for (int x = x0 + (tid & 127); x < x1; x += 128)
        reinterpret_cast<uint4 *>(out)[x] = make_uint4(0u, 0u, 0u, 0u);
      heard(k);
    }
    if (lane == 0) tma_store_wait_read();
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
