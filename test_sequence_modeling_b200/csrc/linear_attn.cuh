// linear_attn.cuh - linear attention with a decay for each head: the chunked form over
// whole sequences on the CUDA cores (any input type), the scan that joins a sequence cut
// into segments, and the recurrent step for single tokens.
//
// The TTT write-up §03.8 makes TTT with a linear f and batch gradient descent equal to
// linear attention; the decay is the forget factor of the Titans article (§二.1(2)) held
// constant per head.  With gamma = exp(log_decay[head]) and the state S [D][D] of one
// (batch, head) unit:
//   S_t = gamma S_{t-1} + k_t^T v_t,    z_t = scale q_t S_t.
//
// One pass ("roles" x, y, w in place of q, k, v) serves the forward and all three
// gradients.  For a chunk of n tokens t, s = 0..n-1 and the state C carried into it:
//   out_t = a sum_s m_ts (x_t . y_s) w_s + c f_t x_t C
//   C    <- gamma^n C + e sum_s h_s y_s^T w_s
// forward pass:  m_ts = gamma^(t-s) for s <= t, f_t = gamma^(t+1), h_s = gamma^(n-1-s)
// reverse pass:  m_ts = gamma^(s-t) for s >= t, f_t = gamma^(n-1-t), h_s = gamma^(s+1),
//                chunks taken from the end of the sequence
//   Z  : x, y, w = Q, K, V    C = S     a = c = scale, e = 1
//   dQ : x, y, w = dZ, V, K   C = S^T   a = c = scale, e = 1
//   dK : x, y, w = V, dZ, Q   C = G^T   a = e = scale, c = 1      (reverse)
//   dV : x, y, w = K, Q, dZ   C = G     a = e = scale, c = 1      (reverse)
// with G the gradient of the state, dS_T after the last token; G before the first token is
// dS0.  The powers of gamma are exp(n log_decay), never a product of negative powers: a
// strong decay cannot overflow, and log_decay = -inf is gamma = 0.
//
// A sequence's tokens end at lengths[b] (clamped to [0, T]); rows behind the end are not
// used, whatever they hold, and their outputs are zeros.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rope.cuh"
#include "simt.cuh"

namespace ttt {
namespace lattn {

using simt::D;
using simt::load_in;

constexpr int CHUNK = 64;
constexpr int THREADS = 128;
constexpr int STEP_THREADS = 256;  // of the single-token step
constexpr int LD = D + 4;  // padded row stride: 8 rows' float4 at one column hit 8 distinct bank groups

// How the units' sequences are dealt out to segments: units below `whole` are one segment each, the others
// are cut into nseg segments of seg_len tokens (whole chunks of every kernel).  For states alone only the
// cut units count, without their last segments, which no segment follows.
struct Cut {
  int whole, nseg, seg_len;
  __host__ __device__ int segments(int units, bool state_only) const {
    return state_only ? (units - whole) * (nseg - 1) : whole + (units - whole) * nseg;
  }
};
struct Segment {
  int unit;
  int t_lo, rows;     // its rows (of T)
  bool last;          // of its unit, in the order of the pass
  int slot;           // of the state that it starts from, or -1: it is its unit's first
};

struct Params {
  const void *X, *Y, *W;   // [units][T][D]
  const float *log_decay;  // [H]
  const int *lengths;      // [B] or NULL
  const float *C0;         // [units][D][D] carried state at the start of the pass, or NULL (zero)
  float *slots;            // [cut units][nseg][D][D] states that the segments of cut units start from
  bool transposed;         // the pass carries the transposes of C0 and of the slots
  float a, c, e;           // the three factors above
  void *out;               // [units][T][D]
  float *C_out;            // [units][D][D] carried state after the pass, or NULL
  float *slots_out;        // [cut units][nseg][D][D], else NULL: no outputs, only the states that the cut
                           // units' segments leave by themselves (the last one's has no reader)
  int H, T;
  Cut cut;
  int segments;            // this launch's
};

// The passes of one launch: the forward's one, or the three of a backward (the first one forward, the
// others in reverse; or one of each for states alone), which have no part in one another.
constexpr int MOST_PASSES = 3;
struct Passes {
  Params p[MOST_PASSES];
};

// Segment k of a launch; its slot, for states alone, is that of the state that it leaves.
template <bool STATE_ONLY>
__device__ __forceinline__ Segment segment_of(const Params &p, int k, bool reverse) {
  Segment g;
  const int rest = STATE_ONLY ? k : k - p.cut.whole, n = STATE_ONLY ? p.cut.nseg - 1 : p.cut.nseg;
  const bool cut = rest >= 0;
  const int q = cut ? rest / n : 0, seg = cut ? rest - q * n + (STATE_ONLY && reverse) : 0;
  const int len = cut ? p.cut.seg_len : p.T;
  g.unit = cut ? p.cut.whole + q : k;
  g.t_lo = seg * len;
  g.rows = min(len, p.T - g.t_lo);
  g.last = !STATE_ONLY && (!cut || seg == (reverse ? 0 : p.cut.nseg - 1));
  g.slot = cut ? q * p.cut.nseg + seg : -1;
  return g;
}
// The state a segment starts from (NULL: zero).
__device__ __forceinline__ const float *start_state(const Params &p, int unit, int slot) {
  if (p.slots_out) return nullptr;
  if (slot >= 0) return p.slots + (long long)slot * (D * D);
  return p.C0 ? p.C0 + (long long)unit * (D * D) : nullptr;
}
// Where the state it ends in goes (NULL: nowhere).
__device__ __forceinline__ float *end_state(const Params &p, int unit, int slot, bool last) {
  if (p.slots_out) return p.slots_out + (long long)slot * (D * D);
  return p.C_out && last ? p.C_out + (long long)unit * (D * D) : nullptr;
}

__device__ __forceinline__ float decay_pow(float g, int n) { return n == 0 ? 1.f : expf(g * (float)n); }

__device__ __forceinline__ int sequence_length(const int *lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

__device__ __forceinline__ void store_out(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16 *p, float4 v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t *>(&lo);
  u.y = *reinterpret_cast<const uint32_t *>(&hi);
  *reinterpret_cast<uint2 *>(p) = u;
}
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// acc += x (u, v): one row of an 8 x 8 register tile, columns 4 tx .. and 32 + 4 tx ...
__device__ __forceinline__ void row_times(float (&acc)[8], float x, float4 u, float4 v) {
  acc[0] = fmaf(x, u.x, acc[0]);
  acc[1] = fmaf(x, u.y, acc[1]);
  acc[2] = fmaf(x, u.z, acc[2]);
  acc[3] = fmaf(x, u.w, acc[3]);
  acc[4] = fmaf(x, v.x, acc[4]);
  acc[5] = fmaf(x, v.y, acc[5]);
  acc[6] = fmaf(x, v.z, acc[6]);
  acc[7] = fmaf(x, v.w, acc[7]);
}
__device__ __forceinline__ float4 lds4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float component(float4 v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// acc (rows ty + 8 i, i0 <= i < i1) += A B for columns k0 .. k1 - 1 of A, rows of B: tiles in shared memory.
template <int I0, int I1>
__device__ __forceinline__ void rows_times_rows(float (&acc)[8][8], const float *A, const float *B, int k0, int k1, int tx,
                                                int ty) {
#pragma unroll 1
  for (int k = k0; k < k1; k += 4) {
    float4 a[8];
#pragma unroll
    for (int i = I0; i < I1; ++i) a[i] = lds4(A + (ty + 8 * i) * LD + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const float4 u = lds4(B + (k + kk) * LD + 4 * tx), v = lds4(B + (k + kk) * LD + 32 + 4 * tx);
#pragma unroll
      for (int i = I0; i < I1; ++i) row_times(acc[i], component(a[i], kk), u, v);
    }
  }
}

constexpr size_t SMEM_BYTES = sizeof(float) * (size_t)(5 * CHUNK * LD + 2 * CHUNK + 4);

// One CTA takes one segment of one unit, in fp32 fused multiply-adds.  Its two halves of 64 threads hold
// an 8 x 8 register tile of one 64 x 64 product each: the first takes m o (x y^T) and then the state's
// y^T w, the second x C and then (m o x y^T) w on top of it, so that each does as much.  8 x 8, because with
// 4 x 4 tiles and 256 threads the operands' reads from shared memory took twice the arithmetic's time:
// forward B6 H8 T1999 145 us, against 124 now, of which the arithmetic is about half.  B16 H12 T2048 436 us
// (26 TFLOP/s without the quarters left out, 35 % of the CUDA cores' 74), backward 863 us.
template <typename InT, bool REVERSE, bool STATE_ONLY>
__device__ __forceinline__ void attn_segment(const Params &p, int segment) {
  extern __shared__ __align__(16) float sm[];
  float *Xs = sm;                // [CHUNK][LD]
  float *Ys = Xs + CHUNK * LD;
  float *Ws = Ys + CHUNK * LD;
  float *Ms = Ws + CHUNK * LD;   // a times the masked, decayed products x_t . y_s
  float *Cs = Ms + CHUNK * LD;   // the carried state
  float *pw = Cs + D * LD;       // gamma^0 .. gamma^CHUNK
  const int tid = threadIdx.x, half = tid >> 6, tx = tid & 7, ty = (tid >> 3) & 7;
  const Segment sg = segment_of<STATE_ONLY>(p, segment, REVERSE);
  const float g = p.log_decay[sg.unit % p.H];
  const int len = sequence_length(p.lengths, sg.unit / p.H, p.T);
  const int n_seg = min(max(len - sg.t_lo, 0), sg.rows);  // its tokens
  const long long row0 = (long long)sg.unit * p.T + sg.t_lo;
  const InT *X = static_cast<const InT *>(p.X) + row0 * D;
  const InT *Y = static_cast<const InT *>(p.Y) + row0 * D;
  const InT *W = static_cast<const InT *>(p.W) + row0 * D;
  InT *out = static_cast<InT *>(p.out) + row0 * D;

  // The state, in registers of the first half: rows 4 ty .. and 32 + 4 ty .., columns 4 tx .. and
  // 32 + 4 tx ...  For states alone each half takes half of the rows.
  constexpr int ROWS = STATE_ONLY ? 4 : 8;
  auto state_row = [&](int i) { return (STATE_ONLY ? 32 * half : 32 * (i >> 2)) + 4 * ty + (i & 3); };
  const bool has_state = STATE_ONLY || half == 0;
  float C[ROWS][8];
  if (has_state) {
    const float *C0 = start_state(p, sg.unit, sg.slot);
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = state_row(i), col = 32 * (j >> 2) + 4 * tx + (j & 3);
        C[i][j] = C0 ? (p.transposed ? C0[col * D + r] : C0[r * D + col]) : 0.f;
      }
  }
  auto state_to = [&](float *to, int ld) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 4)
        *reinterpret_cast<float4 *>(to + state_row(i) * ld + 8 * j + 4 * tx) =
            make_float4(C[i][j], C[i][j + 1], C[i][j + 2], C[i][j + 3]);
  };
  if (!STATE_ONLY && half == 0) state_to(Cs, LD);
  if (tid <= CHUNK) pw[tid] = decay_pow(g, tid);

  const int nchunks = (n_seg + CHUNK - 1) / CHUNK;
  for (int ci = 0; ci < nchunks; ++ci) {
    const int c0 = (REVERSE ? nchunks - 1 - ci : ci) * CHUNK;
    const int n = min(CHUNK, n_seg - c0);
    // Tiles: 16 lanes a row of 64 values, rows past the end as zeros.
    const int lr = tid >> 4, lc = 4 * (tid & 15);
#pragma unroll
    for (int i = 0; i < CHUNK; i += THREADS / 16) {
      const int r = lr + i;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x, w = x;
      if (r < n) {
        const long long at = (long long)(c0 + r) * D + lc;
        if (!STATE_ONLY) x = load4(X + at);
        y = load4(Y + at);
        w = load4(W + at);
      }
      if (!STATE_ONLY) *reinterpret_cast<float4 *>(Xs + r * LD + lc) = x;
      *reinterpret_cast<float4 *>(Ys + r * LD + lc) = y;
      *reinterpret_cast<float4 *>(Ws + r * LD + lc) = w;
    }
    if (ci + 1 < nchunks) {  // the next chunk's rows on their way to L2, 128 bytes a request
      constexpr int LINE = 128 / (int)sizeof(InT), LINES = CHUNK * D / LINE;
      const long long at = (long long)(REVERSE ? c0 - CHUNK : c0 + CHUNK) * D + tid * LINE;
      if (tid < LINES && at < (long long)n_seg * D) {
        if (!STATE_ONLY) prefetch_l2(X + at);
        prefetch_l2(Y + at);
        prefetch_l2(W + at);
      }
    }
    __syncthreads();
    if (!STATE_ONLY && half == 0) {
      // a m_ts x_t . y_s for rows t = ty + 8 i, columns s = tx + 8 j; the quarter of the tile that the
      // mask empties (i < 4 <= j; reverse: j < 4 <= i) is left out here and below.
      float acc[8][8] = {};
#pragma unroll 1
      for (int k = 0; k < D; k += 4) {
        float4 x[8], y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = lds4(Xs + (ty + 8 * i) * LD + k);
          y[i] = lds4(Ys + (tx + 8 * i) * LD + k);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (REVERSE ? (i < 4 || j >= 4) : (i >= 4 || j < 4))
              acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, acc[i][j]))));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = ty + 8 * i, s = tx + 8 * j, gap = REVERSE ? s - t : t - s;
          if (REVERSE ? (i < 4 || j >= 4) : (i >= 4 || j < 4)) Ms[t * LD + s] = gap >= 0 ? p.a * pw[gap] * acc[i][j] : 0.f;
        }
      asm volatile("bar.arrive 1, %0;" ::"n"(THREADS) : "memory");
    } else if (!STATE_ONLY) {
      float o[8][8] = {};
      rows_times_rows<0, 8>(o, Xs, Cs, 0, D, tx, ty);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = ty + 8 * i;
        const float f = t < n ? p.c * pw[REVERSE ? n - 1 - t : t + 1] : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[i][j] *= f;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");  // the first half has written m
      if (REVERSE) {
        rows_times_rows<0, 4>(o, Ms, Ws, 0, 32, tx, ty);
        rows_times_rows<0, 8>(o, Ms, Ws, 32, 64, tx, ty);
      } else {
        rows_times_rows<0, 8>(o, Ms, Ws, 0, 32, tx, ty);
        rows_times_rows<4, 8>(o, Ms, Ws, 32, 64, tx, ty);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = ty + 8 * i;
        if (t < n) {
          InT *to = out + (long long)(c0 + t) * D + 4 * tx;
          store_out(to, make_float4(o[i][0], o[i][1], o[i][2], o[i][3]));
          store_out(to + 32, make_float4(o[i][4], o[i][5], o[i][6], o[i][7]));
        }
      }
    }
    if (has_state) {
      // C <- gamma^n C + e sum_s h_s y_s^T w_s.  The chunk's sum is one of its own: added token by token C
      // would be rounded T times, not T / 64 times, which without decay costs digits (T = 32768: ~1e-6).
      float M[ROWS][8] = {};
#pragma unroll 2
      for (int s = 0; s < n; ++s) {
        const float h = p.e * pw[REVERSE ? s + 1 : n - 1 - s];
        const float4 u = lds4(Ws + s * LD + 4 * tx), v = lds4(Ws + s * LD + 32 + 4 * tx);
#pragma unroll
        for (int i = 0; i < ROWS; i += 4) {
          const float4 y = lds4(Ys + s * LD + state_row(i));
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) row_times(M[i + ii], h * component(y, ii), u, v);
        }
      }
      const float dn = pw[n];
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) C[i][j] = fmaf(dn, C[i][j], M[i][j]);
    }
    __syncthreads();  // every read of the state and of the tiles is done
    if (!STATE_ONLY && half == 0) state_to(Cs, LD);
  }
  // Rows behind the end.
  if (!STATE_ONLY) {
    for (int r = n_seg + (tid >> 4); r < sg.rows; r += THREADS / 16)
      store_out(out + (long long)r * D + 4 * (tid & 15), make_float4(0.f, 0.f, 0.f, 0.f));
  }
  if (has_state) {
    if (float *Co = end_state(p, sg.unit, sg.slot, sg.last)) state_to(Co, D);
  }
}

template <typename InT, bool STATE_ONLY>
__global__ void __launch_bounds__(THREADS, 2) attn_kernel(const __grid_constant__ Passes ps) {
  int k = blockIdx.x;
  if (k < ps.p[0].segments) return attn_segment<InT, false, STATE_ONLY>(ps.p[0], k);
  k -= ps.p[0].segments;
  const int which = k < ps.p[1].segments ? 1 : 2;
  attn_segment<InT, true, STATE_ONLY>(ps.p[which], which == 1 ? k : k - ps.p[1].segments);
}

// The states at the segments' starts of the cut units, in place: slot i of a unit holds the state that
// its segment alone leaves (M_i) and gets the state that it starts from,
//   C_0 = C0,  C_{i+1} = gamma^(n_i) C_i + M_i     (reverse: from the last segment down).
// Reads and writes nseg x 16 KB a unit once: bound by memory, and small beside the tokens.
struct ScanParams {
  float *slots[2];  // [cut units][nseg][D][D] of the forward and the reverse pass
  const float *C0[2];
  const float *log_decay;
  const int *lengths;
  int H, T;
  Cut cut;
  int blocks;       // of one pass
};

constexpr int SCAN_THREADS = 256;  // 4 values a thread: 4 CTAs a unit

__global__ void __launch_bounds__(SCAN_THREADS) scan_kernel(const ScanParams p) {
  const bool reverse = (int)blockIdx.x >= p.blocks;
  const int block = reverse ? blockIdx.x - p.blocks : blockIdx.x;
  const int q = block >> 2, unit = p.cut.whole + q;
  const int at = ((block & 3) * SCAN_THREADS + threadIdx.x) * 4;
  const float g = p.log_decay[unit % p.H];
  const int len = sequence_length(p.lengths, unit / p.H, p.T);
  float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
  const float *C0 = p.C0[reverse];
  if (C0) c = *reinterpret_cast<const float4 *>(C0 + (long long)unit * (D * D) + at);
  float *slots = p.slots[reverse] + (long long)q * p.cut.nseg * (D * D) + at;
  auto slot = [&](int k) {
    return reinterpret_cast<float4 *>(slots + (long long)(reverse ? p.cut.nseg - 1 - k : k) * (D * D));
  };
  // In batches, whose loads do not wait for one another.
  constexpr int BATCH = 8;
  for (int k0 = 0; k0 < p.cut.nseg; k0 += BATCH) {
    float4 m[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
      if (k0 + j + 1 < p.cut.nseg) m[j] = *slot(k0 + j);
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const int k = k0 + j;
      if (k < p.cut.nseg) *slot(k) = c;
      if (k + 1 < p.cut.nseg) {
        const int t_lo = (reverse ? p.cut.nseg - 1 - k : k) * p.cut.seg_len;
        const float dn = decay_pow(g, min(max(len - t_lo, 0), min(p.cut.seg_len, p.T - t_lo)));
        c = make_float4(fmaf(dn, c.x, m[j].x), fmaf(dn, c.y, m[j].y), fmaf(dn, c.z, m[j].z), fmaf(dn, c.w, m[j].w));
      }
    }
  }
}

// One token of every unit: S <- gamma S + k^T v, z = scale q S, with q and k turned by the
// token's position first when a rotary plan is given.  One CTA a unit: each thread takes four
// float4 of the state (rows ty + 16 i, columns 4 tx ..), all loaded before anything waits.
// 32 KB of state move a unit against 16 KFLOP: bound by memory (B512 H32: 85 us, 6.4 TB/s, 98 % of
// the measured copy; B1 H32: 3.1 us, a launch).
struct DecodeParams {
  const void *q, *k, *v;   // [units][D]
  const float *log_decay;  // [H]
  float scale;
  float *S;                // [units][D][D], in place
  rope::Plan plan;         // rotary == 0: none
  const int *positions;    // [B]
  int H;
  void *z;                 // [units][D]
};

template <typename InT>
__global__ void __launch_bounds__(STEP_THREADS) decode_kernel(const DecodeParams p) {
  __shared__ float qk[2][D];
  __shared__ __align__(16) float part[STEP_THREADS / 32][D];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, warp = tid >> 5, lane = tid & 31;
  const long long unit = blockIdx.x;
  float4 *S = reinterpret_cast<float4 *>(p.S + unit * (D * D)) + tx;
  float4 s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = S[(ty + 16 * i) * (D / 4)];
  const float gamma = decay_pow(p.log_decay[unit % p.H], 1);
  const float4 v = load4(static_cast<const InT *>(p.v) + unit * D + 4 * tx);
  if (tid < 2 * D) {
    const int which = tid >> 6, j = tid & (D - 1);
    const InT *row = static_cast<const InT *>(which ? p.k : p.q) + unit * D;
    float x = load_in(row, j);
    if (j < p.plan.rotary) {
      int pair, sign;
      const int partner = rope::partner_of(p.plan, j, pair, sign);
      const float2 cs = rope::cos_sin(p.positions[unit / p.H], p.plan.inv_freq[pair], p.plan.mscale);
      x = fmaf(x, cs.x, (float)sign * cs.y * load_in(row, partner));
    }
    qk[which][j] = x;
  }
  __syncthreads();
  float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    const float k = qk[1][r], q = qk[0][r];
    s[i].x = fmaf(gamma, s[i].x, k * v.x);
    s[i].y = fmaf(gamma, s[i].y, k * v.y);
    s[i].z = fmaf(gamma, s[i].z, k * v.z);
    s[i].w = fmaf(gamma, s[i].w, k * v.w);
    S[r * (D / 4)] = s[i];
    z.x = fmaf(q, s[i].x, z.x);
    z.y = fmaf(q, s[i].y, z.y);
    z.z = fmaf(q, s[i].z, z.z);
    z.w = fmaf(q, s[i].w, z.w);
  }
  // The warp's two row groups, then the eight warps.
  z.x += __shfl_xor_sync(0xffffffffu, z.x, 16);
  z.y += __shfl_xor_sync(0xffffffffu, z.y, 16);
  z.z += __shfl_xor_sync(0xffffffffu, z.z, 16);
  z.w += __shfl_xor_sync(0xffffffffu, z.w, 16);
  if (lane < 16) *reinterpret_cast<float4 *>(&part[warp][4 * tx]) = z;
  __syncthreads();
  if (tid < D / 4) {
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < STEP_THREADS / 32; ++w) {
      const float4 a = *reinterpret_cast<const float4 *>(&part[w][4 * tid]);
      t.x += a.x;
      t.y += a.y;
      t.z += a.z;
      t.w += a.w;
    }
    store_out(static_cast<InT *>(p.z) + unit * D + 4 * tid,
              make_float4(p.scale * t.x, p.scale * t.y, p.scale * t.z, p.scale * t.w));
  }
}

}  // namespace lattn
}  // namespace ttt
