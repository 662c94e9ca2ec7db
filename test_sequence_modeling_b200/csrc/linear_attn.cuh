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
constexpr int THREADS = 256;
constexpr int LD = D + 4;  // padded row stride: 8 rows' float4 at one column hit 8 distinct bank groups

// How the units' sequences are dealt out to segments: units below `whole` are one segment each, the others are
// cut into nseg segments of seg_len tokens (whole chunks of every kernel).  Segment k of the grid:
struct Cut {
  int whole, nseg, seg_len;
  __host__ __device__ int segments(int units) const { return whole + (units - whole) * nseg; }
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
  int first_segment, segments;  // this launch's
};

template <bool REVERSE>
__device__ __forceinline__ Segment segment_of(const Params &p, int k) {
  Segment g;
  const int rest = k - p.cut.whole;
  const bool cut = rest >= 0;
  const int q = cut ? rest / p.cut.nseg : 0, seg = cut ? rest - q * p.cut.nseg : 0;
  const int n = cut ? p.cut.nseg : 1, len = cut ? p.cut.seg_len : p.T;
  g.unit = cut ? p.cut.whole + q : k;
  g.t_lo = seg * len;
  g.rows = min(len, p.T - g.t_lo);
  g.last = REVERSE ? seg == 0 : seg == n - 1;
  g.slot = cut ? rest : -1;
  return g;
}
// The state a segment starts from (NULL: zero).
__device__ __forceinline__ const float *start_state(const Params &p, const Segment &g) {
  if (p.slots_out) return nullptr;
  if (g.slot >= 0) return p.slots + (long long)g.slot * (D * D);
  return p.C0 ? p.C0 + (long long)g.unit * (D * D) : nullptr;
}
// Where the state it ends in goes (NULL: nowhere).
__device__ __forceinline__ float *end_state(const Params &p, const Segment &g) {
  if (p.slots_out) return g.last ? nullptr : p.slots_out + (long long)g.slot * (D * D);
  return p.C_out && g.last ? p.C_out + (long long)g.unit * (D * D) : nullptr;
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

constexpr size_t SMEM_BYTES = sizeof(float) * (size_t)(5 * CHUNK * LD + 2 * CHUNK + 4);

// One CTA takes one segment of one unit.  Each of the 64 x 64 x 64 products is a 4 x 4
// register tile of each of 16 x 16 threads, in fp32 fused multiply-adds.
template <typename InT, bool REVERSE>
__global__ void __launch_bounds__(THREADS) attn_kernel(const Params p) {
  extern __shared__ __align__(16) float sm[];
  float *Xs = sm;                // [CHUNK][LD]
  float *Ys = Xs + CHUNK * LD;
  float *Ws = Ys + CHUNK * LD;
  float *Ms = Ws + CHUNK * LD;   // the masked, decayed products x_t . y_s
  float *Cs = Ms + CHUNK * LD;   // the carried state
  float *pw = Cs + D * LD;       // gamma^0 .. gamma^CHUNK
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const Segment sg = segment_of<REVERSE>(p, p.first_segment + blockIdx.x);
  const bool state_only = p.slots_out != nullptr;
  if (state_only && sg.last) return;
  const float g = p.log_decay[sg.unit % p.H];
  const int len = sequence_length(p.lengths, sg.unit / p.H, p.T);
  const int n_seg = min(max(len - sg.t_lo, 0), sg.rows);  // its tokens
  const long long row0 = (long long)sg.unit * p.T + sg.t_lo;
  const InT *X = static_cast<const InT *>(p.X) + row0 * D;
  const InT *Y = static_cast<const InT *>(p.Y) + row0 * D;
  const InT *W = static_cast<const InT *>(p.W) + row0 * D;
  InT *out = state_only ? nullptr : static_cast<InT *>(p.out) + row0 * D;

  // The state at the start of the pass: this thread's rows ty + 16 i, columns 4 tx .. 4 tx + 3.
  const float *C0 = start_state(p, sg);
  float C[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = ty + 16 * i, col = 4 * tx + j;
      C[i][j] = C0 ? (p.transposed ? C0[col * D + r] : C0[r * D + col]) : 0.f;
      Cs[r * LD + col] = C[i][j];
    }
  }
  if (tid <= CHUNK) pw[tid] = decay_pow(g, tid);

  const int nchunks = (n_seg + CHUNK - 1) / CHUNK;
  for (int ci = 0; ci < nchunks; ++ci) {
    const int c0 = (REVERSE ? nchunks - 1 - ci : ci) * CHUNK;
    const int n = min(CHUNK, n_seg - c0);
    // Tiles: 16 lanes a row of 64 values, rows past the end as zeros.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 16 * i;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x, w = x;
      if (r < n) {
        const long long at = (long long)(c0 + r) * D + 4 * tx;
        if (out) x = load4(X + at);
        y = load4(Y + at);
        w = load4(W + at);
      }
      *reinterpret_cast<float4 *>(Xs + r * LD + 4 * tx) = x;
      *reinterpret_cast<float4 *>(Ys + r * LD + 4 * tx) = y;
      *reinterpret_cast<float4 *>(Ws + r * LD + 4 * tx) = w;
    }
    __syncthreads();
    if (out) {
      // m_ts x_t . y_s for rows t = ty + 16 i, columns s = tx + 16 j.
      float acc[4][4] = {};
      for (int k = 0; k < D; k += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = *reinterpret_cast<const float4 *>(Xs + (ty + 16 * i) * LD + k);
          y[i] = *reinterpret_cast<const float4 *>(Ys + (tx + 16 * i) * LD + k);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, acc[i][j]))));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = ty + 16 * i, s = tx + 16 * j;
          const int gap = REVERSE ? s - t : t - s;
          Ms[t * LD + s] = gap >= 0 ? acc[i][j] * pw[gap] : 0.f;
        }
      __syncthreads();
      // out rows t = ty + 16 i, columns 4 tx ..: the state's part, then the chunk's own.
      float o[4][4] = {};
      for (int k = 0; k < D; k += 4) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(Xs + (ty + 16 * i) * LD + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const float4 c = *reinterpret_cast<const float4 *>(Cs + (k + kk) * LD + 4 * tx);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float xv = kk == 0 ? x[i].x : kk == 1 ? x[i].y : kk == 2 ? x[i].z : x[i].w;
            o[i][0] = fmaf(xv, c.x, o[i][0]);
            o[i][1] = fmaf(xv, c.y, o[i][1]);
            o[i][2] = fmaf(xv, c.z, o[i][2]);
            o[i][3] = fmaf(xv, c.w, o[i][3]);
          }
        }
      }
      float in[4][4] = {};
      for (int s = 0; s < n; s += 4) {
        float4 m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = *reinterpret_cast<const float4 *>(Ms + (ty + 16 * i) * LD + s);
#pragma unroll
        for (int ss = 0; ss < 4; ++ss) {
          const float4 w = *reinterpret_cast<const float4 *>(Ws + (s + ss) * LD + 4 * tx);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float mv = ss == 0 ? m[i].x : ss == 1 ? m[i].y : ss == 2 ? m[i].z : m[i].w;
            in[i][0] = fmaf(mv, w.x, in[i][0]);
            in[i][1] = fmaf(mv, w.y, in[i][1]);
            in[i][2] = fmaf(mv, w.z, in[i][2]);
            in[i][3] = fmaf(mv, w.w, in[i][3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = ty + 16 * i;
        if (t < n) {
          const float f = p.c * pw[REVERSE ? n - 1 - t : t + 1];
          store_out(out + (long long)(c0 + t) * D + 4 * tx,
                    make_float4(fmaf(f, o[i][0], p.a * in[i][0]), fmaf(f, o[i][1], p.a * in[i][1]),
                                fmaf(f, o[i][2], p.a * in[i][2]), fmaf(f, o[i][3], p.a * in[i][3])));
        }
      }
    }
    // C <- gamma^n C + e sum_s h_s y_s^T w_s for rows 4 ty .., columns 4 tx .. of the sum; the
    // state's rows of this thread are ty + 16 i, so the products are taken there.
    float acc[4][4] = {};
    for (int s = 0; s < n; ++s) {
      const float h = pw[REVERSE ? s + 1 : n - 1 - s];
      const float4 w = *reinterpret_cast<const float4 *>(Ws + s * LD + 4 * tx);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = h * Ys[s * LD + ty + 16 * i];
        acc[i][0] = fmaf(y, w.x, acc[i][0]);
        acc[i][1] = fmaf(y, w.y, acc[i][1]);
        acc[i][2] = fmaf(y, w.z, acc[i][2]);
        acc[i][3] = fmaf(y, w.w, acc[i][3]);
      }
    }
    __syncthreads();  // every read of the state and of the tiles is done
    const float dn = pw[n];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) C[i][j] = fmaf(dn, C[i][j], p.e * acc[i][j]);
      *reinterpret_cast<float4 *>(Cs + (ty + 16 * i) * LD + 4 * tx) = make_float4(C[i][0], C[i][1], C[i][2], C[i][3]);
    }
  }
  // Rows behind the end.
  if (out) {
    for (int r = n_seg + ty; r < sg.rows; r += 16) store_out(out + (long long)r * D + 4 * tx, make_float4(0.f, 0.f, 0.f, 0.f));
  }
  if (float *Co = end_state(p, sg)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4 *>(Co + (ty + 16 * i) * D + 4 * tx) = make_float4(C[i][0], C[i][1], C[i][2], C[i][3]);
  }
}

// The states at the segments' starts of the cut units, in place: slot i of a unit holds the state that
// its segment alone leaves (M_i) and gets the state that it starts from,
//   C_0 = C0,  C_{i+1} = gamma^(n_i) C_i + M_i     (reverse: from the last segment down).
// Reads and writes nseg x 16 KB a unit once: bound by memory, and small beside the tokens.
struct ScanParams {
  float *slots;  // [cut units][nseg][D][D]
  const float *C0;
  const float *log_decay;
  const int *lengths;
  int H, T;
  Cut cut;
};

constexpr int SCAN_THREADS = 256;  // 4 values a thread: 4 CTAs a unit

template <bool REVERSE>
__global__ void __launch_bounds__(SCAN_THREADS) scan_kernel(const ScanParams p) {
  const int q = blockIdx.x >> 2, unit = p.cut.whole + q;
  const int at = ((blockIdx.x & 3) * SCAN_THREADS + threadIdx.x) * 4;
  const float g = p.log_decay[unit % p.H];
  const int len = sequence_length(p.lengths, unit / p.H, p.T);
  float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.C0) c = *reinterpret_cast<const float4 *>(p.C0 + (long long)unit * (D * D) + at);
  float *slots = p.slots + (long long)q * p.cut.nseg * (D * D) + at;
  auto slot = [&](int k) {
    return reinterpret_cast<float4 *>(slots + (long long)(REVERSE ? p.cut.nseg - 1 - k : k) * (D * D));
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
        const int t_lo = (REVERSE ? p.cut.nseg - 1 - k : k) * p.cut.seg_len;
        const float dn = decay_pow(g, min(max(len - t_lo, 0), min(p.cut.seg_len, p.T - t_lo)));
        c = make_float4(fmaf(dn, c.x, m[j].x), fmaf(dn, c.y, m[j].y), fmaf(dn, c.z, m[j].z), fmaf(dn, c.w, m[j].w));
      }
    }
  }
}

// One token of every unit: S <- gamma S + k^T v, z = scale q S, with q and k turned by the
// token's position first when a rotary plan is given.  One CTA a unit: each thread takes four
// float4 of the state (rows ty + 16 i, columns 4 tx ..), all loaded before anything waits.
// 32 KB of state move a unit against 16 KFLOP: bound by memory.
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
__global__ void __launch_bounds__(THREADS) decode_kernel(const DecodeParams p) {
  __shared__ float qk[2][D];
  __shared__ __align__(16) float part[THREADS / 32][D];
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
    for (int w = 0; w < THREADS / 32; ++w) {
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
