// rope.cuh - rotary positions: pairs of a row's leading `rotary` values turned by position x
// frequency, and the rows brought from any strided layout (a joint projection's [B][T][H][D])
// into the dense [B][H][T][D] that the layer's entry points take.
//
// Pair i of a token at position p, values (a, b), angle = p inv_freq[i]:
//   (a, b) -> mscale (a cos - b sin, a sin + b cos)         inverse: the angle's sign turned
// half layout: the pair is (i, i + rotary / 2); interleaved: (2 i, 2 i + 1).  The inverse with the
// same mscale is the transpose, so it is the gradient's way back.
//
// The angle of a far position loses its digits in fp32 (at position 10^6 a step of the product is
// 0.06 rad), so the product and its reduction to one turn are in fp64, the product's own rounding
// (from position 2^29 on) carried beside it, and only the reduced angle goes through sincosf, its
// rounding carried to first order.  A token's 32 angles serve all its heads of Q and K: a CTA makes
// them once for a tile of tokens.  Bound by memory: each row is read and written once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "simt.cuh"

namespace ttt {
namespace rope {

using simt::D;

struct Plan {
  const float *inv_freq;  // [rotary / 2]
  int rotary;             // values of a row that turn (even, <= D)
  bool interleaved;
  float mscale;
};

// (cos, sin) of position x frequency, times mscale.
__device__ __forceinline__ float2 cos_sin(int position, float inv_freq, float mscale) {
  const double p = position, f = inv_freq, a = p * f;
  const double beyond = fma(p, f, -a);                         // what a's rounding left out (31 x 24 bits), exact
  const double turns = rint(a * 0.15915494309189535);          // 1 / (2 pi)
  double r = fma(turns, -6.283185307179586, a);                // 2 pi, high part
  r = fma(turns, -2.4492935982947064e-16, r + beyond);         // and the rest of it
  const float x = (float)r, rest = (float)(r - (double)x);
  float s, c;
  sincosf(x, &s, &c);
  return make_float2(mscale * fmaf(-rest, s, c), mscale * fmaf(rest, c, s));
}

// The other value of the pair that holds value j < rotary: its pair, and the sign of sin in
// y_j = x_j cos + sign x_partner sin.
__device__ __forceinline__ int partner_of(const Plan &plan, int j, int &pair, int &sign) {
  if (plan.interleaved) {
    pair = j >> 1;
    sign = (j & 1) ? 1 : -1;
    return j ^ 1;
  }
  const int half = plan.rotary >> 1;
  const bool upper = j >= half;
  pair = upper ? j - half : j;
  sign = upper ? 1 : -1;
  return upper ? j - half : j + half;
}

constexpr int THREADS = 256;
constexpr int MOST_TILE = 16;  // tokens of a CTA at most

struct Tensor {
  const void *x;
  long long sb, sh, st;  // strides of batch, head and token in values
  void *y;               // [B][heads][T][D]
  int heads;
};

struct Params {
  Tensor t[2];           // Q and K (heads = 0: none)
  Plan plan;
  const int *positions;  // [B][T], or NULL: first + t
  int first;
  float sin_sign;        // -1: inverse
  int T;
  long long tokens;      // B T
  int tile;              // tokens of a CTA: a power of two up to MOST_TILE
  int head_groups;       // CTAs that share a tile's heads
};

// V neighbouring values of a row, moved as one.
template <typename InT, int V>
struct Piece;
template <int V>
struct alignas(4 * V) Piece<float, V> {
  float v[V];
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = v[i];
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = f[i];
  }
};
template <int V>
struct alignas(2 * V) Piece<__nv_bfloat16, V> {  // in words of two
  uint32_t w[V / 2];
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
};
template <>
struct Piece<__nv_bfloat16, 1> {
  __nv_bfloat16 v;
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(v); }
  __device__ __forceinline__ void set(const float (&f)[1]) { v = __float2bfloat16_rn(f[0]); }
};

// A thread takes two pieces of V values of a row.  Half layout: a piece and its partner, V the most
// values up to 16 bytes that rotary / 2 is a multiple of (a narrower piece costs more instructions:
// bf16, B16 H32 T2048: 87 us at V = 8, 6.2 TB/s, 94 % of the measured copy; 92 us at V = 4, rotary 40).
// Interleaved: two neighbouring pieces of 16 bytes, whose pairs are inside.
template <typename InT, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rope_kernel(const Params p) {
  constexpr int ITEMS = D / V / 2;       // threads a row
  constexpr int ROWS = THREADS / ITEMS;  // rows a step
  __shared__ float2 table[MOST_TILE][D / 2];
  const int tid = threadIdx.x;
  const long long tile0 = (long long)(blockIdx.x / p.head_groups) * p.tile;
  const int group = blockIdx.x % p.head_groups;
  const int ntok = (int)min((long long)p.tile, p.tokens - tile0);
  const int half = p.plan.rotary >> 1;
  for (int x = tid; x < ntok * half; x += THREADS) {
    const int tok = x / half, i = x - tok * half;
    const long long at = tile0 + tok;
    const int pos = p.positions ? p.positions[at] : p.first + (int)(at % p.T);
    float2 cs = cos_sin(pos, p.plan.inv_freq[i], p.plan.mscale);
    cs.y *= p.sin_sign;
    table[tok][i] = cs;
  }
  __syncthreads();

  const int item = tid % ITEMS, r = tid / ITEMS, tok = r & (p.tile - 1);
  if (tok >= ntok) return;
  const long long at = tile0 + tok, bi = at / p.T, t = at - bi * p.T;
  const int hv = half / V;
  const bool turn = INTERLEAVED || item < hv;
  const int a = INTERLEAVED ? 2 * item : turn ? item : 2 * hv + 2 * (item - hv);
  const int b = !INTERLEAVED && turn ? item + hv : a + 1;
  // The turn of this thread's V pairs: a V + i, or, interleaved, those inside the two pieces.
  float2 cs[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int pair = INTERLEAVED ? a * (V / 2) + i : a * V + i;
    cs[i] = turn && pair < half ? table[tok][pair] : make_float2(1.f, 0.f);
  }
  using P = Piece<InT, V>;
  auto turned = [&](P &va, P &vb) {
    if (!turn) return;
    float fa[V], fb[V];
    va.get(fa);
    vb.get(fb);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (INTERLEAVED) {
        constexpr int H = V / 2;
        if (a * H + i < half) {
          float &u = i < H ? fa[2 * (i % H)] : fb[2 * (i % H)], &w = i < H ? fa[2 * (i % H) + 1] : fb[2 * (i % H) + 1];
          const float x = u, y = w;
          u = fmaf(x, cs[i].x, -y * cs[i].y);
          w = fmaf(y, cs[i].x, x * cs[i].y);
        }
      } else {
        const float x = fa[i], y = fb[i];
        fa[i] = fmaf(x, cs[i].x, -y * cs[i].y);
        fb[i] = fmaf(y, cs[i].x, x * cs[i].y);
      }
    }
    va.set(fa);
    vb.set(fb);
  };
  // This thread's heads, of Q and then of K: four at a time, whose loads do not wait for one another.
  const int step = ROWS / p.tile * p.head_groups, h0 = group * (ROWS / p.tile) + r / p.tile;
  constexpr int BATCH = 4;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const Tensor &T = p.t[which];
    const InT *x = static_cast<const InT *>(T.x) + bi * T.sb + t * T.st;
    InT *y = static_cast<InT *>(T.y) + (bi * T.heads * p.T + t) * D;
    const long long y_head = (long long)p.T * D;
    for (int h = h0; h < T.heads; h += BATCH * step) {
      P va[BATCH], vb[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int hh = h + k * step;
        if (hh < T.heads) {
          va[k] = *reinterpret_cast<const P *>(x + hh * T.sh + a * V);
          vb[k] = *reinterpret_cast<const P *>(x + hh * T.sh + b * V);
        }
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int hh = h + k * step;
        if (hh < T.heads) {
          turned(va[k], vb[k]);
          *reinterpret_cast<P *>(y + hh * y_head + a * V) = va[k];
          *reinterpret_cast<P *>(y + hh * y_head + b * V) = vb[k];
        }
      }
    }
  }
}

}  // namespace rope
}  // namespace ttt
