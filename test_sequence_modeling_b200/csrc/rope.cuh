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
// 0.06 rad), so the product and its reduction to one turn are in fp64 and only the reduced angle
// goes through sincosf, its rounding carried to first order.  A token's 32 angles serve all its
// heads of Q and K: a CTA makes them once for a tile of tokens.  Bound by memory: each row is read
// and written once.
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
  const double a = (double)position * (double)inv_freq;
  const double turns = rint(a * 0.15915494309189535);          // 1 / (2 pi)
  double r = fma(turns, -6.283185307179586, a);                // 2 pi, high part
  r = fma(turns, -2.4492935982947064e-16, r);                  // and the rest of it
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
constexpr int TILE = 16;  // tokens of a CTA

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
  int head_groups;       // CTAs that share a tile's heads
};

enum { PAIRED = 0, INTERLEAVED = 1, ANY = 2 };

template <typename InT>
struct Vec {
  static constexpr int N = 16 / sizeof(InT);
  uint4 raw;
  __device__ __forceinline__ void load(const InT *p) { raw = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void store(InT *p) const { *reinterpret_cast<uint4 *>(p) = raw; }
  __device__ __forceinline__ void get(float (&f)[N]) const;
  __device__ __forceinline__ void set(const float (&f)[N]);
};
template <>
__device__ __forceinline__ void Vec<float>::get(float (&f)[4]) const {
  f[0] = __uint_as_float(raw.x);
  f[1] = __uint_as_float(raw.y);
  f[2] = __uint_as_float(raw.z);
  f[3] = __uint_as_float(raw.w);
}
template <>
__device__ __forceinline__ void Vec<float>::set(const float (&f)[4]) {
  raw = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ void Vec<__nv_bfloat16>::get(float (&f)[8]) const {
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void Vec<__nv_bfloat16>::set(const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  raw = make_uint4(u[0], u[1], u[2], u[3]);
}

// A thread takes two 16-byte pieces of a row: PAIRED (half layout, rotary / 2 whole pieces): a
// piece and its partner; INTERLEAVED: two neighbours, whose pairs are inside; ANY (half layout
// with a pair's values at unlike places of their pieces): two neighbours, partners read singly.
template <typename InT, int MODE>
__global__ void __launch_bounds__(THREADS) rope_kernel(const Params p) {
  constexpr int N = Vec<InT>::N;
  constexpr int ITEMS = D / N / 2;  // threads a row
  __shared__ float2 table[TILE][D / 2];
  const int tid = threadIdx.x;
  const long long tile0 = (long long)(blockIdx.x / p.head_groups) * TILE;
  const int group = blockIdx.x % p.head_groups;
  const int ntok = (int)min((long long)TILE, p.tokens - tile0);
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

  const int item = tid % ITEMS;
  const int heads = p.t[0].heads + p.t[1].heads;
  const int rows = ntok * heads;
  constexpr int ROWS = THREADS / ITEMS;  // rows a step
  const int hv = half / N;
  int a, b;
  bool turn = true;
  if (MODE == PAIRED) {
    turn = item < hv;
    a = turn ? item : 2 * hv + 2 * (item - hv);
    b = turn ? item + hv : a + 1;
  } else {
    a = 2 * item;
    b = a + 1;
  }
  for (int r = group * ROWS + tid / ITEMS; r < rows; r += ROWS * p.head_groups) {
    const int h = r / ntok, tok = r - h * ntok;
    const long long at = tile0 + tok;
    const long long bi = at / p.T, t = at - bi * p.T;
    const int which = h >= p.t[0].heads;
    const Tensor &T = p.t[which];
    const int head = which ? h - p.t[0].heads : h;
    const InT *x = static_cast<const InT *>(T.x) + bi * T.sb + head * T.sh + t * T.st;
    InT *y = static_cast<InT *>(T.y) + ((bi * T.heads + head) * p.T + t) * D;
    Vec<InT> va, vb;
    va.load(x + a * N);
    vb.load(x + b * N);
    if (MODE == PAIRED) {
      if (turn) {
        float fa[N], fb[N];
        va.get(fa);
        vb.get(fb);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float2 cs = table[tok][a * N + i];
          const float u = fa[i], w = fb[i];
          fa[i] = fmaf(u, cs.x, -w * cs.y);
          fb[i] = fmaf(w, cs.x, u * cs.y);
        }
        va.set(fa);
        vb.set(fb);
      }
    } else {
#pragma unroll
      for (int which_vec = 0; which_vec < 2; ++which_vec) {
        Vec<InT> &v = which_vec ? vb : va;
        const int j0 = (which_vec ? b : a) * N;
        if (j0 < p.plan.rotary) {
          float f[N];
          v.get(f);
          if (MODE == INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
              if (j0 + i < p.plan.rotary) {
                const float2 cs = table[tok][(j0 + i) >> 1];
                const float u = f[i], w = f[i + 1];
                f[i] = fmaf(u, cs.x, -w * cs.y);
                f[i + 1] = fmaf(w, cs.x, u * cs.y);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const int j = j0 + i;
              if (j < p.plan.rotary) {
                const bool upper = j >= half;
                const float2 cs = table[tok][upper ? j - half : j];
                const float w = simt::load_in(x, upper ? j - half : j + half);
                f[i] = fmaf(f[i], cs.x, upper ? w * cs.y : -w * cs.y);
              }
            }
          }
          v.set(f);
        }
      }
    }
    va.store(y + a * N);
    vb.store(y + b * N);
  }
}

}  // namespace rope
}  // namespace ttt
