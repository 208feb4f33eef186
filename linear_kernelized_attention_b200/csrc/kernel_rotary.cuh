// kernel_rotary.cuh - rotary positions of q and k, in one launch.
//
// What it computes. Columns 0 .. rot-1 of a head are rot/2 pairs, (2i, 2i+1) interleaved or
// (i, i + rot/2) in halves; pair i of a token at position t turns by the angle t freq[i]:
//   (x1, x2) -> scale rot_scale (x1 cos - x2 sin, x1 sin + x2 cos); other columns are scaled by
//   `scale`. inverse turns the other way, which is the transposed map: the gradient.
// The angle is reduced in double (t freq / pi, less the nearest even integer) before sin and cos of
// an fp32 argument in [-1, 1] half turns: fp32 products of far positions lose the angle itself.
//
// Reading and writing q and k bounds it at best. One thread computes the sines of V pairs of one token once
// and applies them to every head of its head group (q's heads, then k's), one after another: outputs may be the
// inputs, so a head's loads stay behind the stores of the head before, and what is in flight comes from the number of
// threads (its 55 registers hold one head's vectors, and of 14 warps a cycle issued 8 wait on loads). Heads
// are split into groups only where there are too few tokens to fill the GPU. Measured: 4 x 4096
// tokens of 8 + 8 heads of 64 columns in 13.7 us, 4900 GB/s (75% of a plain copy); twice as many groups, each
// with the sines again, 15.9 us, and sines shared through shared memory 17.9 us.
#pragma once
#include "kernels_decay.cuh"

namespace favor {
namespace rot {

using dcy::View;

constexpr int kThreads = 128;

struct Params {
  View q, k, qy, ky;
  const double* freq;  // [rot / 2], radians per position
  const int* pos;      // [B, L] or null
  long long first;     // position of token 0 where pos is null
  float scale, rot_scale;
  int B, Hq, Hk, L, d, rot, inverse;
  int groups, per_group;  // head groups, heads per group
  int npair, npass;       // vectors of pairs and of unrotated columns per token
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T x[V];
};

// V: pairs per thread in halves layout; 2 V consecutive columns in interleaved layout.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) k_rotary(const Params p) {
  const int items = p.npair + p.npass;
  const long long tokens = (long long)p.B * p.L;
  const long long total = tokens * items;
  const int h0 = blockIdx.y * p.per_group, h1 = min(p.Hq + p.Hk, h0 + p.per_group);
  for (long long w = (long long)blockIdx.x * kThreads + threadIdx.x; w < total;
       w += (long long)gridDim.x * kThreads) {
    const int it = (int)(w % items);
    const long long tok = w / items;
    const int b = (int)(tok / p.L), t = (int)(tok % p.L);
    const bool pass = it >= p.npair;
    const int half = p.rot / 2;
    int c1, c2;  // the two vectors' first columns (one vector, twice, for unrotated columns)
    float cs[V], sn[V];
    if (pass) {
      c1 = c2 = p.rot + (it - p.npair) * V;
    } else {
      const int i0 = it * V;
      c1 = INTER ? 2 * i0 : i0;
      c2 = INTER ? c1 + V : i0 + half;
      const double ps = (double)(p.pos ? (long long)p.pos[tok] : p.first + t);
      const float sc = p.scale * p.rot_scale;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const double x = ps * (p.freq[i0 + e] * 0.31830988618379067154);  // half turns
        const float r = (float)(x - 2.0 * rint(0.5 * x));
        float s, c;
        sincospif(r, &s, &c);
        cs[e] = sc * c;
        sn[e] = p.inverse ? -sc * s : sc * s;
      }
    }
#pragma unroll 8
    for (int h = h0; h < h1; ++h) {
      const bool isq = h < p.Hq;
      const int hh = isq ? h : h - p.Hq;
      const View& vi = isq ? p.q : p.k;
      const View& vo = isq ? p.qy : p.ky;
      const T* x = static_cast<const T*>(vi.p) + b * vi.sb + hh * vi.sh + t * vi.st;
      T* y = static_cast<T*>(vo.p) + b * vo.sb + hh * vo.sh + t * vo.st;
      const Vec<T, V> a = *reinterpret_cast<const Vec<T, V>*>(x + c1);
      Vec<T, V> ya, yb;
      if (pass) {
#pragma unroll
        for (int e = 0; e < V; ++e) dcy::from_f(ya.x[e], dcy::to_f(a.x[e]) * p.scale);
        *reinterpret_cast<Vec<T, V>*>(y + c1) = ya;
      } else {
        const Vec<T, V> c = *reinterpret_cast<const Vec<T, V>*>(x + c2);
        if (INTER) {
          T in[2 * V], ou[2 * V];
#pragma unroll
          for (int e = 0; e < V; ++e) in[e] = a.x[e], in[V + e] = c.x[e];
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float x1 = dcy::to_f(in[2 * e]), x2 = dcy::to_f(in[2 * e + 1]);
            dcy::from_f(ou[2 * e], x1 * cs[e] - x2 * sn[e]);
            dcy::from_f(ou[2 * e + 1], x1 * sn[e] + x2 * cs[e]);
          }
#pragma unroll
          for (int e = 0; e < V; ++e) ya.x[e] = ou[e], yb.x[e] = ou[V + e];
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float x1 = dcy::to_f(a.x[e]), x2 = dcy::to_f(c.x[e]);
            dcy::from_f(ya.x[e], x1 * cs[e] - x2 * sn[e]);
            dcy::from_f(yb.x[e], x1 * sn[e] + x2 * cs[e]);
          }
        }
        *reinterpret_cast<Vec<T, V>*>(y + c1) = ya;
        *reinterpret_cast<Vec<T, V>*>(y + c2) = yb;
      }
    }
  }
}

}  // namespace rot
}  // namespace favor
