// kernel_decay_step.cuh - one token per head of linear attention with a decay, against the carried state.
//
// What it computes, for every (batch, head), in place:  S = lambda S + k v^T,  out = S^T q,
// lambda = exp(log_decay[h]); S [d, d] fp32.
//
// The step reads and writes the state once and does five flops on each element, so HBM bounds it.
// Columns of S are independent, so a block takes W columns of one head (all d rows): a warp's loads
// are whole 16-byte pieces of consecutive columns, every thread has its rows in flight before it
// needs the token, and only the block's row groups are summed through shared memory (fixed order:
// results do not depend on timing). Few heads take narrow slices, so that more SMs share the state.
// Measured: 512 x 8 states of 64 x 64 in 25.5 us, 5350 GB/s read and written in place (82% of a plain copy);
// 8 states of one sequence in 2.8 us, which is launch and latency.
//
// lambda is carried as an fp32 pair (value and remainder): its rounding alone would grow with the
// number of steps.
#pragma once
#include "kernels_decay.cuh"

namespace favor {
namespace dcy {

struct StepParams {
  View q, k, v, y;  // token stride unused
  const float* log_decay;
  float* state;  // [B * H, d, d]
  int H, d, slices, cols;  // column slices per head, columns per slice
};

constexpr int kStepThreads = 256;

// VEC columns per thread (4 when d % 4 == 0, else 1), IT rows per thread and pass.
template <typename T, int VEC, int IT>
__global__ void __launch_bounds__(kStepThreads) k_decay_step(const StepParams p) {
  __shared__ float sq[kMaxD], sk[kMaxD], red[kStepThreads * VEC];
  const int tid = threadIdx.x, d = p.d;
  const int bh = blockIdx.x / p.slices, c0 = (blockIdx.x % p.slices) * p.cols;
  const int b = bh / p.H, h = bh % p.H;
  const int cg = p.cols / VEC;            // column groups of the slice
  const int rg = kStepThreads / cg;       // row groups
  const int my_c = c0 + (tid % cg) * VEC, my_r = tid / cg;
  const bool live = my_r < rg && my_c < d;
  float* S = p.state + (long long)bh * d * d + my_c;

  float s[IT][VEC];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int r = r0 + i * rg;
      if (live && r < d) {
        if (VEC == 4) {
          const float4 x = *reinterpret_cast<const float4*>(S + (long long)r * d);
          s[i][0] = x.x, s[i][1 % VEC] = x.y, s[i][2 % VEC] = x.z, s[i][3 % VEC] = x.w;
        } else {
          s[i][0] = S[(long long)r * d];
        }
      }
    }
  };
  load(my_r);  // in flight while the token arrives
  const T* q = static_cast<const T*>(p.q.p) + b * p.q.sb + h * p.q.sh;
  const T* k = static_cast<const T*>(p.k.p) + b * p.k.sb + h * p.k.sh;
  const T* v = static_cast<const T*>(p.v.p) + b * p.v.sb + h * p.v.sh;
  for (int i = tid; i < d; i += kStepThreads) {
    sq[i] = to_f(q[i]);
    sk[i] = to_f(k[i]);
  }
  float vv[VEC], o[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    vv[e] = live ? to_f(v[my_c + e]) : 0.f;
    o[e] = 0.f;
  }
  const double ld = decay_pow(p.log_decay[h], 1);
  const float lh = (float)ld, ll = isinf(lh) ? 0.f : (float)(ld - (double)lh);
  __syncthreads();
  for (int r0 = my_r; r0 < d; r0 += IT * rg) {
    if (r0 != my_r) load(r0);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int r = r0 + i * rg;
      if (live && r < d) {
        const float kr = sk[r], qr = sq[r];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s[i][e] = fmaf(s[i][e], lh, fmaf(s[i][e], ll, kr * vv[e]));
          o[e] = fmaf(qr, s[i][e], o[e]);
        }
        if (VEC == 4)
          *reinterpret_cast<float4*>(S + (long long)r * d) =
              make_float4(s[i][0], s[i][1 % VEC], s[i][2 % VEC], s[i][3 % VEC]);
        else
          S[(long long)r * d] = s[i][0];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) red[e * kStepThreads + tid] = o[e];
  __syncthreads();
  if (tid < p.cols && c0 + tid < d) {
    const int e = tid % VEC, c = tid / VEC;
    float t = 0.f;
    for (int r = 0; r < rg; ++r) t += red[e * kStepThreads + r * cg + c];
    T* y = static_cast<T*>(p.y.p) + b * p.y.sb + h * p.y.sh;
    from_f(y[c0 + tid], t);
  }
}

}  // namespace dcy
}  // namespace favor
