// kernels_decay.cuh - causal linear attention with one decay per head, and its gradients, on CUDA
// cores in fp32: every type, head size and stride the entry points take.
//
// What it computes. With lambda = exp(log_decay[h]) and, for every (batch, head),
//   S_t = lambda S_{t-1} + k_t v_t^T,   out_t = S_t^T q_t          (S_{-1} = state_in or 0)
//   G_t = lambda G_{t+1} + q_t dout_t^T (beyond the last token: dstate_out or 0, undecayed)
//   dq_t = S_t dout_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,  dstate_in = lambda G_0.
// All four products have one form, a scan job (a, b, c, direction):
//   y_i = sum_j lambda^|i-j| (a_i . b_j) c_j + (boundary state), j <= i (forward) or j >= i (reverse):
//   out = (q, k, v, forward), dq = (dout, v, k, forward), dk = (v, dout, q, reverse),
//   dv = (k, q, dout, reverse).
//
// Blocking. Tokens in chunks of kChunk; X is the state a chunk is handed, the sum of its direction's
// earlier tokens. In a chunk of n tokens, row r sees it as lambda^(r+1) a_r X (forward) or
// lambda^(n-1-r) a_r X (reverse), and it is handed on as
//   forward: X' = lambda^n X + sum_r lambda^(n-1-r) b_r c_r^T   (first X: state_in; last X': state_out)
//   reverse: X' = lambda^n X + sum_r lambda^(r+1) b_r c_r^T     (first X: dstate_out; last X': dstate_in)
// so no exponent is negative and lambda = 0 needs no division.
// Three launches: chunk updates (every chunk at once), the scan over chunks (one thread per state
// element, in double), the outputs (every chunk at once). Powers of lambda are evaluated in double:
// the library is built with fast single-precision intrinsics.
//
// A product whose weight the mask removes is never formed (it is skipped, not multiplied by zero),
// so infinities and NaN in later tokens do not reach earlier rows. Tokens at and past the sequence's
// length are read as zero and their rows are not written.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace favor {
namespace dcy {

constexpr int kChunk = 64;
constexpr int kThreads = 256;
constexpr int kMaxD = 128;

// A [B, H, L, d] operand: element strides of the three outer dimensions, d contiguous.
struct View {
  void* p;
  long long sb, sh, st;
};

// One state (forward: state_in -> state_out; reverse: dstate_out -> dstate_in), [B*H, d, d] fp32.
struct StateJob {
  View b, c;
  const float* in;  // may be null (zeros)
  float* out;       // may be null (not wanted)
  int reverse;
};

// One output: y from a, b, c and state job `state` (transposed: X is read as its transpose).
struct OutJob {
  View a, b, c, y;
  int state, trans, reverse;
};

struct Params {
  StateJob s[2];
  OutJob o[3];
  const float* log_decay;  // [H]
  const int* lengths;      // [B] or null
  float* ws;               // [states][BH][nch][d * d]
  int nstates, nouts, B, H, L, d, nch;
};

struct ScanParams {
  const float* in[2];  // may be null (zeros)
  float* out[2];       // may be null (not wanted)
  int reverse[2];
  float* ws;           // [states][BH][nseg][d * d]
  const float* log_decay;
  const int* lengths;
  int nstates, B, H, L, d, nseg, seg;  // segments, tokens in each
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// lambda^n for n >= 0 (lambda^0 = 1 for every lambda, 0 among them).
__device__ __forceinline__ double decay_pow(float g, long long n) {
  return n == 0 ? 1.0 : exp(static_cast<double>(g) * static_cast<double>(n));
}

// Tokens of sequence b: lengths[b] held to [0, L], or L.
__device__ __forceinline__ int seq_len(const int* lengths, int b, int L) {
  return lengths ? max(0, min(lengths[b], L)) : L;
}

// Rows row0 .. row0 + 63 of one head into dst[64][DP] as fp32; zero past n rows and d columns.
template <typename T, int DP>
__device__ __forceinline__ void load_tile(float* dst, const View& x, int b, int h, int row0, int n, int d) {
  const T* src = static_cast<const T*>(x.p) + b * x.sb + h * x.sh + (long long)row0 * x.st;
  for (int i = threadIdx.x; i < kChunk * DP; i += kThreads) {
    const int r = i / DP, m = i % DP;
    dst[i] = r < n && m < d ? to_f(src[r * x.st + m]) : 0.f;
  }
}

// ws[state][bh][chunk][m][n] = sum_r w_r b_r[m] c_r[n]. Grid: states x BH x chunks, chunk fastest.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) k_chunk_update(const Params p) {
  extern __shared__ float sm[];
  pdl_launch_dependents();
  float* sb = sm;                 // [kChunk][DP], rows scaled by w_r
  float* sc = sm + kChunk * DP;   // [kChunk][DP]
  const int ch = blockIdx.x % p.nch, q = blockIdx.x / p.nch;
  const int bh = q % (p.B * p.H), js = q / (p.B * p.H);
  const int b = bh / p.H, h = bh % p.H;
  const StateJob& job = p.s[js];
  const int len = seq_len(p.lengths, b, p.L);
  const int row0 = ch * kChunk, n = min(kChunk, len - row0);
  if (n <= 0) return;
  load_tile<T, DP>(sb, job.b, b, h, row0, n, p.d);
  load_tile<T, DP>(sc, job.c, b, h, row0, n, p.d);
  __syncthreads();
  const float g = p.log_decay[h];
  {
    const int r = threadIdx.x >> 2;  // four threads scale one row
    if (r < n) {
      const float w = (float)decay_pow(g, job.reverse ? r + 1 : n - 1 - r);
      for (int m = threadIdx.x & 3; m < DP; m += 4) sb[r * DP + m] *= w;
    }
  }
  __syncthreads();
  constexpr int R = DP / 16;
  const int m0 = (threadIdx.x >> 4) * R, n0 = (threadIdx.x & 15) * R;
  float acc[R][R];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < R; ++j) acc[i][j] = 0.f;
  for (int r = 0; r < n; ++r) {
    float x[R], y[R];
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = sb[r * DP + m0 + i], y[i] = sc[r * DP + n0 + i];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
  }
  float* out = p.ws + ((long long)q * p.nch + ch) * p.d * p.d;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (m0 + i < p.d && n0 + j < p.d) out[(m0 + i) * p.d + n0 + j] = acc[i][j];
}

// Each segment's update (p.seg tokens; a chunk is one) replaced by the state it is handed; the
// boundary states read and written. One thread per (state job, head, element); the running state is
// held in double. Eight segments' loads are in flight at a time: the chain itself is one fma a segment.
static __global__ void __launch_bounds__(kThreads) k_chunk_scan(const __grid_constant__ ScanParams p) {
  constexpr int G = 8;
  __shared__ double pw[2];  // lambda^seg, lambda^(tokens of the last segment)
  const int dd = p.d * p.d, nb = (dd + kThreads - 1) / kThreads;
  const int q = blockIdx.x / nb, el = (blockIdx.x % nb) * kThreads + threadIdx.x;
  const int bh = q % (p.B * p.H), js = q / (p.B * p.H);
  const int len = seq_len(p.lengths, bh / p.H, p.L);
  const int ns = (int)(((long long)len + p.seg - 1) / p.seg);
  if (threadIdx.x < 64 && threadIdx.x % 32 == 0 && ns > 0)
    pw[threadIdx.x / 32] = decay_pow(p.log_decay[bh % p.H], threadIdx.x ? len - (ns - 1) * p.seg : p.seg);
  pdl_launch_dependents();
  __syncthreads();
  pdl_wait();
  if (el >= dd) return;
  float* u = p.ws + (long long)q * p.nseg * dd + el;
  double x = p.in[js] ? (double)p.in[js][(long long)bh * dd + el] : 0.0;
  const int rev = p.reverse[js];
  for (int i0 = 0; i0 < ns; i0 += G) {
    float w[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (i0 + i < ns) w[i] = u[(long long)(rev ? ns - 1 - i0 - i : i0 + i) * dd];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int c = rev ? ns - 1 - i0 - i : i0 + i;
      if (i0 + i < ns) {
        u[(long long)c * dd] = (float)x;
        x = fma(x, pw[c == ns - 1], (double)w[i]);
      }
    }
  }
  if (p.out[js]) p.out[js][(long long)bh * dd + el] = (float)x;
}

// y rows of one chunk. Grid: outs x BH x chunks, chunk fastest.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) k_chunk_out(const Params p) {
  constexpr int PS = kChunk + 1;  // row stride of the weighted scores (no bank conflicts down a column)
  constexpr int AS = DP + 1;
  constexpr int XR = 32;          // state rows staged at a time
  extern __shared__ float sm[];
  float* sa = sm;                       // [kChunk][AS]
  float* sb = sa + kChunk * AS;         // [kChunk][AS], then state rows [XR][DP]
  float* sc = sb + kChunk * AS;         // [kChunk][DP]
  float* sp = sc + kChunk * DP;         // [kChunk][PS]
  float* pw = sp + kChunk * PS;         // lambda^0 .. lambda^64
  const int ch = blockIdx.x % p.nch, q = blockIdx.x / p.nch;
  const int bh = q % (p.B * p.H), jo = q / (p.B * p.H);
  const int b = bh / p.H, h = bh % p.H;
  const OutJob& job = p.o[jo];
  const int len = seq_len(p.lengths, b, p.L);
  const int row0 = ch * kChunk, n = min(kChunk, len - row0);
  pdl_wait();
  if (n <= 0) return;
  const int rev = job.reverse;
  auto load_padded = [&](float* dst, const View& x) {
    const T* src = static_cast<const T*>(x.p) + b * x.sb + h * x.sh + (long long)row0 * x.st;
    for (int i = threadIdx.x; i < kChunk * DP; i += kThreads) {
      const int r = i / DP, m = i % DP;
      dst[r * AS + m] = r < n && m < p.d ? to_f(src[r * x.st + m]) : 0.f;
    }
  };
  load_padded(sa, job.a);
  load_padded(sb, job.b);
  load_tile<T, DP>(sc, job.c, b, h, row0, n, p.d);
  if (threadIdx.x <= kChunk) pw[threadIdx.x] = (float)decay_pow(p.log_decay[h], threadIdx.x);
  __syncthreads();

  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int i0 = 4 * ty;
  {  // scores of rows 4 ty .. + 3 and columns tx, tx + 16, ...
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    for (int m = 0; m < p.d; ++m) {
      float x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = sa[(i0 + i) * AS + m], y[i] = sb[(tx + 16 * i) * AS + m];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = fmaf(x[i], y[j], s[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int gap = rev ? (tx + 16 * j) - (i0 + i) : (i0 + i) - (tx + 16 * j);
        sp[(i0 + i) * PS + tx + 16 * j] = gap >= 0 ? s[i][j] * pw[gap] : 0.f;
      }
  }
  __syncthreads();

  constexpr int R = DP / 16;
  float acc[4][R];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < R; ++j) acc[i][j] = 0.f;
  // the carried state: acc = a X
  const float* X = p.ws + (((long long)job.state * p.B * p.H + bh) * p.nch + ch) * p.d * p.d;
  float* sx = sb;
  for (int m0 = 0; m0 < p.d; m0 += XR) {
    const int nm = min(XR, p.d - m0);
    for (int i = threadIdx.x; i < XR * DP; i += kThreads) {
      int m, c;
      if (job.trans) m = i % XR, c = i / XR; else m = i / DP, c = i % DP;
      const bool ok = m < nm && c < p.d;
      sx[m * DP + c] = ok ? (job.trans ? X[c * p.d + m0 + m] : X[(m0 + m) * p.d + c]) : 0.f;
    }
    __syncthreads();
    for (int m = 0; m < nm; ++m) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = sa[(i0 + i) * AS + m0 + m];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const float y = sx[m * DP + tx + 16 * j];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = fmaf(x[i], y, acc[i][j]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i0 + i;
    const float w = r < n ? pw[rev ? n - 1 - r : r + 1] : 0.f;
#pragma unroll
    for (int j = 0; j < R; ++j) acc[i][j] *= w;
  }
  // the chunk itself: every key all four rows see, then the diagonal 4 x 4 block element by element
  const int lo = rev ? i0 + 4 : 0, hi = rev ? n : i0;
  for (int r = lo; r < hi; ++r) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = sp[(i0 + i) * PS + r];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const float y = sc[r * DP + tx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i][j] = fmaf(x[i], y, acc[i][j]);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((rev ? r >= i : r <= i) && i0 + r < n) {
        const float x = sp[(i0 + i) * PS + i0 + r];
#pragma unroll
        for (int j = 0; j < R; ++j) acc[i][j] = fmaf(x, sc[(i0 + r) * DP + tx + 16 * j], acc[i][j]);
      }
  T* y = static_cast<T*>(job.y.p) + b * job.y.sb + h * job.y.sh;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i0 + i >= n) continue;
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (tx + 16 * j < p.d) from_f(y[(long long)(row0 + i0 + i) * job.y.st + tx + 16 * j], acc[i][j]);
  }
}

constexpr int update_smem(int dp) { return 2 * kChunk * dp * 4; }
constexpr int out_smem(int dp) {
  return (2 * kChunk * (dp + 1) + kChunk * dp + kChunk * (kChunk + 1) + kChunk + 1) * 4;
}

}  // namespace dcy
}  // namespace favor
