// kernels_decay.cuh - causal linear attention with one decay per head, and its gradients, on CUDA
// cores in fp32: fp32 operands, and bf16 ones whose rows are not whole 16-byte pieces.
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
// Three launches overlap through programmatic dependent launch. Measured: fp32 prompts of 2 x 8 heads x 1023
// tokens, d = 64, in 32.8 us (update 9, scan 7, outputs 20 alone), gradients of 8 heads x 777 tokens in 32.9;
// bound by fp32 FMA from shared memory at 256 to 312 blocks. Scalar shared reads took 73 us.
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
  int vec;  // fp32 rows and strides of whole 16-byte pieces
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

// Four consecutive elements as fp32, zeros past `left` of them.
__device__ __forceinline__ float4 load4(const float* p, int left, bool vec) {
  if (left <= 0) return make_float4(0.f, 0.f, 0.f, 0.f);
  if (vec) return *reinterpret_cast<const float4*>(p);
  return make_float4(p[0], left > 1 ? p[1] : 0.f, left > 2 ? p[2] : 0.f, left > 3 ? p[3] : 0.f);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p, int left, bool) {
  return make_float4(left > 0 ? to_f(p[0]) : 0.f, left > 1 ? to_f(p[1]) : 0.f, left > 2 ? to_f(p[2]) : 0.f,
                     left > 3 ? to_f(p[3]) : 0.f);
}

// A thread's pieces of 64 rows x DP columns (piece i: row i / (DP / 4), columns 4 (i % (DP / 4)) ..): all in
// flight together, then into shared memory.
template <typename T, int DP>
struct Rows {
  static constexpr int NP = kChunk * DP / 4 / kThreads;
  float4 v[NP];
  __device__ __forceinline__ void load(const View& x, int b, int h, int row0, int n, int d, bool vec) {
    const T* src = static_cast<const T*>(x.p) + b * x.sb + h * x.sh + (long long)row0 * x.st;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int i = threadIdx.x + k * kThreads, r = i / (DP / 4), m = 4 * (i % (DP / 4));
      v[k] = load4(src + (r < n ? r * x.st : 0) + m, r < n ? d - m : 0, vec);
    }
  }
  // rows `stride` floats apart; scale: a factor per row, or null
  __device__ __forceinline__ void store(float* dst, int stride, const float* scale) const {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int i = threadIdx.x + k * kThreads, r = i / (DP / 4), m = 4 * (i % (DP / 4));
      const float w = scale ? scale[r] : 1.f;
      *reinterpret_cast<float4*>(dst + r * stride + m) = make_float4(v[k].x * w, v[k].y * w, v[k].z * w, v[k].w * w);
    }
  }
};

__device__ __forceinline__ void fma4(float (&acc)[4], float x, const float4& y) {
  acc[0] = fmaf(x, y.x, acc[0]);
  acc[1] = fmaf(x, y.y, acc[1]);
  acc[2] = fmaf(x, y.z, acc[2]);
  acc[3] = fmaf(x, y.w, acc[3]);
}
__device__ __forceinline__ float dot4(const float4& x, const float4& y, float s) {
  return fmaf(x.w, y.w, fmaf(x.z, y.z, fmaf(x.y, y.y, fmaf(x.x, y.x, s))));
}
__device__ __forceinline__ float part(const float4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

// ws[state][bh][chunk][m][n] = sum_r w_r b_r[m] c_r[n]. Grid: states x BH x chunks, chunk fastest.
// A thread sums tiles of 4 x 4 elements: 16 fma on two 16-byte reads a token.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) k_chunk_update(const __grid_constant__ Params p) {
  constexpr int K = DP / 64;
  extern __shared__ float sm[];
  pdl_launch_dependents();
  float* sb = sm;                 // [kChunk][DP], rows scaled by w_r
  float* sc = sm + kChunk * DP;   // [kChunk][DP]
  float* sw = sc + kChunk * DP;   // w_r
  const int ch = blockIdx.x % p.nch, q = blockIdx.x / p.nch;
  const int bh = q % (p.B * p.H), js = q / (p.B * p.H);
  const int b = bh / p.H, h = bh % p.H;
  const StateJob& job = p.s[js];
  const int len = seq_len(p.lengths, b, p.L);
  const int row0 = ch * kChunk, n = min(kChunk, len - row0);
  if (n <= 0) return;
  Rows<T, DP> xb, xc;
  xb.load(job.b, b, h, row0, n, p.d, p.vec);
  xc.load(job.c, b, h, row0, n, p.d, p.vec);
  if (threadIdx.x < kChunk)
    sw[threadIdx.x] =
        threadIdx.x < n ? (float)decay_pow(p.log_decay[h], job.reverse ? threadIdx.x + 1 : n - 1 - threadIdx.x) : 0.f;
  __syncthreads();
  xb.store(sb, DP, sw);
  xc.store(sc, DP, nullptr);
  __syncthreads();
  const int m0 = 4 * (threadIdx.x >> 4), n0 = 4 * (threadIdx.x & 15);
  if (m0 >= p.d) return;
  float acc[K][4][K][4];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int l = 0; l < K; ++l)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[k][i][l][j] = 0.f;
#pragma unroll 4
  for (int r = 0; r < n; ++r) {
    float4 x[K], y[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k] = *reinterpret_cast<const float4*>(sb + r * DP + m0 + 64 * k);
      y[k] = *reinterpret_cast<const float4*>(sc + r * DP + n0 + 64 * k);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int l = 0; l < K; ++l) fma4(acc[k][i][l], part(x[k], i), y[l]);
  }
  float* out = p.ws + ((long long)q * p.nch + ch) * p.d * p.d;
  const bool v4 = p.d % 4 == 0;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int l = 0; l < K; ++l) {
        const int m = m0 + 64 * k + i, c = n0 + 64 * l;
        if (m < p.d && c < p.d) {
          const float* a = acc[k][i][l];
          if (v4) {
            *reinterpret_cast<float4*>(out + m * p.d + c) = make_float4(a[0], a[1], a[2], a[3]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (c + j < p.d) out[m * p.d + c + j] = a[j];
          }
        }
      }
}

// Each segment's update (p.seg tokens; a chunk is one) replaced by the state it is handed; the
// boundary states read and written. One thread per (state job, head, element); the running state is
// held in double. G segments' loads are in flight at a time: the chain itself is one fma a segment.
template <int G>
__global__ void __launch_bounds__(kThreads) k_chunk_scan(const __grid_constant__ ScanParams p) {
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

// y rows of one chunk. Grid: outs x BH x chunks, chunk fastest. A thread sums 4 rows by 4 (or twice 4)
// columns of each product, 64 fma on eight 16-byte reads; the score rows overwrite b. Operands arrive
// while the scan runs; the carried state follows it.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) k_chunk_out(const __grid_constant__ Params p) {
  constexpr int AS = DP + 4;      // row stride: 16-byte pieces, eight rows on distinct banks
  constexpr int PS = kChunk + 4;
  constexpr int K = DP / 64;
  extern __shared__ float sm[];
  float* sa = sm;                       // [kChunk][AS]
  float* sb = sa + kChunk * AS;         // [kChunk][AS], then the weighted scores [kChunk][PS]
  float* sc = sb + kChunk * AS;         // [kChunk][AS]
  float* sx = sc + kChunk * AS;         // [DP][AS], X or its transpose
  float* pw = sx + DP * AS;             // lambda^0 .. lambda^64
  float* sp = sb;
  pdl_launch_dependents();
  const int ch = blockIdx.x % p.nch, q = blockIdx.x / p.nch;
  const int bh = q % (p.B * p.H), jo = q / (p.B * p.H);
  const int b = bh / p.H, h = bh % p.H;
  const OutJob& job = p.o[jo];
  const int len = seq_len(p.lengths, b, p.L);
  const int row0 = ch * kChunk, n = min(kChunk, len - row0), d = p.d;
  if (n <= 0) {
    pdl_wait();
    return;
  }
  const int rev = job.reverse;
  {
    Rows<T, DP> xa, xb, xc;
    xa.load(job.a, b, h, row0, n, d, p.vec);
    xb.load(job.b, b, h, row0, n, d, p.vec);
    xc.load(job.c, b, h, row0, n, d, p.vec);
    if (threadIdx.x <= kChunk) pw[threadIdx.x] = (float)decay_pow(p.log_decay[h], threadIdx.x);
    xa.store(sa, AS, nullptr);
    xb.store(sb, AS, nullptr);
    xc.store(sc, AS, nullptr);
  }
  __syncthreads();

  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int i0 = 4 * ty, d4 = (d + 3) / 4 * 4;
  {  // scores of rows 4 ty .. + 3 and columns tx, tx + 16, ...
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    for (int m = 0; m < d4; m += 4) {
      float4 x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = *reinterpret_cast<const float4*>(sa + (i0 + i) * AS + m);
        y[i] = *reinterpret_cast<const float4*>(sb + (tx + 16 * i) * AS + m);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = dot4(x[i], y[j], s[i][j]);
    }
    __syncthreads();  // b is read
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int gap = rev ? (tx + 16 * j) - (i0 + i) : (i0 + i) - (tx + 16 * j);
        sp[(i0 + i) * PS + tx + 16 * j] = gap >= 0 ? s[i][j] * pw[gap] : 0.f;
      }
  }
  {  // the carried state, zeros past d; columns of X are X's own unless transposed
    pdl_wait();
    const float* X = p.ws + (((long long)job.state * p.B * p.H + bh) * p.nch + ch) * d * d;
    const bool v4 = d % 4 == 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < DP * DP / 4; i += kThreads) {
      const int r = i / (DP / 4), c = 4 * (i % (DP / 4));
      const float4 v = load4(X + (r < d ? r * d : 0) + c, r < d ? d - c : 0, v4);
      if (job.trans) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sx[(c + e) * AS + r] = part(v, e);
      } else {
        *reinterpret_cast<float4*>(sx + r * AS + c) = v;
      }
    }
  }
  __syncthreads();

  float acc[4][K][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][k][j] = 0.f;
  // rows of `x` times rows m .. m + 3 of `y`
  auto step = [&](const float* x, int xs, const float* y) {
    float4 a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(x + i * xs);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(y + e * AS + 4 * tx + 64 * k);
#pragma unroll
        for (int i = 0; i < 4; ++i) fma4(acc[i][k], part(a[i], e), v);
      }
  };
  for (int m = 0; m < d4; m += 4) step(sa + i0 * AS + m, AS, sx + m * AS);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i0 + i;
    const float w = r < n ? pw[rev ? n - 1 - r : r + 1] : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][k][j] *= w;
  }
  // the chunk itself: every key all four rows see, then the diagonal 4 x 4 block element by element
  const int lo = rev ? i0 + 4 : 0, hi = rev ? (n + 3) / 4 * 4 : i0;
  for (int r = lo; r < hi; r += 4) step(sp + i0 * PS + r, PS, sc + r * AS);
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((rev ? r >= i : r <= i) && i0 + r < n) {
        const float x = sp[(i0 + i) * PS + i0 + r];
#pragma unroll
        for (int k = 0; k < K; ++k)
          fma4(acc[i][k], x, *reinterpret_cast<const float4*>(sc + (i0 + r) * AS + 4 * tx + 64 * k));
      }
  T* y = static_cast<T*>(job.y.p) + b * job.y.sb + h * job.y.sh;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i0 + i >= n) continue;
    T* yr = y + (long long)(row0 + i0 + i) * job.y.st;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = 4 * tx + 64 * k;
      if (c >= d) continue;
      if (p.vec && sizeof(T) == 4) {
        *reinterpret_cast<float4*>(yr + c) = make_float4(acc[i][k][0], acc[i][k][1], acc[i][k][2], acc[i][k][3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < d) from_f(yr[c + j], acc[i][k][j]);
      }
    }
  }
}

constexpr int update_smem(int dp) { return (2 * kChunk * dp + kChunk) * 4; }
constexpr int out_smem(int dp) { return (3 * kChunk * (dp + 4) + dp * (dp + 4) + kChunk + 4) * 4; }

}  // namespace dcy
}  // namespace favor
