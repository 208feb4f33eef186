// kernel_decay_tc.cuh - linear attention with a decay per head, and its gradients, on sm_100a
// tensor cores (bf16 operands, fp32 accumulation).
//
// What it computes: the scan jobs of kernels_decay.cuh,
//   y_i = sum_j lambda^|i-j| (a_i . b_j) c_j + lambda^(distance) a_i X,   j <= i, or j >= i (reverse),
// with X the state carried into the segment (X = sum b c^T of the tokens before it, decayed).
//
// Blocking. A CTA walks one segment of one head in chunks of 128 tokens. With n tokens in the chunk,
// row weight f_r = lambda^(r+1) (reverse: lambda^(n-1-r)) and update weight w_r = lambda^(n-1-r)
// (reverse: lambda^(r+1)):
//   scores    P = (A B^T) o lambda^|i-j|, masked          128 x 128 x d   -> bf16, in TMEM
//   y         = f (A X) + P C                             128 x d x d, 128 x d x 128
//   state     X <- lambda^n X + (w B)^T C                 d x d x 128
// Every exponent is >= 0: lambda = 0 and strong decays need no division and lose nothing.
//
// Precision. The state stays in fp32 in TMEM; each chunk it is read once, scaled by lambda^n, written
// back, and its bf16 image goes to shared memory for A X. The update accumulates onto it. Rounding
// w B to bf16 would cost the fp32 state 2^-9 of every product, so w B goes in as two bf16 terms, hi =
// bf16(w b) and lo = bf16(w b - hi): 2^-18 per product. hi overwrites B in place once the scores have
// read it. d <= 64 stacks hi and lo as the 128 rows of one operand (rows 64.. of the state collect the
// lo products and are added when it is read out); d <= 128 accumulates hi, then lo.
//
// The state update is the only dependence between chunks: update -> state read and rescaled -> next
// update, about 1000 cycles against the 2700 in which an SM's share of HBM delivers a d = 64 chunk, so a
// walk is bound by memory as long as the loads run ahead (2 or 3 chunks) and every other step
// overlaps. Long sequences of few heads are cut into segments: kernel OUT = false computes each
// segment's own state from b and c alone, k_chunk_scan carries them, and kernel OUT = true walks all
// segments at once.
//
// Warps: 0 TMA; 1 TMEM allocation and every MMA; 4-7 w B; 8-11 state; and with OUT 12-15 scores,
// 16-19 rows out. Thread = row of its 128 (token or state row).
//
// Non-finite values. The mask removes a product by selecting zero into P, but zero times an infinity
// or NaN in a later token's c would still reach earlier rows of the chunk. Rows out notice a
// non-finite P C and sum that element again over its own tokens alone. Rows of c behind the
// sequence's end are zeroed in shared memory.
#pragma once
#include <cuda_bf16.h>

#include "kernels_decay.cuh"
#include "ptx.cuh"

namespace favor {
namespace dtc {

using dcy::View;

constexpr int kTok = 128;
constexpr int kAtomB = kTok * 128;  // 128 rows of 64 bf16 columns, 128-byte swizzle

struct Job {
  int a, b, c;  // operands (indices into Params::m)
  int state, trans, reverse;
  int final;    // 1: writes its state's `out` (one segment only)
  View y;
};

struct Params {
  CUtensorMap m[4];
  int bm[4], hm[4];  // 0 where an operand repeats over batch entries or heads
  Job j[3];
  const float* in[2];  // carried-in states, used where `ws` is null
  float* out[2];
  float* ws;           // [states][BH][nseg][d * d]: OUT = false writes it, OUT = true reads it
  const float* log_decay;
  const int* lengths;
  int njobs, B, H, L, d, nseg, cps;  // chunks per segment
};

template <int DP, bool OUT>
struct Cfg {
  static constexpr int NB = DP / 64;
  static constexpr int kOpB = NB * kAtomB;
  static constexpr int kStageB = (OUT ? 3 : 2) * kOpB;  // b, c, a
  static constexpr int NS = DP == 64 ? (OUT ? 3 : 4) : 2;
  static constexpr int NLO = DP == 64 ? 2 : 1;
  static constexpr int kLo = NS * kStageB;
  // d > 64: the image of X and the lo operand share one buffer (the image is read before lo is written)
  static constexpr int kX = DP == 64 ? kLo + NLO * kOpB : kLo;
  static constexpr int kMisc = kX + (OUT || DP > 64 ? kOpB : 0);
  static constexpr int kSmem = kMisc + 2048 + 1024;
  static constexpr int kThreads = OUT ? 640 : 384;
  static constexpr int SB = OUT && DP == 64 ? 2 : 1;  // score buffers
  static constexpr uint32_t kTO1 = DP, kTO2 = 2 * DP, kTS = DP == 64 ? 192 : 384;
  static constexpr uint32_t kCols = OUT ? 512 : DP;
  static_assert(kSmem <= 232448, "shared memory");
};

struct Misc {
  int abort_flag;
  uint32_t tmem_base;
  alignas(16) float pw[132];   // lambda^0 .. lambda^128
  alignas(16) float pwr[32];   // lambda^31 .. lambda^0
  uint64_t full[4], empty[4];
  uint64_t s_full[2], s_free[2], p_full[2];
  uint64_t x_full, qx_done, bh_full[2], u_done[2], o_full, o_free, st_sync, drain;
};
static_assert(sizeof(Misc) <= 2048, "misc block");

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

template <int DP, bool OUT>
__global__ void __launch_bounds__(Cfg<DP, OUT>::kThreads, 1) k_decay_walk(const __grid_constant__ Params p) {
  using C = Cfg<DP, OUT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gb = smem_raw + (base - raw);
  Misc* ms = reinterpret_cast<Misc*>(gb + C::kMisc);
  volatile int* abort_flag = &ms->abort_flag;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int jid = blockIdx.x % p.njobs;
  const int seg = (blockIdx.x / p.njobs) % p.nseg;
  const int bh = blockIdx.x / p.njobs / p.nseg;
  const int b = bh / p.H, h = bh % p.H;
  const Job& job = p.j[jid];
  const int rev = job.reverse, d = p.d;
  const int len = dcy::seq_len(p.lengths, b, p.L);
  const int nch = (int)(((long long)len + kTok - 1) / kTok);
  const int c0 = seg * p.cps, c1 = min(nch, c0 + p.cps);
  const int N = c1 - c0;  // chunks to walk
  const float* x_in = p.ws && OUT ? p.ws + (((long long)job.state * p.B * p.H + bh) * p.nseg + seg) * d * d
                      : OUT && p.in[job.state] ? p.in[job.state] + (long long)bh * d * d
                                               : nullptr;
  float* x_out = !OUT ? p.ws + (((long long)job.state * p.B * p.H + bh) * p.nseg + seg) * d * d
                 : job.final && p.out[job.state] ? p.out[job.state] + (long long)bh * d * d
                                                 : nullptr;
  // a segment behind the sequence's end; an empty sequence still hands its state on
  if (N <= 0 && !(OUT && x_out)) {
    pdl_launch_dependents();
    if (OUT) pdl_wait();
    return;
  }

  if (tid == 0) {
    ms->abort_flag = 0;
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(bar(ms->full[s]), 1);
      mbar_init(bar(ms->empty[s]), OUT ? 5 : 1);  // the last MMA's commit; rows out
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(ms->s_full[s]), 1);
      mbar_init(bar(ms->s_free[s]), 4);
      mbar_init(bar(ms->p_full[s]), 4);
      mbar_init(bar(ms->u_done[s]), 1);
      mbar_init(bar(ms->bh_full[s]), 4);
    }
    mbar_init(bar(ms->x_full), 4);
    mbar_init(bar(ms->qx_done), 1);
    mbar_init(bar(ms->o_full), 1);
    mbar_init(bar(ms->o_free), 4);
    mbar_init(bar(ms->st_sync), 128);
    mbar_init(bar(ms->drain), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ms->tmem_base), C::kCols);
    tmem_relinquish();
  }
  {
    const float g = p.log_decay[h];
    if (tid <= kTok) {
      const float w = (float)dcy::decay_pow(g, tid);
      ms->pw[tid] = w;
      if (tid < 32) ms->pwr[31 - tid] = w;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = ms->tmem_base;
  auto chunk = [&](int i) { return rev ? c1 - 1 - i : c0 + i; };
  auto tokens = [&](int i) { return min(kTok, len - chunk(i) * kTok); };

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    const bool leader = elect_one();
    const int op[3] = {job.b, job.c, job.a};
    if (leader)
      for (int o = 0; o < (OUT ? 3 : 2); ++o) tma_prefetch_desc(&p.m[op[o]]);
    int issued = 0;
    for (int i = 0; i < N; ++i) {
      const int s = i % C::NS;
      if (i >= C::NS && !mbar_wait(bar(ms->empty[s]), ((i / C::NS) - 1) & 1, abort_flag)) break;
      if (leader) {
        mbar_arrive_expect_tx(bar(ms->full[s]), C::kStageB);
        const int row = chunk(i) * kTok;
#pragma unroll
        for (int o = 0; o < (OUT ? 3 : 2); ++o)
#pragma unroll
          for (int x = 0; x < C::NB; ++x)
            tma_load_4d(base + s * C::kStageB + o * C::kOpB + x * kAtomB, &p.m[op[o]], bar(ms->full[s]), 64 * x, row,
                        h * p.hm[op[o]], b * p.bm[op[o]]);
      }
      issued = i + 1;
      __syncwarp();
    }
    if (*abort_flag)  // let the copies already issued land before the CTA can exit
      for (int i = max(0, issued - C::NS); i < issued; ++i)
        mbar_wait(bar(ms->full[i % C::NS]), (i / C::NS) & 1, nullptr, kWaitLimitCycles / 8);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    const bool leader = elect_one();
    constexpr uint32_t id_s = idesc_f16(128, 128, 1, 1, 0, 0);
    constexpr uint32_t id_x = idesc_f16(128, DP, 1, 1, 0, 1);  // A X and P C
    constexpr uint32_t id_u = idesc_f16(128, DP, 1, 1, 1, 1);
    constexpr uint64_t kRows16 = (16 * 128) >> 4;  // 16 rows of an MN-major operand
    auto kmaj = [](int kk) { return uint64_t(((kk >> 2) * kAtomB + (kk & 3) * 32) >> 4); };
    // scores of chunk i into buffer i % SB
    auto scores = [&](int i) -> bool {
      const int s = i % C::NS, sb = i % C::SB;
      if (!mbar_wait(bar(ms->full[s]), (i / C::NS) & 1, abort_flag)) return false;
      if (i >= C::SB && !mbar_wait(bar(ms->s_free[sb]), ((i / C::SB) - 1) & 1, abort_flag)) return false;
      tc_fence_after();
      if (leader) {
        const uint64_t db = sdesc_sw128(base + s * C::kStageB, 16, 1024);
        const uint64_t da = sdesc_sw128(base + s * C::kStageB + 2 * C::kOpB, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
          mma_ss(tmem + C::kTS + sb * 128, da + kmaj(kk), db + kmaj(kk), id_s, kk > 0 ? 1u : 0u);
        mma_commit(bar(ms->s_full[sb]));
      }
      __syncwarp();
      return true;
    };
    bool ok = !OUT || N <= 0 || scores(0);
    for (int i = 0; ok && i < N; ++i) {
      const int s = i % C::NS, sb = i % C::SB;
      const uint32_t st = base + s * C::kStageB;
      const uint64_t dc = sdesc_sw128(st + C::kOpB, kAtomB, 1024);
      if (OUT) {
        if (C::SB == 2 && i + 1 < N && !(ok = scores(i + 1))) break;
        // A X
        if (!(ok = mbar_wait(bar(ms->x_full), i & 1, abort_flag))) break;
        if (i >= 1 && !(ok = mbar_wait(bar(ms->o_free), (i - 1) & 1, abort_flag))) break;
        tc_fence_after();
        if (leader) {
          const uint64_t da = sdesc_sw128(st + 2 * C::kOpB, 16, 1024);
          const uint64_t dx = sdesc_sw128(base + C::kX, kAtomB, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // 128 rows of X: hi and lo (d <= 64), or d
            mma_ss(tmem + C::kTO1, da + kmaj(DP == 64 ? kk & 3 : kk), dx + kk * kRows16, id_x, kk > 0 ? 1u : 0u);
          if (DP > 64) mma_commit(bar(ms->qx_done));
        }
        __syncwarp();
      } else {
        if (!(ok = mbar_wait(bar(ms->full[s]), (i / C::NS) & 1, abort_flag))) break;
        if (!(ok = mbar_wait(bar(ms->x_full), i & 1, abort_flag))) break;
      }
      // X += (w B)^T C
      if (!(ok = mbar_wait(bar(ms->bh_full[i & 1]), (i >> 1) & 1, abort_flag))) break;
      tc_fence_after();
      if (leader) {
        const uint32_t lo = base + C::kLo + (i % C::NLO) * C::kOpB;
        if (DP == 64) {
          const uint64_t dw = sdesc_sw128(st, lo - st, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mma_ss(tmem, dw + kk * kRows16, dc + kk * kRows16, id_u, 1u);
        } else {
          const uint64_t dh = sdesc_sw128(st, kAtomB, 1024), dl = sdesc_sw128(lo, kAtomB, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mma_ss(tmem, dh + kk * kRows16, dc + kk * kRows16, id_u, 1u);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mma_ss(tmem, dl + kk * kRows16, dc + kk * kRows16, id_u, 1u);
        }
        mma_commit(bar(ms->u_done[i & 1]));
        if (!OUT) mma_commit(bar(ms->empty[s]));
      }
      __syncwarp();
      if (OUT) {
        // P C
        if (!(ok = mbar_wait(bar(ms->p_full[sb]), (i / C::SB) & 1, abort_flag))) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tmem + C::kTO2, tmem + C::kTS + sb * 128 + 8 * kk, dc + kk * kRows16, id_x, kk > 0 ? 1u : 0u);
          mma_commit(bar(ms->o_full));
          mma_commit(bar(ms->empty[s]));
        }
        __syncwarp();
        if (C::SB == 1 && i + 1 < N && !(ok = scores(i + 1))) break;
      }
    }
    if (leader) mma_commit(bar(ms->drain));
    __syncwarp();
    mbar_wait(bar(ms->drain), 0, nullptr, kWaitLimitCycles / 8);
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ w B, in place (hi) and beside it (lo)
    const int t = tid - 128;
    for (int i = 0; i < N; ++i) {
      const int s = i % C::NS, n = tokens(i);
      if (!mbar_wait(bar(ms->full[s]), (i / C::NS) & 1, abort_flag)) break;
      // the lo buffer's last reader is update i - NLO
      if (i >= C::NLO && !mbar_wait(bar(ms->u_done[(i - C::NLO) & 1]), ((i - C::NLO) >> 1) & 1, abort_flag)) break;
      if (OUT && !mbar_wait(bar(ms->s_full[i % C::SB]), (i / C::SB) & 1, abort_flag)) break;  // B has been read
      if (OUT && DP > 64 && !mbar_wait(bar(ms->qx_done), i & 1, abort_flag)) break;           // so has X's image
      uint8_t* hi = gb + s * C::kStageB;
      uint8_t* lo = gb + C::kLo + (i % C::NLO) * C::kOpB;
#pragma unroll 4
      for (int e = t; e < C::kOpB / 16; e += 128) {
        const int r = (e >> 3) & (kTok - 1);
        uint4 x = *reinterpret_cast<const uint4*>(hi + 16 * e), y;
        if (r < n) {
          const float w = ms->pw[rev ? r + 1 : n - 1 - r];
          uint32_t* px = &x.x;
          uint32_t* py = &y.x;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float u0 = bf_lo(px[q]) * w, u1 = bf_hi(px[q]) * w;
            px[q] = pack_bf16x2(u0, u1);
            py[q] = pack_bf16x2(u0 - bf_lo(px[q]), u1 - bf_hi(px[q]));
          }
        } else {
          x = y = make_uint4(0u, 0u, 0u, 0u);
        }
        *reinterpret_cast<uint4*>(hi + 16 * e) = x;
        *reinterpret_cast<uint4*>(lo + 16 * e) = y;
      }
      if (n < kTok) {  // rows of c behind the end take part in products with zero: they must be finite
        uint8_t* cc = hi + C::kOpB;
        for (int e = t; e < C::kOpB / 16; e += 128)
          if (((e >> 3) & (kTok - 1)) >= n) *reinterpret_cast<uint4*>(cc + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ms->bh_full[i & 1]));
    }
  } else if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------ state (thread = row of X, b's column)
    const int q4 = warp & 3, row = q4 * 32 + lane;
    const uint32_t la = uint32_t(q4 * 32) << 16;
    const bool real = row < d && (DP > 64 || row < 64);
    if (OUT && x_in) pdl_wait();  // the carried states are written by the kernel before
    bool ok = true;
    uint32_t ph = 0;
    for (int i = 0; ok && i <= N; ++i) {
      if (i > 0) {
        if (!(ok = mbar_wait(bar(ms->u_done[(i - 1) & 1]), ((i - 1) >> 1) & 1, abort_flag))) break;
        tc_fence_after();
      }
      if (i == N && !x_out) break;
      const float f = i < N ? ms->pw[tokens(i)] : 1.f;
      float* scr = reinterpret_cast<float*>(gb + C::kLo);  // free once the last update is done
#pragma unroll 1
      for (int x = 0; x < DP / 32; ++x) {
        uint32_t v[32];
        if (i > 0) {
          tmem_ld32(tmem + la + 32 * x, v);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int n = 32 * x + e;
            v[e] = __float_as_uint(x_in && real && n < d ? (job.trans ? x_in[n * d + row] : x_in[row * d + n]) : 0.f);
          }
        }
        if (i < N) {
          if (OUT) {
            uint8_t* img = gb + C::kX + (x >> 1) * kAtomB + row * 128;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint4 o;
              o.x = pack_bf16x2(__uint_as_float(v[8 * q]), __uint_as_float(v[8 * q + 1]));
              o.y = pack_bf16x2(__uint_as_float(v[8 * q + 2]), __uint_as_float(v[8 * q + 3]));
              o.z = pack_bf16x2(__uint_as_float(v[8 * q + 4]), __uint_as_float(v[8 * q + 5]));
              o.w = pack_bf16x2(__uint_as_float(v[8 * q + 6]), __uint_as_float(v[8 * q + 7]));
              *reinterpret_cast<uint4*>(img + ((((x & 1) * 4 + q) ^ (row & 7)) << 4)) = o;
            }
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
          tmem_st32(tmem + la + 32 * x, v);
        } else {
          if (DP == 64) {  // rows 64.. hold the lo products' sums
            if (!(ok = __all_sync(0xffffffffu, group_sync(bar(ms->st_sync), ph, abort_flag)))) break;
            if (row >= 64)
#pragma unroll
              for (int e = 0; e < 32; ++e) scr[e * 64 + row - 64] = N > 0 ? __uint_as_float(v[e]) : 0.f;
            if (!(ok = __all_sync(0xffffffffu, group_sync(bar(ms->st_sync), ph, abort_flag)))) break;
            if (row < 64)
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + scr[e * 64 + row]);
          }
          if (real) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int n = 32 * x + e;
              if (n < d) x_out[job.trans ? n * d + row : row * d + n] = __uint_as_float(v[e]);
            }
          }
        }
      }
      if (i < N) {
        tmem_wait_st();
        if (OUT) fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ms->x_full));
      }
    }
  } else if (OUT && warp >= 12 && warp < 16) {
    // ------------------------------------------------------------ scores -> P (thread = row)
    const int q4 = warp & 3, row = q4 * 32 + lane;
    const uint32_t la = uint32_t(q4 * 32) << 16;
    const float* wt = rev ? ms->pw : ms->pwr;
    for (int i = 0; i < N; ++i) {
      const int sb = i % C::SB, n = tokens(i);
      if (!mbar_wait(bar(ms->s_full[sb]), (i / C::SB) & 1, abort_flag)) break;
      tc_fence_after();
      const uint32_t ts = tmem + la + C::kTS + sb * 128;
      // P's 16 columns of block x lie in scores that are read or masked by then
#pragma unroll 1
      for (int x = 0; x < 4; ++x) {
        uint32_t pk[16];
        if (rev ? x < q4 : x > q4) {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0u;
        } else {
          uint32_t v[32];
          tmem_ld32(ts + 32 * x, v);
          tmem_wait_ld();
          if (x == q4) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int gap = rev ? e - lane : lane - e;
              const float u = __uint_as_float(v[e]) * ms->pw[max(gap, 0)];
              v[e] = __float_as_uint(gap >= 0 ? u : 0.f);
            }
          } else {
            // lambda^(i-j) = lambda^(i-32x-31) lambda^(31-(j-32x)), reversed lambda^(32x-i) lambda^(j-32x)
            const float w1 = ms->pw[rev ? 32 * x - row : row - 32 * x - 31];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 w = *reinterpret_cast<const float4*>(wt + e);
              v[e] = __float_as_uint(__uint_as_float(v[e]) * (w1 * w.x));
              v[e + 1] = __float_as_uint(__uint_as_float(v[e + 1]) * (w1 * w.y));
              v[e + 2] = __float_as_uint(__uint_as_float(v[e + 2]) * (w1 * w.z));
              v[e + 3] = __float_as_uint(__uint_as_float(v[e + 3]) * (w1 * w.w));
            }
          }
          if (rev && n < kTok) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * x + e >= n) v[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
        }
        tmem_st16(ts + 16 * x, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ms->p_full[sb]));
    }
  } else if (OUT && warp >= 16) {
    // ------------------------------------------------------------ rows out (thread = row)
    const int q4 = warp & 3, row = q4 * 32 + lane;
    const uint32_t la = uint32_t(q4 * 32) << 16;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(job.y.p) + b * job.y.sb + h * job.y.sh;
    for (int i = 0; i < N; ++i) {
      const int s = i % C::NS, sb = i % C::SB, n = tokens(i);
      if (!mbar_wait(bar(ms->o_full), i & 1, abort_flag)) break;
      tc_fence_after();
      const bool live = row < n;
      const float f = ms->pw[live ? (rev ? n - 1 - row : row + 1) : 0];
      __nv_bfloat16* yr = y + ((long long)chunk(i) * kTok + row) * job.y.st;
#pragma unroll 1
      for (int x = 0; x < DP / 32; ++x) {
        uint32_t o1[32], o2[32];
        tmem_ld32(tmem + la + C::kTO2 + 32 * x, o2);
        tmem_ld32(tmem + la + C::kTO1 + 32 * x, o1);
        tmem_wait_ld();
        float z = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) z = fmaf(__uint_as_float(o2[e]), 0.f, z);  // NaN if any is not finite
        if (__any_sync(0xffffffffu, live && !(z == 0.f))) {
          // an infinity or NaN in this chunk's c (or P): sum such elements over the row's own tokens
          mbar_wait(bar(ms->full[s]), (i / C::NS) & 1, abort_flag);
          const uint8_t* cc = gb + s * C::kStageB + C::kOpB + (x >> 1) * kAtomB;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float acc[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
              uint32_t pp;
              tmem_ld1(tmem + la + C::kTS + sb * 128 + (j >> 1), pp);
              tmem_wait_ld();
              if (rev ? j >= row : j <= row) {
                const float pj = j & 1 ? bf_hi(pp) : bf_lo(pp);
                const uint4 u = *reinterpret_cast<const uint4*>(cc + j * 128 + ((((x & 1) * 4 + q) ^ (j & 7)) << 4));
                const uint32_t* pu = &u.x;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  acc[2 * k] = fmaf(pj, bf_lo(pu[k]), acc[2 * k]);
                  acc[2 * k + 1] = fmaf(pj, bf_hi(pu[k]), acc[2 * k + 1]);
                }
              }
              __syncwarp();
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (!(__uint_as_float(o2[8 * q + e]) * 0.f == 0.f)) o2[8 * q + e] = __float_as_uint(acc[e]);
          }
        }
        if (live) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (32 * x + 8 * q >= d) continue;
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 8 * q + 2 * k;
              o[k] = pack_bf16x2(fmaf(f, __uint_as_float(o1[e]), __uint_as_float(o2[e])),
                                 fmaf(f, __uint_as_float(o1[e + 1]), __uint_as_float(o2[e + 1])));
            }
            *reinterpret_cast<uint4*>(yr + 32 * x + 8 * q) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(ms->o_free));
        mbar_arrive(bar(ms->s_free[sb]));
        mbar_arrive(bar(ms->empty[s]));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

}  // namespace dtc
}  // namespace favor
