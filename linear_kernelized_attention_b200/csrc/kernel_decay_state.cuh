// kernel_decay_state.cuh - the states of linear attention with a decay, to fp32 accuracy, on sm_100a
// tensor cores.
//
// What it computes, for a segment of one head: X = sum_r w_r b_r c_r^T over the segment's tokens, w_r =
// lambda^(tokens of the segment beyond r in the state's direction). As the only segment of a sequence it
// adds lambda^len of the state carried in: state_out, or dstate_in.
//
// Precision. The caller gets X in fp32, so three things that the bf16 rows of kernel_decay_tc.cuh do
// without are done here. w b is fed to the MMAs as three bf16 terms, hi + mid + lo, each the rounding of
// what the ones before leave: 2^-26 of a product. Each 128-token chunk is summed from zero and added to
// running sums in registers with fp32's own rounding: tensor cores truncate every accumulation, which
// over a whole segment pulls a slowly decaying state towards zero (measured at 57 chunks and lambda^128
// near 1: 1.4e-5 of the state's norm, against 4e-7 as it is). hi and the smaller terms have accumulators of
// their own, so the large sums are truncated eight times a chunk, no more.
//
// Chunks are taken against the state's direction, so that a chunk's factor, the decay over the tokens
// beyond it, grows from 1 by one product (in double) a chunk, and nothing is ever rescaled.
//
// Reading b and c bounds it at best: 32 KB a chunk and head at d = 64, 1400 cycles of an SM's share of HBM.
// Measured: 1.3 us (2300 cycles) a chunk at d = 64 and 2.0 at d = 128, most of it the products, which alone
// take 770 and 1540 cycles. Terms are made in units of 8192 elements (128 tokens, or 64 at
// d > 64) with two buffers, so that one unit's products run beside the next one's arithmetic; with one
// buffer d = 128 took 3.2 us, and units of 64 tokens at d = 64 took 1.6.
//
// Warps: 0 TMA; 1 TMEM allocation and MMAs; 4-11 the three terms of w b (hi in place, mid and lo beside
// it); from 12 on the running sums, thread = row of X (b's column).
// d <= 64: [hi; mid] as the 128 rows of one operand, [lo; mid] as another whose second half is unused.
#pragma once
#include "kernel_decay_tc.cuh"

namespace favor {
namespace dst {

using dtc::kAtomB;
using dtc::kTok;

struct Job {
  int b, c;  // operands (indices into Params::m)
  int reverse;
  const float* in;  // one segment only: carried in (null: zeros)
  float* out;       // one segment only
};

struct Params {
  CUtensorMap m[4];
  int bm[4], hm[4];  // 0 where an operand repeats over batch entries or heads
  Job j[2];
  float* ws;         // several segments: [states][BH][nseg][d * d]
  const float* log_decay;
  const int* lengths;
  int njobs, B, H, L, d, nseg, cps;  // chunks per segment
};

template <int DP>
struct Cfg {
  static constexpr int NB = DP / 64;
  static constexpr int kOpB = NB * kAtomB;
  static constexpr int kStageB = 2 * kOpB;  // b, c
  static constexpr int NS = DP == 64 ? 4 : 2;
  static constexpr int UPC = NB;                    // units of terms a chunk: 128 tokens of 64 columns, or 64 of 128
  static constexpr int kUnitB = kOpB / UPC, kUnitAtomB = kAtomB / UPC;
  static constexpr int NT = 2;                      // buffers of a unit's (lo, mid)
  static constexpr int kTerms = NS * kStageB;
  static constexpr int kMisc = kTerms + NT * 2 * kUnitB;
  static constexpr int kSmem = kMisc + 2048 + 1024;
  static constexpr int kThreads = DP == 64 ? 512 : 640;
  static constexpr uint32_t kAcc = 2 * DP;          // columns of one chunk's accumulators: hi (and mid), the rest
  static constexpr uint32_t kCols = 512;
  static_assert(kSmem <= 232448, "shared memory");
};

struct Misc {
  int abort_flag;
  uint32_t tmem_base;
  float pw[132];  // lambda^0 .. lambda^128
  uint64_t full[4], empty[4], t_full[2], t_free[2], done[2], d_free[2], sync, drain;
};

// The state of block `block`: job, segment and head. SC: columns a thread sums, 64, or 32 where the block has the
// walk's many threads and few registers each.
template <int DP, int SC>
__device__ __forceinline__ void state_block(const Params& p, unsigned block) {
  constexpr int kSumWarps = 4 * DP / SC;
  using C = Cfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gb = smem_raw + (base - raw);
  Misc* ms = reinterpret_cast<Misc*>(gb + C::kMisc);
  volatile int* abort_flag = &ms->abort_flag;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };

  // What decides control flow is broadcast from lane 0, so that the compiler knows it to be uniform: loop
  // counters and MMA descriptors then live in uniform registers (otherwise an MMA takes 100 to 150 cycles to
  // issue; the products themselves take 32 to 64).
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int jid = block % p.njobs;
  const int seg = (block / p.njobs) % p.nseg;
  const int bh = block / p.njobs / p.nseg;
  const int b = bh / p.H, h = bh % p.H;
  const Job& job = p.j[jid];
  const int rev = job.reverse, d = p.d;
  const int len = __shfl_sync(0xffffffffu, dcy::seq_len(p.lengths, b, p.L), 0);
  const int nch = (int)(((long long)len + kTok - 1) / kTok);
  const int c0 = seg * p.cps, c1 = min(nch, c0 + p.cps);
  const int N = max(0, c1 - c0);
  if (N == 0 && p.ws) {  // a segment behind the sequence's end
    pdl_launch_dependents();
    pdl_wait();
    return;
  }
  auto chunk = [&](int i) { return rev ? c0 + i : c1 - 1 - i; };
  auto tokens = [&](int i) { return min(kTok, len - chunk(i) * kTok); };
  auto load = [&](int i) {  // one lane: chunk i into its stage
    const int s = i % C::NS, row = chunk(i) * kTok;
    const int op[2] = {job.b, job.c};
    mbar_arrive_expect_tx(bar(ms->full[s]), C::kStageB);
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int x = 0; x < C::NB; ++x)
        dtc::tma_load_4d(base + s * C::kStageB + o * C::kOpB + x * kAtomB, &p.m[op[o]], bar(ms->full[s]), 64 * x, row,
                         h * p.hm[op[o]], b * p.bm[op[o]]);
  };
  if (tid == 0) {
    ms->abort_flag = 0;
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(bar(ms->full[s]), 1);
      mbar_init(bar(ms->empty[s]), 1);
    }
    for (int s = 0; s < C::NT; ++s) {
      mbar_init(bar(ms->t_full[s]), 8);
      mbar_init(bar(ms->t_free[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(ms->done[s]), 1);
      mbar_init(bar(ms->d_free[s]), kSumWarps);
    }
    mbar_init(bar(ms->sync), 32 * kSumWarps);
    mbar_init(bar(ms->drain), 1);
    fence_mbar_init();
    for (int i = 0; i < min(N, C::NS); ++i) load(i);  // in flight while the block sets up
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ms->tmem_base), C::kCols);
    tmem_relinquish();
  }
  if (tid >= 96 && tid <= 96 + kTok) ms->pw[tid - 96] = (float)dcy::decay_pow(p.log_decay[h], tid - 96);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  constexpr uint32_t tmem = 0;  // all 512 columns are this block's

  if (warp == 0) {
    const bool leader = elect_one();
    int issued = min(N, C::NS);
    for (int i = issued; i < N; ++i) {
      if (!mbar_wait(bar(ms->empty[i % C::NS]), ((i / C::NS) - 1) & 1, abort_flag)) break;
      if (leader) load(i);
      issued = i + 1;
      __syncwarp();
    }
    if (*abort_flag)  // let the copies already issued land before the CTA can exit
      for (int i = max(0, issued - C::NS); i < issued; ++i)
        mbar_wait(bar(ms->full[i % C::NS]), (i / C::NS) & 1, nullptr, kWaitLimitCycles / 8);
    __syncwarp();
  } else if (warp == 1) {
    // straight-line for the whole warp, as in kernel_decay_tc.cuh
    const uint32_t lead = elect_one();
    constexpr uint32_t id_u = idesc_f16(128, DP, 1, 1, 1, 1);
    constexpr uint64_t kRows16 = (16 * 128) >> 4;
    for (int i = 0; i < N; ++i) {
      const int s = i % C::NS;
      mbar_wait(bar(ms->full[s]), (i / C::NS) & 1, abort_flag);
      if (i >= 2) mbar_wait(bar(ms->d_free[i & 1]), ((i >> 1) - 1) & 1, abort_flag);
      const uint32_t acc = tmem + (i & 1) * C::kAcc;
#pragma unroll
      for (int f = 0; f < C::UPC; ++f) {
        const int u = C::UPC * i + f, t = u % C::NT;
        mbar_wait(bar(ms->t_full[t]), (u / C::NT) & 1, abort_flag);
        tc_fence_after();
        const uint32_t hi = base + s * C::kStageB + f * C::kUnitAtomB, lo = base + C::kTerms + t * 2 * C::kUnitB, mid = lo + C::kUnitB;
        const uint64_t dc = sdesc_sw128(hi + C::kOpB, kAtomB, 1024);
        const uint64_t dh = sdesc_sw128(hi, DP == 64 ? mid - hi : kAtomB, 1024);
        const uint64_t dl = sdesc_sw128(lo, C::kUnitAtomB, 1024);  // d <= 64: mid is its second half
#pragma unroll
        for (int kk = 0; kk < 8 / C::UPC; ++kk)
          dtc::mma_ss_if(lead, acc, dh + kk * kRows16, dc + kk * kRows16, id_u, f > 0 || kk > 0 ? 1u : 0u);
        if (DP > 64) {
          const uint64_t dm = sdesc_sw128(mid, C::kUnitAtomB, 1024);
#pragma unroll
          for (int kk = 0; kk < 8 / C::UPC; ++kk)
            dtc::mma_ss_if(lead, acc + DP, dm + kk * kRows16, dc + kk * kRows16, id_u, f > 0 || kk > 0 ? 1u : 0u);
        }
#pragma unroll
        for (int kk = 0; kk < 8 / C::UPC; ++kk)
          dtc::mma_ss_if(lead, acc + DP, dl + kk * kRows16, dc + kk * kRows16, id_u, DP > 64 || f > 0 || kk > 0 ? 1u : 0u);
        dtc::commit_if(lead, bar(ms->t_free[t]));
      }
      dtc::commit_if(lead, bar(ms->done[i & 1]));
      dtc::commit_if(lead, bar(ms->empty[s]));
    }
    dtc::commit_if(lead, bar(ms->drain));
    __syncwarp();
    mbar_wait(bar(ms->drain), 0, nullptr, kWaitLimitCycles / 8);
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ w b, a unit at a time
    constexpr int UR = kTok / C::UPC, NR = UR / 32;  // rows of a unit, and of a thread in each 64 columns
    const int t = tid - 128, r0 = t >> 3;
    const uint64_t m1 = dtc::pair(-1.f, -1.f);
    double cf = 1.0;  // decay over the segment's tokens beyond the chunk
    const double full = dcy::decay_pow(p.log_decay[h], kTok);
    for (int u = 0; u < C::UPC * N; ++u) {
      const int i = u / C::UPC, f = u % C::UPC, s = i % C::NS, n = tokens(i), tb = u % C::NT;
      float w[NR];
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int r = UR * f + r0 + 32 * k;
        w[k] = r < n ? ms->pw[rev ? r + 1 : n - 1 - r] * (float)cf : 0.f;
      }
      if (f == C::UPC - 1) cf *= n == kTok ? full : dcy::decay_pow(p.log_decay[h], n);
      if (!mbar_wait(bar(ms->full[s]), (i / C::NS) & 1, abort_flag)) break;
      if (u >= C::NT && !mbar_wait(bar(ms->t_free[tb]), ((u / C::NT) - 1) & 1, abort_flag)) break;
      uint8_t* hi = gb + s * C::kStageB + C::kUnitAtomB * f + 16 * t;
      uint8_t* lo = gb + C::kTerms + tb * 2 * C::kUnitB + 16 * t;
      uint8_t* mid = lo + C::kUnitB;
      uint4 v[4];  // NB atoms x NR rows
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const uint4*>(hi + (k / NR) * kAtomB + (k % NR) * 4096);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t ww = dtc::pair(w[k % NR], w[k % NR]);
        uint32_t ph[4] = {v[k].x, v[k].y, v[k].z, v[k].w}, pm[4], pl[4];
        const bool past = UR * f + r0 + 32 * (k % NR) >= n;  // rows behind the end may hold anything
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint64_t y = dtc::mul2(dtc::pair(ph[q] << 16, ph[q] & 0xffff0000u), ww);
          ph[q] = dtc::pack2(y);
          const uint64_t y1 = dtc::fma2(dtc::pair(ph[q] << 16, ph[q] & 0xffff0000u), m1, y);
          pm[q] = dtc::pack2(y1);
          pl[q] = dtc::pack2(dtc::fma2(dtc::pair(pm[q] << 16, pm[q] & 0xffff0000u), m1, y1));
          if (past) ph[q] = pm[q] = pl[q] = 0u;
        }
        *reinterpret_cast<uint4*>(hi + (k / NR) * kAtomB + (k % NR) * 4096) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
        *reinterpret_cast<uint4*>(mid + (k / NR) * C::kUnitAtomB + (k % NR) * 4096) = make_uint4(pm[0], pm[1], pm[2], pm[3]);
        *reinterpret_cast<uint4*>(lo + (k / NR) * C::kUnitAtomB + (k % NR) * 4096) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
      }
      if (n < UR * f + UR) {  // rows of c behind the end take part in products with zero: they must be finite
        uint8_t* cc = gb + s * C::kStageB + C::kOpB;
        for (int e = t; e < C::kOpB / 16; e += 256) {
          const int r = (e >> 3) & (kTok - 1);
          if (r >= n && r / UR == f) *reinterpret_cast<uint4*>(cc + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ms->t_full[tb]));
    }
  } else if (warp >= 12 && warp < 12 + kSumWarps) {
    // ------------------------------------------------------------ running sums (thread = row of X, SC columns)
    const int q4 = warp & 3, row = q4 * 32 + lane, col0 = SC * ((warp - 12) >> 2);
    const uint32_t la = uint32_t(q4 * 32) << 16;
    const bool second = DP > 64 || q4 < 2;  // d <= 64: rows 64.. of the second accumulator are unused
    float x[SC];
#pragma unroll
    for (int e = 0; e < SC; ++e) x[e] = 0.f;
    bool ok = true;
    for (int i = 0; i < N; ++i) {
      if (!(ok = mbar_wait(bar(ms->done[i & 1]), (i >> 1) & 1, abort_flag))) break;
      tc_fence_after();
      const uint32_t acc = tmem + la + (i & 1) * C::kAcc + col0;
#pragma unroll
      for (int y = 0; y < SC; y += 8) {
        uint32_t v[8], u[8];
        if (second) tmem_ld8(acc + DP + y, v);
        tmem_ld8(acc + y, u);
        tmem_wait_ld();
        if (second) {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) + __uint_as_float(v[e]));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[y + e] += __uint_as_float(u[e]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ms->d_free[i & 1]));
    }
    if (DP == 64) {  // rows 64.. hold the mid terms' sums: through shared memory to rows 0 .. 63
      uint32_t ph = 0;
      float* scr = reinterpret_cast<float*>(gb + C::kTerms);  // free: the last product is done
      ok = __all_sync(0xffffffffu, ok);
      if (ok && row >= 64) {
#pragma unroll
        for (int e = 0; e < SC; ++e) scr[(col0 + e) * 64 + row - 64] = x[e];
      }
      ok = group_sync(bar(ms->sync), ph, abort_flag) && ok;
      if (ok && row < 64) {
#pragma unroll
        for (int e = 0; e < SC; ++e) x[e] += scr[(col0 + e) * 64 + row];
      }
    }
    if (ok && row < d && row < DP && (DP > 64 || row < 64)) {
      const long long dd = (long long)d * d;
      float* out = p.ws ? p.ws + (((long long)jid * p.B * p.H + bh) * p.nseg + seg) * dd : job.out + bh * dd;
      const float* in = !p.ws && job.in ? job.in + bh * dd : nullptr;
      const double f = in ? dcy::decay_pow(p.log_decay[h], len) : 0.0;
#pragma unroll
      for (int e = 0; e < SC; e += 4) {
        if (col0 + e >= d) continue;
        const long long at = (long long)row * d + col0 + e;
        float4 y = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        if (in) {
          const float4 z = *reinterpret_cast<const float4*>(in + at);
          y = make_float4((float)(f * z.x + y.x), (float)(f * z.y + y.y), (float)(f * z.z + y.z),
                          (float)(f * z.w + y.w));
        }
        *reinterpret_cast<float4*>(out + at) = y;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(ms->tmem_base, C::kCols);
  }
}

template <int DP>
__global__ void __launch_bounds__(Cfg<DP>::kThreads, 1) k_decay_state(const __grid_constant__ Params p) {
  state_block<DP, 64>(p, blockIdx.x);
  pdl_wait();  // where this kernel was started beside the walk: it ends after it
}

// Walks and, in the blocks behind them, the whole sequences' states, in one launch for short calls. The blocks
// share nothing.
struct Both {
  dtc::Params w;
  Params s;
  int nwalk;
};
template <int DP>
__global__ void __launch_bounds__(dtc::Cfg<DP>::kThreads, 1) k_decay_both(const __grid_constant__ Both p) {
  if ((int)blockIdx.x < p.nwalk)
    dtc::walk_block<DP>(p.w, blockIdx.x);
  else
    state_block<DP, 32>(p.s, blockIdx.x - p.nwalk);
}

}  // namespace dst
}  // namespace favor
