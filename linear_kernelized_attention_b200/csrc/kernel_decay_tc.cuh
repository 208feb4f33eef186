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
// Precision. The walk's state serves its bf16 rows; the states a caller gets back are summed to fp32
// accuracy by kernel_decay_state.cuh. It stays in fp32 in TMEM; each chunk it is read once, scaled by
// lambda^n, written back, and its bf16 image goes to shared memory for A X. The update accumulates onto
// it. Rounding w B to bf16 would put a second rounding of 2^-8 on every product that reaches a later
// chunk, beside the image's, so w B goes in as two bf16 terms, hi = bf16(w b) and lo = bf16(w b - hi). hi
// overwrites B in place once the scores have read it. d <= 64 stacks hi and lo as the 128 rows of one
// operand: rows 64.. of the state and of its image are the lo products' sums, and A X reads A twice.
// d <= 128 accumulates hi, then lo. The image of X and the weighted scores P are operands of the MMAs in bf16: one
// rounding of 2^-8 of each product, with independent signs. Measured, random inputs, rows are 2.35e-3 of their norm from
// 64 bits: 1.66e-3 from that rounding and 1.66e-3 from the result's own, which the plain form has too. A second term
// of P would take eight more products a chunk (256 of its 2700 cycles at d = 64), one of the image 32 KB, a stage's room.
//
// What bounds it. An SM's share of HBM delivers a d = 64 chunk in about 2700 cycles and a d = 128 one in
// 5400; a chunk takes 2600 to 3000 and 5500 (measured: 16 heads x 65536 tokens, d = 64, in 98 us). The
// products themselves take 1100 and 2300 of them; shared memory is busy for about 2300 at d = 64 (operands of
// the MMAs, loads, w B in place, the image), and each role's instructions and hand-overs for 1000 to 1600.
// Long sequences of few heads are cut into segments: the state kernel sums each segment's own state from
// b and c alone, k_chunk_scan carries them, and this kernel walks all segments at once.
//
// Warps: 0 TMA; 1 TMEM allocation and every MMA; 4-11 w B and state; 12-19 scores; 20-27
// rows out. Thread = row of its 128 (token or state row).
//
// Non-finite values. The mask removes a product by selecting zero into P, but zero times an infinity
// or NaN in a later token's c would still reach earlier rows of the chunk. Rows out notice a
// non-finite P C where A X is finite and sum that element again, from global memory, over its own tokens
// alone, so that nothing on chip waits for them. Measured, 2 x 8 heads x 2048 tokens: one such token's chunk
// adds up to 0.9 ms to a call at d = 64 and 3.3 ms at d = 128, wherever the next ones are (X carries them);
// with every element of an operand NaN calls take 1 to 2 times a clean one's. Rows of c behind the
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
  View va, vb, vc, y;  // rows in global memory: a, b, c for elements summed again
};

struct Params {
  CUtensorMap m[4], my[3];  // operands (boxes of 64 columns x 128 tokens), outputs by job (32 x 32)
  int bm[4], hm[4];  // 0 where an operand repeats over batch entries or heads
  Job j[3];
  const float* in[2];  // carried-in states, used where `ws` is null
  const float* ws;     // [states][BH][nseg][d * d], the states carried into each segment
  const float* log_decay;
  const int* lengths;
  int njobs, B, H, L, d, nseg, cps;  // chunks per segment
};

template <int DP>
struct Cfg {
  static constexpr int NB = DP / 64;
  static constexpr int kOpB = NB * kAtomB;
  static constexpr int kStageB = 3 * kOpB;  // b, c, a
  static constexpr int NS = DP == 64 ? 3 : 2;
  static constexpr int NLO = DP == 64 ? 2 : 1;
  static constexpr int kLo = NS * kStageB;
  // d > 64: the image of X and the lo operand share one buffer (the image is read before lo is
  // written), and rows out are staged over the chunk's own A, which every product has read by then.
  static constexpr int NX = DP == 64 ? 2 : 1;
  static constexpr int kX = DP == 64 ? kLo + NLO * kOpB : kLo;
  static constexpr int kY = kX + NX * kOpB;
  static constexpr int kMisc = kY + (DP == 64 ? kOpB : 0);
  static constexpr int kSmem = kMisc + 2048 + 1024;
  // 72 registers a thread: k_decay_walk<128> spills 28 bytes, the joint kernel of kernel_decay_state.cuh 56 and 92
  // (d <= 64 reloads 260 bytes of it), k_decay_walk<64> none
  static constexpr int kThreads = 896;
  static constexpr int kBT = DP == 64 ? 128 : 256;  // threads that weight B
  static constexpr int SB = DP == 64 ? 2 : 1;  // score buffers
  static constexpr uint32_t kTO1 = DP, kTO2 = 2 * DP, kTS = DP == 64 ? 192 : 384;
  static constexpr uint32_t kCols = 512;
  static_assert(kSmem <= 232448, "shared memory");
};

struct Misc {
  int abort_flag;
  uint32_t tmem_base;
  float pw[132];               // lambda^0 .. lambda^128
  float pwz[64];               // 31 zeros, then lambda^0 .. lambda^31
  uint64_t full[4], empty[4];
  uint64_t s_full[2], p_full[2];
  uint64_t x_full, img_full[2], qx_done, pc_done[2], bh_full[2], u_done[2], o_full, o_free, drain;
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

__device__ __forceinline__ void tma_store_4d(const void* tmap, uint32_t src, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}

// MMAs and commits of the one lane with `lead` set, without a branch: the descriptors stay warp-uniform.
__device__ __forceinline__ void mma_ss_if(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint64_t pair(float x, float y) { return pair(__float_as_uint(x), __float_as_uint(y)); }
__device__ __forceinline__ void unpair(uint64_t v, uint32_t& x, uint32_t& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {  // (low, high) to bf16x2
  uint32_t x, y;
  unpair(v, x, y);
  return pack_bf16x2(__uint_as_float(x), __uint_as_float(y));
}

// Column of P's tokens j, j + 1 (bf16 pairs) in their score buffer: each half over its own scores.
__host__ __device__ constexpr int p_col(int j) { return (j & 64) + ((j & 63) >> 1); }

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// One token's row of an operand, and eight of its elements.
__device__ __forceinline__ const __nv_bfloat16* row_of(const View& v, int b, int h, long long t) {
  return static_cast<const __nv_bfloat16*>(v.p) + b * v.sb + h * v.sh + t * v.st;
}
__device__ __forceinline__ void load8(float (&x)[8], const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  x[0] = bf_lo(u.x), x[1] = bf_hi(u.x), x[2] = bf_lo(u.y), x[3] = bf_hi(u.y);
  x[4] = bf_lo(u.z), x[5] = bf_hi(u.z), x[6] = bf_lo(u.w), x[7] = bf_hi(u.w);
}

// Columns 32 x .. of one row of X from a [d, d] state, or its transpose; zeros where there is none.
__device__ __forceinline__ void load_state(uint32_t (&v)[32], const float* in, int x, int row, int d, int trans) {
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = 0u;
  if (!in || row >= d) return;  // d <= 64: rows 64.. are the lo products', from zero
  if (trans) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (32 * x + e < d) v[e] = __float_as_uint(in[(32 * x + e) * d + row]);
  } else {
#pragma unroll
    for (int e = 0; e < 32; e += 4)
      if (32 * x + e < d) {
        const uint4 u = *reinterpret_cast<const uint4*>(in + row * d + 32 * x + e);
        v[e] = u.x, v[e + 1] = u.y, v[e + 2] = u.z, v[e + 3] = u.w;
      }
  }
}

// The walk of block `block`: job, segment and head.
template <int DP>
__device__ __forceinline__ void walk_block(const Params& p, unsigned block) {
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
  const int N = c1 - c0;  // chunks to walk
  const float* x_in = p.ws ? p.ws + (((long long)job.state * p.B * p.H + bh) * p.nseg + seg) * d * d
                      : p.in[job.state] ? p.in[job.state] + (long long)bh * d * d
                                        : nullptr;
  if (N <= 0) {  // a segment behind the sequence's end
    pdl_launch_dependents();
    pdl_wait();
    return;
  }
  auto chunk = [&](int i) { return rev ? c1 - 1 - i : c0 + i; };
  auto tokens = [&](int i) { return min(kTok, len - chunk(i) * kTok); };
  const int op[3] = {job.b, job.c, job.a};
  auto load = [&](int i) {  // one lane: chunk i into its stage
    const int s = i % C::NS, row = chunk(i) * kTok;
    mbar_arrive_expect_tx(bar(ms->full[s]), C::kStageB);
#pragma unroll
    for (int o = 0; o < 3; ++o)
#pragma unroll
      for (int x = 0; x < C::NB; ++x)
        tma_load_4d(base + s * C::kStageB + o * C::kOpB + x * kAtomB, &p.m[op[o]], bar(ms->full[s]), 64 * x, row,
                    h * p.hm[op[o]], b * p.bm[op[o]]);
  };
  if (tid == 0) {
    ms->abort_flag = 0;
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(bar(ms->full[s]), 1);
      mbar_init(bar(ms->empty[s]), DP > 64 ? 9 : 1);  // the last MMA's commit; rows staged over a
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(ms->s_full[s]), 1);
      mbar_init(bar(ms->p_full[s]), 8);
      mbar_init(bar(ms->pc_done[s]), 1);
      mbar_init(bar(ms->u_done[s]), 1);
      mbar_init(bar(ms->img_full[s]), DP / 16);
      mbar_init(bar(ms->bh_full[s]), C::kBT / 32);
    }
    mbar_init(bar(ms->x_full), DP / 16);
    mbar_init(bar(ms->qx_done), 1);
    mbar_init(bar(ms->o_full), 1);
    mbar_init(bar(ms->o_free), 8);
    mbar_init(bar(ms->drain), 1);
    fence_mbar_init();
    for (int i = 0; i < min(N, C::NS); ++i) load(i);  // in flight while the block sets up
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ms->tmem_base), C::kCols);
    tmem_relinquish();
  }
  if (tid >= 96 && tid <= 96 + kTok) {
    const int e = tid - 96;
    const float w = (float)dcy::decay_pow(p.log_decay[h], e);
    ms->pw[e] = w;
    if (e < 32) {
      ms->pwz[31 + e] = w;
      if (e < 31) ms->pwz[e] = 0.f;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  constexpr uint32_t tmem = 0;  // all 512 columns are this block's

  if (warp == 0) {
    // ------------------------------------------------------------ loads
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
    // ------------------------------------------------------------ MMAs
    // Straight-line for the whole warp: loop counters and descriptors stay in uniform registers, which a
    // divergent exit on a failed wait would forbid (an MMA then takes about 70 cycles to issue). After a
    // timeout every wait returns at once and the remaining products run on whatever shared memory holds.
    const uint32_t lead = elect_one();
    constexpr uint32_t id_s = idesc_f16(128, 128, 1, 1, 0, 0);
    constexpr uint32_t id_x = idesc_f16(128, DP, 1, 1, 0, 1);  // A X and P C
    constexpr uint32_t id_u = idesc_f16(128, DP, 1, 1, 1, 1);
    constexpr uint64_t kRows16 = (16 * 128) >> 4;  // 16 rows of an MN-major operand
    auto kmaj = [](int kk) { return uint64_t(((kk >> 2) * kAtomB + (kk & 3) * 32) >> 4); };
    // scores of chunk i into buffer i % SB
    auto scores = [&](int i) {
      const int s = i % C::NS, sb = i % C::SB;
      mbar_wait(bar(ms->full[s]), (i / C::NS) & 1, abort_flag);
      if (i >= C::SB) mbar_wait(bar(ms->pc_done[sb]), ((i / C::SB) - 1) & 1, abort_flag);
      tc_fence_after();
      const uint64_t db = sdesc_sw128(base + s * C::kStageB, 16, 1024);
      const uint64_t da = sdesc_sw128(base + s * C::kStageB + 2 * C::kOpB, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
        mma_ss_if(lead, tmem + C::kTS + sb * 128, da + kmaj(kk), db + kmaj(kk), id_s, kk > 0 ? 1u : 0u);
      commit_if(lead, bar(ms->s_full[sb]));
    };
    // X += (w B)^T C
    auto update = [&](int i, bool last) {  // last: of the chunk's products, as below
      const int s = i % C::NS;
      mbar_wait(bar(ms->full[s]), (i / C::NS) & 1, abort_flag);
      mbar_wait(bar(ms->x_full), i & 1, abort_flag);
      mbar_wait(bar(ms->bh_full[i & 1]), (i >> 1) & 1, abort_flag);
      tc_fence_after();
      const uint32_t st = base + s * C::kStageB, lo = base + C::kLo + (i % C::NLO) * C::kOpB;
      const uint64_t dc = sdesc_sw128(st + C::kOpB, kAtomB, 1024);
      const uint64_t dw = sdesc_sw128(st, DP == 64 ? lo - st : kAtomB, 1024);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ss_if(lead, tmem, dw + kk * kRows16, dc + kk * kRows16, id_u, 1u);
      if (DP > 64) {
        const uint64_t dl = sdesc_sw128(lo, kAtomB, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mma_ss_if(lead, tmem, dl + kk * kRows16, dc + kk * kRows16, id_u, 1u);
      }
      commit_if(lead, bar(ms->u_done[i & 1]));
      if (last) commit_if(lead, bar(ms->empty[s]));
    };
    // A X
    auto carried = [&](int i) {
      mbar_wait(bar(ms->img_full[i & 1]), (i >> 1) & 1, abort_flag);
      if (i >= 1) mbar_wait(bar(ms->o_free), (i - 1) & 1, abort_flag);
      tc_fence_after();
      const uint64_t da = sdesc_sw128(base + (i % C::NS) * C::kStageB + 2 * C::kOpB, 16, 1024);
      const uint64_t dx = sdesc_sw128(base + C::kX + (i % C::NX) * C::kOpB, kAtomB, 1024);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)  // 128 rows of X: hi and lo (d <= 64), or d
        mma_ss_if(lead, tmem + C::kTO1, da + kmaj(DP == 64 ? kk & 3 : kk), dx + kk * kRows16, id_x, kk > 0 ? 1u : 0u);
      if (DP > 64) commit_if(lead, bar(ms->qx_done));
    };
    // P C
    auto values = [&](int i, bool last) {
      const int s = i % C::NS, sb = i % C::SB;
      mbar_wait(bar(ms->p_full[sb]), (i / C::SB) & 1, abort_flag);
      tc_fence_after();
      const uint64_t dc = sdesc_sw128(base + s * C::kStageB + C::kOpB, kAtomB, 1024);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ts_if(lead, tmem + C::kTO2, tmem + C::kTS + sb * 128 + p_col(16 * kk), dc + kk * kRows16, id_x, kk > 0 ? 1u : 0u);
      commit_if(lead, bar(ms->o_full));
      commit_if(lead, bar(ms->pc_done[sb]));
      if (last) commit_if(lead, bar(ms->empty[s]));
    };
    // The next chunk's scores go first: they wait for the products P C that read their buffer, no more.
    // With one score buffer (d > 64) that is this chunk's; and the update follows A X, whose image its lo
    // operand overwrites, and P C, which lets the rows out start, but where the update's operand pass
    // zeroes c's tail.
    scores(0);
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      if (C::SB == 2) {
        if (i + 1 < N) scores(i + 1);
        update(i, false);
        carried(i);
        values(i, true);
      } else {
        const bool tail = tokens(i) < kTok;
        carried(i);
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          if ((k == 0) == tail)
            update(i, k == 1);
          else
            values(i, k == 1);
        }
        if (i + 1 < N) scores(i + 1);
      }
    }
    commit_if(lead, bar(ms->drain));
    __syncwarp();
    mbar_wait(bar(ms->drain), 0, nullptr, kWaitLimitCycles / 8);
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ w B and the state
    // w B in place (hi) and beside it (lo); thread = every (T / 8)-th row of each 64 columns.
    // State: thread = row of X (b's column). d <= 64: one warpgroup each, side by side. d > 64: the update
    // waits for w B, w B for A X (its lo lies over X's image) and A X for the state, so both warpgroups
    // take half the state's columns, then half of w B.
    constexpr int T = C::kBT;
    constexpr int NR = kTok / (T / 8);
    const bool does_b = DP > 64 || warp < 8, does_x = DP > 64 || warp >= 8;
    const int t = tid - 128, r0 = t >> 3;
    const int q4 = warp & 3, row = q4 * 32 + lane, half = DP > 64 ? t >> 7 : 0;
    const uint32_t la = uint32_t(q4 * 32) << 16;
    const uint64_t m1 = pair(-1.f, -1.f);
    float w[NR];
    int nw = 0;  // tokens the weights are for
    auto scale_b = [&](int i) -> bool {
      const int s = i % C::NS, n = tokens(i);
      if (n != nw) {
#pragma unroll
        for (int k = 0; k < NR; ++k) {
          const int r = r0 + k * (T / 8);
          w[k] = r < n ? ms->pw[rev ? r + 1 : n - 1 - r] : 0.f;
        }
        nw = n;
      }
      if (!mbar_wait(bar(ms->full[s]), (i / C::NS) & 1, abort_flag)) return false;
      // the lo buffer's last reader is update i - NLO
      if (i >= C::NLO && !mbar_wait(bar(ms->u_done[(i - C::NLO) & 1]), ((i - C::NLO) >> 1) & 1, abort_flag)) return false;
      if (!mbar_wait(bar(ms->s_full[i % C::SB]), (i / C::SB) & 1, abort_flag)) return false;  // B has been read
      if (DP > 64 && !mbar_wait(bar(ms->qx_done), i & 1, abort_flag)) return false;           // so has X's image
      uint8_t* hi = gb + s * C::kStageB + 16 * t;
      uint8_t* lo = gb + C::kLo + (i % C::NLO) * C::kOpB + 16 * t;
#pragma unroll 1
      for (int x = 0; x < C::NB; ++x) {
#pragma unroll
        for (int k0 = 0; k0 < NR; k0 += 4) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const uint4*>(hi + x * kAtomB + (k0 + k) * 16 * T);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t ww = pair(w[k0 + k], w[k0 + k]);
            uint32_t px[4] = {v[k].x, v[k].y, v[k].z, v[k].w}, py[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint64_t u = mul2(pair(px[q] << 16, px[q] & 0xffff0000u), ww);
              px[q] = pack2(u);
              py[q] = pack2(fma2(pair(px[q] << 16, px[q] & 0xffff0000u), m1, u));
            }
            if (n < kTok && r0 + (k0 + k) * (T / 8) >= n) {  // rows behind the end may hold anything
#pragma unroll
              for (int q = 0; q < 4; ++q) px[q] = py[q] = 0u;
            }
            *reinterpret_cast<uint4*>(hi + x * kAtomB + (k0 + k) * 16 * T) = make_uint4(px[0], px[1], px[2], px[3]);
            *reinterpret_cast<uint4*>(lo + x * kAtomB + (k0 + k) * 16 * T) = make_uint4(py[0], py[1], py[2], py[3]);
          }
        }
      }
      if (n < kTok) {  // rows of c behind the end take part in products with zero: they must be finite
        uint8_t* cc = gb + s * C::kStageB + C::kOpB;
        for (int e = t; e < C::kOpB / 16; e += T)
          if (((e >> 3) & (kTok - 1)) >= n) *reinterpret_cast<uint4*>(cc + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ms->bh_full[i & 1]));
      return true;
    };
    // The image of X for chunk i and X scaled for its update
    auto hand_on = [&](int i) {
      const float f = ms->pw[tokens(i)];
      const uint64_t ff = pair(f, f);
#pragma unroll 1
      for (int x = 2 * half; x < 2 * half + 2; ++x) {
        uint32_t v[32];
        tmem_ld32(tmem + la + 32 * x, v);
        tmem_wait_ld();
        {
          uint8_t* img = gb + C::kX + (i % C::NX) * C::kOpB + (x >> 1) * kAtomB + row * 128;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(img + ((((x & 1) * 4 + q) ^ (row & 7)) << 4)) =
                make_uint4(pack2(pair(v[8 * q], v[8 * q + 1])), pack2(pair(v[8 * q + 2], v[8 * q + 3])),
                           pack2(pair(v[8 * q + 4], v[8 * q + 5])), pack2(pair(v[8 * q + 6], v[8 * q + 7])));
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) unpair(mul2(pair(v[e], v[e + 1]), ff), v[e], v[e + 1]);
        tmem_st32(tmem + la + 32 * x, v);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ms->x_full));  // the update may go ahead
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ms->img_full[i & 1]));
    };
    auto updated = [&](int i) -> bool {
      const bool ok = mbar_wait(bar(ms->u_done[i & 1]), (i >> 1) & 1, abort_flag);
      tc_fence_after();
      return __all_sync(0xffffffffu, ok);
    };
    if (does_x) {  // X carried in, to TMEM
      if (x_in) pdl_wait();  // written by the kernel before
#pragma unroll 1
      for (int x = 2 * half; x < 2 * half + 2; ++x) {
        uint32_t v[32];
        load_state(v, x_in, x, row, d, job.trans);
        tmem_st32(tmem + la + 32 * x, v);
      }
      tmem_wait_st();
    }
    bool ok = true;
#pragma unroll 1
    for (int i = 0; ok && i < N; ++i) {
      if (does_x) {
        if (i > 0 && !(ok = updated(i - 1))) break;
        hand_on(i);
      }
      if (does_b) ok = scale_b(i);
    }
  } else if (warp >= 12 && warp < 20) {
    // ------------------------------------------------------------ scores -> P (thread = row, half the columns)
    const int q4 = warp & 3, row = q4 * 32 + lane, half = (warp - 12) >> 2;
    const uint32_t la = uint32_t(q4 * 32) << 16;
    const uint64_t l4 = pair(ms->pw[4], ms->pw[4]);
    const float* wz = ms->pwz + 31 + (rev ? -lane : lane);
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      const int sb = i % C::SB, n = tokens(i);
      if (!mbar_wait(bar(ms->s_full[sb]), (i / C::SB) & 1, abort_flag)) break;
      tc_fence_after();
      const uint32_t ts = tmem + la + C::kTS + sb * 128;
      // In order of columns: P's 16 columns of block x lie in scores of this half that are read, or
      // masked, by then.
#pragma unroll 1
      for (int x = 2 * half; x < 2 * half + 2; ++x) {
        const uint32_t tp = ts + p_col(32 * x);
        uint32_t pk[16];
        if (rev ? x < q4 : x > q4) {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0u;
        } else {
          uint32_t v[32];
          tmem_ld32(ts + 32 * x, v);
          if (x == q4) {  // lambda^|i-j|; a masked score may be anything, of a later token or behind the end
            tmem_wait_ld();
            if (rev) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                uint32_t u0, u1;
                unpair(mul2(pair(v[e], v[e + 1]), pair(wz[e], wz[e + 1])), u0, u1);
                pk[e / 2] = pack_bf16x2(__uint_as_float(e < lane ? 0u : u0), __uint_as_float(e + 1 < lane ? 0u : u1));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                uint32_t u0, u1;
                unpair(mul2(pair(v[e], v[e + 1]), pair(wz[-e], wz[-e - 1])), u0, u1);
                pk[e / 2] = pack_bf16x2(__uint_as_float(e > lane ? 0u : u0), __uint_as_float(e + 1 > lane ? 0u : u1));
              }
            }
          } else {
            // Weights run along the row by products with lambda^4, from the nearest token outwards: 8 roundings
            // of 2^-24 under P's own of 2^-8, and no shared-memory reads beside those of the MMAs.
            const float* near = ms->pw + (rev ? 32 * x - row : row - 32 * x - 31);
            uint64_t w0 = rev ? pair(near[0], near[1]) : pair(near[1], near[0]);
            uint64_t w1 = rev ? pair(near[2], near[3]) : pair(near[3], near[2]);
            tmem_wait_ld();
            if (rev) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                pk[e / 2] = pack2(mul2(pair(v[e], v[e + 1]), w0));
                pk[e / 2 + 1] = pack2(mul2(pair(v[e + 2], v[e + 3]), w1));
                w0 = mul2(w0, l4);
                w1 = mul2(w1, l4);
              }
            } else {
#pragma unroll
              for (int e = 28; e >= 0; e -= 4) {
                pk[e / 2 + 1] = pack2(mul2(pair(v[e + 2], v[e + 3]), w0));
                pk[e / 2] = pack2(mul2(pair(v[e], v[e + 1]), w1));
                w0 = mul2(w0, l4);
                w1 = mul2(w1, l4);
              }
            }
          }
          if (rev && n < 32 * x + 32) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              pk[e] = 32 * x + 2 * e + 1 < n ? pk[e] : 32 * x + 2 * e < n ? pk[e] & 0xffffu : 0u;
          }
        }
        tmem_st16(tp, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ms->p_full[sb]));
    }
  } else if (warp >= 20) {
    // ------------------------------------------------------------ rows out (thread = row, half the columns)
    const int q4 = warp & 3, row = q4 * 32 + lane, half = (warp - 20) >> 2;
    const uint32_t la = uint32_t(q4 * 32) << 16;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(job.y.p) + b * job.y.sb + h * job.y.sh;
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      const int s = i % C::NS, n = tokens(i);
      if (DP == 64) {
        if (lane == 0) bulk_wait_read0();  // the last chunk's rows have left their place
        __syncwarp();
      }
      if (!mbar_wait(bar(ms->o_full), i & 1, abort_flag)) break;
      tc_fence_after();
      const bool live = row < n;
      const float f = ms->pw[live ? (rev ? n - 1 - row : row + 1) : 0];
      const uint64_t ff = pair(f, f);
      const bool whole = 32 * q4 + 32 <= n;  // the warp's 32 rows leave as boxes of 32 columns
      const uint32_t slab = (DP == 64 ? C::kY : s * C::kStageB + 2 * C::kOpB) + q4 * (DP / 32) * 2048;
      __nv_bfloat16* yr = y + ((long long)chunk(i) * kTok + row) * job.y.st;
#pragma unroll 1
      for (int g = half * (DP / 32); g < (half + 1) * (DP / 32); ++g) {  // 16 columns
        uint32_t o1[16], o2[16];
        tmem_ld16(tmem + la + C::kTO2 + 16 * g, o2);
        tmem_ld16(tmem + la + C::kTO1 + 16 * g, o1);
        tmem_wait_ld();
        uint64_t z2 = 0ull, z3 = 0ull;  // NaN if any is not finite
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          z2 = fma2(pair(o2[e], o2[e + 1]), 0ull, z2);
          z3 = fma2(pair(o2[e + 2], o2[e + 3]), 0ull, z3);
        }
        uint32_t za, zb;
        unpair(fma2(z3, 0ull, z2), za, zb);
        if (__any_sync(0xffffffffu, live && !(__uint_as_float(za) + __uint_as_float(zb) == 0.f))) {
          // An infinity or NaN in this chunk's a, b or c. Sum again, over the row's own tokens, the elements that may
          // yet be finite: where A X is not finite (the row's own a, or a token of an earlier chunk), neither is the
          // result. So a column is summed again in one chunk of a walk at most, and there until its sum is not finite.
          uint32_t need = 0u;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (live && !(__uint_as_float(o2[e]) * 0.f == 0.f) && __uint_as_float(o1[e]) * 0.f == 0.f) need |= 1u << e;
          const long long t0 = (long long)chunk(i) * kTok;
          const __nv_bfloat16* ga = row_of(job.va, b, h, t0 + (live ? row : 0));
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            const int col = 16 * g + 8 * q;
            const uint32_t nq = need >> (8 * q) & 0xffu;
            if (col >= d || !nq) continue;
            float acc[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.f;
            const int j1 = rev ? n : row + 1;
#pragma unroll 1
            for (int j = rev ? row : 0; j < j1; ++j) {
              const __nv_bfloat16* gbj = row_of(job.vb, b, h, t0 + j);
              float sc = 0.f;
#pragma unroll 1
              for (int m = 0; m < d; m += 8) {
                float x[8], z[8];
                load8(x, ga + m);
                load8(z, gbj + m);
#pragma unroll
                for (int e = 0; e < 8; ++e) sc = fmaf(x[e], z[e], sc);
              }
              sc *= ms->pw[rev ? j - row : row - j];
              float z[8];
              load8(z, row_of(job.vc, b, h, t0 + j) + col);
              bool open = false;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                acc[e] = fmaf(sc, z[e], acc[e]);
                open = open || ((nq >> e & 1u) && acc[e] * 0.f == 0.f);
              }
              if (!open) break;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if ((e >> 3) == q && (nq >> (e & 7) & 1u)) o2[e] = __float_as_uint(acc[e & 7]);
          }
          __syncwarp();
        }
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = pack2(fma2(ff, pair(o1[2 * e], o1[2 * e + 1]), pair(o2[2 * e], o2[2 * e + 1])));
        if (whole) {  // 32 rows of 64 bytes, 64-byte swizzle
          uint8_t* ys = gb + slab + (g >> 1) * 2048 + lane * 64;
#pragma unroll
          for (int q = 0; q < 2; ++q)
            *reinterpret_cast<uint4*>(ys + ((((g & 1) * 2 + q) ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        } else if (live) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (16 * g + 8 * q < d)
              *reinterpret_cast<uint4*>(yr + 16 * g + 8 * q) = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ms->o_free));  // the accumulators are read
      if (whole) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (whole) {
#pragma unroll
          for (int x = half * (DP / 64); x < (half + 1) * (DP / 64); ++x)
            if (32 * x < d) tma_store_4d(&p.my[jid], base + slab + x * 2048, 32 * x, chunk(i) * kTok + 32 * q4, h, b);
          bulk_commit();
        }
        if (DP > 64) {
          bulk_wait_read0();  // the rows lie in the stage
          mbar_arrive(bar(ms->empty[s]));
        }
      }
    }
    if (lane == 0) bulk_wait0();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(ms->tmem_base, C::kCols);
  }
}

template <int DP>
__global__ void __launch_bounds__(Cfg<DP>::kThreads, 1) k_decay_walk(const __grid_constant__ Params p) {
  walk_block<DP>(p, blockIdx.x);
}

}  // namespace dtc
}  // namespace favor
