// host_decay.cuh - host side of the decayed linear attention and rotary entry points: argument
// checks, scratch, launches. Included by favor_lib.cu after its helpers.
#pragma once
#include <cmath>

#include "kernel_decay_state.cuh"
#include "kernel_decay_step.cuh"
#include "kernel_decay_tc.cuh"
#include "kernel_rotary.cuh"
#include "kernels_decay.cuh"

namespace {

using favor::dcy::View;
namespace dcy = favor::dcy;

// Strides of operand `i` of a call ([B, H, L, d] contiguous where none are given). Inputs may
// repeat (stride 0); the offset of the last element stays below 2^42.
int make_view(View* v, const void* p, const favor_strides* s, int i, int B, int H, int L, int d) {
  v->p = const_cast<void*>(p);
  if (!s) {
    v->st = d;
    v->sh = (long long)L * d;
    v->sb = (long long)H * L * d;
    return FAVOR_OK;
  }
  v->sb = s[i].batch;
  v->sh = s[i].head;
  v->st = s[i].token;
  const long long lim = 1ll << 42;
  if (v->sb < 0 || v->sh < 0 || v->st < 0) return FAVOR_ERR_SHAPE;
  // a dimension of one element takes no step
  if (B == 1) v->sb = 0;
  if (H == 1) v->sh = 0;
  if (L == 1) v->st = 0;
  if (v->sb > lim || v->sh > lim || v->st > lim) return FAVOR_ERR_SHAPE;
  const double last = (double)(B - 1) * v->sb + (double)(H - 1) * v->sh + (double)(L - 1) * v->st + d;
  return last < (double)lim ? FAVOR_OK : FAVOR_ERR_SHAPE;
}

// Where an operand's rows are whole 16-byte pieces they are moved as such, and its base must lie on one; other rows
// are read element by element, and slices of them start anywhere.
bool view_aligned(const View& v, int d, int dtype_code) {
  const int es = dtype_code == 1 ? 2 : 4, n = 16 / es;
  const bool pieces = d % n == 0 && v.sb % n == 0 && v.sh % n == 0 && v.st % n == 0;
  return (reinterpret_cast<uintptr_t>(v.p) & (pieces ? 15u : es - 1u)) == 0;
}

// An output's rows must not overlap one another: in order of stride, each dimension steps past
// everything the smaller ones span.
bool rows_distinct(const View& v, int B, int H, int L, int d) {
  long long st[3] = {v.sb, v.sh, v.st}, n[3] = {B, H, L};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (st[j] > st[j + 1]) std::swap(st[j], st[j + 1]), std::swap(n[j], n[j + 1]);
  long long span = d;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (st[i] < span) return false;
    span += (n[i] - 1) * st[i];
  }
  return true;
}

int check_decay_sizes(int B, int H, int L, int d, int dtype_code) {
  if (B <= 0 || H <= 0 || L <= 0 || d <= 0) return FAVOR_ERR_SHAPE;
  if ((long long)B * H > INT_MAX / 2 || (long long)B * H * L > (1ll << 40) || (long long)B * H * L * d > (1ll << 40))
    return FAVOR_ERR_SHAPE;
  if (d > dcy::kMaxD || (dtype_code != 0 && dtype_code != 1)) return FAVOR_ERR_UNSUPPORTED;
  return FAVOR_OK;
}

int decay_chunks(int L) { return (int)(((long long)L + dcy::kChunk - 1) / dcy::kChunk); }

size_t decay_cc_workspace(int B, int H, int L, int d, int nstates) {
  return (size_t)nstates * B * H * decay_chunks(L) * d * d * sizeof(float);
}

// A launch that may start while the kernel before it in the stream drains (the kernel waits for that
// one's results itself) where `pdl` is set. Its own status alone is looked at: an error that an earlier call of the
// process left behind is not this call's, and one of this call is not left for the next.
template <typename P>
int launch_with(void (*kern)(P), dim3 grid, int threads, int smem, cudaStream_t st, bool pdl, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess) return FAVOR_OK;
  cudaGetLastError();
  return FAVOR_ERR_CUDA;
}

// The scan over `nseg` segments of `seg` tokens whose updates lie in ws.
int launch_scan(const dcy::Params& p, float* ws, int nseg, int seg, cudaStream_t st) {
  dcy::ScanParams sp{};
  for (int i = 0; i < p.nstates; ++i) {
    sp.in[i] = p.s[i].in;
    sp.out[i] = p.s[i].out;
    sp.reverse[i] = p.s[i].reverse;
  }
  sp.ws = ws;
  sp.log_decay = p.log_decay;
  sp.lengths = p.lengths;
  sp.nstates = p.nstates, sp.B = p.B, sp.H = p.H, sp.L = p.L, sp.d = p.d, sp.nseg = nseg, sp.seg = seg;
  const long long grid = (long long)p.B * p.H * p.nstates * ((p.d * p.d + dcy::kThreads - 1) / dcy::kThreads);
  if (grid > INT_MAX) return FAVOR_ERR_UNSUPPORTED;
  // 32 segments' loads in flight where there are many, 8 (a third of the registers, so more blocks an SM) where few.
  // Measured, whole fp32 calls of d = 64 in us, 8 against 32. 16 heads: 16 segments 29.0 and 30.2, 32 46.1 and 47.5, 48
  // 60.7 and 60.5, 64 79.6 and 77.9, 96 123 and 115, 128 161 and 150. One head: 32 segments 15.2 and 14.8, 64 18.8 and
  // 18.0, 1024 201 and 165. 256 heads of 2 segments 52 and 83. Between 24 and 64 either does.
  return nseg >= 64 ? launch_with<dcy::ScanParams>(dcy::k_chunk_scan<32>, grid, dcy::kThreads, 0, st, true, sp)
                    : launch_with<dcy::ScanParams>(dcy::k_chunk_scan<8>, grid, dcy::kThreads, 0, st, true, sp);
}

template <typename T, int DP>
int launch_decay_cc_t(const dcy::Params& p, cudaStream_t st) {
  const long long heads = (long long)p.B * p.H;
  const long long g_up = heads * p.nstates * p.nch, g_out = heads * p.nouts * p.nch;
  if (g_up > INT_MAX || g_out > INT_MAX) return FAVOR_ERR_UNSUPPORTED;
  auto ku = dcy::k_chunk_update<T, DP>;
  auto ko = dcy::k_chunk_out<T, DP>;
  if (ensure_smem_attr(reinterpret_cast<const void*>(ku), dcy::update_smem(DP)) != FAVOR_OK ||
      ensure_smem_attr(reinterpret_cast<const void*>(ko), dcy::out_smem(DP)) != FAVOR_OK)
    return FAVOR_ERR_CUDA;
  int rc = launch_with<dcy::Params>(ku, g_up, dcy::kThreads, dcy::update_smem(DP), st, false, p);
  if (rc == FAVOR_OK) rc = launch_scan(p, p.ws, p.nch, dcy::kChunk, st);
  if (rc == FAVOR_OK) rc = launch_with<dcy::Params>(ko, g_out, dcy::kThreads, dcy::out_smem(DP), st, true, p);
  return rc;
}

// The CUDA-core route: every type, head size and stride.
int launch_decay_cc(dcy::Params p, int dtype_code, cudaStream_t st) {
  p.nch = decay_chunks(p.L);
  void* ws = nullptr;
  int rc = scratch_alloc(&ws, decay_cc_workspace(p.B, p.H, p.L, p.d, p.nstates), st);
  if (rc != FAVOR_OK) return rc;
  p.ws = static_cast<float*>(ws);
  p.vec = dtype_code == 0 && p.d % 4 == 0;
  for (int i = 0; i < p.nouts; ++i)
    for (const View* v : {&p.o[i].a, &p.o[i].b, &p.o[i].c, &p.o[i].y})
      if (v->sb % 4 != 0 || v->sh % 4 != 0 || v->st % 4 != 0) p.vec = 0;
  if (dtype_code == 0)
    rc = p.d <= 64 ? launch_decay_cc_t<float, 64>(p, st) : launch_decay_cc_t<float, 128>(p, st);
  else
    rc = p.d <= 64 ? launch_decay_cc_t<__nv_bfloat16, 64>(p, st) : launch_decay_cc_t<__nv_bfloat16, 128>(p, st);
  cudaFreeAsync(ws, st);
  return rc;
}

// ------------------------------------------------------------------ tensor-core route
// How a call's walk is cut: chunks per segment, segments. `scan` (several segments): segment states,
// their scan and the walk, three launches; else one walk per head from the carried-in state, and the states a
// caller wants back.
struct WalkPlan {
  int cps, nseg;
  bool scan;
};

// The number of segments with the least estimated time, in microseconds. The estimate: a block of the walk takes
// 3 and 1.55 (d <= 64) or 2.95 a chunk, one of the states 3 and 1.0 or 2.2 a chunk, the scan and the gaps of
// two further launches 7 and its traffic at 3 TB/s. The terms were fitted together, on whole calls with an earlier state
// kernel; the present one takes 1.3 and 2.0 a chunk by itself. States that a caller wants back cost nothing more
// with segments; without, their own pass over b and c, beside the walk, is not in the estimate.
// Measured on the device, the pick against the best of 1 to 128 segments: prompts of 4 x 8 heads x 4096 tokens, d = 64,
// 33.0 and 32.9; 16 x 65536 165 and 165; 65536 tokens of one head 31.4 and 31.4; 32 x 4096, d = 128, 62 and 62;
// 8 x 8192, d = 128, 46.5 and 43.8; gradients 8 x 4096, d = 64, 27.7 and 27.7; 4 x 8 x 4096 47.2 and 47.2; 16 x 4096,
// d = 128, 76 and 76. It misses on short prompts of few heads: 8 x 2048, d = 64, 16 segments 19.1 and 8 14.2; 2 x 8 x
// 1024 with states, one segment 18.1 and 4 14.5.
WalkPlan plan_walk(int BH, int L, int d, int nstates, int njobs) {
  const int nch = (int)(((long long)L + dtc::kTok - 1) / dtc::kTok), sms = sm_count();
  const double tw = d <= 64 ? 1.55 : 2.95, ts = d <= 64 ? 1.0 : 2.2;
  auto waves = [&](long long ctas) { return (double)((ctas + sms - 1) / sms); };
  WalkPlan best{};
  double cost = 1e300;
  for (int k = 1; k <= std::min(nch, 1024); ++k) {
    const int cps = (nch + k - 1) / k, nseg = (nch + cps - 1) / cps;
    if (nseg != k) continue;  // as many segments as the chunks per segment need
    double t = waves((long long)BH * njobs * nseg) * (tw * cps + 3.0);
    if (k > 1) t += waves((long long)BH * nstates * nseg) * (ts * cps + 3.0) + 7.0 + 8.0 * BH * nstates * nseg * d * d / 3e6;
    if (t < cost) cost = t, best = WalkPlan{cps, nseg, k > 1};
    if ((long long)BH * nseg > 8ll * sms) break;
  }
  return best;
}

// Operands the tensor-core route reads in place: bf16 rows and strides of whole 16-byte pieces.
bool tc_view_ok(const View& v) {
  const long long lim = 1ll << 39;
  for (long long s : {v.sb, v.sh, v.st})
    if (s % 8 != 0 || s >= lim) return false;
  return true;
}

// Everything they can read goes to the tensor cores. Measured against the CUDA-core route on the device, 8 heads,
// d = 64: one token 5.8 and 13.0 us, 128 tokens 6.0 and 27.5; 128 heads x 512 tokens of d = 128 16 and 380.
bool tc_route(const dcy::Params& p, int dtype_code) {
  if (dtype_code != 1 || p.d % 8 != 0) return false;
  for (int i = 0; i < p.nouts; ++i)
    for (const View* v : {&p.o[i].a, &p.o[i].b, &p.o[i].c, &p.o[i].y})
      if (!tc_view_ok(*v) || (v != &p.o[i].y && p.L > 1 && v->st == 0)) return false;
  return true;
}

// [B][H][L][d] bf16 in boxes of 64 columns x 128 tokens (128-byte swizzle), an output in boxes of
// 32 x 32 (64-byte swizzle). A dimension an operand repeats over (stride
// 0) is a dimension of one, walked at coordinate 0: bm, hm.
bool make_map_view(CUtensorMap* m, int* bm, int* hm, const View& v, int B, int H, int L, int d, bool output) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  *bm = v.sb != 0, *hm = v.sh != 0;
  const cuuint64_t row = (cuuint64_t)(d + 7) / 8 * 16;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)L, (cuuint64_t)(*hm ? H : 1), (cuuint64_t)(*bm ? B : 1)};
  const cuuint64_t strides[3] = {v.st ? (cuuint64_t)v.st * 2 : row, v.sh ? (cuuint64_t)v.sh * 2 : row,
                                 v.sb ? (cuuint64_t)v.sb * 2 : row};
  const cuuint32_t box[4] = {output ? 32u : 64u, output ? 32u : 128u, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            output ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t walk_workspace(const WalkPlan& pl, int BH, int d, int nstates) {
  return pl.scan ? (size_t)nstates * BH * pl.nseg * d * d * sizeof(float) : 0;
}

// Tensor maps of a call's operands, by pointer and strides: forward q, k, v; backward q, k, v, dout.
struct OperandMaps {
  CUtensorMap m[4];
  int bm[4], hm[4], n = 0;
  View seen[4];
  int add(const View& v, const dcy::Params& p) {
    for (int i = 0; i < n; ++i)
      if (seen[i].p == v.p && seen[i].sb == v.sb && seen[i].sh == v.sh && seen[i].st == v.st) return i;
    if (n == 4 || !make_map_view(&m[n], &bm[n], &hm[n], v, p.B, p.H, p.L, p.d, false)) return -1;
    seen[n] = v;
    return n++;
  }
};

void set_maps(const OperandMaps& om, CUtensorMap* m, int* bm, int* hm) {
  std::copy(om.m, om.m + 4, m);
  std::copy(om.bm, om.bm + 4, bm);
  std::copy(om.hm, om.hm + 4, hm);
}

// The states in p.s that have a use: every segment's (ws), or the whole sequences' written to their `out`.
int state_params(dst::Params& sp, const dcy::Params& p, OperandMaps& om, float* ws, int nseg, int cps) {
  for (int i = 0; i < p.nstates; ++i) {
    if (!ws && !p.s[i].out) continue;
    dst::Job& j = sp.j[sp.njobs++];
    j.b = om.add(p.s[i].b, p);
    j.c = om.add(p.s[i].c, p);
    if (j.b < 0 || j.c < 0) return FAVOR_ERR_CUDA;
    j.reverse = p.s[i].reverse;
    j.in = p.s[i].in;
    j.out = p.s[i].out;
  }
  set_maps(om, sp.m, sp.bm, sp.hm);
  sp.ws = ws;
  sp.log_decay = p.log_decay;
  sp.lengths = p.lengths;
  sp.B = p.B, sp.H = p.H, sp.L = p.L, sp.d = p.d, sp.nseg = nseg, sp.cps = cps;
  return FAVOR_OK;
}

int walk_params(dtc::Params& tp, const dcy::Params& p, OperandMaps& om, const float* ws, const WalkPlan& pl) {
  tp.njobs = p.nouts;
  for (int i = 0; i < p.nouts; ++i) {
    dtc::Job& j = tp.j[i];
    j.a = om.add(p.o[i].a, p);
    j.b = om.add(p.o[i].b, p);
    j.c = om.add(p.o[i].c, p);
    if (j.a < 0 || j.b < 0 || j.c < 0) return FAVOR_ERR_CUDA;
    j.state = p.o[i].state;
    j.trans = p.o[i].trans;
    j.reverse = p.o[i].reverse;
    j.va = p.o[i].a, j.vb = p.o[i].b, j.vc = p.o[i].c, j.y = p.o[i].y;
    int bm, hm;
    if (!make_map_view(&tp.my[i], &bm, &hm, j.y, p.B, p.H, p.L, p.d, true)) return FAVOR_ERR_CUDA;
  }
  set_maps(om, tp.m, tp.bm, tp.hm);
  for (int i = 0; i < p.nstates; ++i) tp.in[i] = p.s[i].in;
  tp.ws = ws;
  tp.log_decay = p.log_decay;
  tp.lengths = p.lengths;
  tp.B = p.B, tp.H = p.H, tp.L = p.L, tp.d = p.d, tp.nseg = pl.nseg, tp.cps = pl.cps;
  return FAVOR_OK;
}

template <typename P>
int launch_blocks(void (*k)(P), long long grid, int threads, int smem, bool pdl, const P& p, cudaStream_t st) {
  if (ensure_smem_attr(reinterpret_cast<const void*>(k), smem) != FAVOR_OK) return FAVOR_ERR_CUDA;
  return launch_with<P>(k, grid, threads, smem, st, pdl, p);
}

template <int DP>
int launch_decay_tc_t(const dcy::Params& p, const WalkPlan& pl, float* ws, cudaStream_t st) {
  using WC = dtc::Cfg<DP>;
  using SC = dst::Cfg<DP>;
  const long long heads = (long long)p.B * p.H;
  if (heads * pl.nseg * 5 > INT_MAX) return FAVOR_ERR_UNSUPPORTED;
  OperandMaps om;
  dst::Both both{};
  dtc::Params& tp = both.w;
  dst::Params& sp = both.s;
  int rc = walk_params(tp, p, om, ws, pl);
  if (rc == FAVOR_OK) rc = state_params(sp, p, om, ws, pl.nseg, pl.cps);
  if (rc != FAVOR_OK) return rc;
  set_maps(om, tp.m, tp.bm, tp.hm);
  const long long nwalk = heads * pl.nseg * p.nouts, nstate = heads * pl.nseg * sp.njobs;
  if (pl.scan) {
    rc = launch_blocks(dst::k_decay_state<DP>, nstate, SC::kThreads, SC::kSmem, false, sp, st);
    if (rc == FAVOR_OK) rc = launch_scan(p, ws, pl.nseg, pl.cps * dtc::kTok, st);
    if (rc == FAVOR_OK) rc = launch_blocks(dtc::k_decay_walk<DP>, nwalk, WC::kThreads, WC::kSmem, true, tp, st);
    return rc;
  }
  if (!sp.njobs) return launch_blocks(dtc::k_decay_walk<DP>, nwalk, WC::kThreads, WC::kSmem, false, tp, st);
  // The whole sequences' states: in the walk's own launch where the call is short (one block an SM, eight chunks
  // at most), since a second launch costs about 3 us but the joint kernel has the walk's few registers a thread for the
  // states too; else beside the walk, or after it where they overwrite what it reads. Measured on the device, two
  // launches against one, prompts of 8 heads with states: d = 64, 1 chunk 11.0 and 7.9 us, 2 12.0 and 9.0, 4 13.9 and
  // 11.7, 8 18.2 and 18.0, 12 22.6 and 24.2, 16 27.0 and 30.6; d = 128, 2 chunks 17.0 and 16.1, 8 30.4 and 29.7, 16
  // 52.8 and 51.2. 74 heads of d = 128: 4 chunks 22.3 and 21.8, 8 32.1 and 33.0, 12 43.3 and 46.1.
  bool in_place = false;
  for (int i = 0; i < p.nstates; ++i) in_place = in_place || (p.s[i].out && p.s[i].out == p.s[i].in);
  if (!in_place && nwalk + nstate <= sm_count() && pl.cps <= 8) {
    both.nwalk = (int)nwalk;
    return launch_blocks(dst::k_decay_both<DP>, nwalk + nstate, WC::kThreads, std::max(WC::kSmem, SC::kSmem), false,
                         both, st);
  }
  rc = launch_blocks(dtc::k_decay_walk<DP>, nwalk, WC::kThreads, WC::kSmem, false, tp, st);
  return rc == FAVOR_OK ? launch_blocks(dst::k_decay_state<DP>, nstate, SC::kThreads, SC::kSmem, !in_place, sp, st) : rc;
}

int launch_decay_tc(const dcy::Params& p, cudaStream_t st) {
  const WalkPlan pl = plan_walk(p.B * p.H, p.L, p.d, p.nstates, p.nouts);
  void* ws = nullptr;
  int rc = scratch_alloc(&ws, walk_workspace(pl, p.B * p.H, p.d, p.nstates), st);
  if (rc != FAVOR_OK) return rc;
  rc = p.d <= 64 ? launch_decay_tc_t<64>(p, pl, static_cast<float*>(ws), st)
                 : launch_decay_tc_t<128>(p, pl, static_cast<float*>(ws), st);
  if (ws) cudaFreeAsync(ws, st);
  return rc;
}

int launch_decay(const dcy::Params& p, int dtype_code, cudaStream_t st) {
  return tc_route(p, dtype_code) ? launch_decay_tc(p, st) : launch_decay_cc(p, dtype_code, st);
}

bool bad_align(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return true;
  return false;
}

template <typename T>
int launch_decay_step(const dcy::StepParams& p0, int BH, int d, cudaStream_t st) {
  dcy::StepParams p = p0;
  const bool vec = d % 4 == 0;
  // Slices of 32 columns (whole 128-byte row pieces) while all heads' slices are one block an SM at most, else
  // whole rows. Measured, slices against whole rows: 8 heads of d = 64 2.49 and 2.56 us, 32 heads of d = 128 2.99
  // and 3.99; past an SM each, 128 heads of d = 64 3.05 and 2.79, 4096 heads 34.2 and 20.2.
  p.cols = d <= 32 || (long long)BH * ((d + 31) / 32) > sm_count() ? d : 32;
  p.slices = (d + p.cols - 1) / p.cols;
  if ((long long)BH * p.slices > INT_MAX) return FAVOR_ERR_UNSUPPORTED;
  const unsigned grid = (unsigned)((long long)BH * p.slices);
  return launch_with<dcy::StepParams>(vec ? dcy::k_decay_step<T, 4, 8> : dcy::k_decay_step<T, 1, 8>, grid,
                                      dcy::kStepThreads, 0, st, false, p);
}

template <typename T, int V, bool INTER>
int launch_rotary_t(favor::rot::Params p, cudaStream_t st) {
  p.npair = p.rot / 2 / V;
  p.npass = (p.d - p.rot) / V;
  const long long items = (long long)p.B * p.L * (p.npair + p.npass);
  const long long blocks = (items + favor::rot::kThreads - 1) / favor::rot::kThreads;
  const int heads = p.Hq + p.Hk, sms = sm_count();
  // every head in one thread, unless that leaves fewer than eight blocks an SM. Measured at 4 x 4096 tokens of 16
  // heads: 2 groups 13.7 us, 4 groups 15.9, 8 groups 18.2; one token of 64 sequences and 20 heads: 20 groups 2.8
  p.groups = (int)std::max<long long>(1, std::min<long long>(heads, 8ll * sms / std::max<long long>(1, blocks)));
  p.per_group = (heads + p.groups - 1) / p.groups;
  p.groups = (heads + p.per_group - 1) / p.per_group;
  const unsigned gx = (unsigned)std::min<long long>(blocks, 64ll * sms);
  if (p.groups > 65535) return FAVOR_ERR_UNSUPPORTED;
  return launch_with<favor::rot::Params>(favor::rot::k_rotary<T, V, INTER>, dim3(gx, p.groups), favor::rot::kThreads, 0,
                                         st, false, p);
}

template <typename T>
int launch_rotary(const favor::rot::Params& p, int interleaved, bool strides_ok, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  // 16-byte pieces where every row starts on one and the pairs and the rest fill whole ones, else single
  // elements, which take any row
  const bool vec = strides_ok && (p.rot / 2) % V == 0 && (p.d - p.rot) % V == 0;
  if (interleaved) return vec ? launch_rotary_t<T, V, true>(p, st) : launch_rotary_t<T, 1, true>(p, st);
  return vec ? launch_rotary_t<T, V, false>(p, st) : launch_rotary_t<T, 1, false>(p, st);
}

}  // namespace

extern "C" {

size_t favor_decay_workspace_bytes(int B, int H, int L, int d, int dtype_code, int backward) {
  if (check_decay_sizes(B, H, L, d, dtype_code) != FAVOR_OK) return 0;
  const int ns = backward ? 2 : 1;
  if (dtype_code == 1 && d % 8 == 0)
    return walk_workspace(plan_walk(B * H, L, d, ns, backward ? 3 : 1), B * H, d, ns);
  return decay_cc_workspace(B, H, L, d, ns);
}

int favor_decay_attention(const void* q, const void* k, const void* v, const float* log_decay, const float* state_in,
                          const int* lengths, void* out, float* state_out, int B, int H, int L, int d,
                          int dtype_code, const favor_strides* strides, void* stream) {
  if (!q || !k || !v || !log_decay || !out) return FAVOR_ERR_NULL;
  if (bad_align({state_in, state_out}) || ((uintptr_t)log_decay & 3) || ((uintptr_t)lengths & 3))
    return FAVOR_ERR_ALIGN;
  int rc = check_decay_sizes(B, H, L, d, dtype_code);
  if (rc != FAVOR_OK) return rc;
  dcy::Params p{};
  View vq, vk, vv, vo;
  if ((rc = make_view(&vq, q, strides, 0, B, H, L, d)) != FAVOR_OK ||
      (rc = make_view(&vk, k, strides, 1, B, H, L, d)) != FAVOR_OK ||
      (rc = make_view(&vv, v, strides, 2, B, H, L, d)) != FAVOR_OK ||
      (rc = make_view(&vo, out, strides, 3, B, H, L, d)) != FAVOR_OK)
    return rc;
  for (const View* x : {&vq, &vk, &vv, &vo})
    if (!view_aligned(*x, d, dtype_code)) return FAVOR_ERR_ALIGN;
  if (!rows_distinct(vo, B, H, L, d)) return FAVOR_ERR_SHAPE;
  if (out == q || out == k || out == v) return FAVOR_ERR_UNSUPPORTED;
  if ((rc = check_device()) != FAVOR_OK) return rc;
  p.s[0] = {vk, vv, state_in, state_out, 0};
  p.o[0] = {vq, vk, vv, vo, 0, 0, 0};
  p.nstates = p.nouts = 1;
  p.log_decay = log_decay;
  p.lengths = lengths;
  p.B = B, p.H = H, p.L = L, p.d = d;
  return launch_decay(p, dtype_code, static_cast<cudaStream_t>(stream));
}

int favor_decay_attention_backward(const void* q, const void* k, const void* v, const float* log_decay,
                                   const float* state_in, const int* lengths, const void* dout,
                                   const float* dstate_out, void* dq, void* dk, void* dv, float* dstate_in, int B,
                                   int H, int L, int d, int dtype_code, const favor_strides* strides, void* stream) {
  if (!q || !k || !v || !log_decay || !dout || !dq || !dk || !dv) return FAVOR_ERR_NULL;
  if (bad_align({state_in, dstate_out, dstate_in}) || ((uintptr_t)log_decay & 3) || ((uintptr_t)lengths & 3))
    return FAVOR_ERR_ALIGN;
  int rc = check_decay_sizes(B, H, L, d, dtype_code);
  if (rc != FAVOR_OK) return rc;
  View x[7];
  const void* ptr[7] = {q, k, v, dout, dq, dk, dv};
  for (int i = 0; i < 7; ++i)
    if ((rc = make_view(&x[i], ptr[i], strides, i, B, H, L, d)) != FAVOR_OK) return rc;
  for (const View& v : x)
    if (!view_aligned(v, d, dtype_code)) return FAVOR_ERR_ALIGN;
  for (int i = 4; i < 7; ++i) {
    if (!rows_distinct(x[i], B, H, L, d)) return FAVOR_ERR_SHAPE;
    for (int j = 0; j < i; ++j)
      if (ptr[i] == ptr[j]) return FAVOR_ERR_UNSUPPORTED;
  }
  // the gradient of the carried-in state may overwrite dstate_out, not the state that dq still reads
  if (dstate_in && dstate_in == state_in) return FAVOR_ERR_UNSUPPORTED;
  if ((rc = check_device()) != FAVOR_OK) return rc;
  dcy::Params p{};
  p.s[0] = {x[1], x[2], state_in, nullptr, 0};      // S: k, v
  p.s[1] = {x[0], x[3], dstate_out, dstate_in, 1};  // G: q, dout
  p.o[0] = {x[3], x[2], x[1], x[4], 0, 1, 0};       // dq = S dout
  p.o[1] = {x[2], x[3], x[0], x[5], 1, 1, 1};       // dk = G v
  p.o[2] = {x[1], x[0], x[3], x[6], 1, 0, 1};       // dv = G^T k
  p.nstates = 2;
  p.nouts = 3;
  p.log_decay = log_decay;
  p.lengths = lengths;
  p.B = B, p.H = H, p.L = L, p.d = d;
  return launch_decay(p, dtype_code, static_cast<cudaStream_t>(stream));
}

int favor_decay_step(const void* q, const void* k, const void* v, const float* log_decay, float* state, void* out,
                     int B, int H, int d, int dtype_code, const favor_strides* strides, void* stream) {
  if (!q || !k || !v || !log_decay || !state || !out) return FAVOR_ERR_NULL;
  if (bad_align({state}) || ((uintptr_t)log_decay & 3)) return FAVOR_ERR_ALIGN;
  int rc = check_decay_sizes(B, H, 1, d, dtype_code);
  if (rc != FAVOR_OK) return rc;
  dcy::StepParams p{};
  if ((rc = make_view(&p.q, q, strides, 0, B, H, 1, d)) != FAVOR_OK ||
      (rc = make_view(&p.k, k, strides, 1, B, H, 1, d)) != FAVOR_OK ||
      (rc = make_view(&p.v, v, strides, 2, B, H, 1, d)) != FAVOR_OK ||
      (rc = make_view(&p.y, out, strides, 3, B, H, 1, d)) != FAVOR_OK)
    return rc;
  for (const View* x : {&p.q, &p.k, &p.v, &p.y})
    if (!view_aligned(*x, d, dtype_code)) return FAVOR_ERR_ALIGN;
  if (!rows_distinct(p.y, B, H, 1, d)) return FAVOR_ERR_SHAPE;
  if (out == q || out == k || out == v) return FAVOR_ERR_UNSUPPORTED;
  if ((rc = check_device()) != FAVOR_OK) return rc;
  p.log_decay = log_decay;
  p.state = state;
  p.H = H, p.d = d;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype_code == 0 ? launch_decay_step<float>(p, B * H, d, st)
                         : launch_decay_step<__nv_bfloat16>(p, B * H, d, st);
}

int favor_rotary(const void* q, const void* k, const double* freq, const int* positions, void* q_out, void* k_out,
                 int B, int Hq, int Hk, int L, int d, int rot, int interleaved, int inverse, int first_position,
                 float scale, float rot_scale, int dtype_code, const favor_strides* strides, void* stream) {
  if (!q || !freq || !q_out || (Hk > 0 && (!k || !k_out))) return FAVOR_ERR_NULL;
  if (Hk < 0) return FAVOR_ERR_SHAPE;
  if (((uintptr_t)freq & 7) || ((uintptr_t)positions & 3)) return FAVOR_ERR_ALIGN;
  if (B <= 0 || Hq <= 0 || L <= 0 || d <= 0 || rot <= 0 || rot % 2 != 0 || rot > d) return FAVOR_ERR_SHAPE;
  const long long heads = (long long)Hq + Hk;
  if ((double)B * heads * L * d > (double)(1ll << 40)) return FAVOR_ERR_SHAPE;
  if (heads > 65535 || d > 65536 || (dtype_code != 0 && dtype_code != 1)) return FAVOR_ERR_UNSUPPORTED;
  favor::rot::Params p{};
  int rc;
  if ((rc = make_view(&p.q, q, strides, 0, B, Hq, L, d)) != FAVOR_OK ||
      (rc = make_view(&p.qy, q_out, strides, 2, B, Hq, L, d)) != FAVOR_OK)
    return rc;
  if (Hk > 0 && ((rc = make_view(&p.k, k, strides, 1, B, Hk, L, d)) != FAVOR_OK ||
                 (rc = make_view(&p.ky, k_out, strides, 3, B, Hk, L, d)) != FAVOR_OK))
    return rc;
  for (const View* x : {&p.q, &p.k, &p.qy, &p.ky})  // views that are not there are null
    if (!view_aligned(*x, d, dtype_code)) return FAVOR_ERR_ALIGN;
  if (!rows_distinct(p.qy, B, Hq, L, d) || (Hk > 0 && !rows_distinct(p.ky, B, Hk, L, d))) return FAVOR_ERR_SHAPE;
  auto same = [](const View& a, const View& b) { return a.sb == b.sb && a.sh == b.sh && a.st == b.st; };
  // in place means the very same rows; q's output over k (or k's over q) has no order
  if ((q_out == q && !same(p.q, p.qy)) || (Hk > 0 && k_out == k && !same(p.k, p.ky)) ||
      (Hk > 0 && (q_out == k || k_out == q || k_out == q_out)))
    return FAVOR_ERR_UNSUPPORTED;
  if ((rc = check_device()) != FAVOR_OK) return rc;
  p.freq = freq;
  p.pos = positions;
  p.first = first_position;
  p.scale = scale;
  p.rot_scale = rot_scale;
  p.B = B, p.Hq = Hq, p.Hk = Hk, p.L = L, p.d = d, p.rot = rot, p.inverse = inverse != 0;
  const long long es = dtype_code == 1 ? 2 : 4;
  bool ok = true;
  for (const View* v : {&p.q, &p.qy, &p.k, &p.ky})
    ok = ok && v->sb * es % 16 == 0 && v->sh * es % 16 == 0 && v->st * es % 16 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype_code == 0 ? launch_rotary<float>(p, interleaved, ok, st)
                         : launch_rotary<__nv_bfloat16>(p, interleaved, ok, st);
}

int favor_rotary_frequencies(double* freq, double* rot_scale, int rot, double base, int scaling, double factor,
                             double trained_length, double beta_fast, double beta_slow) {
  if (!freq || !rot_scale) return FAVOR_ERR_NULL;
  if (rot <= 0 || rot % 2 != 0 || !(base > 1.0) || !std::isfinite(base)) return FAVOR_ERR_SHAPE;
  if (scaling < FAVOR_ROTARY_PLAIN || scaling > FAVOR_ROTARY_PARTS) return FAVOR_ERR_KIND;
  if (scaling != FAVOR_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return FAVOR_ERR_SHAPE;
  if (scaling == FAVOR_ROTARY_BASE && rot == 2) return FAVOR_ERR_SHAPE;
  if (scaling == FAVOR_ROTARY_PARTS &&
      (!(trained_length > 0.0) || !std::isfinite(trained_length) || !(beta_fast > beta_slow) || !(beta_slow >= 0.0) ||
       !std::isfinite(beta_fast)))
    return FAVOR_ERR_SHAPE;
  const double two_pi = 6.28318530717958647693;
  if (scaling == FAVOR_ROTARY_BASE) base *= std::pow(factor, (double)rot / (rot - 2));
  *rot_scale = scaling == FAVOR_ROTARY_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0;
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == FAVOR_ROTARY_LINEAR) f /= factor;
    if (scaling == FAVOR_ROTARY_PARTS) {
      const double turns = trained_length * f / two_pi;
      const double keep = std::min(1.0, std::max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)));
      f *= keep + (1.0 - keep) / factor;
    }
    freq[i] = f;
  }
  return FAVOR_OK;
}

}  // extern "C"
