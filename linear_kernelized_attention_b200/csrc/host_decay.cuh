// host_decay.cuh - host side of the decayed linear attention and rotary entry points: argument
// checks, scratch, launches. Included by favor_lib.cu after its helpers.
#pragma once
#include <cmath>

#include "kernel_decay_step.cuh"
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

template <typename T, int DP>
int launch_decay_cc_t(const dcy::Params& p, cudaStream_t st) {
  const long long heads = (long long)p.B * p.H;
  const long long g_up = heads * p.nstates * p.nch, g_out = heads * p.nouts * p.nch;
  const long long g_scan = (heads * p.nstates * p.d * p.d + dcy::kThreads - 1) / dcy::kThreads;
  if (g_up > INT_MAX || g_out > INT_MAX || g_scan > INT_MAX) return FAVOR_ERR_UNSUPPORTED;
  auto ku = dcy::k_chunk_update<T, DP>;
  auto ko = dcy::k_chunk_out<T, DP>;
  if (ensure_smem_attr(reinterpret_cast<const void*>(ku), dcy::update_smem(DP)) != FAVOR_OK ||
      ensure_smem_attr(reinterpret_cast<const void*>(ko), dcy::out_smem(DP)) != FAVOR_OK)
    return FAVOR_ERR_CUDA;
  ku<<<(unsigned)g_up, dcy::kThreads, dcy::update_smem(DP), st>>>(p);
  dcy::k_chunk_scan<<<(unsigned)g_scan, dcy::kThreads, 0, st>>>(p);
  ko<<<(unsigned)g_out, dcy::kThreads, dcy::out_smem(DP), st>>>(p);
  return cudaGetLastError() == cudaSuccess ? FAVOR_OK : FAVOR_ERR_CUDA;
}

// The CUDA-core route: every type, head size and stride.
int launch_decay_cc(dcy::Params p, int dtype_code, cudaStream_t st) {
  p.nch = decay_chunks(p.L);
  void* ws = nullptr;
  int rc = scratch_alloc(&ws, decay_cc_workspace(p.B, p.H, p.L, p.d, p.nstates), st);
  if (rc != FAVOR_OK) return rc;
  p.ws = static_cast<float*>(ws);
  if (dtype_code == 0)
    rc = p.d <= 32   ? launch_decay_cc_t<float, 32>(p, st)
         : p.d <= 64 ? launch_decay_cc_t<float, 64>(p, st)
                     : launch_decay_cc_t<float, 128>(p, st);
  else
    rc = p.d <= 32   ? launch_decay_cc_t<__nv_bfloat16, 32>(p, st)
         : p.d <= 64 ? launch_decay_cc_t<__nv_bfloat16, 64>(p, st)
                     : launch_decay_cc_t<__nv_bfloat16, 128>(p, st);
  cudaFreeAsync(ws, st);
  return rc;
}

int launch_decay(const dcy::Params& p, int dtype_code, cudaStream_t st) { return launch_decay_cc(p, dtype_code, st); }

bool bad_align(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return true;
  return false;
}

template <typename T>
int launch_decay_step(const dcy::StepParams& p0, int BH, int d, cudaStream_t st) {
  dcy::StepParams p = p0;
  const bool vec = d % 4 == 0;
  // Slices of 32 columns (whole 128-byte row pieces) while all heads' slices are below two blocks
  // an SM, else whole rows.
  p.cols = d <= 32 || (long long)BH * ((d + 31) / 32) > 2ll * sm_count() ? d : 32;
  p.slices = (d + p.cols - 1) / p.cols;
  if ((long long)BH * p.slices > INT_MAX) return FAVOR_ERR_UNSUPPORTED;
  const unsigned grid = (unsigned)((long long)BH * p.slices);
  if (vec)
    dcy::k_decay_step<T, 4, 8><<<grid, dcy::kStepThreads, 0, st>>>(p);
  else
    dcy::k_decay_step<T, 1, 8><<<grid, dcy::kStepThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? FAVOR_OK : FAVOR_ERR_CUDA;
}

template <typename T, int V, bool INTER>
int launch_rotary_t(favor::rot::Params p, cudaStream_t st) {
  p.npair = p.rot / 2 / V;
  p.npass = (p.d - p.rot) / V;
  const long long items = (long long)p.B * p.L * (p.npair + p.npass);
  const long long blocks = (items + favor::rot::kThreads - 1) / favor::rot::kThreads;
  const int heads = p.Hq + p.Hk, sms = sm_count();
  // every head in one thread, unless that leaves fewer than four blocks an SM
  p.groups = (int)std::max<long long>(1, std::min<long long>(heads, 4ll * sms / std::max<long long>(1, blocks)));
  p.per_group = (heads + p.groups - 1) / p.groups;
  p.groups = (heads + p.per_group - 1) / p.per_group;
  const unsigned gx = (unsigned)std::min<long long>(blocks, 64ll * sms);
  if (p.groups > 65535) return FAVOR_ERR_UNSUPPORTED;
  favor::rot::k_rotary<T, V, INTER><<<dim3(gx, p.groups), favor::rot::kThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? FAVOR_OK : FAVOR_ERR_CUDA;
}

template <typename T>
int launch_rotary(const favor::rot::Params& p, int interleaved, bool strides_ok, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  // 16-byte pieces where every row starts on one and the pairs and the rest fill whole ones
  const bool vec = strides_ok && (p.rot / 2) % V == 0 && (p.d - p.rot) % V == 0;
  if (interleaved) return vec ? launch_rotary_t<T, V, true>(p, st) : launch_rotary_t<T, 1, true>(p, st);
  return vec ? launch_rotary_t<T, V, false>(p, st) : launch_rotary_t<T, 1, false>(p, st);
}

}  // namespace

extern "C" {

size_t favor_decay_workspace_bytes(int B, int H, int L, int d, int dtype_code, int backward) {
  if (check_decay_sizes(B, H, L, d, dtype_code) != FAVOR_OK) return 0;
  return decay_cc_workspace(B, H, L, d, backward ? 2 : 1);
}

int favor_decay_attention(const void* q, const void* k, const void* v, const float* log_decay, const float* state_in,
                          const int* lengths, void* out, float* state_out, int B, int H, int L, int d,
                          int dtype_code, const favor_strides* strides, void* stream) {
  if (!q || !k || !v || !log_decay || !out) return FAVOR_ERR_NULL;
  if (bad_align({q, k, v, out, state_in, state_out}) || ((uintptr_t)log_decay & 3) || ((uintptr_t)lengths & 3))
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
  if (bad_align({q, k, v, dout, dq, dk, dv, state_in, dstate_out, dstate_in}) || ((uintptr_t)log_decay & 3) ||
      ((uintptr_t)lengths & 3))
    return FAVOR_ERR_ALIGN;
  int rc = check_decay_sizes(B, H, L, d, dtype_code);
  if (rc != FAVOR_OK) return rc;
  View x[7];
  const void* ptr[7] = {q, k, v, dout, dq, dk, dv};
  for (int i = 0; i < 7; ++i)
    if ((rc = make_view(&x[i], ptr[i], strides, i, B, H, L, d)) != FAVOR_OK) return rc;
  for (int i = 4; i < 7; ++i) {
    if (!rows_distinct(x[i], B, H, L, d)) return FAVOR_ERR_SHAPE;
    for (int j = 0; j < i; ++j)
      if (ptr[i] == ptr[j]) return FAVOR_ERR_UNSUPPORTED;
  }
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
  if (bad_align({q, k, v, out, state}) || ((uintptr_t)log_decay & 3)) return FAVOR_ERR_ALIGN;
  int rc = check_decay_sizes(B, H, 1, d, dtype_code);
  if (rc != FAVOR_OK) return rc;
  dcy::StepParams p{};
  if ((rc = make_view(&p.q, q, strides, 0, B, H, 1, d)) != FAVOR_OK ||
      (rc = make_view(&p.k, k, strides, 1, B, H, 1, d)) != FAVOR_OK ||
      (rc = make_view(&p.v, v, strides, 2, B, H, 1, d)) != FAVOR_OK ||
      (rc = make_view(&p.y, out, strides, 3, B, H, 1, d)) != FAVOR_OK)
    return rc;
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
  if (bad_align({q, q_out}) || (Hk > 0 && bad_align({k, k_out})) || ((uintptr_t)freq & 7) || ((uintptr_t)positions & 3))
    return FAVOR_ERR_ALIGN;
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
