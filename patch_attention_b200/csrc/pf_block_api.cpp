// pf_block_api.cpp -- host side of the transformer-block operators declared in
// include/patchattn.h: layer norm, QK norm + rotary, masked attention, and their gradients.  Checks every
// argument before anything is enqueued; holds no state.

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "patchattn.h"
#include "pf_internal.h"

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int t) { return t == PF_BF16 || t == PF_F16 || t == PF_F32; }
size_t elem_bytes(int t) { return t == PF_F32 ? 4 : 2; }
pf_status from_cuda(cudaError_t e) { return e == cudaSuccess ? PF_OK : PF_ERR_CUDA; }

// Sizes every layer-norm call checks: launch grids and row counts fit 31 bits.
pf_status check_ln_sizes(int64_t groups, int64_t rows_per_group, int channels) {
  if (groups < 1 || rows_per_group < 0 || channels < 1 || channels > pf::kLnMaxChannels) return PF_ERR_SHAPE;
  if (groups > INT32_MAX || rows_per_group > INT32_MAX || groups * rows_per_group > INT32_MAX) return PF_ERR_SHAPE;
  if (groups * 2 * ((channels + 31) / 32) > INT32_MAX) return PF_ERR_SHAPE;
  return PF_OK;
}

pf_status check_ln(const pf::LnArgs& a) {
  const pf_status st = check_ln_sizes(a.groups, a.rows_per_group, a.channels);
  if (st != PF_OK) return st;
  if (!dtype_ok(a.dtype) || (a.wdtype != a.dtype && a.wdtype != PF_F32)) return PF_ERR_UNSUPPORTED;
  if (!std::isfinite(a.weight_offset)) return PF_ERR_INVALID_ARG;
  if (a.groups > 1 && ((a.weight && a.weight_stride < a.channels) || (a.bias && a.bias_stride < a.channels)))
    return PF_ERR_INVALID_ARG;
  const size_t e = elem_bytes(a.dtype), we = elem_bytes(a.wdtype);
  if (!aligned(a.x, e) || !aligned(a.dy, e) || !aligned(a.y, e) || !aligned(a.weight, we) || !aligned(a.bias, we) ||
      !aligned(a.mean, 4) || !aligned(a.rstd, 4))
    return PF_ERR_ALIGN;
  return PF_OK;
}

// The pairs of a head vector, section by section; the rest of the vector is a section that
// does not turn.
pf_status make_rope(const pf_rope_config* c, pf::RopeArgs& a) {
  if (!c) return PF_ERR_INVALID_ARG;
  if (c->batch < 0 || c->tokens < 0 || c->heads_q < 0 || c->heads_k < 0 || c->heads_q + c->heads_k < 1 ||
      c->heads_q > 65536 || c->heads_k > 65536)
    return PF_ERR_SHAPE;
  if (c->head_dim < 8 || c->head_dim > 256 || c->head_dim % 8 != 0) return PF_ERR_SHAPE;
  if (c->n_axes < 1 || c->n_axes > 4) return PF_ERR_SHAPE;
  if (!dtype_ok(c->dtype)) return PF_ERR_UNSUPPORTED;
  if (!(c->eps >= 0.f) || std::isinf(c->eps)) return PF_ERR_INVALID_ARG;
  if (c->pos_batch_stride < 0) return PF_ERR_INVALID_ARG;
  // a block takes one to four tokens, on a 31-bit grid
  if (static_cast<int64_t>(c->batch) * c->tokens > INT32_MAX) return PF_ERR_SHAPE;
  std::memset(&a, 0, sizeof(a));
  a.batch = c->batch;
  a.tokens = c->tokens;
  a.n_axes = c->n_axes;
  a.heads[0] = c->heads_q;
  a.heads[1] = c->heads_k;
  a.head_dim = c->head_dim;
  a.dtype = c->dtype;
  a.interleaved = c->interleaved != 0;
  a.eps = c->eps;
  a.pos_batch = c->pos_batch_stride;
  int base = 0, pair = 0, half_bits = 4;
  for (int ax = 0; ax <= c->n_axes; ++ax) {
    const bool rest = ax == c->n_axes;
    const int w = rest ? c->head_dim - base : c->axis_dim[ax];
    if (w < 0 || w % 2 != 0 || (!rest && w == 0) || base + w > c->head_dim) return PF_ERR_SHAPE;
    if (!rest && (!(c->theta[ax] > 0.0) || std::isinf(c->theta[ax]))) return PF_ERR_INVALID_ARG;
    for (int i = 0; i < w / 2; ++i, ++pair) {
      a.tab.axis[pair] = static_cast<uint8_t>(ax);
      a.tab.e0[pair] = static_cast<uint8_t>(base + (a.interleaved ? 2 * i : i));
      a.tab.e1[pair] = static_cast<uint8_t>(base + (a.interleaved ? 2 * i + 1 : i + w / 2));
      a.tab.turns[pair] = rest ? 0.0 : std::pow(c->theta[ax], -2.0 * i / w) / 6.283185307179586476925;
    }
    half_bits |= w / 2;
    base += w;
  }
  a.tab.half_align = half_bits & -half_bits;
  return PF_OK;
}

// One operand of a rotary call: present exactly when it has heads, 16-byte aligned throughout.
pf_status take_operand(const pf::RopeArgs& a, int which, const void* p, const pf_strides* st, bool needed,
                       const void** out, long long (*strides)[3]) {
  *out = nullptr;
  if (a.heads[which] == 0) return p == nullptr ? PF_OK : PF_ERR_INVALID_ARG;
  if (!needed) return PF_OK;
  if (a.batch == 0 || a.tokens == 0) return PF_OK;
  if (!p || !st) return PF_ERR_INVALID_ARG;
  const int64_t unit = 16 / static_cast<int64_t>(elem_bytes(a.dtype));
  if (!aligned(p, 16) || st->batch % unit != 0 || st->token % unit != 0 || st->head % unit != 0) return PF_ERR_ALIGN;
  *out = p;
  strides[which][0] = st->batch;
  strides[which][1] = st->token;
  strides[which][2] = st->head;
  return PF_OK;
}

pf_status take_gain(pf::RopeArgs& a, int which, const void* g) {
  if (!g) return PF_OK;
  if (a.eps == 0.f || a.heads[which] == 0) return PF_ERR_INVALID_ARG;
  if (!aligned(g, 16)) return PF_ERR_ALIGN;
  a.gain[which] = g;
  return PF_OK;
}

// ------------------------------------------------------------------ masked attention

constexpr int kMaxTokens = 1 << 30;

// Strides of one operand: positive multiples of 16 bytes below 2^40 where the extent is above 1.
pf_status check_strides(const pf_strides& s, int batch, int rows, int heads) {
  const int64_t v[3] = {s.batch, s.token, s.head};
  const int extent[3] = {batch, rows, heads};
  for (int i = 0; i < 3; ++i) {
    if (extent[i] <= 1) continue;
    if (v[i] <= 0 || v[i] >= (int64_t{1} << 39)) return PF_ERR_INVALID_ARG;
    if (v[i] % 8 != 0) return PF_ERR_ALIGN;
  }
  return PF_OK;
}

constexpr float kLog2e = 1.4426950408889634f;

float scale_of(const pf_masked_attn_config& c) {
  return c.softmax_scale > 0.f ? c.softmax_scale : 1.0f / std::sqrt(static_cast<float>(c.head_dim));
}
// scale / cap: a raw product's argument of the cap's tanh.
float cap_in_of(const pf_masked_attn_config& c) { return c.softcap > 0.f ? scale_of(c) / c.softcap : 0.f; }

pf_status check_masked(const pf_masked_attn_config* c) {
  if (!c) return PF_ERR_INVALID_ARG;
  if (c->batch < 1 || c->heads_q < 1 || c->heads_kv < 1 || c->heads_q % c->heads_kv != 0) return PF_ERR_SHAPE;
  if (c->n_q < 0 || c->n_k < 0 || c->n_q > kMaxTokens || c->n_k > kMaxTokens) return PF_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 72 && c->head_dim != 128) return PF_ERR_UNSUPPORTED;
  if (!(c->softmax_scale >= 0.f) || std::isinf(c->softmax_scale)) return PF_ERR_INVALID_ARG;
  if (!(c->softcap >= 0.f) || !std::isfinite(c->softcap * kLog2e) || !std::isfinite(scale_of(*c) * kLog2e) ||
      !std::isfinite(3.f * cap_in_of(*c)))
    return PF_ERR_INVALID_ARG;
  // products are divided by cap / scale, in 32 bits: below this the quotients would lose bits or vanish
  if (c->softcap > 0.f && cap_in_of(*c) < 1e-30f) return PF_ERR_INVALID_ARG;
  // CTAs (at most 8 per query tile and head, or per key tile) on a 31-bit grid
  const double longest = c->n_q > c->n_k ? c->n_q : c->n_k;
  if (static_cast<double>(c->batch) * c->heads_q * (longest / 128 + 1) * 8 > 2147483647.0) return PF_ERR_SHAPE;
  pf_status st = check_strides(c->q, c->batch, c->n_q, c->heads_q);
  if (st == PF_OK) st = check_strides(c->k, c->batch, c->n_k, c->heads_kv);
  if (st == PF_OK) st = check_strides(c->v, c->batch, c->n_k, c->heads_kv);
  return st;
}

pf_status make_mask(const pf_masked_attn_config& c, const float* slopes, const int32_t* prefix, const int32_t* doc_q,
                    const int32_t* doc_k, pf::MaskParams& m) {
  if (prefix && !c.causal) return PF_ERR_INVALID_ARG;
  if ((doc_q != nullptr) != (doc_k != nullptr) && c.n_q > 0 && c.n_k > 0) return PF_ERR_INVALID_ARG;
  const bool docs = doc_q && doc_k;
  if (docs && c.n_k > pf::kMaskedDocTiles * 128) return PF_ERR_SHAPE;
  if (slopes && scale_of(c) < 1e-20f) return PF_ERR_INVALID_ARG;  // the forward kernel divides them by the scale
  if (!aligned(slopes, 4) || !aligned(prefix, 4) || !aligned(doc_q, 4) || !aligned(doc_k, 4)) return PF_ERR_ALIGN;
  m.prefix = prefix;
  m.doc_q = docs ? doc_q : nullptr;
  m.doc_k = docs ? doc_k : nullptr;
  m.slopes = slopes;
  m.causal = c.causal != 0;
  m.n_q = c.n_q;
  m.n_k = c.n_k;
  m.scale_log2 = scale_of(c) * kLog2e;
  m.cap_log2 = c.softcap * kLog2e;
  m.cap_in = cap_in_of(c);
  m.cap_half = c.softcap > 0.f ? 0.5f / m.cap_in : 0.f;
  return PF_OK;
}

// The device's status word and number of SMs, looked up once per device.
struct DeviceInfo {
  unsigned* watchdog;
  int sms;
};
cudaError_t device_info(DeviceInfo* out) {
  static std::atomic<unsigned*> words[64];
  static std::atomic<int> sms[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  out->watchdog = words[dev].load();
  out->sms = sms[dev].load();
  if (out->watchdog != nullptr && out->sms > 0) return cudaSuccess;
  e = pf::watchdog_word(&out->watchdog);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&out->sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  words[dev].store(out->watchdog);
  sms[dev].store(out->sms);
  return cudaSuccess;
}

pf_status from_attn(cudaError_t e) { return e == cudaErrorNotSupported ? PF_ERR_UNSUPPORTED : from_cuda(e); }

}  // namespace

extern "C" {

pf_status pf_layernorm(const void* x, void* y, int64_t groups, int64_t rows_per_group, int channels,
                       const void* weight, int64_t weight_stride, const void* bias, int64_t bias_stride,
                       float weight_offset, float eps, int dtype, int wdtype, float* mean, float* rstd, void* stream) {
  pf::LnArgs a = {x, nullptr, y, weight, bias, mean, rstd, groups, rows_per_group, weight_stride,
                  bias_stride, channels, dtype, wdtype, weight_offset, eps};
  const pf_status st = check_ln(a);
  if (st != PF_OK) return st;
  if (!(eps > 0.f) || std::isinf(eps)) return PF_ERR_INVALID_ARG;
  if (rows_per_group == 0) return PF_OK;
  if (!x || !y) return PF_ERR_INVALID_ARG;
  return from_cuda(pf::launch_layernorm(a, static_cast<cudaStream_t>(stream)));
}

size_t pf_layernorm_bwd_workspace_bytes(int64_t groups, int64_t rows_per_group, int channels) {
  if (check_ln_sizes(groups, rows_per_group, channels) != PF_OK || rows_per_group == 0) return 0;
  return static_cast<size_t>(groups) * pf::ln_bwd_parts(groups, rows_per_group) * 2 * channels * 4;
}

pf_status pf_layernorm_bwd(const void* dy, const void* x, int64_t groups, int64_t rows_per_group, int channels,
                           const void* weight, int64_t weight_stride, float weight_offset, int dtype, int wdtype,
                           const float* mean, const float* rstd, void* dx, void* dweight, void* dbias,
                           void* workspace, size_t workspace_bytes, void* stream) {
  pf::LnArgs a = {x, dy, dx, weight, nullptr, const_cast<float*>(mean), const_cast<float*>(rstd), groups,
                  rows_per_group, weight_stride, 0, channels, dtype, wdtype, weight_offset, 0.f};
  const pf_status st = check_ln(a);
  if (st != PF_OK) return st;
  if (rows_per_group > 0 && (!dy || !x || !dx || !mean || !rstd)) return PF_ERR_INVALID_ARG;
  const size_t we = elem_bytes(wdtype);
  if (!aligned(dweight, we) || !aligned(dbias, we) || !aligned(workspace, 16)) return PF_ERR_ALIGN;
  if (dweight || dbias) {
    const size_t need = pf_layernorm_bwd_workspace_bytes(groups, rows_per_group, channels);
    if (workspace_bytes < need || (need > 0 && !workspace)) return PF_ERR_INVALID_ARG;
  }
  return from_cuda(pf::launch_layernorm_bwd(a, dweight, dbias, static_cast<float*>(workspace),
                                            static_cast<cudaStream_t>(stream)));
}

pf_status pf_qk_norm_rope(const pf_rope_config* cfg, const float* pos, const void* q, const pf_strides* q_st,
                          const void* k, const pf_strides* k_st, const void* gain_q, const void* gain_k,
                          void* q_out, const pf_strides* q_out_st, void* k_out, const pf_strides* k_out_st,
                          void* stream) {
  pf::RopeArgs a;
  pf_status st = make_rope(cfg, a);
  const void* in[2] = {q, k};
  const pf_strides* in_st[2] = {q_st, k_st};
  const void* out[2] = {q_out, k_out};
  const pf_strides* out_st[2] = {q_out_st, k_out_st};
  const void* gain[2] = {gain_q, gain_k};
  for (int w = 0; w < 2 && st == PF_OK; ++w) {
    const void* y = nullptr;
    st = take_operand(a, w, in[w], in_st[w], true, &a.x[w], a.xs);
    if (st == PF_OK) st = take_operand(a, w, out[w], out_st[w], true, &y, a.ys);
    a.y[w] = const_cast<void*>(y);
    if (st == PF_OK) st = take_gain(a, w, gain[w]);
  }
  if (st != PF_OK) return st;
  if (a.batch == 0 || a.tokens == 0) return PF_OK;
  if (!pos) return PF_ERR_INVALID_ARG;
  if (!aligned(pos, 4)) return PF_ERR_ALIGN;
  a.pos = pos;
  return from_cuda(pf::launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

size_t pf_qk_norm_rope_bwd_workspace_bytes(const pf_rope_config* cfg) {
  pf::RopeArgs a;
  if (make_rope(cfg, a) != PF_OK) return 0;
  return static_cast<size_t>(pf::rope_bwd_blocks(a)) * 2 * a.head_dim * 4;
}

pf_status pf_qk_norm_rope_bwd(const pf_rope_config* cfg, const float* pos, const void* dq_out,
                              const pf_strides* dq_out_st, const void* dk_out, const pf_strides* dk_out_st,
                              const void* q, const pf_strides* q_st, const void* k, const pf_strides* k_st,
                              const void* gain_q, const void* gain_k, void* dq, const pf_strides* dq_st, void* dk,
                              const pf_strides* dk_st, void* dgain_q, void* dgain_k, void* workspace,
                              size_t workspace_bytes, void* stream) {
  pf::RopeArgs a;
  pf_status st = make_rope(cfg, a);
  const void* up[2] = {dq_out, dk_out};
  const pf_strides* up_st[2] = {dq_out_st, dk_out_st};
  const void* in[2] = {q, k};
  const pf_strides* in_st[2] = {q_st, k_st};
  const void* out[2] = {dq, dk};
  const pf_strides* out_st[2] = {dq_st, dk_st};
  const void* gain[2] = {gain_q, gain_k};
  const void* dgain[2] = {dgain_q, dgain_k};
  for (int w = 0; w < 2 && st == PF_OK; ++w) {
    const void* y = nullptr;
    st = take_operand(a, w, up[w], up_st[w], true, &a.dy[w], a.ds);
    if (st == PF_OK) st = take_operand(a, w, in[w], in_st[w], a.eps > 0.f, &a.x[w], a.xs);
    if (st == PF_OK) st = take_operand(a, w, out[w], out_st[w], true, &y, a.ys);
    a.y[w] = const_cast<void*>(y);
    if (st == PF_OK) st = take_gain(a, w, gain[w]);
    if (st == PF_OK && dgain[w] && (a.eps == 0.f || a.heads[w] == 0)) st = PF_ERR_INVALID_ARG;
    if (st == PF_OK && !aligned(dgain[w], elem_bytes(a.dtype))) st = PF_ERR_ALIGN;
  }
  if (st != PF_OK) return st;
  if (!aligned(workspace, 16) || !aligned(pos, 4)) return PF_ERR_ALIGN;
  if (dgain_q || dgain_k) {
    const size_t need = pf_qk_norm_rope_bwd_workspace_bytes(cfg);
    if (workspace_bytes < need || (need > 0 && !workspace)) return PF_ERR_INVALID_ARG;
  }
  if (a.batch > 0 && a.tokens > 0 && !pos) return PF_ERR_INVALID_ARG;
  a.pos = pos;
  return from_cuda(pf::launch_qk_norm_rope_bwd(a, dgain_q, dgain_k, static_cast<float*>(workspace),
                                               static_cast<cudaStream_t>(stream)));
}

pf_status pf_masked_attn(const pf_masked_attn_config* cfg, const void* q, const void* k, const void* v,
                         const float* slopes, const int32_t* prefix, const int32_t* doc_q, const int32_t* doc_k,
                         void* o, float* lse, void* stream) {
  pf_status st = check_masked(cfg);
  if (st != PF_OK) return st;
  const pf_masked_attn_config& c = *cfg;
  pf::MaskedFwdParams p;
  std::memset(&p, 0, sizeof(p));
  st = make_mask(c, slopes, prefix, doc_q, doc_k, p.m);
  if (st != PF_OK) return st;
  if (c.n_q == 0) return PF_OK;
  if (!q || !o || (c.n_k > 0 && (!k || !v))) return PF_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4)) return PF_ERR_ALIGN;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return PF_ERR_CUDA;
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.watchdog = dev.watchdog;
  p.batch = c.batch;
  p.heads_q = c.heads_q;
  p.heads_kv = c.heads_kv;
  p.head_dim = c.head_dim;
  pf::masked_fwd_plan(p, dev.sms);
  if (!pf::encode_heads_map(&p.tm_q, q, c.batch, c.n_q, c.heads_q, c.head_dim, c.q, p.pack, 128 / p.pack) ||
      (c.n_k > 0 && (!pf::encode_heads_map(&p.tm_k, k, c.batch, c.n_k, c.heads_kv, c.head_dim, c.k, 1, 128) ||
                     !pf::encode_heads_map(&p.tm_v, v, c.batch, c.n_k, c.heads_kv, c.head_dim, c.v, 1, 128))))
    return PF_ERR_CUDA;
  return from_attn(pf::launch_masked_fwd(p, static_cast<cudaStream_t>(stream)));
}

size_t pf_masked_attn_bwd_workspace_bytes(const pf_masked_attn_config* cfg) {
  if (check_masked(cfg) != PF_OK) return 0;
  return static_cast<size_t>(cfg->batch) * cfg->heads_q * cfg->n_q * 4;
}

pf_status pf_masked_attn_bwd(const pf_masked_attn_config* cfg, const void* dout, const void* q, const void* k,
                             const void* v, const void* o, const float* lse, const float* slopes,
                             const int32_t* prefix, const int32_t* doc_q, const int32_t* doc_k, void* dq, void* dk,
                             void* dv, void* workspace, size_t workspace_bytes, void* stream) {
  pf_status st = check_masked(cfg);
  if (st != PF_OK) return st;
  const pf_masked_attn_config& c = *cfg;
  pf::MaskedBwdParams p;
  std::memset(&p, 0, sizeof(p));
  st = make_mask(c, slopes, prefix, doc_q, doc_k, p.m);
  if (st != PF_OK) return st;
  if (p.m.doc_q && c.n_q > pf::kMaskedDocTiles * 128) return PF_ERR_SHAPE;
  if (c.n_q > 0 && (!dout || !q || !o || !lse || !dq || !workspace)) return PF_ERR_INVALID_ARG;
  if (c.n_k > 0 && (!k || !v || !dk || !dv)) return PF_ERR_INVALID_ARG;
  const void* all[] = {dout, q, k, v, o, dq, dk, dv, workspace};
  for (const void* x : all)
    if (!aligned(x, 16)) return PF_ERR_ALIGN;
  if (!aligned(lse, 4)) return PF_ERR_ALIGN;
  if (workspace_bytes < pf_masked_attn_bwd_workspace_bytes(cfg)) return PF_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return PF_ERR_CUDA;
  p.o = static_cast<const uint16_t*>(o);
  p.dout = static_cast<const uint16_t*>(dout);
  p.lse = lse;
  p.delta = static_cast<float*>(workspace);
  p.dq = static_cast<uint16_t*>(dq);
  p.dk = static_cast<uint16_t*>(dk);
  p.dv = static_cast<uint16_t*>(dv);
  p.watchdog = dev.watchdog;
  p.batch = c.batch;
  p.heads_q = c.heads_q;
  p.heads_kv = c.heads_kv;
  p.head_dim = c.head_dim;
  p.scale = scale_of(c);
  const int64_t row = static_cast<int64_t>(c.heads_q) * c.head_dim;
  const pf_strides whole = {row * c.n_q, row, c.head_dim};
  CUtensorMap maps[2][4];
  std::memset(maps, 0, sizeof(maps));
  for (int box = 0; box < 2; ++box) {
    const int rows = box == 0 ? 128 : 64;
    auto map = [&](int which, const void* base, int n, int heads, const pf_strides& strides) {
      return n == 0 || pf::encode_heads_map(&maps[box][which], base, c.batch, n, heads, c.head_dim, strides, 1, rows);
    };
    if (!map(0, q, c.n_q, c.heads_q, c.q) || !map(1, k, c.n_k, c.heads_kv, c.k) || !map(2, v, c.n_k, c.heads_kv, c.v) ||
        !map(3, dout, c.n_q, c.heads_q, whole))
      return PF_ERR_CUDA;
  }
  return from_attn(pf::launch_masked_bwd(p, maps, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
