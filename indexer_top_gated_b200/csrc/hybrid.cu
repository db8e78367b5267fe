// hybrid.cu - C ABI of the operators around the layer (include/dsa.h): the rotary append, the
// short convolution and the gated delta rule.  Argument validation and launch configuration;
// the kernels are in the headers included here.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "dsa.h"
#include "gated_delta.cuh"
#include "gated_delta_umma.cuh"
#include "hybrid.h"
#include "rope.cuh"
#include "short_conv.cuh"

namespace dsa {
namespace {

#define DSA_TRY(x)                   \
  do {                               \
    dsa_status _s = (x);             \
    if (_s != DSA_OK) return _s;     \
  } while (0)

// Status of the launch just made, which it counts; one line on stderr when it failed.
dsa_status launched(const char* kernel) {
  count_launches(1);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return DSA_OK;
  std::fprintf(stderr, "dsa: launch of %s failed: %s\n", kernel, cudaGetErrorString(e));
  return DSA_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct Span {
  uintptr_t at = 0;
  size_t bytes = 0;
};
Span span(const void* p, int64_t rows, int64_t stride, int64_t width, int elem) {
  Span s;
  if (!p || rows <= 0) return s;
  s.at = reinterpret_cast<uintptr_t>(p);
  s.bytes = (size_t)((rows - 1) * stride + width) * elem;
  return s;
}
bool overlap(const Span& a, const Span& b) {
  return a.bytes && b.bytes && a.at < b.at + b.bytes && b.at < a.at + a.bytes;
}

dsa_status check_rows(const dsa_ragged* R) {
  if (!R || R->batch < 1 || !R->q_offsets || R->total_q < 0) return DSA_ERR_INVALID_ARG;
  if (R->total_q > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}
dsa_status check_lens(const dsa_ragged* R) {
  DSA_TRY(check_rows(R));
  return R->max_q_len < 0 ? DSA_ERR_INVALID_ARG : DSA_OK;
}

// The row stride to use: `stride`, or `width` when it is 0; -1 when invalid.
int64_t row_stride(int64_t stride, int64_t width) {
  if (stride == 0) return width;
  return stride < width || stride % 8 != 0 ? -1 : stride;
}

// ---------------------------------------------------------------- rotary append
// Turns per position of each pair.
dsa_status rope_freqs(const dsa_rope_params* O, int rot, double* f) {
  if (rot == 0) return DSA_OK;
  long double theta = O->theta;
  if (O->scaling == DSA_ROPE_SCALE_NTK && rot > 2)
    theta *= std::pow((long double)O->factor, (long double)rot / (rot - 2));
  const double two_pi = 6.283185307179586477;
  // powers by multiplication: 64 steps in 64-bit mantissas stay below a double's half step
  const long double ratio = std::pow(theta, -2.0L / rot);
  long double power = 1;
  for (int i = 0; i < rot / 2; ++i, power *= ratio) {
    double x = (double)power;
    if (O->scaling == DSA_ROPE_SCALE_LINEAR) x /= O->factor;
    if (O->scaling == DSA_ROPE_SCALE_BY_PARTS) {
      const double turns = O->orig_len * x / two_pi;
      double keep = (turns - O->beta_slow) / (O->beta_fast - O->beta_slow);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      x *= keep + (1 - keep) / O->factor;
    }
    if (!std::isfinite(x)) return DSA_ERR_INVALID_ARG;
    f[i] = x / two_pi;
  }
  return DSA_OK;
}

dsa_status check_rot(int rot, int off, int dim) {
  if (rot < 0 || rot > dim || off < 0 || off > dim - rot) return DSA_ERR_INVALID_ARG;
  if (rot % 16 != 0 || off % 8 != 0) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

}  // namespace

cudaError_t hybrid_allow_smem() {
  auto allow = [](const void* f, int bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  cudaError_t e = allow((const void*)delta_prep_kernel<false>, (int)sizeof(PrepSmem));
  e = e ? e : allow((const void*)delta_prep_kernel<true>, (int)sizeof(PrepSmem));
  e = e ? e : allow((const void*)delta_umma_kernel, kUmmaSmem);
  e = e ? e : allow((const void*)delta_scan_kernel<1>, ScanGeo<1>::kSmem);
  e = e ? e : allow((const void*)delta_scan_kernel<2>, ScanGeo<2>::kSmem);
  return e;
}

}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_rope_append(const dsa_params* P, const dsa_ragged* R, const dsa_rope_params* O,
                           const dsa_rope_buffers* B, const int32_t* positions,
                           int32_t* err_count, void* stream) {
  DSA_TRY(check_lens(R));
  if (!P || !O || !B || !R->kv_offsets || R->total_kv < 0) return DSA_ERR_INVALID_ARG;
  if (R->total_kv > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  const bool att = B->q || B->k || B->v, idx = B->q_idx || B->k_idx;
  const bool cached = B->k || B->v || B->k_idx;
  RopeArgs a = {};
  if (R->block_table && cached) {
    const int ps = R->page_size;
    if (ps < 128 || ps > (1 << 24) || (ps & (ps - 1)) != 0) return DSA_ERR_INVALID_ARG;
    if (R->max_pages < 1 || (int64_t)R->max_pages * ps < R->max_kv_len) return DSA_ERR_INVALID_ARG;
    if (R->total_kv % ps != 0) return DSA_ERR_INVALID_ARG;
    a.pg.table = R->block_table;
    a.pg.max_pages = R->max_pages;
    while ((1 << a.pg.shift) < ps) ++a.pg.shift;
    a.pg.n_pages = (int)(R->total_kv >> a.pg.shift);
  }
  if (att) {
    if (P->head_dim != 128) return DSA_ERR_UNSUPPORTED;
    DSA_TRY(check_rot(O->rot_dim, O->rot_offset, 128));
    if ((B->q && P->n_q_heads < 1) || ((B->k || B->v) && P->n_kv_heads < 1))
      return DSA_ERR_INVALID_ARG;
    if ((B->q && P->n_q_heads > 65536) || ((B->k || B->v) && P->n_kv_heads > 65536))
      return DSA_ERR_UNSUPPORTED;
  }
  if (idx) {
    if (P->idx_dim != 64 || P->n_idx_heads < 1 || P->n_idx_heads > 4) return DSA_ERR_UNSUPPORTED;
    if (P->idx_dtype != DSA_BF16 && P->idx_dtype != DSA_FP8_E4M3) return DSA_ERR_INVALID_ARG;
    if ((B->q_idx && (!(P->idx_scale_q > 0.f) || !std::isfinite(P->idx_scale_q))) ||
        (B->k_idx && (!(P->idx_scale_k > 0.f) || !std::isfinite(P->idx_scale_k))))
      return DSA_ERR_INVALID_ARG;
    DSA_TRY(check_rot(O->idx_rot_dim, O->idx_rot_offset, 64));
  }
  if (O->layout != DSA_ROPE_HALF && O->layout != DSA_ROPE_INTERLEAVED) return DSA_ERR_INVALID_ARG;
  if (O->scaling < DSA_ROPE_SCALE_NONE || O->scaling > DSA_ROPE_SCALE_BY_PARTS)
    return DSA_ERR_INVALID_ARG;
  if (!(O->theta > 0) || !std::isfinite(O->theta) || !std::isfinite(O->magnitude))
    return DSA_ERR_INVALID_ARG;
  if (O->scaling != DSA_ROPE_SCALE_NONE && (!(O->factor > 0) || !std::isfinite(O->factor)))
    return DSA_ERR_INVALID_ARG;
  if (O->scaling == DSA_ROPE_SCALE_BY_PARTS &&
      (!(O->orig_len > 0) || !std::isfinite(O->orig_len) || !std::isfinite(O->beta_fast) ||
       !std::isfinite(O->beta_slow) || !(O->beta_fast > O->beta_slow)))
    return DSA_ERR_INVALID_ARG;

  const bool fp8 = idx && P->idx_dtype == DSA_FP8_E4M3;
  struct Item {
    RopeTensor* t;
    const void* src;
    void* dst;
    int64_t stride;
    int heads, dim;
    bool cache;
  };
  const Item items[5] = {
      {&a.t[0], B->q, B->q_out, O->q_row_stride, P->n_q_heads, 128, false},
      {&a.t[1], B->k, B->k_cache, O->k_row_stride, P->n_kv_heads, 128, true},
      {&a.t[2], B->v, B->v_cache, O->v_row_stride, P->n_kv_heads, 128, true},
      {&a.t[3], B->q_idx, B->q_idx_out, O->q_idx_row_stride, P->n_idx_heads, 64, false},
      {&a.t[4], B->k_idx, B->k_idx_cache, O->k_idx_row_stride, P->n_idx_heads, 64, true}};
  Span in[5], out[5];
  for (int i = 0; i < 5; ++i) {
    const Item& t = items[i];
    if (!t.src) continue;
    const int64_t width = (int64_t)t.heads * t.dim, stride = row_stride(t.stride, width);
    if (!t.dst || stride < 0 || !aligned16(t.src) || !aligned16(t.dst)) return DSA_ERR_INVALID_ARG;
    *t.t = {static_cast<const __nv_bfloat16*>(t.src), t.dst, stride, t.heads};
    in[i] = span(t.src, R->total_q, stride, width, 2);
    out[i] = span(t.dst, t.cache ? R->total_kv : R->total_q, width, width, t.dim == 64 && fp8 ? 1 : 2);
  }
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < 5; ++j) {
      if (i < j && overlap(out[i], out[j])) return DSA_ERR_INVALID_ARG;
      if (!overlap(out[i], in[j])) continue;
      const bool in_place = i == j && !items[i].cache && out[i].at == in[i].at &&
                            out[i].bytes == in[i].bytes;
      if (!in_place) return DSA_ERR_INVALID_ARG;
    }
  if (att) DSA_TRY(rope_freqs(O, O->rot_dim, a.turns));
  if (idx) DSA_TRY(rope_freqs(O, O->idx_rot_dim, a.idx_turns));
  a.q_offsets = R->q_offsets;
  a.kv_offsets = R->kv_offsets;
  a.positions = positions;
  a.batch = R->batch;
  a.total_q = R->total_q;
  a.cache_rows = R->total_kv;
  a.err_count = cached ? err_count : nullptr;
  a.interleaved = O->layout == DSA_ROPE_INTERLEAVED;
  a.idx_fp8 = fp8;
  a.rot = att ? O->rot_dim : 0;
  a.off = att ? O->rot_offset : 0;
  a.idx_rot = idx ? O->idx_rot_dim : 0;
  a.idx_off = idx ? O->idx_rot_offset : 0;
  a.mscale = O->magnitude == 0 ? 1.f : (float)O->magnitude;
  a.idx_scale_q = P->idx_scale_q;
  a.idx_scale_k = P->idx_scale_k;
  if (R->total_q == 0 || !(att || idx)) return DSA_OK;
  HybridDevice dev;
  DSA_TRY(hybrid_device(&dev));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // One row per CTA for few rows (64 rows 4.4 us, by four 6.1 us; 592 rows 7.3 and 6.9 us, 4736
  // rows 57 and 43 us)
  if (R->total_q < (int64_t)dev.num_sms * 3)
    rope_append_kernel<1><<<(unsigned)R->total_q, kRopeThreads, 0, st>>>(a);
  else
    rope_append_kernel<4><<<(unsigned)((R->total_q + 3) / 4), kRopeThreads, 0, st>>>(a);
  return launched("rope_append_kernel");
}

}  // extern "C"

// ---------------------------------------------------------------- short convolution
namespace dsa {
namespace {
constexpr int kConvRun = 48;  // rows of a run in a large batch

template <int W>
dsa_status launch_conv(const ConvArgs& a, const dsa_ragged* R, int sms, cudaStream_t st) {
  const int groups = (a.channels / 8 + kConvThreads - 1) / kConvThreads;
  // Long runs read fewer rows twice; short ones spread a small batch over the GPU (4 taps, 8192
  // channels, runs of 8 and of 48 rows: 300 rows 6.2 and 9.6 us, 900 rows 11.6 and 11.2 us, 1500
  // rows 16.7 and 14.0 us, 8000 rows 66 and 49 us; 2 taps, one row twice: 8000 rows 44 and 48 us)
  const bool wide = R->total_q / kConvRun * groups * 2 >= 3 * (int64_t)sms;
  // (max_q_len may be unset: either form takes sequences of any length)
  const bool single = R->max_q_len == 1;
  const int64_t runs = single ? R->batch : R->total_q / (wide ? kConvRun : 8) + R->batch;
  const unsigned y = (unsigned)std::min<int64_t>(runs, 32768);
  const dim3 grid((unsigned)groups, y, (unsigned)((runs + y - 1) / y));
  if (single) short_conv_kernel<W, 1><<<grid, kConvThreads, 0, st>>>(a);
  else if (wide) short_conv_kernel<W, kConvRun><<<grid, kConvThreads, 0, st>>>(a);
  else short_conv_kernel<W, 8><<<grid, kConvThreads, 0, st>>>(a);
  return launched("short_conv_kernel");
}
}  // namespace
}  // namespace dsa

extern "C" {

dsa_status dsa_short_conv(const dsa_conv_params* P, const dsa_ragged* R, const void* x,
                          const void* weight, const void* bias, const void* state_in,
                          void* state_out, const int32_t* state_index, void* out, void* stream) {
  DSA_TRY(check_rows(R));
  if (!P || !weight) return DSA_ERR_INVALID_ARG;
  if (R->total_q > 0 && (!x || !out)) return DSA_ERR_INVALID_ARG;
  if (P->channels < 1 || P->channels % 8 != 0) return DSA_ERR_INVALID_ARG;
  if (P->width < 2 || P->width > kConvMaxWidth) return DSA_ERR_UNSUPPORTED;
  if (P->channels > (1 << 24)) return DSA_ERR_UNSUPPORTED;
  if (P->n_states < 0 || ((state_in || state_out) && P->n_states < 1)) return DSA_ERR_INVALID_ARG;
  ConvArgs a = {};
  a.x_stride = row_stride(P->x_row_stride, P->channels);
  a.out_stride = row_stride(P->out_row_stride, P->channels);
  if (a.x_stride < 0 || a.out_stride < 0) return DSA_ERR_INVALID_ARG;
  for (const void* p : {x, weight, bias, state_in, (const void*)state_out, (const void*)out})
    if (!aligned16(p)) return DSA_ERR_INVALID_ARG;
  const int64_t slot = (int64_t)(P->width - 1) * P->channels;
  const Span so = span(out, R->total_q, a.out_stride, P->channels, 2);
  const Span sx = span(x, R->total_q, a.x_stride, P->channels, 2);
  const Span s0 = span(state_in, P->n_states, slot, slot, 2);
  const Span s1 = span(state_out, P->n_states, slot, slot, 2);
  const Span sw = span(weight, 1, 0, (int64_t)P->channels * P->width, 2);
  const Span sb = span(bias, 1, 0, P->channels, 2);
  if (overlap(so, sx) || overlap(so, s0) || overlap(so, s1) || overlap(sx, s1) ||
      overlap(so, sw) || overlap(so, sb) || overlap(s1, sw) || overlap(s1, sb))
    return DSA_ERR_INVALID_ARG;
  if (state_in != state_out && overlap(s0, s1)) return DSA_ERR_INVALID_ARG;
  a.q_offsets = R->q_offsets;
  a.batch = R->batch;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.weight = static_cast<const __nv_bfloat16*>(weight);
  a.bias = static_cast<const __nv_bfloat16*>(bias);
  a.state_in = static_cast<const __nv_bfloat16*>(state_in);
  a.state_out = static_cast<__nv_bfloat16*>(state_out);
  a.state_index = state_index;
  a.n_states = P->n_states;
  a.channels = P->channels;
  a.silu = P->silu;
  a.out = static_cast<__nv_bfloat16*>(out);
  HybridDevice dev;
  DSA_TRY(hybrid_device(&dev));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return P->width == 2 ? launch_conv<2>(a, R, dev.num_sms, st)
         : P->width == 3 ? launch_conv<3>(a, R, dev.num_sms, st)
                         : launch_conv<4>(a, R, dev.num_sms, st);
}

}  // extern "C"

// ---------------------------------------------------------------- gated delta rule
namespace dsa {
namespace {

// Sequences of up to this many tokens run token by token (at 24 tokens, against the chunks: 16
// sequences x 16 heads 61 and 68 us, 64 x 32 281 and 346 us; the cost grows with each token).
constexpr int kDeltaShort = 24;

dsa_status check_delta(const dsa_delta_params* P, const dsa_ragged* R) {
  DSA_TRY(check_lens(R));
  if (!P) return DSA_ERR_INVALID_ARG;
  if (P->head_dim != kDeltaDim) return DSA_ERR_UNSUPPORTED;
  if (P->n_k_heads < 1 || P->n_v_heads < 1 || P->n_v_heads % P->n_k_heads != 0)
    return DSA_ERR_INVALID_ARG;
  if (P->n_v_heads > 65536) return DSA_ERR_UNSUPPORTED;
  // (a CTA of the scan takes 16 or more of a head's 128 value columns)
  if ((int64_t)R->batch * P->n_v_heads * 8 > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  if (P->reserved != 0 || P->n_states < 0) return DSA_ERR_INVALID_ARG;
  if (P->qk_norm && (!(P->norm_eps > 0.f) || !std::isfinite(P->norm_eps)))
    return DSA_ERR_INVALID_ARG;
  if (P->scale < 0.f || !std::isfinite(P->scale)) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

int64_t delta_slots(const dsa_ragged* R) { return R->total_q / kDeltaChunk + R->batch; }

dsa_status delta_args(const dsa_delta_params* P, const dsa_ragged* R, const void* q, const void* k,
                      const void* v, const float* g, const float* beta, const float* state_in,
                      float* state_out, const int32_t* state_index, void* out, DeltaArgs* a) {
  if (R->total_q > 0 && (!q || !k || !v || !g || !beta || !out)) return DSA_ERR_INVALID_ARG;
  if ((state_in || state_out) && P->n_states < 1) return DSA_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, (const void*)g, (const void*)beta, (const void*)state_in,
                        (const void*)state_out, (const void*)out})
    if (!aligned16(p)) return DSA_ERR_INVALID_ARG;
  const int64_t wk = (int64_t)P->n_k_heads * kDeltaDim, wv = (int64_t)P->n_v_heads * kDeltaDim;
  a->q_stride = row_stride(P->q_row_stride, wk);
  a->k_stride = row_stride(P->k_row_stride, wk);
  a->v_stride = row_stride(P->v_row_stride, wv);
  if (a->q_stride < 0 || a->k_stride < 0 || a->v_stride < 0) return DSA_ERR_INVALID_ARG;
  const int64_t n = R->total_q, slot = wv * kDeltaDim;
  const Span so = span(out, n, wv, wv, 2);
  const Span s0 = span(state_in, P->n_states, slot, slot, 4);
  const Span s1 = span(state_out, P->n_states, slot, slot, 4);
  const Span in[5] = {span(q, n, a->q_stride, wk, 2), span(k, n, a->k_stride, wk, 2),
                      span(v, n, a->v_stride, wv, 2), span(g, n, P->n_v_heads, P->n_v_heads, 4),
                      span(beta, n, P->n_v_heads, P->n_v_heads, 4)};
  for (const Span& s : in)
    if (overlap(so, s) || overlap(s1, s)) return DSA_ERR_INVALID_ARG;
  if (overlap(so, s0) || overlap(so, s1)) return DSA_ERR_INVALID_ARG;
  if (state_in != state_out && overlap(s0, s1)) return DSA_ERR_INVALID_ARG;
  a->q_offsets = R->q_offsets;
  a->batch = R->batch;
  a->q = static_cast<const __nv_bfloat16*>(q);
  a->k = static_cast<const __nv_bfloat16*>(k);
  a->v = static_cast<const __nv_bfloat16*>(v);
  a->g = g;
  a->beta = beta;
  a->state_in = state_in;
  a->state_out = state_out;
  a->state_index = state_index;
  a->n_states = P->n_states;
  a->out = static_cast<__nv_bfloat16*>(out);
  a->hk = P->n_k_heads;
  a->hv = P->n_v_heads;
  a->norm = P->qk_norm != 0;
  a->scale = P->scale == 0.f ? (float)(1.0 / std::sqrt((double)kDeltaDim)) : P->scale;
  a->eps = P->norm_eps;
  return DSA_OK;
}

dsa_status launch_recurrent(DeltaArgs a, int max_len, cudaStream_t st) {
  a.min_len = 0;
  a.max_len = max_len;
  const int64_t ctas = (int64_t)a.batch * a.hv * kRecParts;
  delta_recurrent_kernel<<<(unsigned)ctas, kRecWarps * 32, 0, st>>>(a);
  return launched("delta_recurrent_kernel");
}

template <int PAIRS>
dsa_status launch_scan(const DeltaArgs& a, const DeltaMaps& maps, cudaStream_t st) {
  using Geo = ScanGeo<PAIRS>;
  const int64_t ctas = (int64_t)a.batch * a.heads * Geo::kParts;
  delta_scan_kernel<PAIRS><<<(unsigned)ctas, Geo::kThreads, Geo::kSmem, st>>>(a, maps);
  return launched("delta_scan_kernel");
}

}  // namespace
}  // namespace dsa

extern "C" {

dsa_status dsa_gated_delta_workspace_size(const dsa_delta_params* P, const dsa_ragged* R,
                                          size_t* min_bytes, size_t* rec_bytes) {
  DSA_TRY(check_delta(P, R));
  const size_t head =
      R->max_q_len <= kDeltaShort ? 0 : (size_t)delta_slots(R) * kDeltaItemBytes;
  if (min_bytes) *min_bytes = head;
  if (rec_bytes) *rec_bytes = head * P->n_v_heads;
  return DSA_OK;
}

dsa_status dsa_gated_delta_prefill(const dsa_delta_params* P, const dsa_ragged* R, const void* q,
                                   const void* k, const void* v, const float* g,
                                   const float* beta, const float* state_in, float* state_out,
                                   const int32_t* state_index, void* out, void* workspace,
                                   size_t ws_bytes, void* stream) {
  DSA_TRY(check_delta(P, R));
  DeltaArgs a = {};
  DSA_TRY(delta_args(P, R, q, k, v, g, beta, state_in, state_out, state_index, out, &a));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  HybridDevice dev;
  if (R->max_q_len <= kDeltaShort || R->total_q == 0) {
    DSA_TRY(hybrid_device(&dev));
    return launch_recurrent(a, INT32_MAX, st);
  }
  const int64_t slots = delta_slots(R);
  const size_t head = (size_t)slots * kDeltaItemBytes;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || ws_bytes < head)
    return DSA_ERR_WORKSPACE;
  int64_t pass = (int64_t)(ws_bytes / head);
  pass = std::min<int64_t>(pass, a.hv);
  if (slots * pass > INT32_MAX) pass = INT32_MAX / slots;
  if (pass < 1) return DSA_ERR_UNSUPPORTED;
  DSA_TRY(hybrid_device(&dev));
  a.status = dev.status;
  DeltaMaps maps;
  DSA_TRY(make_row_map(&maps.q, q, R->total_q, P->n_k_heads * kDeltaDim, a.q_stride, 64, kDeltaChunk));
  DSA_TRY(make_row_map(&maps.k, k, R->total_q, P->n_k_heads * kDeltaDim, a.k_stride, 64, kDeltaChunk));
  DSA_TRY(make_row_map(&maps.v, v, R->total_q, P->n_v_heads * kDeltaDim, a.v_stride, kScanNV,
                       kDeltaChunk));
  DSA_TRY(make_row_map(&maps.out, out, R->total_q, P->n_v_heads * kDeltaDim,
                       (int64_t)P->n_v_heads * kDeltaDim, 32, kDeltaChunk));
  bool any_short = true;
  if (R->q_offsets_host) {
    any_short = false;
    for (int b = 0; b < R->batch && !any_short; ++b)
      any_short = R->q_offsets_host[b + 1] - R->q_offsets_host[b] <= kDeltaShort;
  }
  if (any_short) DSA_TRY(launch_recurrent(a, kDeltaShort, st));
  a.min_len = kDeltaShort + 1;
  a.max_len = INT32_MAX;
  a.ws = static_cast<unsigned char*>(workspace);
  // A head's scan as one CTA on tcgen05, or as CTAs of 16 or 32 of its 128 columns with mma.sync
  // (shorter steps, a quarter of the work a CTA): tcgen05 once the heads of the longest sequence's
  // length that the batch amounts to are more than the GPU holds by four CTAs each (8192 tokens,
  // mma.sync and tcgen05, the whole call: 36 heads 380 and 456 us, 38 heads 641 and 459 us, 64
  // heads 702 and 515 us, 128 heads 1361 and 656 us; 8 uneven sequences, 8 heads 448 and 456 us, 10
  // heads 504 and 475 us, 16 heads 713 and 531 us).  Of the whole call, not of a pass, so that the workspace does not change results.
  const bool umma = (int64_t)R->total_q * a.hv * 4 > (int64_t)R->max_q_len * dev.num_sms;
  for (int h0 = 0; h0 < a.hv; h0 += (int)pass) {
    a.head0 = h0;
    a.heads = (int)std::min<int64_t>(pass, a.hv - h0);
    // The value heads of a key head in one preparation CTA, where a pass is whole groups of them
    // and enough CTAs remain (4 key and 16 value heads, apart and together: 2048 tokens 102 and
    // 110 us the whole call, 8192 tokens 291 and 284 us, 32768 tokens 1047 and 1012 us)
    const int group = a.hv / a.hk;
    const bool whole = h0 % group == 0 && a.heads % group == 0;
    a.per_cta = whole && slots * (a.heads / group) >= 3 * (int64_t)dev.num_sms ? group : 1;
    const unsigned ctas = (unsigned)(slots * (a.heads / a.per_cta));
    if (a.per_cta > 1)
      delta_prep_kernel<true><<<ctas, kPrepThreads, sizeof(PrepSmem), st>>>(a, maps);
    else
      delta_prep_kernel<false><<<ctas, kPrepThreads, sizeof(PrepSmem), st>>>(a, maps);
    DSA_TRY(launched("delta_prep_kernel"));
    // (Without tcgen05:) 16 value columns a CTA while those CTAs fit the GPU at once: the schedulers
    // of an SM then carry one warp each (4096 tokens, 16 and 32 columns: 8 heads 148 and 179 us, 18
    // heads 159 and 188 us, 20 heads 264 and 194 us)
    if (umma) {
      const int64_t ctas = (int64_t)a.batch * a.heads;
      delta_umma_kernel<<<(unsigned)ctas, kUmmaThreads, kUmmaSmem, st>>>(a, maps);
      DSA_TRY(launched("delta_umma_kernel"));
    } else if ((int64_t)a.batch * a.heads * ScanGeo<1>::kParts <= dev.num_sms) {
      DSA_TRY(launch_scan<1>(a, maps, st));
    } else {
      DSA_TRY(launch_scan<2>(a, maps, st));
    }
  }
  return DSA_OK;
}

dsa_status dsa_gated_delta_decode(const dsa_delta_params* P, const dsa_ragged* R, const void* q,
                                  const void* k, const void* v, const float* g, const float* beta,
                                  const float* state_in, float* state_out,
                                  const int32_t* state_index, void* out, void* stream) {
  DSA_TRY(check_delta(P, R));
  if (R->max_q_len > 1 || R->total_q > R->batch) return DSA_ERR_INVALID_ARG;
  DeltaArgs a = {};
  DSA_TRY(delta_args(P, R, q, k, v, g, beta, state_in, state_out, state_index, out, &a));
  HybridDevice dev;
  DSA_TRY(hybrid_device(&dev));
  return launch_recurrent(a, INT32_MAX, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
