// The C ABI of rotary positions, the 16-bit paged cache with attention over it, and attention of packed prompts.

#include <cmath>
#include <new>

#include "attn.h"
#include "common.cuh"
#include "host.h"
#include "prompt.h"
#include "rope.h"

using vbs::aligned16;
using vbs::num_sms;

struct vbs_rope {
  vbs::RopeGeom g;
  int D;
  void* dev_block;
};

struct vbs_kv16 {
  vbs_pkv* kv;
  vbs::Kv16Geom g;                // layer is set per call
  int q_heads, max_q;
  int n_q;                        // of the last plan, 0: none yet
  int64_t planned;                // kv->tables at the last plan
  vbs::Kv8Plan plan;
  float* part;                    // partials of segments in pieces (pieces: where each one's are)
  int2* pieces;
  void* dev_block;
};

struct vbs_pattn {
  cudaStream_t stream;
  int q_heads, kv_heads, head_dim;
  int tiles;                      // the kernel of the last run: 1 the tiles, 0 the rows' kernel, -1: no run yet
  int* status;
};

// Whether an output's rows (n by tok, heads by head elements apart) are different memory, as far as strides of 0 go.
static bool apart(int64_t n, int64_t tok, int64_t heads, int64_t head) { return (n < 2 || tok != 0) && (heads < 2 || head != 0); }

// =====================================================================================
// rotary positions
// =====================================================================================

VBS_EXPORT int rope_frequencies(int rot, double base, int scaling, double factor, double original, double low, double high,
                                double* freq) {
  if (!freq || rot < 0 || rot > vbs::ROPE_MAX_D || rot % 2 != 0) return VBS_EINVAL;
  if (!(base > 0) || !std::isfinite(base) || scaling < VBS_ROPE_NONE || scaling > VBS_ROPE_PARTS) return VBS_EINVAL;
  if (scaling != VBS_ROPE_NONE && (!(factor > 0) || !std::isfinite(factor))) return VBS_EINVAL;
  if (scaling == VBS_ROPE_BASE && rot <= 2) return VBS_EINVAL;
  if (scaling == VBS_ROPE_PARTS && (!(original > 0) || !std::isfinite(original) || !std::isfinite(low) || !(high > low) ||
                                    !std::isfinite(high)))
    return VBS_EINVAL;
  if (scaling == VBS_ROPE_BASE) base *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
  if (!(base > 0) || !std::isfinite(base)) return VBS_EINVAL;
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == VBS_ROPE_LINEAR) f /= factor;
    if (scaling == VBS_ROPE_PARTS) {
      const double turns = original * f / 6.283185307179586476925;
      const double keep = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
      f = f * keep + f / factor * (1.0 - keep);
    }
    if (!std::isfinite(f)) return VBS_EINVAL;
    freq[i] = f;
  }
  return VBS_OK;
}

// x modulo 1 in units of 2^-64 (cut, so that x and -x make 0).
static unsigned long long fraction(double x) {
  const double r = x - std::nearbyint(x);   // exact
  const unsigned long long u = static_cast<unsigned long long>(std::ldexp(std::fabs(r), 64));
  return r < 0 ? 0 - u : u;
}
// The turns that a position makes, modulo 1, in units of 2^-64: freq times 1 / (2 pi) in two doubles, which leave some
// 2^-108 freq of it.  (One double leaves up to 2^-55 freq: 2^-24 of a turn at position 2^31 for a frequency of 1.)
static unsigned long long turn_fraction(double freq) {
  constexpr double HI = 0x1.45f306dc9c883p-3, LO = -0x1.6b01ec5417056p-57;
  const double p = freq * HI;
  return fraction(p) + fraction(std::fma(freq, HI, -p) + freq * LO);
}

VBS_EXPORT int rope_init(vbs_rope** out, int head_dim, int rot, int layout, const double* freq, double amplitude) {
  if (!out) return VBS_EINVAL;
  *out = nullptr;
  if (head_dim < 1 || head_dim > vbs::ROPE_MAX_D || rot < 0 || rot > head_dim || rot % 2 != 0) return VBS_EINVAL;
  if ((layout != VBS_ROPE_HALF && layout != VBS_ROPE_INTERLEAVED) || !std::isfinite(static_cast<float>(amplitude)) ||
      (rot > 0 && !freq))
    return VBS_EINVAL;
  unsigned long long turns[vbs::ROPE_MAX_D / 2] = {};
  for (int i = 0; i < rot / 2; ++i) {
    if (!std::isfinite(freq[i])) return VBS_EINVAL;
    turns[i] = turn_fraction(freq[i]);
  }
  vbs_rope* c = new (std::nothrow) vbs_rope{};
  if (!c) return VBS_ENOMEM;
  if (cudaMalloc(&c->dev_block, sizeof(turns)) != cudaSuccess) {
    cudaGetLastError();
    delete c;
    return VBS_ENOMEM;
  }
  if (cudaMemcpy(c->dev_block, turns, sizeof(turns), cudaMemcpyHostToDevice) != cudaSuccess) {
    cudaFree(c->dev_block);
    delete c;
    return VBS_ECUDA;
  }
  c->g = {static_cast<const unsigned long long*>(c->dev_block), rot, layout, static_cast<float>(amplitude)};
  c->D = head_dim;
  *out = c;
  return VBS_OK;
}

VBS_EXPORT int rope_apply(const vbs_rope* c, int64_t n, const int32_t* pos, int dtype, const void* q, int64_t q_tok, int64_t q_head,
                          void* q_out, int64_t qo_tok, int64_t qo_head, int q_heads, const void* k, int64_t k_tok, int64_t k_head,
                          void* k_out, int64_t ko_tok, int64_t ko_head, int k_heads, vbs_stream_t stream) {
  if (!c || n < 0 || n >= (int64_t{1} << 31) || (dtype != VBS_F32 && dtype != VBS_BF16) || q_heads < 0 || k_heads < 0 ||
      q_heads > VBS_MAX_HEADS || k_heads > VBS_MAX_HEADS)
    return VBS_EINVAL;
  if (n == 0 || q_heads + k_heads == 0) return VBS_OK;
  if (!pos || (q_heads > 0 && (!q || !q_out)) || (k_heads > 0 && (!k || !k_out))) return VBS_EINVAL;
  if (!apart(q_heads > 0 ? n : 0, qo_tok, q_heads, qo_head) || !apart(k_heads > 0 ? n : 0, ko_tok, k_heads, ko_head)) return VBS_EINVAL;
  vbs::RopeArgs a{};
  a.n = n;
  a.pos = pos;
  a.r = c->g;
  a.q = {q, q_out, q_tok, q_head, qo_tok, qo_head, q_heads};
  a.k = {k, k_out, k_tok, k_head, ko_tok, ko_head, k_heads};
  a.D = c->D;
  a.dtype = dtype;
  return vbs::launch_rope(a, num_sms(), reinterpret_cast<cudaStream_t>(stream));
}
VBS_EXPORT int rope_apply_args(const vbs_rope* c, const vbs_rope_args* a) {
  if (!a) return VBS_EINVAL;
  return rope_apply(c, a->n, a->pos, a->dtype, a->q, a->q_tok, a->q_head, a->q_out, a->qo_tok, a->qo_head, a->q_heads, a->k,
                    a->k_tok, a->k_head, a->k_out, a->ko_tok, a->ko_head, a->k_heads, a->stream);
}

VBS_EXPORT int rope_destroy(vbs_rope* c) {
  if (!c) return VBS_OK;
  cudaFree(c->dev_block);
  delete c;
  return VBS_OK;
}

// =====================================================================================
// the 16-bit paged cache
// =====================================================================================

VBS_EXPORT int kv16_init(vbs_kv16** out, vbs_pkv* kv, int q_heads, int max_q) {
  if (!out) return VBS_EINVAL;
  *out = nullptr;
  if (!kv) return VBS_EINVAL;
  const vbs::PagedArgs& a = kv->a;
  if (kv->elem_bytes != 2 || a.slot_bytes % 16 != 0 || a.slot_bytes > 512) return VBS_EINVAL;
  if (q_heads < 1 || q_heads > VBS_MAX_HEADS || q_heads % a.H != 0 || max_q < 1 || max_q > 32) return VBS_EINVAL;
  if (!aligned16(a.pool)) return VBS_EALIGN;
  vbs_kv16* c = new (std::nothrow) vbs_kv16{};
  if (!c) return VBS_ENOMEM;
  c->kv = kv;
  c->q_heads = q_heads;
  c->max_q = max_q;
  vbs::Kv16Geom& g = c->g;
  g.pool = reinterpret_cast<uint16_t*>(a.pool);
  g.NB = static_cast<int64_t>(a.B) * a.S;
  g.L = a.L;
  g.H = a.H;
  g.block = a.block;
  g.D = static_cast<int>(a.slot_bytes / 2);
  g.status = a.status;
  vbs::Carver cv;
  for (int pass = 0; pass < 2; ++pass) {
    c->plan.list = cv.take<int4>(g.NB);
    c->plan.n_pages = cv.take<int>(a.B);
    c->plan.seen = cv.take<int>(kv->R);
    c->part = cv.take<float>(vbs::attn_part_floats(g.D, num_sms()));
    c->pieces = cv.take<int2>(vbs::attn_segments(a.B, a.W, g.H, g.D, q_heads, max_q));
    if (pass == 0) {
      if (cudaMalloc(&c->dev_block, cv.off) != cudaSuccess) {
        cudaGetLastError();
        delete c;
        return VBS_ENOMEM;
      }
      cv = vbs::Carver{};
      cv.base = static_cast<char*>(c->dev_block);
    }
  }
  if (cudaMemsetAsync(c->dev_block, 0, cv.off, kv->stream) != cudaSuccess) {
    cudaFree(c->dev_block);
    delete c;
    return VBS_ECUDA;
  }
  *out = c;
  return VBS_OK;
}

VBS_EXPORT int kv16_append(vbs_kv16* c, int layer, int64_t n, const int64_t* slots, int dtype, const void* k, int64_t k_tok,
                           int64_t k_head, const void* v, int64_t v_tok, int64_t v_head, const vbs_rope* rope, const int32_t* pos,
                           void* k_out, int64_t ko_tok, int64_t ko_head, const void* q, int64_t q_tok, int64_t q_head, void* q_out,
                           int64_t qo_tok, int64_t qo_head) {
  if (!c || layer < 0 || layer >= c->g.L || n < 0 || n >= (int64_t{1} << 31) || (dtype != VBS_F32 && dtype != VBS_BF16))
    return VBS_EINVAL;
  if (rope ? rope->D != c->g.D || (n > 0 && !pos) : pos || k_out || q || q_out) return VBS_EINVAL;
  if (n > 0 && (!k || !v || !slots || (q != nullptr) != (q_out != nullptr))) return VBS_EINVAL;
  if ((q_out && !apart(n, qo_tok, c->q_heads, qo_head)) || (k_out && !apart(n, ko_tok, c->g.H, ko_head))) return VBS_EINVAL;
  if (c->kv->copy_pending) return VBS_ESTATE;
  vbs::RopeArgs a{};
  a.n = n;
  a.pos = rope ? pos : nullptr;
  a.slots = slots;
  if (rope) a.r = rope->g;
  if (q) a.q = {q, q_out, q_tok, q_head, qo_tok, qo_head, c->q_heads};
  a.k = {k, k_out, k_tok, k_head, ko_tok, ko_head, c->g.H};
  a.v = {v, nullptr, v_tok, v_head, 0, 0, c->g.H};
  a.kv = c->g;
  a.kv.layer = layer;
  a.D = c->g.D;
  a.dtype = dtype;
  return vbs::launch_rope(a, num_sms(), c->kv->stream);
}
VBS_EXPORT int kv16_append_args(vbs_kv16* c, const vbs_kv16_args* a) {
  if (!a) return VBS_EINVAL;
  return kv16_append(c, a->layer, a->n, a->slots, a->dtype, a->k, a->k_tok, a->k_head, a->v, a->v_tok, a->v_head, a->rope,
                     a->pos, a->k_out, a->ko_tok, a->ko_head, a->q, a->q_tok, a->q_head, a->q_out, a->qo_tok, a->qo_head);
}

VBS_EXPORT int kv16_plan(vbs_kv16* c, const int32_t* ctx_len, int n_q) {
  if (!c || !ctx_len || n_q < 1 || n_q > c->max_q) return VBS_EINVAL;
  if (c->kv->copy_pending) return VBS_ESTATE;
  const int st = vbs::launch_kv8_plan(c->kv->a, ctx_len, c->plan, c->kv->stream);
  c->n_q = st == VBS_OK ? n_q : 0;
  c->planned = c->kv->tables;
  return st;
}

VBS_EXPORT int kv16_attention(vbs_kv16* c, int layer, const void* q, int64_t q_row, int64_t q_tok, int64_t q_head, float scale,
                              void* out, int64_t o_row, int64_t o_tok, int64_t o_head) {
  if (!c || !q || !out || layer < 0 || layer >= c->g.L || !std::isfinite(scale)) return VBS_EINVAL;
  if (c->n_q == 0 || c->planned != c->kv->tables || c->kv->copy_pending) return VBS_ESTATE;
  if (!apart(c->kv->R, o_row, c->q_heads, o_head) || !apart(c->n_q, o_tok, 0, 0)) return VBS_EINVAL;
  const vbs::QO io{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(out), q_row, q_tok, q_head, o_row, o_tok,
                   o_head, c->n_q, c->q_heads, scale};
  vbs::Kv16Geom g = c->g;
  g.layer = layer;
  return vbs::launch_kv16_attention(c->kv->a, g, io, c->plan, c->part, c->pieces, num_sms(), c->kv->stream);
}
VBS_EXPORT int kv16_attention_args(vbs_kv16* c, const vbs_kv16_query* a) {
  if (!a) return VBS_EINVAL;
  return kv16_attention(c, a->layer, a->q, a->q_row, a->q_tok, a->q_head, a->scale, a->out, a->o_row, a->o_tok, a->o_head);
}

VBS_EXPORT int kv16_destroy(vbs_kv16* c) {
  if (!c) return VBS_OK;
  cudaStreamSynchronize(c->kv->stream);
  cudaFree(c->dev_block);
  delete c;
  return VBS_OK;
}

// =====================================================================================
// packed prompts
// =====================================================================================

VBS_EXPORT int pattn_init(vbs_pattn** out, int q_heads, int kv_heads, int head_dim, vbs_stream_t stream) {
  if (!out) return VBS_EINVAL;
  *out = nullptr;
  if (kv_heads < 1 || q_heads < 1 || q_heads > VBS_MAX_HEADS || q_heads % kv_heads != 0) return VBS_EINVAL;
  if (head_dim < 8 || head_dim > 256 || head_dim % 8 != 0) return VBS_EINVAL;
  vbs_pattn* c = new (std::nothrow) vbs_pattn{};
  if (!c) return VBS_ENOMEM;
  c->stream = reinterpret_cast<cudaStream_t>(stream);
  c->q_heads = q_heads;
  c->kv_heads = kv_heads;
  c->head_dim = head_dim;
  c->tiles = -1;
  void* p = nullptr;
  if (cudaMalloc(&p, sizeof(int)) != cudaSuccess) {
    cudaGetLastError();
    delete c;
    return VBS_ENOMEM;
  }
  c->status = static_cast<int*>(p);
  if (cudaMemsetAsync(p, 0, sizeof(int), c->stream) != cudaSuccess) {
    cudaFree(p);
    delete c;
    return VBS_ECUDA;
  }
  *out = c;
  return VBS_OK;
}

VBS_EXPORT int pattn_run(vbs_pattn* c, int64_t n, int batch, const int32_t* cu, const void* q, int64_t q_tok, int64_t q_head,
                         const void* k, int64_t k_tok, int64_t k_head, const void* v, int64_t v_tok, int64_t v_head, int causal,
                         float scale, void* out, int64_t o_tok, int64_t o_head) {
  if (!c || n < 0 || n > (1 << 30) || batch < 0 || batch > (1 << 30) || !std::isfinite(scale)) return VBS_EINVAL;
  if (n == 0 || batch == 0) return VBS_OK;
  if (!cu || !q || !k || !v || !out || !apart(n, o_tok, c->q_heads, o_head)) return VBS_EINVAL;
  const vbs::PromptArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                          static_cast<uint16_t*>(out), q_tok, q_head, k_tok, k_head, v_tok, v_head, o_tok, o_head, cu,
                          static_cast<int>(n), batch, c->q_heads, c->kv_heads, c->head_dim, causal != 0, scale, c->status};
  c->tiles = vbs::prompt_tc_takes(a) ? 1 : 0;
  return c->tiles ? vbs::launch_prompt_tc(a, num_sms(), c->stream) : vbs::launch_prompt_rows(a, c->stream);
}
VBS_EXPORT int pattn_run_args(vbs_pattn* c, const vbs_pattn_args* a) {
  if (!a) return VBS_EINVAL;
  return pattn_run(c, a->n, a->batch, a->cu, a->q, a->q_tok, a->q_head, a->k, a->k_tok, a->k_head, a->v, a->v_tok, a->v_head,
                   a->causal, a->scale, a->out, a->o_tok, a->o_head);
}

VBS_EXPORT int pattn_kernel(vbs_pattn* c, int* tiles) {
  if (!c || !tiles) return VBS_EINVAL;
  *tiles = c->tiles;
  return VBS_OK;
}

VBS_EXPORT int pattn_status(vbs_pattn* c) {
  if (!c) return VBS_EINVAL;
  if (cudaStreamSynchronize(c->stream) != cudaSuccess) return VBS_ECUDA;
  int h = 0;
  if (cudaMemcpy(&h, c->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return VBS_ECUDA;
  if (h != 0) cudaMemset(c->status, 0, sizeof(int));
  return h;
}

VBS_EXPORT int pattn_destroy(vbs_pattn* c) {
  if (!c) return VBS_OK;
  cudaStreamSynchronize(c->stream);
  cudaFree(c->status);
  delete c;
  return VBS_OK;
}
