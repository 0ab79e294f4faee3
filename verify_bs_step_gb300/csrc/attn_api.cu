// The C ABI of the attention operators: the 8-bit paged cache.

#include <new>

#include "common.cuh"
#include "host.h"
#include "kv8.h"

using vbs::aligned16;
using vbs::num_sms;

struct vbs_kv8 {
  vbs_pkv* kv;
  vbs::Kv8Geom g;                 // layer is set per call
  int q_heads, max_q;
};

VBS_EXPORT int kv8_init(vbs_kv8** out, vbs_pkv* kv, int format, float* scales, int q_heads, int max_q) {
  if (!out) return VBS_EINVAL;
  *out = nullptr;
  if (!kv || !scales || (format != VBS_I8 && format != VBS_E4M3)) return VBS_EINVAL;
  const vbs::PagedArgs& a = kv->a;
  if (kv->elem_bytes != 1 || a.slot_bytes % 16 != 0 || a.slot_bytes > 256) return VBS_EINVAL;
  if (q_heads < 1 || q_heads % a.H != 0 || max_q < 1 || max_q > 32) return VBS_EINVAL;
  if (!aligned16(a.pool)) return VBS_EALIGN;
  if (a.scales) return VBS_ESTATE;
  vbs_kv8* c = new (std::nothrow) vbs_kv8{};
  if (!c) return VBS_ENOMEM;
  c->kv = kv;
  c->q_heads = q_heads;
  c->max_q = max_q;
  vbs::Kv8Geom& g = c->g;
  g.pool = a.pool;
  g.scales = scales;
  g.fmt = format;
  g.NB = static_cast<int64_t>(a.B) * a.S;
  g.L = a.L;
  g.H = a.H;
  g.block = a.block;
  g.D = static_cast<int>(a.slot_bytes);
  g.status = a.status;
  kv->a.scales = scales;          // copy-on-write carries a page's scales along
  *out = c;
  return VBS_OK;
}

VBS_EXPORT int kv8_append(vbs_kv8* c, int layer, const void* k, const void* v, int64_t k_tok, int64_t k_head,
                          int64_t v_tok, int64_t v_head, int dtype, int64_t n, const int64_t* slots) {
  if (!c || layer < 0 || layer >= c->g.L || n < 0 || (dtype != VBS_F32 && dtype != VBS_BF16)) return VBS_EINVAL;
  if (n > 0 && (!k || !v || !slots)) return VBS_EINVAL;
  const vbs::Kv8Src src{k, v, k_tok, k_head, v_tok, v_head, dtype};
  vbs::Kv8Geom g = c->g;
  g.layer = layer;
  return vbs::launch_kv8_append(g, src, n, slots, num_sms(), c->kv->stream);
}

VBS_EXPORT int kv8_read(vbs_kv8* c, int layer, int64_t n, const int64_t* slots, void* k_out, void* v_out) {
  if (!c || layer < 0 || layer >= c->g.L || n < 0) return VBS_EINVAL;
  if (n > 0 && (!slots || !k_out || !v_out)) return VBS_EINVAL;
  if (!aligned16(k_out) || !aligned16(v_out)) return VBS_EALIGN;
  vbs::Kv8Geom g = c->g;
  g.layer = layer;
  return vbs::launch_kv8_read(g, n, slots, k_out, v_out, num_sms(), c->kv->stream);
}

VBS_EXPORT int kv8_destroy(vbs_kv8* c) {
  if (!c) return VBS_OK;
  cudaStreamSynchronize(c->kv->stream);
  c->kv->a.scales = nullptr;
  delete c;
  return VBS_OK;
}
