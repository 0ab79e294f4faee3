// The C ABI of the attention operators: the 8-bit paged cache, attention over it, cross attention.

#include <cmath>
#include <new>

#include "attn.h"
#include "common.cuh"
#include "host.h"
#include "kv8.h"

using vbs::aligned16;
using vbs::num_sms;

struct vbs_kv8 {
  vbs_pkv* kv;
  vbs::Kv8Geom g;                 // layer is set per call
  int q_heads, max_q;
  int n_q;                        // of the last plan, 0: none yet
  int64_t planned;                // kv->tables at the last plan
  vbs::Kv8Plan plan;
  float* part;                    // partials of segments in pieces (pieces: where each one's are)
  int2* pieces;
  void* dev_block;
};

struct vbs_xattn {
  vbs::EncKV e;                   // the tensors are set per call
  cudaStream_t stream;
  int q_heads, max_q, max_len;
  int tiles;                      // the kernel of the last run: 1 the tiles, 0 the split kernel, -1: no run yet
  float* part;
  int2* pieces;
  void* dev_block;
};

VBS_EXPORT int kv8_init(vbs_kv8** out, vbs_pkv* kv, int format, float* scales, int q_heads, int max_q) {
  if (!out) return VBS_EINVAL;
  *out = nullptr;
  if (!kv || !scales || (format != VBS_I8 && format != VBS_E4M3)) return VBS_EINVAL;
  const vbs::PagedArgs& a = kv->a;
  if (kv->elem_bytes != 1 || a.slot_bytes % 16 != 0 || a.slot_bytes > 256) return VBS_EINVAL;
  if (q_heads < 1 || q_heads % a.H != 0 || max_q < 1 || max_q > 32) return VBS_EINVAL;
  if (!aligned16(a.pool)) return VBS_EALIGN;
  if (kv->scales) return VBS_ESTATE;
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
  kv->scales = scales;
  *out = c;
  return VBS_OK;
}

VBS_EXPORT int kv8_append(vbs_kv8* c, int layer, const void* k, const void* v, int64_t k_tok, int64_t k_head,
                          int64_t v_tok, int64_t v_head, int dtype, int64_t n, const int64_t* slots) {
  if (!c || layer < 0 || layer >= c->g.L || n < 0 || (dtype != VBS_F32 && dtype != VBS_BF16)) return VBS_EINVAL;
  if (n > 0 && (!k || !v || !slots)) return VBS_EINVAL;
  if (c->kv->copy_pending) return VBS_ESTATE;
  const vbs::Kv8Src src{k, v, k_tok, k_head, v_tok, v_head, dtype};
  vbs::Kv8Geom g = c->g;
  g.layer = layer;
  return vbs::launch_kv8_append(g, src, n, slots, num_sms(), c->kv->stream);
}

VBS_EXPORT int kv8_read(vbs_kv8* c, int layer, int64_t n, const int64_t* slots, void* k_out, void* v_out) {
  if (!c || layer < 0 || layer >= c->g.L || n < 0) return VBS_EINVAL;
  if (n > 0 && (!slots || !k_out || !v_out)) return VBS_EINVAL;
  if (!aligned16(k_out) || !aligned16(v_out)) return VBS_EALIGN;
  if (c->kv->copy_pending) return VBS_ESTATE;
  vbs::Kv8Geom g = c->g;
  g.layer = layer;
  return vbs::launch_kv8_read(g, n, slots, k_out, v_out, num_sms(), c->kv->stream);
}

VBS_EXPORT int kv8_plan(vbs_kv8* c, const int32_t* ctx_len, int n_q) {
  if (!c || !ctx_len || n_q < 1 || n_q > c->max_q) return VBS_EINVAL;
  if (c->kv->copy_pending) return VBS_ESTATE;
  const int st = vbs::launch_kv8_plan(c->kv->a, ctx_len, c->plan, c->kv->stream);
  c->n_q = st == VBS_OK ? n_q : 0;
  c->planned = c->kv->tables;
  return st;
}

VBS_EXPORT int kv8_attention(vbs_kv8* c, int layer, const void* q, int64_t q_row, int64_t q_tok, int64_t q_head,
                             float scale, void* out, int64_t o_row, int64_t o_tok, int64_t o_head) {
  if (!c || !q || !out || layer < 0 || layer >= c->g.L || !std::isfinite(scale)) return VBS_EINVAL;
  if (c->n_q == 0 || c->planned != c->kv->tables || c->kv->copy_pending) return VBS_ESTATE;
  const vbs::QO io{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(out), q_row, q_tok, q_head, o_row, o_tok,
                   o_head, c->n_q, c->q_heads, scale};
  vbs::Kv8Geom g = c->g;
  g.layer = layer;
  return vbs::launch_kv8_attention(c->kv->a, g, io, c->plan, c->part, c->pieces, num_sms(), c->kv->stream);
}

VBS_EXPORT int kv8_destroy(vbs_kv8* c) {
  if (!c) return VBS_OK;
  cudaStreamSynchronize(c->kv->stream);
  c->kv->scales = nullptr;
  cudaFree(c->dev_block);
  delete c;
  return VBS_OK;
}

// =====================================================================================
// cross attention
// =====================================================================================

VBS_EXPORT int xattn_init(vbs_xattn** out, int batch, int W, int q_heads, int kv_heads, int head_dim, int max_q,
                          int max_len, vbs_stream_t stream) {
  if (!out) return VBS_EINVAL;
  *out = nullptr;
  if (batch < 1 || W < 1 || W > vbs::WMAX || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0) return VBS_EINVAL;
  if (head_dim < 8 || head_dim > 256 || head_dim % 8 != 0 || max_q < 1 || max_len < 1) return VBS_EINVAL;
  if (static_cast<int64_t>(batch) * W * q_heads >= (int64_t{1} << 31) ||
      static_cast<int64_t>(batch) * W * q_heads * max_q >= (int64_t{1} << 31)) return VBS_EINVAL;
  vbs_xattn* c = new (std::nothrow) vbs_xattn{};
  if (!c) return VBS_ENOMEM;
  c->stream = reinterpret_cast<cudaStream_t>(stream);
  c->q_heads = q_heads;
  c->max_q = max_q;
  c->max_len = max_len;
  c->tiles = -1;
  vbs::EncKV& e = c->e;
  e.B = batch;
  e.W = W;
  e.H = kv_heads;
  e.D = head_dim;
  vbs::Carver cv;
  for (int pass = 0; pass < 2; ++pass) {
    e.status = cv.take<int>(1);
    c->part = cv.take<float>(vbs::attn_part_floats(head_dim, num_sms()));
    c->pieces = cv.take<int2>(vbs::attn_segments(batch, W, kv_heads, head_dim, q_heads, max_q));
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
  if (cudaMemsetAsync(c->dev_block, 0, cv.off, c->stream) != cudaSuccess) {
    cudaFree(c->dev_block);
    delete c;
    return VBS_ECUDA;
  }
  *out = c;
  return VBS_OK;
}

VBS_EXPORT int xattn_run(vbs_xattn* c, const void* q, int64_t q_row, int64_t q_tok, int64_t q_head, int n_q,
                         const void* k, int64_t k_sent, int64_t k_pos, int64_t k_head, const void* v, int64_t v_sent,
                         int64_t v_pos, int64_t v_head, int len, const int32_t* enc_len, float scale, void* out,
                         int64_t o_row, int64_t o_tok, int64_t o_head) {
  if (!c || n_q < 1 || n_q > c->max_q || len < 0 || len > c->max_len || !std::isfinite(scale)) return VBS_EINVAL;
  if (!q || !out || !enc_len || (len > 0 && (!k || !v))) return VBS_EINVAL;
  const vbs::QO io{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(out), q_row, q_tok, q_head, o_row, o_tok,
                   o_head, n_q, c->q_heads, scale};
  vbs::EncKV e = c->e;
  e.k = static_cast<const uint16_t*>(k);
  e.v = static_cast<const uint16_t*>(v);
  e.k_sent = k_sent;
  e.k_pos = k_pos;
  e.k_head = k_head;
  e.v_sent = v_sent;
  e.v_pos = v_pos;
  e.v_head = v_head;
  e.len = enc_len;
  e.S = len;
  return vbs::launch_xattn(e, io, c->part, c->pieces, num_sms(), c->stream, &c->tiles);
}

VBS_EXPORT int xattn_kernel(vbs_xattn* c, int* tiles) {
  if (!c || !tiles) return VBS_EINVAL;
  *tiles = c->tiles;
  return VBS_OK;
}

VBS_EXPORT int xattn_status(vbs_xattn* c) {
  if (!c) return VBS_EINVAL;
  if (cudaStreamSynchronize(c->stream) != cudaSuccess) return VBS_ECUDA;
  int h = 0;
  if (cudaMemcpy(&h, c->e.status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return VBS_ECUDA;
  if (h != 0) cudaMemset(c->e.status, 0, sizeof(int));
  return h;
}

VBS_EXPORT int xattn_destroy(vbs_xattn* c) {
  if (!c) return VBS_OK;
  cudaStreamSynchronize(c->stream);
  cudaFree(c->dev_block);
  delete c;
  return VBS_OK;
}
