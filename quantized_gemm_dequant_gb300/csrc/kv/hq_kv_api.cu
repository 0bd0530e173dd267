// C ABI of the paged key-value cache: argument validation and kernel launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../../include/hq.h"
#include "hq_kv.h"
#include "hq_kv_attention.cuh"

namespace hq {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int kMaxHeads = 1024;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

hq_status_t check_format(const hq_kv_format_t* f) {
  if (!f) return HQ_ERR_INVALID_ARG;
  if (f->kind != HQ_KV_BF16 && f->kind != HQ_KV_E4M3 && f->kind != HQ_KV_NVFP4) return HQ_ERR_UNSUPPORTED;
  if (f->head_dim != 64 && f->head_dim != 128 && f->head_dim != 256) return HQ_ERR_UNSUPPORTED;
  if (f->page_size < 1 || f->page_size > 1024 || f->num_heads < 1 || f->num_heads > kMaxHeads || f->num_pages < 1 ||
      f->num_pages > INT32_MAX)
    return HQ_ERR_INVALID_ARG;
  if (f->page_size % KV_BLOCK) return HQ_ERR_ALIGNMENT;
  // the kernels count a pool's 16-token blocks in 31 bits: more than any device holds
  return f->num_pages * f->num_heads * (f->page_size / KV_BLOCK) > INT32_MAX ? HQ_ERR_INVALID_ARG : HQ_OK;
}

hq_status_t check_q_heads(const hq_kv_format_t* f, int32_t num_q_heads) {
  return num_q_heads < 1 || num_q_heads > 16 * kMaxHeads || num_q_heads % f->num_heads ? HQ_ERR_INVALID_ARG : HQ_OK;
}

hq_status_t check_cache(const hq_kv_format_t* f, const hq_kv_cache_t* c) {
  if (!c || !c->k || !c->v) return HQ_ERR_INVALID_ARG;
  if (f->kind != HQ_KV_BF16 && (!c->k_scale || !c->v_scale)) return HQ_ERR_INVALID_ARG;
  if (f->kind == HQ_KV_NVFP4 && (!c->k_global || !c->v_global)) return HQ_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) ||
      !aligned(c->k_global, 4) || !aligned(c->v_global, 4))
    return HQ_ERR_ALIGNMENT;
  return HQ_OK;
}

// (sequence, head, row tile) triples of the attention
int64_t pairs(const hq_kv_format_t* f, int64_t batch, int32_t num_q_heads) {
  return batch * f->num_heads * ((num_q_heads / f->num_heads + KA_ROWS - 1) / KA_ROWS);
}

// The attention counts its work in 31 bits, and a triple as one unit at least beside its own: a batch past that is refused
// here, lengths that are past it by the kernel.
bool countable(const hq_kv_format_t* f, int64_t batch, int32_t num_q_heads) {
  return pairs(f, batch, num_q_heads) <= INT32_MAX / (ka_extra(f->kind, f->head_dim) + 1);
}

hq_status_t check_workspace(const hq_kv_format_t* f, int64_t batch, int32_t num_q_heads, const void* ws,
                            size_t ws_bytes) {
  if (!ws || ws_bytes < hq_kv_workspace_bytes(f, batch, num_q_heads)) return HQ_ERR_WORKSPACE;
  return aligned(ws, 16) ? HQ_OK : HQ_ERR_ALIGNMENT;
}

KvView view(const hq_kv_format_t* f, const hq_kv_cache_t* c) {
  KvView v;
  v.k = (uint8_t*)c->k;
  v.v = (uint8_t*)c->v;
  v.k_scale = (uint8_t*)c->k_scale;
  v.v_scale = (uint8_t*)c->v_scale;
  v.k_global = c->k_global;
  v.v_global = c->v_global;
  v.num_pages = f->num_pages;
  v.page_size = f->page_size;
  v.heads = f->num_heads;
  return v;
}

// SMs of the current device, looked up once per device (without a device: a GB300's, for host-only queries)
int num_sms() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

hq_status_t launched(cudaError_t e) { return e == cudaSuccess ? HQ_OK : HQ_ERR_CUDA; }

}  // namespace
}  // namespace hq

using namespace hq;

extern "C" {

size_t hq_kv_workspace_bytes(const hq_kv_format_t* fmt, int64_t batch, int32_t num_q_heads) {
  if (check_format(fmt) != HQ_OK || batch < 0 || batch > kMaxRows) return 0;
  if (batch == 0) return KV_HEADER_BYTES;
  if (check_q_heads(fmt, num_q_heads) != HQ_OK || batch * num_q_heads > kMaxRows || !countable(fmt, batch, num_q_heads))
    return 0;
  return ka_counters_at(num_sms()) + sizeof(int) * (size_t)pairs(fmt, batch, num_q_heads);
}

hq_status_t hq_kv_write(const hq_kv_format_t* fmt, const hq_kv_cache_t* cache, const hq_kv_rows_t* r, void* workspace,
                        size_t ws_bytes, hq_stream_t stream) {
  hq_status_t st = check_format(fmt);
  if (st != HQ_OK) return st;
  if (!r || r->T < 0 || r->T > kMaxRows || !(r->eps >= 0.0f) || isinf(r->eps)) return HQ_ERR_INVALID_ARG;
  if ((st = check_q_heads(fmt, r->num_q_heads)) != HQ_OK) return st;
  if (r->rotary_dim < 0 || r->rotary_dim > fmt->head_dim || r->interleaved < 0 || r->interleaved > 1)
    return HQ_ERR_INVALID_ARG;
  if (r->rotary_dim % 16) return HQ_ERR_ALIGNMENT;
  const int64_t row = ((int64_t)r->num_q_heads + 2 * fmt->num_heads) * fmt->head_dim;
  if (r->row_stride < row || r->row_stride > ((int64_t)1 << 40)) return HQ_ERR_INVALID_ARG;
  if (r->row_stride % 8) return HQ_ERR_ALIGNMENT;
  if (r->T == 0) return HQ_OK;
  if ((st = check_cache(fmt, cache)) != HQ_OK) return st;
  if (!r->qkv || !r->slots || !r->q_out) return HQ_ERR_INVALID_ARG;
  if (r->rotary_dim && (!r->cos_sin || !r->positions || r->num_positions < 1)) return HQ_ERR_INVALID_ARG;
  if (!aligned(r->qkv, 16) || !aligned(r->slots, 8) || !aligned(r->q_out, 16) || !aligned(r->cos_sin, 16) ||
      !aligned(r->positions, 4) || !aligned(r->q_norm, 16) || !aligned(r->k_norm, 16))
    return HQ_ERR_ALIGNMENT;
  if ((st = check_workspace(fmt, 0, 1, workspace, ws_bytes)) != HQ_OK) return st;
  KvWriteArgs a;
  a.kv = view(fmt, cache);
  a.qkv = (const uint16_t*)r->qkv;
  a.row_stride = r->row_stride;
  a.T = r->T;
  a.q_heads = r->num_q_heads;
  a.rotary = r->rotary_dim;
  a.interleaved = r->interleaved;
  a.eps = r->eps;
  a.q_norm = (const uint16_t*)r->q_norm;
  a.k_norm = (const uint16_t*)r->k_norm;
  a.cos_sin = r->cos_sin;
  a.num_positions = r->num_positions;
  a.positions = r->positions;
  a.slots = r->slots;
  a.q_out = (uint16_t*)r->q_out;
  a.status = (int*)workspace;
  return launched(launch_kv_write(fmt->kind, fmt->head_dim, a, (cudaStream_t)stream));
}

hq_status_t hq_kv_read(const hq_kv_format_t* fmt, const hq_kv_cache_t* cache, const hq_kv_read_t* x, void* workspace,
                       size_t ws_bytes, hq_stream_t stream) {
  hq_status_t st = check_format(fmt);
  if (st != HQ_OK) return st;
  if (!x || x->B < 0 || x->B > kMaxRows || x->total < 0 || x->total > ((int64_t)1 << 34) || x->table_stride < 0 ||
      x->table_stride > kMaxRows)
    return HQ_ERR_INVALID_ARG;
  if (x->B == 0 || x->total == 0) return HQ_OK;
  if ((st = check_cache(fmt, cache)) != HQ_OK) return st;
  if ((x->table_stride && !x->page_table) || !x->starts || !x->k_out || !x->v_out) return HQ_ERR_INVALID_ARG;
  if (!aligned(x->page_table, 4) || !aligned(x->starts, 8) || !aligned(x->first, 4) || !aligned(x->k_out, 16) ||
      !aligned(x->v_out, 16))
    return HQ_ERR_ALIGNMENT;
  if ((st = check_workspace(fmt, 0, 1, workspace, ws_bytes)) != HQ_OK) return st;
  KvReadArgs a;
  a.kv = view(fmt, cache);
  a.page_table = x->page_table;
  a.table_stride = x->table_stride;
  a.starts = x->starts;
  a.first = x->first;
  a.B = x->B;
  a.total = x->total;
  a.k_out = (uint16_t*)x->k_out;
  a.v_out = (uint16_t*)x->v_out;
  a.status = (int*)workspace;
  return launched(launch_kv_read(fmt->kind, fmt->head_dim, a, (cudaStream_t)stream));
}

hq_status_t hq_paged_attention(const hq_kv_format_t* fmt, const hq_kv_cache_t* cache, const hq_kv_attention_t* x,
                               void* workspace, size_t ws_bytes, hq_stream_t stream) {
  hq_status_t st = check_format(fmt);
  if (st != HQ_OK) return st;
  if (!x) return HQ_ERR_INVALID_ARG;
  if ((st = check_q_heads(fmt, x->num_q_heads)) != HQ_OK) return st;
  if (x->B < 0 || x->B > kMaxRows || x->B * x->num_q_heads > kMaxRows || !countable(fmt, x->B, x->num_q_heads) ||
      x->table_stride < 0 || x->table_stride > kMaxRows || x->window < 0 || !isfinite(x->scale) || !(x->softcap >= 0.0f) ||
      isinf(x->softcap))
    return HQ_ERR_INVALID_ARG;
  if (x->B == 0) return HQ_OK;
  if ((st = check_cache(fmt, cache)) != HQ_OK) return st;
  if (!x->q || (x->table_stride && !x->page_table) || !x->lens || !x->out) return HQ_ERR_INVALID_ARG;
  if (!aligned(x->q, 16) || !aligned(x->page_table, 4) || !aligned(x->lens, 4) || !aligned(x->out, 16) ||
      !aligned(x->lse, 4))
    return HQ_ERR_ALIGNMENT;
  if ((st = check_workspace(fmt, x->B, x->num_q_heads, workspace, ws_bytes)) != HQ_OK) return st;
  KvAttnArgs a;
  a.kv = view(fmt, cache);
  a.q = (const uint16_t*)x->q;
  a.group = x->num_q_heads / fmt->num_heads;
  a.page_table = x->page_table;
  a.table_stride = x->table_stride;
  a.lens = x->lens;
  a.B = x->B;
  const int64_t most = x->table_stride * fmt->page_size;
  a.most = most < kMaxRows ? most : kMaxRows;
  a.scale = x->scale;
  a.window = x->window;
  a.softcap = x->softcap;
  a.out = (uint16_t*)x->out;
  a.lse = x->lse;
  a.status = (int*)workspace;
  const int sms = num_sms();
  const int64_t seen = a.window > 0 && a.window < a.most ? a.window + KV_BLOCK : a.most;
  const auto launch = fmt->kind == HQ_KV_BF16 ? launch_kv_attention_bf16
                                              : (fmt->kind == HQ_KV_E4M3 ? launch_kv_attention_e4m3
                                                                         : launch_kv_attention_nvfp4);
  return launched(launch(fmt->head_dim, a, sms, seen, (uint8_t*)workspace, (cudaStream_t)stream));
}

}  // extern "C"
