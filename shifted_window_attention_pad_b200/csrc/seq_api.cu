// seq_api.cu -- the C ABI of include/swin_seqattn.h: host-side checks, workspace
// sizing and the choice of kernel family. Nothing is allocated and no stream is
// synchronised here.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "seq.h"

namespace swin {
namespace {

bool al16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }
bool al4(const void* p) { return p && ((uintptr_t)p & 3u) == 0; }
int status_of(cudaError_t e) { return e == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA; }
int elem_bytes(int dtype) { return dtype == SWIN_DTYPE_BF16 ? 2 : 4; }

// Two ranges of bytes share an address.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + nb && y < x + na;
}

int check_heads(int heads, int kv_heads, int hd, int dtype) {
  if (heads < 1 || kv_heads < 1 || heads % kv_heads) return SWIN_ERR_INVALID_ARG;
  if (hd < 8 || hd > 256 || (hd & 7)) return SWIN_ERR_INVALID_ARG;
  if (dtype != SWIN_DTYPE_F32 && dtype != SWIN_DTYPE_BF16) return SWIN_ERR_UNSUPPORTED;
  return SWIN_OK;
}

bool bad_stride(int stride, int heads, int hd, int dtype) {
  if (stride == 0) return false;
  return stride < 0 || stride < (long long)heads * hd || (stride * (long long)elem_bytes(dtype)) % 16;
}

int check_seq(const swin_seqattn_desc* d) {
  if (!d) return SWIN_ERR_INVALID_ARG;
  if (d->B < 1 || d->S < 1 || d->S > (1 << 30)) return SWIN_ERR_INVALID_ARG;
  const int rc = check_heads(d->heads, d->kv_heads, d->head_dim, d->dtype);
  if (rc) return rc;
  if (d->window < 0 || d->sinks < 0) return SWIN_ERR_INVALID_ARG;
  if (bad_stride(d->q_stride, d->heads, d->head_dim, d->dtype) ||
      bad_stride(d->kv_stride, d->kv_heads, d->head_dim, d->dtype))
    return SWIN_ERR_INVALID_ARG;
  const long long rows = (long long)d->B * d->S;
  if (rows > 0x7fffffffLL || rows * d->heads * d->head_dim > (1LL << 40))
    return SWIN_ERR_INVALID_ARG;
  if (rows * d->heads > (1LL << 33)) return SWIN_ERR_INVALID_ARG;   // grids of rows
  return SWIN_OK;
}

bool seq_fast(const swin_seqattn_desc* d) {
  return !(d->flags & SWIN_FLAG_FORCE_GENERIC) && seq_fast_supported(d->dtype, d->head_dim);
}

SeqParams seq_params(const swin_seqattn_desc* d) {
  SeqParams p;
  memset(&p, 0, sizeof(p));
  p.B = d->B; p.S = d->S; p.H = d->heads; p.K = d->kv_heads; p.G = d->heads / d->kv_heads;
  p.hd = d->head_dim;
  // a window that hides nothing needs no sinks
  p.window = d->window == 0 || d->window > d->S ? d->S : d->window;
  p.sinks = p.window == d->S ? 0 : (d->sinks > d->S ? d->S : d->sinks);
  p.qs = d->q_stride ? d->q_stride : (long long)d->heads * d->head_dim;
  p.ks = d->kv_stride ? d->kv_stride : (long long)d->kv_heads * d->head_dim;
  p.scale = 1.f / sqrtf((float)d->head_dim);
  p.scale_log2 = kSeqLog2e / sqrtf((float)d->head_dim);
  p.test_timeout = (d->flags & SWIN_FLAG_TEST_TIMEOUT) ? 1 : 0;
  p.ld_stride = ((long long)d->S + 127) / 128 * 128;
  p.plan = make_dkv_plan(p.B, p.S, p.K, p.G, p.hd, p.window, p.sinks,
                         seq_fast(d) ? 128 : seq_generic_tile(p.B, p.S, p.H, p.hd));
  return p;
}

// Header, (lse, D) of every row, partials of the key-side backward.
size_t seq_workspace(const SeqParams& p) {
  return kWsHeader + align256((size_t)p.B * p.H * p.ld_stride * 8) + align256(p.plan.main_bytes) +
         align256(p.plan.sink_bytes);
}
void seq_carve(SeqParams& p, void* ws) {
  char* w = (char*)ws;
  p.status = (int*)w;
  p.nl = (float*)(w += kWsHeader);
  p.nd = p.nl + (size_t)p.B * p.H * p.ld_stride;
  p.main_part = (float*)(w += align256((size_t)p.B * p.H * p.ld_stride * 8));
  p.sink_part = (float*)(w + align256(p.plan.main_bytes));
}

int check_ws(const void* ws, size_t have, size_t need) {
  return !ws || ((uintptr_t)ws & 255u) || have < need ? SWIN_ERR_WORKSPACE : SWIN_OK;
}

// Bytes from the first to behind the last element of a strided operand.
size_t span(long long tokens, long long stride, int heads, int hd, int dtype) {
  return (size_t)((tokens - 1) * stride + (long long)heads * hd) * elem_bytes(dtype);
}

size_t cache_bytes(const CacheParams& p, int dtype) {
  return (size_t)p.pages * p.K * p.ps * p.hd * elem_bytes(dtype);
}

int check_cache(const swin_kvcache_desc* d) {
  if (!d) return SWIN_ERR_INVALID_ARG;
  const int rc = check_heads(d->heads, d->kv_heads, d->head_dim, d->dtype);
  if (rc) return rc;
  if (d->B < 1 || d->page_size < 1 || d->page_size > 65536 || d->num_pages < 1 || d->max_pages < 1)
    return SWIN_ERR_INVALID_ARG;
  if (d->window < 0 || d->sinks < 0) return SWIN_ERR_INVALID_ARG;
  if (bad_stride(d->q_stride, d->heads, d->head_dim, d->dtype) ||
      bad_stride(d->kv_stride, d->kv_heads, d->head_dim, d->dtype))
    return SWIN_ERR_INVALID_ARG;
  const long long len = (long long)d->max_pages * d->page_size;
  if (len > (1LL << 30) || len * d->B > (1LL << 40) / d->kv_heads) return SWIN_ERR_INVALID_ARG;
  if (d->heads / d->kv_heads > 1024 || (long long)d->B * d->heads > 0x7fffffffLL)
    return SWIN_ERR_INVALID_ARG;
  if ((double)d->num_pages * d->kv_heads * d->page_size * d->head_dim > (double)(1LL << 48))
    return SWIN_ERR_INVALID_ARG;
  // evict's own fields are checked by that call; here only that they can size a workspace
  if (d->budget < 0 || d->budget > len || d->recent < 0) return SWIN_ERR_INVALID_ARG;
  return SWIN_OK;
}

CacheParams cache_params(const swin_kvcache_desc* d) {
  CacheParams p;
  memset(&p, 0, sizeof(p));
  p.B = d->B; p.H = d->heads; p.K = d->kv_heads; p.G = d->heads / d->kv_heads; p.hd = d->head_dim;
  p.ps = d->page_size; p.pages = d->num_pages; p.mp = d->max_pages;
  p.max_len = (long long)d->max_pages * d->page_size;
  p.window = d->window == 0 || d->window > p.max_len ? (int)p.max_len : d->window;
  p.sinks = d->sinks > p.max_len ? (int)p.max_len : d->sinks;
  p.with_weights = (d->flags & SWIN_FLAG_KV_WEIGHTS) != 0;
  p.recent = d->recent; p.budget = d->budget;
  p.qs = d->q_stride ? d->q_stride : (long long)d->heads * d->head_dim;
  p.ks = d->kv_stride ? d->kv_stride : (long long)d->kv_heads * d->head_dim;
  p.scale_log2 = kSeqLog2e / sqrtf((float)d->head_dim);
  return p;
}

}  // namespace
}  // namespace swin

using namespace swin;

extern "C" {

int swin_seqattn_path(const swin_seqattn_desc* desc) {
  const int rc = check_seq(desc);
  if (rc) return rc;
  return seq_fast(desc) ? 1 : 0;
}

int swin_seqattn_workspace_size(const swin_seqattn_desc* desc, size_t* bytes) {
  const int rc = check_seq(desc);
  if (rc) return rc;
  if (!bytes) return SWIN_ERR_INVALID_ARG;
  *bytes = seq_workspace(seq_params(desc));
  return SWIN_OK;
}

int swin_seqattn_fwd(const swin_seqattn_desc* desc, const void* q, const void* k, const void* v,
                     const int32_t* lengths, void* out, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int rc = check_seq(desc);
  if (rc) return rc;
  if (!al16(q) || !al16(k) || !al16(v) || !al16(out) || (lse && !al16(lse)) ||
      (lengths && !al4(lengths)))
    return SWIN_ERR_INVALID_ARG;
  SeqParams p = seq_params(desc);
  const long long tok = (long long)p.B * p.S;
  const size_t nq = span(tok, p.qs, p.H, p.hd, desc->dtype);
  const size_t nk = span(tok, p.ks, p.K, p.hd, desc->dtype);
  const size_t no = (size_t)tok * p.H * p.hd * elem_bytes(desc->dtype);
  if (overlap(out, no, q, nq) || overlap(out, no, k, nk) || overlap(out, no, v, nk) ||
      overlap(lse, (size_t)tok * p.H * 4, q, nq) || overlap(lse, (size_t)tok * p.H * 4, k, nk) ||
      overlap(lse, (size_t)tok * p.H * 4, v, nk) || overlap(lse, (size_t)tok * p.H * 4, out, no))
    return SWIN_ERR_INVALID_ARG;
  rc = check_ws(workspace, workspace_bytes, seq_workspace(p));
  if (rc) return rc;
  seq_carve(p, workspace);
  p.q = q; p.k = k; p.v = v; p.lengths = lengths; p.out = out; p.lse = lse;
  cudaStream_t st = (cudaStream_t)stream;
  return status_of(seq_fast(desc) ? seq_fast_forward(p, st)
                                  : seq_generic_forward(p, desc->dtype, st));
}

int swin_seqattn_bwd(const swin_seqattn_desc* desc, const void* q, const void* k, const void* v,
                     const int32_t* lengths, const void* out, const float* lse, const void* dout,
                     void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                     void* stream) {
  int rc = check_seq(desc);
  if (rc) return rc;
  const void* ptrs[] = {q, k, v, out, lse, dout, dq, dk, dv};
  for (const void* x : ptrs)
    if (!al16(x)) return SWIN_ERR_INVALID_ARG;
  if (lengths && !al4(lengths)) return SWIN_ERR_INVALID_ARG;
  SeqParams p = seq_params(desc);
  const long long tok = (long long)p.B * p.S;
  const size_t no = (size_t)tok * p.H * p.hd * elem_bytes(desc->dtype);
  const size_t nq = span(tok, p.qs, p.H, p.hd, desc->dtype);
  const size_t nk = span(tok, p.ks, p.K, p.hd, desc->dtype);
  // dq, dk, dv may interleave in one buffer, never with out, lse or dout, and each
  // starts where nothing else does
  if (dq == dk || dq == dv || dk == dv || dq == q || dk == k || dv == v)
    return SWIN_ERR_INVALID_ARG;
  const void* grads[] = {dq, dk, dv};
  for (const void* x : grads) {
    const size_t n = x == dq ? nq : nk;
    if (overlap(x, n, out, no) || overlap(x, n, dout, no) || overlap(x, n, lse, (size_t)tok * p.H * 4))
      return SWIN_ERR_INVALID_ARG;
  }
  rc = check_ws(workspace, workspace_bytes, seq_workspace(p));
  if (rc) return rc;
  seq_carve(p, workspace);
  p.q = q; p.k = k; p.v = v; p.lengths = lengths; p.o = out; p.lse_in = lse; p.dout = dout;
  p.dq = dq; p.dk = dk; p.dv = dv;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = seq_prep(p, desc->dtype, st);
  if (e == cudaSuccess)
    e = seq_fast(desc) ? seq_fast_backward(p, st) : seq_generic_backward(p, desc->dtype, st);
  if (e == cudaSuccess) e = seq_reduce(p, desc->dtype, st);
  return status_of(e);
}

int swin_kvcache_workspace_size(const swin_kvcache_desc* desc, size_t* bytes) {
  const int rc = check_cache(desc);
  if (rc) return rc;
  if (!bytes) return SWIN_ERR_INVALID_ARG;
  *bytes = kWsHeader + cache_workspace(cache_params(desc), desc->dtype);
  return SWIN_OK;
}

int swin_kvcache_append(const swin_kvcache_desc* desc, int32_t T, const void* k, const void* v,
                        const int32_t* counts, const int32_t* lengths, const int32_t* page_table,
                        void* k_cache, void* v_cache, void* workspace, size_t workspace_bytes,
                        void* stream) {
  int rc = check_cache(desc);
  if (rc) return rc;
  if (T < 1 || !al16(k) || !al16(v) || !al4(lengths) || !al4(page_table) || !al16(k_cache) ||
      !al16(v_cache) || (counts && !al4(counts)))
    return SWIN_ERR_INVALID_ARG;
  rc = check_ws(workspace, workspace_bytes, kWsHeader);
  if (rc) return rc;
  CacheParams p = cache_params(desc);
  const size_t nc = cache_bytes(p, desc->dtype);
  const size_t nn = span((long long)p.B * T, p.ks, p.K, p.hd, desc->dtype);
  if (overlap(k_cache, nc, v_cache, nc) || overlap(k, nn, k_cache, nc) ||
      overlap(k, nn, v_cache, nc) || overlap(v, nn, k_cache, nc) || overlap(v, nn, v_cache, nc))
    return SWIN_ERR_INVALID_ARG;
  if ((long long)T * p.K * p.hd > (1LL << 31) || (long long)T * p.B * p.K * p.hd > (1LL << 38))
    return SWIN_ERR_INVALID_ARG;
  p.status = (int*)workspace;
  p.T = T; p.k_new = k; p.v_new = v; p.counts = counts; p.lengths = lengths; p.table = page_table;
  p.kc = k_cache; p.vc = v_cache;
  return status_of(cache_append(p, desc->dtype, (cudaStream_t)stream));
}

int swin_kvcache_decode(const swin_kvcache_desc* desc, const void* q, const void* k_new,
                        const void* v_new, const int32_t* lengths, const int32_t* page_table,
                        void* k_cache, void* v_cache, const float* weights, float* new_weights,
                        void* out, float* lse, void* workspace, size_t workspace_bytes,
                        void* stream) {
  int rc = check_cache(desc);
  if (rc) return rc;
  if (!al16(q) || !al4(lengths) || !al4(page_table) || !al16(k_cache) || !al16(v_cache) ||
      !al16(out) || (lse && !al16(lse)))
    return SWIN_ERR_INVALID_ARG;
  if ((k_new == nullptr) != (v_new == nullptr)) return SWIN_ERR_INVALID_ARG;
  if (k_new && (!al16(k_new) || !al16(v_new))) return SWIN_ERR_INVALID_ARG;
  if ((weights == nullptr) != (new_weights == nullptr)) return SWIN_ERR_INVALID_ARG;
  if (weights && (!al16(weights) || !al16(new_weights) || !(desc->flags & SWIN_FLAG_KV_WEIGHTS)))
    return SWIN_ERR_INVALID_ARG;
  CacheParams p = cache_params(desc);
  // out is written while other blocks still read q and the new rows
  const size_t nc = cache_bytes(p, desc->dtype), nw = (size_t)p.B * p.K * p.max_len * 4;
  const size_t no = (size_t)p.B * p.H * p.hd * elem_bytes(desc->dtype);
  const size_t nn = span(p.B, p.ks, p.K, p.hd, desc->dtype);
  if (overlap(k_cache, nc, v_cache, nc) ||
      overlap(out, no, q, span(p.B, p.qs, p.H, p.hd, desc->dtype)) || overlap(out, no, k_new, nn) ||
      overlap(out, no, v_new, nn) || overlap(out, no, k_cache, nc) || overlap(out, no, v_cache, nc) ||
      overlap(lse, (size_t)p.B * p.H * 4, out, no) ||
      (weights != new_weights && overlap(weights, nw, new_weights, nw)))
    return SWIN_ERR_INVALID_ARG;
  rc = check_ws(workspace, workspace_bytes, kWsHeader + cache_workspace(p, desc->dtype));
  if (rc) return rc;
  p.status = (int*)workspace;
  p.ws = (char*)workspace + kWsHeader;
  p.q = q; p.k_new = k_new; p.v_new = v_new; p.lengths = lengths; p.table = page_table;
  p.kc = k_cache; p.vc = v_cache; p.w = weights; p.w_out = new_weights; p.out = out; p.lse = lse;
  return status_of(cache_decode(p, desc->dtype, (cudaStream_t)stream));
}

int swin_kvcache_evict(const swin_kvcache_desc* desc, const float* weights,
                       const int32_t* lengths, const int32_t* page_table,
                       const int32_t* dst_page_table, void* k_cache, void* v_cache,
                       float* new_weights, int32_t* new_lengths, int32_t* kept, void* workspace,
                       size_t workspace_bytes, void* stream) {
  int rc = check_cache(desc);
  if (rc) return rc;
  if (desc->budget < 1 || (long long)desc->sinks + desc->recent > desc->budget)
    return SWIN_ERR_INVALID_ARG;
  if (!al16(weights) || !al16(new_weights) || !al4(lengths) || !al4(new_lengths) ||
      !al4(page_table) || !al4(dst_page_table) || !al16(k_cache) || !al16(v_cache) ||
      (kept && !al4(kept)))
    return SWIN_ERR_INVALID_ARG;
  CacheParams p = cache_params(desc);
  const size_t nw = (size_t)p.B * p.K * p.max_len * 4, nc = cache_bytes(p, desc->dtype);
  if (overlap(k_cache, nc, v_cache, nc) || overlap(weights, nw, new_weights, nw) || overlap(lengths, p.B * 4, new_lengths, p.B * 4) ||
      page_table == dst_page_table)
    return SWIN_ERR_INVALID_ARG;
  rc = check_ws(workspace, workspace_bytes, kWsHeader + cache_workspace(p, desc->dtype));
  if (rc) return rc;
  p.status = (int*)workspace;
  p.ws = (char*)workspace + kWsHeader;
  p.w = weights; p.w_out = new_weights; p.lengths = lengths; p.table = page_table;
  p.dst_table = dst_page_table; p.kc = k_cache; p.vc = v_cache; p.new_len = new_lengths;
  p.kept = kept;
  return status_of(cache_evict(p, desc->dtype, (cudaStream_t)stream));
}

}  // extern "C"
