// C ABI of the rotation and of the paged 4-bit cache: argument checks and
// launches.  See include/vq_kivi.h.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "paged.cuh"
#include "vqk_internal.cuh"

using namespace vqk;

namespace {

int fail(int code, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return code;
}

int cuda_fail(cudaError_t e, const char *what) {
  return fail(VQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// SMs of the current device
int sm_count(int *out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "device query");
}

int check_dtype(int dtype, bool with_f32, int *elem) {
  if (dtype != VQ_F16 && dtype != VQ_BF16 && !(with_f32 && dtype == VQ_F32))
    return fail(VQ_ERR_UNSUPPORTED, "dtype %d (supported: %s)", dtype,
                with_f32 ? "fp16, bf16, fp32" : "fp16, bf16");
  *elem = dtype == VQ_F32 ? 4 : 2;
  return VQ_OK;
}

int check_rows(const vq_kivi_rows *r, const char *name, int elem, int64_t tokens, bool out,
               HeadRows *to) {
  if (r->heads < 1 || r->heads > 1024)
    return fail(VQ_ERR_ARG, "%s: heads=%d outside [1, 1024]", name, r->heads);
  if (tokens > 0 && (!r->x || (out && !r->out)))
    return fail(VQ_ERR_ARG, "%s: NULL pointer", name);
  const int v = 16 / elem;
  if (!aligned(r->x, 16) || r->x_token % v || r->x_head % v || !aligned(r->weight, 16) ||
      (out && (!aligned(r->out, 16) || r->out_token % v || r->out_head % v)))
    return fail(VQ_ERR_ARG, "%s: rows must be 16-byte aligned", name);
  to->x = r->x;
  to->out = out ? r->out : nullptr;
  to->weight = r->weight;
  to->x_token = r->x_token;
  to->x_head = r->x_head;
  to->out_token = r->out_token;
  to->out_head = r->out_head;
  to->heads = r->heads;
  return VQ_OK;
}

int check_rope(const vq_kivi_rope *p, int D, int64_t tokens, const void *positions, int pos_64,
               int64_t pos_stride, bool places, RopeArgs *to) {
  *to = RopeArgs();
  if (!p) return VQ_OK;
  if (p->rot_dim < 0 || p->rot_dim > D || p->rot_dim % 16)
    return fail(VQ_ERR_UNSUPPORTED, "rot_dim=%d: a multiple of 16 in [0, D=%d]", p->rot_dim, D);
  if (p->n_axes < 1 || p->n_axes > 4)
    return fail(VQ_ERR_ARG, "n_axes=%d outside [1, 4]", p->n_axes);
  if (!std::isfinite(p->scale)) return fail(VQ_ERR_ARG, "the rotation's scale is not finite");
  if (p->rot_dim > 0) {
    if (!p->turns || (p->n_axes > 1 && !p->axis))
      return fail(VQ_ERR_ARG, "rotation: NULL turns or axis");
    if (!aligned(p->turns, 8)) return fail(VQ_ERR_ARG, "turns must be 8-byte aligned");
    if (!positions && !places && tokens > 0) return fail(VQ_ERR_ARG, "positions is NULL");
    if (positions && !aligned(positions, pos_64 ? 8 : 4))
      return fail(VQ_ERR_ARG, "positions are misaligned");
    // stride 0: the same positions on every axis
    if (positions && p->n_axes > 1 && pos_stride != 0 && pos_stride < tokens)
      return fail(VQ_ERR_ARG, "pos_stride=%lld < %lld tokens", (long long)pos_stride,
                  (long long)tokens);
  }
  to->turns = static_cast<const unsigned long long *>(p->turns);
  to->axis = p->n_axes > 1 ? static_cast<const uint8_t *>(p->axis) : nullptr;
  to->pos = positions;
  to->pos_stride = pos_stride;
  to->half = p->rot_dim / 2;
  to->interleaved = p->interleaved ? 1 : 0;
  to->pos64 = pos_64 ? 1 : 0;
  to->axes = p->n_axes;
  to->scale = p->scale;
  return VQ_OK;
}

int check_pool(const vq_kivi_paged *p) {
  if (!p) return fail(VQ_ERR_ARG, "cache is NULL");
  if (p->H_q < 1 || p->H_kv < 1 || p->n_pages < 1)
    return fail(VQ_ERR_ARG, "sizes must be positive (H_q=%d H_kv=%d n_pages=%d)", p->H_q,
                p->H_kv, p->n_pages);
  if (p->H_q % p->H_kv)
    return fail(VQ_ERR_UNSUPPORTED, "H_q=%d is not a multiple of H_kv=%d", p->H_q, p->H_kv);
  if (p->H_q / p->H_kv > kMaxGroupHeads)
    return fail(VQ_ERR_UNSUPPORTED, "H_q/H_kv=%d > %d", p->H_q / p->H_kv, kMaxGroupHeads);
  if (p->H_q > 1024) return fail(VQ_ERR_UNSUPPORTED, "H_q=%d > 1024", p->H_q);
  if (p->D != 64 && p->D != 128)
    return fail(VQ_ERR_UNSUPPORTED, "D=%d (supported: 64, 128)", p->D);
  if ((p->group != 32 && p->group != 64 && p->group != 128) || p->group > p->D)
    return fail(VQ_ERR_UNSUPPORTED, "group=%d (supported: 32, 64, 128, at most D=%d)", p->group,
                p->D);
  if (p->page < 16 || p->page > 1024 || (p->page & (p->page - 1)))
    return fail(VQ_ERR_UNSUPPORTED, "page=%d: a power of two in [16, 1024]", p->page);
  return VQ_OK;
}

int check_batch(const vq_kivi_paged *p, const vq_kivi_paged_batch *s, PagedArgs *to) {
  if (!s) return fail(VQ_ERR_ARG, "batch is NULL");
  if (s->B < 0 || s->tokens < 0 || s->max_pages < 0)
    return fail(VQ_ERR_ARG, "negative size (B=%d tokens=%lld max_pages=%d)", s->B,
                (long long)s->tokens, s->max_pages);
  if (s->B > kMaxSeqs) return fail(VQ_ERR_UNSUPPORTED, "B=%d > %d", s->B, kMaxSeqs);
  if (s->tokens > (1 << 24))
    return fail(VQ_ERR_UNSUPPORTED, "%lld new tokens > 2^24", (long long)s->tokens);
  if (!s->cu_new && s->tokens != s->B)
    return fail(VQ_ERR_ARG, "without cu_new every sequence has one new token, got %lld for "
                "B=%d", (long long)s->tokens, s->B);
  int lg = 4;
  while ((1 << lg) < p->page) ++lg;
  // the work line of the attention counts blocks in 31 bits
  if ((int64_t)s->B * s->max_pages * (p->page / 16) * p->H_kv > 0x7fffffffLL)
    return fail(VQ_ERR_UNSUPPORTED, "B * max_pages * page * H_kv too large");
  if (s->B > 0) {
    if (!s->lens || !p->pool || !p->status || (s->max_pages > 0 && !s->table))
      return fail(VQ_ERR_ARG, "NULL pointer");
    if (s->table_stride < s->max_pages)
      return fail(VQ_ERR_ARG, "table_stride=%lld < max_pages=%d", (long long)s->table_stride,
                  s->max_pages);
    if (!aligned(p->pool, 16)) return fail(VQ_ERR_ARG, "the pool must be 16-byte aligned");
    if (!aligned(s->table, 4) || !aligned(s->lens, 4) || !aligned(s->cu_new, 4) ||
        !aligned(p->status, 4))
      return fail(VQ_ERR_ARG, "int32 arrays must be 4-byte aligned");
  }
  to->pool = static_cast<uint8_t *>(p->pool);
  to->status = static_cast<unsigned *>(p->status);
  to->table = s->table;
  to->lens = s->lens;
  to->cu = s->cu_new;
  to->table_stride = s->table_stride;
  to->tokens = s->tokens;
  to->n_pages = p->n_pages;
  to->page_log2 = lg;
  to->max_pages = s->max_pages;
  to->B = s->B;
  to->H_q = p->H_q;
  to->H_kv = p->H_kv;
  to->g = p->group;
  return VQ_OK;
}

// Only the bits that were read: kernels of other streams may set others
// meanwhile.  (A bit that one sets again before this is among those reported.)
__global__ void k_clear_bits(unsigned *status, unsigned bits) { atomicAnd(status, ~bits); }

// whether contiguous rows `out` lie within the range that rows `x` span: tiles
// of queries are read while others' outputs are written
bool overlap(const HeadRows &h, int64_t tokens, int D, int elem) {
  const int64_t t = (tokens - 1) * h.x_token, e = (int64_t)(h.heads - 1) * h.x_head;
  const int64_t lo = (t < 0 ? t : 0) + (e < 0 ? e : 0);
  const int64_t hi = (t > 0 ? t : 0) + (e > 0 ? e : 0) + D;
  const intptr_t x = reinterpret_cast<intptr_t>(h.x), o = reinterpret_cast<intptr_t>(h.out);
  return o < x + hi * elem && x + lo * elem < o + tokens * h.heads * D * elem;
}

// The split-KV kernel serves up to 16 rows of a kv head, which is all that its
// products take; there it is the faster one at both head sizes.  Replayed
// graphs, 8 kv heads, cold caches, split-KV against tensor-memory kernel, us:
//   D = 128     1 x 1024     1 x 32768    16 x 8192     64 x 2048
//   8 rows     15.5 / 23.7   33.9 / 49.3   56.5 / 118   62.6 / 148
//   16 rows    19.6 / 23.7   35.9 / 51.4   65.7 / 117   75.9 / 150
//   20, 32        23.7, 25      53, 56      120, 120     151, 153
//   D = 64
//   8 rows     15.5 / 19.6   25.8 / 44.1   40.1 / 108   44.2 / 128
//   16 rows    17.5 / 21.6   29.8 / 44.2   46.2 / 108   56.4 / 128
//   20, 32        21.6, 22      46, 46      107, 109     128, 129
bool few_rows(const vq_kivi_paged *p, int max_new) {
  return (int64_t)max_new * (p->H_q / p->H_kv) <= 16;
}

}  // namespace

extern "C" {

int vq_kivi_norm_rope(int dtype, int64_t tokens, int D, const vq_kivi_rows *q,
                      const vq_kivi_rows *k, const vq_kivi_rope *rope, const void *positions,
                      int positions_64, int64_t positions_stride, float eps, void *stream) {
  int elem, sms;
  int rc = check_dtype(dtype, true, &elem);
  if (rc) return rc;
  if (tokens < 0) return fail(VQ_ERR_ARG, "tokens=%lld < 0", (long long)tokens);
  if (tokens > (1 << 24))
    return fail(VQ_ERR_UNSUPPORTED, "%lld tokens > 2^24", (long long)tokens);
  if (D < 16 || D > kMaxD || D % 16)
    return fail(VQ_ERR_UNSUPPORTED, "D=%d: a multiple of 16 in [16, %d]", D, kMaxD);
  if (!q) return fail(VQ_ERR_ARG, "q is NULL");
  if (!std::isfinite(eps) || eps < 0.f) return fail(VQ_ERR_ARG, "eps must be finite and >= 0");
  HeadRows hq, hk;
  if ((rc = check_rows(q, "q", elem, tokens, true, &hq))) return rc;
  if (k && (rc = check_rows(k, "k", elem, tokens, true, &hk))) return rc;
  RopeArgs r;
  if ((rc = check_rope(rope, D, tokens, positions, positions_64, positions_stride, false, &r)))
    return rc;
  if (tokens == 0) return VQ_OK;
  if ((rc = sm_count(&sms))) return rc;
  cudaError_t e = launch_norm_rope(dtype, hq, hk, r, D, tokens, eps, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "norm_rope launch");
}

size_t vq_kivi_paged_pool_bytes(const vq_kivi_paged *p) {
  if (check_pool(p)) return 0;
  return (size_t)p->n_pages * p->H_kv * (p->page / 16) * paged_block_bytes(p->D, p->group);
}

size_t vq_kivi_paged_workspace_bytes(const vq_kivi_paged *p, int32_t B, int32_t max_new) {
  int sms;
  if (check_pool(p) || B < 0 || max_new < 1 || sm_count(&sms)) return 0;
  const int GQ = p->H_q / p->H_kv;
  const size_t n = few_rows(p, max_new) ? paged_decode_ws(B, p->H_kv, p->D, max_new * GQ, sms)
                                        : paged_chunk_ws(B, p->H_kv, p->D, sms);
  return n < 256 ? 256 : n;
}

int vq_kivi_paged_append(const vq_kivi_paged *p, const vq_kivi_paged_batch *batch, int dtype,
                         const vq_kivi_rows *q, const vq_kivi_rows *k, const vq_kivi_rows *v,
                         const vq_kivi_rope *rope, const void *positions, int positions_64,
                         int64_t positions_stride, float eps, void *stream) {
  int elem, sms;
  int rc = check_pool(p);
  if (rc) return rc;
  if ((rc = check_dtype(dtype, false, &elem))) return rc;
  PagedArgs a;
  if ((rc = check_batch(p, batch, &a))) return rc;
  if (!k || !v) return fail(VQ_ERR_ARG, "k or v is NULL");
  if (!std::isfinite(eps) || eps < 0.f) return fail(VQ_ERR_ARG, "eps must be finite and >= 0");
  HeadRows hq, hk, hv;
  if (q && (rc = check_rows(q, "q", elem, a.tokens, true, &hq))) return rc;
  if ((rc = check_rows(k, "k", elem, a.tokens, false, &hk))) return rc;
  if ((rc = check_rows(v, "v", elem, a.tokens, false, &hv))) return rc;
  if ((q && hq.heads != p->H_q) || hk.heads != p->H_kv || hv.heads != p->H_kv)
    return fail(VQ_ERR_ARG, "heads: q %d, k %d, v %d for H_q=%d, H_kv=%d", hq.heads, hk.heads,
                hv.heads, p->H_q, p->H_kv);
  if (hv.weight) return fail(VQ_ERR_ARG, "values are not normed");
  RopeArgs r;
  if ((rc = check_rope(rope, p->D, a.tokens, positions, positions_64, positions_stride, true,
                       &r)))
    return rc;
  if (a.tokens == 0 || a.B == 0) return VQ_OK;
  if ((rc = sm_count(&sms))) return rc;
  cudaError_t e = launch_paged_append(dtype, a, hq, hk, hv, r, positions == nullptr, p->D, eps,
                                      sms, (cudaStream_t)stream);
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "paged append launch");
}

int vq_kivi_paged_dequantize(const vq_kivi_paged *p, const vq_kivi_paged_batch *batch,
                             void *K_hat, void *V_hat, void *stream) {
  int sms;
  int rc = check_pool(p);
  if (rc) return rc;
  PagedArgs a;
  if ((rc = check_batch(p, batch, &a))) return rc;
  if (a.tokens == 0 || a.B == 0) return VQ_OK;
  if (!K_hat || !V_hat) return fail(VQ_ERR_ARG, "K_hat or V_hat is NULL");
  if (!aligned(K_hat, 16) || !aligned(V_hat, 16))
    return fail(VQ_ERR_ARG, "K_hat and V_hat must be 16-byte aligned");
  if ((rc = sm_count(&sms))) return rc;
  cudaError_t e = launch_paged_dequantize(a, static_cast<__half *>(K_hat),
                                          static_cast<__half *>(V_hat), p->D, sms,
                                          (cudaStream_t)stream);
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "paged dequantize launch");
}

int vq_kivi_paged_attend(const vq_kivi_paged *p, const vq_kivi_paged_batch *batch, int dtype,
                         const vq_kivi_rows *q, int32_t max_new, float softmax_scale,
                         void *workspace, size_t workspace_bytes, void *stream) {
  int elem, sms;
  int rc = check_pool(p);
  if (rc) return rc;
  if ((rc = check_dtype(dtype, false, &elem))) return rc;
  PagedArgs a;
  if ((rc = check_batch(p, batch, &a))) return rc;
  if (!q) return fail(VQ_ERR_ARG, "q is NULL");
  HeadRows h;
  if ((rc = check_rows(q, "q", elem, a.tokens, true, &h))) return rc;
  if (h.heads != p->H_q) return fail(VQ_ERR_ARG, "q has %d heads, H_q=%d", h.heads, p->H_q);
  if (h.weight) return fail(VQ_ERR_ARG, "attend does not norm its queries");
  if (h.out_head != p->D || h.out_token != (int64_t)p->D * p->H_q)
    return fail(VQ_ERR_ARG, "the output must be contiguous [tokens][H_q][D]");
  if (max_new < 1) return fail(VQ_ERR_ARG, "max_new=%d < 1", max_new);
  if (!batch->cu_new && max_new != 1)
    return fail(VQ_ERR_ARG, "without cu_new max_new is 1, got %d", max_new);
  if (!std::isfinite(softmax_scale)) return fail(VQ_ERR_ARG, "softmax_scale is not finite");
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)p->D);
  const float scale2 = scale * 1.4426950408889634f;      // base 2
  if (!std::isfinite(scale2)) return fail(VQ_ERR_ARG, "softmax_scale=%g is too large", scale);
  if (a.tokens == 0 || a.B == 0) return VQ_OK;
  if (overlap(h, a.tokens, p->D, elem))
    return fail(VQ_ERR_ARG, "the output overlaps the queries");
  if ((rc = sm_count(&sms))) return rc;
  const int GQ = p->H_q / p->H_kv;
  const bool few = few_rows(p, max_new);
  const size_t need = few ? paged_decode_ws(a.B, p->H_kv, p->D, max_new * GQ, sms)
                          : paged_chunk_ws(a.B, p->H_kv, p->D, sms);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
    return fail(VQ_ERR_ARG, "the workspace must be 16-byte aligned and hold %zu bytes", need);
  PagedAttend t;
  t.q = h.x;
  t.out = h.out;
  t.q_token = h.x_token;
  t.q_head = h.x_head;
  t.scale = scale2;
  t.max_new = max_new;
  t.ws = static_cast<float *>(workspace);
  cudaError_t e = few ? launch_paged_decode(dtype, a, t, p->D, sms, (cudaStream_t)stream)
                      : launch_paged_chunk(dtype, a, t, p->D, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "paged attend launch");
}

int vq_kivi_paged_status(const vq_kivi_paged *p, void *stream) {
  int rc = check_pool(p);
  if (rc) return rc;
  if (!p->status) return fail(VQ_ERR_ARG, "NULL pointer");
  unsigned flags = 0;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaMemcpyAsync(&flags, p->status, sizeof flags, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && flags) {
    k_clear_bits<<<1, 1, 0, st>>>(static_cast<unsigned *>(p->status), flags);
    count_launch();
    e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  if (e != cudaSuccess) return cuda_fail(e, "reading the status word");
  if (!flags) return VQ_OK;
  return fail(flags & kGaveUp ? VQ_ERR_CUDA : VQ_ERR_ARG, "%s%s%s",
              flags & kGaveUp ? "an attention kernel gave up waiting for its copies; its outputs "
                                "are not valid. " : "",
              flags & kBadPage ? "a block table names a page outside the pool: its tokens were "
                                 "not stored, and rows that see it are not valid. " : "",
              flags & kBadLength ? "a sequence's length or its new tokens lie outside their "
                                   "ranges; the sequence was left out." : "");
}

}  // extern "C"
