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

// whether two ranges of bytes meet
bool meet(const void *a, int64_t na, const void *b, int64_t nb) {
  const intptr_t x = reinterpret_cast<intptr_t>(a), y = reinterpret_cast<intptr_t>(b);
  return x < y + nb && y < x + na;
}

// whether what is written at `o` meets the batch's table or offsets
bool over_batch(const PagedArgs &a, const void *o, int64_t bytes) {
  if (a.max_pages > 0 &&
      meet(o, bytes, a.table, 4 * ((a.B - 1) * a.table_stride + a.max_pages)))
    return true;
  return a.cu && meet(o, bytes, a.cu, 4 * ((int64_t)a.B + 1));
}

// workspace of an eviction: none where no sequence can pass the budget
size_t evict_bytes(const vq_kivi_paged *p, int B, int max_pages, int budget, int recent) {
  return (int64_t)max_pages * p->page <= budget ? 0
                                                : paged_evict_ws(B, p->H_kv, budget, recent);
}

// whether the work line of the attention counts more blocks than 31 bits hold
bool too_many(const vq_kivi_paged *p, int B, int max_pages) {
  return (int64_t)B * max_pages * (p->page / 16) * p->H_kv > 0x7fffffffLL;
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
  if (too_many(p, s->B, s->max_pages))
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
  const int64_t room = (int64_t)s->max_pages << lg;
  to->max_len = (int)(room < kMaxLen ? room : kMaxLen);
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
//   8 rows     16.5 / 23.7   34.0 / 51.4   57.5 / 115   62.6 / 169
//   16 rows    19.6 / 25.7   36.0 / 54.4   66.7 / 117   76.9 / 171
//   20, 32      25.7, 25.8    54.4, 57.5    117, 118     173, 174
//   D = 64
//   8 rows     16.5 / 20.6   27.8 / 44.2   42.1 / 104   46.2 / 127
//   16 rows    18.6 / 21.6   29.9 / 44.2   48.3 / 104   58.5 / 127
//   20, 32      20.6, 21.7    44.2, 44.3    104, 104     128, 128
bool few_rows(const vq_kivi_paged *p, int max_new) {
  return (int64_t)max_new * (p->H_q / p->H_kv) <= 16;
}

int check_weights(const vq_kivi_paged *p, const PagedArgs &a, const vq_kivi_weights *w,
                  const char *name, PagedWeights *to) {
  if (!w) return fail(VQ_ERR_ARG, "%s is NULL", name);
  const int64_t room = (int64_t)a.max_pages << a.page_log2;
  if (w->capacity < 0)
    return fail(VQ_ERR_ARG, "%s: capacity=%lld < 0", name, (long long)w->capacity);
  // (an eviction clears all places, also of a table without pages)
  if (a.B > 0 && (room > 0 || w->capacity > 0)) {
    if (!w->at || !aligned(w->at, 4)) return fail(VQ_ERR_ARG, "%s is NULL or misaligned", name);
    if (w->capacity < room)
      return fail(VQ_ERR_ARG, "%s has room for %lld tokens, the table for %lld", name,
                  (long long)w->capacity, (long long)room);
    // no two rows may share a place
    const int64_t s = w->seq_stride, h = w->head_stride, H = p->H_kv, B = a.B, n = w->capacity;
    const bool one_b = B == 1, one_h = H == 1;
    if ((!one_b && s < n) || (!one_h && h < n) ||
        (!one_b && !one_h && s < (H - 1) * h + n && h < (B - 1) * s + n))
      return fail(VQ_ERR_ARG, "%s: rows overlap", name);
  }
  to->at = w->at;
  to->seq = a.B == 1 ? 0 : w->seq_stride;
  to->head = p->H_kv == 1 ? 0 : w->head_stride;
  to->capacity = w->capacity;
  return VQ_OK;
}

// bytes that an array of weights spans
int64_t span(const PagedWeights &w, const PagedArgs &a) {
  return 4 * ((a.B - 1) * w.seq + (a.H_kv - 1) * w.head + w.capacity);
}

// what the three attentions share; tree: masks, weights: where weights are added
int attend(const vq_kivi_paged *p, const vq_kivi_paged_batch *batch, int dtype,
           const vq_kivi_rows *q, const void *tree, const vq_kivi_weights *weights,
           int32_t max_new, float softmax_scale, void *workspace, size_t workspace_bytes,
           void *stream, bool with_tree = false) {
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
  if (with_tree) {
    if ((!tree && a.tokens > 0) || !aligned(tree, 8))
      return fail(VQ_ERR_ARG, "tree is NULL or misaligned");
    if (max_new > kMaxTree)
      return fail(VQ_ERR_UNSUPPORTED, "a tree has at most %d nodes, max_new=%d", kMaxTree,
                  max_new);
  }
  PagedWeights w;
  if (weights) {
    if ((rc = check_weights(p, a, weights, "weights", &w))) return rc;
    if (!few_rows(p, max_new))
      return fail(VQ_ERR_UNSUPPORTED, "weights: max_new=%d * H_q/H_kv=%d > 16", max_new,
                  p->H_q / p->H_kv);
  }
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
  const size_t need =
      weights ? paged_weigh_ws(a.B, p->H_kv, p->D, max_new * GQ,
                               (int64_t)a.max_pages << a.page_log2, sms)
      : few   ? paged_decode_ws(a.B, p->H_kv, p->D, max_new * GQ, sms)
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
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (with_tree) {
    t.tree = static_cast<const unsigned long long *>(tree);
    e = few ? launch_paged_decode_tree(dtype, a, t, p->D, sms, st)
            : launch_paged_chunk_tree(dtype, a, t, p->D, sms, st);
  } else if (weights) {
    e = launch_paged_weigh(dtype, a, t, w, p->D, sms, st);
  } else {
    e = few ? launch_paged_decode(dtype, a, t, p->D, sms, st)
            : launch_paged_chunk(dtype, a, t, p->D, sms, st);
  }
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "paged attend launch");
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

size_t vq_kivi_paged_weights_workspace_bytes(const vq_kivi_paged *p, int32_t B, int32_t max_pages,
                                             int32_t max_new) {
  int sms;
  if (check_pool(p) || B < 0 || max_pages < 0 || max_new < 1 || sm_count(&sms)) return 0;
  if (!few_rows(p, max_new)) {
    fail(VQ_ERR_UNSUPPORTED, "weights: max_new=%d * H_q/H_kv=%d > 16", max_new, p->H_q / p->H_kv);
    return 0;
  }
  if (too_many(p, B, max_pages)) {
    fail(VQ_ERR_UNSUPPORTED, "B * max_pages * page * H_kv too large");
    return 0;
  }
  const size_t n = paged_weigh_ws(B, p->H_kv, p->D, max_new * (p->H_q / p->H_kv),
                                  (int64_t)max_pages * p->page, sms);
  return n < 256 ? 256 : n;
}

int vq_kivi_paged_attend(const vq_kivi_paged *p, const vq_kivi_paged_batch *batch, int dtype,
                         const vq_kivi_rows *q, int32_t max_new, float softmax_scale,
                         void *workspace, size_t workspace_bytes, void *stream) {
  return attend(p, batch, dtype, q, nullptr, nullptr, max_new, softmax_scale, workspace,
                workspace_bytes, stream);
}

int vq_kivi_paged_attend_tree(const vq_kivi_paged *p, const vq_kivi_paged_batch *batch, int dtype,
                              const vq_kivi_rows *q, const void *tree, int32_t max_new,
                              float softmax_scale, void *workspace, size_t workspace_bytes,
                              void *stream) {
  return attend(p, batch, dtype, q, tree, nullptr, max_new, softmax_scale, workspace,
                workspace_bytes, stream, true);
}

int vq_kivi_paged_attend_weights(const vq_kivi_paged *p, const vq_kivi_paged_batch *batch,
                                 int dtype, const vq_kivi_rows *q, const vq_kivi_weights *weights,
                                 int32_t max_new, float softmax_scale, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  if (!weights) return fail(VQ_ERR_ARG, "weights is NULL");
  return attend(p, batch, dtype, q, nullptr, weights, max_new, softmax_scale, workspace,
                workspace_bytes, stream);
}

int vq_kivi_paged_keep(const vq_kivi_paged *p, const vq_kivi_paged_batch *batch,
                       const int32_t *path, const int32_t *counts, int32_t *lens_out,
                       void *stream) {
  int rc = check_pool(p);
  if (rc) return rc;
  PagedArgs a;
  if ((rc = check_batch(p, batch, &a))) return rc;
  if (a.B == 0) return VQ_OK;
  if (!counts || !lens_out || (a.tokens > 0 && !path)) return fail(VQ_ERR_ARG, "NULL pointer");
  if (!aligned(path, 4) || !aligned(counts, 4) || !aligned(lens_out, 4))
    return fail(VQ_ERR_ARG, "int32 arrays must be 4-byte aligned");
  // (in place a sequence's length is read and written by one CTA)
  const int64_t bytes = 4 * (int64_t)a.B;
  if (lens_out != a.lens && meet(lens_out, bytes, a.lens, bytes))
    return fail(VQ_ERR_ARG, "lens_out overlaps lens (it may be the same array)");
  // (so are the counts)
  if ((lens_out != counts && meet(lens_out, bytes, counts, bytes)) ||
      (a.tokens > 0 && meet(lens_out, bytes, path, 4 * a.tokens)) ||
      over_batch(a, lens_out, bytes))
    return fail(VQ_ERR_ARG, "lens_out overlaps what other sequences' CTAs read");
  cudaError_t e = launch_paged_keep(a, path, counts, lens_out, p->D, (cudaStream_t)stream);
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "paged keep launch");
}

size_t vq_kivi_paged_evict_workspace_bytes(const vq_kivi_paged *p, int32_t B, int32_t max_pages,
                                           int32_t budget, int32_t recent) {
  if (check_pool(p) || B < 0 || max_pages < 0 || budget < 1 || recent < 0 || recent > budget)
    return 0;
  const size_t n = evict_bytes(p, B, max_pages, budget, recent);
  return n < 256 ? 256 : n;
}

int vq_kivi_paged_evict(const vq_kivi_paged *p, const vq_kivi_paged_batch *batch,
                        const vq_kivi_weights *weights, const vq_kivi_weights *weights_out,
                        int32_t budget, int32_t recent, int32_t first, int32_t *lens_out,
                        void *workspace, size_t workspace_bytes, void *stream) {
  int sms;
  int rc = check_pool(p);
  if (rc) return rc;
  PagedArgs a;
  if ((rc = check_batch(p, batch, &a))) return rc;
  if (batch->cu_new) return fail(VQ_ERR_ARG, "evict takes whole sequences: cu_new must be NULL");
  if (budget < 1 || recent < 0 || first < 0 || (int64_t)recent + first > budget)
    return fail(VQ_ERR_ARG, "budget=%d, recent=%d, first=%d: recent + first must be in [0, budget]",
                budget, recent, first);
  PagedEvict v;
  if ((rc = check_weights(p, a, weights, "weights", &v.in))) return rc;
  if ((rc = check_weights(p, a, weights_out, "weights_out", &v.out))) return rc;
  if (a.B == 0) return VQ_OK;
  if (v.in.at == v.out.at ? v.in.seq != v.out.seq || v.in.head != v.out.head ||
                                v.in.capacity != v.out.capacity
                          : meet(v.in.at, span(v.in, a), v.out.at, span(v.out, a)))
    return fail(VQ_ERR_ARG, "weights_out overlaps weights (it may be the same array)");
  if (!lens_out || !aligned(lens_out, 4))
    return fail(VQ_ERR_ARG, "lens_out is NULL or misaligned");
  // heads read the lengths while another's sequence is done
  const int64_t bytes = 4 * (int64_t)a.B;
  if (meet(lens_out, bytes, a.lens, bytes))
    return fail(VQ_ERR_ARG, "lens_out overlaps lens");
  // (weights in place, too, change while other heads' CTAs read the batch)
  const int64_t n = span(v.out, a);
  if (over_batch(a, lens_out, bytes) || meet(lens_out, bytes, v.in.at, span(v.in, a)) ||
      meet(lens_out, bytes, v.out.at, n))
    return fail(VQ_ERR_ARG, "lens_out overlaps another array of the call");
  if (over_batch(a, v.out.at, n) || meet(v.out.at, n, a.lens, bytes))
    return fail(VQ_ERR_ARG, "weights_out overlaps the batch's arrays");
  const size_t need = evict_bytes(p, a.B, a.max_pages, budget, recent);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
    return fail(VQ_ERR_ARG, "the workspace must be 16-byte aligned and hold %zu bytes", need);
  if ((rc = sm_count(&sms))) return rc;
  v.lens_out = lens_out;
  v.budget = budget;
  v.recent = recent;
  v.first = first;
  v.pairs = static_cast<int2 *>(workspace);
  cudaError_t e = launch_paged_evict(a, v, p->D, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "paged evict launch");
}

int vq_kivi_verify_drafts(const vq_kivi_drafts *d, int dtype, int32_t *path, int32_t *counts,
                          void *after, void *stream) {
  int elem, sms;
  int rc = check_dtype(dtype, true, &elem);
  if (rc) return rc;
  if (!d) return fail(VQ_ERR_ARG, "drafts is NULL");
  if (d->B < 0 || d->tokens < 0 || d->V < 1)
    return fail(VQ_ERR_ARG, "sizes: B=%d, tokens=%lld, V=%d", d->B, (long long)d->tokens, d->V);
  if (d->B > kMaxSeqs) return fail(VQ_ERR_UNSUPPORTED, "B=%d > %d", d->B, kMaxSeqs);
  if (d->V > (1 << 19)) return fail(VQ_ERR_UNSUPPORTED, "V=%d > 2^19", d->V);
  if (d->tokens > (1 << 24))
    return fail(VQ_ERR_UNSUPPORTED, "%lld new tokens > 2^24", (long long)d->tokens);
  if (d->B == 0) return VQ_OK;
  if (!d->cu_new || !counts || !after ||
      (d->tokens > 0 && (!d->target || !d->token || !d->uniforms || !path)))
    return fail(VQ_ERR_ARG, "NULL pointer");
  if (d->tokens > 1 && (d->target_row < d->V || (d->draft && d->draft_row < d->V)))
    return fail(VQ_ERR_ARG, "rows of probabilities overlap: strides %lld and %lld for V=%d",
                (long long)d->target_row, (long long)d->draft_row, d->V);
  const int wide = d->token_64 ? 8 : 4;
  if (!aligned(d->target, elem) || !aligned(d->draft, elem) || !aligned(d->token, wide) ||
      !aligned(after, wide) || !aligned(d->parent, 4) || !aligned(d->cu_new, 4) ||
      !aligned(d->uniforms, 4) || !aligned(path, 4) || !aligned(counts, 4))
    return fail(VQ_ERR_ARG, "misaligned pointer");
  // the CTAs of a sequence read its nodes and rows each for itself
  auto rows = [&](const void *p, int64_t row) {
    return p && d->tokens > 0 ? elem * ((d->tokens - 1) * row + d->V) : (int64_t)0;
  };
  const struct { const void *at; int64_t bytes; } outs[3] = {
      {path, 4 * d->tokens}, {counts, 4 * (int64_t)d->B}, {after, wide * (int64_t)d->B}},
      ins[6] = {{d->token, wide * d->tokens}, {d->parent, d->parent ? 4 * d->tokens : 0},
                {d->uniforms, 4 * d->tokens}, {d->cu_new, 4 * ((int64_t)d->B + 1)},
                {d->target, rows(d->target, d->target_row)},
                {d->draft, rows(d->draft, d->draft_row)}};
  for (const auto &o : outs) {
    for (const auto &i : ins)
      if (o.bytes > 0 && i.bytes > 0 && meet(o.at, o.bytes, i.at, i.bytes))
        return fail(VQ_ERR_ARG, "an output overlaps an input");
    for (const auto &x : outs)
      if (&x != &o && o.bytes > 0 && x.bytes > 0 && meet(o.at, o.bytes, x.at, x.bytes))
        return fail(VQ_ERR_ARG, "two outputs overlap");
  }
  if ((rc = sm_count(&sms))) return rc;
  Drafts x;
  x.target = d->target;
  x.draft = d->draft;
  x.target_row = d->target_row;
  x.draft_row = d->draft_row;
  x.tokens = d->token;
  x.parents = d->parent;
  x.cu = d->cu_new;
  x.uniforms = d->uniforms;
  x.path = path;
  x.counts = counts;
  x.after = after;
  x.rows = d->tokens;
  x.B = d->B;
  x.V = d->V;
  x.tokens64 = d->token_64 ? 1 : 0;
  cudaError_t e = launch_verify(dtype, x, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? VQ_OK : cuda_fail(e, "verify launch");
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
  return fail(flags & kGaveUp ? VQ_ERR_CUDA : VQ_ERR_ARG, "%s%s%s%s",
              flags & kGaveUp ? "an attention kernel gave up waiting for its copies; its outputs "
                                "are not valid. " : "",
              flags & kBadPage ? "a block table names a page outside the pool: its tokens were "
                                 "not stored, and rows that see it are not valid. " : "",
              flags & kBadLength ? "a sequence's length or its new tokens lie outside their "
                                   "ranges; the sequence was left out. " : "",
              flags & kBadPath ? "a path of kept tokens does not rise within its tree; the "
                                 "sequence was left as it was." : "");
}

}  // extern "C"
