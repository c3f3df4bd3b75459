// attend_api.cu -- the C ABI entry points of the softmax layers (treewy_attend,
// treewy_append, treewy_add_norm): argument validation and dispatch.
#include <cmath>

#include "treewy_internal.h"

namespace {

using treewy::cuda_fail;
using treewy::fail;

constexpr int64_t kMax31 = (int64_t(1) << 31) - 1;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known(int32_t dtype) { return dtype == TREEWY_DTYPE_BF16 || dtype == TREEWY_DTYPE_F32; }
uintptr_t bytes_of(int32_t dtype) { return dtype == TREEWY_DTYPE_BF16 ? 2 : 4; }
// A stride as the kernels use it: 0 stands for dense rows.
int64_t stride_or(int64_t stride, int64_t dense) { return stride == 0 ? dense : stride; }

treewy_status validate_cache_sizes(const treewy_cache& c) {
  if (c.Hkv < 1) return fail(TREEWY_ERR_INVALID_ARG, "Hkv = %d must be >= 1", c.Hkv);
  if (c.d < 1) return fail(TREEWY_ERR_INVALID_ARG, "d = %d must be >= 1", c.d);
  if (c.d > 256) return fail(TREEWY_ERR_UNSUPPORTED, "d = %d: head sizes above 256 are not supported", c.d);
  if (c.page_len != 16 && c.page_len != 32 && c.page_len != 64 && c.page_len != 128)
    return fail(TREEWY_ERR_UNSUPPORTED, "page_len = %d is not 16, 32, 64 or 128", c.page_len);
  if (c.max_pages < 0) return fail(TREEWY_ERR_INVALID_ARG, "max_pages = %d is negative", c.max_pages);
  if (c.num_pages < 0) return fail(TREEWY_ERR_INVALID_ARG, "num_pages = %lld is negative", (long long)c.num_pages);
  if (c.Hkv > (1 << 20) || c.num_pages > kMax31 / c.Hkv)
    return fail(TREEWY_ERR_UNSUPPORTED, "num_pages * Hkv exceeds 2^31 - 1, or Hkv 2^20");
  return TREEWY_OK;
}

treewy_status validate_cache_pointers(const treewy_cache& c) {
  if (!c.length) return fail(TREEWY_ERR_INVALID_ARG, "cache.length must be non-NULL");
  if (c.max_pages > 0 && !c.page_table) return fail(TREEWY_ERR_INVALID_ARG, "cache.page_table must be non-NULL");
  if (c.num_pages > 0 && (!c.k || !c.v || !c.k_scale || !c.v_scale))
    return fail(TREEWY_ERR_INVALID_ARG, "the cache's codes and scales must be non-NULL");
  if (!aligned(c.k, 16) || !aligned(c.v, 16)) return fail(TREEWY_ERR_INVALID_ARG, "the cache's codes must be 16-byte aligned");
  if (!aligned(c.k_scale, 4) || !aligned(c.v_scale, 4) || !aligned(c.page_table, 4) || !aligned(c.length, 4))
    return fail(TREEWY_ERR_INVALID_ARG, "scales, page_table and length must be aligned to their elements");
  return TREEWY_OK;
}

treewy_status validate_stride(int64_t stride, int64_t row) {
  if (stride != 0 && stride < row) return fail(TREEWY_ERR_INVALID_ARG, "a token stride is shorter than its row");
  if (stride > (int64_t(1) << 31) || row > (int64_t(1) << 31))
    return fail(TREEWY_ERR_UNSUPPORTED, "token rows are too long");
  return TREEWY_OK;
}

treewy_status validate_attn_sizes(const treewy_attn* a) {
  if (a == nullptr) return fail(TREEWY_ERR_INVALID_ARG, "attn is NULL");
  treewy_status st = validate_cache_sizes(a->cache);
  if (st != TREEWY_OK) return st;
  if (a->R < 0) return fail(TREEWY_ERR_INVALID_ARG, "R = %d is negative", a->R);
  if (a->Hq < 1 || a->Hq % a->cache.Hkv != 0)
    return fail(TREEWY_ERR_INVALID_ARG, "Hq = %d must be a positive multiple of Hkv = %d", a->Hq, a->cache.Hkv);
  if (a->Hq > (1 << 20)) return fail(TREEWY_ERR_UNSUPPORTED, "more than 2^20 heads");
  if (a->max_nodes < 1 || a->max_nodes > TREEWY_MAX_NODES)
    return fail(a->max_nodes < 1 ? TREEWY_ERR_INVALID_ARG : TREEWY_ERR_UNSUPPORTED, "max_nodes = %d outside [1, %d]",
                a->max_nodes, TREEWY_MAX_NODES);
  if (a->T < 0 || a->T > kMax31) return fail(TREEWY_ERR_INVALID_ARG, "T = %lld outside [0, 2^31)", (long long)a->T);
  if (a->max_context < 0) return fail(TREEWY_ERR_INVALID_ARG, "max_context = %d is negative", a->max_context);
  if (!known(a->qkv_dtype) || !known(a->o_dtype))
    return fail(TREEWY_ERR_INVALID_ARG, "qkv_dtype = %d, o_dtype = %d: not TREEWY_DTYPE_BF16/F32", a->qkv_dtype, a->o_dtype);
  if (a->flags & ~TREEWY_FLAG_FORCE_GENERIC)
    return fail(TREEWY_ERR_INVALID_ARG, "flags = 0x%x has unknown bits", a->flags);
  return TREEWY_OK;
}

treewy_status validate_attn(const treewy_attn* a) {
  treewy_status st = validate_attn_sizes(a);
  if (st != TREEWY_OK) return st;
  const treewy_cache& c = a->cache;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return fail(TREEWY_ERR_INVALID_ARG, "scale must be positive and finite");
  for (auto [stride, heads] : {std::pair<int64_t, int64_t>{a->q_stride, a->Hq}, {a->k_stride, c.Hkv}, {a->v_stride, c.Hkv}})
    if ((st = validate_stride(stride, heads * c.d)) != TREEWY_OK) return st;
  if (a->R == 0) return TREEWY_OK;
  if (!a->node_offset || !a->status) return fail(TREEWY_ERR_INVALID_ARG, "node_offset and status must be non-NULL");
  if (a->T > 0 && (!a->q || !a->k || !a->v || !a->o)) return fail(TREEWY_ERR_INVALID_ARG, "q, k, v and o must be non-NULL");
  const uintptr_t e = bytes_of(a->qkv_dtype);
  if (!aligned(a->q, e) || !aligned(a->k, e) || !aligned(a->v, e) || !aligned(a->o, bytes_of(a->o_dtype)) ||
      !aligned(a->node_offset, 4) || !aligned(a->parent, 4) || !aligned(a->status, 4))
    return fail(TREEWY_ERR_INVALID_ARG, "rows, node_offset, parent and status must be aligned to their elements");
  if ((st = validate_cache_pointers(c)) != TREEWY_OK) return st;
  const uint64_t need = treewy::attend_workspace(*a);
  if (a->workspace_bytes < need || (need > 0 && (!a->workspace || !aligned(a->workspace, 16))))
    return fail(TREEWY_ERR_INVALID_ARG, "a workspace of %llu bytes, 16-byte aligned, is needed", (unsigned long long)need);
  return TREEWY_OK;
}

treewy_status validate_append(const treewy_append_args* a) {
  if (a == nullptr) return fail(TREEWY_ERR_INVALID_ARG, "args is NULL");
  const treewy_cache& c = a->cache;
  treewy_status st = validate_cache_sizes(c);
  if (st != TREEWY_OK) return st;
  if (a->R < 0) return fail(TREEWY_ERR_INVALID_ARG, "R = %d is negative", a->R);
  if (a->max_new < 0) return fail(TREEWY_ERR_INVALID_ARG, "max_new = %d is negative", a->max_new);
  if (a->accepted != nullptr && a->max_new > TREEWY_MAX_NODES)
    return fail(TREEWY_ERR_UNSUPPORTED, "max_new = %d: accepted nodes are of trees of at most %d", a->max_new, TREEWY_MAX_NODES);
  if (!known(a->kv_dtype)) return fail(TREEWY_ERR_INVALID_ARG, "kv_dtype = %d is not TREEWY_DTYPE_BF16/F32", a->kv_dtype);
  if (a->T < 0 || a->T > kMax31) return fail(TREEWY_ERR_INVALID_ARG, "T = %lld outside [0, 2^31)", (long long)a->T);
  for (int64_t stride : {a->k_stride, a->v_stride})
    if ((st = validate_stride(stride, int64_t(c.Hkv) * c.d)) != TREEWY_OK) return st;
  if (a->R == 0) return TREEWY_OK;
  if (!a->node_offset || !a->status) return fail(TREEWY_ERR_INVALID_ARG, "node_offset and status must be non-NULL");
  if (a->T > 0 && a->max_new > 0 && (!a->k || !a->v)) return fail(TREEWY_ERR_INVALID_ARG, "k and v must be non-NULL");
  const uintptr_t e = bytes_of(a->kv_dtype);
  if (!aligned(a->k, e) || !aligned(a->v, e) || !aligned(a->node_offset, 4) || !aligned(a->parent, 4) ||
      !aligned(a->accepted, 4) || !aligned(a->new_length, 4) || !aligned(a->status, 4))
    return fail(TREEWY_ERR_INVALID_ARG, "rows, node_offset, parent, accepted, new_length and status must be aligned to their elements");
  if (a->new_length != nullptr && a->new_length == c.length)
    return fail(TREEWY_ERR_INVALID_ARG, "new_length must not be cache.length");
  return validate_cache_pointers(c);
}

treewy_status validate_norm(const treewy_norm* a) {
  if (a == nullptr) return fail(TREEWY_ERR_INVALID_ARG, "norm is NULL");
  if (a->T < 0 || a->T > kMax31) return fail(TREEWY_ERR_INVALID_ARG, "T = %lld outside [0, 2^31)", (long long)a->T);
  if (a->n < 1) return fail(TREEWY_ERR_INVALID_ARG, "n = %d must be >= 1", a->n);
  if (a->n > 32768) return fail(TREEWY_ERR_UNSUPPORTED, "n = %d: rows above 32768 are not supported", a->n);
  if (!known(a->x_dtype) || (a->residual != nullptr && !known(a->residual_dtype)))
    return fail(TREEWY_ERR_INVALID_ARG, "x_dtype = %d, residual_dtype = %d: not TREEWY_DTYPE_BF16/F32", a->x_dtype, a->residual_dtype);
  if (a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128)
    return fail(TREEWY_ERR_UNSUPPORTED, "group = %d is not 0, 32, 64 or 128", a->group);
  if (!(a->eps >= 0.f)) return fail(TREEWY_ERR_INVALID_ARG, "eps must be >= 0");
  treewy_status st = validate_stride(a->x_stride, a->n);
  if (st == TREEWY_OK) st = validate_stride(a->residual_stride, a->n);
  if (st != TREEWY_OK || a->T == 0) return st;
  if (!a->x) return fail(TREEWY_ERR_INVALID_ARG, "x must be non-NULL");
  if (!a->y && !a->y8 && !a->residual) return fail(TREEWY_ERR_INVALID_ARG, "an output (y, y8 or residual_out) is needed");
  if ((a->residual != nullptr) != (a->residual_out != nullptr))
    return fail(TREEWY_ERR_INVALID_ARG, "residual and residual_out go together");
  if (a->y8 != nullptr && !a->y8_scale) return fail(TREEWY_ERR_INVALID_ARG, "y8_scale is needed with y8");
  const uintptr_t e = bytes_of(a->x_dtype), er = bytes_of(a->residual_dtype);
  if (!aligned(a->x, e) || !aligned(a->y, e) || !aligned(a->weight, 4) || !aligned(a->y8_scale, 4) ||
      (a->residual != nullptr && (!aligned(a->residual, er) || !aligned(a->residual_out, er))))
    return fail(TREEWY_ERR_INVALID_ARG, "rows, weight and scales must be aligned to their elements");
  if (a->residual != nullptr && a->residual_out == a->residual && stride_or(a->residual_stride, a->n) != a->n)
    return fail(TREEWY_ERR_INVALID_ARG, "residual_out = residual needs dense rows");
  if (a->y == a->x && stride_or(a->x_stride, a->n) != a->n)
    return fail(TREEWY_ERR_INVALID_ARG, "y = x needs dense rows");
  return TREEWY_OK;
}

}  // namespace

extern "C" {

treewy_status treewy_attend_workspace(const treewy_attn* attn, uint64_t* bytes) {
  treewy::clear_error();
  const treewy_status st = validate_attn_sizes(attn);
  if (st != TREEWY_OK) return st;
  if (bytes == nullptr) return fail(TREEWY_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = treewy::attend_workspace(*attn);
  return TREEWY_OK;
}

treewy_status treewy_attend(const treewy_attn* attn, cudaStream_t stream) {
  treewy::clear_error();
  const treewy_status st = validate_attn(attn);
  if (st != TREEWY_OK || attn->R == 0) return st;
  treewy_attn a = *attn;
  a.q_stride = stride_or(a.q_stride, int64_t(a.Hq) * a.cache.d);
  a.k_stride = stride_or(a.k_stride, int64_t(a.cache.Hkv) * a.cache.d);
  a.v_stride = stride_or(a.v_stride, int64_t(a.cache.Hkv) * a.cache.d);
  const cudaError_t err = treewy::attend_on_tensor_cores(a) ? treewy::launch_attend_tc(a, stream) : treewy::launch_attend_scan(a, stream);
  if (err == cudaErrorNotSupported)
    return fail(TREEWY_ERR_UNSUPPORTED, "%d requests of %d nodes and %d heads are too many for one call", a.R, a.max_nodes, a.Hq);
  return err == cudaSuccess ? TREEWY_OK : cuda_fail(err, "treewy_attend launch");
}

treewy_status treewy_append(const treewy_append_args* args, cudaStream_t stream) {
  treewy::clear_error();
  const treewy_status st = validate_append(args);
  if (st != TREEWY_OK || args->R == 0) return st;
  treewy_append_args a = *args;
  a.k_stride = stride_or(a.k_stride, int64_t(a.cache.Hkv) * a.cache.d);
  a.v_stride = stride_or(a.v_stride, int64_t(a.cache.Hkv) * a.cache.d);
  const cudaError_t err = treewy::launch_append(a, stream);
  if (err == cudaErrorNotSupported)
    return fail(TREEWY_ERR_UNSUPPORTED, "%d requests of %d rows and %d heads are too many for one call", a.R, a.max_new, a.cache.Hkv);
  return err == cudaSuccess ? TREEWY_OK : cuda_fail(err, "treewy_append launch");
}

treewy_status treewy_add_norm(const treewy_norm* norm, cudaStream_t stream) {
  treewy::clear_error();
  const treewy_status st = validate_norm(norm);
  if (st != TREEWY_OK || norm->T == 0) return st;
  treewy_norm a = *norm;
  a.x_stride = stride_or(a.x_stride, a.n);
  a.residual_stride = stride_or(a.residual_stride, a.n);
  const cudaError_t err = treewy::launch_add_norm(a, stream);
  return err == cudaSuccess ? TREEWY_OK : cuda_fail(err, "treewy_add_norm launch");
}

}  // extern "C"
