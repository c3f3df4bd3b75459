// serving_api.cu -- the C ABI entry points around verification (treewy_extend,
// treewy_qk_norm, treewy_copy_slots): argument validation and dispatch.
#include "treewy_internal.h"

namespace {

using treewy::cuda_fail;
using treewy::fail;

constexpr int64_t kMax31 = (int64_t(1) << 31) - 1;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A stride as the kernels use it: 0 stands for dense rows.
int64_t stride_or(int64_t stride, int64_t dense) { return stride == 0 ? dense : stride; }

treewy_status validate_seqs(const treewy_seqs* s) {
  if (s == nullptr) return fail(TREEWY_ERR_INVALID_ARG, "seqs is NULL");
  if (s->R < 0) return fail(TREEWY_ERR_INVALID_ARG, "R = %d is negative", s->R);
  if (s->H < 1 || s->Hk < 1 || s->H % s->Hk != 0)
    return fail(TREEWY_ERR_INVALID_ARG, "H = %d must be a positive multiple of Hk = %d", s->H, s->Hk);
  if (s->dk < 1 || s->dv < 1)
    return fail(TREEWY_ERR_INVALID_ARG, "dk = %d, dv = %d must be >= 1", s->dk, s->dv);
  if (s->dk > 128 || s->dv > 128)
    return fail(TREEWY_ERR_UNSUPPORTED, "dk = %d, dv = %d: head sizes above 128 are not supported",
                s->dk, s->dv);
  if (s->max_len < 0) return fail(TREEWY_ERR_INVALID_ARG, "max_len = %d is negative", s->max_len);
  if (s->qkv_dtype != TREEWY_DTYPE_BF16 && s->qkv_dtype != TREEWY_DTYPE_F32)
    return fail(TREEWY_ERR_INVALID_ARG, "qkv_dtype = %d is not TREEWY_DTYPE_BF16/F32", s->qkv_dtype);
  if (s->o_dtype != TREEWY_DTYPE_BF16 && s->o_dtype != TREEWY_DTYPE_F32)
    return fail(TREEWY_ERR_INVALID_ARG, "o_dtype = %d is not TREEWY_DTYPE_BF16/F32", s->o_dtype);
  if (s->flags & ~(TREEWY_FLAG_FORCE_GENERIC | TREEWY_FLAG_STATE_BF16))
    return fail(TREEWY_ERR_INVALID_ARG, "flags = 0x%x has unknown bits", s->flags);
  if (s->T < 0 || s->T > kMax31)
    return fail(TREEWY_ERR_INVALID_ARG, "T = %lld outside [0, 2^31)", (long long)s->T);
  if (int64_t(s->R) * s->H > kMax31)
    return fail(TREEWY_ERR_UNSUPPORTED, "R * H = %lld (sequence, head) pairs exceed 2^31 - 1",
                (long long)(int64_t(s->R) * s->H));
  if (s->num_slots < 1)
    return fail(TREEWY_ERR_INVALID_ARG, "num_slots = %lld must be >= 1", (long long)s->num_slots);
  if (s->num_slots > kMax31 || s->num_slots * s->H > kMax31 ||
      s->num_slots * s->H * int64_t(s->dv) > kMax31)
    return fail(TREEWY_ERR_UNSUPPORTED, "state pool rows num_slots*H*dv exceed 2^31");
  const int64_t wq = int64_t(s->Hk) * s->dk, wv = int64_t(s->H) * s->dv;
  if ((s->q_stride != 0 && s->q_stride < wq) || (s->k_stride != 0 && s->k_stride < wq) ||
      (s->v_stride != 0 && s->v_stride < wv))
    return fail(TREEWY_ERR_INVALID_ARG, "a token stride is shorter than its row");
  const int64_t limit = int64_t(1) << 31;
  if (s->q_stride > limit || s->k_stride > limit || s->v_stride > limit || wq > limit || wv > limit)
    return fail(TREEWY_ERR_UNSUPPORTED, "token rows are too long");
  if (s->R == 0) return TREEWY_OK;
  if (!s->seq_offset || !s->state || !s->state_slot || !s->status)
    return fail(TREEWY_ERR_INVALID_ARG, "seq_offset, state, state_slot and status must be non-NULL");
  if (s->T > 0 && s->max_len > 0 && (!s->q || !s->k || !s->v || !s->alpha || !s->beta || !s->o))
    return fail(TREEWY_ERR_INVALID_ARG, "q, k, v, alpha, beta and o must be non-NULL");
  if (!aligned(s->state, 16)) return fail(TREEWY_ERR_INVALID_ARG, "state must be 16-byte aligned");
  const uintptr_t e = s->qkv_dtype == TREEWY_DTYPE_BF16 ? 2 : 4;
  const uintptr_t eo = s->o_dtype == TREEWY_DTYPE_BF16 ? 2 : 4;
  if (!aligned(s->q, e) || !aligned(s->k, e) || !aligned(s->v, e) || !aligned(s->o, eo) ||
      !aligned(s->alpha, 4) || !aligned(s->beta, 4))
    return fail(TREEWY_ERR_INVALID_ARG, "q, k, v, o, alpha and beta must be aligned to their elements");
  if (!aligned(s->seq_offset, 4) || !aligned(s->state_slot, 4) || !aligned(s->status, 4))
    return fail(TREEWY_ERR_INVALID_ARG, "seq_offset, state_slot and status must be aligned to their elements");
  return TREEWY_OK;
}

// Batches whose longest sequence has at least this many tokens run in chunks.
// A chunk takes 14 (bf16 pool) to 17 us whatever its length; token by token it
// is 0.2 to 0.3 us a token (128 x 128 heads) while a head's rows have the SMs
// to themselves, more when heads share them.  Chunks against tokens, us, on a
// bf16 pool and on an f32 one:
//   40 heads,   33 tokens   14.4 / 14.5   16.5 / 14.7
//               40          14.4 / 15.6   16.5 / 15.8
//               48          14.4 / 17.8   16.5 / 18.1
//   80 heads,   12          14.4 / 11.5   16.5 / 12.8
//               16          14.4 / 14.5   16.5 / 16.3
//               20          14.4 / 18.6   16.5 / 19.1
//   2048 heads, 10           164 / 154     208 / 137
//               13           166 / 195     209 / 171
//               16           166 / 234     209 / 215
int chunked_len(const treewy_seqs& s) {
  const bool sb = (s.flags & TREEWY_FLAG_STATE_BF16) != 0;
  return int64_t(s.R) * s.H > 64 ? (sb ? 13 : 16) : (sb ? 33 : 43);
}

// Whether the chunked kernel takes the batch (s: strides resolved).  f32
// outputs over a bf16 pool go token by token: chunks are 4e-6 to 5e-6 off, so
// that one value in 500 of the state that a call stores rounds to the other
// side, 2^-8 away (one in 10^4 with f32 sums), and the next call's f32 outputs
// show it: the second of two calls of 70 tokens (decays above 0.97) is 6.3e-5
// off in the norm, 2.3e-5 token by token; of 1000 tokens 2.1e-5 and 2.4e-6.
// bf16 outputs do not show it beside their own 2^-9.  So the sequences that
// gain are those whose calls all have f32 outputs: after a call with bf16
// outputs that ran in chunks its roundings are in the state, unless that call
// set TREEWY_FLAG_FORCE_GENERIC.  It costs time: 1010 us for 4096 tokens of 32
// heads, where chunks with bf16 outputs take 290 us.
bool use_chunks(const treewy_seqs& s) {
  const bool rounded_state = (s.flags & TREEWY_FLAG_STATE_BF16) != 0 && s.o_dtype == TREEWY_DTYPE_F32;
  auto rows_on16 = [](const void* p, int64_t stride) { return aligned(p, 16) && stride % 8 == 0; };
  return s.qkv_dtype == TREEWY_DTYPE_BF16 && s.dk % 8 == 0 && s.dv % 8 == 0 && s.T > 0 && !rounded_state &&
         s.max_len >= chunked_len(s) && (s.flags & TREEWY_FLAG_FORCE_GENERIC) == 0 &&
         rows_on16(s.q, s.q_stride) && rows_on16(s.k, s.k_stride) && rows_on16(s.v, s.v_stride) &&
         aligned(s.o, 16);
}

treewy_status make_extend_maps(const treewy_seqs& s, treewy::ExtendMaps* m) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = treewy::encode_fn();
  if (enc == nullptr) return fail(TREEWY_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint32_t ones[3] = {1, 1, 1};
  struct {
    CUtensorMap* map;
    const void* p;
    int heads, d;
    int64_t stride;
    cuuint32_t cols;
  } const of[3] = {{&m->q, s.q, s.Hk, s.dk, s.q_stride, 64},
                   {&m->k, s.k, s.Hk, s.dk, s.k_stride, 64},
                   {&m->v, s.v, s.H, s.dv, s.v_stride, 128}};
  for (const auto& x : of) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(x.d), static_cast<cuuint64_t>(x.heads),
                                static_cast<cuuint64_t>(s.T)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(x.d) * 2, static_cast<cuuint64_t>(x.stride) * 2};
    const cuuint32_t box[3] = {x.cols, 1, 64};
    const CUresult rc = enc(x.map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x.p), dims, strides, box,
                            ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            x.cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (rc != CUDA_SUCCESS) return fail(TREEWY_ERR_CUDA, "tensor map for q, k or v failed (%d)", (int)rc);
  }
  return TREEWY_OK;
}

treewy_status validate_qk(const treewy_qk* a) {
  if (a == nullptr) return fail(TREEWY_ERR_INVALID_ARG, "qk is NULL");
  if (a->T < 0 || a->T > kMax31)
    return fail(TREEWY_ERR_INVALID_ARG, "T = %lld outside [0, 2^31)", (long long)a->T);
  if (a->Hq < 0 || a->Hk < 0 || int64_t(a->Hq) + a->Hk < 1)
    return fail(TREEWY_ERR_INVALID_ARG, "Hq = %d, Hk = %d: at least one head is needed", a->Hq, a->Hk);
  if (a->d < 1) return fail(TREEWY_ERR_INVALID_ARG, "d = %d must be >= 1", a->d);
  if (a->d > 256) return fail(TREEWY_ERR_UNSUPPORTED, "d = %d: head sizes above 256 are not supported", a->d);
  if (a->dtype != TREEWY_DTYPE_BF16 && a->dtype != TREEWY_DTYPE_F32)
    return fail(TREEWY_ERR_INVALID_ARG, "dtype = %d is not TREEWY_DTYPE_BF16/F32", a->dtype);
  if (a->norm != TREEWY_NORM_L2 && a->norm != TREEWY_NORM_RMS)
    return fail(TREEWY_ERR_INVALID_ARG, "norm = %d is not TREEWY_NORM_L2/RMS", a->norm);
  if (!(a->eps >= 0.f)) return fail(TREEWY_ERR_INVALID_ARG, "eps must be >= 0");
  if (a->rope_dims < 0 || a->rope_dims > a->d || a->rope_dims % 2 != 0)
    return fail(TREEWY_ERR_INVALID_ARG, "rope_dims = %d must be even and in [0, d]", a->rope_dims);
  if (a->q_repeat < 1 || a->k_repeat < 1)
    return fail(TREEWY_ERR_INVALID_ARG, "q_repeat = %d, k_repeat = %d must be >= 1", a->q_repeat, a->k_repeat);
  const int64_t heads = int64_t(a->Hq) + a->Hk;
  if (heads > (1 << 20) || a->q_repeat > (1 << 20) || a->k_repeat > (1 << 20))
    return fail(TREEWY_ERR_UNSUPPORTED, "more than 2^20 heads or repeats");
  // the element-wise kernel's grid: eight rows per CTA
  if (a->T * heads > 8 * kMax31)
    return fail(TREEWY_ERR_UNSUPPORTED, "T * (Hq + Hk) = %lld rows are too many", (long long)(a->T * heads));
  if ((a->q_stride != 0 && a->q_stride < int64_t(a->Hq) * a->d) ||
      (a->k_stride != 0 && a->k_stride < int64_t(a->Hk) * a->d))
    return fail(TREEWY_ERR_INVALID_ARG, "a token stride is shorter than its row");
  if (a->q_stride > (int64_t(1) << 31) || a->k_stride > (int64_t(1) << 31))
    return fail(TREEWY_ERR_UNSUPPORTED, "token rows are too long");
  if (a->T == 0) return TREEWY_OK;
  const uintptr_t e = a->dtype == TREEWY_DTYPE_BF16 ? 2 : 4;
  if (a->Hq > 0 && (!a->q || !a->q_out)) return fail(TREEWY_ERR_INVALID_ARG, "q and q_out must be non-NULL");
  if (a->Hk > 0 && (!a->k || !a->k_out)) return fail(TREEWY_ERR_INVALID_ARG, "k and k_out must be non-NULL");
  if (!aligned(a->q, e) || !aligned(a->k, e) || !aligned(a->q_out, e) || !aligned(a->k_out, e) ||
      !aligned(a->q_weight, 4) || !aligned(a->k_weight, 4) || !aligned(a->rope, 4) || !aligned(a->position, 4) ||
      !aligned(a->status, 4))
    return fail(TREEWY_ERR_INVALID_ARG, "rows, weights, table, position and status must be aligned to their elements");
  if (a->Hq > 0 && a->q_out == a->q &&
      (a->q_repeat != 1 || stride_or(a->q_stride, int64_t(a->Hq) * a->d) != int64_t(a->Hq) * a->d))
    return fail(TREEWY_ERR_INVALID_ARG, "q_out = q needs q_repeat = 1 and dense rows");
  if (a->Hk > 0 && a->k_out == a->k &&
      (a->k_repeat != 1 || stride_or(a->k_stride, int64_t(a->Hk) * a->d) != int64_t(a->Hk) * a->d))
    return fail(TREEWY_ERR_INVALID_ARG, "k_out = k needs k_repeat = 1 and dense rows");
  if (a->rope_dims > 0) {
    if (!a->rope || !a->position || !a->status)
      return fail(TREEWY_ERR_INVALID_ARG, "rope, position and status must be non-NULL with a rotation");
    if (a->rope_rows < 1)
      return fail(TREEWY_ERR_INVALID_ARG, "rope_rows = %lld must be >= 1", (long long)a->rope_rows);
  }
  return TREEWY_OK;
}

treewy_status validate_slots(const treewy_slots* a) {
  if (a == nullptr) return fail(TREEWY_ERR_INVALID_ARG, "slots is NULL");
  if (a->n < 0 || a->layers < 0)
    return fail(TREEWY_ERR_INVALID_ARG, "n = %d, layers = %d must be >= 0", a->n, a->layers);
  if (a->num_slots < 1 || a->slot_bytes < 1)
    return fail(TREEWY_ERR_INVALID_ARG, "num_slots = %lld, slot_bytes = %lld must be >= 1",
                (long long)a->num_slots, (long long)a->slot_bytes);
  if (a->num_slots > kMax31 || a->slot_bytes > (int64_t(1) << 40) / a->num_slots)
    return fail(TREEWY_ERR_UNSUPPORTED, "a pool above 2^40 bytes is not supported");
  if (a->layer_stride < 0 || a->layer_stride > (int64_t(1) << 40) ||
      (a->layers > 1 && a->layer_stride != 0 && a->layer_stride < a->num_slots * a->slot_bytes))
    return fail(TREEWY_ERR_INVALID_ARG, "layer_stride = %lld is shorter than a pool or above 2^40",
                (long long)a->layer_stride);
  if (a->n == 0 || a->layers == 0) return TREEWY_OK;
  if (!a->state || !a->src || !a->dst || !a->status)
    return fail(TREEWY_ERR_INVALID_ARG, "state, src, dst and status must be non-NULL");
  if (!aligned(a->src, 4) || !aligned(a->dst, 4) || !aligned(a->status, 4))
    return fail(TREEWY_ERR_INVALID_ARG, "src, dst and status must be aligned to their elements");
  return TREEWY_OK;
}

}  // namespace

extern "C" {

treewy_status treewy_extend(const treewy_seqs* seqs, cudaStream_t stream) {
  treewy::clear_error();
  treewy_status st = validate_seqs(seqs);
  if (st != TREEWY_OK || seqs->R == 0) return st;
  treewy_seqs s = *seqs;
  s.q_stride = stride_or(s.q_stride, int64_t(s.Hk) * s.dk);
  s.k_stride = stride_or(s.k_stride, int64_t(s.Hk) * s.dk);
  s.v_stride = stride_or(s.v_stride, int64_t(s.H) * s.dv);
  cudaError_t err;
  if (use_chunks(s)) {
    treewy::ExtendMaps maps;
    st = make_extend_maps(s, &maps);
    if (st != TREEWY_OK) return st;
    err = treewy::launch_extend_chunk(s, maps, stream);
  } else {
    err = treewy::launch_extend_scan(s, stream);
  }
  return err == cudaSuccess ? TREEWY_OK : cuda_fail(err, "treewy_extend launch");
}

treewy_status treewy_qk_norm(const treewy_qk* qk, cudaStream_t stream) {
  treewy::clear_error();
  treewy_status st = validate_qk(qk);
  if (st != TREEWY_OK || qk->T == 0) return st;
  treewy_qk a = *qk;
  a.q_stride = stride_or(a.q_stride, int64_t(a.Hq) * a.d);
  a.k_stride = stride_or(a.k_stride, int64_t(a.Hk) * a.d);
  const cudaError_t err = treewy::launch_qk_norm(a, stream);
  return err == cudaSuccess ? TREEWY_OK : cuda_fail(err, "treewy_qk_norm launch");
}

treewy_status treewy_copy_slots(const treewy_slots* slots, cudaStream_t stream) {
  treewy::clear_error();
  treewy_status st = validate_slots(slots);
  if (st != TREEWY_OK || slots->n == 0 || slots->layers == 0) return st;
  const cudaError_t err = treewy::launch_copy_slots(*slots, stream);
  if (err == cudaErrorNotSupported)
    return fail(TREEWY_ERR_UNSUPPORTED, "%d moves in %d layers of %lld bytes each are too many for one call", slots->n,
                slots->layers, (long long)slots->slot_bytes);
  return err == cudaSuccess ? TREEWY_OK : cuda_fail(err, "treewy_copy_slots launch");
}

}  // extern "C"
