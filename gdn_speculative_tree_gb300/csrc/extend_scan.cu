// extend_scan.cu -- the gated delta rule token by token on CUDA cores
// (TreeWY paper §1 Eq. (1)), for any head size dk, dv <= 128:
//
//   u_t = beta_t (v_t - alpha_t S k_t),  S <- alpha_t S + u_t k_t^T,
//   o_t = S q_t = alpha_t (S_old q_t) + (k_t . q_t) u_t,
//
// so that S k_t and S q_t are both taken of the old state in one sweep over
// it, and the state is touched once per token.
//
// The state lives in registers, f32 whatever the pool's type: eight lanes
// share a row of S (each holds 16 of its dk columns, in pieces of 16 bytes of
// the pool, so that a warp's load covers whole 128-byte lines), a warp holds
// four rows per register row, and dot products over a row are three shuffles.
// The type of q, k and v is a template argument: behind a branch on it every
// load would be followed by its conversion, one load's latency after the other
// (64 tokens x 32 heads on a bf16 pool: 25 us, 32 with the branch).
//
// decode_kernel: at most one token per sequence, 16 rows per warp.  Its time is the state's way in and out of HBM (2 x 64 KB per f32
// head against 1.3 KB of everything else); nothing depends on the state's load
// but the token's own arithmetic.  256 tokens x 32 heads, f32: 159 us, 6.8 TB/s,
// the rate of a plain copy.
//
// few_kernel: the same for up to 12 or 16 tokens (2048 heads x 4 tokens: 67 us,
// 92 to 126 us by the staged kernel below), bound by the chain of shuffles.
//
// scan_kernel: any number of tokens, for the sizes and types that the chunked
// kernel does not take.  Four tokens take one sweep of the state: with G_n the
// product of the decays from the first of them to n,
//
//   u_n = beta_n (v_n - G_n S k_n) - sum_{j<n} beta_n (G_n/G_j) (k_n . k_j) u_j,
//   o_n = G_n S q_n + sum_{j<=n} (G_n/G_j) (q_n . k_j) u_j,
//   S <- G_4 S + sum_j (G_4/G_j) u_j k_j^T
//
// (the quotients as products of the decays between, so that a decay of zero is
// right), which turns eight sums over a row's lanes into seven shuffles for
// all four tokens and one chain per four tokens.  Four warps of a CTA stage
// the next 16 tokens and their blocks' products meanwhile.  Bound by issue and
// by the reads of k and q from shared memory: 4096 tokens of 32 heads 996 us
// (3262 us a token at a time, staged by the warps that use it); with one head
// per eight SMs by the staging, 0.15 us a token.
#include <type_traits>

#include "serving_device.cuh"
#include "treewy_device.cuh"
#include "treewy_internal.h"

namespace treewy {
namespace {

constexpr int kFewWarps = 1, kFewThreads = 32 * kFewWarps;
constexpr int kStage = 16;  // tokens staged at a time
constexpr int kPrep = 128;  // threads that stage them
constexpr int kBlock = 4;   // tokens that take one sweep of the state
constexpr unsigned kFull = 0xffffffffu;

struct Seq {
  int64_t tok0;
  int len, slot, flags;
  bool fresh;
};

// Sequence r's range and slot, and the status bits of what is wrong with them.
__device__ __forceinline__ Seq load_seq(const treewy_seqs& a, int r) {
  const int lo = __ldg(a.seq_offset + r), hi = __ldg(a.seq_offset + r + 1);
  Seq s;
  s.slot = __ldg(a.state_slot + r);
  s.fresh = a.fresh != nullptr && __ldg(a.fresh + r) != 0;
  const int64_t len = static_cast<int64_t>(hi) - lo;
  s.flags = 0;
  if (len < 0 || len > a.max_len) s.flags |= TREEWY_STATUS_TOO_MANY_NODES;
  else if (lo < 0 || hi > a.T) s.flags |= TREEWY_STATUS_BAD_TREE;
  if (s.slot < 0 || s.slot >= a.num_slots) s.flags |= TREEWY_STATUS_BAD_SLOT;
  s.tok0 = lo;
  s.len = static_cast<int>(len);
  return s;
}

// First column of piece i of lane l (0..7) of a row group: pieces of V columns.
template <int V>
__device__ __forceinline__ int piece_col(int l, int i) {
  return V * (l + 8 * i);
}

// The CL columns (16 of up to 128, 8 of up to 64) of lane l of a row of n elements, zero beyond it.  WIDE: the
// row starts on a 16-byte boundary of the pool's type (a q/k row on a
// boundary of V elements) and n is a multiple of V.
template <int V, bool WIDE, int CL>
__device__ __forceinline__ void load_row(const void* base, bool bf16, int64_t at, int n, int l,
                                         float (&x)[CL]) {
#pragma unroll
  for (int i = 0; i < CL / V; ++i) {
    const int c0 = piece_col<V>(l, i);
#pragma unroll
    for (int e = 0; e < V; ++e) x[V * i + e] = 0.f;
    if constexpr (WIDE) {
      if (c0 < n) {
        if (bf16) {
          const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at + c0;
          uint32_t w[V / 2];
          if constexpr (V == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[0] = u.x; w[1] = u.y;
          }
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            x[V * i + 2 * e] = __uint_as_float(w[e] << 16);
            x[V * i + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
          }
        } else {
          const float* p = reinterpret_cast<const float*>(base) + at + c0;
#pragma unroll
          for (int e = 0; e < V; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(p + e);
            x[V * i + e] = f.x;
            x[V * i + e + 1] = f.y;
            x[V * i + e + 2] = f.z;
            x[V * i + e + 3] = f.w;
          }
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (c0 + e < n) {
          x[V * i + e] = bf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(base)[at + c0 + e])
                              : reinterpret_cast<const float*>(base)[at + c0 + e];
        }
      }
    }
  }
}

// The same columns back to the pool, which the next layers' pools push out of
// L2 before it is read again; a bf16 pool rounds to nearest even.
template <int V, bool WIDE, int CL>
__device__ __forceinline__ void store_row(void* base, bool bf16, int64_t at, int n, int l,
                                          const float (&x)[CL]) {
#pragma unroll
  for (int i = 0; i < CL / V; ++i) {
    const int c0 = piece_col<V>(l, i);
    if constexpr (WIDE) {
      if (c0 < n) {
        if (bf16) {
          uint32_t w[V / 2];
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[V * i + 2 * e], x[V * i + 2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&p);
          }
          uint16_t* p = reinterpret_cast<uint16_t*>(base) + at + c0;
          if constexpr (V == 8) __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
          else __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
        } else {
          float* p = reinterpret_cast<float*>(base) + at + c0;
#pragma unroll
          for (int e = 0; e < V; e += 4)
            __stcs(reinterpret_cast<float4*>(p + e), make_float4(x[V * i + e], x[V * i + e + 1],
                                                                 x[V * i + e + 2], x[V * i + e + 3]));
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (c0 + e < n) {
          if (bf16) reinterpret_cast<__nv_bfloat16*>(base)[at + c0 + e] = __float2bfloat16_rn(x[V * i + e]);
          else reinterpret_cast<float*>(base)[at + c0 + e] = x[V * i + e];
        }
      }
    }
  }
}

__device__ __forceinline__ float sum8(float x) {
  x += __shfl_xor_sync(kFull, x, 4);
  x += __shfl_xor_sync(kFull, x, 2);
  x += __shfl_xor_sync(kFull, x, 1);
  return x;
}

__device__ __forceinline__ void store_o(const treewy_seqs& a, int64_t at, float x) {
  if (a.o_dtype == TREEWY_DTYPE_BF16) reinterpret_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(x);
  else reinterpret_cast<float*>(a.o)[at] = x;
}

// Row of register row j of this lane's group, `first` the CTA's first row: a
// warp's four groups hold neighbouring rows.
template <int RPT>
__device__ __forceinline__ int group_row(int first, int j) {
  const int warp = threadIdx.x >> 5, grp = (threadIdx.x & 31) >> 3;
  return first + 4 * (warp * RPT + j) + grp;
}

// The 16 columns of a row as they are stored: pieces of 16 bytes.
template <bool SB>
struct RawRow {
  uint4 w[SB ? 2 : 4];
};
template <bool SB>
__device__ __forceinline__ void unpack_row(const RawRow<SB>& r, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < (SB ? 2 : 4); ++i) {
    const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (SB) {
        x[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
        x[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      } else {
        x[4 * i + e] = __uint_as_float(w[e]);
      }
    }
  }
}

// One (sequence, head) and 4 WARPS RPT of its rows per CTA, one token
// at most.  WIDE: every load of the state, q and k is a whole piece; the rows
// then wait in registers as they are stored, all of them in flight at once,
// and are taken one after the other.
template <int RPT, int WARPS, bool SB, bool QB, bool WIDE>
__global__ void __launch_bounds__(32 * WARPS) decode_kernel(const treewy_seqs a) {
  after_previous();
  constexpr int V = SB ? 8 : 4;
  const int r = blockIdx.x / a.H, h = blockIdx.x - r * a.H;
  const int l = threadIdx.x & 7;
  const int first = static_cast<int>(blockIdx.y) * (4 * WARPS * RPT);
  const Seq s = load_seq(a, r);
  if (s.flags) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && h == 0) atomicOr(a.status + r, s.flags);
    return;
  }
  if (s.len == 0 && !s.fresh) return;
  const int64_t block = (static_cast<int64_t>(s.slot) * a.H + h) * a.dv;
  RawRow<SB> raw[RPT];
  if constexpr (WIDE) {
    const unsigned char* p = reinterpret_cast<const unsigned char*>(a.state);
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
      const int row = group_row<RPT>(first, j);
#pragma unroll
      for (int i = 0; i < 16 / V; ++i) {
        raw[j].w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (!s.fresh && row < a.dv && piece_col<V>(l, i) < a.dk)
          raw[j].w[i] = __ldcs(reinterpret_cast<const uint4*>(p + ((block + row) * a.dk + piece_col<V>(l, i)) * (SB ? 2 : 4)));
      }
    }
  }
  const int64_t t = s.tok0;
  float k[16], q[16], v[RPT], alpha = 1.f, beta = 0.f, kq = 0.f;
  if (s.len > 0) {
    const int hk = h / (a.H / a.Hk);
    load_row<V, WIDE>(a.k, QB, t * a.k_stride + static_cast<int64_t>(hk) * a.dk, a.dk, l, k);
    load_row<V, WIDE>(a.q, QB, t * a.q_stride + static_cast<int64_t>(hk) * a.dk, a.dk, l, q);
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
      const int row = group_row<RPT>(first, j);
      v[j] = row < a.dv ? load_qkv(a.v, t * a.v_stride + static_cast<int64_t>(h) * a.dv + row, QB) : 0.f;
    }
    alpha = __ldg(a.alpha + t * a.H + h);
    beta = __ldg(a.beta + t * a.H + h);
#pragma unroll
    for (int c = 0; c < 16; ++c) kq = fmaf(k[c], q[c], kq);
    kq = sum8(kq);
  }
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
    const int row = group_row<RPT>(first, j);
    float S[16];
    if constexpr (WIDE) {
      unpack_row<SB>(raw[j], S);
    } else if (!s.fresh && row < a.dv) {
      load_row<V, false>(a.state, SB, (block + row) * a.dk, a.dk, l, S);
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) S[c] = 0.f;
    }
    if (s.len > 0) {
      float sk = 0.f, sq = 0.f;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        sk = fmaf(S[c], k[c], sk);
        sq = fmaf(S[c], q[c], sq);
      }
      sk = sum8(sk);
      sq = sum8(sq);
      const float u = beta * (v[j] - alpha * sk);
#pragma unroll
      for (int c = 0; c < 16; ++c) S[c] = fmaf(u, k[c], alpha * S[c]);
      if (l == 0 && row < a.dv) store_o(a, (t * a.H + h) * a.dv + row, fmaf(kq, u, alpha * sq));
    }
    if (row < a.dv) store_row<V, WIDE>(a.state, SB, (block + row) * a.dk, a.dk, l, S);
  }
}

// The same split for a few tokens: S in f32 registers over all of them, the
// next token's rows on their way meanwhile.
template <int RPT, bool SB, bool QB, bool WIDE>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const treewy_seqs a) {
  after_previous();
  constexpr int V = SB ? 8 : 4;
  const int r = blockIdx.x / a.H, h = blockIdx.x - r * a.H;
  const int l = threadIdx.x & 7;
  const int first = static_cast<int>(blockIdx.y) * (4 * kFewWarps * RPT);
  const Seq s = load_seq(a, r);
  if (s.flags) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && h == 0) atomicOr(a.status + r, s.flags);
    return;
  }
  if (s.len == 0 && !s.fresh) return;
  const int64_t block = (static_cast<int64_t>(s.slot) * a.H + h) * a.dv;
  float S[RPT][16];
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
    const int row = group_row<RPT>(first, j);
    if (!s.fresh && row < a.dv) {
      load_row<V, WIDE>(a.state, SB, (block + row) * a.dk, a.dk, l, S[j]);
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) S[j][c] = 0.f;
    }
  }
  const int hk = h / (a.H / a.Hk);
  float k[2][16], q[2][16], v[2][RPT], alpha[2], beta[2];
  auto next = [&](int n, int slot) {
    const int64_t t = s.tok0 + n;
    load_row<V, WIDE>(a.k, QB, t * a.k_stride + static_cast<int64_t>(hk) * a.dk, a.dk, l, k[slot]);
    load_row<V, WIDE>(a.q, QB, t * a.q_stride + static_cast<int64_t>(hk) * a.dk, a.dk, l, q[slot]);
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
      const int row = group_row<RPT>(first, j);
      v[slot][j] = row < a.dv ? load_qkv(a.v, t * a.v_stride + static_cast<int64_t>(h) * a.dv + row, QB) : 0.f;
    }
    alpha[slot] = __ldg(a.alpha + t * a.H + h);
    beta[slot] = __ldg(a.beta + t * a.H + h);
  };
  if (s.len > 0) next(0, 0);
#pragma unroll 1
  for (int n0 = 0; n0 < s.len; n0 += 2) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int n = n0 + p;
      if (n >= s.len) break;
      if (n + 1 < s.len) next(n + 1, p ^ 1);
      float2 prod = make_float2(0.f, 0.f), sk[RPT], sq[RPT];
#pragma unroll
      for (int j = 0; j < RPT; ++j) sk[j] = sq[j] = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        const float2 kc = make_float2(k[p][c], k[p][c + 1]), qc = make_float2(q[p][c], q[p][c + 1]);
        prod = fma2(kc, qc, prod);
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
          const float2 s2 = make_float2(S[j][c], S[j][c + 1]);
          sk[j] = fma2(s2, kc, sk[j]);
          sq[j] = fma2(s2, qc, sq[j]);
        }
      }
      const float kq = sum8(prod.x + prod.y);
      // lanes 0-3 of a row get S k, the others S q
      float x[RPT], u[RPT];
#pragma unroll
      for (int j = 0; j < RPT; ++j) {
        const float y = sk[j].x + sk[j].y, z = sq[j].x + sq[j].y;
        x[j] = ((l & 4) ? z : y) + __shfl_xor_sync(kFull, (l & 4) ? y : z, 4);
      }
#pragma unroll
      for (int j = 0; j < RPT; ++j) x[j] += __shfl_xor_sync(kFull, x[j], 2);
#pragma unroll
      for (int j = 0; j < RPT; ++j) x[j] = alpha[p] * (x[j] + __shfl_xor_sync(kFull, x[j], 1));
#pragma unroll
      for (int j = 0; j < RPT; ++j) u[j] = __shfl_sync(kFull, beta[p] * (v[p][j] - x[j]), 0, 8);
#pragma unroll
      for (int j = 0; j < RPT; ++j) {
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          const float2 y = fma2(make_float2(u[j], u[j]), make_float2(k[p][c], k[p][c + 1]),
                                mul2(make_float2(alpha[p], alpha[p]), make_float2(S[j][c], S[j][c + 1])));
          S[j][c] = y.x;
          S[j][c + 1] = y.y;
        }
        const int row = group_row<RPT>(first, j);
        if (l == 4 && row < a.dv) store_o(a, ((s.tok0 + n) * a.H + h) * a.dv + row, fmaf(kq, u[j], x[j]));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
    const int row = group_row<RPT>(first, j);
    if (row < a.dv) store_row<V, WIDE>(a.state, SB, (block + row) * a.dk, a.dk, l, S[j]);
  }
}

// Staged tokens, f32: 8 CL columns of k and q (zero beyond dk) and the CTA's
// rows of v (zero beyond dv); behind the sequence's end k, q, v and beta are
// zero and alpha is one.  The factors of a block of kBlock tokens, with G_n the
// product of the decays from the block's first token to n:
template <int CL, int ROWS>
struct Stage {
  float k[kStage][8 * CL];
  float q[kStage][8 * CL];
  float v[kStage][ROWS];
  float kk[kStage][kBlock];    // beta_n (G_n / G_j) k_n . k_j   (j < n)
  float kq[kStage][kBlock];    // (G_n / G_j) q_n . k_j          (j <= n)
  float dec[kStage];           // G of the block's last token / G_n
  float gate[kStage];          // G_n
  float alpha[kStage], beta[kStage];
};

// Sums over the eight lanes of a row group of eight values per row: lane l gets
// value l's.  Step by step for all rows, so that one's shuffle need not wait
// for another's.
template <int RPT>
__device__ __forceinline__ void sum8_each(const float (&x)[RPT][8], int l, float (&out)[RPT]) {
  float y[RPT][4], z[RPT][2];
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      y[j][e] = ((l & 4) ? x[j][e + 4] : x[j][e]) + __shfl_xor_sync(kFull, (l & 4) ? x[j][e] : x[j][e + 4], 4);
  }
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      z[j][e] = ((l & 2) ? y[j][e + 2] : y[j][e]) + __shfl_xor_sync(kFull, (l & 2) ? y[j][e] : y[j][e + 2], 2);
  }
#pragma unroll
  for (int j = 0; j < RPT; ++j)
    out[j] = ((l & 1) ? z[j][1] : z[j][0]) + __shfl_xor_sync(kFull, (l & 1) ? z[j][0] : z[j][1], 1);
}

template <int ID, int N>
__device__ __forceinline__ void bar_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(N) : "memory");
}

// One (sequence, head) and THREADS / 8 x RPT of its rows per CTA, CL columns
// of a row per lane, any number of tokens.  kPrep more threads stage the next
// tokens and their blocks' factors meanwhile.
template <int RPT, bool SB, bool QB, bool WIDE, int CL, int THREADS>
__global__ void __launch_bounds__(THREADS + kPrep) scan_kernel(const treewy_seqs a) {
  constexpr int V = 4, kRows = THREADS / 8 * RPT, kCols = 8 * CL, kAll = THREADS + kPrep;
  __shared__ __align__(16) Stage<CL, kRows> stages[2];
  after_previous();
  const int idx = blockIdx.x / a.H, h = blockIdx.x - idx * a.H, r = longest_first(a, idx);
  const int l = threadIdx.x & 7;
  const Seq s = load_seq(a, r);
  if (s.flags) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && h == 0) atomicOr(a.status + r, s.flags);
    return;
  }
  if (s.len == 0 && !s.fresh) return;
  const int first = static_cast<int>(blockIdx.y) * kRows;

  if (threadIdx.x >= THREADS) {
    const int tid = threadIdx.x - THREADS, hk = h / (a.H / a.Hk);
    constexpr int kPer = kStage * kCols / kPrep;  // staged elements of k (and q) per thread
    constexpr int kPerV = kStage * kRows / kPrep;
    // as they are stored: a conversion here would wait for its load
    using Raw = std::conditional_t<QB, uint16_t, float>;
    const Raw *pk = static_cast<const Raw*>(a.k), *pq = static_cast<const Raw*>(a.q), *pv = static_cast<const Raw*>(a.v);
    auto value = [](Raw x) {
      if constexpr (QB) return bf16_bits_to_float(x);
      else return x;
    };
    Raw nk[kPer], nq[kPer], nv[kPerV];
    float ngate = 0.f;
    auto fetch = [&](int t0) {  // the stage from token t0 on, into registers
      {
        constexpr int kHop = kPrep / kCols;  // tokens between a thread's elements, all of one column
        const int n0 = tid / kCols, c = tid % kCols;
        const Raw* k = pk + (s.tok0 + t0 + n0) * a.k_stride + static_cast<int64_t>(hk) * a.dk + c;
        const Raw* q = pq + (s.tok0 + t0 + n0) * a.q_stride + static_cast<int64_t>(hk) * a.dk + c;
#pragma unroll
        for (int i = 0; i < kPer; ++i, k += kHop * a.k_stride, q += kHop * a.q_stride) {
          nk[i] = nq[i] = 0;
          if (t0 + n0 + i * kHop < s.len && c < a.dk) {
            nk[i] = __ldg(k);
            nq[i] = __ldg(q);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kPerV; ++i) {
        const int e = tid + i * kPrep, n = e / kRows, c = first + e % kRows;
        nv[i] = 0;
        if (t0 + n < s.len && c < a.dv)
          nv[i] = __ldg(pv + (s.tok0 + t0 + n) * a.v_stride + static_cast<int64_t>(h) * a.dv + c);
      }
      if (tid < 2 * kStage) {
        const int n = tid & (kStage - 1);
        ngate = tid < kStage ? 1.f : 0.f;
        const float* g = tid < kStage ? a.alpha : a.beta;
        if (t0 + n < s.len) ngate = __ldg(g + (s.tok0 + t0 + n) * a.H + h);
      }
    };
    fetch(0);
    for (int t0 = 0; t0 < s.len; t0 += kStage) {
      Stage<CL, kRows>& st = stages[t0 / kStage & 1];  // its last tokens were done before the last barrier
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        (&st.k[0][0])[tid + i * kPrep] = value(nk[i]);
        (&st.q[0][0])[tid + i * kPrep] = value(nq[i]);
      }
#pragma unroll
      for (int i = 0; i < kPerV; ++i) (&st.v[0][0])[tid + i * kPrep] = value(nv[i]);
      if (tid < kStage) st.alpha[tid] = ngate;
      else if (tid < 2 * kStage) st.beta[tid - kStage] = ngate;
      bar_sync<1, kPrep>();
      fetch(t0 + kStage);
      const int m = min(kStage, s.len - t0);
      // 10 products q_n . k_j and 6 k_n . k_j of each block, eight lanes per product
#pragma unroll 2
      for (int p = tid >> 3; p < kStage / kBlock * 16; p += kPrep / 8) {
        const int b = p / 16 * kBlock, e = p % 16;
        if (b >= m) break;  // whole warps: 4 products of one block each
        const bool isq = e < 10;
        const int f = isq ? e : e - 10;
        const int n = isq ? (f >= 6 ? 3 : f >= 3 ? 2 : f >= 1 ? 1 : 0) : (f >= 3 ? 3 : f >= 1 ? 2 : 1);
        const int j = f - (isq ? n * (n + 1) / 2 : n * (n - 1) / 2);
        float x[CL], y[CL];
        float2 sum = make_float2(0.f, 0.f);
        load_row<V, true>(isq ? st.q[b + n] : st.k[b + n], false, 0, kCols, l, x);
        load_row<V, true>(st.k[b + j], false, 0, kCols, l, y);
#pragma unroll
        for (int c = 0; c < CL; c += 2) sum = fma2(make_float2(x[c], x[c + 1]), make_float2(y[c], y[c + 1]), sum);
        const float4 al = *reinterpret_cast<const float4*>(st.alpha + b);
        const float beta = st.beta[b + n];
        const float a1 = j < 1 && n >= 1 ? al.y : 1.f, a2 = j < 2 && n >= 2 ? al.z : 1.f, a3 = n >= 3 && j < 3 ? al.w : 1.f;
        const float z = sum8(sum.x + sum.y) * (isq ? 1.f : beta) * (a1 * a2 * a3);
        if (l == 0) (isq ? st.kq : st.kk)[b + n][j] = z;
      }
      if (tid < kStage) {
        const int n = tid & (kBlock - 1);
        const float4 al = *reinterpret_cast<const float4*>(st.alpha + tid - n);
        const float g = al.x * (n >= 1 ? al.y : 1.f) * (n >= 2 ? al.z : 1.f) * (n >= 3 ? al.w : 1.f);
        const float d = (n < 1 ? al.y : 1.f) * (n < 2 ? al.z : 1.f) * (n < 3 ? al.w : 1.f);
        st.gate[tid] = g;
        st.dec[tid] = d;
      }
      bar_sync<0, kAll>();
    }
    return;
  }

  const int64_t block = (static_cast<int64_t>(s.slot) * a.H + h) * a.dv;
  float S[RPT][CL];
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
    const int row = group_row<RPT>(first, j);
    if (!s.fresh && row < a.dv) {
      load_row<V, WIDE>(a.state, SB, (block + row) * a.dk, a.dk, l, S[j]);
    } else {
#pragma unroll
      for (int c = 0; c < CL; ++c) S[j][c] = 0.f;
    }
  }
  // row 0's output of this lane's token of the first block
  const int64_t at0 = ((s.tok0 + (l & (kBlock - 1))) * a.H + h) * a.dv + group_row<RPT>(first, 0);
  for (int t0 = 0; t0 < s.len; t0 += kStage) {
    const Stage<CL, kRows>& st = stages[t0 / kStage & 1];
    const int m = min(kStage, s.len - t0);
    bar_sync<0, kAll>();
#pragma unroll 1
    for (int b = 0; b < m; b += kBlock) {
      float dot[RPT][2 * kBlock];  // S k_n, then S q_n: this lane's columns
      float k[kBlock][CL];
#pragma unroll
      for (int n = 0; n < kBlock; ++n) {
        float q[CL];
        load_row<V, true>(st.k[b + n], false, 0, kCols, l, k[n]);
        load_row<V, true>(st.q[b + n], false, 0, kCols, l, q);
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
          const float2 s0 = make_float2(S[j][0], S[j][1]);
          float2 x = mul2(s0, make_float2(k[n][0], k[n][1])), y = mul2(s0, make_float2(q[0], q[1]));
#pragma unroll
          for (int c = 2; c < CL; c += 2) {
            const float2 sc = make_float2(S[j][c], S[j][c + 1]);
            x = fma2(sc, make_float2(k[n][c], k[n][c + 1]), x);
            y = fma2(sc, make_float2(q[c], q[c + 1]), y);
          }
          dot[j][n] = x.x + x.y;
          dot[j][kBlock + n] = y.x + y.y;
        }
      }
      // lane l < 4: token l's S k, the others token l - 4's S q
      const int mine = b + (l & (kBlock - 1));
      const float gate = st.gate[mine], beta = st.beta[mine], last = st.gate[b + kBlock - 1];
      const float4 m4 = *reinterpret_cast<const float4*>(st.kq[mine]);
      const float mq[kBlock] = {m4.x, m4.y, m4.z, m4.w};
      const float4 k1 = *reinterpret_cast<const float4*>(st.kk[b + 1]), k2 = *reinterpret_cast<const float4*>(st.kk[b + 2]),
                   k3 = *reinterpret_cast<const float4*>(st.kk[b + 3]);
      float v[RPT], y[RPT], u[RPT][kBlock];
#pragma unroll
      for (int j = 0; j < RPT; ++j) v[j] = st.v[mine][group_row<RPT>(0, j)];
      // the rows' chains side by side
      sum8_each<RPT>(dot, l, y);
#pragma unroll
      for (int j = 0; j < RPT; ++j) {
        y[j] *= gate;
        const float rhs = mine < m ? beta * (v[j] - y[j]) : 0.f;
#pragma unroll
        for (int n = 0; n < kBlock; ++n) u[j][n] = __shfl_sync(kFull, rhs, n, 8);
      }
#pragma unroll
      for (int j = 0; j < RPT; ++j) {
        u[j][1] = b + 1 < m ? fmaf(-k1.x, u[j][0], u[j][1]) : 0.f;
        u[j][2] = b + 2 < m ? fmaf(-k2.y, u[j][1], fmaf(-k2.x, u[j][0], u[j][2])) : 0.f;
        u[j][3] = b + 3 < m ? fmaf(-k3.z, u[j][2], fmaf(-k3.y, u[j][1], fmaf(-k3.x, u[j][0], u[j][3]))) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < RPT; ++j) {
#pragma unroll
        for (int n = 0; n < kBlock; ++n) {
          if (n <= (l & (kBlock - 1))) y[j] = fmaf(mq[n], u[j][n], y[j]);
        }
        const int row = group_row<RPT>(first, j);
        if (l >= kBlock && mine < m && row < a.dv) store_o(a, at0 + (t0 + b) * static_cast<int64_t>(a.H) * a.dv + 4 * j, y[j]);
      }
#pragma unroll
      for (int n = 0; n < kBlock; ++n) {
        const float dec = st.dec[b + n];
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
          const float w = dec * u[j][n];
#pragma unroll
          for (int c = 0; c < CL; c += 2) {
            float2 x = make_float2(S[j][c], S[j][c + 1]);
            if (n == 0) x = mul2(make_float2(last, last), x);
            x = fma2(make_float2(w, w), make_float2(k[n][c], k[n][c + 1]), x);
            S[j][c] = x.x;
            S[j][c + 1] = x.y;
          }
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < RPT; ++j) {
    const int row = group_row<RPT>(first, j);
    if (row < a.dv) store_row<V, WIDE>(a.state, SB, (block + row) * a.dk, a.dk, l, S[j]);
  }
}

template <int RPT, int WARPS, bool SB, bool QB, bool WIDE>
cudaError_t launch_decode(const treewy_seqs& a, cudaStream_t stream) {
  constexpr int kRows = 4 * WARPS * RPT;
  const dim3 grid(static_cast<unsigned>(a.R) * static_cast<unsigned>(a.H),
                  static_cast<unsigned>((a.dv + kRows - 1) / kRows));
  return launch_after(decode_kernel<RPT, WARPS, SB, QB, WIDE>, grid, 32 * WARPS, stream, a);
}

template <int RPT, bool SB, bool QB, bool WIDE>
cudaError_t launch_few(const treewy_seqs& a, cudaStream_t stream) {
  constexpr int kRows = 4 * kFewWarps * RPT;
  const dim3 grid(static_cast<unsigned>(a.R) * static_cast<unsigned>(a.H),
                  static_cast<unsigned>((a.dv + kRows - 1) / kRows));
  return launch_after(few_kernel<RPT, SB, QB, WIDE>, grid, kFewThreads, stream, a);
}

template <int RPT, bool SB, bool QB, bool WIDE, int CL, int THREADS>
cudaError_t launch_scan(const treewy_seqs& a, cudaStream_t stream) {
  constexpr int kRows = THREADS / 8 * RPT;
  const dim3 grid(static_cast<unsigned>(a.R) * static_cast<unsigned>(a.H),
                  static_cast<unsigned>((a.dv + kRows - 1) / kRows));
  return launch_after(scan_kernel<RPT, SB, QB, WIDE, CL, THREADS>, grid, THREADS + kPrep, stream, a);
}

template <bool SB, bool QB, bool WIDE>
cudaError_t launch(const treewy_seqs& a, cudaStream_t stream) {
  const int64_t heads = static_cast<int64_t>(a.R) * a.H;
  // Up to 75 heads spread over as many CTAs as they have rows for; more take 16
  // rows per warp and 64 per CTA (32 on a bf16 pool): 8192 heads 159 us, 177 us
  // with 16 per CTA, 159 us with all 128; on a bf16 pool 94, 94 and 100 us.
  if (a.max_len <= 1)
    return 4 * heads >= 304 ? launch_decode<4, SB ? 2 : 4, SB, QB, WIDE>(a, stream)
                            : launch_decode<1, 1, SB, QB, WIDE>(a, stream);
  // 12 tokens of 32 heads 8.0 us, 16 10.0 us, 20 staged 8.7 us; of 2048 heads 16
  // 210 us, 20 staged 256 us
  if (a.max_len <= (4 * heads >= 304 ? 16 : 12))
    return 4 * heads >= 304 ? launch_few<2, SB, QB, WIDE>(a, stream) : launch_few<1, SB, QB, WIDE>(a, stream);
  // 16 rows of a head per CTA while two CTAs per SM hold them all, then 64;
  // half as many columns per lane for small keys.
  if (8 * heads > 304)
    return a.dk <= 64 ? launch_scan<2, SB, QB, WIDE, 8, 256>(a, stream) : launch_scan<2, SB, QB, WIDE, 16, 256>(a, stream);
  return a.dk <= 64 ? launch_scan<1, SB, QB, WIDE, 8, 128>(a, stream) : launch_scan<1, SB, QB, WIDE, 16, 128>(a, stream);
}

}  // namespace

cudaError_t launch_extend_scan(const treewy_seqs& a, cudaStream_t stream) {
  // pieces of 16 bytes of the pool's type; wide loads where every row of the
  // state, and of q and k for the single-token kernel, starts on a piece
  const int e = a.qkv_dtype == TREEWY_DTYPE_BF16 ? 2 : 4;
  auto rows_on = [&](const void* p, int64_t stride, int64_t piece) {
    return (reinterpret_cast<uintptr_t>(p) % piece) == 0 && (stride * e) % piece == 0;
  };
  const bool sb = (a.flags & TREEWY_FLAG_STATE_BF16) != 0;
  const int v = sb ? 8 : 4;
  const int64_t piece = (v * e < 16) ? v * e : 16;
  const bool wide = a.dk % v == 0 && rows_on(a.q, a.q_stride, piece) && rows_on(a.k, a.k_stride, piece);
  if (e == 2) {
    if (sb) return wide ? launch<true, true, true>(a, stream) : launch<true, true, false>(a, stream);
    return wide ? launch<false, true, true>(a, stream) : launch<false, true, false>(a, stream);
  }
  if (sb) return wide ? launch<true, false, true>(a, stream) : launch<true, false, false>(a, stream);
  return wide ? launch<false, false, true>(a, stream) : launch<false, false, false>(a, stream);
}

}  // namespace treewy
