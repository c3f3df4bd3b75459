// extend_chunk.cu -- the gated delta rule over long sequences in chunks of 64
// tokens on the 5th-generation tensor cores (tcgen05, TMEM, TMA), for bf16
// q/k/v and head sizes that are multiples of 8 up to 128 (smaller heads are
// zero-padded to 128 by the tensor maps).
//
// Within a chunk, with g_t the product of its decays up to token t, the
// recurrence S_t = a_t S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T unrolls to
//
//   (I + A) U = diag(b) W,  A[n,i] = b_n (g_n/g_i) k_n.k_i (i < n),  W_i = v_i - g_i S k_i,
//   o_n = g_n S q_n + sum_{i<=n} M[n,i] u_i,  M[n,i] = (g_n/g_i) q_n.k_i,
//   S'  = g_C S + sum_n (g_C/g_n) u_n k_n^T.
//
// With T = (I + A)^-1 neither sum needs U:
//
//   o_n = g_n S q_n + (MT W)_n,   S' = g_C S + sum_i W_i kt_i^T,
//   MT = M T diag(b),   kt_i = b_i sum_n T[n,i] (g_C/g_n) k_n,
//
// and MT and kt depend on the tokens alone.  So the chain from one
// chunk's state to the next is two products long, S k and W kt; everything
// else is prepared one chunk ahead or follows behind.
//
// One CTA per (sequence, head).  Value rows are TMEM lanes throughout: S, W
// and their products are [dv = 128 lanes][columns], so that a thread owns a
// row, and the left operands S and W go back to TMEM as bf16 without passing
// through shared memory.
//
//   warps 0-7    state: two threads per row (64 of S's columns and 32 tokens
//                each); S stays in f32 registers for the whole sequence
//   warps 8-15   preparation of the next chunk: [K;Q] K^T, T, kt
//   warps 16-19  o; 18 and 19 also MT
//   warp 20      issues the chain's products
//   warp 21      loads K, Q and V, two chunks in flight
//   warp 22      gates
//   warp 23      issues the preparation's products
//
// Products accumulate in f32; keys, queries and values are exact operands, and
// an f32 operand is two bf16 terms x = hi + lo, lo times lo left out: S, W, kt,
// M and MT, each 2^-17 off at most (a third term of all five has no room in
// TMEM and shared memory).  T21 and what it is made from, T and T'' have three
// terms and all products that count: where keys are alike, they are large and
// cancel in what they are multiplied by.  Errors against 64 bits, in the norm
// (512 tokens, heads of 128; sums in f32 token by token: 1e-7 to 1e-6):
//
//   cosine of the keys, b, decay     o (f32)  S       (two terms throughout)
//   0.08, 0 to 1, 0.9 to 1           5e-6     4e-6    (5e-6, 5e-6)
//   0.9, 1, 1                        7e-6     6e-6    (2e-5, 2e-5)
//   0.99, 1, 1                       1e-5     6e-6    (3e-5, 3e-5)
//   0.9, 1.9, 1                      1e-5     1e-5    (1e-4, 1e-4)
//   0.99, 2, 1                       5e-5     5e-5    (1e-3, 1e-3)
//
// bf16 outputs leave M T's smallest products out: up to 2e-4 in the last two
// lines, against the 2^-9 of their own rounding (290 against 306 us for 4096
// tokens of 32 heads; the state does not depend on it).  Ratios g_n/g_i are
// running products of the decays between i and n, never quotients, so they are
// right however small g has become, a decay of zero included.
//
// Bound by what a CTA's warps issue between the products, not by the products
// or by HBM: a chunk takes about 8700 cycles, of which [K;Q] K^T, T, kt and
// the tiles for the products are the longest way, and the SM's tensor pipe is
// busy for a third and its issue slots for half of them.  The roles' code
// together (81 KB) does not fit the instruction cache, so that its size shows
// in every figure (a full batch of 16 prompts x 32 heads of 4096 tokens, with
// two terms throughout: 125 KB 1684 us, 92 KB 1294 us, 83 KB 1205 us, 76 KB
// 1050 us): loops stay rolled where the registers allow it, and f32 work is
// packed in pairs.  4096 tokens of 32 heads 289 us (15 us of HBM time; 268 us
// with two terms), the full batch 1152 us (243 us; 1050 us).
#include "serving_device.cuh"
#include "treewy_device.cuh"
#include "treewy_internal.h"

namespace treewy {
namespace {

constexpr int kC = 64;                       // tokens per chunk
constexpr int kStateWarps = 8, kPrepWarps = 8, kOutWarps = 4;
constexpr int kPrepWarp = kStateWarps, kOutWarp = kPrepWarp + kPrepWarps, kMmaWarp = kOutWarp + kOutWarps,
              kLoadWarp = kMmaWarp + 1, kGateWarp = kLoadWarp + 1, kWarps = kGateWarp + 2;
constexpr int kPrepThreads = 32 * kPrepWarps;
constexpr int kThreads = 32 * kWarps;
// Registers per thread: kLaunchRegs at launch (six warps share the 512 x 32 of
// a quarter of the SM); the state and output warps take what the others give
// back.  An increase waits for registers of the launch, so the shares must not
// add up to more than it has: launch() holds the compiled kernel to it.
constexpr int kLaunchRegs = 80, kStateRegs = 112, kPrepRegs = 64, kOutRegs = 96, kMiscRegs = 32;
static_assert(2 * kStateRegs + 2 * kPrepRegs + kOutRegs + kMiscRegs <= 6 * kLaunchRegs, "the launch's registers");

// TMEM columns
constexpr uint32_t kColS = 0;                // S: hi in 64 columns, lo in 64 (bf16 pairs)
constexpr uint32_t kColW = 128;              // W (16 columns per 16 tokens: hi 8, lo 8)
constexpr uint32_t kColO = 192;              // S q, then MT (lanes 64-127), then MT W
constexpr uint32_t kColD = 256;              // S k in the first 64, then sum W kt^T
constexpr uint32_t kColG = 384;              // [K;Q] K^T
constexpr uint32_t kColK = 448;              // kt^T
constexpr uint32_t kTmemCols = 512;

// Shared memory.  A stage holds K and Q as 64-column boxes of 64 rows in the
// order K0 Q0 K1 Q1 (8 KB each, 128-byte swizzle; so [K;Q] is one operand of
// 128 rows), then V as plain rows.
constexpr uint32_t kBox = 8192;
constexpr uint32_t kStageBytes = 6 * kBox;
constexpr uint32_t kOffKt = 2 * kStageBytes;      // kt^T: 128 rows (dk) of 64 tokens, hi then lo
constexpr uint32_t kOffMT = kOffKt + 4 * kBox;    // MT: 64 rows of 64 tokens, hi then lo
constexpr uint32_t kOffM = kOffMT + 2 * kBox;     // M, hi then lo
constexpr uint32_t kOffT = kOffM + 2 * kBox;      // T hi, lo, then T'' = diag(g_C/g_n) T diag(b) hi, lo
constexpr uint32_t kOffT3 = kOffT + 4 * kBox;     // T's third term; A21's hi in its lower left quarter until T21 is there
constexpr uint32_t kOffA = kOffT3 + kBox;         // A21's lo and third term (rows 32-63), T22 A21's lo (rows 0-31)
constexpr uint32_t kOffX = kOffA + kBox;          // A's, then T's diagonal blocks of 32, f32; then the third term of T''
constexpr int kPitchX = 36;
constexpr uint32_t kOffY = kOffX + kC * kPitchX * 4;  // T22 A21's hi and third term
constexpr uint32_t kSmemBytes = kOffY + kBox / 2 + 1024;
static_assert(kC * kPitchX * 4 >= kBox && kOffY % 1024 == 0, "a tile in the place of the diagonal blocks");

struct __align__(16) Gates {
  float a[kC], b[kC], g[kC];          // decay, write strength and the product of the decays up to every token
  float dec[kC];                      // g_C / g_n: the product of the decays behind token n
  float mid[kC];                      // product of the decays from token 32 to n (1 for n < 32)
  float mid16[32];                    // product of the decays from token 16 to n (16 <= n < 32)
  float gC;
};

// Barriers count warps (lane 0 arrives for its warp) or commits of products.
struct ChunkSmem {
  Gates gates[2];
  uint64_t full[2], full_v[2], stage_free[2], v_free[2], gates_ready[2], gates_free[2];
  uint64_t fix, gram_done, kt_done, mt_done, kt_ready, mt_ready, s_ready[2], d1_done, qs_done, rhs_ready, qs_read, d2_done[2], o2_done,
      o_read, o_tile, t_ready, drain[3];
  uint64_t deadline;
  uint32_t tmem;
  int fail;
};

// A bounded wait: every wait of the CTA gives up at the same time, a second
// and 100 us per chunk (fifteen times what one takes) after its start.  Kept
// short: the roles' code together outgrows the instruction cache, and its size
// is what a chunk's time has gone down with.
__device__ __forceinline__ bool wait(ChunkSmem& cs, uint64_t* bar, uint32_t parity) {
  while (!mbar_try_wait(bar, parity & 1u)) {
    if (globaltimer_ns() > cs.deadline) {
      cs.fail = 1;
      return false;
    }
  }
  return true;
}

// One arrival for the warp, after everything its threads have done.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0)
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// One lane of a converged warp.  Products are issued by the lane that this
// elects: the compiler knows that branch to be taken by one lane and keeps the
// descriptors in uniform registers (a 128 x 64 x 16 product every 37 cycles,
// against 56 from a branch on the lane number and 76 under a predicate).
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// D(tmem) (+)= A(tmem, bf16 pairs) * B(smem desc)^T
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int N>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Descriptor of an operand whose rows run along the contraction (MN-major),
// 128-byte swizzle: blocks of 64 columns `lbo` bytes apart, groups of eight
// rows 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t saddr, uint32_t lbo) {
  uint64_t d = smem_desc_sw128(saddr, 1024);
  d &= ~(static_cast<uint64_t>(0x3FFFu) << 16);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  return d;
}
constexpr uint32_t kAmajorMN = 1u << 15, kBmajorMN = 1u << 16;

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// As tmem_wait16 for one array of eight.
__device__ __forceinline__ void tmem_wait8(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}

// x = hi + lo in bf16 terms, as split_pair, two elements per instruction.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const float2 d = fma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), make_float2(-1.f, -1.f),
                        make_float2(x0, x1));
  const __nv_bfloat162 l = __floats2bfloat162_rn(d.x, d.y);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// x = hi + lo + third, to 2^-26 of x.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t& hi, uint32_t& lo, uint32_t& third) {
  const float2 minus = make_float2(-1.f, -1.f);
  const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const float2 d = fma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), minus, make_float2(x0, x1));
  const __nv_bfloat162 l = __floats2bfloat162_rn(d.x, d.y);
  lo = *reinterpret_cast<const uint32_t*>(&l);
  const float2 e = fma2(make_float2(__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u)), minus, d);
  const __nv_bfloat162 t = __floats2bfloat162_rn(e.x, e.y);
  third = *reinterpret_cast<const uint32_t*>(&t);
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Row `row`, 16-byte piece `j` of a K-major operand with 128-byte rows.
__device__ __forceinline__ uint4* operand_piece(unsigned char* tile, int row, int j) {
  return reinterpret_cast<uint4*>(tile + row * 128 + ((j ^ (row & 7)) << 4));
}

__device__ __forceinline__ void prep_sync() { named_bar_sync<1, kPrepThreads>(); }
// The same, and whether a wait of any preparation thread has given up: all of
// them leave together, so that none is left at a barrier.
__device__ __forceinline__ bool prep_failed(bool ok) { return named_bar_or<1, kPrepThreads>(!ok); }

// acc = sum over N of left (a row L) times right (rows of R, V columns from
// there), N a multiple of 4; all f32 in shared memory.
template <int N, int V>
__device__ __forceinline__ void dot_rows(const float* L, const float* R, float (&acc)[V]) {
  float2 sum[V / 2];
#pragma unroll
  for (int e = 0; e < V / 2; ++e) sum[e] = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int i = 0; i < N; i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(L + i);
    const float ls[4] = {l.x, l.y, l.z, l.w};
    float4 y[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
      y[k] = *reinterpret_cast<const float4*>(R + (i + k / (V / 4)) * kPitchX + 4 * (k % (V / 4)));
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int e = 2 * (k % (V / 4));
      const float2 f = make_float2(ls[k / (V / 4)], ls[k / (V / 4)]);
      sum[e] = fma2(f, make_float2(y[k].x, y[k].y), sum[e]);
      sum[e + 1] = fma2(f, make_float2(y[k].z, y[k].w), sum[e + 1]);
    }
  }
#pragma unroll
  for (int e = 0; e < V; e += 2) acc[e] = sum[e / 2].x, acc[e + 1] = sum[e / 2].y;
}

// T21 = -T22 (A21 T11) for the block of 2 N at B (A21 and then T21 at row N,
// T22 at row and column N), V columns per lane: row r, from column c.
template <int N, int V>
__device__ __forceinline__ void merge(float* B, int r, int c) {
  float4* out = reinterpret_cast<float4*>(B + (N + r) * kPitchX + c);
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    float t[V];
    dot_rows<N, V>(B + (N + r) * kPitchX + pass * N, B + pass * N * kPitchX + c, t);
    __syncwarp();
#pragma unroll
    for (int e = 0; e < V; e += 4)
      out[e / 4] = pass ? make_float4(-t[e], -t[e + 1], -t[e + 2], -t[e + 3])
                        : make_float4(t[e], t[e + 1], t[e + 2], t[e + 3]);
    __syncwarp();
  }
}

// The diagonal block of 32 at X (unit lower triangular, zeros above) becomes
// its inverse, by one warp: blocks of 8 by substitution, a column per lane;
// then of 16 and of 32 by T21 = -T22 (A21 T11).
__device__ __forceinline__ void solve32(float* X, int lane) {
  {
    const int j = lane & 7;
    float* B = X + 8 * (lane >> 3) * (kPitchX + 1);
    float x[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) x[n] = n == j ? 1.f : 0.f;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      float4 a[8];
#pragma unroll
      for (int n = i + 1; n < 8; ++n) a[n] = *reinterpret_cast<const float4*>(B + n * kPitchX + i);
#pragma unroll
      for (int n = i + 1; n < 8; ++n) {
        x[n] = fmaf(-a[n].x, x[i], x[n]);
        if (n > i + 1) x[n] = fmaf(-a[n].y, x[i + 1], x[n]);
        if (n > i + 2) x[n] = fmaf(-a[n].z, x[i + 2], x[n]);
        if (n > i + 3) x[n] = fmaf(-a[n].w, x[i + 3], x[n]);
      }
    }
    __syncwarp();
#pragma unroll
    for (int n = 0; n < 8; ++n) B[n * kPitchX + j] = x[n];
  }
  __syncwarp();
  merge<8, 4>(X + 16 * (lane >> 4) * (kPitchX + 1), (lane & 15) >> 1, 4 * (lane & 1));
  merge<16, 8>(X, lane >> 1, 8 * (lane & 1));
}

__device__ __forceinline__ void put_piece(unsigned char* hi, int row, int j, const float (&x)[8]) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) split2(x[2 * e], x[2 * e + 1], h[e], l[e]);
  uint4* out = operand_piece(hi, row, j);
  out[0] = make_uint4(h[0], h[1], h[2], h[3]);
  out[kBox / 16] = make_uint4(l[0], l[1], l[2], l[3]);
}

// The same, and the third term.
__device__ __forceinline__ uint4 put_piece3(unsigned char* hi, int row, int j, const float (&x)[8]) {
  uint32_t h[4], l[4], t[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) split3(x[2 * e], x[2 * e + 1], h[e], l[e], t[e]);
  uint4* out = operand_piece(hi, row, j);
  out[0] = make_uint4(h[0], h[1], h[2], h[3]);
  out[kBox / 16] = make_uint4(l[0], l[1], l[2], l[3]);
  return make_uint4(t[0], t[1], t[2], t[3]);
}

// A 16 x 8 result tile of warp-level products whose operands are three terms
// each, products below 2^-25 of the largest left out; three accumulators of
// two products each, so that they need not all wait for one another.
struct Left {
  uint32_t hi[4], lo[4], third[4];
};
struct Right {
  uint32_t hl[4], third[2];  // hi in hl[0..1], lo in hl[2..3]
};
struct Tile {
  float x[4], y[4], z[4];
  __device__ __forceinline__ Tile() {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = y[e] = z[e] = 0.f;
  }
  __device__ __forceinline__ void add(const Left& a, const Right& b) {
    mma16816_bf16_nv(z, a.third[0], a.third[1], a.third[2], a.third[3], b.hl[0], b.hl[1]);
    mma16816_bf16_nv(y, a.lo[0], a.lo[1], a.lo[2], a.lo[3], b.hl[0], b.hl[1]);
    mma16816_bf16_nv(x, a.hi[0], a.hi[1], a.hi[2], a.hi[3], b.hl[0], b.hl[1]);
    mma16816_bf16_nv(z, a.hi[0], a.hi[1], a.hi[2], a.hi[3], b.third[0], b.third[1]);
    mma16816_bf16_nv(y, a.hi[0], a.hi[1], a.hi[2], a.hi[3], b.hl[2], b.hl[3]);
    mma16816_bf16_nv(x, a.lo[0], a.lo[1], a.lo[2], a.lo[3], b.hl[2], b.hl[3]);
  }
  __device__ __forceinline__ float at(int e) const { return x[e] + (y[e] + z[e]); }
};
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(p)));
}
__device__ __forceinline__ void ldsm_x2_trans(uint32_t (&r)[2], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];\n"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(smem_addr(p)));
}
// The 16 x 16 block at (row, col) of an operand's tiles as a left operand, the
// third term's from column col3 of its tile.
__device__ __forceinline__ Left left_frag(const unsigned char* hi, const unsigned char* lo, const unsigned char* third,
                                          int row, int col, int col3, int lane) {
  const uint32_t at = sw128_off(row + (lane & 15), col + 8 * (lane >> 4));
  Left f;
  ldsm_x4(f.hi, hi + at);
  ldsm_x4(f.lo, lo + at);
  ldsm_x4(f.third, third + sw128_off(row + (lane & 15), col3 + 8 * (lane >> 4)));
  return f;
}
// 16 rows (the contraction) and 8 columns as a right operand; lo is a tile
// behind hi.
__device__ __forceinline__ Right right_frag(const unsigned char* hi, const unsigned char* third, int row, int col,
                                            int col3, int lane) {
  Right f;
  ldsm_x4_trans(f.hl, hi + (lane >> 4) * kBox + sw128_off(row + (lane & 15), col));
  ldsm_x2_trans(f.third, third + sw128_off(row + (lane & 15), col3));
  return f;
}

// The operands T and T'' = diag(g_C/g_n) T diag(b) from T's diagonal blocks of
// 32 (in X) and A21: the lower left quarter T21 = -(T22 A21) T11 by warp-level
// MMAs, a tile of 16 x 8 per warp.  (These take turns with the tcgen05
// products; on FMAs the two products took 4500 cycles against 1500 with two
// terms.)  The upper right quarter stays zero in the tiles.
__device__ __forceinline__ void solve64(unsigned char* base, const Gates& g, int p) {
  float* X = reinterpret_cast<float*>(base + kOffX);
  unsigned char *tb = base + kOffT, *t3 = base + kOffT3, *ab = base + kOffA, *u3 = base + kOffX, *yb = base + kOffY;
  {
    // the diagonal blocks: eight values per thread
    const int r = p >> 2, c = 8 * (p & 3), col = (r & 32) + c;
    const float dec = g.dec[r];
    const float4 u = *reinterpret_cast<const float4*>(X + r * kPitchX + c);
    const float4 v = *reinterpret_cast<const float4*>(X + r * kPitchX + c + 4);
    const float4 b0 = *reinterpret_cast<const float4*>(g.b + col), b1 = *reinterpret_cast<const float4*>(g.b + col + 4);
    const float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    const float bs[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 z = mul2(mul2(make_float2(dec, dec), make_float2(bs[e], bs[e + 1])), make_float2(x[e], x[e + 1]));
      y[e] = z.x, y[e + 1] = z.y;
    }
    *operand_piece(t3, r, col / 8) = put_piece3(tb, r, col / 8, x);
    const uint4 late = put_piece3(tb + 2 * kBox, r, col / 8, y);
    prep_sync();
    // X has been read: the third term of T'' takes its place
    *operand_piece(u3, r, col / 8) = late;
    if (r < 32) *operand_piece(u3, r, 4 + (p & 3)) = make_uint4(0u, 0u, 0u, 0u);
  }
  // T22 and T11 are lower triangular: only blocks k <= m of the one, k >= t/2
  // of the other
  const int lane = p & 31, m = (p >> 5) & 1, t = p >> 6;
  const int at = lane >> 2, c = 8 * t + 2 * (lane & 3);
  {
    Tile d;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k > m) continue;
      d.add(left_frag(tb, tb + kBox, t3, 32 + 16 * m, 32 + 16 * k, 32 + 16 * k, lane),
            right_frag(t3, ab, 32 + 16 * k, 8 * t, 32 + 8 * t, lane));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t h, l, h3;
      split3(d.at(2 * e), d.at(2 * e + 1), h, l, h3);
      const uint32_t to = sw128_off(16 * m + 8 * e + at, c);
      *reinterpret_cast<uint32_t*>(yb + to) = h;
      *reinterpret_cast<uint32_t*>(ab + to) = l;
      *reinterpret_cast<uint32_t*>(yb + sw128_off(16 * m + 8 * e + at, 32 + c)) = h3;
    }
  }
  prep_sync();
  {
    const float2 b = *reinterpret_cast<const float2*>(g.b + c);
    const float dec[2] = {-g.dec[32 + 16 * m + at], -g.dec[40 + 16 * m + at]};
    Tile d;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k < (t >> 1)) continue;
      d.add(left_frag(yb, ab, yb, 16 * m, 16 * k, 32 + 16 * k, lane), right_frag(tb, t3, 16 * k, 8 * t, 8 * t, lane));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float x = d.at(2 * e), y = d.at(2 * e + 1);
      uint32_t h, l, h3, h2, l2, h23;
      split3(-x, -y, h, l, h3);
      split3(dec[e] * b.x * x, dec[e] * b.y * y, h2, l2, h23);
      const uint32_t to = sw128_off(32 + 16 * m + 8 * e + at, c);
      unsigned char* out = tb + to;
      *reinterpret_cast<uint32_t*>(out) = h;
      *reinterpret_cast<uint32_t*>(out + kBox) = l;
      *reinterpret_cast<uint32_t*>(out + 2 * kBox) = h2;
      *reinterpret_cast<uint32_t*>(out + 3 * kBox) = l2;
      *reinterpret_cast<uint32_t*>(t3 + to) = h3;
      *reinterpret_cast<uint32_t*>(u3 + to) = h23;
    }
  }
}

struct SeqInfo {
  int64_t tok0;
  int len, slot;
  bool fresh;
};

// 64 columns of a row of S (from column 64 half) of the pool.
template <bool SB>
__device__ __forceinline__ void load_state(const treewy_seqs& a, int64_t row, int half, float (&S)[64]) {
#pragma unroll
  for (int i = 0; i < 64; i += 8) {
    const int c = 64 * half + i;
#pragma unroll
    for (int e = 0; e < 8; ++e) S[i + e] = 0.f;
    if (c < a.dk) {
      if constexpr (SB) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.state) + row * a.dk + c);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          S[i + 2 * e] = __uint_as_float(w[e] << 16);
          S[i + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
      } else {
        const float* p = reinterpret_cast<const float*>(a.state) + row * a.dk + c;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 f = *reinterpret_cast<const float4*>(p + e);
          S[i + e] = f.x;
          S[i + e + 1] = f.y;
          S[i + e + 2] = f.z;
          S[i + e + 3] = f.w;
        }
      }
    }
  }
}

template <bool SB>
__device__ __forceinline__ void store_state(const treewy_seqs& a, int64_t row, int half, const float (&S)[64]) {
#pragma unroll
  for (int i = 0; i < 64; i += 8) {
    const int c = 64 * half + i;
    if (c < a.dk) {
      if constexpr (SB) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(S[i + 2 * e], S[i + 2 * e + 1]);
          w[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.state) + row * a.dk + c) =
            make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        float* p = reinterpret_cast<float*>(a.state) + row * a.dk + c;
        *reinterpret_cast<float4*>(p) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(S[i + 4], S[i + 5], S[i + 6], S[i + 7]);
      }
    }
  }
}

// Columns 16 b .. 16 b + 15 of this thread's half of S as the left operand.
__device__ __forceinline__ void put_state16(uint32_t tm, int half, int b, const float (&S)[64]) {
  uint32_t hi[8], lo[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) split2(S[16 * b + 2 * e], S[16 * b + 2 * e + 1], hi[e], lo[e]);
  tmem_st8(tm + kColS + 32 * half + 8 * b, hi);
  tmem_st8(tm + kColS + 64 + 32 * half + 8 * b, lo);
}

// The state warps.
template <bool SB>
__device__ __forceinline__ void run_state(const treewy_seqs& a, ChunkSmem& cs, unsigned char* base, const SeqInfo& q,
                                          int h, int nchunk) {
  const int t = threadIdx.x, d = t & 127, half = t >> 7;
  const uint32_t tm = cs.tmem + (static_cast<uint32_t>(d & 96) << 16);
  const int64_t row = (static_cast<int64_t>(q.slot) * a.H + h) * a.dv + d;
  float S[64];
  if (d < a.dv && !q.fresh) {
    load_state<SB>(a, row, half, S);
  } else {
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0.f;
  }
  bool ok = true;
  const int n0 = 32 * half;
  for (int c = 0; c < nchunk; ++c) {
    // the state as the left operand of S k and S q
#pragma unroll
    for (int b = 0; b < 4; ++b) put_state16(tm, half, b, S);
    tmem_wait_st();
    tc_fence_before_sync();
    warp_arrive(&cs.s_ready[half]);
    const int sg = c & 1;
    const uint32_t ph2 = c >> 1;
    const Gates& g = cs.gates[sg];
    const int left = q.len - c * kC - n0;  // tokens of this thread's half
    ok = wait(cs, &cs.full_v[sg], ph2) && wait(cs, &cs.gates_ready[sg], ph2) && wait(cs, &cs.d1_done, c);
    if (!__all_sync(0xffffffffu, ok)) break;
    tc_fence_after_sync();
    {
      // W = v - g (S k), with v zero past the sequence's end (each thread reads,
      // and clears, only its own column of its half's rows)
      unsigned char* vt = base + sg * kStageBytes + 4 * kBox + n0 * 256 + 2 * d;
      for (int n = max(left, 0); n < 32; ++n) *reinterpret_cast<uint16_t*>(vt + n * 256) = 0;
#pragma unroll 1
      for (int b = 0; b < 2; ++b, vt += 16 * 256) {
        uint32_t x[16], hi[8], lo[8];
        tmem_ld16_async(tm + kColD + n0 + 16 * b, x);
        tmem_wait16(x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 f = *reinterpret_cast<const float4*>(g.g + n0 + 16 * b + 4 * j);
          const float fs[4] = {f.x, f.y, f.z, f.w};
          float v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(vt + (4 * j + k) * 256));
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const float2 w = fma2(make_float2(-fs[k], -fs[k + 1]),
                                  make_float2(__uint_as_float(x[4 * j + k]), __uint_as_float(x[4 * j + k + 1])),
                                  make_float2(v[k], v[k + 1]));
            split2(w.x, w.y, hi[2 * j + k / 2], lo[2 * j + k / 2]);
          }
        }
        // 16 tokens: hi in 8 columns, lo in 8
        tmem_st8(tm + kColW + n0 + 16 * b, hi);
        tmem_st8(tm + kColW + n0 + 16 * b + 8, lo);
      }
    }
    tmem_wait_st();
    tc_fence_before_sync();
    warp_arrive(&cs.rhs_ready);
    // S' = g_C S + W kt
    const float gC = g.gC;
    ok = wait(cs, &cs.d2_done[half], c);
    if (!__all_sync(0xffffffffu, ok)) break;
    tc_fence_after_sync();
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t x[16];
      tmem_ld16_async(tm + kColD + 64 * half + 16 * b, x);
      tmem_wait16(x);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 y = fma2(make_float2(gC, gC), make_float2(S[16 * b + e], S[16 * b + e + 1]),
                              make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
        S[16 * b + e] = y.x;
        S[16 * b + e + 1] = y.y;
      }
    }
    warp_arrive(&cs.gates_free[sg]);
  }
  if (ok && d < a.dv) store_state<SB>(a, row, half, S);
}

// The output warps: o = g (S q) + MT W, a row of 64 tokens per thread.
template <bool OF32>
__device__ __forceinline__ void run_out(const treewy_seqs& a, ChunkSmem& cs, unsigned char* base, const SeqInfo& q,
                                        int h, int nchunk) {
  const int t = threadIdx.x - 32 * kOutWarp, d = t;
  const uint32_t tm = cs.tmem + (static_cast<uint32_t>(d & 96) << 16);
  const int64_t step = static_cast<int64_t>(a.H) * a.dv;
  for (int c = 0; c < nchunk; ++c) {
    const int sg = c & 1;
    const uint32_t ph2 = c >> 1;
    const Gates& g = cs.gates[sg];
    float o[64];
    bool ok = wait(cs, &cs.gates_ready[sg], ph2) && wait(cs, &cs.qs_done, c);
    if (!__all_sync(0xffffffffu, ok)) break;
    tc_fence_after_sync();
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t x[16];
      tmem_ld16_async(tm + kColO + 16 * b, x);
      tmem_wait16(x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 f = *reinterpret_cast<const float4*>(g.g + 16 * b + 4 * j);
        const float2 y = mul2(make_float2(f.x, f.y), make_float2(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1])));
        const float2 z = mul2(make_float2(f.z, f.w), make_float2(__uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3])));
        o[16 * b + 4 * j] = y.x, o[16 * b + 4 * j + 1] = y.y;
        o[16 * b + 4 * j + 2] = z.x, o[16 * b + 4 * j + 3] = z.y;
      }
    }
    tc_fence_before_sync();
    warp_arrive(&cs.qs_read);
    if (d >= 64) {
      // MT = M T diag(b), in lanes 64-127, as an operand while these warps have
      // nothing else to do; rows 0-31 of it end in column 31
      ok = wait(cs, &cs.mt_done, c);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after_sync();
      unsigned char* mtb = base + kOffMT;
      const int last = d < 96 ? 4 : 8;
#pragma unroll 1
      for (int j = 0; j < last; ++j) {
        const float4 u = *reinterpret_cast<const float4*>(g.b + 8 * j), v = *reinterpret_cast<const float4*>(g.b + 8 * j + 4);
        uint32_t x[8];
        tmem_ld8_async(tm + kColO + 8 * j, x);
        tmem_wait8(x);
        const float bs[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 z = mul2(make_float2(bs[e], bs[e + 1]), make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
          y[e] = z.x, y[e + 1] = z.y;
        }
        put_piece(mtb, d - 64, j, y);
      }
      tc_fence_before_sync();
      fence_proxy_async_smem();
      warp_arrive(&cs.mt_ready);
    }
    warp_arrive(&cs.gates_free[sg]);
    ok = wait(cs, &cs.o2_done, c);
    if (!__all_sync(0xffffffffu, ok)) break;
    tc_fence_after_sync();
    const int rows = min(kC, q.len - c * kC);
    const int64_t at0 = ((q.tok0 + c * kC) * a.H + h) * static_cast<int64_t>(a.dv);
    // bf16: o takes V's place (the state warps have read it: W is made) and
    // leaves from there in pieces of 16 bytes
    unsigned char* tile = base + sg * kStageBytes + 4 * kBox;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t x[16];
      tmem_ld16_async(tm + kColO + 16 * b, x);
      tmem_wait16(x);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const int n = 16 * b + e;
        const float2 y = fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), make_float2(1.f, 1.f),
                              make_float2(o[n], o[n + 1]));
        if constexpr (OF32) {
          float* out = reinterpret_cast<float*>(a.o) + at0 + n * step + d;
          if (n < rows && d < a.dv) out[0] = y.x;
          if (n + 1 < rows && d < a.dv) out[step] = y.y;
        } else {
          const __nv_bfloat162 p = __floats2bfloat162_rn(y.x, y.y);
          *reinterpret_cast<__nv_bfloat16*>(tile + n * 256 + 2 * d) = p.x;
          *reinterpret_cast<__nv_bfloat16*>(tile + (n + 1) * 256 + 2 * d) = p.y;
        }
      }
    }
    tc_fence_before_sync();
    warp_arrive(&cs.o_read);
    if constexpr (!OF32) {
      warp_arrive(&cs.o_tile);
      ok = wait(cs, &cs.o_tile, c);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int piece = t & 15;
      if (8 * piece < a.dv) {
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.o) + at0 + 8 * piece;
#pragma unroll 2
        for (int n = t >> 4; n < rows; n += 8)
          *reinterpret_cast<uint4*>(out + n * step) = *reinterpret_cast<const uint4*>(tile + n * 256 + 16 * piece);
      }
      fence_proxy_async_smem();
    }
    warp_arrive(&cs.v_free[sg]);
  }
}

// One warp: the gates of every chunk.
__device__ __forceinline__ void run_gates(const treewy_seqs& a, ChunkSmem& cs, const SeqInfo& q, int h, int nchunk) {
  const int lane = threadIdx.x & 31;
  float na[2] = {1.f, 1.f}, nb[2] = {0.f, 0.f};
  // one turn ahead: turn c works on what turn c - 1 has requested
#pragma unroll 1
  for (int c = -1; c < nchunk; ++c) {
    const float al[2] = {na[0], na[1]}, be[2] = {nb[0], nb[1]};
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // tokens `lane` and `lane + 32`; past the end they change nothing
      const int i = (c + 1) * kC + lane + 32 * k;
      na[k] = 1.f;
      nb[k] = 0.f;
      if (i < q.len) {
        na[k] = __ldg(a.alpha + (q.tok0 + i) * a.H + h);
        nb[k] = __ldg(a.beta + (q.tok0 + i) * a.H + h);
      }
    }
    if (c < 0) continue;
    const int sg = c & 1;
    // products of the decays up to and behind every token, by doubling
    float up[2] = {al[0], al[1]}, down[2] = {al[0], al[1]};
#pragma unroll 1
    for (int s = 1; s < 32; s <<= 1) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float y = __shfl_up_sync(0xffffffffu, up[k], s), z = __shfl_down_sync(0xffffffffu, down[k], s);
        if (lane >= s) up[k] *= y;
        if (lane + s < 32) down[k] *= z;
      }
    }
    const float mid = up[1];
    // within tokens 16-31: by doubling over 16 lanes
    float mid16 = al[0];
#pragma unroll 1
    for (int s = 1; s < 16; s <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, mid16, s, 16);
      if ((lane & 15) >= s) mid16 *= y;
    }
    up[1] *= __shfl_sync(0xffffffffu, up[0], 31);
    const float half = __shfl_sync(0xffffffffu, down[1], 0);
    const float next0 = __shfl_down_sync(0xffffffffu, down[0], 1), next1 = __shfl_down_sync(0xffffffffu, down[1], 1);
    const float dec[2] = {lane < 31 ? next0 * half : half, lane < 31 ? next1 : 1.f};
    const bool ok = c < 2 || wait(cs, &cs.gates_free[sg], (c >> 1) - 1);
    if (!__all_sync(0xffffffffu, ok)) break;
    Gates& g = cs.gates[sg];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = lane + 32 * k;
      g.a[i] = al[k];
      g.b[i] = be[k];
      g.g[i] = up[k];
      g.dec[i] = dec[k];
      g.mid[i] = k ? mid : 1.f;
    }
    g.mid16[lane] = mid16;
    if (lane == 31) g.gC = up[1];
    warp_arrive(&cs.gates_ready[sg]);
  }
}

// [K;Q] K^T of chunk c (one elected lane).
__device__ __forceinline__ void issue_gram(ChunkSmem& cs, unsigned char* base, int c) {
  constexpr uint32_t id = idesc_bf16_f32(128, kC);
  const uint64_t s0 = smem_desc_sw128(smem_addr(base + (c & 1) * kStageBytes), 1024);
  uint64_t at = s0;
#pragma unroll 2
  for (int k = 0; k < 8; ++k) {
    mma_bf16(cs.tmem + kColG, at, at, id, k > 0);
    at += k == 3 ? (2 * kBox - 96) >> 4 : 2;
  }
  mma_commit(&cs.gram_done);
}

// One warp: the preparation's other products, once T and the next chunk's K
// and Q are there.
template <bool OF32>
__device__ __forceinline__ void run_issue(ChunkSmem& cs, unsigned char* base, int nchunk) {
  constexpr uint32_t idk = idesc_bf16_f32(128, kC) | kAmajorMN | kBmajorMN;
  constexpr uint32_t idm = idesc_bf16_f32(128, kC) | kBmajorMN;
  const uint64_t t1 = smem_desc_sw128_mn(smem_addr(base + kOffT), kBox), t2 = t1 + ((2 * kBox) >> 4);
  const uint64_t m0 = smem_desc_sw128(smem_addr(base + kOffM - kBox), 1024);
  for (int c = 0; c < nchunk; ++c) {
    const uint64_t k0 = smem_desc_sw128_mn(smem_addr(base + (c & 1) * kStageBytes), 2 * kBox);
    const bool ok = wait(cs, &cs.t_ready, c);
    if (!__all_sync(0xffffffffu, ok)) return;
    if (elect_one()) {
      tc_fence_after_sync();
      // kt^T[dk][i] = sum_n K[n][dk] T''[n][i]
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        mma_bf16(cs.tmem + kColK, k0 + k * 128, t2 + k * 128, idk, k > 0);
        mma_bf16(cs.tmem + kColK, k0 + k * 128, t2 + (kBox >> 4) + k * 128, idk, 1u);
        mma_bf16(cs.tmem + kColK, k0 + k * 128, t1 + ((kOffX - kOffT) >> 4) + k * 128, idk, 1u);
      }
      mma_commit(&cs.kt_done);
      mma_commit(&cs.stage_free[c & 1]);
      if (c + 1 < nchunk) issue_gram(cs, base, c + 1);
    }
    __syncwarp();
    // MT takes the place of the chunk's S q for a while
    const bool free = wait(cs, &cs.qs_read, c);
    if (!__all_sync(0xffffffffu, free)) return;
    if (elect_one()) {
      tc_fence_after_sync();
      // M T in lanes 64-127: rows 64.. of the left operand are M's (hi, then
      // lo), the tile before them fills lanes that nothing reads
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const uint64_t mh = m0 + 2 * k, ml = mh + (kBox >> 4), th = t1 + 128 * k, tl = th + (kBox >> 4);
        mma_bf16(cs.tmem + kColO, mh, th, idm, k > 0);
        mma_bf16(cs.tmem + kColO, mh, tl, idm, 1u);
        mma_bf16(cs.tmem + kColO, ml, th, idm, 1u);
        if constexpr (OF32) {
          mma_bf16(cs.tmem + kColO, ml, tl, idm, 1u);
          mma_bf16(cs.tmem + kColO, mh, th + ((kOffT3 - kOffT) >> 4), idm, 1u);
        }
      }
      mma_commit(&cs.mt_done);
    }
    __syncwarp();
  }
}

// Columns 16 b .. of the 32 from 32 cb, for b from b1 - 1 down to b0, of row n
// of A or M from [K;Q] K^T: entry i times the
// decays between i and n (and b_n for A), from the diagonal (or column
// 32 cb + 31) leftwards; zero right of the diagonal.  A's diagonal blocks go to
// `row` in f32 (their diagonal is never read), the others to a tile.
__device__ __forceinline__ void form_row(uint32_t tm_row, const Gates& g, bool isM, int n, int cb, int b0, int b1,
                                         unsigned char* tile, float* out_row) {
  const float f0 = isM ? 1.f : g.b[n];
  const int dl = n - 32 * cb;
  float f = dl > 31 ? f0 * g.mid[n] : 0.f;
  if (b1 == 1) f = dl > 15 ? f0 * g.mid16[n] : 0.f;
#pragma unroll 1
  for (int b = b1 - 1; b >= b0; --b) {
    const int db = dl - 16 * b;
    float as[16], y[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 u = *reinterpret_cast<const float4*>(g.a + 32 * cb + 16 * b + 4 * j);
      as[4 * j] = u.x, as[4 * j + 1] = u.y, as[4 * j + 2] = u.z, as[4 * j + 3] = u.w;
    }
    uint32_t x[16];
    tmem_ld16_async(tm_row + kColG + 32 * cb + 16 * b, x);
    tmem_wait16(x);
#pragma unroll
    for (int k = 15; k >= 0; --k) {
      if (k == db) f = f0;
      y[k] = k <= db ? f * __uint_as_float(x[k]) : 0.f;
      f *= as[k];
    }
    if (out_row == nullptr) {
      uint32_t h[8], l[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) split2(y[2 * k], y[2 * k + 1], h[k], l[k]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint4* out = operand_piece(tile, n, 4 * cb + 2 * b + j);
        out[0] = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
        out[kBox / 16] = make_uint4(l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]);
      }
      if (!isM) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t t[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t hh, ll;
            split3(y[8 * j + 2 * k], y[8 * j + 2 * k + 1], hh, ll, t[k]);
          }
          *operand_piece(tile + kBox, n, 4 + 2 * b + j) = make_uint4(t[0], t[1], t[2], t[3]);
        }
      }
    } else {
      float4* r = reinterpret_cast<float4*>(out_row + 16 * b);
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
    }
  }
}

// Columns 16 b .. of a row of kt^T as operands, for b from b0 to b1 - 1.
__device__ __forceinline__ void put_kt(uint32_t tm_row, unsigned char* ktb, int row, int b0, int b1) {
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    uint32_t x[16], h[8], l[8];
    tmem_ld16_async(tm_row + kColK + 16 * b, x);
    tmem_wait16(x);
#pragma unroll
    for (int k = 0; k < 8; ++k) split2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]), h[k], l[k]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint4* out = operand_piece(ktb, row, 2 * b + j);
      out[0] = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
      out[2 * kBox / 16] = make_uint4(l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]);
    }
  }
}

// The preparation warps: M, T and kt of every chunk, one chunk ahead of the
// state, and [K;Q] K^T one more chunk ahead.  The way from a chunk's
// [K;Q] K^T to its T is the longest, so two warps (0 and 5, whose TMEM lanes
// hold the rows of A's diagonal blocks of 32) do nothing else, and the others
// finish the chunk before and form the rest of A and M beside them:
//
//   0, 5          A's diagonal blocks of chunk c, then T's
//   1             kt of c - 1 (64 columns); A21 of c
//   4             kt of c - 1 (64 columns)
//   2, 3, 6, 7    kt of c - 1 (32 columns each); M of c (2, 6: rows 0-31, 16 columns
//                 each; 3, 7: rows 32-63, 32 columns each)
//
// then all of them T21 of c, and [K;Q] K^T of c + 1, kt^T and MT of c are
// issued.  kt is what the chain waits for, so it comes first.
__device__ __forceinline__ void run_prep(ChunkSmem& cs, unsigned char* base, int len, int nchunk) {
  const int p = threadIdx.x - 32 * kPrepWarp, lane = p & 31, w = p >> 5;
  const int quad = w & 3, row = 32 * quad + lane, n = row & 63;
  const uint32_t tm = cs.tmem + (static_cast<uint32_t>(32 * quad) << 16);
  const bool solver = w == 0 || w == 5;
  float* X = reinterpret_cast<float*>(base + kOffX);
  unsigned char *ktb = base + kOffKt, *mtb = base + kOffMT, *mb = base + kOffM;
  // the upper right quarters of MT, M, T, T'' and T's third term stay zero
  for (int i = 16 * p; i < static_cast<int>(9 * kBox); i += 16 * kPrepThreads)
    *reinterpret_cast<uint4*>(mtb + i) = make_uint4(0u, 0u, 0u, 0u);
  // K and Q of chunk c are there; rows of K past the sequence's end (the next
  // one's) become zero
  auto stage_in = [&](int c) {
    const bool there = wait(cs, &cs.full[c & 1], c >> 1);
    __syncwarp();
    const int nt = len - c * kC;
    if (nt < kC) {
      unsigned char* st = base + (c & 1) * kStageBytes;
      for (int i = nt * 128 + 16 * p; i < static_cast<int>(kBox); i += 16 * kPrepThreads) {
        *reinterpret_cast<uint4*>(st + i) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(st + 2 * kBox + i) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      warp_arrive(&cs.fix);
    }
    return there;
  };
  bool ok = stage_in(0);
  if (prep_failed(ok)) return;
  if (w == 0 && elect_one()) {
    tc_fence_after_sync();
    issue_gram(cs, base, 0);
  }
  __syncwarp();
  for (int c = 0; c <= nchunk; ++c) {
    const bool cur = c < nchunk;
    const Gates& g = cs.gates[c & 1];
    if (!solver && c > 0) {
      // the operands of c - 2 have been read, the products of c - 1 are done
      if (c > 1 && !wait(cs, &cs.o2_done, c - 2)) ok = false;
      if (!wait(cs, &cs.kt_done, c - 1)) ok = false;
      __syncwarp();
      tc_fence_after_sync();
      const int b0 = w == 6 || w == 7 ? 2 : 0, b1 = w == 2 || w == 3 ? 2 : 4;
      put_kt(tm, ktb, row, b0, b1);
      tc_fence_before_sync();
      fence_proxy_async_smem();
      warp_arrive(&cs.kt_ready);
      // M and T of c - 1 have been read
      if (!wait(cs, &cs.mt_done, c - 1)) ok = false;
    }
    if (c > 0) warp_arrive(&cs.gates_free[(c - 1) & 1]);
    if (!cur) break;
    if (!wait(cs, &cs.gates_ready[c & 1], c >> 1) || !wait(cs, &cs.gram_done, c)) ok = false;
    __syncwarp();
    tc_fence_after_sync();
    // rows 0-31 of M end in column 31: 16 columns each for warps 2 and 6
    if (w != 4)
      form_row(tm, g, quad >= 2, n, w == 5 || w == 7, w == 2, w == 6 ? 1 : 2, quad >= 2 ? mb : base + kOffT3,
               solver ? X + n * kPitchX : nullptr);
    tc_fence_before_sync();
    if (solver) {
      __syncwarp();
      solve32(X + (w == 5 ? 32 * kPitchX : 0), lane);
    }
    if (c + 1 < nchunk && !stage_in(c + 1)) ok = false;
    if (prep_failed(ok)) break;
    solve64(base, g, p);
    fence_proxy_async_smem();
    warp_arrive(&cs.t_ready);
    prep_sync();  // X is written again once the next [K;Q] K^T is there, and so kt of this chunk
  }
}

// The products that this warp has issued are done (or the limit is over)
// before the CTA frees its TMEM, also after a wait that gave up.
__device__ __forceinline__ void drain(uint64_t* bar) {
  __syncwarp();
  if (elect_one()) mma_commit(bar);
  mbar_wait(bar, 0);
  __syncwarp();
}

// One warp: the chain's products.
__device__ __forceinline__ void run_mma(ChunkSmem& cs, unsigned char* base, int len, int nchunk) {
  constexpr uint32_t id = idesc_bf16_f32(128, kC);
  const uint32_t tm = cs.tmem;
  const uint64_t kt = smem_desc_sw128(smem_addr(base + kOffKt), 1024);
  const uint64_t mt = smem_desc_sw128(smem_addr(base + kOffMT), 1024);
  auto held = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = wait(cs, bar, parity);
    return __all_sync(0xffffffffu, ok) != 0;
  };
  for (int c = 0; c < nchunk; ++c) {
    const int sg = c & 1;
    const uint64_t s0 = smem_desc_sw128(smem_addr(base + sg * kStageBytes), 1024);
    if (!held(&cs.full[sg], c >> 1)) return;
    if (len - c * kC < kC && !held(&cs.fix, 0)) return;
    // S k in the columns of W kt, half of the columns of S at a time
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      if (!held(&cs.s_ready[half], c)) return;
      if (elect_one()) {
      tc_fence_after_sync();
#pragma unroll 2
      for (int k = 0; k < 4; ++k) {
        const uint64_t kd = s0 + ((half * 2 * kBox + 32 * k) >> 4);
        mma_ts(tm + kColD, tm + kColS + 32 * half + 8 * k, kd, id, half > 0 || k > 0);
        mma_ts(tm + kColD, tm + kColS + 64 + 32 * half + 8 * k, kd, id, 1u);
      }
      }
      __syncwarp();
    }
    // the columns of W may be written again
    if (c > 0 && !held(&cs.o2_done, c - 1)) return;
    if (elect_one()) mma_commit(&cs.d1_done);
    __syncwarp();
    // S q
    if (c > 0 && !held(&cs.o_read, c - 1)) return;
    if (elect_one()) {
    tc_fence_after_sync();
    uint64_t qd = s0 + (kBox >> 4);
#pragma unroll 1
    for (int k = 0; k < 8; ++k, qd += k == 4 ? (2 * kBox - 96) >> 4 : 2) {
      mma_ts(tm + kColO, tm + kColS + 8 * k, qd, id, k > 0);
      mma_ts(tm + kColO, tm + kColS + 64 + 8 * k, qd, id, 1u);
    }
    mma_commit(&cs.qs_done);
    mma_commit(&cs.stage_free[sg]);
    }
    __syncwarp();
    // W kt, half of its columns at a time
    if (!held(&cs.kt_ready, c) || !held(&cs.rhs_ready, c)) return;
    if (elect_one()) {
    tc_fence_after_sync();
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const uint32_t wh = tm + kColW + 16 * k;
        const uint64_t kh = kt + ((half * kBox + 32 * k) >> 4), kl = kh + ((2 * kBox) >> 4);
        mma_ts(tm + kColD + 64 * half, wh, kh, id, k > 0);
        mma_ts(tm + kColD + 64 * half, wh, kl, id, 1u);
        mma_ts(tm + kColD + 64 * half, wh + 8, kh, id, 1u);
      }
      mma_commit(&cs.d2_done[half]);
    }
    }
    __syncwarp();
    // MT W over the columns of S q
    if (!held(&cs.mt_ready, c)) return;
    if (elect_one()) {
    tc_fence_after_sync();
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const uint32_t wh = tm + kColW + 16 * k;
      const uint64_t mh = mt + 2 * k, ml = mh + (kBox >> 4);
      mma_ts(tm + kColO, wh, mh, id, k > 0);
      mma_ts(tm + kColO, wh, ml, id, 1u);
      mma_ts(tm + kColO, wh + 8, mh, id, 1u);
    }
    mma_commit(&cs.o2_done);
    }
    __syncwarp();
  }
}

// One thread: K, Q and V of every chunk, two in flight.
__device__ __forceinline__ void run_load(const CUtensorMap* map_q, const CUtensorMap* map_k, const CUtensorMap* map_v,
                                         ChunkSmem& cs, unsigned char* base, const SeqInfo& q, int hk, int h,
                                         int nchunk) {
  int issued = 0, issued_v = 0;
#pragma unroll 1
  for (int c = 0; c < nchunk; ++c) {
    const int sg = c & 1;
    if (c >= 2 && !wait(cs, &cs.stage_free[sg], (c >> 1) - 1)) break;
    unsigned char* st = base + sg * kStageBytes;
    const int tok = static_cast<int>(q.tok0) + c * kC;
    mbar_arrive_expect_tx(&cs.full[sg], 4 * kBox);
    tma_load_3d(st, map_k, &cs.full[sg], 0, hk, tok);
    tma_load_3d(st + 2 * kBox, map_k, &cs.full[sg], 64, hk, tok);
    tma_load_3d(st + kBox, map_q, &cs.full[sg], 0, hk, tok);
    tma_load_3d(st + 3 * kBox, map_q, &cs.full[sg], 64, hk, tok);
    ++issued;
    if (c >= 2 && !wait(cs, &cs.v_free[sg], (c >> 1) - 1)) break;
    mbar_arrive_expect_tx(&cs.full_v[sg], 2 * kBox);
    tma_load_3d(st + 4 * kBox, map_v, &cs.full_v[sg], 0, h, tok);
    ++issued_v;
  }
  // no copy targets this CTA's memory once it has ended
  for (int c = max(0, issued - 2); c < issued; ++c) mbar_wait(&cs.full[c & 1], (c >> 1) & 1);
  for (int c = max(0, issued_v - 2); c < issued_v; ++c) mbar_wait(&cs.full_v[c & 1], (c >> 1) & 1);
}

template <bool SB, bool OF32>
__global__ void __launch_bounds__(kThreads, 1)
    extend_chunk_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const treewy_seqs a) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ ChunkSmem cs;
  // by an offset, so that the compiler still knows the pointer to be a shared one
  unsigned char* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int idx = blockIdx.x / a.H, h = blockIdx.x - idx * a.H, r = longest_first(a, idx);
  const int t = threadIdx.x, warp = t >> 5;

  const int lo = __ldg(a.seq_offset + r), hi = __ldg(a.seq_offset + r + 1);
  SeqInfo q;
  q.slot = __ldg(a.state_slot + r);
  q.fresh = a.fresh != nullptr && __ldg(a.fresh + r) != 0;
  const int64_t len = static_cast<int64_t>(hi) - lo;
  int flags = 0;
  if (len < 0 || len > a.max_len) flags |= TREEWY_STATUS_TOO_MANY_NODES;
  else if (lo < 0 || hi > a.T) flags |= TREEWY_STATUS_BAD_TREE;
  if (q.slot < 0 || q.slot >= a.num_slots) flags |= TREEWY_STATUS_BAD_SLOT;
  q.tok0 = lo;
  q.len = static_cast<int>(len);
  if (flags) {
    if (t == 0 && h == 0) atomicOr(a.status + r, flags);
    return;
  }
  if (q.len == 0) {
    if (q.fresh) {
      const int64_t at = (static_cast<int64_t>(q.slot) * a.H + h) * a.dv * a.dk;
      for (int i = t; i < a.dv * a.dk; i += kThreads) {
        if constexpr (SB) reinterpret_cast<uint16_t*>(a.state)[at + i] = 0;
        else reinterpret_cast<float*>(a.state)[at + i] = 0.f;
      }
    }
    return;
  }
  const int nchunk = (q.len + kC - 1) / kC;

  if (t == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&cs.full[i], 1);
      mbar_init(&cs.full_v[i], 1);
      mbar_init(&cs.stage_free[i], 2);
      mbar_init(&cs.v_free[i], kOutWarps);
      mbar_init(&cs.gates_ready[i], 1);
      mbar_init(&cs.gates_free[i], kStateWarps + kPrepWarps + kOutWarps);
      mbar_init(&cs.s_ready[i], kStateWarps / 2);
      mbar_init(&cs.d2_done[i], 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&cs.drain[i], 1);
    mbar_init(&cs.t_ready, kPrepWarps);
    mbar_init(&cs.fix, kPrepWarps);
    mbar_init(&cs.gram_done, 1);
    mbar_init(&cs.kt_done, 1);
    mbar_init(&cs.mt_done, 1);
    mbar_init(&cs.mt_ready, kOutWarps / 2);
    mbar_init(&cs.kt_ready, kPrepWarps - 2);
    mbar_init(&cs.d1_done, 1);
    mbar_init(&cs.qs_done, 1);
    mbar_init(&cs.rhs_ready, kStateWarps);
    mbar_init(&cs.qs_read, kOutWarps);
    mbar_init(&cs.o2_done, 1);
    mbar_init(&cs.o_read, kOutWarps);
    mbar_init(&cs.o_tile, kOutWarps);
    cs.fail = 0;
    cs.deadline = globaltimer_ns() + kWaitLimitNs + 100000ull * static_cast<uint64_t>(nchunk);
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&cs.tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();

  if (warp < kPrepWarp) {
    set_regs_up<kStateRegs>();
    run_state<SB>(a, cs, base, q, h, nchunk);
  } else if (warp < kOutWarp) {
    set_regs_down<kPrepRegs>();
    run_prep(cs, base, q.len, nchunk);
    if (warp == kPrepWarp) drain(&cs.drain[1]);
  } else if (warp < kMmaWarp) {
    set_regs_up<kOutRegs>();
    run_out<OF32>(a, cs, base, q, h, nchunk);
  } else {
    set_regs_down<kMiscRegs>();
    if (warp == kMmaWarp) {
      run_mma(cs, base, q.len, nchunk);
      drain(&cs.drain[0]);
    } else if (warp == kLoadWarp) {
      if ((t & 31) == 0) run_load(&map_q, &map_k, &map_v, cs, base, q, h / (a.H / a.Hk), h, nchunk);
    } else if (warp == kGateWarp) {
      run_gates(a, cs, q, h, nchunk);
    } else {
      run_issue<OF32>(cs, base, nchunk);
      drain(&cs.drain[2]);
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (t == 0 && cs.fail) atomicOr(a.status + r, TREEWY_STATUS_TIMEOUT);
  if (warp == kMmaWarp) tmem_dealloc(cs.tmem, kTmemCols);
}

template <bool SB, bool OF32>
cudaError_t launch(const treewy_seqs& a, const ExtendMaps& m, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  const cudaError_t attr = once_per_device(attr_done, [] {
    cudaFuncAttributes f;
    const cudaError_t e = cudaFuncGetAttributes(&f, extend_chunk_kernel<SB, OF32>);
    if (e != cudaSuccess) return e;
    if (f.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(extend_chunk_kernel<SB, OF32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSmemBytes));
  });
  if (attr != cudaSuccess) return attr;
  const unsigned grid = static_cast<unsigned>(a.R) * static_cast<unsigned>(a.H);
  extend_chunk_kernel<SB, OF32><<<grid, kThreads, kSmemBytes, stream>>>(m.q, m.k, m.v, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_extend_chunk(const treewy_seqs& a, const ExtendMaps& m, cudaStream_t stream) {
  if (a.flags & TREEWY_FLAG_STATE_BF16)  // with bf16 outputs only
    return a.o_dtype == TREEWY_DTYPE_F32 ? cudaErrorInvalidValue : launch<true, false>(a, m, stream);
  return a.o_dtype == TREEWY_DTYPE_F32 ? launch<false, true>(a, m, stream) : launch<false, false>(a, m, stream);
}

}  // namespace treewy
