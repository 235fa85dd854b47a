// Softmax attention over 8-bit KV rows of the paged cache: for token t, head h
// and the positions J (listed, or causally visible),
//   kv_j = c_j s_j,  z_j = scale q . kv_j,
//   o = sum_j e^(z_j - m) kv_j / sum_j e^(z_j - m),  lse = m + ln sum.
//
// With x_j = z_j log2 e, y_j = x_j + log2 s_j and a running reference M >=
// max y_j - kSlack, the weight p_j = 2^(y_j - M + kShift) carries the row's
// scale, so the value product runs on the codes themselves,
//   o = sum p_j c_j / sum (p_j / s_j),
// and p_j never leaves FP16 whatever the scales are: at most 2^(kSlack +
// kShift) = 2^14, and what falls below 2^-25 is under 2^-31 of the largest.
// Codes of both types are FP16 values; a BF16 query times a power of two per
// head is one too (11 significand bits >= 8). So both contractions are
// kind::f16 with exact products, and only p_j is rounded (2^-11).
//
// A unit of work is (token, 64 heads, 64 positions). The units of a launch are
// split evenly and contiguously over one CTA per SM; a row tile (token, 64
// heads) that lies across CTAs leaves normalised FP32 pieces and their LSE in
// the workspace, joined by merge_pieces_kernel. Twenty warps:
//   0-7   softmax: S from TMEM, weights to shared memory, at the end of a row
//         tile the output from TMEM
//   8-15  loaders: a unit's 64 rows of codes in flight in registers, widened to
//         FP16 and stored in one of two 128-byte-swizzled tiles; at the start
//         of a row tile its queries
//   16    issues the score products, 17 the value products: each waits for its
//         own operands, and the tensor core takes what is there
//   18-19 the units' rows: pages, scales, fetches into L2, up to four units ahead
// The scores are S[64 positions, 64 heads] = K Q^T as M = 64 products (36 cycles
// each, against 52 with M = 128, whose tile would leave no room for a second
// one, so that products, softmax and conversion would take turns); the values
// O^T[128 values, 64 heads] += V^T P^T for each quarter of the values, from the
// same tile read MN-major.
// TMEM: two S buffers of 64 columns, four O^T quarters of 64. Shared memory:
// two FP16 tiles (128 KB), the queries (64 KB), two buffers of weights (16 KB).
//
// What bounds it. In a long run a unit takes about 3.1k cycles, most of them on the
// path between shared memory, L1 and the rest, 128 bytes a clock. Counted over a call
// of 64 tokens over 8192 positions (ncu, 3.5k cycles a unit with the start and the
// outputs): the products' operands 1792 wavefronts a unit (224 KB; issued alone they
// take 1984 cycles, 32 score products of 36 and 16 value products of 52), loads and
// stores 1417 (the tile's stores and the codes' loads are 768, the rest weights,
// factors, lookups, pieces and outputs) and 411 more in conflicts between the two.
// It is not all: copies of the kernel without half of the stores are 0.22k cycles a
// unit faster, without the loads 0.24k, with half the score products 0.26k (of 0.58k
// that these take to issue), without the exponentials 0.03k; loads issued a half
// earlier, conversion before the wait and weights stored before the vote changed
// nothing or lost. Around a CTA's units lie 7k cycles up to its first rows (planning,
// dependent lookups, cold instructions), and 4.1k for each output or piece of 64 heads
// (a piece's 128 KB leave the SM at 32 bytes a clock; an output is half as long, in
// stores of 2 bytes). Measured on one GB300: 1021 tokens over some 8K
// positions each, 64 heads, INT8: 1.34 ms, 0.75 PFLOP/s; 12 tokens over 64K
// positions, E4M3: 150 us, 2.6 TB/s and 0.67 PFLOP/s; 64 tokens over 2048 listed
// positions, E4M3: 49 us, 1.5 TB/s; one token over 512 listed positions: 15 us,
// nearly all of it fixed cost.
// 64 positions a unit: with 128 a tile's 128 KB leave room for one only, and
// conversion, products and softmax take turns (the first case 2.01 ms against
// 1.85 when the two were compared).

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "qli_internal.h"
#include "qli_meta.cuh"
#include "qli_ptx.cuh"

namespace qli {
namespace kvattn {
namespace {

constexpr int kD = 512;
constexpr int kHT = 64;                        // heads per row tile (MMA N)
constexpr int kPos = 64;                       // positions per unit
constexpr int kSoftWarps = 8, kLoadWarps = 8;
constexpr int kLoadWarp0 = kSoftWarps, kScoreWarp = kSoftWarps + kLoadWarps;
constexpr int kValueWarp = kScoreWarp + 1, kRowWarp0 = kScoreWarp + 2, kRowWarps = 2;
constexpr int kThreads = 32 * (kRowWarp0 + kRowWarps);
// Registers of the warpgroups' threads, within the CTA's 640 x 96. A spill in a
// role's loop costs an L2 round trip: the streamed codes leave L1 to nothing else.
constexpr int kSoftRegs = 104, kLoadRegs = 104, kIssueRegs = 64;
static_assert(2 * kSoftRegs + 2 * kLoadRegs + kIssueRegs <= 5 * 96, "registers of the CTA");
constexpr int kSlots = 4;                      // units whose rows are looked up ahead
constexpr int kRegion = kPos * 128;            // 64 values of every row of a tile (or query)
constexpr int kTile = 8 * kRegion;
constexpr int kChunkT = 512;                   // tokens planned per launch, one a thread
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 0, kOCol = 256;
constexpr float kSlack = 8.0f, kShift = 6.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kPieceRow = kHT * kD;            // floats of a piece

struct Smem {
  uint8_t kv[2][kTile];                        // 1024-aligned, by unit parity
  uint8_t q[kTile];                            // 1024-aligned
  uint8_t p[2][kPos * 128];                    // 1024-aligned, by unit parity
  int32_t tokV[kChunkT], tokB[kChunkT];        // visible positions and request of the launch's tokens
  const uint8_t* row[kSlots][kPos];            // the rows' codes, by unit modulo kSlots
  float rs[kSlots][kPos];                      // and scales; 0: no position
  float sl2[2][kHT];                           // by row tile parity: softmax scale in log2 over the
                                               // queries' power of two
  float m[kHT], alpha[kHT], delta[kHT];
  float part[2][4][32];                        // [32 heads][softmax warp of them][head]
  int32_t warp_sum[kThreads / 32];
  int32_t count, start_t, start_g, start_i;    // the CTA's share: units, first token, row tile, unit
  // tiles by unit parity and half of the values. What the softmax warps arrive
  // on is by unit parity too: four of them may be a unit ahead of the others.
  uint64_t full[2][2], empty[2][2], sfull[2], sfree[2], rowfull[kSlots], rowfree[kSlots], qfull, qempty, pready[2], done;
  uint32_t tmem_base;
};
constexpr int kSmemBytes = static_cast<int>(sizeof(Smem)) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct Args {
  const uint16_t* q;
  int64_t q_st, q_sh;
  int32_t T, H, B;
  const int32_t* cu;
  const int32_t* k_lens;
  const int32_t* residual;
  int32_t ratio, window;
  int64_t cap;                 // positions a block-table row holds
  const uint8_t* cache;
  int64_t page_stride, num_pages, kv_off, sc_off;
  int32_t R, log2R;
  const int32_t* bt;
  int32_t bt_stride;
  const int32_t* idx;
  int32_t K;
  float scale;
  uint16_t* out;
  int64_t o_st, o_sh;
  float* lse;
  uint32_t* err;
  int32_t t0, tc;              // tokens of this launch: t0 .. t0 + tc
  int32_t ht;                  // heads per row tile, at most kHT
  int32_t hg;                  // row tiles per token
  int32_t whole;               // 1: CTA c has row tile c, whole; 0: even shares
  // workspace
  int4* cut;                   // [CTAs] the row tile that goes on in the next CTA: token, row tile,
                               // first unit past it (token -1: none)
  float* piece;                // [2 * CTAs][64][512]
  float* piece_lse;            // [2 * CTAs][64], log2
};

// Instruction descriptor, kind::f16 with FP16 A and B, FP32 D, M = m, N = n;
// a_mn / b_mn select MN-major operands.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) |
         ((m >> 4) << 24);
}

// Shared-memory descriptor, 128-byte swizzle. K-major: sbo = bytes between
// 8-row groups (lbo unused). MN-major: lbo = bytes between 64-value atoms
// along M or N, sbo = bytes between 8-row groups along K. `off` bytes further
// on is lo + (off >> 4): shared addresses stay within the 14 address bits.
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
__host__ __device__ constexpr uint32_t sdesc_hi(uint32_t sbo) {
  return (sbo >> 4) | (1u << 14) | (2u << 29);
}

// Byte offset of 16-byte unit u of row r in a swizzled region of 128-byte rows.
__device__ __forceinline__ uint32_t sw(uint32_t r, uint32_t u) {
  return r * 128u + ((u ^ (r & 7u)) << 4);
}

__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t x, uint32_t y, uint32_t z,
                                             uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Two FP32 numbers in one register pair, and the packed FP32 operations on
// them (each half rounded as the scalar operation would be).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair_of(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 both(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ void st_shared(uint32_t at, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}

// 2^x by the SFU's approximation (a few ulp; 2^-inf = +0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Waits, as a whole warp, for the phase with the given parity; false once it
// has been probed 2^16 times (0.1 us each while the CTA is busy, 20 us when
// nothing happens: some ms to a second or so). A loop of five instructions: the
// roles' loops together have to stay within the instruction cache.
#ifdef QLI_TEST_STALL_EPILOGUE
constexpr int kProbes = 1 << 13;               // a test build, in which CTA 1 waits for what never comes
#else
constexpr int kProbes = 1 << 16;
#endif
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 i;\n\t"
      "mov.u32 i, %3;\n"
      "PROBE:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "sub.u32 i, i, 1;\n\t"
      "setp.ne.u32 q, i, 0;\n\t"
      "@q bra PROBE;\n"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "n"(kProbes)
      : "memory");
  return __all_sync(0xffffffffu, ok);
}

// 32 lanes x 16 consecutive 32-bit columns of TMEM.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// The first 16 of the warp's 32 lanes x 32 columns: lane t gets, of the i-th
// eight columns, 2 (t & 3) and the next, of rows t / 4 (r[4i], r[4i + 1]) and
// t / 4 + 8 (r[4i + 2], r[4i + 3]).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// log2 x likewise (log2 0 = -inf).
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void named_bar(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// The same, and whether any of the n threads has p.
__device__ __forceinline__ bool named_bar_any(int id, int n, bool p) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(n), "r"(static_cast<uint32_t>(p))
      : "memory");
  return any != 0;
}

// The warpgroup's registers per thread.
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// 16 codes to 16 FP16 values (exact), lowest byte first.
template <bool kFp8>
__device__ __forceinline__ void widen16(const uint4 v, uint32_t (&o)[8]) {
  if constexpr (kFp8) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
          "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
          : "=r"(o[2 * k]), "=r"(o[2 * k + 1])
          : "r"(w[k]));
  } else {
    // 0x64xx is the FP16 number 1024 + xx; the code plus 128 is xx
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const __half2 bias = __floats2half2_rn(-1152.0f, -1152.0f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t u = w[k] ^ 0x80808080u;
      const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
      const __half2 a = __hadd2(*reinterpret_cast<const __half2*>(&lo), bias);
      const __half2 b = __hadd2(*reinterpret_cast<const __half2*>(&hi), bias);
      o[2 * k] = *reinterpret_cast<const uint32_t*>(&a);
      o[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// The launch's units in order: token, row tile of the token, unit of kPos
// positions. A token has at least one unit, so that every output is written.
__device__ __forceinline__ int32_t positions_of(const Args& a, int32_t V) {
  return a.idx ? a.K : (a.window > 0 ? min(V, a.window) : V);
}
__device__ __forceinline__ int32_t units_of(const Args& a, int32_t V) {
  const int32_t n = positions_of(a, V);
  return n <= kPos ? 1 : (n - 1) / kPos + 1;
}

// First unit of CTA c of `ctas`, out of `total` (below 2^30).
__device__ __forceinline__ int32_t share_begin(int32_t total, int32_t ctas, int32_t c) {
  const int32_t each = total / ctas;
  return each * c + min(c, total - each * ctas);
}

// A CTA's share, unit by unit.
struct Walk {
  int32_t k, count;            // units behind, units of the share
  int32_t t, g, i, n;          // token (within the launch), row tile, unit of it, its units
  __device__ __forceinline__ Walk(const Args& a, const Smem& S)
      : k(0), count(S.count), t(S.start_t), g(S.start_g), i(S.start_i) {
    n = units_of(a, S.tokV[t]);
  }
  __device__ __forceinline__ bool valid() const { return k < count; }
  // first and last unit of the row tile in this CTA
  __device__ __forceinline__ bool first() const { return k == 0 || i == 0; }
  __device__ __forceinline__ bool last() const { return i == n - 1 || k + 1 == count; }
  // at its last unit: whether the row tile began in this CTA
  __device__ __forceinline__ bool began_here() const { return k >= i; }
  __device__ __forceinline__ void next(const Args& a, const Smem& S) {
    ++k;
    if (++i < n) return;
    i = 0;
    if (++g < a.hg) return;
    g = 0;
    if (++t < a.tc) n = units_of(a, S.tokV[t]);
  }
};

// Request of token t (absolute): the last one starting at or before it.
// `cu` is the raw array or its copy in shared memory.
__device__ __forceinline__ int32_t request_of(const int32_t* cu, int32_t B, int32_t T, int32_t t) {
  int32_t lo = 0, hi = B - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (min(max(cu[mid], 0), T) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Flags requests with bad metadata, once a call.
__device__ __forceinline__ void flag_requests(const Args& a, int tid) {
  if (a.idx || a.t0 != 0 || !a.err) return;
  uint32_t e = 0u;
#pragma unroll 1
  for (int b = tid; b < a.B; b += kThreads) {
    int32_t q0, q1, lk, res;
    e |= sanitize_request(a, b, q0, q1, lk, res);
  }
  if (e) atomicOr(a.err, e);
}

// The requests' boundaries and lengths, as sanitize_request reads them: copies in
// the still unused tiles, where they fit.
struct Requests {
  const int32_t *cu, *k_lens, *residual;
  int32_t T, B, ratio;
  int64_t cap;
};
constexpr int kRequestsInSmem = 10000;
static_assert((3 * kRequestsInSmem + 1) * 4 <= 2 * kTile, "the requests fit in the tiles");

// What a thread loads before the CTA has set itself up, so that the latencies
// overlap: its request's metadata, and in listed mode (where the CTA's share
// follows from sizes alone) a row warp's entry of the CTA's first unit.
struct Early {
  int32_t cu, k_len, residual, entry;
};

// The CTA's share [u0, u1) of `total` units.
__device__ __forceinline__ void share_of(const Args& a, int32_t total, int32_t& u0, int32_t& u1) {
  const int32_t ctas = static_cast<int32_t>(gridDim.x), c = static_cast<int32_t>(blockIdx.x);
  u0 = share_begin(total, ctas, c);
  u1 = share_begin(total, ctas, c + 1);
}

__device__ __forceinline__ Early load_early(const Args& a) {
  const int tid = threadIdx.x, r = tid - 32 * kRowWarp0;
  Early v{0, 0, 0, -1};
  if (tid <= a.B) v.cu = __ldg(a.cu + tid);
  if (!a.idx) {
    if (tid < a.B) v.k_len = __ldg(a.k_lens + tid);
    if (tid < a.B && a.residual) v.residual = __ldg(a.residual + tid);
  } else if (r >= 0) {
    const int32_t units = units_of(a, 0);
    int32_t u0, u1;
    share_of(a, a.tc * a.hg * units, u0, u1);
    const int32_t e = u0 % units * kPos + r;
    if (u0 < u1 && e < a.K) v.entry = __ldg(a.idx + static_cast<int64_t>(a.t0 + u0 / units / a.hg) * a.K + e);
  }
  return v;
}

// The last row tile of the share, which began at unit `first` of the launch:
// cut if it goes on in the next CTA, and the first cut of it if it began here.
__device__ __forceinline__ void record_cut(const Args& a, int32_t t, int32_t g, int32_t first, int32_t end,
                                           int32_t u0, int32_t u1, int32_t total) {
  a.cut[blockIdx.x] = make_int4(end > u1 && first >= u0 ? t : -1, g, end, total);
}

// Plans the launch: every token's request and visible positions, and the CTA's
// share. A thread takes one token.
__device__ __forceinline__ void plan(const Args& a, Smem& S, const Early& early) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Requests req{a.cu, a.k_lens, a.residual, a.T, a.B, a.ratio, a.cap};
  if (a.B <= kRequestsInSmem) {
    int32_t* cu = reinterpret_cast<int32_t*>(S.kv);
    int32_t *k_lens = cu + a.B + 1, *residual = k_lens + a.B;
#pragma unroll 1
    for (int b = tid; b <= a.B; b += kThreads) {
      const bool more = b >= kThreads, len = b < a.B && !a.idx;
      cu[b] = more ? __ldg(a.cu + b) : early.cu;
      if (len) k_lens[b] = more ? __ldg(a.k_lens + b) : early.k_len;
      if (len && a.residual) residual[b] = more ? __ldg(a.residual + b) : early.residual;
    }
    req.cu = cu;
    req.k_lens = k_lens;
    if (a.residual) req.residual = residual;
  }
  __syncthreads();
  int32_t V = 0, units = 0;
  if (tid < a.tc) {
    const int32_t t = a.t0 + tid, b = request_of(req.cu, a.B, a.T, t);
    if (!a.idx) {
      int32_t q0, q1, lk, res;
      sanitize_request(req, b, q0, q1, lk, res);
      if (q0 <= t && t < q1) V = visible_count(lk, res, a.ratio, q1 - q0, t - q0);
    }
    S.tokV[tid] = V;
    S.tokB[tid] = b;
    units = units_of(a, V);
  }
  if (blockIdx.x == 0) flag_requests(a, tid);
  if (a.whole) {
    __syncthreads();
    if (tid == 0) {
      S.start_t = static_cast<int32_t>(blockIdx.x) / a.hg;
      S.start_g = static_cast<int32_t>(blockIdx.x) % a.hg;
      S.start_i = 0;
      S.count = units_of(a, S.tokV[S.start_t]);
    }
    __syncthreads();
    return;
  }
  int32_t u0, u1;
  if (a.idx) {
    // every token has as many units
    if (tid == 0) {
      const int32_t each = units_of(a, 0), total = a.tc * a.hg * each;
      share_of(a, total, u0, u1);
      const int32_t tile = u0 / each, last = (u1 - 1) / each;
      S.start_t = tile / a.hg;
      S.start_g = tile % a.hg;
      S.start_i = u0 - tile * each;
      S.count = u1 - u0;
      if (u1 <= u0) a.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
      else record_cut(a, last / a.hg, last % a.hg, last * each, (last + 1) * each, u0, u1, total);
    }
    __syncthreads();
    return;
  }
  const int32_t mine = units * a.hg;
  int32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) S.warp_sum[warp] = incl;
  __syncthreads();
  int32_t sums = lane < kThreads / 32 ? S.warp_sum[lane] : 0;
  const int32_t own = __shfl_sync(0xffffffffu, sums, warp);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += y;
  }
  const int32_t total = __shfl_sync(0xffffffffu, sums, 31);
  const int32_t at = __shfl_sync(0xffffffffu, sums, warp) - own + incl - mine;
  share_of(a, total, u0, u1);
  if (at <= u0 && u0 < at + mine) {
    S.start_t = tid;
    S.start_g = (u0 - at) / units;
    S.start_i = (u0 - at) % units;
  }
  if (tid == 0) S.count = u1 - u0;
  if (u1 <= u0) {
    if (tid == 0) a.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
  } else if (at <= u1 - 1 && u1 - 1 < at + mine) {
    const int32_t g = (u1 - 1 - at) / units, first = at + g * units;
    record_cut(a, tid, g, first, first + units, u0, u1, total);
  }
  __syncthreads();
}

// ---- loaders ----------------------------------------------------------------
// Quarter c of the values is in regions 2c and 2c + 1, in this order: 16-byte
// unit j of region 2c + b holds values 128c + 16j + 8b .. + 7, so that a lane's 16
// loaded codes fill unit j of two regions and eight lanes cover all banks. The
// queries are stored alike, and row 64b + 8j + x of O^T's quarter c is that
// value + x.
__device__ __forceinline__ int value_of(int c, int row) {
  return 128 * c + 16 * ((row >> 3) & 7) + 8 * (row >> 6) + (row & 7);
}

// What rows without a position, and rows of zeros, are filled from.
__device__ __align__(16) const uint8_t kZeroRow[kD] = {};

// The row tile's queries as FP16 times a power of two per head that brings the
// head's largest magnitude to [2^13, 2^14); rows past the row tile's heads are
// zero. A warp takes every eighth row.
__device__ __forceinline__ void load_queries(const Args& a, Smem& S, int32_t t, int32_t g,
                                             uint32_t parity, int lw) {
  const int lane = threadIdx.x & 31;
  constexpr int kRows = kHT / kLoadWarps, kBatch = 4;
  // lane l holds values 16l .. 16l + 15: unit l & 7 of quarter l >> 3
  const uint32_t dst = smem_u32(S.q) + (lane >> 3) * 2 * kRegion;
  const int heads = min(a.ht, a.H - g * a.ht);
  const uint16_t* q = a.q + static_cast<int64_t>(a.t0 + t) * a.q_st + g * a.ht * a.q_sh + 16 * lane;
#pragma unroll 1
  for (int k0 = 0; k0 < kRows; k0 += kBatch) {
    uint4 v[kBatch][2];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = kLoadWarps * (k0 + k) + lw;
      v[k][0] = v[k][1] = make_uint4(0u, 0u, 0u, 0u);
      if (r < heads) {
        const uint4* src = reinterpret_cast<const uint4*>(q + r * a.q_sh);
        v[k][0] = __ldg(src);
        v[k][1] = __ldg(src + 1);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = kLoadWarps * (k0 + k) + lw;
      uint32_t w[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                       v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
      // magnitudes compare as integers (NaN above all)
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        top = max(top, max((w[i] << 16) & 0x7fff0000u, w[i] & 0x7fff0000u));
      top = __reduce_max_sync(0xffffffffu, top);
      const int e = min(100, 13 - (static_cast<int>(top >> 23) - 127));
      const float f = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = pack_half2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
      const uint32_t at = dst + sw(r, lane & 7);
      st_shared_v4(at, w[0], w[1], w[2], w[3]);
      st_shared_v4(at + kRegion, w[4], w[5], w[6], w[7]);
      if (lane == 0)
        S.sl2[parity][r] = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    }
  }
}

// The rows of the units, one a lane: iteration m publishes unit m and takes one
// step each of the lookup of units m + 1 (page to codes and scale, the codes
// fetched into L2), m + 2 (position to page) and m + 3 (listed entry to
// position; `entry` is the first unit's), so that no step waits for the load of the
// one before. Positions
// past the table and pages outside the pool are skipped and flagged.
__device__ __forceinline__ bool run_rows(const Args& a, Smem& S, int32_t entry) {
  const int lane = threadIdx.x & 31, r = threadIdx.x - 32 * kRowWarp0;
  bool bad = false;
  Walk w(a, S);                                       // unit m + 3
  int32_t j3 = -1, b3 = 0;                            // position, request
  int32_t j2 = -1, page2 = -1;                        // position, page
  const uint8_t* codes1 = kZeroRow;                   // codes and scale
  uint16_t s1 = 0;
  bool live1 = false;
#pragma unroll 1
  for (int32_t m = -3; m < w.count; ++m) {
    if (m >= 0) {
      const uint32_t slot = m & (kSlots - 1);
      if (!wait(&S.rowfree[slot], ((m / kSlots) & 1) ^ 1)) return false;
      // a row under a zero scale stands for zeros whatever its codes are: it
      // counts in the normaliser only, under the smallest scale there is, so
      // that it does not set the reference
      const float s = __half2float(__ushort_as_half(s1));
      const bool zero = live1 && s == 0.0f;
      S.row[slot][r] = zero ? kZeroRow : codes1;
      S.rs[slot][r] = live1 ? (zero ? 5.9604645e-8f : s) : 0.0f;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.rowfull[slot]);
    }
    // unit m + 1
    codes1 = kZeroRow;
    live1 = j2 >= 0 && page2 >= 0 && page2 < a.num_pages;
    bad |= j2 >= 0 && !live1;
    if (live1) {
      const uint8_t* base = a.cache + static_cast<int64_t>(page2) * a.page_stride;
      const int32_t row = j2 & (a.R - 1);
      codes1 = base + a.kv_off + row * kD;
      s1 = __ldg(reinterpret_cast<const uint16_t*>(base + a.sc_off + row * 2));
#pragma unroll
      for (int c = 0; c < 4; ++c) asm volatile("prefetch.global.L2 [%0];" ::"l"(codes1 + c * 128));
    }
    // unit m + 2
    bad |= j3 >= a.cap;
    j2 = j3 < a.cap ? j3 : -1;
    if (j2 >= 0) page2 = __ldg(a.bt + static_cast<int64_t>(b3) * a.bt_stride + (j2 >> a.log2R));
    // unit m + 3
    j3 = -1;
    if (w.valid()) {
      const int32_t V = S.tokV[w.t], n = positions_of(a, V), e = w.i * kPos + r;
      b3 = S.tokB[w.t];
      if (e < n)
        j3 = !a.idx ? V - n + e : m == -3 ? entry : __ldg(a.idx + static_cast<int64_t>(a.t0 + w.t) * a.K + e);
      if (w.first()) {
        // the row tile's queries, into L2: head r, 128 bytes at a time
        const int h = w.g * a.ht + r, end = r < a.ht ? a.H : 0;
        const uint16_t* q = a.q + static_cast<int64_t>(a.t0 + w.t) * a.q_st + h * a.q_sh;
#pragma unroll 1
        for (int c = 0; c < 8 && h < end; ++c) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + c * 64));
      }
      w.next(a, S);
    }
  }
  if (bad && a.err) atomicOr(a.err, QLI_DEVERR_PAGE);
  return true;
}

// Iteration n stores unit n from registers, one half of the values after the
// other as they come free, then loads unit n + 1 (32 KB in flight on the SM
// while unit n is worked on). A warp has eight rows; a warp
// instruction loads one quarter of four.
template <bool kFp8>
__device__ __forceinline__ bool run_loaders(const Args& a, Smem& S) {
  const int lane = threadIdx.x & 31, lw = (threadIdx.x >> 5) - kLoadWarp0;
  const int r0 = kPos / kLoadWarps * lw + (lane >> 3), off = (lane & 7) * 16;
  // rows 4 apart: 512 bytes on, and bit 2 of the swizzled unit flips
  const uint32_t at0 = smem_u32(S.kv) + sw(r0, lane & 7), at1 = (at0 ^ 64u) + 512;
  uint32_t seg = 0;
  Walk w(a, S);                                       // unit n + 1
  uint4 x[2][4];
#pragma unroll 1
  for (int32_t n = -1; n < w.count; ++n) {
    if (n >= 0) {
      const int buf = n & 1;
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        if (!wait(&S.empty[buf][f], ((n >> 1) & 1) ^ 1)) return false;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int c = 2 * f; c < 2 * f + 2; ++c) {
            uint32_t o[8];
            widen16<kFp8>(x[k][c], o);
            const uint32_t at = (k ? at1 : at0) + buf * kTile + c * 2 * kRegion;
            st_shared_v4(at, o[0], o[1], o[2], o[3]);
            st_shared_v4(at + kRegion, o[4], o[5], o[6], o[7]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.full[buf][f]);
      }
    }
    if (n + 1 == w.count) break;
    // unit n + 1: its codes, and at the start of a row tile its queries; the
    // codes first, but at the very start, where their rows are not known yet
#pragma unroll 1
    for (int step = 0; step < 2; ++step) {
      if ((step == 0) == (n >= 0)) {
        const uint32_t slot = (n + 1) & (kSlots - 1);
        if (!wait(&S.rowfull[slot], ((n + 1) / kSlots) & 1)) return false;
        const uint8_t* r[2] = {S.row[slot][r0] + off, S.row[slot][r0 + 4] + off};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int c = 0; c < 4; ++c) x[k][c] = __ldg(reinterpret_cast<const uint4*>(r[k] + c * 128));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.rowfree[slot]);
      } else if (w.first()) {
        // the products with the previous row tile's queries are done, and the
        // softmax is past its wait for them
        if (!wait(&S.qempty, (seg & 1) ^ 1)) return false;
        load_queries(a, S, w.t, w.g, seg & 1, lw);
        ++seg;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.qfull);
      }
    }
    w.next(a, S);
  }
  return true;
}

// ---- products (a warp for the scores, one for the values) -------------------------
// The whole warp runs the loop and an elected lane issues each batch of
// products with constant descriptor steps, about ten instructions a product;
// one thread's loop with 64-bit descriptors took 100-180 cycles a product.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// D (+)= A B^T from descriptors given as low and high words.
__device__ __forceinline__ void mma(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                    uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, 1;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc)
      : "memory");
}
__device__ __forceinline__ void mma_first(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// At the end each warp waits for the products of both.
__device__ __forceinline__ bool drain(Smem& S) {
  if (elect_one()) mma_commit(&S.done);
  __syncwarp();
  return wait(&S.done, 0);
}

__device__ __forceinline__ bool run_scores(const Args& a, Smem& S, uint32_t tmem_any) {
  constexpr uint32_t id = idesc_f16(kPos, kHT, false, false), hi = sdesc_hi(1024);
  const uint32_t k_lo = sdesc_lo(smem_u32(S.kv), 16), q_lo = sdesc_lo(smem_u32(S.q), 16);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
  bool ok = true;
  uint32_t n = 0, seg = 0;
#pragma unroll 1
  for (Walk w(a, S); ok && w.valid(); w.next(a, S), ++n) {
    const uint32_t buf = n & 1, parity = (n >> 1) & 1;
    const bool last = w.last();
    if (w.first()) ok = wait(&S.qfull, seg++ & 1);
    ok = ok && wait(&S.sfree[buf], parity ^ 1);
#pragma unroll 1
    for (uint32_t f = 0; f < 2 && ok; ++f) {
      ok = wait(&S.full[buf][f], parity);
      tc_fence_after();
      if (ok && elect_one()) {
        const uint32_t step = f * (4 * kRegion >> 4), ke = k_lo + buf * (kTile >> 4) + step;
        const uint32_t qe = q_lo + step, se = tmem + kSCol + buf * kHT;
        mma_first(se, ke, qe, hi, id, f);
#pragma unroll
        for (uint32_t k = 1; k < 16; ++k) {
          const uint32_t on = ((k >> 2) * kRegion + (k & 3) * 32) >> 4;
          mma(se, ke + on, qe + on, hi, id);
        }
        if (f) {
          mma_commit(&S.sfull[buf]);
          if (last) mma_commit(&S.qempty);
        }
      }
      __syncwarp();
    }
  }
  return drain(S) && ok;
}

__device__ __forceinline__ bool run_values(const Args& a, Smem& S, uint32_t tmem_any) {
  constexpr uint32_t id = idesc_f16(128, kHT, true, true), hi = sdesc_hi(1024);
  const uint32_t v_lo = sdesc_lo(smem_u32(S.kv), kRegion), p_lo = sdesc_lo(smem_u32(S.p), 1024);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
  bool ok = true;
#ifdef QLI_TEST_STALL_EPILOGUE
  ok = blockIdx.x != 1;
#endif
  uint32_t n = 0;
#pragma unroll 1
  for (Walk w(a, S); ok && w.valid(); w.next(a, S), ++n) {
    const uint32_t more = w.first() ? 0u : 1u, tile = v_lo + (n & 1) * (kTile >> 4);
    const uint32_t pe = p_lo + (n & 1) * (kPos * 128 >> 4);
    ok = wait(&S.pready[n & 1], (n >> 1) & 1);
    tc_fence_after();
    if (ok && elect_one()) {
#pragma unroll
      for (uint32_t f = 0; f < 2; ++f) {
#pragma unroll
        for (uint32_t c = 2 * f; c < 2 * f + 2; ++c) {
          const uint32_t ve = tile + c * (2 * kRegion >> 4), oe = tmem + kOCol + c * kHT;
          mma_first(oe, ve, pe, hi, id, more);
#pragma unroll
          for (uint32_t k = 1; k < 4; ++k) mma(oe, ve + (k * 2048 >> 4), pe + (k * 2048 >> 4), hi, id);
        }
        mma_commit(&S.empty[n & 1][f]);
      }
    }
    __syncwarp();
  }
  return drain(S) && ok;
}

// ---- softmax ------------------------------------------------------------------
// Combines 8 values a lane (pair i: heads 8i + 2 (lane & 3) and the next) across
// the eight lanes that share lane & 3; the lane gets the one of head_of(lane).
template <class F>
__device__ __forceinline__ float across(const f32x2 (&x)[4], int lane, F f) {
  float v[4];
  {
    const bool up = (lane & 16) != 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 lo = both(x[i]), hi = both(x[i + 2]);
      v[2 * i] = f(up ? hi.x : lo.x, __shfl_xor_sync(0xffffffffu, up ? lo.x : hi.x, 16));
      v[2 * i + 1] = f(up ? hi.y : lo.y, __shfl_xor_sync(0xffffffffu, up ? lo.y : hi.y, 16));
    }
  }
#pragma unroll
  for (int o = 8; o > 2; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o / 4; ++i) {
      const float send = up ? v[i] : v[i + o / 4], keep = up ? v[i + o / 4] : v[i];
      v[i] = f(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return v[0];
}
__device__ __forceinline__ int head_of(int lane) {
  return 8 * (lane >> 3) + 2 * (lane & 3) + ((lane >> 2) & 1);
}

// O^T's row `pos` of each quarter times the heads' factors, the 32 heads from h0
// on. BF16 outputs (kOut), of the first `nh` heads: head i at dst + i * stride,
// in the order of the values (a warp stores to one 128-byte line). FP32 pieces,
// of at least those: head i at dst + i * kD, in the order of the rows (likewise;
// merge_pieces_kernel reorders). A row tile without positions (`none`) gives zeros
// whatever a query that is not finite has left in the accumulators.
template <bool kOut, class T>
__device__ __forceinline__ void output(const Smem& S, uint32_t tmem, int h0, int pos, int32_t nh, bool none,
                                       T* dst, int64_t stride) {
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {
    const int i0 = (c & 1) * 16;
    if (i0 >= nh) continue;
    uint32_t o[16];
    tmem_ld_x16(tmem + (c >> 1) * kHT + i0, o);
    float al[16];                                     // before the stores, which loads may not pass
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(al + 4 * i) =
        *reinterpret_cast<const float4*>(S.alpha + h0 + i0 + 4 * i);
    tmem_ld_wait();
    T* at = dst + i0 * stride + (kOut ? value_of(c >> 1, pos) : 128 * (c >> 1) + pos);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float v = none ? 0.0f : __uint_as_float(o[i]) * al[i];
      if constexpr (kOut) {
        const __nv_bfloat16 y = __float2bfloat16_rn(v);
        if (i0 + i < nh) *at = *reinterpret_cast<const uint16_t*>(&y);
        at += stride;
      } else {
        at[i * kD] = v;
      }
    }
  }
}

// Warp (qw, sub) has positions 16 qw .. 16 qw + 15 (M = 64 scores lie in the first
// 16 of every 32 TMEM lanes) of the 32 heads from 32 sub on; a lane has two
// positions, lane / 4 and 8 further, of four pairs of heads. The four warps of a
// `sub` share a named barrier.
__device__ __forceinline__ bool run_softmax(const Args& a, Smem& S, uint32_t tmem) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int qw = warp & 3, sub = warp >> 2, bar = 1 + sub;
  const uint32_t lanes = static_cast<uint32_t>(32 * qw) << 16;
  const int pos = 16 * qw + (lane >> 2), h0 = 32 * sub + 2 * (lane & 3);
  float* part = S.part[sub][0];
  // pair i: heads h0 + 8i, h0 + 8i + 1
  const f32x2* m2 = reinterpret_cast<const f32x2*>(S.m + h0);
  const f32x2* de2 = reinterpret_cast<const f32x2*>(S.delta + h0);
  const f32x2* al2 = reinterpret_cast<const f32x2*>(S.alpha + h0);
  // the lane's word of unit 4 sub of its first position; unit 4 sub + i flips bits 4, 5
  const uint32_t p_at = smem_u32(S.p) + sw(pos, 4 * sub) + 4 * (lane & 3);
  bool ok = true, seen = false, live = false;          // live: one of the lane's positions is there
  f32x2 l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) l[i] = pair_of(0.0f, 0.0f);
  uint32_t n = 0, seg = 0;
  // A wait that gives up clears `ok`. The warp still runs through the named
  // barriers, on whatever TMEM holds, but arrives nowhere else, so that nobody
  // goes on with what it should have made and the units after this one end in
  // waits that give up too. What it adds to a normaliser is NaN, and so are its
  // outputs: a row tile that was not finished does not look like a result, in
  // `out` or, by way of its piece, in a join.
  for (Walk w(a, S); w.valid(); w.next(a, S), ++n) {
    const uint32_t buf = n & 1, parity = (n >> 1) & 1;
    if (w.first()) {                                  // the heads' factors
      if (ok && !wait(&S.qfull, seg & 1)) ok = false;
      ++seg;
      seen = live = false;
      // the queries after these wait for this warp too, so that it sees every
      // phase of the barrier
      if (lane == 0 && ok) mbar_arrive(&S.qempty);
    }
    const uint32_t slot = n & (kSlots - 1);
    if (ok && !wait(&S.rowfull[slot], (n / kSlots) & 1)) ok = false;
    // d = y - M + kShift = score * cs + es; no position here: -inf, weight 0.
    // 1 / s is taken from the logarithm that d uses, so that p / s is free of
    // its error.
    f32x2 cs[2][4], es[2][4], inv2[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float s = S.rs[slot][pos + 8 * k], ls = lg2(s), inv_s = s != 0.0f ? ex2(-ls) : 0.0f;
      live |= s != 0.0f;
      const f32x2* c2 = reinterpret_cast<const f32x2*>(S.sl2[(seg - 1) & 1] + h0);
      const f32x2 s2 = pair_of(s, s), ls2 = pair_of(ls + kShift, ls + kShift);
      inv2[k] = pair_of(inv_s, inv_s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[k][i] = mul2(c2[4 * i], s2);
        es[k][i] = sub2(ls2, m2[4 * i]);
      }
    }
    if (ok && !wait(&S.sfull[buf], parity)) ok = false;
    tc_fence_after();
    f32x2 d[2][4];
    float over = -INFINITY;
    {
      uint32_t r[16];
      tmem_ld_16x256b_x4(tmem + lanes + kSCol + kHT * buf + 32 * sub, r);
      tmem_ld_wait();
      tc_fence_before();
      if (lane == 0 && ok) mbar_arrive(&S.sfree[buf]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          d[k][i] = fma2(pair_of(__uint_as_float(r[4 * i + 2 * k]), __uint_as_float(r[4 * i + 2 * k + 1])),
                         cs[k][i], es[k][i]);
          const float2 u = both(d[k][i]);
          over = fmaxf(over, fmaxf(u.x, u.y));
        }
      }
    }
    // until something was seen, any position sets the references
    const bool rises = over > (seen ? kSlack + kShift : -INFINITY);
    // the weights of the unit before last have been used
    if (ok && !wait(&S.empty[buf][1], parity ^ 1)) ok = false;
    if (named_bar_any(bar, 128, rises)) {
      // move references to the maxima so far: each head decides for itself, a
      // non-finite one keeps its reference
      f32x2 t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = both(d[0][i]), v = both(d[1][i]);
        t[i] = pair_of(fmaxf(u.x, v.x), fmaxf(u.y, v.y));
      }
      part[qw * 32 + head_of(lane)] = across(t, lane, [](float p, float q) { return fmaxf(p, q); });
      named_bar(bar, 128);
      float up = fmaxf(fmaxf(part[lane], part[32 + lane]), fmaxf(part[64 + lane], part[96 + lane])) - kShift;
      if ((seen && !(up > kSlack)) || !(fabsf(up) < INFINITY)) up = 0.0f;
      if (qw == 0) {
        S.m[32 * sub + lane] += up;
        S.delta[32 * sub + lane] = up;
        S.alpha[32 * sub + lane] = seen ? ex2(-up) : 1.0f;
      }
      named_bar(bar, 128);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[0][i] = sub2(d[0][i], de2[4 * i]);
        d[1][i] = sub2(d[1][i], de2[4 * i]);
        l[i] = mul2(l[i], al2[4 * i]);
      }
      if (seen) {
        // the products of the units before are done
        if (ok && !wait(&S.empty[buf ^ 1][1], ((n - 1) >> 1) & 1)) ok = false;
        tc_fence_after();
        // 16 heads at a time, those whose reference moved
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          const float* al = S.alpha + 32 * sub + 16 * g;
          if (!__any_sync(0xffffffffu, al[lane & 15] != 1.0f)) continue;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[16];
            const uint32_t oe = tmem + lanes + kOCol + c * kHT + 32 * sub + 16 * g;
            tmem_ld_x16(oe, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al[i]);
            tmem_st_x16(oe, o);
          }
        }
        tmem_st_wait();
      }
      seen = true;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = both(d[k][i]);
        const float px = ex2(v.x), py = ex2(v.y);
        d[k][i] = pair_of(px, py);
        st_shared((p_at ^ (i << 4)) + buf * (kPos * 128) + k * 1024, pack_half2(px, py));
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0 && ok) {
      mbar_arrive(&S.pready[buf]);
      mbar_arrive(&S.rowfree[slot]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) l[i] = fma2(d[1][i], inv2[1], fma2(d[0][i], inv2[0], l[i]));
    if (!w.last()) continue;

    // ---- the row tile's end in this CTA: totals, then the output
    // A query that is not finite makes NaN weights of rows without a position too:
    // a warp that has no position adds nothing.
    const float mine = across(l, lane, [](float p, float q) { return p + q; });
    part[qw * 32 + head_of(lane)] = !ok ? NAN : __any_sync(0xffffffffu, live) ? mine : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) l[i] = pair_of(0.0f, 0.0f);
    named_bar(bar, 128);
    // lane: head 32 sub + lane
    const float total = (part[lane] + part[32 + lane]) + (part[64 + lane] + part[96 + lane]);
    const bool none = __all_sync(0xffffffffu, total == 0.0f);
    float lse2 = total == 0.0f ? -INFINITY : S.m[32 * sub + lane] - kShift + log2f(total);
    named_bar(bar, 128);
    if (qw == 0) {
      S.alpha[32 * sub + lane] = total == 0.0f ? 0.0f : 1.0f / total;
      S.m[32 * sub + lane] = 0.0f;
    }
    named_bar(bar, 128);
    if (ok && !wait(&S.empty[buf][1], parity)) ok = false;
    if (!ok) {
      lse2 = NAN;
      S.alpha[32 * sub + lane] = NAN;
      __syncwarp();
    }
    tc_fence_after();
    const int32_t h = w.g * a.ht + 32 * sub;          // first head of this sub
    const int32_t nh = min(min(32, a.ht - 32 * sub), a.H - h);  // heads to write
    const uint32_t oe = tmem + lanes + kOCol + 32 * sub;
    if (w.i == w.n - 1 && w.began_here()) {
      if (qw == 0 && lane < nh && a.lse)
        a.lse[static_cast<int64_t>(a.t0 + w.t) * a.H + h + lane] = lse2 * kLn2;
      uint16_t* orow = a.out + static_cast<int64_t>(a.t0 + w.t) * a.o_st + h * a.o_sh;
      output<true>(S, oe, 32 * sub, 32 * qw + lane, nh, none, orow, a.o_sh);
    } else {
      // a row tile that began in an earlier CTA goes to slot 0, one that goes
      // on in the next to slot 1
      const int64_t piece = 2 * static_cast<int64_t>(blockIdx.x) + (w.began_here() ? 1 : 0);
      if (qw == 0) a.piece_lse[piece * kHT + 32 * sub + lane] = lse2;
      output<false>(S, oe, 32 * sub, 32 * qw + lane, nh, none, a.piece + piece * kPieceRow + (32 * sub) * kD,
                    static_cast<int64_t>(kD));
    }
    named_bar(bar, 128);                              // the factors are read
  }
  return ok;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1) kv_attn_kernel(const Args a) {
  extern __shared__ uint8_t smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  const Early early = load_early(a);
  if (warp == kScoreWarp) tmem_alloc(&S.tmem_base, kTmemCols);
  if (tid < kHT) S.m[tid] = 0.0f;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int f = 0; f < 2; ++f) {
        mbar_init(&S.full[i][f], kLoadWarps);
        mbar_init(&S.empty[i][f], 1);
      }
      mbar_init(&S.sfull[i], 1);
      mbar_init(&S.sfree[i], kSoftWarps);
      mbar_init(&S.pready[i], kSoftWarps);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&S.rowfull[i], kRowWarps);
      mbar_init(&S.rowfree[i], kLoadWarps + kSoftWarps);
    }
    mbar_init(&S.qfull, kLoadWarps);
    mbar_init(&S.qempty, 1 + kSoftWarps);
    mbar_init(&S.done, 2);
    fence_mbar_init();
  }
  tc_fence_before();
  plan(a, S, early);                          // ends with a barrier of the CTA
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  if (S.count > 0) {
    bool ok = true;
    if (warp < kSoftWarps) {
      more_registers<kSoftRegs>();
      ok = run_softmax(a, S, tmem);
    } else if (warp < kScoreWarp) {
      more_registers<kLoadRegs>();
      ok = run_loaders<kFp8>(a, S);
    } else {
      fewer_registers<kIssueRegs>();
      if (warp == kScoreWarp) ok = run_scores(a, S, tmem);
      if (warp == kValueWarp) ok = run_values(a, S, tmem);
      if (warp >= kRowWarp0) ok = run_rows(a, S, early.entry);
    }
    if (!ok && lane == 0 && a.err) atomicOr(a.err, QLI_DEVERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kScoreWarp) tmem_dealloc(tmem, kTmemCols);
}

// ---- joining the pieces ---------------------------------------------------------
// Bound by latency: pieces of up to all SMs, 128 KB each, come out of L2 (10 us
// alone, most of it before the first load; it starts while its predecessor ends).
// Block (c - 1, k): the row tile that began in CTA c - 1 and goes on in CTA c, if
// there is one; rows 8k .. 8k+7 of it, a warp per row.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = kJoinThreads / 32;

__global__ void __launch_bounds__(kJoinThreads) merge_pieces_kernel(const Args a, int32_t ctas) {
  pdl_wait();
  const int lane = threadIdx.x & 31, c = blockIdx.x + 1;
  const int row = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
  const int4 tile = __ldcg(a.cut + c - 1);
  const int32_t h = tile.y * a.ht + row;
  if (tile.x < 0 || h >= a.H || row >= a.ht) return;
  // pieces: CTA c - 1's slot 1, then slot 0 of CTA c, c + 1, ... up to the end
  // (a CTA with units has all its predecessors with units)
  int32_t count = 2;
#pragma unroll 1
  while (c + count - 1 < ctas && share_begin(tile.w, ctas, c + count - 1) < tile.z) ++count;
  const auto slot = [&](int32_t k) -> int64_t {
    return k == 0 ? 2 * static_cast<int64_t>(c - 1) + 1 : 2 * static_cast<int64_t>(c - 1 + k);
  };
  const auto lse_of = [&](int32_t k) -> float {
    return k < count ? __ldcg(a.piece_lse + slot(k) * kHT + row) : -INFINITY;
  };
  const float first = lse_of(lane);
  float m = first;
#pragma unroll 1
  for (int32_t k = lane + 32; k < count; k += 32) m = fmaxf(m, lse_of(k));
  float acc[16], total = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  const float4* src = reinterpret_cast<const float4*>(a.piece + static_cast<int64_t>(row) * kD) + lane;
  constexpr int kBatch = 4;                           // pieces whose loads are in flight together
#pragma unroll 1
  for (int32_t k0 = 0; k0 < count; k0 += kBatch) {
    float4 v[kBatch][4];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[k][i] = k0 + k < count ? __ldcg(src + slot(k0 + k) * (kPieceRow / 4) + 32 * i)
                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    if (k0 == 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const float mine = k0 < 32 ? first : lse_of(k0 - k0 % 32 + lane);
    const float wk = mine == -INFINITY ? 0.0f : ex2(mine - m);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float w = __shfl_sync(0xffffffffu, wk, (k0 + k) & 31);
      if (w == 0.0f) continue;
      total += w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[4 * i] = fmaf(w, v[k][i].x, acc[4 * i]);
        acc[4 * i + 1] = fmaf(w, v[k][i].y, acc[4 * i + 1]);
        acc[4 * i + 2] = fmaf(w, v[k][i].z, acc[4 * i + 2]);
        acc[4 * i + 3] = fmaf(w, v[k][i].w, acc[4 * i + 3]);
      }
    }
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t t = a.t0 + tile.x;
  // the lane's rows 4l .. 4l + 3 of each quarter are four values in a row
  uint16_t* dst = a.out + t * a.o_st + h * a.o_sh;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(acc[4 * i] * inv, acc[4 * i + 1] * inv);
    const __nv_bfloat162 y = __floats2bfloat162_rn(acc[4 * i + 2] * inv, acc[4 * i + 3] * inv);
    *reinterpret_cast<uint2*>(dst + value_of(i, 4 * lane)) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  if (lane == 0 && a.lse)
    a.lse[t * a.H + h] = total == 0.0f ? -INFINITY : (m + log2f(total)) * kLn2;
}

std::atomic<uint64_t> g_smem_kv_attn[2];

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

qli_status validate(const qli_kv_attn_args* a) {
  if (a == nullptr) return QLI_ERR_INVALID_ARG;
  if (a->D != kD || a->H < 1 || a->H > 128) return QLI_ERR_UNSUPPORTED;
  if (a->rows_per_page != 64 && a->rows_per_page != 128) return QLI_ERR_UNSUPPORTED;
  if (a->quant_mode != QLI_QUANT_INT8 && a->quant_mode != QLI_QUANT_FP8) return QLI_ERR_UNSUPPORTED;
  if (a->T < 0 || a->B < 0 || (a->B == 0 && a->T != 0)) return QLI_ERR_INVALID_ARG;
  if (!std::isfinite(a->scale)) return QLI_ERR_INVALID_ARG;
  if (a->indices != nullptr) {
    if (a->K < 1 || a->window != 0) return QLI_ERR_INVALID_ARG;
  } else {
    if (a->ratio != 1 && a->ratio != 2) return QLI_ERR_UNSUPPORTED;
    if (a->ratio == 1 && a->residual != nullptr) return QLI_ERR_RESIDUAL_WITH_RATIO1;
    if (a->window < 0) return QLI_ERR_INVALID_ARG;
    if (a->T > 0 && a->k_lens == nullptr) return QLI_ERR_INVALID_ARG;
  }
  if (a->T == 0) return QLI_OK;
  if (a->q == nullptr || a->cu_seqlens_q == nullptr || a->cache == nullptr ||
      a->block_table == nullptr || a->out == nullptr)
    return QLI_ERR_INVALID_ARG;
  if (a->bt_stride < 1 || a->bt_width < 0 || a->num_pages < 1 || a->page_stride <= 0 || a->kv_offset < 0 ||
      a->kv_scale_offset < 0 ||
      a->kv_offset + static_cast<int64_t>(a->rows_per_page) * kD > a->page_stride ||
      a->kv_scale_offset + static_cast<int64_t>(a->rows_per_page) * 2 > a->page_stride)
    return QLI_ERR_INVALID_ARG;
  if (a->q_stride_h < kD || a->q_stride_t < kD || a->out_stride_h < kD || a->out_stride_t < kD)
    return QLI_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || a->q_stride_t % 8 || a->q_stride_h % 8 || !aligned(a->out, 16) ||
      a->out_stride_t % 8 || a->out_stride_h % 8 || !aligned(a->cache, 16) ||
      a->page_stride % 16 || a->kv_offset % 16 || a->kv_scale_offset % 2 ||
      !aligned(a->cu_seqlens_q, 4) || !aligned(a->block_table, 4) || !aligned(a->indices, 4) ||
      !aligned(a->k_lens, 4) || !aligned(a->residual, 4) || !aligned(a->lse, 4) ||
      !aligned(a->err_word, 4))
    return QLI_ERR_ALIGNMENT;
  return QLI_OK;
}

Args make_args(const qli_kv_attn_args& a) {
  Args d{};
  d.q = a.q;
  d.q_st = a.q_stride_t;
  d.q_sh = a.q_stride_h;
  d.T = a.T;
  d.H = a.H;
  d.B = a.B;
  d.cu = a.cu_seqlens_q;
  d.k_lens = a.k_lens;
  d.residual = a.residual;
  d.ratio = a.ratio;
  d.window = a.window;
  d.cap = static_cast<int64_t>(a.bt_width ? a.bt_width : a.bt_stride) * a.rows_per_page;
  d.cache = a.cache;
  d.page_stride = a.page_stride;
  d.num_pages = a.num_pages;
  d.kv_off = a.kv_offset;
  d.sc_off = a.kv_scale_offset;
  d.R = a.rows_per_page;
  d.log2R = a.rows_per_page == 64 ? 6 : 7;
  d.bt = a.block_table;
  d.bt_stride = a.bt_stride;
  d.idx = a.indices;
  d.K = a.K;
  d.scale = a.scale;
  d.out = a.out;
  d.o_st = a.out_stride_t;
  d.o_sh = a.out_stride_h;
  d.lse = a.lse;
  d.err = a.err_word;
  return d;
}

// Most units a row tile can have.
int64_t most_units(const Args& d) {
  int64_t n = d.idx ? static_cast<int64_t>(d.K) : d.cap < INT32_MAX ? d.cap : INT32_MAX;
  if (!d.idx && d.window > 0 && d.window < n) n = d.window;
  return n <= kPos ? 1 : (n - 1) / kPos + 1;
}

// Row tiles of at most this many units are not cut while there is an SM for
// each. 64 tokens over a window of 128 positions (two units): 21.6 us cut and
// joined, 19.6 us whole.
constexpr int kWholeUnits = 2;

// Heads per row tile: 64, what the products are made for, or 32 or 16 while
// every unit (or uncut row tile) still has an SM of its own. The conversions and
// products of a unit stay the same, but its queries and its output, which leaves
// an SM at 32 bytes a clock, shrink with the heads. One token of 64 heads over 512
// positions: 16.6 us with 64 heads a tile, 14.6 with 16; 64 tokens of 32 heads over
// a window of 128: 14.5 and 13.1.
int32_t heads_per_tile(const Args& d, int64_t most, int sms) {
  int32_t ht = kHT;
  while (ht > 16 && (most <= kWholeUnits ? 1 : most) * d.T * ((d.H + ht / 2 - 1) / (ht / 2)) <= sms) ht /= 2;
  return ht;
}

// Workspace, per SM: the row tile it cuts, two pieces and their LSE.
struct Layout {
  size_t piece, lse, total;
};
Layout layout_for(int sms) {
  Layout L{};
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  L.piece = up(sizeof(int4) * static_cast<size_t>(sms));
  L.lse = L.piece + up(sizeof(float) * 2 * static_cast<size_t>(sms) * kPieceRow);
  L.total = L.lse + up(sizeof(float) * 2 * static_cast<size_t>(sms) * kHT);
  return L;
}

template <bool kFp8>
cudaError_t launch(Args d, int sms, cudaStream_t s) {
  const auto kernel = kv_attn_kernel<kFp8>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), kSmemBytes,
                                    g_smem_kv_attn[kFp8 ? 1 : 0]);
  const int64_t most = most_units(d);
  d.ht = heads_per_tile(d, most, sms);
  d.hg = (d.H + d.ht - 1) / d.ht;
  // tokens per launch: what one plan holds, and fewer than 2^30 units
  const int64_t fit = (int64_t{1} << 30) / (most * d.hg);
  const int32_t chunk = static_cast<int32_t>(fit < kChunkT ? fit : kChunkT);
  for (d.t0 = 0; e == cudaSuccess && d.t0 < d.T; d.t0 += chunk) {
    d.tc = d.T - d.t0 < chunk ? d.T - d.t0 : chunk;
    const int64_t tiles = static_cast<int64_t>(d.tc) * d.hg;
    d.whole = most <= kWholeUnits && tiles <= sms ? 1 : 0;
    // one CTA per SM, and no more than there can be units
    const int64_t units = tiles * most;
    const int32_t ctas = static_cast<int32_t>(d.whole ? tiles : units < sms ? units : sms);
    kernel<<<static_cast<unsigned>(ctas), kThreads, kSmemBytes, s>>>(d);
    e = cudaGetLastError();
    if (e == cudaSuccess && ctas > 1 && !d.whole)
      e = launch_pdl(merge_pieces_kernel,
                     dim3(static_cast<unsigned>(ctas - 1),
                          static_cast<unsigned>(((d.H < d.ht ? d.H : d.ht) + kJoinRows - 1) / kJoinRows)),
                     dim3(kJoinThreads), 0, s, d, ctas);
  }
  return e;
}

}  // namespace
}  // namespace kvattn
}  // namespace qli

extern "C" qli_status qli_kv_attention_workspace_size(const qli_kv_attn_args* a, size_t* bytes) {
  if (bytes == nullptr) return QLI_ERR_INVALID_ARG;
  qli_status st = qli::kvattn::validate(a);
  if (st != QLI_OK) return st;
  *bytes = 0;
  if (a->T == 0) return QLI_OK;
  int sms = 0;
  st = qli::device_sms(&sms);
  if (st == QLI_OK) *bytes = qli::kvattn::layout_for(sms).total;
  return st;
}

extern "C" qli_status qli_kv_attention(const qli_kv_attn_args* a, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  using namespace qli::kvattn;
  qli_status st = validate(a);
  if (st != QLI_OK) return st;
  if (a->T == 0) return QLI_OK;
  int sms = 0;
  st = qli::device_sms(&sms);
  if (st != QLI_OK) return st;
  const Layout L = layout_for(sms);
  if (workspace == nullptr || workspace_bytes < L.total) return QLI_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256)) return QLI_ERR_ALIGNMENT;
  Args d = make_args(*a);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  d.cut = reinterpret_cast<int4*>(w);
  d.piece = reinterpret_cast<float*>(w + L.piece);
  d.piece_lse = reinterpret_cast<float*>(w + L.lse);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->quant_mode == QLI_QUANT_FP8 ? launch<true>(d, sms, s) : launch<false>(d, sms, s);
  return e == cudaSuccess ? QLI_OK : QLI_ERR_CUDA;
}

extern "C" int64_t qli_kv_attn_args_size(void) {
  return static_cast<int64_t>(sizeof(qli_kv_attn_args));
}
