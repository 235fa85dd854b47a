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
// A unit of work is (token, 64 heads, 128 positions). The units of a launch
// are split evenly and contiguously over one CTA per SM; a row tile (token,
// 64 heads) that lies across CTAs leaves normalised FP32 pieces and their LSE
// in the workspace, joined by merge_pieces_kernel. Twenty warps:
//   0-7   softmax: S (lane = position, column = head) from TMEM, weights to
//         shared memory, at the end of a row tile the output from TMEM
//   8-15  loaders: per unit the 128 rows' codes, two 128-value quarters of the
//         tile in flight in registers, widened to FP16 and stored in the
//         128-byte-swizzled tile
//   17-19 the row tile's queries
//   16    MMA issuer: S[128 positions, 64 heads] = K Q^T quarter by quarter as
//         the tile fills, then O^T[128 values, 64 heads] += V^T P^T for each
//         quarter, from the same tile read MN-major; a quarter is handed back as
//         soon as its products are done
// TMEM: S (64 columns) and four O^T quarters of 64. Shared memory: the FP16 tile (128 KB), the queries
// (64 KB), the weights (16 KB).
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
constexpr int kPos = 128;                      // positions per unit
constexpr int kSoftWarps = 8, kLoadWarps = 8;
constexpr int kLoadWarp0 = kSoftWarps, kMmaWarp = kSoftWarps + kLoadWarps, kQueryWarps = 3;
constexpr int kThreads = 640;                  // five warpgroups
// Registers of the warpgroups' threads, within the CTA's 640 x 96.
constexpr int kSoftRegs = 144, kLoadRegs = 72, kMmaRegs = 48;
static_assert(2 * kSoftRegs + 2 * kLoadRegs + kMmaRegs <= 5 * 96, "registers of the CTA");
constexpr int kRegion = kPos * 128;            // 64 values of every row of the tile
constexpr int kQRegion = kHT * 128;            // 64 values of every query row
constexpr int kChunkT = 2048;                  // tokens planned per launch
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 0, kOCol = kHT;
constexpr float kSlack = 8.0f, kShift = 6.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kPieceRow = kHT * kD;            // floats of a piece

struct Smem {
  uint8_t kv[8 * kRegion];                     // 1024-aligned
  uint8_t q[8 * kQRegion];                     // 1024-aligned
  uint8_t p[kPos * 128];                       // 1024-aligned
  int32_t tokV[kChunkT];                       // visible positions of the launch's tokens
  const uint8_t* row[2][kPos];                 // the rows' codes by unit parity
  float rs[2][kPos];                           // row scales by unit parity; 0: no position
  float sl2[2][kHT];                           // by row tile parity: softmax scale in log2 over the
                                               // queries' power of two
  float m[kHT], alpha[kHT], delta[kHT];
  float part[2][4][32];                        // [head half][lane quarter][head]
  alignas(16) int32_t flag[2][2][4];                       // [unit parity][head half][lane quarter]
  int64_t warp_sum[kThreads / 32];
  int32_t count, start_t, start_g, start_i;    // the CTA's share: units, first token, row tile, unit
  uint64_t full[4], empty[4], qfull, qempty, sfull, pready, pvdone, done;
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
  int64_t cap;                 // bt_stride * R
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
  int32_t hg;                  // row tiles per token
  // workspace
  int64_t* tok_start;          // [tc + 1] first unit of each token
  float* piece;                // [2 * CTAs][64][512]
  float* piece_lse;            // [2 * CTAs][64], log2
};

// Instruction descriptor, kind::f16 with FP16 A and B, FP32 D, M = 128, N = n;
// a_mn / b_mn select MN-major operands.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) |
         ((128u >> 4) << 24);
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
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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
#ifndef QLI_KV_ATTN_PROBES
#define QLI_KV_ATTN_PROBES (1 << 16)
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
      : "r"(smem_u32(bar)), "r"(parity), "n"(QLI_KV_ATTN_PROBES)
      : "memory");
  return __all_sync(0xffffffffu, ok);
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

// The warpgroup's registers per thread (out of those the CTA was launched with).
template <int kRegs>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// 16 codes to 16 FP16 values (exact), lowest byte first.
template <bool kFp8>
__device__ __forceinline__ void widen16(const uint4 v, uint32_t (&o)[8]) {
  if constexpr (kFp8) {
    e4m3x16_to_f16x16(v, o);
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

// The launch's units in order: token, row tile of the token, unit of 128
// positions. A token has at least one unit, so that every output is written.
__device__ __forceinline__ int32_t positions_of(const Args& a, int32_t V) {
  return a.idx ? a.K : (a.window > 0 ? min(V, a.window) : V);
}
__device__ __forceinline__ int32_t units_of(const Args& a, int32_t V) {
  const int32_t n = positions_of(a, V);
  return n <= kPos ? 1 : (n - 1) / kPos + 1;
}

// A CTA's share, unit by unit (fewer than 2^31 of them).
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

// Plans the launch: every token's visible positions and the CTA's first unit.
// One pass over the tokens by the whole CTA.
__device__ __forceinline__ void plan(const Args& a, Smem& S) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the boundaries go through the (still unused) tile when they fit
  int32_t* cu_s = reinterpret_cast<int32_t*>(S.kv);
  const bool local = a.B <= static_cast<int32_t>(sizeof(S.kv) / 4);
  if (!a.idx) {
    if (local)
      for (int b = tid; b < a.B; b += kThreads) cu_s[b] = __ldg(a.cu + b);
    if (blockIdx.x == 0 && a.t0 == 0 && a.err) {
      uint32_t e = 0u;
      for (int b = tid; b < a.B; b += kThreads) {
        int32_t q0, q1, lk, res;
        e |= sanitize_request(a, b, q0, q1, lk, res);
      }
      if (e) atomicOr(a.err, e);
    }
    __syncthreads();
    for (int i = tid; i < a.tc; i += kThreads) {
      const int32_t t = a.t0 + i;
      const int32_t b = request_of(local ? cu_s : a.cu, a.B, a.T, t);
      int32_t q0, q1, lk, res;
      sanitize_request(a, b, q0, q1, lk, res);
      S.tokV[i] = q0 <= t && t < q1 ? visible_count(lk, res, a.ratio, q1 - q0, t - q0) : 0;
    }
  } else {
    for (int i = tid; i < a.tc; i += kThreads) S.tokV[i] = 0;
  }
  __syncthreads();
  const int per = (a.tc + kThreads - 1) / kThreads;
  const int lo = min(a.tc, tid * per), hi = min(a.tc, lo + per);
  int64_t mine = 0;
  for (int i = lo; i < hi; ++i) mine += units_of(a, S.tokV[i]);
  mine *= a.hg;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) S.warp_sum[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t v = S.warp_sum[w];
    if (w < warp) before += v;
    total += v;
  }
  int64_t at = before + incl - mine;
  const int64_t u0 = total * blockIdx.x / gridDim.x;
  const int64_t u1 = total * (blockIdx.x + 1) / gridDim.x;
  if (tid == 0) S.count = static_cast<int32_t>(u1 - u0);
  for (int i = lo; i < hi; ++i) {
    const int64_t n = units_of(a, S.tokV[i]);
    if (blockIdx.x == 0) a.tok_start[i] = at;
    if (at <= u0 && u0 < at + n * a.hg) {
      S.start_t = i;
      S.start_g = static_cast<int32_t>((u0 - at) / n);
      S.start_i = static_cast<int32_t>((u0 - at) % n);
    }
    at += n * a.hg;
  }
  if (blockIdx.x == 0 && tid == 0) a.tok_start[a.tc] = total;
  __syncthreads();
}

// ---- loaders ----------------------------------------------------------------
// The order of a quarter's 128 values in the tile: 16-byte unit j of region
// 2e + b holds values 128e + 16j + 8b .. + 7, so that a lane's 16 loaded codes
// fill unit j of two regions and eight lanes cover all banks. The queries are
// stored alike, and row 64b + 8j + x of O^T's quarter e is that value + x.
__device__ __forceinline__ int value_of(int e, int row) {
  return 128 * e + 16 * ((row >> 3) & 7) + 8 * (row >> 6) + (row & 7);
}

// What rows without a position, and rows of zeros, are filled from.
__device__ __align__(16) const uint8_t kZeroRow[kD] = {};

// Row r of the walk's unit: its codes into S.row, its scale (0: no position
// there). Positions past the table and pages outside the pool are skipped and
// flagged. A row under a zero scale stands for zeros whatever its codes are:
// it counts in the normaliser only, under the smallest scale there is, so that
// it does not set the reference. The codes are fetched into L2 a unit ahead.
__device__ __forceinline__ float find_row(const Args& a, Smem& S, const Walk& w, int32_t b, int r,
                                          uint32_t parity, bool& bad) {
  const int32_t V = S.tokV[w.t], n = positions_of(a, V), e = w.i * kPos + r;
  const uint8_t* codes = kZeroRow;
  float s = 0.0f;
  int64_t j = -1;
  if (e < n) j = a.idx ? __ldg(a.idx + static_cast<int64_t>(a.t0 + w.t) * a.K + e) : V - n + e;
  if (j >= a.cap) {
    bad = true;
  } else if (j >= 0) {
    const int32_t page = __ldg(a.bt + static_cast<int64_t>(b) * a.bt_stride + (j >> a.log2R));
    if (page < 0 || page >= a.num_pages) {
      bad = true;
    } else {
      const uint8_t* base = a.cache + static_cast<int64_t>(page) * a.page_stride;
      const int32_t row = static_cast<int32_t>(j) & (a.R - 1);
      codes = base + a.kv_off + row * kD;
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(codes), "n"(kD));
      s = __half2float(__ushort_as_half(
          __ldg(reinterpret_cast<const uint16_t*>(base + a.sc_off + row * 2))));
      if (s == 0.0f) {
        s = 5.9604645e-8f;
        codes = kZeroRow;
      }
    }
  }
  S.row[parity][r] = codes;
  return s;
}

// The row tile's queries as FP16 times a power of two per head that brings the
// head's largest magnitude to [2^13, 2^14); rows past H are zero.
__device__ __forceinline__ void load_queries(const Args& a, Smem& S, int32_t t, int32_t g,
                                             uint32_t parity, int qw) {
  const int lane = threadIdx.x & 31;
  constexpr int kBatch = 2;
  // lane l holds values 16l .. 16l + 15: unit l & 7 of regions 2 (l >> 3), + 1
  uint8_t* dst = S.q + (lane >> 3) * 2 * kQRegion;
#pragma unroll 1
  for (int r0 = qw * kBatch; r0 < kHT; r0 += kBatch * kQueryWarps) {
    uint4 v[kBatch][2];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = g * kHT + r0 + k;
      v[k][0] = v[k][1] = make_uint4(0u, 0u, 0u, 0u);
      if (h < a.H) {
        const uint4* src = reinterpret_cast<const uint4*>(
                               a.q + static_cast<int64_t>(a.t0 + t) * a.q_st + h * a.q_sh) + 2 * lane;
        v[k][0] = __ldg(src);
        v[k][1] = __ldg(src + 1);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k;
      const uint32_t w[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                             v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
      // magnitudes compare as integers (NaN above all)
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        top = max(top, max((w[i] << 16) & 0x7fff0000u, w[i] & 0x7fff0000u));
      top = __reduce_max_sync(0xffffffffu, top);
      const int e = min(100, 13 - (static_cast<int>(top >> 23) - 127));
      const float f = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] = pack_half2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
      const uint32_t at = smem_u32(dst) + sw(r, lane & 7);
      st_shared_v4(at, o[0], o[1], o[2], o[3]);
      st_shared_v4(at + kQRegion, o[4], o[5], o[6], o[7]);
      if (lane == 0)
        S.sl2[parity][r] = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    }
  }
}

__device__ __forceinline__ bool run_queries(const Args& a, Smem& S) {
  const int qw = (threadIdx.x >> 5) - kMmaWarp - 1;
  uint32_t seg = 0;
  for (Walk w(a, S); w.valid(); w.next(a, S)) {
    if (!w.first()) continue;
    // the products with the previous row tile's queries are done, and the
    // softmax is past its wait for them
    if (!wait(&S.qempty, (seg & 1) ^ 1)) return false;
    load_queries(a, S, w.t, w.g, seg & 1, qw);
    ++seg;
    fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&S.qfull);
  }
  return true;
}

// A warp's 16 rows of one quarter of the tile: four loads a lane, each warp
// instruction 128 bytes of four rows.
constexpr int kWarpRows = kPos / kLoadWarps, kSteps = kWarpRows / 4;
struct Quarter {
  uint4 v[kSteps];
};

// rows: the lane's first row pointer (rows 4k apart follow); off: byte of the row.
__device__ __forceinline__ void load_quarter(Quarter& b, const uint8_t* const* rows, int off) {
#pragma unroll
  for (int k = 0; k < kSteps; ++k) b.v[k] = __ldg(reinterpret_cast<const uint4*>(rows[4 * k] + off));
}

// dst: the lane's unit of its first row in the quarter's first region. Rows
// 4k apart are 512 bytes apart; the swizzle flips bit 2 of the unit between
// even and odd k.
template <bool kFp8>
__device__ __forceinline__ void store_quarter(uint32_t even, uint32_t odd, const Quarter& b) {
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    uint32_t o[8];
    widen16<kFp8>(b.v[k], o);
    const uint32_t at = ((k & 1) ? odd : even) + k * 512;
    st_shared_v4(at, o[0], o[1], o[2], o[3]);
    st_shared_v4(at + kRegion, o[4], o[5], o[6], o[7]);
  }
}

template <bool kFp8>
__device__ __forceinline__ bool run_loaders(const Args& a, Smem& S) {
  const int lane = threadIdx.x & 31, lw = (threadIdx.x >> 5) - kLoadWarp0;
  const int r = kWarpRows * lw + lane;                // lanes 0-15: the row looked up
  const int r0 = kWarpRows * lw + (lane >> 3), off = (lane & 7) * 16;
  const uint32_t even = smem_u32(S.kv) + sw(r0, lane & 7), odd = even ^ 64u;
  bool bad = false, ok = true;
  Walk w(a, S);                                       // one unit ahead of the tile being filled
  int32_t bt = w.t, b = request_of(a.cu, a.B, a.T, a.t0 + bt);
  float s = 0.0f;
  if (lane < kWarpRows) s = find_row(a, S, w, b, r, 0u, bad);
  __syncwarp();
  Quarter x, y;
  load_quarter(x, &S.row[0][r0], off);
  load_quarter(y, &S.row[0][r0], off + 128);
  for (uint32_t n = 0; w.valid(); ++n) {
    // the next unit's rows, whose loads go out during this one
    w.next(a, S);
    float s_next = 0.0f;
    if (w.valid()) {
      if (w.t != bt) {
        bt = w.t;
        b = request_of(a.cu, a.B, a.T, a.t0 + bt);
      }
      if (lane < kWarpRows) s_next = find_row(a, S, w, b, r, (n + 1) & 1, bad);
    } else if (lane < kWarpRows) {
      S.row[(n + 1) & 1][r] = kZeroRow;
    }
    __syncwarp();
    const uint32_t parity = (n & 1) ^ 1;
#pragma unroll 1
    for (uint32_t pair = 0; pair < 2; ++pair) {
      // this unit's second pair, or the next unit's first
      const uint8_t* const* rows = &S.row[(n + pair) & 1][r0];
      const int next = off + (pair ? 0 : 256);
      const uint32_t base = pair * 4 * kRegion;
      if (!wait(&S.empty[2 * pair], parity)) {
        ok = false;
        break;
      }
      if (pair == 0 && lane < kWarpRows) S.rs[n & 1][r] = s;
      store_quarter<kFp8>(even + base, odd + base, x);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.full[2 * pair]);
      load_quarter(x, rows, next);
      if (!wait(&S.empty[2 * pair + 1], parity)) {
        ok = false;
        break;
      }
      store_quarter<kFp8>(even + base + 2 * kRegion, odd + base + 2 * kRegion, y);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.full[2 * pair + 1]);
      load_quarter(y, rows, next + 128);
    }
    if (!ok) break;
    s = s_next;
  }
  if (bad && a.err) atomicOr(a.err, QLI_DEVERR_PAGE);
  return ok;
}

// ---- MMA issuer (one warp) ------------------------------------------------------
// The whole warp runs the loop and an elected lane issues each batch of
// products with constant descriptor steps, about ten instructions a product;
// one thread's loop with 64-bit descriptors took 100-180 cycles a product,
// where the tensor core takes 42.
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

__device__ __forceinline__ bool run_mma(const Args& a, Smem& S, uint32_t tmem_any) {
  constexpr uint32_t id_qk = idesc_f16(kHT, false, false), id_pv = idesc_f16(kHT, true, true);
  constexpr uint32_t hi = sdesc_hi(1024);
  const uint32_t k_lo = sdesc_lo(smem_u32(S.kv), 16), q_lo = sdesc_lo(smem_u32(S.q), 16);
  const uint32_t v_lo = sdesc_lo(smem_u32(S.kv), kRegion), p_lo = sdesc_lo(smem_u32(S.p), 1024);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
  bool ok = true;
  uint32_t n = 0, seg = 0;
  for (Walk w(a, S); w.valid(); w.next(a, S), ++n) {
    const bool last = w.last();
    if (w.first() && !wait(&S.qfull, seg++ & 1)) {
      ok = false;
      break;
    }
#pragma unroll 1
    for (uint32_t e = 0; e < 4; ++e) {
      if (!wait(&S.full[e], n & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint32_t ke = k_lo + e * (2 * kRegion >> 4), qe = q_lo + e * (2 * kQRegion >> 4);
        mma_first(tmem + kSCol, ke, qe, hi, id_qk, e);
#pragma unroll
        for (uint32_t k = 1; k < 8; ++k)
          mma(tmem + kSCol, ke + (((k >> 2) * kRegion + (k & 3) * 32) >> 4),
              qe + (((k >> 2) * kQRegion + (k & 3) * 32) >> 4), hi, id_qk);
        if (e == 3) {
          mma_commit(&S.sfull);
          if (last) mma_commit(&S.qempty);
        }
      }
      __syncwarp();
    }
    if (!ok) break;
    const uint32_t more = w.first() ? 0u : 1u;
    if (!wait(&S.pready, n & 1)) {
      ok = false;
      break;
    }
    tc_fence_after();
#pragma unroll 1
    for (uint32_t e = 0; e < 4; ++e) {
      if (elect_one()) {
        const uint32_t ve = v_lo + e * (2 * kRegion >> 4), oe = tmem + kOCol + e * kHT;
        mma_first(oe, ve, p_lo, hi, id_pv, more);
#pragma unroll
        for (uint32_t k = 1; k < 8; ++k) mma(oe, ve + (k * 2048 >> 4), p_lo + (k * 2048 >> 4), hi, id_pv);
        mma_commit(&S.empty[e]);
        if (e == 3) mma_commit(&S.pvdone);
      }
      __syncwarp();
    }
  }
  if (elect_one()) mma_commit(&S.done);               // every product of the CTA
  __syncwarp();
  return wait(&S.done, 0) && ok;
}

// ---- softmax ------------------------------------------------------------------
// Combines 32 values a lane (as 16 pairs) across the warp's 32 lanes: lane l
// gets value l's result.
template <class F>
__device__ __forceinline__ float across(const f32x2 (&x)[16], int lane, F f) {
  float v[16];
  {
    const bool up = (lane & 16) != 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 lo = both(x[i]), hi = both(x[i + 8]);
      v[2 * i] = f(up ? hi.x : lo.x, __shfl_xor_sync(0xffffffffu, up ? lo.x : hi.x, 16));
      v[2 * i + 1] = f(up ? hi.y : lo.y, __shfl_xor_sync(0xffffffffu, up ? lo.y : hi.y, 16));
    }
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = f(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return v[0];
}

__device__ __forceinline__ bool run_softmax(const Args& a, Smem& S, uint32_t tmem) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int qw = warp & 3, half = warp >> 2;          // TMEM lane quarter; heads 32 half ..
  const uint32_t lanes = static_cast<uint32_t>(32 * qw) << 16;
  const int pos = 32 * qw + lane, bar = 1 + half;
  float* part = S.part[half][0];
  const float4* m4 = reinterpret_cast<const float4*>(S.m + 32 * half);
  const f32x2* de2 = reinterpret_cast<const f32x2*>(S.delta + 32 * half);
  const f32x2* al2 = reinterpret_cast<const f32x2*>(S.alpha + 32 * half);
  bool ok = true, seen = false;
  f32x2 l[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) l[i] = pair_of(0.0f, 0.0f);
  uint32_t n = 0, seg = 0;
  // A wait that gives up clears `ok`; the warps still run through the same
  // named barriers, on whatever TMEM holds, and write no output.
  for (Walk w(a, S); w.valid(); w.next(a, S), ++n) {
    if (w.first()) {                                  // the heads' factors
      if (ok && !wait(&S.qfull, seg & 1)) ok = false;
      ++seg;
      // the queries after these wait for this warp too, so that it sees every
      // phase of the barrier
      if (lane == 0) mbar_arrive(&S.qempty);
    }
    if (ok && !wait(&S.full[0], n & 1)) ok = false;                  // the row scales
    if (ok && !wait(&S.sfull, n & 1)) ok = false;
    tc_fence_after();
    if (w.first()) seen = false;
    uint32_t xr[32];
    tmem_ld_32x32b_x32(tmem + lanes + kSCol + 32 * half, xr);
    tmem_ld_wait();
    // d = y - M + kShift; no position here: -inf, weight 0. 1 / s is taken from
    // the logarithm that d uses, so that p / s is free of its error.
    const float s = S.rs[n & 1][pos];
    const bool some = s != 0.0f;
    const float ls = lg2(s), inv_s = some ? ex2(-ls) : 0.0f;
    const float4* c4 = reinterpret_cast<const float4*>(S.sl2[(seg - 1) & 1] + 32 * half);
    f32x2 d[16];
    float over = -INFINITY;
    {
      const f32x2 s2 = pair_of(s, s), ls2 = pair_of(ls + kShift, ls + kShift);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 c = c4[i], m = m4[i];
        d[2 * i] = fma2(mul2(pair_of(__uint_as_float(xr[4 * i]), __uint_as_float(xr[4 * i + 1])),
                             pair_of(c.x, c.y)),
                        s2, sub2(ls2, pair_of(m.x, m.y)));
        d[2 * i + 1] = fma2(mul2(pair_of(__uint_as_float(xr[4 * i + 2]), __uint_as_float(xr[4 * i + 3])),
                                 pair_of(c.z, c.w)),
                            s2, sub2(ls2, pair_of(m.z, m.w)));
        const float2 u = both(d[2 * i]), v = both(d[2 * i + 1]);
        over = fmaxf(over, fmaxf(fmaxf(u.x, u.y), fmaxf(v.x, v.y)));
      }
    }
    const uint32_t mine = (__any_sync(0xffffffffu, over > kSlack + kShift) ? 1u : 0u) |
                          (__any_sync(0xffffffffu, some) ? 2u : 0u);
    if (lane == 0) S.flag[n & 1][half][qw] = static_cast<int32_t>(mine);
    named_bar(bar, 128);
    const int4 fl = *reinterpret_cast<const int4*>(S.flag[n & 1][half]);
    const int32_t flags = fl.x | fl.y | fl.z | fl.w;
    if ((flags & 1) || ((flags & 2) && !seen)) {
      // move references to the maxima so far: each head decides for itself, a
      // non-finite one keeps its reference
      part[qw * 32 + lane] = across(d, lane, [](float p, float q) { return fmaxf(p, q); });
      named_bar(bar, 128);
      float up = fmaxf(fmaxf(part[lane], part[32 + lane]), fmaxf(part[64 + lane], part[96 + lane])) - kShift;
      if ((seen && !(up > kSlack)) || !(fabsf(up) < INFINITY)) up = 0.0f;
      if (qw == 0) {
        S.m[32 * half + lane] += up;
        S.delta[32 * half + lane] = up;
        S.alpha[32 * half + lane] = seen ? ex2(-up) : 1.0f;
      }
      named_bar(bar, 128);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        d[i] = sub2(d[i], de2[i]);
        l[i] = mul2(l[i], al2[i]);
      }
      if (seen) {
        // the products of the units before are done: this unit's tile was
        // filled after them
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
          uint32_t o[32];
          const uint32_t at = tmem + lanes + kOCol + e * kHT + 32 * half;
          tmem_ld_32x32b_x32(at, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = __float_as_uint(__uint_as_float(o[i]) * S.alpha[32 * half + i]);
          tmem_st_32x32b_x32(at, o);
        }
        tmem_st_wait();
      }
      seen = true;
    }
    const f32x2 is2 = pair_of(inv_s, inv_s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = both(d[4 * i + k]);
        const float px = ex2(v.x), py = ex2(v.y);
        l[4 * i + k] = fma2(pair_of(px, py), is2, l[4 * i + k]);
        h[k] = pack_half2(px, py);
      }
      *reinterpret_cast<uint4*>(&S.p[sw(pos, 4 * half + i)]) = make_uint4(h[0], h[1], h[2], h[3]);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.pready);
    if (!w.last()) continue;

    // ---- the row tile's end in this CTA: totals, then the output
    part[qw * 32 + lane] = across(l, lane, [](float p, float q) { return p + q; });
#pragma unroll
    for (int i = 0; i < 16; ++i) l[i] = pair_of(0.0f, 0.0f);
    named_bar(bar, 128);
    const float total = (part[lane] + part[32 + lane]) + (part[64 + lane] + part[96 + lane]);
    const float lse2 = total == 0.0f ? -INFINITY : S.m[32 * half + lane] - kShift + log2f(total);
    named_bar(bar, 128);
    if (qw == 0) {
      S.alpha[32 * half + lane] = total == 0.0f ? 0.0f : 1.0f / total;
      S.m[32 * half + lane] = 0.0f;
    }
    named_bar(bar, 128);
    if (ok && !wait(&S.pvdone, n & 1)) ok = false;
    tc_fence_after();
    const int32_t h = w.g * kHT + 32 * half;          // first head of this half
    const bool whole = w.i == w.n - 1 && w.began_here();
    if (!ok) {
      // nothing to write
    } else if (whole) {
      if (qw == 0 && h + lane < a.H && a.lse)
        a.lse[static_cast<int64_t>(a.t0 + w.t) * a.H + h + lane] = lse2 * kLn2;
      uint16_t* orow = a.out + static_cast<int64_t>(a.t0 + w.t) * a.o_st + h * a.o_sh;
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(tmem + lanes + kOCol + e * kHT + 32 * half, o);
        tmem_ld_wait();
        const int v = value_of(e, pos);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float inv = S.alpha[32 * half + i];
          const __nv_bfloat16 y = __float2bfloat16_rn(__uint_as_float(o[i]) * inv);
          if (h + i < a.H) orow[i * a.o_sh + v] = *reinterpret_cast<const uint16_t*>(&y);
        }
      }
    } else {
      // a row tile that began in an earlier CTA goes to slot 0, one that goes
      // on in the next to slot 1
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (w.began_here() ? 1 : 0);
      if (qw == 0) a.piece_lse[slot * kHT + 32 * half + lane] = lse2;
      float* dst = a.piece + slot * kPieceRow + (32 * half) * kD;
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(tmem + lanes + kOCol + e * kHT + 32 * half, o);
        tmem_ld_wait();
        const int v = value_of(e, pos);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (h + i < a.H) dst[i * kD + v] = __uint_as_float(o[i]) * S.alpha[32 * half + i];
      }
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
  if (warp == kMmaWarp) tmem_alloc(&S.tmem_base, kTmemCols);
  if (tid == 0) {
    for (int h = 0; h < kHT; ++h) S.m[h] = 0.0f;
    for (int e = 0; e < 4; ++e) {
      mbar_init(&S.full[e], kLoadWarps);
      mbar_init(&S.empty[e], 1);
    }
    mbar_init(&S.qfull, kQueryWarps);
    mbar_init(&S.qempty, 1 + kSoftWarps);
    mbar_init(&S.sfull, 1);
    mbar_init(&S.pready, kSoftWarps);
    mbar_init(&S.pvdone, 1);
    mbar_init(&S.done, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  plan(a, S);                                 // ends with a barrier of the CTA
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  if (S.count > 0) {
    bool ok = true;
    if (warp < kSoftWarps) {
      setmaxnreg_inc<kSoftRegs>();
      ok = run_softmax(a, S, tmem);
    } else if (warp < kMmaWarp) {
      setmaxnreg_dec<kLoadRegs>();
      ok = run_loaders<kFp8>(a, S);
    } else {
      setmaxnreg_dec<kMmaRegs>();
      ok = warp == kMmaWarp ? run_mma(a, S, tmem) : run_queries(a, S);
    }
    if (!ok && lane == 0 && a.err) atomicOr(a.err, QLI_DEVERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// ---- joining the pieces ---------------------------------------------------------
// Block (c, k): the row tile that boundary c (between CTA c - 1 and CTA c) is
// the first to cut, rows 8k .. 8k+7 of it, a warp per row.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = kJoinThreads / 32;

__global__ void __launch_bounds__(kJoinThreads) merge_pieces_kernel(const Args a, int32_t ctas) {
  pdl_wait();
  const int lane = threadIdx.x & 31, c = blockIdx.x + 1;
  const int row = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
  const int64_t U = a.tok_start[a.tc];
  const int64_t uc = U * c / ctas, ub = U * (c - 1) / ctas;
  if (uc == ub || uc >= U) return;
  int32_t lo = 0, hi = a.tc - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (a.tok_start[mid] <= uc) lo = mid; else hi = mid - 1;
  }
  const int64_t base = a.tok_start[lo], n = (a.tok_start[lo + 1] - base) / a.hg;
  const int32_t g = static_cast<int32_t>((uc - base) / n);
  const int64_t start = base + g * n, end = start + n;
  const int32_t h = g * kHT + row;
  if (uc == start || ub > start || h >= a.H) return;   // not cut, or cut before
  // pieces: CTA c - 1's slot 1, then slot 0 of CTA c, c + 1, ... up to the end
  int32_t last = c;
  while (last + 1 < ctas && U * (last + 1) / ctas < end) ++last;
  const int32_t count = last - c + 2;
  const auto slot = [&](int32_t k) -> int64_t {
    return k == 0 ? 2 * static_cast<int64_t>(c - 1) + 1 : 2 * static_cast<int64_t>(c - 1 + k);
  };
  // a CTA without units left no piece
  const auto lse_of = [&](int32_t k) -> float {
    const int64_t cta = c - 1 + k;
    if (U * cta / ctas == U * (cta + 1) / ctas) return -INFINITY;
    return a.piece_lse[slot(k) * kHT + row];
  };
  float m = -INFINITY;
  for (int32_t k = lane; k < count; k += 32) m = fmaxf(m, lse_of(k));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float acc[16], total = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  for (int32_t k0 = 0; k0 < count; k0 += 32) {
    const float mine = k0 + lane < count ? lse_of(k0 + lane) : -INFINITY;
    const float wk = mine == -INFINITY ? 0.0f : ex2(mine - m);
    const int32_t some = min(32, count - k0);
#pragma unroll 4
    for (int32_t k = 0; k < some; ++k) {
      const float w = __shfl_sync(0xffffffffu, wk, k);
      if (w == 0.0f) continue;
      total += w;
      const float4* src = reinterpret_cast<const float4*>(
          a.piece + slot(k0 + k) * kPieceRow + static_cast<int64_t>(row) * kD);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = src[(i >> 1) * 64 + 2 * lane + (i & 1)];
        acc[4 * i] = fmaf(w, v.x, acc[4 * i]);
        acc[4 * i + 1] = fmaf(w, v.y, acc[4 * i + 1]);
        acc[4 * i + 2] = fmaf(w, v.z, acc[4 * i + 2]);
        acc[4 * i + 3] = fmaf(w, v.w, acc[4 * i + 3]);
      }
    }
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t t = a.t0 + lo;
  uint4* dst = reinterpret_cast<uint4*>(a.out + t * a.o_st + h * a.o_sh) + lane;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 y = __floats2bfloat162_rn(acc[8 * i + 2 * k] * inv, acc[8 * i + 2 * k + 1] * inv);
      w[k] = *reinterpret_cast<const uint32_t*>(&y);
    }
    dst[32 * i] = make_uint4(w[0], w[1], w[2], w[3]);
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
  if (a->bt_stride < 1 || a->num_pages < 1 || a->page_stride <= 0 || a->kv_offset < 0 ||
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
  d.cap = static_cast<int64_t>(a.bt_stride) * a.rows_per_page;
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
  d.hg = (a.H + kHT - 1) / kHT;
  return d;
}

// CTAs of a launch over tc tokens: one per SM, and no more than there can be
// units (known on the host for lists only).
int32_t ctas_for(const Args& d, int32_t tc, int sms) {
  if (d.idx == nullptr) return sms;
  const int64_t units = static_cast<int64_t>(tc) * d.hg * ((static_cast<int64_t>(d.K) - 1) / kPos + 1);
  return static_cast<int32_t>(units < sms ? units : sms);
}

// Workspace: the tokens' first units, then two pieces and their LSE per SM.
struct Layout {
  size_t piece, lse, total;
};
Layout layout_for(int sms) {
  Layout L{};
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  L.piece = up(sizeof(int64_t) * (kChunkT + 1));
  L.lse = L.piece + up(sizeof(float) * 2 * static_cast<size_t>(sms) * kPieceRow);
  L.total = L.lse + up(sizeof(float) * 2 * static_cast<size_t>(sms) * kHT);
  return L;
}

template <bool kFp8>
cudaError_t launch(Args d, int sms, cudaStream_t s) {
  const auto kernel = kv_attn_kernel<kFp8>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), kSmemBytes,
                                    g_smem_kv_attn[kFp8 ? 1 : 0]);
  for (d.t0 = 0; e == cudaSuccess && d.t0 < d.T; d.t0 += kChunkT) {
    d.tc = d.T - d.t0 < kChunkT ? d.T - d.t0 : kChunkT;
    const int32_t ctas = ctas_for(d, d.tc, sms);
    kernel<<<static_cast<unsigned>(ctas), kThreads, kSmemBytes, s>>>(d);
    e = cudaGetLastError();
    if (e == cudaSuccess && ctas > 1)
      e = launch_pdl(merge_pieces_kernel,
                     dim3(static_cast<unsigned>(ctas - 1),
                          static_cast<unsigned>(((d.H < kHT ? d.H : kHT) + kJoinRows - 1) / kJoinRows)),
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
  d.tok_start = reinterpret_cast<int64_t*>(w);
  d.piece = reinterpret_cast<float*>(w + L.piece);
  d.piece_lse = reinterpret_cast<float*>(w + L.lse);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->quant_mode == QLI_QUANT_FP8 ? launch<true>(d, sms, s) : launch<false>(d, sms, s);
  return e == cudaSuccess ? QLI_OK : QLI_ERR_CUDA;
}

extern "C" int64_t qli_kv_attn_args_size(void) {
  return static_cast<int64_t>(sizeof(qli_kv_attn_args));
}
