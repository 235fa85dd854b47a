// Rows on their way to the indexer, the attention and the cache: the rotation of
// positions on its own (qli_rotate), and norm, rotation and one rounding in a
// single pass over queries (qli_prepare_q) or over new cache rows, which go into
// their page slots (qli_append_kv).
//
//   norm      rms:   y = x / sqrt(mean x^2 + eps) * w
//             layer: y = (x - mean x) / sqrt(mean (x - mean x)^2 + eps) * w + b
//   rotation  pair i of a row at position p, values (a, b):
//             (a cos t - b sin t, b cos t + a sin t) * magnitude,  t = 2 pi p f_i
//   rounding  BF16, or 8-bit codes under an FP16 scale (the writer's, applied to
//             the FP32 values)
// Statistics and products are FP32. The angle is exact before it becomes FP32:
// f_i is a whole number of 2^-64 turns, so p f_i modulo 2^64 is the fraction of a
// turn whatever the position (an FP32 product would be 0.06 rad off at 10^6), and
// its top 32 bits are exact in 2^-32 turns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstring>

#include "qli_codes.cuh"
#include "qli_internal.h"

namespace qli {
namespace rows {
namespace {

constexpr int kThreads = 128;
constexpr int kKvRow = 512, kIndexRow = 128;
constexpr int64_t kMostRows = int64_t{1} << 30;   // of a call: row numbers and a block's beyond are 32 bits
constexpr int32_t kMostValues = 1 << 16;          // of a row that is rotated

// A rotation: pairs of a row's values from unit `o8` on (units are 8 values).
struct Turn {
  int32_t pairs, half, o8;
  uint32_t per_pair;                       // 2^32 / pairs, rounded up
  float scale, scale_lo;                   // the magnitude, in two numbers
  int32_t inverse;
  uint64_t turns[QLI_ROTARY_PAIRS];
};

struct Prep {
  int32_t norm;
  float eps;
  const float *weight, *bias;
  Turn turn;
};

// Cosine and sine of 2^-32 `frac` turns, times the magnitude. Within an eighth of a turn
// of the nearest quarter, |t| <= pi / 4, the Taylor series up to t^9 and t^10 leave 2^-29
// and 2^-33. The angle is t + e and the magnitude has two parts, so that little more than
// the last rounding is off (2^-24 without them, which moved twice as many 8-bit codes over
// the borders of their steps).
__device__ __forceinline__ void turn_of(uint32_t frac, const Turn& w, float& c, float& s) {
  constexpr float kHi = 1.4629181200e-09f, kLo = -4.0709402679e-17f;   // 2 pi / 2^32
  const uint32_t quarter = (frac + 0x20000000u) >> 30;
  const int32_t rest = static_cast<int32_t>(frac - (quarter << 30));
  const float hi = static_cast<float>(rest), lo = static_cast<float>(rest - static_cast<int32_t>(hi));
  const float t = hi * kHi, e = fmaf(hi, kHi, -t) + fmaf(hi, kLo, lo * kHi);
  const float t2 = t * t, t2e = fmaf(t, t, -t2);
  float p = fmaf(t2, 1.0f / 362880.0f, -1.0f / 5040.0f);
  p = fmaf(p, t2, 1.0f / 120.0f);
  p = fmaf(p, t2, -1.0f / 6.0f);
  float q = fmaf(t2, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  q = fmaf(q, t2, -1.0f / 720.0f);
  q = fmaf(q, t2, 1.0f / 24.0f);
  // sin = t + sin_r, cos = one + cos_r, where one is 1 - t2 / 2 rounded
  const float sin_r = fmaf(t * t2, p, fmaf(-0.5f * t2, e, e));
  const float one = 1.0f - 0.5f * t2;
  const float cos_r = fmaf(t2 * t2, q, ((1.0f - one) - 0.5f * t2) - fmaf(t, e, 0.5f * t2e));
  const float sin_t = fmaf(w.scale, t, fmaf(w.scale, sin_r, w.scale_lo * t));
  const float cos_t = fmaf(w.scale, one, fmaf(w.scale, cos_r, w.scale_lo * one));
  const float a = quarter & 1u ? sin_t : cos_t, b = quarter & 1u ? cos_t : sin_t;
  c = (quarter + 1u) & 2u ? -a : a;
  s = ((quarter >> 1) & 1u) != static_cast<uint32_t>(w.inverse) ? -b : b;
}

// (cos, sin) times the magnitude of the tokens t0 .. t0 + n, two pairs to a float4. The
// pairs of a unit (four neighbouring ones, or eight of which it holds one half) are a
// column: float4 i of unit u of a token at kColumns i + u, so that lanes side by side
// read side by side. In the order of the pairs they met in the same banks, four to
// eight at a time: 3561 tokens of 64 heads x 128, all rotated by halves, to INT8 took 45 us
// where they take 26.
constexpr int kTokenEntries = QLI_ROTARY_PAIRS;       // of the table, whatever the number of pairs
constexpr int64_t kTableBytes = 16 * 1024;            // of a table at most: 32 tokens
template <bool kHalf>
constexpr int kColumns = kHalf ? QLI_ROTARY_PAIRS / 8 : QLI_ROTARY_PAIRS / 4;
__device__ __forceinline__ int32_t table_place(const Turn& w, int32_t pair) {
  return w.half ? 2 * (((pair & 7) >> 1) * kColumns<true> + (pair >> 3)) + (pair & 1)
                : 2 * (((pair & 3) >> 1) * kColumns<false> + (pair >> 2)) + (pair & 1);
}
__device__ __forceinline__ void fill_table(float2* table, const Turn& w, const int32_t* positions,
                                           int32_t t0, int32_t n) {
#pragma unroll 1
  for (uint32_t i = threadIdx.x; i < static_cast<uint32_t>(n * w.pairs); i += kThreads) {
    const uint32_t t = __umulhi(i, w.per_pair), p = i - t * w.pairs;
    // by its generic address: lanes that index the constant bank apart take turns
    uint64_t f;
    asm volatile("ld.u64 %0, [%1];" : "=l"(f) : "l"(w.turns + p));
    const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(__ldg(positions + t0 + t))) * f;
    float s, c;
    turn_of(static_cast<uint32_t>(frac >> 32), w, c, s);
    table[t * kTokenEntries + table_place(w, p)] = make_float2(c, s);
  }
}

// Two FP32 numbers in one register pair, and the packed operations on them.
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
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

constexpr f32x2 kOnes = 0x3f8000003f800000ull;

// Eight values of a row, in pairs of neighbours.
struct Unit {
  f32x2 p[4];
};

__device__ __forceinline__ Unit unpack8(const uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  Unit u;
#pragma unroll
  for (int i = 0; i < 4; ++i) u.p[i] = pair_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return u;
}

__device__ __forceinline__ uint4 pack8(const Unit& u) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = both(u.p[i]);
    const __nv_bfloat162 p = __floats2bfloat162_rn(x.x, x.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four neighbouring pairs in one unit, column `u`.
__device__ __forceinline__ void turn_neighbours(Unit& x, const float2* cs, int u) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float4 t = reinterpret_cast<const float4*>(cs)[k * kColumns<false> + u];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float c = i ? t.z : t.x, s = i ? t.w : t.y;
      f32x2& p = x.p[2 * k + i];
      const float2 v = both(p);
      p = fma2(pair_of(-v.y, v.x), pair_of(s, s), mul2(p, pair_of(c, c)));
    }
  }
}

// Eight values and the eight that are their pairs' other halves (`w`), column `u`:
// a cos + sign w sin, the sign -1 for first halves and 1 for second.
__device__ __forceinline__ void turn_half(Unit& x, const Unit& w, const float2* cs, int u, float sign) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = reinterpret_cast<const float4*>(cs)[i * kColumns<true> + u];
    x.p[i] = fma2(mul2(w.p[i], pair_of(sign, sign)), pair_of(t.y, t.w), mul2(x.p[i], pair_of(t.x, t.z)));
  }
}

// ---- a row in the registers of its lanes --------------------------------------
// G = D / 16 lanes have a row: lane l units l and l + G (eight values each), so a
// warp instruction loads or stores 16 G contiguous bytes of each of its rows.
template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The lane's values of a weight or bias vector: out of L1, which holds them for every
// row; kept in registers they would cost more warps than they save loads.
template <int G>
__device__ __forceinline__ Unit vector_of(const float* from, int at) {
  Unit u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(from) + 2 * at + i);
    u.p[2 * i] = pair_of(v.x, v.y);
    u.p[2 * i + 1] = pair_of(v.z, v.w);
  }
  return u;
}

// Under an eps that does not cover them, squares of values below 2^-63 leave FP32's range.
// Rows up to 2^-40 are taken 2^90 times as large then: 2^50 at most, and from 2^-43 (the
// smallest BF16 number) on. Of others a value is a multiple of 2^-48, or a mean at least
// 2^-57 off some value. Returns the row's eps.
constexpr float kSmallEps = 7.888609052e-31f;         // 2^-100
bool small_eps(const Prep& p) { return p.norm != QLI_NORM_NONE && p.eps < kSmallEps; }
template <int G>
__device__ __forceinline__ float enlarge(Unit (&v)[2], float eps) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = both(v[i >> 2].p[i & 3]);
    m = fmaxf(fmaxf(m, fabsf(x.x)), fabsf(x.y));
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float up = m < 0x1p-40f ? 0x1p90f : 1.0f;
  const f32x2 up2 = pair_of(up, up);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i >> 2].p[i & 3] = mul2(v[i >> 2].p[i & 3], up2);
  return eps * up * up;
}

template <int G, int kNorm>
__device__ __forceinline__ void normalise(Unit (&v)[2], const Prep& p, int l, float eps) {
  constexpr float kInv = 1.0f / (16 * G);
  if constexpr (kNorm == QLI_NORM_LAYER) {
    f32x2 s = add2(v[0].p[0], v[1].p[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s = add2(s, add2(v[0].p[i], v[1].p[i]));
    const float2 e = both(s);
    const float mean = row_sum<G>(e.x + e.y) * -kInv;
    const f32x2 m = pair_of(mean, mean);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i >> 2].p[i & 3] = add2(v[i >> 2].p[i & 3], m);
  }
  f32x2 s = mul2(v[0].p[0], v[0].p[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) s = fma2(v[i >> 2].p[i & 3], v[i >> 2].p[i & 3], s);
  const float2 e = both(s);
  // with one step of Newton's, since what is off here moves the whole row
  const float x = fmaf(row_sum<G>(e.x + e.y), kInv, eps), y = rsqrtf(x);
  const float r = y > 0.0f && y < INFINITY ? fmaf(0.5f * y, fmaf(-x * y, y, 1.0f), y) : y;
  const f32x2 r2 = pair_of(r, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i >> 2].p[i & 3] = mul2(v[i >> 2].p[i & 3], r2);
  if (!p.weight && !(kNorm == QLI_NORM_LAYER && p.bias)) return;
  const Unit ones = {{kOnes, kOnes, kOnes, kOnes}};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Unit w = p.weight ? vector_of<G>(p.weight, l + k * G) : ones;
    if (kNorm == QLI_NORM_LAYER && p.bias) {
      const Unit b = vector_of<G>(p.bias, l + k * G);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[k].p[i] = fma2(v[k].p[i], w.p[i], b.p[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[k].p[i] = mul2(v[k].p[i], w.p[i]);
    }
  }
}

// `cs`: the row's token in the table.
enum : int { kNeighbours = 0, kHalves = 1, kOwnHalves = 2 };   // the last: pairs half a row apart, in one lane
constexpr int kAny = -1;                               // of layouts and norms: see Rows
template <int G, int kLayout>
__device__ __forceinline__ void turn_row(Unit (&v)[2], const Turn& w, const float2* cs, int l) {
  const int r8 = w.pairs / 4;
  if constexpr (kLayout == kNeighbours) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int u = l + k * G - w.o8;
      if (u >= 0 && u < r8) turn_neighbours(v[k], cs, u);
    }
    return;
  }
  if constexpr (kLayout == kOwnHalves) {
    const Unit was = v[0];
    turn_half(v[0], v[1], cs, l, -1.0f);
    turn_half(v[1], was, cs, l, 1.0f);
    return;
  }
  // a value's partner is h8 units away, in another lane or in this one's other
  // unit; the slots that hold part of the rotation are the same for every lane
  const int h8 = r8 / 2;
  const bool slot0 = w.o8 < G, slot1 = w.o8 + r8 > G;
  const auto partner = [&](int u) { return u < 0 || u >= r8 ? l : (u < h8 ? u + h8 : u - h8) + w.o8; };
  const auto turn = [&](Unit& x, const Unit& y, int u) {
    if (u >= 0 && u < r8) turn_half(x, y, cs, u < h8 ? u : u - h8, u < h8 ? -1.0f : 1.0f);
  };
  Unit other[2];
  if (slot0 && slot1) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int from = partner(l + k * G - w.o8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 a = __shfl_sync(0xffffffffu, v[0].p[i], from & (G - 1), G);
        const f32x2 b = __shfl_sync(0xffffffffu, v[1].p[i], from & (G - 1), G);
        other[k].p[i] = from < G ? a : b;
      }
    }
    turn(v[0], other[0], l - w.o8);
    turn(v[1], other[1], l + G - w.o8);
    return;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k ? !slot1 : !slot0) continue;
    const int u = l + k * G - w.o8, from = partner(u) & (G - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) other[k].p[i] = __shfl_sync(0xffffffffu, v[k].p[i], from, G);
    turn(v[k], other[k], u);
  }
}

// The largest of three. Of KV rows NaN is above all, as for the KV writer: the scale is NaN
// then, and so is what attends to the row (without that a norm over a NaN leaves a row of
// zeros). The quantisers of queries and index K pass over it.
template <int G>
__device__ __forceinline__ float largest(float a, float b, float c) {
  if constexpr (16 * G != kKvRow) return fmaxf(fmaxf(a, b), c);
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The row's codes and the FP16 bits of its scale: s = FP16(max |x| / Q), code(x / s),
// the quotient as the other writers take it (qli_codes.cuh), two at a time. E4M3 has two
// zeros, and the quotient's is x's: the correction step ends in +0 where x / s is a zero, so
// it works on -x / s, whose zeros are +0 then for x < 0 and -0 for x > 0, and the codes'
// signs are turned over (4096 tokens of 64 heads: 23.1 us, 22.8 without).
template <int G, bool kFp8>
__device__ __forceinline__ uint16_t quantise(const Unit (&v)[2], uint2 (&codes)[2]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = both(v[i >> 2].p[i & 3]);
    m = largest<G>(m, fabsf(x.x), fabsf(x.y));
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) m = largest<G>(m, m, __shfl_xor_sync(0xffffffffu, m, o));
  const uint16_t sb = scale_bits_of<kFp8>(m);
  const float sf = __half2float(__ushort_as_half(sb));
  codes[0] = codes[1] = make_uint2(0u, 0u);
  if (sf == 0.0f) return 0u;
  constexpr float kSign = kFp8 ? -1.0f : 1.0f;
  const float y = kSign * __frcp_rn(sf);
  const f32x2 y2 = pair_of(y, y), s2 = pair_of(-kSign * sf, -kSign * sf);
  // A scale that is a normal number is within 2^-11 of amax / Q, so that quotients end
  // at Q and a fraction. A subnormal one may be smaller, and the largest one cuts.
  const bool clamp = !kFp8 && (sb < 0x0400u || sb == 0x7bffu);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f32x2 q[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f32x2 x = v[k].p[2 * j + i], q0 = mul2(x, y2);
        q[i] = fma2(fma2(q0, s2, x), y2, q0);
      }
      if constexpr (kFp8) {
        const float2 lo = both(q[0]), hi = both(q[1]);
        w[j] = (e4m3x2_of(lo.x, lo.y) | (e4m3x2_of(hi.x, hi.y) << 16)) ^ 0x80808080u;
      } else {
        if (clamp) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 x = both(q[i]);
            q[i] = pair_of(fminf(fmaxf(x.x, -127.0f), 127.0f), fminf(fmaxf(x.y, -127.0f), 127.0f));
          }
        }
        // adding 1.5 * 2^23 rounds to an integer, ties to even, in the low bits
        const f32x2 magic = pair_of(12582912.0f, 12582912.0f);
        const float2 lo = both(add2(q[0], magic)), hi = both(add2(q[1], magic));
        w[j] = __byte_perm(__byte_perm(__float_as_uint(lo.x), __float_as_uint(lo.y), 0x0040),
                           __byte_perm(__float_as_uint(hi.x), __float_as_uint(hi.y), 0x0040), 0x5410);
      }
    }
    codes[k] = make_uint2(w[0], w[1]);
  }
  return sb;
}

// ---- where rows come from and go ------------------------------------------------
// Quotients of numbers below 2^31: with 2^s >= d and m = ceil(2^(31 + s) / d), m d is at
// most 2^s over 2^(31 + s), which moves r m / 2^(31 + s) by less than 1 / d.
struct Divide {
  uint32_t m;
  int32_t shift;                           // s - 1; -1: by one
  __device__ __forceinline__ int32_t operator()(int32_t r) const {
    return shift < 0 ? r : static_cast<int32_t>(__umulhi(static_cast<uint32_t>(r), m) >> shift);
  }
};
Divide divide_by(int32_t d) {
  int32_t s = 0;
  while ((int64_t{1} << s) < d) ++s;
  return Divide{static_cast<uint32_t>(((uint64_t{1} << (31 + s)) + static_cast<uint64_t>(d) - 1) / static_cast<uint64_t>(d)),
                s - 1};
}

struct DenseIn {
  const uint16_t* x;
  int64_t st, sh;
  int32_t H;
  Divide by_H;
  __device__ __forceinline__ int32_t token(int32_t r) const { return by_H(r); }
  __device__ __forceinline__ const uint16_t* row(int32_t r, int32_t t) const {
    return x + t * st + (r - t * H) * sh;
  }
};

// One row a token.
struct FlatIn {
  const uint16_t* x;
  int64_t st;
  __device__ __forceinline__ int32_t token(int32_t r) const { return r; }
  __device__ __forceinline__ const uint16_t* row(int32_t r, int32_t) const { return x + r * st; }
};

// kMode: 0 BF16, QLI_QUANT_INT8 or QLI_QUANT_FP8.
template <int kMode>
struct DenseOut {
  uint8_t* out;
  int64_t st, sh;                          // bytes
  uint16_t* scale;                         // [T, H]
  int32_t H;
  struct Key {};
  __device__ __forceinline__ Key key(int32_t) const { return {}; }
  __device__ __forceinline__ uint8_t* dest(int32_t r, int32_t t, Key, uint16_t*& s) const {
    s = scale + r;
    return out + t * st + (r - t * H) * sh;
  }
};

// Page slots; a negative one is padding, one past the pool is flagged.
template <int kMode>
struct PagedOut {
  const int64_t* slot;
  uint8_t* cache;
  int64_t slots, page_stride, offset, scale_offset;
  int32_t log2R, row_bytes;
  uint32_t* err;
  typedef int64_t Key;
  __device__ __forceinline__ Key key(int32_t r) const { return __ldg(slot + r); }
  __device__ __forceinline__ uint8_t* dest(int32_t, int32_t, Key m, uint16_t*& s) const {
    if (m < 0) return nullptr;
    if (m >= slots) {
      if (err != nullptr) atomicOr(err, QLI_DEVERR_PAGE);
      return nullptr;
    }
    const int64_t row = m & ((int64_t{1} << log2R) - 1);
    uint8_t* p = cache + (m >> log2R) * page_stride;
    s = reinterpret_cast<uint16_t*>(p + scale_offset + row * 2);
    return p + offset + row * row_bytes;
  }
};

// Rows r0 .. end of a block, kThreads / G at a time: construct (loads the first ones),
// fill the table of the rows' tokens from `t0` on, synchronise, run
// (works on one set of rows while the next one loads). kSmall: under an eps that does not
// cover small rows; kernels of their own, since the others took up to 2% longer with a test
// of the eps and up to 5% with a loop beside theirs (registers).
template <int D, int kMode, bool kSmall, class In, class Out>
struct Rows {
  static constexpr int G = D / 16, kRows = kThreads / G;
  const In& in;
  const Out& out;
  const Prep& p;
  const int l;
  int32_t r;
  const int32_t end;
  uint4 raw[2];
  int32_t tok;
  typename Out::Key key;

  __device__ __forceinline__ Rows(const In& in_, const Out& out_, const Prep& p_, int32_t r0, int32_t end_)
      : in(in_), out(out_), p(p_), l(threadIdx.x & (G - 1)), r(r0 + static_cast<int32_t>(threadIdx.x) / G), end(end_) {
    load();
  }
  __device__ __forceinline__ void load() {
    // lanes past the end read the last row, so that every lane takes part in the sums
    const int32_t at = min(r, end - 1);
    tok = in.token(at);
    const uint4* src = reinterpret_cast<const uint4*>(in.row(at, tok)) + l;
    raw[0] = src[0];                       // coherent: the output may be the input
    raw[1] = src[G];
    key = out.key(at);
  }
  __device__ __forceinline__ void run(const float2* table, int32_t t0) {
    if constexpr (kSmall) run_all<kAny, kAny>(table, t0);
    else if (!p.turn.half) run_norm<kNeighbours>(table, t0);
    else if (p.turn.pairs == 8 * G) run_norm<kOwnHalves>(table, t0);
    else run_norm<kHalves>(table, t0);
  }
  template <int kLayout>
  __device__ __forceinline__ void run_norm(const float2* table, int32_t t0) {
    if (p.norm == QLI_NORM_RMS) run_all<kLayout, QLI_NORM_RMS>(table, t0);
    else if (p.norm == QLI_NORM_LAYER) run_all<kLayout, QLI_NORM_LAYER>(table, t0);
    else run_all<kLayout, QLI_NORM_NONE>(table, t0);
  }
  // kAny: any layout and norm.
  template <int kLayout, int kNorm>
  __device__ __forceinline__ void run_all(const float2* table, int32_t t0) {
    // the same number of turns for every thread of the block
    const int32_t first = r - static_cast<int32_t>(threadIdx.x) / G;
#pragma unroll 1
    for (int32_t n = first; n < end; n += kRows) {
      Unit v[2] = {unpack8(raw[0]), unpack8(raw[1])};
      const int32_t t = tok, at = r;
      const typename Out::Key to = key;
      r += kRows;
      if (n + kRows < end) load();
      const float2* cs = table + (t - t0) * kTokenEntries;
      if constexpr (kNorm == kAny) {
        if (p.norm != QLI_NORM_NONE) {
          const float eps = p.eps < kSmallEps ? enlarge<G>(v, p.eps) : p.eps;
          if (p.norm == QLI_NORM_RMS) normalise<G, QLI_NORM_RMS>(v, p, l, eps);
          else normalise<G, QLI_NORM_LAYER>(v, p, l, eps);
        }
        if (p.turn.pairs && p.turn.half) turn_row<G, kHalves>(v, p.turn, cs, l);
        else if (p.turn.pairs) turn_row<G, kNeighbours>(v, p.turn, cs, l);
      } else {
        if constexpr (kNorm != QLI_NORM_NONE) normalise<G, kNorm>(v, p, l, p.eps);
        if (p.turn.pairs) turn_row<G, kLayout>(v, p.turn, cs, l);
      }
      uint16_t* scale = nullptr;
      if constexpr (kMode == 0) {
        uint8_t* dst = at < end ? out.dest(at, t, to, scale) : nullptr;
        if (dst == nullptr) continue;
        reinterpret_cast<uint4*>(dst)[l] = pack8(v[0]);
        reinterpret_cast<uint4*>(dst)[l + G] = pack8(v[1]);
      } else {
        uint2 codes[2];
        const uint16_t sb = quantise<G, kMode == QLI_QUANT_FP8>(v, codes);
        uint8_t* dst = at < end ? out.dest(at, t, to, scale) : nullptr;
        if (dst == nullptr) continue;
        reinterpret_cast<uint2*>(dst)[l] = codes[0];
        reinterpret_cast<uint2*>(dst)[l + G] = codes[1];
        if (l == 0) *scale = sb;
      }
    }
  }
};

// Tokens that `count` rows in a row can belong to, of `rows` with H a token.
int64_t tokens_of(int64_t count, int64_t rows, int64_t H) {
  const int64_t in = rows < count ? rows : count;
  const int64_t n = (in - 2 + H) / H + 1;
  return n < in ? n : in;
}

// Blocks an SM holds, by way of the registers: 8 with codes (64 registers a thread: half
// again as many without spills, and fewer with more of them, took 8% and 5% longer), 9
// with BF16 results. Blocks of 256 threads, half as many, took 2 to 5% longer.
constexpr int kBlocksPerSm = 8, kBlocksPerSmBf16 = 9;
// Sets of rows per block at most: the table and the start are paid once for them (with
// 2 the queries below took 7% longer, with 8 the same).
constexpr int kSets = 4;

// ---- queries --------------------------------------------------------------------
// Bound by HBM with BF16 results: 2047 tokens of 64 heads x 512 with RMS norm and a
// rotated tail (268 MB) take 43 us, 6.2 TB/s. With codes by the instructions, some 16 a
// value: 4096 tokens of 64 heads x 128 to E4M3 (101 MB) take 23.1 us, 4.4 TB/s, with 68%
// of the issue slots taken. One set of rows a block, without the next one in flight,
// took 59 and 32 us; the norm's and the layout's branches inside the loop 51 and 26.
template <int D, int kMode, bool kSmall>
__global__ void __launch_bounds__(kThreads, kMode == 0 ? kBlocksPerSmBf16 : kBlocksPerSm)
    prepare_kernel(const __grid_constant__ Prep p, DenseIn in, DenseOut<kMode> out, const int32_t* positions,
                   int32_t rows, int32_t block_rows) {
  extern __shared__ float4 table4[];
  float2* table = reinterpret_cast<float2*>(table4);
  const int32_t r0 = static_cast<int32_t>(blockIdx.x) * block_rows, end = min(rows - r0, block_rows) + r0;
  Rows<D, kMode, kSmall, DenseIn, DenseOut<kMode>> work(in, out, p, r0, end);
  const int32_t t0 = in.token(r0);
  if (p.turn.pairs) {
    fill_table(table, p.turn, positions, t0, in.token(end - 1) - t0 + 1);
    __syncthreads();
  }
  work.run(table, t0);
}

template <int D, int kMode>
cudaError_t launch_prepare(const Prep& p, const DenseIn& in, const DenseOut<kMode>& out,
                           const int32_t* positions, int32_t rows, int sms, cudaStream_t s) {
  constexpr int kRows = kThreads / (D / 16);
  const int64_t sets = (static_cast<int64_t>(rows) - 1) / kRows + 1;
  int64_t each = sets / (static_cast<int64_t>(sms) * kBlocksPerSm);
  each = each < 1 ? 1 : each > kSets ? kSets : each;
  const auto bytes = [&] {
    return p.turn.pairs ? static_cast<int64_t>(sizeof(float2)) * tokens_of(each * kRows, rows, in.H) * kTokenEntries : 0;
  };
  while (each > 1 && bytes() > kTableBytes) --each;
  const int32_t block_rows = static_cast<int32_t>(each) * kRows;
  const size_t smem = static_cast<size_t>(bytes());
  const auto kernel = small_eps(p) ? prepare_kernel<D, kMode, true> : prepare_kernel<D, kMode, false>;
  kernel<<<static_cast<unsigned>((rows - 1) / block_rows + 1), kThreads, smem, s>>>(p, in, out, positions, rows,
                                                                                    block_rows);
  return cudaGetLastError();
}

// ---- cache rows -----------------------------------------------------------------
template <int kKv, int kIndex>
struct AppendArgs {
  Prep kv, index;
  FlatIn kv_in, index_in;
  PagedOut<kKv> kv_out;
  PagedOut<kIndex> index_out;
  const int32_t* positions;
  int32_t n, block_rows;
  int32_t index_table;                     // entry of the table where the index K's begins; 0: the same one
};

// A block takes a few tokens: their KV rows, then their index K rows, by one table where
// they turn alike. Bound by the instructions, some 450 of a warp a token: 65536 tokens to
// E4M3 (127 MB) take 38.6 us, 3.3 TB/s; separate blocks for the two kinds, each with its
// table, took 54.
template <int kKv, int kIndex, bool kSmall>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    append_kernel(const __grid_constant__ AppendArgs<kKv, kIndex> a) {
  extern __shared__ float4 table4[];
  float2* table = reinterpret_cast<float2*>(table4);
  const int32_t r0 = static_cast<int32_t>(blockIdx.x) * a.block_rows, end = min(a.n - r0, a.block_rows) + r0;
  const auto turns = [&] {
    if (a.kv.turn.pairs) fill_table(table, a.kv.turn, a.positions, r0, end - r0);
    if (a.index.turn.pairs && (a.index_table || !a.kv.turn.pairs))
      fill_table(table + a.index_table, a.index.turn, a.positions, r0, end - r0);
    __syncthreads();
  };
  if (a.kv_in.x) {
    Rows<kKvRow, kKv, kSmall, FlatIn, PagedOut<kKv>> work(a.kv_in, a.kv_out, a.kv, r0, end);
    turns();
    work.run(table, r0);
  } else {
    turns();
  }
  if (a.index_in.x) {
    Rows<kIndexRow, kIndex, kSmall, FlatIn, PagedOut<kIndex>> work(a.index_in, a.index_out, a.index, r0, end);
    work.run(table + a.index_table, r0);
  }
}

// ---- rotation alone ---------------------------------------------------------------
// A thread has two units of a row, h8 apart: eight pairs of the half layout, or
// two times four neighbouring ones. In place nothing else of the row is touched;
// otherwise the block copies the rest of its rows. Bound by HBM: 4093 tokens of 33 heads
// x 512 out of wider rows (277 MB) take 44.8 us, 6.2 TB/s; 64 tokens of 64 heads in
// place 1.8 us, the time of a launch.
struct RotateArgs {
  const uint16_t* x;
  int64_t x_st, x_sh;
  uint16_t* out;
  int64_t o_st, o_sh;
  const int32_t* positions;
  int32_t rows, H, units, block_rows;      // units of a row (0: in place), rows of a block
  Turn turn;
};

__global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ RotateArgs a) {
  extern __shared__ float4 table4[];
  float2* table = reinterpret_cast<float2*>(table4);
  const int32_t r0 = static_cast<int32_t>(blockIdx.x) * a.block_rows;
  const int32_t n = min(a.block_rows, a.rows - r0), t0 = r0 / a.H;
  const int h8 = a.turn.pairs / 8;
  const int32_t mine = static_cast<int32_t>(threadIdx.x) / h8, u = a.turn.o8 + static_cast<int32_t>(threadIdx.x) % h8;
  const bool some = mine < n;
  const int32_t r = r0 + mine, t = r / a.H;
  uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
  if (some) {
    const uint4* src = reinterpret_cast<const uint4*>(a.x + t * a.x_st + (r - t * a.H) * a.x_sh) + u;
    v0 = *src;
    v1 = src[h8];
  }
  fill_table(table, a.turn, a.positions, t0, (r0 + n - 1) / a.H - t0 + 1);
  __syncthreads();
  if (some) {
    Unit x = unpack8(v0), y = unpack8(v1);
    const int w = u - a.turn.o8;
    const float2* cs = table + (t - t0) * kTokenEntries;
    if (a.turn.half) {
      const Unit was = x;
      turn_half(x, y, cs, w, -1.0f);
      turn_half(y, was, cs, w, 1.0f);
    } else {
      turn_neighbours(x, cs, w);
      turn_neighbours(y, cs, w + h8);
    }
    uint4* dst = reinterpret_cast<uint4*>(a.out + t * a.o_st + (r - t * a.H) * a.o_sh) + u;
    *dst = pack8(x);
    dst[h8] = pack8(y);
  }
  if (a.units == 0) return;
  const int rest = a.units - 2 * h8;
#pragma unroll 4
  for (int32_t i = threadIdx.x; i < n * rest; i += kThreads) {
    const int32_t row = i / rest, c = i - row * rest, at = c < a.turn.o8 ? c : c + 2 * h8;
    const int32_t rr = r0 + row, tt = rr / a.H;
    reinterpret_cast<uint4*>(a.out + tt * a.o_st + (rr - tt * a.H) * a.o_sh)[at] =
        __ldg(reinterpret_cast<const uint4*>(a.x + tt * a.x_st + (rr - tt * a.H) * a.x_sh) + at);
  }
}

// ---- host -------------------------------------------------------------------------
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

qli_status check_rotary(const qli_rotary& r, int64_t width) {
  if (r.layout != QLI_ROTARY_INTERLEAVED && r.layout != QLI_ROTARY_HALF) return QLI_ERR_UNSUPPORTED;
  if (r.pairs < 8 || r.pairs > QLI_ROTARY_PAIRS || r.pairs % 8 != 0 || r.offset % 8 != 0)
    return QLI_ERR_UNSUPPORTED;
  if (r.offset < 0 || r.offset + 2 * static_cast<int64_t>(r.pairs) > width ||
      !std::isfinite(static_cast<float>(r.magnitude)))
    return QLI_ERR_INVALID_ARG;
  return QLI_OK;
}

Turn make_turn(const qli_rotary& r, bool inverse) {
  Turn w{};
  w.pairs = r.pairs;
  w.half = r.layout == QLI_ROTARY_HALF ? 1 : 0;
  w.o8 = r.offset / 8;
  w.per_pair = static_cast<uint32_t>(((uint64_t{1} << 32) - 1) / static_cast<uint32_t>(r.pairs) + 1);
  const double scale = inverse ? 1.0 / r.magnitude : r.magnitude;
  w.scale = static_cast<float>(scale);
  w.scale_lo = static_cast<float>(scale - static_cast<double>(w.scale));
  w.inverse = inverse ? 1 : 0;
  std::memcpy(w.turns, r.turns, sizeof(uint64_t) * static_cast<size_t>(r.pairs));
  return w;
}

qli_status check_prep(const qli_row_prep* p) {
  if (p == nullptr) return QLI_ERR_INVALID_ARG;
  if (p->norm != QLI_NORM_NONE && p->norm != QLI_NORM_RMS && p->norm != QLI_NORM_LAYER) return QLI_ERR_UNSUPPORTED;
  if ((p->norm == QLI_NORM_NONE && p->weight != nullptr) || (p->norm != QLI_NORM_LAYER && p->bias != nullptr))
    return QLI_ERR_INVALID_ARG;
  if (!std::isfinite(p->eps) || p->eps < 0.0f) return QLI_ERR_INVALID_ARG;
  if (!aligned(p->weight, 16) || !aligned(p->bias, 16)) return QLI_ERR_ALIGNMENT;
  return p->rotary.pairs == 0 ? QLI_OK : check_rotary(p->rotary, p->width);
}

Prep make_prep(const qli_row_prep& p) {
  Prep d{};
  d.norm = p.norm;
  d.eps = p.eps;
  d.weight = p.weight;
  d.bias = p.bias;
  if (p.rotary.pairs) d.turn = make_turn(p.rotary, false);
  return d;
}

// Rows of `width` elements at these strides lie apart.
bool apart(int64_t T, int64_t H, int64_t st, int64_t sh, int64_t width) {
  if (T <= 1 && H <= 1) return true;
  if (T <= 1) return sh >= width;
  if (H <= 1) return st >= width;
  return (sh >= width && st >= (H - 1) * sh + width) || (st >= width && sh >= (T - 1) * st + width);
}

qli_status check_dense(const void* x, int64_t x_st, int64_t x_sh, int32_t T, int32_t H, int64_t width,
                       const void* out, int64_t o_st, int64_t o_sh, int64_t out_unit) {
  if (x == nullptr || out == nullptr || x_st < 0 || x_sh < 0) return QLI_ERR_INVALID_ARG;
  if (!aligned(x, 16) || x_st % 8 || x_sh % 8 || !aligned(out, 16) || o_st % out_unit || o_sh % out_unit)
    return QLI_ERR_ALIGNMENT;
  if (!apart(T, H, o_st, o_sh, width)) return QLI_ERR_INVALID_ARG;
  // in place: the same rows
  if (x == out && ((T > 1 && x_st != o_st) || (H > 1 && x_sh != o_sh))) return QLI_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * H > kMostRows) return QLI_ERR_UNSUPPORTED;
  return QLI_OK;
}

template <int kMode>
cudaError_t launch_width(const qli_prepare_args& a, const Prep& p, int32_t width, int sms, cudaStream_t s) {
  const DenseIn in{a.x, a.x_stride_t, a.x_stride_h, a.H, divide_by(a.H)};
  const int64_t unit = kMode == 0 ? 2 : 1;
  const DenseOut<kMode> out{static_cast<uint8_t*>(a.out), a.out_stride_t * unit, a.out_stride_h * unit, a.scale_out, a.H};
  const int32_t rows = a.T * a.H;
  if constexpr (kMode == 0) {
    if (width == 64) return launch_prepare<64, 0>(p, in, out, a.positions, rows, sms, s);
    if (width == 256) return launch_prepare<256, 0>(p, in, out, a.positions, rows, sms, s);
    if (width == 512) return launch_prepare<512, 0>(p, in, out, a.positions, rows, sms, s);
  }
  return launch_prepare<128, kMode>(p, in, out, a.positions, rows, sms, s);
}

// Tokens per block: enough for whole warps of index K rows while that leaves each SM two
// blocks, down to one set of KV rows. (12000 tokens: 12.8 us with 4 a block, 9.1 with 16;
// 1000: 4.3 and 6.2.)
constexpr int kMinBlocks = 2;
constexpr int kFewTokens = kThreads / (kKvRow / 16), kManyTokens = kThreads / (kIndexRow / 16);

template <int kKv, int kIndex>
cudaError_t launch_append(const qli_append_args& a, const qli_row_prep* kv, const qli_row_prep* index, int sms,
                          cudaStream_t s) {
  AppendArgs<kKv, kIndex> d{};
  d.positions = a.positions;
  d.n = static_cast<int32_t>(a.n);
  d.block_rows = kManyTokens;
  while (d.block_rows > kFewTokens && a.n < kMinBlocks * sms * static_cast<int64_t>(d.block_rows)) d.block_rows /= 2;
  const int64_t slots = a.num_pages * a.rows_per_page;
  const int32_t log2R = a.rows_per_page == 64 ? 6 : 7;
  const int64_t tokens = tokens_of(d.block_rows, a.n, 1);
  if (a.kv) {
    d.kv = make_prep(*kv);
    d.kv_in = FlatIn{a.kv, a.kv_stride};
    d.kv_out = PagedOut<kKv>{a.slot_mapping, a.cache, slots, a.page_stride, a.kv_offset, a.kv_scale_offset, log2R,
                             kKv == 0 ? 2 * kKvRow : kKvRow, a.err_word};
  }
  int64_t entries = d.kv.turn.pairs ? tokens * kTokenEntries : 0;
  if (a.index_k) {
    d.index = make_prep(*index);
    d.index_in = FlatIn{a.index_k, a.index_stride};
    d.index_out = PagedOut<kIndex>{a.slot_mapping, a.cache, slots, a.page_stride, a.k_offset, a.scale_offset, log2R,
                                   kIndexRow, a.err_word};
    const Turn &x = d.kv.turn, &y = d.index.turn;
    // the same angles, magnitude and layout: one table, whatever the offsets
    const bool same = x.pairs == y.pairs && x.half == y.half && x.scale == y.scale && x.scale_lo == y.scale_lo &&
                      std::memcmp(x.turns, y.turns, sizeof(x.turns)) == 0;
    if (!same) {
      d.index_table = static_cast<int32_t>(entries);
      entries += y.pairs ? tokens * kTokenEntries : 0;
    }
  }
  const auto kernel = small_eps(d.kv) || small_eps(d.index) ? append_kernel<kKv, kIndex, true>
                                                            : append_kernel<kKv, kIndex, false>;
  kernel<<<static_cast<unsigned>((a.n - 1) / d.block_rows + 1), kThreads,
           sizeof(float2) * static_cast<size_t>(entries), s>>>(d);
  return cudaGetLastError();
}

struct Span {
  int64_t at, bytes;
};

}  // namespace
}  // namespace rows
}  // namespace qli

extern "C" qli_status qli_rotate(const qli_rotate_args* a, const qli_rotary* rotary, void* stream) {
  using namespace qli::rows;
  if (a == nullptr || rotary == nullptr) return QLI_ERR_INVALID_ARG;
  if (a->T < 0 || a->H < 1) return QLI_ERR_INVALID_ARG;
  if (a->D < 16 || a->D > kMostValues || a->D % 8 != 0) return QLI_ERR_UNSUPPORTED;
  qli_status st = check_rotary(*rotary, a->D);
  if (st != QLI_OK) return st;
  if (a->inverse && !std::isfinite(static_cast<float>(1.0 / rotary->magnitude))) return QLI_ERR_INVALID_ARG;
  if (a->T == 0) return QLI_OK;
  st = check_dense(a->x, a->x_stride_t, a->x_stride_h, a->T, a->H, a->D, a->out, a->out_stride_t, a->out_stride_h, 8);
  if (st != QLI_OK) return st;
  if (a->positions == nullptr) return QLI_ERR_INVALID_ARG;
  if (!aligned(a->positions, 4)) return QLI_ERR_ALIGNMENT;
  int sms = 0;
  st = qli::device_sms(&sms);
  if (st != QLI_OK) return st;
  RotateArgs d{};
  d.x = a->x;
  d.x_st = a->x_stride_t;
  d.x_sh = a->x_stride_h;
  d.out = a->out;
  d.o_st = a->out_stride_t;
  d.o_sh = a->out_stride_h;
  d.positions = a->positions;
  d.rows = a->T * a->H;
  d.H = a->H;
  d.units = a->x == a->out ? 0 : a->D / 8;
  d.block_rows = kThreads / (rotary->pairs / 8);
  d.turn = make_turn(*rotary, a->inverse != 0);
  const auto bytes = [&] {
    return static_cast<int64_t>(sizeof(float2)) * tokens_of(d.block_rows, d.rows, a->H) * kTokenEntries;
  };
  while (bytes() > kTableBytes) d.block_rows /= 2;
  const size_t smem = static_cast<size_t>(bytes());
  rotate_kernel<<<static_cast<unsigned>((d.rows - 1) / d.block_rows + 1), kThreads, smem,
                  static_cast<cudaStream_t>(stream)>>>(d);
  return cudaGetLastError() == cudaSuccess ? QLI_OK : QLI_ERR_CUDA;
}

extern "C" qli_status qli_prepare_q(const qli_prepare_args* a, const qli_row_prep* prep, void* stream) {
  using namespace qli::rows;
  if (a == nullptr) return QLI_ERR_INVALID_ARG;
  qli_status st = check_prep(prep);
  if (st != QLI_OK) return st;
  const int32_t D = prep->width;
  if (D != 64 && D != 128 && D != 256 && D != 512) return QLI_ERR_UNSUPPORTED;
  if (a->quant_mode != 0 && a->quant_mode != QLI_QUANT_INT8 && a->quant_mode != QLI_QUANT_FP8)
    return QLI_ERR_UNSUPPORTED;
  if (a->quant_mode != 0 && D != kIndexRow) return QLI_ERR_UNSUPPORTED;
  if (a->T < 0 || a->H < 1) return QLI_ERR_INVALID_ARG;
  if (a->T == 0) return QLI_OK;
  st = check_dense(a->x, a->x_stride_t, a->x_stride_h, a->T, a->H, D, a->out, a->out_stride_t, a->out_stride_h,
                   a->quant_mode == 0 ? 8 : 16);
  if (st != QLI_OK) return st;
  if (prep->rotary.pairs != 0 && a->positions == nullptr) return QLI_ERR_INVALID_ARG;
  if (a->quant_mode != 0 && (a->scale_out == nullptr || static_cast<const void*>(a->x) == a->out))
    return QLI_ERR_INVALID_ARG;
  if (!aligned(a->positions, 4) || !aligned(a->scale_out, 2)) return QLI_ERR_ALIGNMENT;
  int sms = 0;
  st = qli::device_sms(&sms);
  if (st != QLI_OK) return st;
  const Prep p = make_prep(*prep);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->quant_mode == 0                ? launch_width<0>(*a, p, D, sms, s)
                        : a->quant_mode == QLI_QUANT_INT8 ? launch_width<QLI_QUANT_INT8>(*a, p, D, sms, s)
                                                          : launch_width<QLI_QUANT_FP8>(*a, p, D, sms, s);
  return e == cudaSuccess ? QLI_OK : QLI_ERR_CUDA;
}

extern "C" qli_status qli_append_kv(const qli_append_args* a, const qli_row_prep* kv_prep,
                                    const qli_row_prep* index_prep, void* stream) {
  using namespace qli::rows;
  if (a == nullptr) return QLI_ERR_INVALID_ARG;
  if (a->kv_mode != 0 && a->kv_mode != QLI_QUANT_INT8 && a->kv_mode != QLI_QUANT_FP8) return QLI_ERR_UNSUPPORTED;
  if (a->quant_mode != QLI_QUANT_INT8 && a->quant_mode != QLI_QUANT_FP8) return QLI_ERR_UNSUPPORTED;
  if (a->n < 0 || a->num_pages < 0) return QLI_ERR_INVALID_ARG;
  if (a->n == 0) return QLI_OK;
  if (a->n > kMostRows) return QLI_ERR_UNSUPPORTED;
  if (a->kv == nullptr && a->index_k == nullptr) return QLI_ERR_INVALID_ARG;
  if (a->cache == nullptr || a->slot_mapping == nullptr) return QLI_ERR_INVALID_ARG;
  const int32_t R = a->rows_per_page;
  if (R != 64 && R != 128) return QLI_ERR_UNSUPPORTED;
  if (a->page_stride <= 0) return QLI_ERR_INVALID_ARG;
  bool turns = false;
  // the parts of a page that the call writes: within it, and apart
  Span part[4];
  int parts = 0;
  if (a->kv != nullptr) {
    const qli_status st = check_prep(kv_prep);
    if (st != QLI_OK) return st;
    if (kv_prep->width != kKvRow) return QLI_ERR_UNSUPPORTED;
    if (a->n > 1 && a->kv_stride < kKvRow) return QLI_ERR_INVALID_ARG;
    turns |= kv_prep->rotary.pairs != 0;
    part[parts++] = Span{a->kv_offset, static_cast<int64_t>(R) * kKvRow * (a->kv_mode == 0 ? 2 : 1)};
    if (a->kv_mode != 0) part[parts++] = Span{a->kv_scale_offset, 2 * R};
    if (!aligned(a->kv, 16) || (a->n > 1 && a->kv_stride % 8) || a->kv_offset % 16 ||
        (a->kv_mode != 0 && a->kv_scale_offset % 2))
      return QLI_ERR_ALIGNMENT;
  }
  if (a->index_k != nullptr) {
    const qli_status st = check_prep(index_prep);
    if (st != QLI_OK) return st;
    if (index_prep->width != kIndexRow) return QLI_ERR_UNSUPPORTED;
    if (a->n > 1 && a->index_stride < kIndexRow) return QLI_ERR_INVALID_ARG;
    turns |= index_prep->rotary.pairs != 0;
    part[parts++] = Span{a->k_offset, static_cast<int64_t>(R) * kIndexRow};
    part[parts++] = Span{a->scale_offset, 2 * R};
    if (!aligned(a->index_k, 16) || (a->n > 1 && a->index_stride % 8) || a->k_offset % 16 || a->scale_offset % 2)
      return QLI_ERR_ALIGNMENT;
  }
  for (int i = 0; i < parts; ++i) {
    if (part[i].at < 0 || part[i].at > a->page_stride - part[i].bytes) return QLI_ERR_INVALID_ARG;
    for (int k = 0; k < i; ++k)
      if (part[i].at < part[k].at + part[k].bytes && part[k].at < part[i].at + part[i].bytes) return QLI_ERR_INVALID_ARG;
  }
  if (turns && a->positions == nullptr) return QLI_ERR_INVALID_ARG;
  if (!aligned(a->cache, 16) || a->page_stride % 16 || !aligned(a->slot_mapping, 8) || !aligned(a->positions, 4) ||
      !aligned(a->err_word, 4))
    return QLI_ERR_ALIGNMENT;
  int sms = 0;
  const qli_status st = qli::device_sms(&sms);
  if (st != QLI_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f8 = a->quant_mode == QLI_QUANT_FP8;
  cudaError_t e = cudaErrorInvalidValue;
  if (a->kv_mode == 0)
    e = f8 ? launch_append<0, QLI_QUANT_FP8>(*a, kv_prep, index_prep, sms, s)
           : launch_append<0, QLI_QUANT_INT8>(*a, kv_prep, index_prep, sms, s);
  else if (a->kv_mode == QLI_QUANT_INT8)
    e = f8 ? launch_append<QLI_QUANT_INT8, QLI_QUANT_FP8>(*a, kv_prep, index_prep, sms, s)
           : launch_append<QLI_QUANT_INT8, QLI_QUANT_INT8>(*a, kv_prep, index_prep, sms, s);
  else
    e = f8 ? launch_append<QLI_QUANT_FP8, QLI_QUANT_FP8>(*a, kv_prep, index_prep, sms, s)
           : launch_append<QLI_QUANT_FP8, QLI_QUANT_INT8>(*a, kv_prep, index_prep, sms, s);
  return e == cudaSuccess ? QLI_OK : QLI_ERR_CUDA;
}

extern "C" int64_t qli_rotary_size(void) { return static_cast<int64_t>(sizeof(qli_rotary)); }
extern "C" int64_t qli_row_prep_size(void) { return static_cast<int64_t>(sizeof(qli_row_prep)); }
extern "C" int64_t qli_rotate_args_size(void) { return static_cast<int64_t>(sizeof(qli_rotate_args)); }
extern "C" int64_t qli_prepare_args_size(void) { return static_cast<int64_t>(sizeof(qli_prepare_args)); }
extern "C" int64_t qli_append_args_size(void) { return static_cast<int64_t>(sizeof(qli_append_args)); }
