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
// its top 32 bits go to sincospif.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstring>

#include "qli_codes.cuh"
#include "qli_internal.h"

namespace qli {
namespace rows {
namespace {

constexpr int kThreads = 256;
constexpr int kKvRow = 512, kIndexRow = 128;

// A rotation: pairs of a row's values from unit `o8` on (units are 8 values).
struct Turn {
  int32_t pairs, half, o8;
  float cos_scale, sin_scale;              // the magnitude; sin's sign is the direction
  uint64_t turns[QLI_ROTARY_PAIRS];
};

struct Prep {
  int32_t norm;
  float eps;
  const float *weight, *bias;
  Turn turn;
};

// (cos, sin) times the magnitude of the tokens t0 .. t0 + n, by token and pair.
__device__ __forceinline__ void fill_table(float2* table, const Turn& w, const int32_t* positions,
                                           int32_t t0, int32_t n) {
#pragma unroll 1
  for (int32_t i = threadIdx.x; i < n * w.pairs; i += kThreads) {
    const int32_t t = i / w.pairs, p = i - t * w.pairs;
    const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(__ldg(positions + t0 + t))) * w.turns[p];
    float s, c;
    // 2^-31: half turns, as sincospif takes them
    sincospif(static_cast<float>(static_cast<int32_t>(frac >> 32)) * 4.656612873077393e-10f, &s, &c);
    table[i] = make_float2(c * w.cos_scale, s * w.sin_scale);
  }
}

__device__ __forceinline__ void unpack8(const uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four neighbouring pairs in one unit.
__device__ __forceinline__ void turn_neighbours(float (&x)[8], const float2* cs) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[2 * i], b = x[2 * i + 1];
    const float2 t = cs[i];
    x[2 * i] = a * t.x - b * t.y;
    x[2 * i + 1] = b * t.x + a * t.y;
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

template <int G>
__device__ __forceinline__ void normalise(float (&v)[2][8], const Prep& p, int l) {
  if (p.norm == QLI_NORM_NONE) return;
  constexpr float kInv = 1.0f / (16 * G);
  if (p.norm == QLI_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += v[i >> 3][i & 7];
    const float mean = row_sum<G>(s) * kInv;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i >> 3][i & 7] -= mean;
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s = fmaf(v[i >> 3][i & 7], v[i >> 3][i & 7], s);
  const float r = rsqrtf(row_sum<G>(s) * kInv + p.eps);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float w[8], b[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = 2 * (l + k * G) + i;
      const float4 one = make_float4(1.0f, 1.0f, 1.0f, 1.0f), zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      *reinterpret_cast<float4*>(w + 4 * i) = p.weight ? __ldg(reinterpret_cast<const float4*>(p.weight) + at) : one;
      *reinterpret_cast<float4*>(b + 4 * i) = p.bias ? __ldg(reinterpret_cast<const float4*>(p.bias) + at) : zero;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = fmaf(v[k][i] * r, w[i], b[i]);
  }
}

// `cs`: the row's token in the table.
template <int G>
__device__ __forceinline__ void turn_row(float (&v)[2][8], const Turn& w, const float2* cs, int l) {
  if (w.pairs == 0) return;
  const int r8 = w.pairs / 4;
  if (!w.half) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int u = l + k * G - w.o8;
      if (u >= 0 && u < r8) turn_neighbours(v[k], cs + 4 * u);
    }
    return;
  }
  // a value's partner is h8 units away, in another lane or in this one's other
  // unit; the slots that hold part of the rotation are the same for every lane
  const int h8 = r8 / 2;
  const bool slot0 = w.o8 < G, slot1 = w.o8 + r8 > G;
  float other[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!(k ? slot1 : slot0)) continue;
    const int u = l + k * G - w.o8;
    const int from = u < 0 || u >= r8 ? l : (u < h8 ? u + h8 : u - h8) + w.o8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = slot0 ? __shfl_sync(0xffffffffu, v[0][i], from & (G - 1), G) : 0.0f;
      const float b = slot1 ? __shfl_sync(0xffffffffu, v[1][i], from & (G - 1), G) : 0.0f;
      other[k][i] = from < G ? a : b;
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int u = l + k * G - w.o8;
    if (u < 0 || u >= r8) continue;
    const bool first = u < h8;
    const float2* t = cs + 8 * (first ? u : u - h8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 c = t[i];
      v[k][i] = first ? v[k][i] * c.x - other[k][i] * c.y : v[k][i] * c.x + other[k][i] * c.y;
    }
  }
}

// The row's codes and the FP16 bits of its scale: s = FP16(max |x| / Q), code(x / s).
template <int G, bool kFp8>
__device__ __forceinline__ uint16_t quantise(const float (&v)[2][8], uint2 (&codes)[2]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i >> 3][i & 7]));
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const uint16_t sb = scale_bits_of<kFp8>(m);
  const float sf = __half2float(__ushort_as_half(sb));
  codes[0] = codes[1] = make_uint2(0u, 0u);
  if (sf == 0.0f) return 0u;
  const float y = __frcp_rn(sf);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = quotient(v[k][4 * j + i], sf, y);
      if constexpr (kFp8) {
        w[j] = e4m3x2_of(q[0], q[1]) | (e4m3x2_of(q[2], q[3]) << 16);
      } else {
        // adding 1.5 * 2^23 rounds to an integer, ties to even, in the low bits
        uint32_t n[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          n[i] = __float_as_uint(__fadd_rn(fminf(fmaxf(q[i], -127.0f), 127.0f), 12582912.0f));
        w[j] = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
      }
    }
    codes[k] = make_uint2(w[0], w[1]);
  }
  return sb;
}

// ---- where rows come from and go ------------------------------------------------
struct DenseIn {
  const uint16_t* x;
  int64_t st, sh;
  int32_t H;
  __device__ __forceinline__ int32_t token(int32_t r) const { return r / H; }
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

// Rows r0 .. r0 + kDepth * kThreads / G of `rows`, those of a warp in flight
// together; the table of their tokens is made while they load.
template <int D, int kMode, int kDepth, class In, class Out>
__device__ __forceinline__ void pass(const In& in, const Out& out, const Prep& p,
                                     const int32_t* positions, int32_t r0, int32_t rows, float2* table) {
  constexpr int G = D / 16, kRows = kThreads / G;
  const int l = threadIdx.x & (G - 1), g = threadIdx.x / G;
  uint4 raw[kDepth][2];
  int32_t tok[kDepth];
  typename Out::Key key[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d) {
    const int32_t r = min(r0 + d * kRows + g, rows - 1);
    tok[d] = in.token(r);
    const uint4* src = reinterpret_cast<const uint4*>(in.row(r, tok[d])) + l;
    raw[d][0] = src[0];                    // coherent: the output may be the input
    raw[d][1] = src[G];
    key[d] = out.key(r);
  }
  const int32_t t0 = in.token(r0);
  if (p.turn.pairs) {
    fill_table(table, p.turn, positions, t0, in.token(min(r0 + kDepth * kRows, rows) - 1) - t0 + 1);
    __syncthreads();
  }
#pragma unroll
  for (int d = 0; d < kDepth; ++d) {
    const int32_t r = r0 + d * kRows + g;
    float v[2][8];
    unpack8(raw[d][0], v[0]);
    unpack8(raw[d][1], v[1]);
    normalise<G>(v, p, l);
    turn_row<G>(v, p.turn, table + (tok[d] - t0) * p.turn.pairs, l);
    uint16_t* scale = nullptr;
    if constexpr (kMode == 0) {
      uint8_t* dst = r < rows ? out.dest(r, tok[d], key[d], scale) : nullptr;
      if (dst == nullptr) continue;
      reinterpret_cast<uint4*>(dst)[l] = pack8(v[0]);
      reinterpret_cast<uint4*>(dst)[l + G] = pack8(v[1]);
    } else {
      uint2 codes[2];
      const uint16_t sb = quantise<G, kMode == QLI_QUANT_FP8>(v, codes);
      uint8_t* dst = r < rows ? out.dest(r, tok[d], key[d], scale) : nullptr;
      if (dst == nullptr) continue;
      reinterpret_cast<uint2*>(dst)[l] = codes[0];
      reinterpret_cast<uint2*>(dst)[l + G] = codes[1];
      if (l == 0) *scale = sb;
    }
  }
}

// Entries of the table that a pass over rows of D values can need.
template <int D, int kDepth>
int64_t table_entries(int64_t rows, int64_t H, int32_t pairs) {
  const int64_t most = kDepth * kThreads / (D / 16), in = rows < most ? rows : most;
  return ((in - 1 + H - 1) / H + 1 < in ? (in - 1 + H - 1) / H + 1 : in) * pairs;
}

// ---- queries --------------------------------------------------------------------
constexpr int kQueryDepth = 1;

template <int D, int kMode>
__global__ void __launch_bounds__(kThreads) prepare_kernel(const __grid_constant__ Prep p, DenseIn in,
                                                           DenseOut<kMode> out, const int32_t* positions,
                                                           int32_t rows) {
  extern __shared__ float2 table[];
  constexpr int kRows = kQueryDepth * kThreads / (D / 16);
  pass<D, kMode, kQueryDepth>(in, out, p, positions, static_cast<int32_t>(blockIdx.x) * kRows, rows, table);
}

template <int D, int kMode>
cudaError_t launch_prepare(const Prep& p, const DenseIn& in, const DenseOut<kMode>& out,
                           const int32_t* positions, int32_t rows, cudaStream_t s) {
  constexpr int kRows = kQueryDepth * kThreads / (D / 16);
  const size_t smem = sizeof(float2) * table_entries<D, kQueryDepth>(rows, in.H, p.turn.pairs);
  prepare_kernel<D, kMode><<<static_cast<unsigned>((rows - 1) / kRows + 1), kThreads, smem, s>>>(
      p, in, out, positions, rows);
  return cudaGetLastError();
}

// ---- cache rows -----------------------------------------------------------------
constexpr int kKvDepth = 1, kIndexDepth = 1;

template <int kKv, int kIndex>
struct AppendArgs {
  Prep kv, index;
  FlatIn kv_in, index_in;
  PagedOut<kKv> kv_out;
  PagedOut<kIndex> index_out;
  const int32_t* positions;
  int32_t n, kv_blocks;
};

// The first blocks take the KV rows, the others the index K rows.
template <int kKv, int kIndex>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs<kKv, kIndex> a) {
  extern __shared__ float2 table[];
  const int32_t b = static_cast<int32_t>(blockIdx.x);
  if (b < a.kv_blocks) {
    constexpr int kRows = kKvDepth * kThreads / (kKvRow / 16);
    pass<kKvRow, kKv, kKvDepth>(a.kv_in, a.kv_out, a.kv, a.positions, b * kRows, a.n, table);
  } else {
    constexpr int kRows = kIndexDepth * kThreads / (kIndexRow / 16);
    pass<kIndexRow, kIndex, kIndexDepth>(a.index_in, a.index_out, a.index, a.positions,
                                         (b - a.kv_blocks) * kRows, a.n, table);
  }
}

// ---- rotation alone ---------------------------------------------------------------
// A thread has two units of a row, h8 apart: eight pairs of the half layout, or
// two times four neighbouring ones. In place nothing else of the row is touched;
// otherwise the block copies the rest of its rows.
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
  extern __shared__ float2 table[];
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
    float x[8], y[8];
    unpack8(v0, x);
    unpack8(v1, y);
    const int w = u - a.turn.o8;
    const float2* cs = table + (t - t0) * a.turn.pairs;
    if (a.turn.half) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 c = cs[8 * w + i];
        const float p = x[i], q = y[i];
        x[i] = p * c.x - q * c.y;
        y[i] = q * c.x + p * c.y;
      }
    } else {
      turn_neighbours(x, cs + 4 * w);
      turn_neighbours(y, cs + 4 * (w + h8));
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
  if (r.offset < 0 || r.offset + 2 * static_cast<int64_t>(r.pairs) > width || !std::isfinite(r.magnitude))
    return QLI_ERR_INVALID_ARG;
  return QLI_OK;
}

Turn make_turn(const qli_rotary& r, bool inverse) {
  Turn w{};
  w.pairs = r.pairs;
  w.half = r.layout == QLI_ROTARY_HALF ? 1 : 0;
  w.o8 = r.offset / 8;
  w.cos_scale = inverse ? 1.0f / r.magnitude : r.magnitude;
  w.sin_scale = inverse ? -w.cos_scale : w.cos_scale;
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
  if (static_cast<int64_t>(T) * H > INT32_MAX) return QLI_ERR_UNSUPPORTED;
  return QLI_OK;
}

template <int kMode>
cudaError_t launch_width(const qli_prepare_args& a, const Prep& p, int32_t width, cudaStream_t s) {
  const DenseIn in{a.x, a.x_stride_t, a.x_stride_h, a.H};
  const int64_t unit = kMode == 0 ? 2 : 1;
  const DenseOut<kMode> out{static_cast<uint8_t*>(a.out), a.out_stride_t * unit, a.out_stride_h * unit, a.scale_out, a.H};
  const int32_t rows = a.T * a.H;
  if constexpr (kMode == 0) {
    if (width == 64) return launch_prepare<64, 0>(p, in, out, a.positions, rows, s);
    if (width == 256) return launch_prepare<256, 0>(p, in, out, a.positions, rows, s);
    if (width == 512) return launch_prepare<512, 0>(p, in, out, a.positions, rows, s);
  }
  return launch_prepare<128, kMode>(p, in, out, a.positions, rows, s);
}

template <int kKv, int kIndex>
cudaError_t launch_append(const qli_append_args& a, const qli_row_prep* kv, const qli_row_prep* index, cudaStream_t s) {
  AppendArgs<kKv, kIndex> d{};
  d.positions = a.positions;
  d.n = static_cast<int32_t>(a.n);
  const int64_t slots = a.num_pages * a.rows_per_page;
  const int32_t log2R = a.rows_per_page == 64 ? 6 : 7;
  int64_t blocks = 0, table = 0;
  if (a.kv) {
    d.kv = make_prep(*kv);
    d.kv_in = FlatIn{a.kv, a.kv_stride};
    d.kv_out = PagedOut<kKv>{a.slot_mapping, a.cache, slots, a.page_stride, a.kv_offset, a.kv_scale_offset, log2R,
                             kKv == 0 ? 2 * kKvRow : kKvRow, a.err_word};
    blocks = (a.n - 1) / (kKvDepth * kThreads / (kKvRow / 16)) + 1;
    table = table_entries<kKvRow, kKvDepth>(a.n, 1, d.kv.turn.pairs);
  }
  d.kv_blocks = static_cast<int32_t>(blocks);
  if (a.index_k) {
    d.index = make_prep(*index);
    d.index_in = FlatIn{a.index_k, a.index_stride};
    d.index_out = PagedOut<kIndex>{a.slot_mapping, a.cache, slots, a.page_stride, a.k_offset, a.scale_offset, log2R,
                                   kIndexRow, a.err_word};
    blocks += (a.n - 1) / (kIndexDepth * kThreads / (kIndexRow / 16)) + 1;
    const int64_t more = table_entries<kIndexRow, kIndexDepth>(a.n, 1, d.index.turn.pairs);
    table = more > table ? more : table;
  }
  append_kernel<kKv, kIndex><<<static_cast<unsigned>(blocks), kThreads, sizeof(float2) * table, s>>>(d);
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
  if (a->D < 16 || a->D % 8 != 0) return QLI_ERR_UNSUPPORTED;
  qli_status st = check_rotary(*rotary, a->D);
  if (st != QLI_OK) return st;
  if (a->inverse && rotary->magnitude == 0.0f) return QLI_ERR_INVALID_ARG;
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
  const int64_t in = d.rows < d.block_rows ? d.rows : d.block_rows;
  const int64_t tokens = (in - 2 + a->H) / a->H + 1;
  const size_t smem = sizeof(float2) * static_cast<size_t>((tokens < in ? tokens : in) * rotary->pairs);
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
  const cudaError_t e = a->quant_mode == 0                ? launch_width<0>(*a, p, D, s)
                        : a->quant_mode == QLI_QUANT_INT8 ? launch_width<QLI_QUANT_INT8>(*a, p, D, s)
                                                          : launch_width<QLI_QUANT_FP8>(*a, p, D, s);
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
  if (a->n > INT32_MAX) return QLI_ERR_UNSUPPORTED;
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
    e = f8 ? launch_append<0, QLI_QUANT_FP8>(*a, kv_prep, index_prep, s)
           : launch_append<0, QLI_QUANT_INT8>(*a, kv_prep, index_prep, s);
  else if (a->kv_mode == QLI_QUANT_INT8)
    e = f8 ? launch_append<QLI_QUANT_INT8, QLI_QUANT_FP8>(*a, kv_prep, index_prep, s)
           : launch_append<QLI_QUANT_INT8, QLI_QUANT_INT8>(*a, kv_prep, index_prep, s);
  else
    e = f8 ? launch_append<QLI_QUANT_FP8, QLI_QUANT_FP8>(*a, kv_prep, index_prep, s)
           : launch_append<QLI_QUANT_FP8, QLI_QUANT_INT8>(*a, kv_prep, index_prep, s);
  return e == cudaSuccess ? QLI_OK : QLI_ERR_CUDA;
}

extern "C" int64_t qli_rotary_size(void) { return static_cast<int64_t>(sizeof(qli_rotary)); }
extern "C" int64_t qli_row_prep_size(void) { return static_cast<int64_t>(sizeof(qli_row_prep)); }
extern "C" int64_t qli_rotate_args_size(void) { return static_cast<int64_t>(sizeof(qli_rotate_args)); }
extern "C" int64_t qli_prepare_args_size(void) { return static_cast<int64_t>(sizeof(qli_prepare_args)); }
extern "C" int64_t qli_append_args_size(void) { return static_cast<int64_t>(sizeof(qli_append_args)); }
