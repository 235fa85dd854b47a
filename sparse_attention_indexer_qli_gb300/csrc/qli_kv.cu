// The 8-bit KV cache around its attention: the row writer (quantises as it
// writes), the row reader, and the merge of attention stages by their
// log-sum-exps. All three are one pass over HBM with a warp per row.
//
//   writer  s = FP16(max |x| / Q) capped at 65504, c = code(x / s), Q = 127
//           (INT8) or 448 (E4M3); s rounding to zero gives codes 0, scale +0
//           (the arithmetic of the index-K writer, on rows of 512)
//   reader  y = BF16(c * s): an 11-bit by 8-bit product is exact in FP32, so
//           there is one rounding
//   merge   M = max_i lse_i, w_i = e^(lse_i - M),
//           o = sum w_i o_i / sum w_i, lse = M + ln sum w_i  (FP32 sums)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qli_codes.cuh"
#include "qli_internal.h"
#include "qli_ptx.cuh"

namespace qli {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRow = 512;                 // values per KV row

// Where a page slot's codes and scale are.
struct Pages {
  uint8_t* cache;
  int64_t slots_total, page_stride, kv_offset, scale_offset;
  int32_t log2R;
  uint32_t* err;
  // false for a negative slot (padding) and for one past the pool (flagged)
  __device__ __forceinline__ bool find(int64_t m, uint8_t*& codes, uint16_t*& scale) const {
    if (m < 0) return false;
    if (m >= slots_total) {
      if (err != nullptr) atomicOr(err, QLI_DEVERR_PAGE);
      return false;
    }
    const int64_t row = m & ((int64_t{1} << log2R) - 1);
    uint8_t* p = cache + (m >> log2R) * page_stride;
    codes = p + kv_offset + row * kRow;
    scale = reinterpret_cast<uint16_t*>(p + scale_offset + row * 2);
    return true;
  }
};

__device__ __forceinline__ void bf16x8_to_f32(const uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Eight codes of BF16 pairs under the scale sf (y = RN(1 / sf)); the same codes
// as code_of and e4m3x2_of give value by value. INT8: adding 1.5 * 2^23 rounds
// the quotient to an integer, ties to even, in the low bits (it is below 1.5 *
// 127 but under the largest scale, where `huge` clamps it first), two are
// clamped at a time as 16-bit halves. E4M3: the quotient's sign is x's; the
// correction step gives +0 for a negative x far below s, so the signs are taken
// from x (the top bytes of its BF16 halves).
template <bool kFp8>
__device__ __forceinline__ uint2 codes8(const uint4 v, float sf, float y, bool huge) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float q[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      q[2 * k] = quotient(__uint_as_float(w[2 * i + k] << 16), sf, y);
      q[2 * k + 1] = quotient(__uint_as_float(w[2 * i + k] & 0xffff0000u), sf, y);
    }
    if constexpr (kFp8) {
      const uint32_t c = e4m3x2_of(q[0], q[1]) | (e4m3x2_of(q[2], q[3]) << 16);
      const uint32_t sign = __byte_perm(w[2 * i], w[2 * i + 1], 0x7531);
      out[i] = (c & 0x7f7f7f7fu) | (sign & 0x80808080u);
    } else {
      uint32_t n[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (huge) q[k] = fminf(fmaxf(q[k], -127.0f), 127.0f);
        n[k] = __float_as_uint(__fadd_rn(q[k], 12582912.0f));
      }
      const uint32_t lo = __vmins2(__vmaxs2(__byte_perm(n[0], n[1], 0x5410), 0xff81ff81u), 0x007f007fu);
      const uint32_t hi = __vmins2(__vmaxs2(__byte_perm(n[2], n[3], 0x5410), 0xff81ff81u), 0x007f007fu);
      out[i] = __byte_perm(lo, hi, 0x6420);
    }
  }
  return make_uint2(out[0], out[1]);
}

// The largest magnitude of a row's BF16 values (a lane has two times eight),
// compared as integers: NaN is above all.
__device__ __forceinline__ float row_amax(const uint4 a, const uint4 b) {
  constexpr uint32_t k = 0x7fff7fffu;
  uint32_t m = __vmaxu2(__vmaxu2(__vmaxu2(a.x & k, a.y & k), __vmaxu2(a.z & k, a.w & k)),
                        __vmaxu2(__vmaxu2(b.x & k, b.y & k), __vmaxu2(b.z & k, b.w & k)));
  m = __reduce_max_sync(0xffffffffu, max(m >> 16, m & 0xffffu));
  return __uint_as_float(m << 16);
}

// ---- writer -----------------------------------------------------------------
// Lane l takes values 8l..8l+7 and 256+8l..256+8l+7 (two coalesced 512-byte
// loads a row, two coalesced 256-byte stores), kDepth rows in flight. Bound by
// HBM with rows scattered over the pages: 65536 rows (101 MB) take 20.5 us, 4.9
// TB/s (the floor at the copy rate is 15 us). Code arithmetic value by value, not
// two at a time, took 23.7; depths of 1 to 4 measured alike.
template <bool kFp8, int kDepth>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const uint16_t* __restrict__ x,
                                                            int64_t x_stride, int64_t rows,
                                                            const int64_t* __restrict__ slot,
                                                            Pages pages) {
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  for (int64_t r0 = warp; r0 < rows; r0 += kDepth * nwarps) {
    uint4 v[kDepth][2];
    int64_t at[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int64_t r = r0 + d * nwarps;
      v[d][0] = v[d][1] = make_uint4(0u, 0u, 0u, 0u);
      at[d] = -1;
      if (r < rows) {
        const uint4* src = reinterpret_cast<const uint4*>(x + r * x_stride) + lane;
        v[d][0] = __ldcs(src);
        v[d][1] = __ldcs(src + 32);
        at[d] = __ldg(slot + r);
      }
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      uint16_t sb = scale_bits_of<kFp8>(row_amax(v[d][0], v[d][1]));
      const float sf = __half2float(__ushort_as_half(sb));
      uint2 c0 = make_uint2(0u, 0u), c1 = c0;
      if (sf != 0.0f) {
        const float y = __frcp_rn(sf);
        c0 = codes8<kFp8>(v[d][0], sf, y, sb == 0x7bffu);
        c1 = codes8<kFp8>(v[d][1], sf, y, sb == 0x7bffu);
      } else {
        sb = 0u;
      }
      uint8_t* codes;
      uint16_t* sc;
      if (pages.find(at[d], codes, sc)) {
        reinterpret_cast<uint2*>(codes)[lane] = c0;
        reinterpret_cast<uint2*>(codes)[32 + lane] = c1;
        if (lane == 0) *sc = sb;
      }
    }
  }
}

// ---- reader -----------------------------------------------------------------
// The writer's layout of lanes; kDepth rows in flight, since slot, codes and
// output are a chain of round trips. Bound by HBM: 131072 rows (203 MB) take 34
// us, 6.0 TB/s. Twice the depth is no faster there and slower for few rows (4097
// rows: 4.3 us with 4 in flight, 6.1 with 8).
// Four codes to FP32 (lowest byte first).
template <bool kFp8>
__device__ __forceinline__ void codes_to_f32(uint32_t w, float* f) {
  if constexpr (kFp8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t h = e4m3x2_to_f16x2((w >> (16 * i)) & 0xffffu);
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = static_cast<float>(static_cast<int8_t>((w >> (8 * i)) & 0xffu));
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <bool kFp8, int kDepth>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(Pages pages, int64_t rows,
                                                           const int64_t* __restrict__ slot,
                                                           uint16_t* __restrict__ out,
                                                           int64_t out_stride) {
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  for (int64_t r0 = warp; r0 < rows; r0 += kDepth * nwarps) {
    int64_t at[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int64_t r = r0 + d * nwarps;
      at[d] = r < rows ? __ldg(slot + r) : -1;
    }
    uint2 v[kDepth][2];
    uint16_t sb[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      v[d][0] = v[d][1] = make_uint2(0u, 0u);
      sb[d] = 0;
      uint8_t* codes;
      uint16_t* sc;
      if (pages.find(at[d], codes, sc)) {
        v[d][0] = __ldcs(reinterpret_cast<const uint2*>(codes) + lane);
        v[d][1] = __ldcs(reinterpret_cast<const uint2*>(codes) + 32 + lane);
        sb[d] = __ldg(sc);
      }
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int64_t r = r0 + d * nwarps;
      if (r >= rows) break;
      const float s = __half2float(__ushort_as_half(sb[d]));
      uint4* dst = reinterpret_cast<uint4*>(out + r * out_stride) + lane;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float f[8];
        codes_to_f32<kFp8>(v[d][i].x, f);
        codes_to_f32<kFp8>(v[d][i].y, f + 4);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = pack_bf16(f[2 * k] * s, f[2 * k + 1] * s);
        __stcs(dst + 32 * i, make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
}

// ---- merge ------------------------------------------------------------------
struct MergeArgs {
  const void* out[QLI_MERGE_MAX];
  int64_t st[QLI_MERGE_MAX], sh[QLI_MERGE_MAX];
  const float* lse[QLI_MERGE_MAX];
  int32_t H;
  int64_t rows;                            // T * H
  uint16_t* o;
  int64_t o_st, o_sh;
  float* o_lse;
};

// Lane l of the row's warp takes values 8l..8l+7 and 256+8l..256+8l+7.
// kParts is a compile-time number so that every part's loads are in flight
// together. Bound by HBM: three parts of 4096 tokens x 64 heads (1.08 GB) take 153
// us, the rate of a plain copy.
template <int kParts, bool kF32>
__global__ void __launch_bounds__(kThreads) merge_kernel(MergeArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < a.rows;
       row += nwarps) {
    const int64_t t = row / a.H, h = row % a.H;
    float l[kParts];
    uint4 v[kParts][kF32 ? 4 : 2];
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      l[p] = __ldg(a.lse[p] + row);
      const int64_t off = t * a.st[p] + h * a.sh[p];
      if constexpr (kF32) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const float*>(a.out[p]) + off);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[p][i] = __ldcs(src + (i >> 1) * 64 + 2 * lane + (i & 1));
      } else {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.out[p]) + off);
#pragma unroll
        for (int i = 0; i < 2; ++i) v[p][i] = __ldcs(src + 32 * i + lane);
      }
    }
    float m = -INFINITY;
#pragma unroll
    for (int p = 0; p < kParts; ++p) m = fmaxf(m, l[p]);
    float total = 0.0f, acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      // a part that found nothing drops out whatever its output holds
      if (l[p] == -INFINITY) continue;
      const float w = expf(l[p] - m);
      total += w;
      float f[16];
      if constexpr (kF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[4 * i] = __uint_as_float(v[p][i].x);
          f[4 * i + 1] = __uint_as_float(v[p][i].y);
          f[4 * i + 2] = __uint_as_float(v[p][i].z);
          f[4 * i + 3] = __uint_as_float(v[p][i].w);
        }
      } else {
        bf16x8_to_f32(v[p][0], f);
        bf16x8_to_f32(v[p][1], f + 8);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = fmaf(w, f[i], acc[i]);
    }
    const bool none = m == -INFINITY && total == 0.0f;
    const float inv = none ? 0.0f : 1.0f / total;
    uint4* dst = reinterpret_cast<uint4*>(a.o + t * a.o_st + h * a.o_sh) + lane;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = pack_bf16(acc[8 * i + 2 * k] * inv, acc[8 * i + 2 * k + 1] * inv);
      __stcs(dst + 32 * i, make_uint4(w[0], w[1], w[2], w[3]));
    }
    if (lane == 0 && a.o_lse != nullptr) a.o_lse[row] = none ? -INFINITY : m + logf(total);
  }
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A warp per row up to the warps the device holds at once; past that each warp
// goes on by the grid's stride, several rows in flight.
unsigned row_grid(int64_t rows, int sms) {
  const int64_t want = (rows + kWarps - 1) / kWarps;
  const int64_t cap = static_cast<int64_t>(sms) * (2048 / kThreads);
  return static_cast<unsigned>(want < cap ? want : cap);
}

qli_status check_pages(const void* cache, int64_t num_pages, int64_t page_stride,
                       int32_t rows_per_page, int64_t kv_offset, int64_t scale_offset,
                       const int64_t* slot, const uint32_t* err_word) {
  if (!cache || !slot) return QLI_ERR_INVALID_ARG;
  if (rows_per_page != 64 && rows_per_page != 128) return QLI_ERR_UNSUPPORTED;
  if (page_stride <= 0 || kv_offset < 0 || scale_offset < 0 ||
      kv_offset + static_cast<int64_t>(rows_per_page) * kRow > page_stride ||
      scale_offset + static_cast<int64_t>(rows_per_page) * 2 > page_stride)
    return QLI_ERR_INVALID_ARG;
  if (!aligned_to(cache, 16) || page_stride % 16 != 0 || kv_offset % 16 != 0 ||
      scale_offset % 2 != 0 || !aligned_to(slot, 8) ||
      (err_word != nullptr && !aligned_to(err_word, 4)))
    return QLI_ERR_ALIGNMENT;
  return QLI_OK;
}

constexpr int kWriteDepth = 2;
constexpr int kReadDepth = 4;

template <int kParts>
cudaError_t launch_merge(const MergeArgs& d, bool f32, unsigned grid, cudaStream_t s) {
  if (f32)
    merge_kernel<kParts, true><<<grid, kThreads, 0, s>>>(d);
  else
    merge_kernel<kParts, false><<<grid, kThreads, 0, s>>>(d);
  return cudaGetLastError();
}

}  // namespace
}  // namespace qli

extern "C" qli_status qli_write_kv(const uint16_t* kv, int64_t kv_stride, int64_t n,
                                   const int64_t* slot_mapping, uint8_t* cache, int64_t num_pages,
                                   int64_t page_stride, int32_t rows_per_page, int64_t kv_offset,
                                   int64_t kv_scale_offset, int32_t quant_mode, uint32_t* err_word,
                                   void* stream) {
  using namespace qli;
  if (quant_mode != QLI_QUANT_INT8 && quant_mode != QLI_QUANT_FP8) return QLI_ERR_UNSUPPORTED;
  if (n < 0 || num_pages < 0) return QLI_ERR_INVALID_ARG;
  if (n == 0) return QLI_OK;
  if (!kv || kv_stride < kRow) return QLI_ERR_INVALID_ARG;
  qli_status st = check_pages(cache, num_pages, page_stride, rows_per_page, kv_offset,
                              kv_scale_offset, slot_mapping, err_word);
  if (st != QLI_OK) return st;
  if (!aligned_to(kv, 16) || kv_stride % 8 != 0) return QLI_ERR_ALIGNMENT;
  int sms = 0;
  st = device_sms(&sms);
  if (st != QLI_OK) return st;
  const Pages p{cache, num_pages * rows_per_page, page_stride, kv_offset, kv_scale_offset,
                rows_per_page == 64 ? 6 : 7, err_word};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = row_grid(n, sms);
  if (quant_mode == QLI_QUANT_FP8)
    kv_write_kernel<true, kWriteDepth><<<grid, kThreads, 0, s>>>(kv, kv_stride, n, slot_mapping, p);
  else
    kv_write_kernel<false, kWriteDepth><<<grid, kThreads, 0, s>>>(kv, kv_stride, n, slot_mapping, p);
  return cudaGetLastError() == cudaSuccess ? QLI_OK : QLI_ERR_CUDA;
}

extern "C" qli_status qli_read_kv(const uint8_t* cache, int64_t num_pages, int64_t page_stride,
                                  int32_t rows_per_page, int64_t kv_offset, int64_t kv_scale_offset,
                                  int32_t quant_mode, const int64_t* slots, int64_t n,
                                  uint16_t* out, int64_t out_stride, uint32_t* err_word,
                                  void* stream) {
  using namespace qli;
  if (quant_mode != QLI_QUANT_INT8 && quant_mode != QLI_QUANT_FP8) return QLI_ERR_UNSUPPORTED;
  if (n < 0 || num_pages < 0) return QLI_ERR_INVALID_ARG;
  if (n == 0) return QLI_OK;
  if (!out || out_stride < kRow) return QLI_ERR_INVALID_ARG;
  qli_status st = check_pages(cache, num_pages, page_stride, rows_per_page, kv_offset,
                              kv_scale_offset, slots, err_word);
  if (st != QLI_OK) return st;
  if (!aligned_to(out, 16) || out_stride % 8 != 0) return QLI_ERR_ALIGNMENT;
  int sms = 0;
  st = device_sms(&sms);
  if (st != QLI_OK) return st;
  // the kernel only reads through `cache`
  const Pages p{const_cast<uint8_t*>(cache), num_pages * rows_per_page, page_stride, kv_offset,
                kv_scale_offset, rows_per_page == 64 ? 6 : 7, err_word};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = row_grid(n, sms);
  if (quant_mode == QLI_QUANT_FP8)
    kv_read_kernel<true, kReadDepth><<<grid, kThreads, 0, s>>>(p, n, slots, out, out_stride);
  else
    kv_read_kernel<false, kReadDepth><<<grid, kThreads, 0, s>>>(p, n, slots, out, out_stride);
  return cudaGetLastError() == cudaSuccess ? QLI_OK : QLI_ERR_CUDA;
}

extern "C" qli_status qli_merge_attention(const qli_merge_args* a, void* stream) {
  using namespace qli;
  if (a == nullptr) return QLI_ERR_INVALID_ARG;
  if (a->D != kRow) return QLI_ERR_UNSUPPORTED;
  if (a->parts < 1 || a->parts > QLI_MERGE_MAX || a->T < 0 || a->H < 1) return QLI_ERR_INVALID_ARG;
  if (a->T == 0) return QLI_OK;
  const bool f32 = a->parts_f32 != 0;
  const int64_t unit = f32 ? 4 : 8;          // elements of 16 bytes
  MergeArgs d{};
  if (a->out == nullptr) return QLI_ERR_INVALID_ARG;
  if (a->out_stride_h < kRow || a->out_stride_t < kRow) return QLI_ERR_INVALID_ARG;
  for (int p = 0; p < a->parts; ++p) {
    if (a->part_out[p] == nullptr || a->part_lse[p] == nullptr) return QLI_ERR_INVALID_ARG;
    if (a->part_stride_t[p] < 0 || a->part_stride_h[p] < 0) return QLI_ERR_INVALID_ARG;
    if (!aligned_to(a->part_out[p], 16) || a->part_stride_t[p] % unit != 0 ||
        a->part_stride_h[p] % unit != 0 || !aligned_to(a->part_lse[p], 4))
      return QLI_ERR_ALIGNMENT;
    d.out[p] = a->part_out[p];
    d.st[p] = a->part_stride_t[p];
    d.sh[p] = a->part_stride_h[p];
    d.lse[p] = a->part_lse[p];
  }
  if (!aligned_to(a->out, 16) || a->out_stride_t % 8 != 0 || a->out_stride_h % 8 != 0 ||
      (a->lse != nullptr && !aligned_to(a->lse, 4)))
    return QLI_ERR_ALIGNMENT;
  int sms = 0;
  const qli_status st = device_sms(&sms);
  if (st != QLI_OK) return st;
  d.H = a->H;
  d.rows = static_cast<int64_t>(a->T) * a->H;
  d.o = a->out;
  d.o_st = a->out_stride_t;
  d.o_sh = a->out_stride_h;
  d.o_lse = a->lse;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = row_grid(d.rows, sms);
  cudaError_t e = cudaErrorInvalidValue;
  switch (a->parts) {
    case 1: e = launch_merge<1>(d, f32, grid, s); break;
    case 2: e = launch_merge<2>(d, f32, grid, s); break;
    case 3: e = launch_merge<3>(d, f32, grid, s); break;
    case 4: e = launch_merge<4>(d, f32, grid, s); break;
  }
  return e == cudaSuccess ? QLI_OK : QLI_ERR_CUDA;
}

extern "C" int64_t qli_merge_args_size(void) { return static_cast<int64_t>(sizeof(qli_merge_args)); }
