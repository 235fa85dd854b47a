// Softmax attention over 8-bit KV rows of the paged cache: for token t, head h
// and the positions J (listed, or causally visible),
//   kv_j = c_j s_j,  z_j = scale q . kv_j,
//   o = sum_j e^(z_j - m) kv_j / sum_j e^(z_j - m),  lse = m + ln sum.
//
// One CTA per (head, token): 32 positions at a time, a warp takes eight of
// their dots (lanes split the 512 values), then every thread adds the 32
// weighted rows to its four values of o.
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
constexpr int kThreads = 128;
constexpr int kChunk = 32;

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
  int32_t R;
  const int32_t* bt;
  int32_t bt_stride;
  const int32_t* idx;
  int32_t K;
  float scale;
  uint16_t* out;
  int64_t o_st, o_sh;
  float* lse;
  uint32_t* err;
};

// Four codes to FP32 (lowest byte first).
template <bool kFp8>
__device__ __forceinline__ void codes4(uint32_t w, float* f) {
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

// Entry e of the token's positions as a row pointer; nullptr when skipped.
__device__ __forceinline__ const uint8_t* row_of(const Args& a, int t, int b, int64_t j,
                                                 int& row, bool& bad) {
  (void)t;
  if (j < 0) return nullptr;
  if (j >= a.cap) {
    bad = true;
    return nullptr;
  }
  const int32_t page = __ldg(a.bt + static_cast<int64_t>(b) * a.bt_stride + j / a.R);
  if (page < 0 || page >= a.num_pages) {
    bad = true;
    return nullptr;
  }
  row = static_cast<int>(j % a.R);
  return a.cache + page * a.page_stride;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads) kv_attn_kernel(Args a) {
  __shared__ float qs[kD];
  __shared__ float z[kChunk], rs[kChunk];
  __shared__ const uint8_t* base[kChunk];
  __shared__ int32_t tok[3];                   // request, first position, end
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, t = blockIdx.y;
  if (tid == 0) {
    int32_t lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    tok[0] = lo;
    tok[1] = 0;
    tok[2] = a.K;
    if (a.idx == nullptr) {
      int32_t q0, q1, lk, res;
      const uint32_t e = sanitize_request(a, lo, q0, q1, lk, res);
      if (e != 0u && a.err != nullptr) atomicOr(a.err, e);
      const int32_t V = q0 <= t && t < q1 ? visible_count(lk, res, a.ratio, q1 - q0, t - q0) : 0;
      tok[1] = a.window > 0 ? max(0, V - a.window) : 0;
      tok[2] = V;
    }
  }
  for (int d = tid; d < kD; d += kThreads)
    qs[d] = __uint_as_float(static_cast<uint32_t>(a.q[t * a.q_st + h * a.q_sh + d]) << 16);
  __syncthreads();
  float qr[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) qr[i] = qs[16 * lane + i];
  float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  bool bad = false;
  for (int64_t p0 = tok[1]; p0 < tok[2]; p0 += kChunk) {
    __syncthreads();
    if (tid < kChunk) {
      const int64_t e = p0 + tid;
      int64_t j = -1;
      if (e < tok[2]) j = a.idx ? __ldg(a.idx + static_cast<int64_t>(t) * a.K + e) : e;
      int row = 0;
      const uint8_t* page = row_of(a, t, tok[0], j, row, bad);
      base[tid] = page ? page + a.kv_off + row * kD : nullptr;
      rs[tid] = page ? __half2float(*reinterpret_cast<const __half*>(page + a.sc_off + row * 2)) : 0.0f;
    }
    __syncthreads();
    for (int i = warp; i < kChunk; i += kThreads / 32) {
      float s = 0.0f;
      if (base[i]) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(base[i]) + lane);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float f[4];
          codes4<kFp8>(w[k], f);
#pragma unroll
          for (int x = 0; x < 4; ++x) s = fmaf(f[x], qr[4 * k + x], s);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      }
      if (lane == 0) z[i] = base[i] ? s * rs[i] * a.scale : -INFINITY;
    }
    __syncthreads();
    float top = m;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) top = fmaxf(top, z[i]);
    if (top == -INFINITY) continue;
    const float alpha = expf(m - top);
    m = top;
    l *= alpha;
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] *= alpha;
    for (int i = 0; i < kChunk; ++i) {
      if (!base[i]) continue;
      const float p = expf(z[i] - m);
      l += p;
      float f[4];
      codes4<kFp8>(__ldg(reinterpret_cast<const uint32_t*>(base[i]) + tid), f);
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] = fmaf(p * rs[i], f[x], o[x]);
    }
  }
  if (bad && a.err != nullptr) atomicOr(a.err, QLI_DEVERR_PAGE);
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  uint16_t* dst = a.out + t * a.o_st + h * a.o_sh + 4 * tid;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const __nv_bfloat16 y = __float2bfloat16_rn(l == 0.0f ? 0.0f : o[x] * inv);
    dst[x] = *reinterpret_cast<const uint16_t*>(&y);
  }
  if (tid == 0 && a.lse != nullptr)
    a.lse[static_cast<int64_t>(t) * a.H + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

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

}  // namespace
}  // namespace kvattn
}  // namespace qli

extern "C" qli_status qli_kv_attention_workspace_size(const qli_kv_attn_args* a, size_t* bytes) {
  if (bytes == nullptr) return QLI_ERR_INVALID_ARG;
  const qli_status st = qli::kvattn::validate(a);
  if (st != QLI_OK) return st;
  *bytes = 0;
  return QLI_OK;
}

extern "C" qli_status qli_kv_attention(const qli_kv_attn_args* a, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  using namespace qli::kvattn;
  (void)workspace;
  (void)workspace_bytes;
  qli_status st = validate(a);
  if (st != QLI_OK) return st;
  if (a->T == 0) return QLI_OK;
  if (a->T > 65535) return QLI_ERR_UNSUPPORTED;
  int sms = 0;
  st = qli::device_sms(&sms);
  if (st != QLI_OK) return st;
  const Args d = make_args(*a);
  const dim3 grid(static_cast<unsigned>(a->H), static_cast<unsigned>(a->T));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->quant_mode == QLI_QUANT_FP8)
    kv_attn_kernel<true><<<grid, kThreads, 0, s>>>(d);
  else
    kv_attn_kernel<false><<<grid, kThreads, 0, s>>>(d);
  return cudaGetLastError() == cudaSuccess ? QLI_OK : QLI_ERR_CUDA;
}

extern "C" int64_t qli_kv_attn_args_size(void) {
  return static_cast<int64_t>(sizeof(qli_kv_attn_args));
}
