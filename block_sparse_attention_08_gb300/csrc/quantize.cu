// quantize.cu -- K and V rows written into the int8 cache, and read back.
//
// A row (a token's 128 values of a KV head) is stored as int8 n and one bf16
// scale s, value n s.  s = 2^(e - 6) with 2^e the power of two at or below the
// row's largest magnitude, so that one takes 64 to 127 of the 127 steps;
// n = x / s rounded to nearest (ties to even), at most 127.  A power of two
// loses up to a bit against s = max / 127, but n s is then a bf16 number, so
// whoever reads the cache in bf16 products reads these values exactly.  Scaling
// by it is exact as well, so n depends on no rounding but its own.
//
// Both kernels move each byte once: 16 lanes take a row, 16 bytes of bf16 and 8
// of int8 each.
#include <algorithm>

#include "launch.h"

namespace msa {

constexpr int kQzThreads = 256;
constexpr int kQzRows = kQzThreads / 16;   // rows that a CTA takes at once
constexpr int kQzBatch = 4;                // and in flight per thread
constexpr int kQzParts = 2 * kKvHeads;     // rows of a token: K's heads, then V's

struct QzArgs {
  const __nv_bfloat16 *k, *v;
  long long k_stride, v_stride;  // elements between tokens
  const int64_t* slots;
  long long tokens, num_slots;
  int8_t *k_cache, *v_cache;
  __nv_bfloat16 *k_scales, *v_scales;
  DevError* err;
};

// The scale of a row whose largest magnitude is `top`, both as bf16 bits.
__device__ __forceinline__ uint32_t qz_scale_bits(uint32_t top) {
  if (top >= 0x7f80u) return 0x7fc0u;  // infinity or NaN in the row: it reads back as NaN
  const uint32_t field = top >> 7;              // biased exponent of 2^e (0: subnormal or zero, e = -127)
  return field > 6 ? (field - 6) << 7 : 1u << field;  // 2^(field - 133), down to a subnormal
}

__global__ void __launch_bounds__(kQzThreads) quantize_kernel(const __grid_constant__ QzArgs a) {
  const int lane16 = threadIdx.x & 15;
  const unsigned half = 0xffffu << (threadIdx.x & 16);
  const long long rows = a.tokens * kQzParts, step = static_cast<long long>(gridDim.x) * kQzRows;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (long long r0 = static_cast<long long>(blockIdx.x) * kQzRows + threadIdx.x / 16; r0 < rows; r0 += kQzBatch * step) {
    uint4 x[kQzBatch];
    int64_t slot[kQzBatch];
#pragma unroll
    for (int b = 0; b < kQzBatch; ++b) {
      const long long r = r0 + b * step;
      if (r >= rows) break;
      const long long t = r / kQzParts;
      const int part = static_cast<int>(r % kQzParts), g = part % kKvHeads;
      const __nv_bfloat16* from = part < kKvHeads ? a.k + t * a.k_stride : a.v + t * a.v_stride;
      x[b] = reinterpret_cast<const uint4*>(from + g * kDim)[lane16];
      slot[b] = a.slots[t];
    }
#pragma unroll
    for (int b = 0; b < kQzBatch; ++b) {
      const long long r = r0 + b * step;
      if (r >= rows) break;
      const int part = static_cast<int>(r % kQzParts), g = part % kKvHeads;
      const uint32_t w[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
      uint32_t top = 0;  // two 16-bit magnitudes
#pragma unroll
      for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) top = __vmaxu2(top, __shfl_xor_sync(half, top, d));
      top = max(top & 0xffffu, top >> 16);
      const uint32_t sb = qz_scale_bits(top);
      // x / s in two factors (one alone may pass the range of fp32): s = 2^(field - 133)
      const int field = min(static_cast<int>(top >> 7), 254), up = 133 - field, u0 = up / 2;
      const float f0 = __uint_as_float(static_cast<uint32_t>(127 + u0) << 23);
      const float f1 = __uint_as_float(static_cast<uint32_t>(127 + up - u0) << 23);
      uint32_t y[2] = {0u, 0u};
      if (top < 0x7f80u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
          const int n = max(-127, min(127, __float2int_rn(v * f0 * f1)));
          y[i / 4] |= (static_cast<uint32_t>(n) & 0xffu) << (8 * (i % 4));
        }
      }
      const int64_t s = slot[b];
      if (s < 0) continue;
      if (s >= a.num_slots) {
        if (lane16 == 0) record_error(a.err, MSA_DEVERR_PAGE, r / kQzParts);
        continue;
      }
      int8_t* cache = part < kKvHeads ? a.k_cache : a.v_cache;
      __nv_bfloat16* scales = part < kKvHeads ? a.k_scales : a.v_scales;
      reinterpret_cast<uint2*>(cache + (s * kKvHeads + g) * kDim)[lane16] = make_uint2(y[0], y[1]);
      if (lane16 == 0)
        reinterpret_cast<uint16_t*>(scales)[((s / kBlock) * kKvHeads + g) * kBlock + s % kBlock] = static_cast<uint16_t>(sb);
    }
  }
}

cudaError_t launch_quantize(const QuantizeLaunch& L, cudaStream_t stream) {
  if (const cudaError_t e = launch_prologue(); e != cudaSuccess) return e;
  const QzArgs a{static_cast<const __nv_bfloat16*>(L.k), static_cast<const __nv_bfloat16*>(L.v), L.k_stride, L.v_stride,
                 L.slots, L.tokens, L.num_slots, static_cast<int8_t*>(L.k_cache), static_cast<int8_t*>(L.v_cache),
                 static_cast<__nv_bfloat16*>(L.k_scales), static_cast<__nv_bfloat16*>(L.v_scales), L.err};
  const long long ctas = (L.tokens * kQzParts + kQzRows - 1) / kQzRows;
  return launch_dependent(quantize_kernel, dim3(static_cast<unsigned>(std::min(ctas, 8LL * kNumSMs))), kQzThreads, 0, stream,
                          a);
}

// ---- read back ------------------------------------------------------------------------

constexpr int kDqTokens = 16;  // tokens that a CTA takes at once

struct DqArgs {
  const int8_t *k_cache, *v_cache;
  const __nv_bfloat16 *k_scales, *v_scales;
  const int32_t *page_table, *starts, *cu;
  int batch, max_blocks, num_pages;
  long long tokens;
  __nv_bfloat16 *k_out, *v_out;
  DevError* err;
};

// The slot of output row t: -1 where its request or page is bad (a row of zeros), -2 where it belongs to no request.
__device__ __forceinline__ long long dq_slot(const DqArgs& a, long long t) {
  int lo = 0, hi = a.batch;  // the first request whose rows end behind t
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (a.cu[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  if (lo == a.batch) return -2;
  const long long c0 = a.cu[lo], c1 = a.cu[lo + 1], start = a.starts ? a.starts[lo] : 0;
  if (c0 > t) return -2;
  if (c0 < 0 || start < 0 || start + (c1 - c0) > static_cast<long long>(a.max_blocks) * kBlock) {
    record_error(a.err, MSA_DEVERR_LENGTH, lo);
    return -1;
  }
  const long long p = start + (t - c0), at = static_cast<long long>(lo) * a.max_blocks + p / kBlock;
  const int page = a.page_table[at];
  if (page < 0 || page >= a.num_pages) {
    record_error(a.err, MSA_DEVERR_PAGE, at);
    return -1;
  }
  return static_cast<long long>(page) * kBlock + p % kBlock;
}

__global__ void __launch_bounds__(kQzThreads) dequantize_kernel(const __grid_constant__ DqArgs a) {
  __shared__ long long slots[kDqTokens];
  const int lane16 = threadIdx.x & 15, row = threadIdx.x / 16;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (long long t0 = static_cast<long long>(blockIdx.x) * kDqTokens; t0 < a.tokens; t0 += static_cast<long long>(gridDim.x) * kDqTokens) {
    if (threadIdx.x < kDqTokens) slots[threadIdx.x] = t0 + threadIdx.x < a.tokens ? dq_slot(a, t0 + threadIdx.x) : -2;
    __syncthreads();
    constexpr int kPasses = kDqTokens * kQzParts / kQzRows;
    uint2 x[kPasses];
    uint16_t s[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int u = i * kQzRows + row, part = u % kQzParts, g = part % kKvHeads;
      const long long slot = slots[u / kQzParts];
      x[i] = make_uint2(0u, 0u);
      s[i] = 0;
      if (slot < 0) continue;
      x[i] = reinterpret_cast<const uint2*>((part < kKvHeads ? a.k_cache : a.v_cache) + (slot * kKvHeads + g) * kDim)[lane16];
      s[i] = reinterpret_cast<const uint16_t*>(part < kKvHeads ? a.k_scales : a.v_scales)
          [((slot / kBlock) * kKvHeads + g) * kBlock + slot % kBlock];
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int u = i * kQzRows + row, part = u % kQzParts, g = part % kKvHeads;
      if (slots[u / kQzParts] == -2) continue;
      const uint32_t ss = s[i] * 0x10001u;
      uint4 y;
      y.x = mul_bf16x2(i8_lo2(x[i].x), ss);
      y.y = mul_bf16x2(i8_hi2(x[i].x), ss);
      y.z = mul_bf16x2(i8_lo2(x[i].y), ss);
      y.w = mul_bf16x2(i8_hi2(x[i].y), ss);
      __nv_bfloat16* out = part < kKvHeads ? a.k_out : a.v_out;
      reinterpret_cast<uint4*>(out + ((t0 + u / kQzParts) * kKvHeads + g) * kDim)[lane16] = y;
    }
    __syncthreads();
  }
}

cudaError_t launch_dequantize(const DequantizeLaunch& L, cudaStream_t stream) {
  if (const cudaError_t e = launch_prologue(); e != cudaSuccess) return e;
  const DqArgs a{static_cast<const int8_t*>(L.k_cache), static_cast<const int8_t*>(L.v_cache),
                 static_cast<const __nv_bfloat16*>(L.k_scales), static_cast<const __nv_bfloat16*>(L.v_scales), L.page_table,
                 L.starts, L.cu, L.batch, L.max_blocks, static_cast<int>(L.num_slots / kBlock), L.tokens,
                 static_cast<__nv_bfloat16*>(L.k_out), static_cast<__nv_bfloat16*>(L.v_out), L.err};
  const long long ctas = (L.tokens + kDqTokens - 1) / kDqTokens;
  return launch_dependent(dequantize_kernel, dim3(static_cast<unsigned>(std::min(ctas, 8LL * kNumSMs))), kQzThreads, 0, stream,
                          a);
}

}  // namespace msa
