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
#include "launch.h"

namespace msa {

constexpr int kQzThreads = 256;
constexpr int kQzRows = kQzThreads / 16;   // rows that a CTA takes at once
constexpr int kQzBatch = 2;                // and in flight per thread
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
// The larger magnitudes of two pairs (NaN where there is one), with some sign.
__device__ __forceinline__ uint32_t qz_max(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Eight values as bytes, with 1 / s = 2^(133 - field).  Added to 1.5 * 2^23, x / s is rounded to a whole number (ties to even) in
// the sum's low bits.  kAny: for any row; else for one with 1 / s in the range of fp32 and no value that rounds to 128.
template <bool kAny>
__device__ __forceinline__ void qz_row(const uint32_t (&w)[4], uint32_t field, uint32_t (&y)[2]) {
  constexpr float kRound = 12582912.f;
  const uint32_t u0 = kAny && field < 13 ? 13 - field : 0;  // 1 / s in two factors
  const float f = __uint_as_float((260 - field - u0) << 23), f0 = __uint_as_float((127 + u0) << 23);
  uint32_t n[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xffff0000u);
    if (kAny) {
      a *= f0;
      b *= f0;
    }
    const float2 t = fma2(a, b, f, f, kRound, kRound);
    n[2 * i] = __float_as_uint(kAny ? fminf(fmaxf(t.x, kRound - 127.f), kRound + 127.f) : t.x);
    n[2 * i + 1] = __float_as_uint(kAny ? fminf(fmaxf(t.y, kRound - 127.f), kRound + 127.f) : t.y);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    y[i] = __byte_perm(__byte_perm(n[4 * i], n[4 * i + 1], 0x0040), __byte_perm(n[4 * i + 2], n[4 * i + 3], 0x0040), 0x5410);
}

// Bound by the instructions of a row, so the offsets are counted in 32 bits where they fit, and rows that need care go another way.
// (17416 tokens, 54 MB: 10.8 us, 5.0 TB/s, the integer pipe 71% busy; 16.2 with a division, a
// conversion and a comparison per value.)
__global__ void __launch_bounds__(kQzThreads) quantize_kernel(const __grid_constant__ QzArgs a) {
  const uint32_t lane16 = threadIdx.x & 15, part = (threadIdx.x / 16) % kQzParts, g = part % kKvHeads;
  const bool is_v = part >= kKvHeads;
  // a warp's two rows are of one token: the lanes stay together
  constexpr uint32_t kTokens = kQzRows / kQzParts;  // that a CTA takes at once
  const uint32_t tokens = static_cast<uint32_t>(a.tokens), t0 = blockIdx.x * (kTokens * kQzBatch) + threadIdx.x / (16 * kQzParts);
  const __nv_bfloat16* from = (is_v ? a.v : a.k) + g * kDim + 8 * lane16;
  const long long stride = is_v ? a.v_stride : a.k_stride;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint4 x[kQzBatch];
  int64_t slot[kQzBatch];
#pragma unroll
  for (int b = 0; b < kQzBatch; ++b) {
    const uint32_t t = t0 + b * kTokens;
    x[b] = make_uint4(0u, 0u, 0u, 0u);
    slot[b] = -1;
    if (t >= tokens) continue;
    x[b] = *reinterpret_cast<const uint4*>(from + t * stride);
    slot[b] = a.slots[t];
  }
#pragma unroll
  for (int b = 0; b < kQzBatch; ++b) {
    const uint32_t w[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
    uint32_t top = qz_max(qz_max(w[0], w[1]), qz_max(w[2], w[3]));
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = qz_max(top, __shfl_xor_sync(0xffffffffu, top, d));
    top = max(top & 0x7fffu, (top >> 16) & 0x7fffu);
    if (slot[b] < 0) continue;  // (also a token behind the last)
    if (slot[b] >= a.num_slots) {
      if (part == 0 && lane16 == 0) record_error(a.err, MSA_DEVERR_PAGE, t0 + b * kTokens);
      continue;
    }
    uint32_t y[2] = {0u, 0u};
    const uint32_t field = top >> 7;
    // 1.992 * 2^e, the last number below 2^(e + 1), is 127.5 steps
    if (field < 13 || (top & 0x7fu) == 0x7fu) {
      if (field < 255) qz_row<true>(w, field, y);
    } else if (field < 255) {
      qz_row<false>(w, field, y);
    }
    const uint32_t s = static_cast<uint32_t>(slot[b]);
    *reinterpret_cast<uint2*>((is_v ? a.v_cache : a.k_cache) + static_cast<size_t>(s) * (kKvHeads * kDim) + g * kDim + 8 * lane16) =
        make_uint2(y[0], y[1]);
    if (lane16 == 0)
      reinterpret_cast<uint16_t*>(is_v ? a.v_scales : a.k_scales)
          [static_cast<size_t>(s / kBlock) * (kKvHeads * kBlock) + g * kBlock + s % kBlock] = static_cast<uint16_t>(qz_scale_bits(top));
  }
}

cudaError_t launch_quantize(const QuantizeLaunch& L, cudaStream_t stream) {
  if (const cudaError_t e = launch_prologue(); e != cudaSuccess) return e;
  const QzArgs a{static_cast<const __nv_bfloat16*>(L.k), static_cast<const __nv_bfloat16*>(L.v), L.k_stride, L.v_stride,
                 L.slots, L.tokens, L.num_slots, static_cast<int8_t*>(L.k_cache), static_cast<int8_t*>(L.v_cache),
                 static_cast<__nv_bfloat16*>(L.k_scales), static_cast<__nv_bfloat16*>(L.v_scales), L.err};
  constexpr long long kTokens = kQzRows / kQzParts * kQzBatch;
  const long long ctas = (L.tokens + kTokens - 1) / kTokens;
  return launch_dependent(quantize_kernel, dim3(static_cast<unsigned>(ctas)), kQzThreads, 0, stream, a);
}

// ---- read back ------------------------------------------------------------------------

// Bound by HBM where contexts are long (8 of up to 32k tokens, 402 MB: 66.6 us, 6.0 TB/s), by the way from cu over starts and the page
// table to the rows where they are short (4 of them: 3.6 us).  So a warp takes two tokens, whose 16 rows it asks for at
// once (one token: 70.8 us), and searches the requests by 32 lanes at a time, one round per factor of 32.

constexpr int kDqTokens = 16;  // tokens of a CTA: two per warp

struct DqArgs {
  const int8_t *k_cache, *v_cache;
  const __nv_bfloat16 *k_scales, *v_scales;
  const int32_t *page_table, *starts, *cu;
  int batch, max_blocks, num_pages;
  long long tokens;
  __nv_bfloat16 *k_out, *v_out;
  DevError* err;
};

// 32 requests, one per lane.
struct DqWindow {
  long long r, c0, c1, start;
  bool in;
};
// The window that begins with the request of output row t, or with one a little before it (the whole warp): the lanes look at
// 32 requests at once, apart as far as the batch wants it and then one after the other.
__device__ __forceinline__ DqWindow dq_window(const DqArgs& a, long long t, int lane) {
  int lo = 0;  // no request before it ends behind t
  for (int step = 1 << (5 * ((31 - __clz(max(a.batch - 1, 1))) / 5)); step > 1; step >>= 5) {
    // lane i: the last of the requests lo + i * step ..
    const long long r = lo + (lane + 1LL) * step - 1;
    const unsigned ends = __ballot_sync(0xffffffffu, r >= a.batch || a.cu[r + 1] > t);
    lo += step * (ends ? __ffs(ends) - 1 : 32);
  }
  const long long r = static_cast<long long>(lo) + lane;
  const bool in = r < a.batch;
  return DqWindow{r, in ? a.cu[r] : 0, in ? a.cu[r + 1] : 0, in && a.starts ? a.starts[r] : 0, in};
}
// The slot of output row t: -1 where its request or page is bad (a row of zeros), -2 where it belongs to no request of the window.
__device__ __forceinline__ long long dq_slot(const DqArgs& a, const DqWindow& w, long long t, int lane) {
  const unsigned ends = __ballot_sync(0xffffffffu, w.in && w.c1 > t);
  const int mine = ends ? __ffs(ends) - 1 : -1;
  long long slot = -2;
  if (lane == mine && w.c0 <= t) {
    slot = -1;
    const long long p = w.start + (t - w.c0), at = w.r * a.max_blocks + p / kBlock;
    if (w.c0 < 0 || w.start < 0 || w.start + (w.c1 - w.c0) > static_cast<long long>(a.max_blocks) * kBlock) {
      record_error(a.err, MSA_DEVERR_LENGTH, w.r);
    } else if (const int page = a.page_table[at]; page < 0 || page >= a.num_pages) {
      record_error(a.err, MSA_DEVERR_PAGE, at);
    } else {
      slot = static_cast<long long>(page) * kBlock + p % kBlock;
    }
  }
  return __shfl_sync(0xffffffffu, slot, max(mine, 0));
}

__global__ void __launch_bounds__(kQzThreads) dequantize_kernel(const __grid_constant__ DqArgs a) {
  const int lane = threadIdx.x & 31, lane16 = lane & 15, half = lane >> 4;
  const long long t0 = static_cast<long long>(blockIdx.x) * kDqTokens + 2 * (threadIdx.x / 32);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // a token's eight rows, two at a time (K's heads, then V's)
  uint2 x[2][4];
  uint16_t s[2][4];
  if (t0 >= a.tokens) return;
  DqWindow w = dq_window(a, t0, lane);
  long long slot[2] = {dq_slot(a, w, t0, lane), -2};
  if (t0 + 1 < a.tokens) {
    // (the same window, unless the second token's request lies behind it)
    if (!__any_sync(0xffffffffu, w.in && w.c1 > t0 + 1)) w = dq_window(a, t0 + 1, lane);
    slot[1] = dq_slot(a, w, t0 + 1, lane);
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int g = (2 * i + half) % kKvHeads;
      x[u][i] = make_uint2(0u, 0u);
      s[u][i] = 0;
      if (slot[u] < 0) continue;
      x[u][i] = reinterpret_cast<const uint2*>((i < 2 ? a.k_cache : a.v_cache) + (slot[u] * kKvHeads + g) * kDim)[lane16];
      s[u][i] = reinterpret_cast<const uint16_t*>(i < 2 ? a.k_scales : a.v_scales)
          [((slot[u] / kBlock) * kKvHeads + g) * kBlock + slot[u] % kBlock];
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (slot[u] == -2) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int g = (2 * i + half) % kKvHeads;
      const uint32_t ss = s[u][i] * 0x10001u;
      stg128(reinterpret_cast<uint4*>((i < 2 ? a.k_out : a.v_out) + ((t0 + u) * kKvHeads + g) * kDim) + lane16,
             mul_bf16x2(i8_lo2(x[u][i].x), ss), mul_bf16x2(i8_hi2(x[u][i].x), ss), mul_bf16x2(i8_lo2(x[u][i].y), ss),
             mul_bf16x2(i8_hi2(x[u][i].y), ss));
    }
  }
}

cudaError_t launch_dequantize(const DequantizeLaunch& L, cudaStream_t stream) {
  if (const cudaError_t e = launch_prologue(); e != cudaSuccess) return e;
  const DqArgs a{static_cast<const int8_t*>(L.k_cache), static_cast<const int8_t*>(L.v_cache),
                 static_cast<const __nv_bfloat16*>(L.k_scales), static_cast<const __nv_bfloat16*>(L.v_scales), L.page_table,
                 L.starts, L.cu, L.batch, L.max_blocks, static_cast<int>(L.num_slots / kBlock), L.tokens,
                 static_cast<__nv_bfloat16*>(L.k_out), static_cast<__nv_bfloat16*>(L.v_out), L.err};
  const long long ctas = (L.tokens + kDqTokens - 1) / kDqTokens;
  return launch_dependent(dequantize_kernel, dim3(static_cast<unsigned>(ctas)), kQzThreads, 0, stream, a);
}

}  // namespace msa
