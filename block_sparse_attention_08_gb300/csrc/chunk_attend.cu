// chunk_attend.cu -- causal attention of each request's new tokens over all its
// keys in the paged cache (bf16 or E4M3).
//
// out[t, h] = sum_j p_j v_j / sum_j p_j, p_j = 2^(x_j - m), x_j = scale log2(e)
// <q, k_j>, over the keys j <= the token's position; the running maximum m and
// the sums are kept in one pass over the keys (when m grows, the sums so far
// are multiplied by 2^(m_old - m_new)).
//
// This form: one warp per (token, query head), four dims per lane, one key at
// a time.
#include <cuda_fp8.h>

#include "launch.h"

namespace msa {

constexpr int kCaWarps = 8;

size_t attend_chunk_bytes(long long, int) { return 0; }

template <bool kFp8>
__device__ __forceinline__ float4 ca_load(const void* cache, long long at, int lane) {
  if (kFp8) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(cache) + at)[lane];
    const __nv_fp8_e4m3* b = reinterpret_cast<const __nv_fp8_e4m3*>(&w);
    return make_float4(float(b[0]), float(b[1]), float(b[2]), float(b[3]));
  }
  const uint2 w = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(cache) + at)[lane];
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

template <bool kFp8>
__global__ void __launch_bounds__(kCaWarps * 32) chunk_attend_kernel(ChunkLaunch a, float scale_log2) {
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * kCaWarps + (threadIdx.x >> 5);
  const long long t = w / kHeads;
  const int h = static_cast<int>(w - t * kHeads), g = h / kGroup;
  if (t >= a.tokens || t >= a.cu[a.batch]) return;
  int lo = 0, hi = a.batch - 1;  // the request r with cu[r] <= t < cu[r + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int len = a.seq_lens[lo], fresh = a.cu[lo + 1] - a.cu[lo];
  long long keys = min(static_cast<long long>(len), len - fresh + (t - a.cu[lo]) + 1);
  if (fresh > len || len > a.max_blocks * static_cast<long long>(kBlock)) {
    if (lane == 0) record_error(a.err, MSA_DEVERR_LENGTH, lo);
    keys = 0;
  }
  const float4 q = ca_load<false>(a.q, (t * kHeads + h) * kDim, lane);
  float m = -INFINITY, l = 0.f, c = 0.f;  // c: what the additions to l have rounded away
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (long long j = 0; j < keys; ++j) {
    const long long e = lo * static_cast<long long>(a.max_blocks) + j / kBlock;
    const int page = a.page_table[e];
    if (page < 0 || (page + 1LL) * kBlock > a.num_slots) {
      if (lane == 0) record_error(a.err, MSA_DEVERR_PAGE, e);
      j |= kBlock - 1;
      continue;
    }
    const long long at = ((static_cast<long long>(page) * kBlock + j % kBlock) * kKvHeads + g) * kDim;
    const float4 k = ca_load<kFp8>(a.k, at, lane), v = ca_load<kFp8>(a.v, at, lane);
    float x = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= scale_log2;
    const float mn = fmaxf(m, x), f = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(x - mn);
    const float lf = l * f, y = fmaf(-c, f, p), sum = lf + y;
    c = (sum - lf) - y;
    l = sum;
    o.x = o.x * f + p * v.x;
    o.y = o.y * f + p * v.y;
    o.z = o.z * f + p * v.z;
    o.w = o.w * f + p * v.w;
    m = mn;
  }
  const float inv = l > 0.f ? a.v_scale / l : 0.f;
  reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (t * kHeads + h) * kDim)[lane] =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (a.lse && lane == 0) a.lse[t * kHeads + h] = l > 0.f ? m + log2f(l) : -INFINITY;
}

cudaError_t launch_attend_chunk(const ChunkLaunch& L, cudaStream_t stream) {
  if (const cudaError_t e0 = launch_prologue(); e0 != cudaSuccess) return e0;
  const long long grid = (L.tokens * kHeads + kCaWarps - 1) / kCaWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const float scale_log2 = L.scale * 1.4426950408889634f * L.k_scale;
  if (L.kv_fp8) chunk_attend_kernel<true><<<static_cast<unsigned>(grid), kCaWarps * 32, 0, stream>>>(L, scale_log2);
  else chunk_attend_kernel<false><<<static_cast<unsigned>(grid), kCaWarps * 32, 0, stream>>>(L, scale_log2);
  return cudaGetLastError();
}

}  // namespace msa
