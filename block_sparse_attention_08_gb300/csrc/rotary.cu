// rotary.cu -- rotary positions with several axes on Q and K, with K and V
// written into the paged cache on the way.
//
// Pair j of a head turns by angle(t, j) = positions[axis[j]][t] * inv_freq[j]:
// a' = a cos - b sin, b' = a sin + b cos.  The turn is orthogonal, so its
// gradient is the turn by the negative angle: the backward is the same kernel.
//
// The product of a 31-bit position and a 24-bit frequency has 55 bits, of
// which fp32 would keep none of the fraction of a far position's angle; so
// each angle is formed and reduced to a fraction of a turn in binary64 (once
// per token and pair, shared by all heads) and sine and cosine are taken of
// that fraction in fp32.  The rotation is fp32, rounded once to the output
// type.
//
// Each row is read once and written once: bound by HBM.  A CTA takes
// kRoTokens tokens; its threads first fill a table of their (cos, sin) in
// shared memory, then take the heads' rows, eight lanes to a row, two 16-byte
// pieces to a lane, chosen so that a lane holds both members of its pairs.
#include <cuda_fp8.h>

#include "launch.h"

namespace msa {

constexpr int kRoThreads = 256;
constexpr int kRoTokens = 4;
constexpr int kRoLanes = 8;  // lanes per row of 128 dims

__device__ __forceinline__ void ro_unpack(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 ro_pack(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
// E4M3 of f / scale, saturating (one rounding of the quotient).
__device__ __forceinline__ uint2 ro_pack_e4m3(const float (&f)[8], float scale) {
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(f[2 * i + 1] / scale), "f"(f[2 * i] / scale));
  return make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
}

__global__ void __launch_bounds__(kRoThreads) rotary_kernel(RotaryLaunch a) {
  __shared__ float2 turn[kRoTokens][kDim / 2];
  const int tid = threadIdx.x;
  const long long t0 = static_cast<long long>(blockIdx.x) * kRoTokens;
  const int nt = static_cast<int>(min(static_cast<long long>(kRoTokens), a.tokens - t0));
  const int pairs = a.rot.rot_dim / 2;

  for (int i = tid; i < nt * pairs; i += kRoThreads) {
    const int tt = i / pairs, j = i - tt * pairs;
    const int p = a.positions[a.rot.axis[j] * a.tokens + t0 + tt];
    constexpr double kTurnsPerRadian = 0.15915494309189535;  // 1 / (2 pi)
    const double turns = static_cast<double>(p) * static_cast<double>(a.inv_freq[j]) * kTurnsPerRadian;
    float s, c;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
    turn[tt][j] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();

  const int kv = a.v ? kKvHeads : 0;
  const int rows = a.q_heads + a.k_heads + kv;  // per token: q, k, v
  const int turned = a.rot.rot_dim / 16;        // lanes of a row that turn their 16 dims
  const bool cross = !a.rot.interleaved;        // a lane's pieces hold the pairs' two members
  for (int u = tid; u < nt * rows * kRoLanes; u += kRoThreads) {
    const int lane = u % kRoLanes, row = u / kRoLanes;
    const int tt = row / rows, h = row - tt * rows;
    const long long t = t0 + tt;
    const bool is_q = h < a.q_heads, is_k = !is_q && h < a.q_heads + a.k_heads;
    const int head = is_q ? h : is_k ? h - a.q_heads : h - a.q_heads - a.k_heads;
    const __nv_bfloat16* src =
        is_q ? static_cast<const __nv_bfloat16*>(a.q) + t * a.q_stride
             : is_k ? static_cast<const __nv_bfloat16*>(a.k) + t * a.k_stride
                    : static_cast<const __nv_bfloat16*>(a.v) + t * a.v_stride;
    // pieces of 8 dims: a turned lane of the split form takes piece l and the one
    // rot_dim / 2 further on; every other lane takes 2 l and 2 l + 1
    const bool rot = lane < turned && (is_q || is_k);
    const bool split = cross && lane < turned;
    const int pa = split ? lane : 2 * lane, pb = split ? lane + turned : 2 * lane + 1;
    const uint4* s4 = reinterpret_cast<const uint4*>(src + head * kDim);
    float x[8], y[8];
    ro_unpack(s4[pa], x);
    ro_unpack(s4[pb], y);
    if (rot) {
      if (cross) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 cs = turn[tt][8 * lane + i];
          const float u0 = x[i], u1 = y[i];
          x[i] = u0 * cs.x - u1 * cs.y;
          y[i] = u0 * cs.y + u1 * cs.x;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 ca = turn[tt][8 * lane + i], cb = turn[tt][8 * lane + 4 + i];
          const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
          x[2 * i] = x0 * ca.x - x1 * ca.y;
          x[2 * i + 1] = x0 * ca.y + x1 * ca.x;
          y[2 * i] = y0 * cb.x - y1 * cb.y;
          y[2 * i + 1] = y0 * cb.y + y1 * cb.x;
        }
      }
    }
    if (is_q || (is_k && a.k_out)) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_q ? a.q_out : a.k_out) +
                           (t * (is_q ? a.q_heads : a.k_heads) + head) * kDim;
      uint4* d4 = reinterpret_cast<uint4*>(dst);
      d4[pa] = ro_pack(x);
      d4[pb] = ro_pack(y);
    }
    if (!is_q && a.k_cache) {
      const long long slot = a.slots[t];
      if (slot >= a.num_slots) {
        record_error(a.err, MSA_DEVERR_PAGE, t);
      } else if (slot >= 0) {
        const long long at = (slot * kKvHeads + head) * kDim;
        void* cache = is_k ? a.k_cache : a.v_cache;
        if (a.kv_fp8) {
          const float scale = is_k ? a.k_scale : a.v_scale;
          uint2* d2 = reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at);
          d2[pa] = ro_pack_e4m3(x, scale);
          d2[pb] = ro_pack_e4m3(y, scale);
        } else {
          uint4* d4 = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + at);
          d4[pa] = ro_pack(x);
          d4[pb] = ro_pack(y);
        }
      }
    }
  }
}

cudaError_t launch_rotary(const RotaryLaunch& L, cudaStream_t stream) {
  if (const cudaError_t e0 = launch_prologue(); e0 != cudaSuccess) return e0;
  const long long grid = (L.tokens + kRoTokens - 1) / kRoTokens;
  rotary_kernel<<<static_cast<unsigned>(grid), kRoThreads, 0, stream>>>(L);
  return cudaGetLastError();
}

}  // namespace msa
