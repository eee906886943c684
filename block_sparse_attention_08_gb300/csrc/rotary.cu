// rotary.cu -- rotary positions with several axes on Q and K, with K and V
// written into the paged cache on the way.
//
// Pair j of a head turns by angle(t, j) = positions[axis[j]][t] * inv_freq[j]:
// a' = a cos - b sin, b' = a sin + b cos.  The turn is orthogonal, so its
// gradient is the turn by the negative angle: the backward is the same kernel.
//
// The angle of a far position keeps nothing of its fraction in fp32, so it is
// reduced to a fraction of a turn before it is rounded: with u = inv_freq /
// (2 pi) as a sum of two floats (exact products by fused multiply-adds), the
// position times u is a sum of two floats, whose whole turns are dropped.  Below
// 2^20 turns, for a position that is a float, the last sum's rounding is 2^-25 of
// a turn and the others together less than 2^-25; a position from 2^24 on, or
// more turns, takes the product in pairs of binary64 (1 / (2 pi) to 106 bits).
// Either way the fraction is within 2^-24 of a turn, for |inv_freq| up to 2^32.
// Sine and cosine are those of that fraction, once per token and pair, shared by
// all heads; the rotation is fp32, rounded once to the output type.
//
// Each row is read once and written once: bound by HBM.  A CTA takes every
// gridDim-th token through a ring of stages in shared memory: a producer warp
// fills the stage's table of (cos, sin) and copies the token's rows in with the
// bulk-copy engine; nine warps turn them where they are, eight lanes to a row of
// 128 dims, two 16-byte pieces to a lane, chosen so that a lane holds both
// members of its pairs; the producer copies the stage out, to q_out and (as they
// lie there, or from the E4M3 bytes that the warps leave beside them) to the
// caches' slots.  So no thread holds data that is on its way, and an SM has
// kRoStages tokens of each of its CTAs in flight, 18 KB each.  16384 tokens with
// insertion (604 MB): 98 us, 6.2 TB/s; 8191 into E4M3 caches (294 MB): 51.5 us,
// 5.7 TB/s; forward and backward of 16384 (1.14 GB): 195 us, 5.9 TB/s; 64
// tokens: 3.6 us.  With few heads a CTA's producer, a token after the other,
// bounds it (65536 tokens of 8 + 1 heads, 302 MB: 210 us).
#include <algorithm>

#include "launch.h"

namespace msa {

constexpr int kRoLanes = 8;    // lanes per row of 128 dims
constexpr int kRoWarps = 9;    // turning warps: four rows each at a time, so 72 rows in two passes
constexpr int kRoStages = 4;
constexpr int kRoThreads = 32 * (kRoWarps + 1);
constexpr int kRoResident = 3;  // CTAs that an SM's registers hold: 64 a thread
constexpr int kRoRow = kDim * 2;
constexpr int kRoMaxStage = 2 * kHeads * kRoRow;  // 64 heads of q and of k (with insertion 72 rows and 1 KB)

// (cos, sin) of position * inv_freq.
__device__ __forceinline__ float2 ro_turn(int position, float inv_freq) {
  // 1 / (2 pi) as the sum of two floats
  constexpr float kHi = 0.15915494f, kLo = static_cast<float>(0.15915494309189535 - static_cast<double>(kHi));
  const float p = static_cast<float>(position);
  const float u = inv_freq * kHi, u_lo = fmaf(inv_freq, kLo, fmaf(inv_freq, kHi, -u)), t = p * u;
  float turns;
  if (position > -(1 << 24) && position < (1 << 24) && fabsf(t) < 0x1p20f) {
    const float t_lo = fmaf(p, u_lo, fmaf(p, u, -t));  // less than 2^-2
    turns = (t - rintf(t)) + t_lo;
  } else {
    constexpr double kHi2 = 0x1.45f306dc9c883p-3, kLo2 = -0x1.6b01ec5417056p-57;
    const double f = inv_freq, x = position * f, x_lo = fma(static_cast<double>(position), f, -x);
    const double y = x * kHi2, y_lo = fma(x, kLo2, fma(x, kHi2, -y)) + x_lo * kHi2;  // at most 2^9 (|y| < 2^61)
    turns = static_cast<float>((y - rint(y)) + (y_lo - rint(y_lo)));
  }
  float s, c;
  sincospif(2.f * turns, &s, &c);
  return make_float2(c, s);
}

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

// Copy shared -> global by the bulk-copy engine (16-byte aligned, bytes % 16 == 0; bulk group).
__device__ __forceinline__ void ro_copy_out(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
// NaN in a token's rows of q_out and k_out (the whole warp): 16 bytes, eight bf16 NaN, at a time.
__device__ __noinline__ void ro_mark(void* q_out, int q_bytes, void* k_out, int k_bytes, long long t) {
  constexpr uint32_t kNan = 0x7fff7fffu;
  const int lane = threadIdx.x & 31;
  for (int o = 16 * lane; o < q_bytes; o += 16 * 32) stg128(static_cast<uint8_t*>(q_out) + t * q_bytes + o, kNan, kNan, kNan, kNan);
  if (k_out)
    for (int o = 16 * lane; o < k_bytes; o += 16 * 32) stg128(static_cast<uint8_t*>(k_out) + t * k_bytes + o, kNan, kNan, kNan, kNan);
}
// A bounded wait; the error word may be missing.
__device__ __forceinline__ bool ro_wait(uint64_t* bar, uint32_t parity, DevError* err, int where) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  do {
    if (mbar_try_wait_suspend(bar, parity)) return true;
  } while (global_ns() - t0 < kWaitNs);
  if (err) record_error(err, MSA_DEVERR_TIMEOUT, where);
  return false;
}

// A stage: the token's q, k and v rows, then (E4M3 caches) 1 KB of K and V bytes.
struct RoGeom {
  int q_bytes, k_bytes, v_bytes, stage;
};

__global__ void __launch_bounds__(kRoThreads) rotary_kernel(const __grid_constant__ RotaryLaunch a, RoGeom geo) {
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ __align__(16) float2 turn[kRoStages][kDim / 2];
  __shared__ uint64_t full[kRoStages], done[kRoStages];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kRoStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&done[i], kRoWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  // the kernel before has completed; the next may be launched behind this one
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long t0 = blockIdx.x;
  const int n = static_cast<int>((a.tokens - t0 + gridDim.x - 1) / gridDim.x);  // tokens of this CTA
  auto token = [&](int i) { return t0 + static_cast<long long>(i) * gridDim.x; };
  const int pairs = a.rot.rot_dim / 2;

  if (warp == kRoWarps) {
    // ---------------- producer ----------------
    // each lane turns two pairs of a token; positions and slot are asked for one token ahead
    const float f0 = lane < pairs ? a.inv_freq[lane] : 0.f, f1 = lane + 32 < pairs ? a.inv_freq[lane + 32] : 0.f;
    const int32_t* at0 = a.positions + (lane < pairs ? a.rot.axis[lane] : 0) * a.tokens;
    const int32_t* at1 = a.positions + (lane + 32 < pairs ? a.rot.axis[lane + 32] : 0) * a.tokens;
    int p0 = at0[t0], p1 = at1[t0];
    long long slots[kRoStages];  // of the tokens in flight
    const bool insert = a.k_cache != nullptr;
    int out = 0;  // where a wait gave up: tokens copied out
    // copies token i's stage out
    auto copy_out = [&](int i, long long slot) {
      const int s = i % kRoStages;
      if (!__all_sync(0xffffffffu, ro_wait(&done[s], (i / kRoStages) & 1, a.err, 850))) {
        out = i;
        return false;
      }
      if (lane == 0) {
        const long long t = token(i);
        const uint8_t* st = stages + s * geo.stage;
        ro_copy_out(static_cast<uint8_t*>(a.q_out) + t * geo.q_bytes, st, geo.q_bytes);
        if (a.k_out) ro_copy_out(static_cast<uint8_t*>(a.k_out) + t * geo.k_bytes, st + geo.q_bytes, geo.k_bytes);
        if (slot >= a.num_slots) {
          record_error(a.err, MSA_DEVERR_PAGE, t);
        } else if (slot >= 0) {
          const int bytes = kKvHeads * kDim * (a.kv_fp8 ? 1 : 2);
          const uint8_t* kv = st + geo.q_bytes + (a.kv_fp8 ? geo.k_bytes + geo.v_bytes : 0);
          ro_copy_out(static_cast<uint8_t*>(a.k_cache) + slot * bytes, kv, bytes);
          ro_copy_out(static_cast<uint8_t*>(a.v_cache) + slot * bytes, kv + bytes, bytes);
        }
        bulk_commit();
      }
      return true;
    };
    bool ok = true;
    for (int base = 0; base < n + kRoStages && ok; base += kRoStages) {
#pragma unroll
      for (int s = 0; s < kRoStages; ++s) {
        const int i = base + s;
        if (i >= n + kRoStages || !ok) break;
        if (i >= kRoStages && i - kRoStages < n) ok = copy_out(i - kRoStages, slots[s]);
        if (!ok || i >= n) continue;
        const int c0 = p0, c1 = p1;
        slots[s] = insert ? a.slots[token(i)] : -1;
        if (i + 1 < n) {
          p0 = at0[token(i + 1)];
          p1 = at1[token(i + 1)];
        }
        if (lane < pairs) {
          const float2 cs = ro_turn(c0, f0);
          turn[s][lane] = make_float2(cs.x, a.inverse ? -cs.y : cs.y);
        }
        if (lane + 32 < pairs) {
          const float2 cs = ro_turn(c1, f1);
          turn[s][lane + 32] = make_float2(cs.x, a.inverse ? -cs.y : cs.y);
        }
        __syncwarp();
        if (lane == 0) {
          bulk_wait_read_all();  // the stage has been copied out
          const long long t = token(i);
          uint8_t* st = stages + s * geo.stage;
          mbar_expect_tx(&full[s], geo.q_bytes + geo.k_bytes + geo.v_bytes);
          tma_bulk_g2s(st, static_cast<const __nv_bfloat16*>(a.q) + t * a.q_stride, geo.q_bytes, &full[s]);
          if (geo.k_bytes)
            tma_bulk_g2s(st + geo.q_bytes, static_cast<const __nv_bfloat16*>(a.k) + t * a.k_stride, geo.k_bytes,
                         &full[s]);
          if (geo.v_bytes)
            tma_bulk_g2s(st + geo.q_bytes + geo.k_bytes, static_cast<const __nv_bfloat16*>(a.v) + t * a.v_stride,
                         geo.v_bytes, &full[s]);
        }
        __syncwarp();
      }
    }
    if (!ok) {
      // after a wait that gave up: the last fill of each stage may still be landing, and the tokens that were not copied out
      // get NaN rows (a call without an error word shows it there)
      const int filled = min(out + kRoStages, n);  // tokens asked for: a stage is filled again once it has been copied out
      for (int s = 0; s < kRoStages; ++s) {
        const int fills = (filled - s + kRoStages - 1) / kRoStages;
        if (fills > 0) ro_wait(&full[s], (fills - 1) & 1, a.err, 852);
      }
      for (int j = out; j < n; ++j) ro_mark(a.q_out, geo.q_bytes, a.k_out, geo.k_bytes, token(j));
    }
    if (lane == 0) bulk_wait_all();
  } else {
    // ---------------- turning warps ----------------
    const int l = lane % kRoLanes, turned = a.rot.rot_dim / 16;  // lanes of a row that turn their 16 dims
    const bool cross = !a.rot.interleaved;
    // pieces of 8 dims: a turned lane of the split form takes piece l and the one rot_dim / 2 further on; every other lane
    // takes 2 l and 2 l + 1
    const bool split = cross && l < turned;
    const int pa = split ? l : 2 * l, pb = split ? l + turned : 2 * l + 1;
    const int qk = a.q_heads + a.k_heads, rows = a.kv_fp8 ? qk + kKvHeads : qk;  // (bf16 V rows pass untouched)
    for (int i = 0; i < n; ++i) {
      const int s = i % kRoStages;
      if (!__all_sync(0xffffffffu, ro_wait(&full[s], (i / kRoStages) & 1, a.err, 851))) break;
      uint8_t* st = stages + s * geo.stage;
      float2 cs[8];
      if (l < turned) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 v = reinterpret_cast<const float4*>(turn[s])[4 * l + j];
          cs[2 * j] = make_float2(v.x, v.y);
          cs[2 * j + 1] = make_float2(v.z, v.w);
        }
      }
#pragma unroll 2
      for (int h = warp * 4 + lane / kRoLanes; h < rows; h += kRoWarps * 4) {
        uint4* row = reinterpret_cast<uint4*>(st + h * kRoRow);
        const bool turns = l < turned && h < qk;
        if (!turns && h < a.q_heads) continue;
        float x[8], y[8];
        ro_unpack(row[pa], x);
        ro_unpack(row[pb], y);
        if (turns) {
          if (cross) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float x0 = x[j], y0 = y[j];
              x[j] = x0 * cs[j].x - y0 * cs[j].y;
              y[j] = x0 * cs[j].y + y0 * cs[j].x;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float x0 = x[2 * j], x1 = x[2 * j + 1], y0 = y[2 * j], y1 = y[2 * j + 1];
              x[2 * j] = x0 * cs[j].x - x1 * cs[j].y;
              x[2 * j + 1] = x0 * cs[j].y + x1 * cs[j].x;
              y[2 * j] = y0 * cs[4 + j].x - y1 * cs[4 + j].y;
              y[2 * j + 1] = y0 * cs[4 + j].y + y1 * cs[4 + j].x;
            }
          }
          row[pa] = ro_pack(x);
          row[pb] = ro_pack(y);
        }
        if (a.kv_fp8 && h >= a.q_heads) {
          uint2* d2 = reinterpret_cast<uint2*>(st + qk * kRoRow + geo.v_bytes + (h - a.q_heads) * kDim);
          const float scale = h < qk ? a.k_scale : a.v_scale;
          d2[pa] = ro_pack_e4m3(x, scale);
          d2[pb] = ro_pack_e4m3(y, scale);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&done[s]);
    }
  }
}

cudaError_t launch_rotary(const RotaryLaunch& L, cudaStream_t stream) {
  if (const cudaError_t e0 = launch_prologue(); e0 != cudaSuccess) return e0;
  RoGeom geo;
  geo.q_bytes = L.q_heads * kRoRow;
  geo.k_bytes = L.k_heads * kRoRow;
  geo.v_bytes = L.v ? kKvHeads * kRoRow : 0;
  geo.stage = (geo.q_bytes + geo.k_bytes + geo.v_bytes + (L.kv_fp8 ? 2 * kKvHeads * kDim : 0) + 127) / 128 * 128;
  const int bytes = kRoStages * geo.stage;
  // The limit belongs to the kernel, not to the call: it is set to the same value by every call, since one thread's smaller
  // limit between another's setting and launch would refuse that launch.
  static_assert(kRoMaxStage >= (kHeads + 2 * kKvHeads) * kRoRow + 2 * kKvHeads * kDim, "a stage with insertion");
  if (const cudaError_t e = cudaFuncSetAttribute(rotary_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kRoStages * kRoMaxStage);
      e != cudaSuccess)
    return e;
  // As many CTAs as are resident at once, by registers and shared memory, each through its share of the tokens.  (Six where
  // shared memory held six: 600 tokens of 8 + 1 heads 6.3 us instead of 5.0, 65536 tokens 204 us either way.)
  const int per_sm = std::min(kRoResident, 228 * 1024 / (bytes + 3584));
  const long long grid = std::min<long long>(L.tokens, static_cast<long long>(kNumSMs) * per_sm);
  return launch_dependent(rotary_kernel, dim3(static_cast<unsigned>(grid)), kRoThreads, bytes, stream, L, geo);
}

}  // namespace msa
