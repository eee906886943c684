// int8_attend.cuh -- one warp's attention of 16 query heads over keys of an int8
// cache, from tiles in shared memory: what the decode attention and the chunk
// attention's one-token items have in common.
//
// Products of m16n8k16, the 16 heads their rows, 32 keys at a time.  A 16-bit ldmatrix of
// K gives a lane four consecutive bytes of one key, dims 16 c + 4 t .. + 3 of
// k-step c; a transposing one of V gives it two dims of two keys.  Both are two
// pairs (bytes 0 and 2, 1 and 3) once widened to bf16, so Q's fragments hold
// dims 4 t, + 2 in the slots of a k-step's first half and 4 t + 1, + 3 in those of its
// second, and O's n-tiles 2 c and 2 c + 1 are the even and the odd dims of block c.
// A key's scale multiplies its scores, a value's scale its weight (rounded to
// bf16 before; a power of two keeps that exact).
//
// Bound by the instructions that it issues: seven for the four values of a word, five of them
// on the half-rate integer pipe.  So no lane masks, tests or counts what a full group of keys does
// not need, and a warp takes 32 keys for each wait on a barrier.  (Three of them on that pipe and six on
// the other, with the sign taken off by a fused operation that ends at zero: 364 us instead of 339 for 16 tokens over 128k
// keys.)
#pragma once

#include "common.cuh"

namespace msa {

// (w & kMask) | magic, in one instruction (of two constants the compiler makes two).
template <uint32_t kMask>
__device__ __forceinline__ uint32_t i8_part(uint32_t w, uint32_t magic) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "n"(kMask), "r"(magic));
  return d;
}
// The halves' upper bytes, as a register whose value the compiler does not know.
__device__ __forceinline__ uint32_t i8_magic() {
  uint32_t m;
  asm volatile("mov.b32 %0, 0x43004300;" : "=r"(m));
  return m;
}
// The even (bytes 0, 2) and the odd (1, 3) values of a word, exactly, as bf16x2 (i8_pair, without the byte permutation).
__device__ __forceinline__ void i8_pairs(uint32_t w, uint32_t& even, uint32_t& odd, uint32_t magic) {
  const uint32_t v = w >> 8;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(even) : "r"(i8_part<0x007f007fu>(w, magic)), "r"(i8_part<0x00800080u>(w, magic)));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(odd) : "r"(i8_part<0x007f007fu>(v, magic)), "r"(i8_part<0x00800080u>(v, magic)));
}
// Q's fragments of a k-step from the words of dims 4 t .. + 3 of rows g8 (a) and g8 + 8 (b).
__device__ __forceinline__ void i8_queries(uint32_t (&q)[4], uint2 a, uint2 b) {
  q[0] = __byte_perm(a.x, a.y, 0x5410);
  q[1] = __byte_perm(b.x, b.y, 0x5410);
  q[2] = __byte_perm(a.x, a.y, 0x7632);
  q[3] = __byte_perm(b.x, b.y, 0x7632);
}

// The sums against a reference m are raised when a maximum passes it by more than this, in base 2.
constexpr float kI8Slack = 8.f;

// rows g8 ([0], o[.][0..1]) and g8 + 8 ([1], o[.][2..3]); l: this lane's part
struct I8State {
  float m[2], l[2];
  float o[16][4];
};
__device__ __forceinline__ void i8_clear(I8State& st) {
  st.m[0] = st.m[1] = -INFINITY;
  st.l[0] = st.l[1] = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
}

// A product that begins a sum.
__device__ __forceinline__ void i8_mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The products of 32 keys, 8 i + 2 t, + 1 (x[i]) of rows g8 (0, 1) and g8 + 8 (2, 3), become weights: ks and vs hold the scales
// of those two keys.  The reference is raised where a maximum passes it by kI8Slack; l takes the weights, pa the A
// operands of the products with V.  kAll: all 32 keys count, else the first `keys`.
template <bool kAll>
__device__ __forceinline__ void i8_weigh(I8State& st, float (&x)[4][4], uint32_t (&pa)[2][4], const uint32_t (&ks)[4],
                                         const uint32_t (&vs)[4], int keys, float scale_log2, int t4) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f0 = scale_log2 * __uint_as_float(ks[i] << 16), f1 = scale_log2 * __uint_as_float(ks[i] & 0xffff0000u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[i][e] *= e & 1 ? f1 : f0;
      if (!kAll && 8 * i + 2 * t4 + (e & 1) >= keys) x[i][e] = -INFINITY;
    }
  }
  float top[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    top[h] = fmaxf(fmax3(fmax3(x[0][2 * h], x[0][2 * h + 1], x[1][2 * h]), x[1][2 * h + 1], x[2][2 * h]),
                   fmax3(x[2][2 * h + 1], x[3][2 * h], x[3][2 * h + 1]));
  if (__any_sync(0xffffffffu, top[0] > st.m[0] + kI8Slack || top[1] > st.m[1] + kI8Slack)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
      const bool raise = top[h] > st.m[h] + kI8Slack;
      const float f = raise && st.m[h] != -INFINITY ? ex2(st.m[h] - top[h]) : 1.f;
      if (raise) st.m[h] = top[h];
      st.l[h] *= f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        st.o[i][2 * h] *= f;
        st.o[i][2 * h + 1] *= f;
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float mu = st.m[h] == -INFINITY ? 0.f : st.m[h];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p0 = ex2(x[i][2 * h] - mu), p1 = ex2(x[i][2 * h + 1] - mu);
      st.l[h] += p0 + p1;
      uint32_t v = vs[i];
      // what lies behind the last key has no weight, whatever its scale
      if (!kAll) v &= (8 * i + 2 * t4 < keys ? 0xffffu : 0u) | (8 * i + 2 * t4 + 1 < keys ? 0xffff0000u : 0u);
      pa[i >> 1][2 * (i & 1) + h] = mul_bf16x2(pack_bf16(p0, p1), v);
    }
  }
}

// This lane's row addresses for ldmatrix in a tile of 128-byte rows (swizzled), of the 16 rows from `row` on: two k-steps of 16
// dims each.  (The 16 rows behind them lie 2048 bytes further on.)
__device__ __forceinline__ void i8_offsets(uint32_t (&at)[4], int row, int lane) {
  const int mi = lane >> 3;
#pragma unroll
  for (int c = 0; c < 4; ++c) at[c] = sw128(row + 8 * (mi & 1) + (lane & 7), 2 * c + (mi >> 1));
}

// 32 keys, from the rows at `at` of the K and V tiles (i8_offsets) on, of which the first `keys` count (at least one).  ks, vs:
// the scales of keys 2 t, + 1 (at [0]), 8 + 2 t, + 1 (at [4]) and so on.  qa(c, a) puts Q's fragments of k-step c into a.
template <class Queries>
__device__ __forceinline__ void i8_attend32(I8State& st, const Queries& qa, uint32_t kt, uint32_t vt,
                                            const uint32_t (&at)[4], const uint32_t* ks, const uint32_t* vs, int keys,
                                            float scale_log2, int t4) {
  constexpr uint32_t kNext = 16 * 128;
  const uint32_t magic = i8_magic();
  uint32_t kw[4], vw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    kw[i] = ks[4 * i];
    vw[i] = vs[4 * i];
  }
  float x[4][4];
  uint32_t r[2][2][4];  // [c & 1][16 keys]: keys 0-7 and 8-15 of k-step 2 c, then of 2 c + 1; the next asked for before
#pragma unroll
  for (int u = 0; u < 2; ++u) ldsm_x4(r[0][u], kt + at[0] + u * kNext);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c < 3)
#pragma unroll
      for (int u = 0; u < 2; ++u) ldsm_x4(r[(c + 1) & 1][u], kt + at[c + 1] + u * kNext);
    else
#pragma unroll
      for (int u = 0; u < 2; ++u) ldsm_x4_t(r[0][u], vt + at[0] + u * kNext);  // dims 32 c .., then 32 c + 16 ..
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t q[4];
      qa(2 * c + h, q);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t e, o;
          i8_pairs(r[c & 1][u][2 * h + i], e, o, magic);
          if (c == 0 && h == 0) i8_mma_first(x[2 * u + i], q, e, o);
          else mma_bf16(x[2 * u + i], q, e, o);
        }
    }
  }
  uint32_t pa[2][4];
  if (keys >= 32) i8_weigh<true>(st, x, pa, kw, vw, keys, scale_log2, t4);
  else i8_weigh<false>(st, x, pa, kw, vw, keys, scale_log2, t4);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c < 3)
#pragma unroll
      for (int u = 0; u < 2; ++u) ldsm_x4_t(r[(c + 1) & 1][u], vt + at[c + 1] + u * kNext);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t e0, o0, e1, o1;
        i8_pairs(r[c & 1][u][2 * i], e0, o0, magic);
        i8_pairs(r[c & 1][u][2 * i + 1], e1, o1, magic);
        mma_bf16(st.o[2 * (2 * c + i)], pa[u], e0, e1);
        mma_bf16(st.o[2 * (2 * c + i) + 1], pa[u], o0, o1);
      }
  }
  // the caller gives the tiles back next: no load of them may be put off until then
#pragma unroll
  for (int u = 0; u < 2; ++u)
    asm volatile("" ::"r"(r[1][u][0]), "r"(r[1][u][1]), "r"(r[1][u][2]), "r"(r[1][u][3]) : "memory");
}

}  // namespace msa
