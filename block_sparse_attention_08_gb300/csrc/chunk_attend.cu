// chunk_attend.cu -- causal attention of each request's new tokens over all its
// keys in the paged cache (bf16 or E4M3).
//
// out[t, h] = sum_j p_j v_j / sum_j p_j, p_j = 2^(x_j - m), x_j = scale log2(e)
// <q, k_j>, over the keys j <= the token's position.  One pass over the keys, a
// block of 128 at a time: the sums are taken against a reference m, and when a
// block's maximum passes it by more than kCaSlack (the weights would grow past
// 2^kCaSlack) m is raised and the sums so far are multiplied by
// 2^(m_old - m_new).
//
// An item is 16 consecutive new tokens of a request and one KV head: 256 rows
// (token, query head) that share their keys, as two tiles of 128 rows.  Its work
// is counted in units: a 128-key block of both tiles, or two blocks of one tile
// (which run side by side, below).  Every CTA takes an equal contiguous share of
// all units of the batch, wherever that cuts an item: a long context with one
// new token is spread over the GPU like a long chunk is.  The
// pieces of a cut item leave (m, sum of p, sum of p v) in scratch, and a second
// kernel joins them.  Each CTA finds its share itself from the lengths (no
// planning launch, nothing kept between calls).
//
// Roles: a producer warp walks the share and copies Q rows and K and V pages by
// TMA; an MMA thread issues S = Q K^T and O += P V on the tensor cores (S, P and
// O in tensor memory, P over the S it came from); two warpgroups turn S into P,
// one row per thread.  With more than 8 tokens each warpgroup owns a tile, and
// all blocks pass both; with 8 or fewer there is one tile, and the warpgroups
// take its blocks in turn, each into sums of its own, joined at the end: the
// tensor cores work on one block while the other's softmax runs.  An E4M3 cache
// has a third warpgroup that widens each page to fp16 (exactly) in shared memory.
//
// That widening writes and reads every tile once more, and shared memory's rate
// then bounds an item of one new token, which needs only 16 of a tile's 128 rows
// (0.48 ms for 16 tokens over 128k E4M3 keys, 0.32 ms as below).  So over an
// E4M3 cache the items of one token are shared out apart, after the others, and
// the softmax warps compute them with warp-level products straight from the
// copied bytes: each warp takes some of a block's keys, with sums of its own in
// registers, joined at the item's end.  Over a bf16 cache that saves an item's
// way through tensor memory (64 tokens over 300 to 900 keys: 28 us instead of
// 36; over 4k to 64k keys 0.58 ms either way), but not what a second kind of
// shares costs: it is done where all items have one token (17 mixed requests
// took 0.118 ms with two kinds, 0.095 with one).
//
// Chunks are bound on chip.  2048 tokens over 32k keys take 1.22 ms in bf16 (1.7
// PFLOP/s, tensor pipe 74% active, 92% of a library product's rate), and 1.31 to
// 1.35 ms in a row, where power bounds the clock:
// what is left is the way from S over the softmax to O.  An item costs about two
// units besides its blocks: 0.5 us for its last O product, 2.4 for its rows'
// stores, 1 for the first block's softmax, none of it beside other products.
// An E4M3 cache adds the widening and leaves the softmax fewer registers:
// 1.38 ms.  Single tokens over long contexts are bound by HBM (64 requests,
// 4.0 GB: 0.58 ms, 6.9 TB/s), short ones by latency: 4.6 us without any work,
// 8.2 with one block.
#include <cuda_fp16.h>

#include <type_traits>

#include "launch.h"

namespace msa {

constexpr int kCaTok = 16;            // new tokens per item
constexpr int kCaTile = 128 * 256;    // 128 rows x 128 dims of 16 bits
constexpr int kCaHalf = kCaTile / 2;  // one 64-dim half
constexpr int kCaQEntry = 4096;       // one token's 16 heads x 128 dims
constexpr int kCaInfo = 4;            // item descriptors in flight
constexpr int kCaOnePlaces = 5;       // blocks in flight of one-token items (32 KB each)
constexpr int kCaBad = 8;             // block flags in flight (at most 5 blocks are)
// warps 0-7 softmax, 8 producer, 9 MMA, 10 bad requests (11 fills their warpgroup), 12-15 widening
constexpr int kCaProducerWarp = 8, kCaMmaWarp = 9, kCaWidenWarp = 12;
constexpr float kCaSlack = 8.f;
// Units that an item counts besides its blocks, for its start and its end: none where shares are short, since a share is
// at least that much longer than a unit, 1 in shares of 4 units on, 2 from 16 on.  (In half units: 17 mixed requests
// 0.103 ms with 0, 0.092 with 2; E4M3 chunks 0.601 with 0, 0.593 with 2, 0.573 with 4; four short single tokens
// 0.016 with 0 and 2, 0.019 with 4.  2048 tokens of a request without a past, 32 units a share: 0.097 with 2, 0.089 with 4.)
__device__ __forceinline__ int ca_item_units(long long total) {
  return total >= 16LL * gridDim.x ? 2 : total >= 4LL * gridDim.x ? 1 : 0;
}
// tensor memory: S of warpgroup w at 128 w, P over its first half, O at 256 + 128 w
constexpr uint32_t kCaOCol = 256;

// The K and V tiles of a piece of nb blocks are loaded in the order K0 K1 V0 K2 V1 ... V(nb-2) V(nb-1): V is needed a
// softmax later than its K, so the next block's K goes before it.  Tile number of K or V of block b:
__device__ __forceinline__ int ca_load_k(int b) { return b == 0 ? 0 : 2 * b - 1; }
__device__ __forceinline__ int ca_load_v(int b, int nb) { return b == nb - 1 ? 2 * nb - 1 : 2 * b + 2; }
// and the other way round (tile j that is not a V tile is K of block (j + 1) / 2)
__device__ __forceinline__ bool ca_is_v(int j, int nb) { return j > 0 && ((j & 1) == 0 || j == 2 * nb - 1); }
__device__ __forceinline__ int ca_block_v(int j, int nb) { return j == 2 * nb - 1 ? nb - 1 : (j - 2) >> 1; }

// A piece of an item: blocks b0 .. b0 + nb - 1.  nb = 0 ends the list.
struct CaItem {
  int t0, ntok, g;  // first row of q, tokens, KV head
  int pos0, len;    // position of the first token, keys of the request
  int b0, nb;
  int slot;         // partial slot, or -1: the piece is the whole item
};
// For the joining kernel: an item that begins in CTA c and ends in CTA `last`.
struct CaCut {
  int t0, ntok, g, last;
};

struct CaArgs {
  const __nv_bfloat16* q;
  const int32_t* seq_lens;
  const int32_t* page_table;
  const int32_t* cu;
  int batch, max_blocks, num_pages;
  long long tokens;
  float scale_log2, v_scale;
  __nv_bfloat16* out;
  float* lse;
  CaCut* cuts;      // [kNumSMs]
  float4* part_o;   // [2 kNumSMs][32][rows]: four dims of each row
  float2* part_ml;  // [2 kNumSMs][rows]
  int rows;         // rows of a partial slot
  // the same for one-token items over an E4M3 cache: 16 rows
  CaCut* cuts1;     // [kNumSMs]
  float4* part1_o;  // [2 kNumSMs][32][16]
  float2* part1_ml; // [2 kNumSMs][16]
  DevError* err;
};

template <bool kFp8>
struct CaShape {
  // 16-bit K / V tiles.  (E4M3: with 3 of them and 4 copied ones, the places of widened tiles came free too late: 0.63 ms
  // instead of 0.60 for 2548 tokens in chunks over 4k to 12k keys.)
  static constexpr int kTiles = kFp8 ? 4 : 5;
  static constexpr int kRaw = kFp8 ? 2 : 1;    // E4M3 tiles as copied
  static constexpr int kWiden = kFp8 ? 4 : 0;  // widening warps
  static constexpr int kThreads = 32 * (kCaWidenWarp + kWiden);
  // registers per thread of the roles, out of the launch's 168 (384 threads) or 128 (512 threads) a thread:
  // 256 * 216 + 128 * 72 = 384 * 168, and 256 * 208 + 128 * 56 + 128 * 40 = 512 * 128.  (With 184 for the softmax, E4M3
  // chunks took 6% more.
  // Two widening warps in the issuing warps' group leave it 216: chunks 1% faster, but items of few tokens, bound by the
  // widening, made 17 mixed requests 126 us instead of 115.)
  static constexpr int kRegsSoftmax = kFp8 ? 208 : 216, kRegsIssue = kFp8 ? 56 : 72, kRegsWiden = 40;
  // fp16 weights are kept near the top of their range (at most 2^(kLift + kCaSlack) = 2^15), so that small ones
  // stay normal down to 2^-21 of the largest
  static constexpr float kLift = kFp8 ? 7.f : 0.f;
};

// A CTA's part [u0, u1) of all units.
struct CaShareOf {
  long long total, ctas, u0, u1;
};
// ---- the units of a request --------------------------------------------------------

// sum of floor(y / 8) over 0 <= y < x
__device__ __forceinline__ long long ca_eighths(long long x) {
  const long long q = x >> 3;
  return 4 * q * (q - 1) + q * (x & 7);
}
// A request's n new tokens at positions len - n .. len - 1, as ceil(n / 16) items per KV head; item i sees the
// blocks up to its last token's.
struct CaReq {
  int t0, n, len;
  bool apart;  // a last item of one token is not counted (it is shared out apart)
  int extra;   // units of an item besides its blocks
  __device__ __forceinline__ bool one() const { return n % kCaTok == 1; }  // the last item has one token
  __device__ __forceinline__ int items() const { return (n + kCaTok - 1) / kCaTok - (apart && one()); }
  __device__ __forceinline__ int blocks(int i) const {
    return (len - n + min(n, kCaTok * (i + 1)) - 1) / kBlock + 1;
  }
  __device__ __forceinline__ bool dual(int i) const { return n - kCaTok * i > kCaTok / 2; }  // both tiles
  // units of the items before item i (all of 16 tokens)
  __device__ __forceinline__ long long before(int i) const {
    const long long a = (static_cast<long long>(len) - n + kCaTok - 1) / kCaTok;
    return ca_eighths(a + i) - ca_eighths(a) + i + static_cast<long long>(extra) * i;
  }
  // units of item i
  __device__ __forceinline__ int units(int i) const { return extra + (dual(i) ? blocks(i) : (blocks(i) + 1) / 2); }
  __device__ __forceinline__ long long per_head() const {
    const int i = items() - 1;
    if (i < 0) return 0;
    return before(i) + units(i);
  }
  // units of the last item where that has one token and is shared out apart
  __device__ __forceinline__ int one_units() const { return one() ? ((len - 1) / kBlock + 2) / 2 : 0; }
};
__device__ __forceinline__ bool ca_good(const CaArgs& a, long long c0, long long c1, int len) {
  return c0 >= 0 && c0 <= c1 && c1 <= a.tokens && c1 - c0 <= len && (len + kBlock - 1LL) / kBlock <= a.max_blocks;
}
// Request r; one with bad lengths has no tokens.
__device__ __forceinline__ CaReq ca_req(const CaArgs& a, int r, bool apart, int extra = 0) {
  const int c0 = a.cu[r], c1 = a.cu[r + 1], len = a.seq_lens[r];
  return ca_good(a, c0, c1, len) ? CaReq{c0, c1 - c0, len, apart, extra} : CaReq{0, 0, 0, apart, extra};
}
// Zeros for the rows of a request with bad lengths (the whole warp).
__device__ __noinline__ void ca_refuse(const CaArgs& a, int r, int lane) {
  if (lane == 0) record_error(a.err, MSA_DEVERR_LENGTH, r);
  const long long c0 = max(0, a.cu[r]), c1 = min(a.tokens, static_cast<long long>(a.cu[r + 1]));
  uint4* out = reinterpret_cast<uint4*>(a.out);
  for (long long i = c0 * (kHeads * kDim / 8) + lane; i < c1 * (kHeads * kDim / 8); i += 32)
    out[i] = make_uint4(0u, 0u, 0u, 0u);
  if (a.lse)
    for (long long i = c0 * kHeads + lane; i < c1 * kHeads; i += 32) a.lse[i] = -INFINITY;
}

// This CTA's part of the requests with bad lengths (one warp).
__device__ __forceinline__ void ca_refuse_bad(const CaArgs& a, int lane) {
  for (long long r0 = blockIdx.x; r0 < a.batch; r0 += 32LL * gridDim.x) {
    const long long r = r0 + static_cast<long long>(lane) * gridDim.x;
    const bool bad = r < a.batch && !ca_good(a, a.cu[r], a.cu[r + 1], a.seq_lens[r]);
    for (unsigned m = __ballot_sync(0xffffffffu, bad); m; m &= m - 1)
      ca_refuse(a, static_cast<int>(r0 + static_cast<long long>(__ffs(m) - 1) * gridDim.x), lane);
  }
}

// The request (and the unit in it) where a share begins.
struct CaStart {
  long long unit;
  int r;
  CaReq q;
};

template <bool kFp8>
struct CaSmem {
  uint8_t q[2][kCaTile];
  uint8_t kv[CaShape<kFp8>::kTiles][kCaTile];
  uint8_t raw[CaShape<kFp8>::kRaw][kFp8 ? kCaHalf : 16];
  float2 ml[2][128];  // before the roles begin: the warps' sums
  uint64_t q_full[2], q_ready[2], q_empty[2];  // q_ready: as fp16 (E4M3 cache)
  uint64_t kv_full[CaShape<kFp8>::kTiles], kv_empty[CaShape<kFp8>::kTiles];
  uint64_t raw_full[CaShape<kFp8>::kRaw], raw_empty[CaShape<kFp8>::kRaw];
  uint64_t s_full[2], p_full[2], o_full[2], x_full, x_done, done;
  uint64_t info_full[kCaInfo], info_empty[kCaInfo];
  // one-token items: K and V bytes of a block per place (over kv and raw), descriptors, the warps' meeting
  uint64_t one_full[kCaOnePlaces], one_empty[kCaOnePlaces], one_info_full[kCaInfo], one_info_empty[kCaInfo];
  uint64_t one_x_full, one_x_done;
  CaItem info[kCaInfo];
  int bad[kCaBad];
  CaStart start[2];  // of the items, and of the one-token items
  CaShareOf share[2];
  int extra;   // units of an item besides its blocks
  bool apart;  // the one-token items are shared out apart, after the others
  uint32_t tmem_base;
};

// The whole CTA: sums up the requests' units and finds this CTA's share of each kind, and where it begins.  The units that an
// item counts besides its blocks depend on the total, so the items are summed up beside their blocks.  (The caller's barrier
// follows.)
template <bool kFp8, bool kOne>
__device__ __forceinline__ void ca_find_shares(const CaArgs& a, CaSmem<kFp8>& sm) {
  constexpr int kThreads = CaShape<kFp8>::kThreads, kWarps = kThreads / 32, kKinds = kOne ? 2 : 1, kN = kOne ? 3 : 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // all KV heads' units without the items' own, items (bf16: the one-token ones too), and units of one-token items: of this
  // thread's request, and of the warp's requests up to and with it (the warps' own sums in wsum)
  long long (*wsum)[kWarps] = reinterpret_cast<long long (*)[kWarps]>(&sm.ml[0][0]);
  static_assert(kN * kWarps * sizeof(long long) <= sizeof(sm.ml), "wsum lies over ml");
  CaReq q{};
  long long u[kN], incl[kN], base[kN] = {};
  auto pass = [&](int r0) {
    const int r = r0 + tid;
    q = r < a.batch ? ca_req(a, r, kOne) : CaReq{};
    u[0] = kKvHeads * q.per_head();
    u[1] = kKvHeads * static_cast<long long>(q.items() + (kOne && !kFp8 && q.one()));
    if constexpr (kOne) u[2] = kKvHeads * static_cast<long long>(q.one_units());
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      incl[n] = u[n];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl[n], d);
        if (lane >= d) incl[n] += y;
      }
      if (lane == 31) wsum[n][warp] = incl[n];
    }
    __syncthreads();
  };
  CaShareOf share[kKinds];
  int extra = 0;
  bool apart = kOne;
  // the units of either kind, out of the sums
  auto units = [&](const long long (&x)[kN], int k) {
    if (!kOne) return x[0] + extra * x[1];
    if (kFp8 || apart) return k ? x[kN - 1] : x[0] + extra * x[1];
    return k ? 0LL : x[0] + x[kN - 1] + extra * x[1];
  };
  auto split = [&](const long long (&total)[kN]) {
    apart = kOne && (kFp8 || total[0] == 0);  // (bf16: only where there are no others)
    extra = 0;
    extra = ca_item_units(units(total, 0));
#pragma unroll
    for (int k = 0; k < kKinds; ++k) {
      CaShareOf& s = share[k];
      s.total = units(total, k);
      // (a share is long enough to hold some block's beginning)
      s.ctas = min(static_cast<long long>(gridDim.x), max(s.total / (k ? 1 : 1 + extra), 1LL));
      s.u0 = min(s.total, s.total * blockIdx.x / s.ctas);
      s.u1 = min(s.total, s.total * (blockIdx.x + 1) / s.ctas);
    }
  };
  const bool once = a.batch <= kThreads;
  if (!once) {
    for (int r0 = 0; r0 < a.batch; r0 += kThreads) {
      pass(r0);
#pragma unroll
      for (int n = 0; n < kN; ++n)
        for (int w = 0; w < kWarps; ++w) base[n] += wsum[n][w];
      __syncthreads();
    }
    split(base);
#pragma unroll
    for (int n = 0; n < kN; ++n) base[n] = 0;
  }
  for (int r0 = 0; r0 < a.batch; r0 += kThreads) {
    pass(r0);
    const int warps = min(kWarps, (a.batch - r0 + 31) / 32);  // that hold requests
    long long before[kN];
#pragma unroll
    for (int n = 0; n < kN; ++n) before[n] = base[n] + incl[n] - u[n];
    for (int w = 0; w < warps; ++w) {
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        const long long x = wsum[n][w];
        if (w < warp) before[n] += x;
        base[n] += x;
      }
    }
    if (once) split(base);
#pragma unroll
    for (int k = 0; k < kKinds; ++k) {
      const CaShareOf& s = share[k];
      const long long from = units(before, k), n = units(u, k);
      if (s.u0 < s.u1 && from <= s.u0 && s.u0 < from + n) {
        q.extra = k ? 0 : extra;
        q.apart = apart;
        sm.start[k] = CaStart{s.u0 - from, r0 + tid, q};
      }
    }
    if (!once) __syncthreads();
  }
  if (tid == 0) {
#pragma unroll
    for (int k = 0; k < kKinds; ++k) sm.share[k] = share[k];
    sm.extra = extra;
    sm.apart = apart;
  }
}

// Instruction descriptors: fp32 accumulation, A and B bf16 (or fp16), M = N = 128; B (V) MN-major for O.
__host__ __device__ constexpr uint32_t ca_idesc(bool fp16) {
  return fp16 ? tc::idesc_bf16_f32(128, 128) & ~((1u << 7) | (1u << 10)) : tc::idesc_bf16_f32(128, 128);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 bytes of a row: where rows begin on 32 bytes (wide) in one store, a whole sector; `out` may begin on 16 bytes
// only, and then in two.
__device__ __forceinline__ void ca_store32(void* p, const uint32_t (&y)[8], bool wide) {
  if (!wide) {
    stg128(p, y[0], y[1], y[2], y[3]);
    stg128(static_cast<uint8_t*>(p) + 16, y[4], y[5], y[6], y[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(y[0]), "r"(y[1]), "r"(y[2]),
               "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
               : "memory");
}
__device__ __forceinline__ bool ca_wait(uint64_t* bar, uint32_t parity, DevError* err, int where) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, where));
}

// One thread of the (whole) warp, always the same: the products' operands are then known to be those of one thread, and
// go straight to the uniform registers that the instruction takes.
__device__ __forceinline__ bool ca_elect() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one != 0;
}
template <int kRegs>
__device__ __forceinline__ void ca_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void ca_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// ---- one-token items ----------------------------------------------------------------

// Two E4M3 values (the low and the high byte of the low half of x) as fp16, exactly.
__device__ __forceinline__ uint32_t ca_widen2(uint32_t x) {
  uint32_t y;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(y) : "r"(x));
  return y;
}

// Products of m16n8k16, the 16 query heads their rows, from the copied pages.  E4M3: warps 0 to 3 take the even blocks, 32
// keys each, warps 4 to 7 the odd ones.  S = Q K^T: a 16-bit ldmatrix of K gives a lane four consecutive bytes of one key,
// dims 16 s + 4 t .. + 3 of k-step s, so Q's fragments hold those dims in the same slots.  O += P V: a transposing ldmatrix
// gives a lane two dims of two keys, which make one value pair for each of two products, one for the even dims and one for the
// odd.  bf16: each warp takes 16 keys of every block, K and V in places of their own.  Bound by HBM: each page is copied in
// and read once.  (16 tokens over 128k keys, E4M3, 2.15 GB: 0.32 ms, 6.7 TB/s.)

// The copies (the producer warp).
template <bool kFp8>
__device__ __forceinline__ void ca_one_produce(const CUtensorMap& kmap, const CUtensorMap& vmap, const CaArgs& a,
                                               const CaShareOf& share, CaSmem<kFp8>& sm) {
  const int lane = threadIdx.x & 31;
  DevError* err = a.err;
  uint8_t* places = &sm.kv[0][0];
  static_assert(sizeof(sm.kv) + sizeof(sm.raw) >= kCaOnePlaces * kCaTile, "the places lie over kv and raw");
  {
    CaCut cut{0, 0, 0, 0};
    int nitem = 0, nplace = 0;  // descriptors and places filled
    bool ok = true;
    if (share.u0 < share.u1) {
      int r = sm.start[1].r;
      const long long start = sm.start[1].unit;
      CaReq q = sm.start[1].q;
      int per = q.one_units();
      int g = (start >= per) + (start >= 2LL * per) + (start >= 3LL * per);
      int u = static_cast<int>(start - static_cast<long long>(g) * per);  // the unit in the item
      long long at = share.u0;
      while (true) {
        const int blocks = (q.len - 1) / kBlock + 1, to = static_cast<int>(min(static_cast<long long>(per), u + share.u1 - at));
        const int b = 2 * u;
        CaItem it{q.t0 + q.n - 1, 1, g, q.len - 1, q.len, b, min(blocks, 2 * to) - b, 0};
        it.slot = u == 0 && to == per ? -1 : static_cast<int>(2 * blockIdx.x + (u == 0));
        if (u == 0 && to < per) cut = CaCut{it.t0, 1, g, static_cast<int>(((at + per) * share.ctas - 1) / share.total)};
        at += to - u;
        const int is = nitem % kCaInfo;
        if (!(ok = ca_wait(&sm.one_info_empty[is], ((nitem / kCaInfo) & 1) ^ 1, err, 840))) break;
        if (lane == 0) {
          sm.info[is] = it;
          mbar_arrive(&sm.one_info_full[is]);
        }
        ++nitem;
        const int32_t* row = a.page_table + static_cast<long long>(r) * a.max_blocks + b;
        int ids = 0, ids_next = lane < it.nb ? row[lane] : 0;
        for (int k = 0; k < it.nb && ok; ++k) {
          if ((k & 31) == 0) {
            ids = ids_next;
            ids_next = k + 32 + lane < it.nb ? row[k + 32 + lane] : 0;
          }
          int page = __shfl_sync(0xffffffffu, ids, k & 31);
          const bool bad = page < 0 || page >= a.num_pages;
          if (bad) {
            if (lane == 0) record_error(err, MSA_DEVERR_PAGE, static_cast<long long>(r) * a.max_blocks + b + k);
            page = 0;
          }
          // E4M3: K and V to one place; bf16: to one each
#pragma unroll
          for (int kv = 0; kv < (kFp8 ? 1 : 2); ++kv, ++nplace) {
            const int s = nplace % kCaOnePlaces;
            if (!(ok = ca_wait(&sm.one_empty[s], ((nplace / kCaOnePlaces) & 1) ^ 1, err, 841))) break;
            if (lane == 0) {
              sm.bad[s] = bad;
              uint8_t* st = places + s * kCaTile;
              mbar_expect_tx(&sm.one_full[s], kCaTile);
              tma_load_3d(st, kv ? &vmap : &kmap, 0, g, page * kBlock, &sm.one_full[s]);
              tma_load_3d(st + kCaHalf, kFp8 || kv ? &vmap : &kmap, kFp8 ? 0 : 64, g, page * kBlock, &sm.one_full[s]);
            }
          }
        }
        if (!ok || at >= share.u1) break;
        u = 0;
        if (++g == kKvHeads) {
          g = 0;
          do {
            q = ca_req(a, ++r, true);
            per = q.one_units();
          } while (per == 0);
        }
      }
    }
    if (lane == 0) (kFp8 ? a.cuts1 : a.cuts)[blockIdx.x] = cut;
    if (ok && ca_wait(&sm.one_info_empty[nitem % kCaInfo], ((nitem / kCaInfo) & 1) ^ 1, err, 842) && lane == 0) {
      sm.info[nitem % kCaInfo] = CaItem{0, 0, 0, 0, 0, 0, 0, 0};
      mbar_arrive(&sm.one_info_full[nitem % kCaInfo]);
    }
    __syncwarp();
    if (lane == 0)  // no copy may still be landing when the CTA exits
      for (int s = 0; s < kCaOnePlaces; ++s) {
        const int fills = (nplace - s + kCaOnePlaces - 1) / kCaOnePlaces;
        if (fills > 0) mbar_wait(&sm.one_full[s], (fills - 1) & 1, err, 843);
      }
  }
}

// The sums (warps 0 to 7).
template <bool kFp8>
__device__ __forceinline__ void ca_one_attend(const CaArgs& a, CaSmem<kFp8>& sm, int warp) {
  const int lane = threadIdx.x & 31;
  DevError* err = a.err;
  uint8_t* places = &sm.kv[0][0];
  {
    const int g8 = lane >> 2, t4 = lane & 3, mi = lane >> 3;
    float* sums = reinterpret_cast<float*>(&sm.q[0][0]);  // [8 warps][16 rows][128] at an item's end
    float2* ml = &sm.ml[0][0];                            // [8 warps][16 rows]
    int nplace = 0;
    uint32_t xcount = 0;
    for (int n = 0;; ++n) {
      const int is = n % kCaInfo;
      if (!ca_wait(&sm.one_info_full[is], (n / kCaInfo) & 1, err, 844)) break;
      const CaItem it = sm.info[is];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.one_info_empty[is]);
      if (it.nb == 0) break;
      // Q rows g8 and g8 + 8, the A operand.  bf16: k-step s holds dims 16 s + 2t, + 1, + 8, + 9.  E4M3 (as fp16): dims
      // 16 s + 4 t .. + 3 in the same slots, which is where a lane's four bytes of K go.
      uint32_t qa[8][4];
      {
        const __nv_bfloat16* q0 = a.q + (static_cast<long long>(it.t0) * kHeads + it.g * kGroup + g8) * kDim;
        const __nv_bfloat16* q1 = q0 + 8 * kDim;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          if constexpr (kFp8) {
            const uint2 x = reinterpret_cast<const uint2*>(q0 + 4 * t4)[4 * s], y = reinterpret_cast<const uint2*>(q1 + 4 * t4)[4 * s];
            qa[s][0] = pack_f16(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u));
            qa[s][1] = pack_f16(__uint_as_float(y.x << 16), __uint_as_float(y.x & 0xffff0000u));
            qa[s][2] = pack_f16(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
            qa[s][3] = pack_f16(__uint_as_float(y.y << 16), __uint_as_float(y.y & 0xffff0000u));
          } else {
            qa[s][0] = *reinterpret_cast<const uint32_t*>(q0 + 16 * s + 2 * t4);
            qa[s][1] = *reinterpret_cast<const uint32_t*>(q1 + 16 * s + 2 * t4);
            qa[s][2] = *reinterpret_cast<const uint32_t*>(q0 + 16 * s + 2 * t4 + 8);
            qa[s][3] = *reinterpret_cast<const uint32_t*>(q1 + 16 * s + 2 * t4 + 8);
          }
        }
      }
      constexpr float kLift = CaShape<kFp8>::kLift;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows g8, g8 + 8; l: this lane's part
      // rows g8 (0, 1) and g8 + 8 (2, 3).  bf16: [n]: dims 8 n + 2t, + 1.  E4M3: [2 c + e]: dims 16 c + 4t + e, + 2 + e.
      float o[16][4];
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      // The weights of a group of keys: x holds their scores, keys 8 i + 2t, + 1 of rows g8 (0, 1) and g8 + 8 (2, 3); the
      // first `keys` count.  Raises the reference where a maximum passes it by kCaSlack, adds to l, and leaves P as the A
      // operand of k-steps of 16 keys.
      auto weigh = [&](auto& x, auto& pa, int keys) {
        constexpr int kTiles = sizeof(x) / sizeof(x[0]);
        if (keys < 8 * kTiles)
#pragma unroll
          for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (8 * i + 2 * t4 + (e & 1) >= keys) x[i][e] = -INFINITY;
        float mx[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v = -INFINITY;
#pragma unroll
          for (int i = 0; i < kTiles; ++i) v = fmax3(v, x[i][2 * h], x[i][2 * h + 1]);
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          mx[h] = v * a.scale_log2 - kLift;
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] + kCaSlack || mx[1] > m[1] + kCaSlack)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool raise = mx[h] > m[h] + kCaSlack;
            const float f = raise && m[h] != -INFINITY ? ex2(m[h] - mx[h]) : 1.f;
            if (raise) m[h] = mx[h];
            l[h] *= f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              o[i][2 * h] *= f;
              o[i][2 * h + 1] *= f;
            }
          }
          __syncwarp();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mu = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            const float p0 = ex2(fmaf(x[i][2 * h], a.scale_log2, -mu)), p1 = ex2(fmaf(x[i][2 * h + 1], a.scale_log2, -mu));
            pa[i >> 1][2 * (i & 1) + h] = kFp8 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
            l[h] += p0 + p1;
          }
        }
      };
      // keys behind the last have no weight, but their values may be anything: they are taken as zero (a register of a
      // transposed V holds keys 2t and 2t + 1, of the first or the second eight)
      auto cut_v = [&](uint32_t (&vr)[4], int keys) {
        const uint32_t lo = (2 * t4 < keys ? 0xffffu : 0u) | (2 * t4 + 1 < keys ? 0xffff0000u : 0u);
        const uint32_t hi = (2 * t4 + 8 < keys ? 0xffffu : 0u) | (2 * t4 + 9 < keys ? 0xffff0000u : 0u);
        vr[0] &= lo;
        vr[1] &= hi;
        vr[2] &= lo;
        vr[3] &= hi;
      };
      auto release = [&](int s) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.one_empty[s]);
      };
      bool ok = true;
      for (int k = 0; k < it.nb; ++k) {
        const int s = nplace % kCaOnePlaces;
        if (!(ok = ca_wait(&sm.one_full[s], (nplace / kCaOnePlaces) & 1, err, 845))) break;
        const int block_keys = sm.bad[s] ? 0 : min(kBlock, it.len - (it.b0 + k) * kBlock);
        const uint32_t kt = smem_u32(places + s * kCaTile);
        if constexpr (kFp8) {
          ++nplace;
          const int keys = block_keys - 32 * (warp & 3);  // of this warp's 32
          if ((nplace & 1) == (warp >> 2) && keys > 0) {
            const uint32_t vt = kt + kCaHalf;
            const int mrow = 32 * (warp & 3) + 8 * (mi & 1) + (lane & 7);  // this lane's row address for ldmatrix
            float x[4][4] = {};
#pragma unroll
            for (int c = 0; c < 8; c += 2)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint32_t kr[4];  // keys 16 u .. + 7 and .. + 15 of k-step c, then of k-step c + 1
                ldsm_x4(kr, kt + sw128(mrow + 16 * u, c + (mi >> 1)));
                mma_f16(x[2 * u], qa[c], ca_widen2(kr[0]), ca_widen2(kr[0] >> 16));
                mma_f16(x[2 * u + 1], qa[c], ca_widen2(kr[1]), ca_widen2(kr[1] >> 16));
                mma_f16(x[2 * u], qa[c + 1], ca_widen2(kr[2]), ca_widen2(kr[2] >> 16));
                mma_f16(x[2 * u + 1], qa[c + 1], ca_widen2(kr[3]), ca_widen2(kr[3] >> 16));
              }
            uint32_t pa[2][4];
            weigh(x, pa, keys);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t vr[4];  // keys 16 u .. + 7 and .. + 15 of dims 32 j .., then of dims 32 j + 16 ..
                ldsm_x4_t(vr, vt + sw128(mrow + 16 * u, 2 * j + (mi >> 1)));
                if (keys < 16 * (u + 1)) cut_v(vr, keys - 16 * u);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  // bytes of a register: key 2t dims 2n and 2n + 1, key 2t + 1 dims 2n and 2n + 1
                  const uint32_t b0 = __byte_perm(vr[2 * c], 0, 0x3120), b1 = __byte_perm(vr[2 * c + 1], 0, 0x3120);
                  mma_f16(o[4 * j + 2 * c], pa[u], ca_widen2(b0), ca_widen2(b1));
                  mma_f16(o[4 * j + 2 * c + 1], pa[u], ca_widen2(b0 >> 16), ca_widen2(b1 >> 16));
                }
              }
          }
          release(s);
        } else {
          const int keys = block_keys - 16 * warp;  // of this warp's 16
          const int mrow = 16 * warp + 8 * (mi >> 1) + (lane & 7), vrow = 16 * warp + 8 * (mi & 1) + (lane & 7);
          uint32_t pa[1][4];
          if (keys > 0) {
            float x[4][4] = {};  // two chains of products per eight keys, added up below
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint32_t kr[4];  // keys 0-7, both halves of k-step c, then keys 8-15
              ldsm_x4(kr, kt + (c >> 2) * kCaHalf + sw128(mrow, 2 * (c & 3) + (mi & 1)));
              mma_bf16(x[2 * (c & 1)], qa[c], kr[0], kr[1]);
              mma_bf16(x[2 * (c & 1) + 1], qa[c], kr[2], kr[3]);
            }
            float y[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) y[i][e] = x[i][e] + x[i + 2][e];
            release(s);
            weigh(y, pa, keys);
          } else {
            release(s);
          }
          ++nplace;
          const int sv = nplace % kCaOnePlaces;
          if (!(ok = ca_wait(&sm.one_full[sv], (nplace / kCaOnePlaces) & 1, err, 848))) break;
          ++nplace;
          if (keys > 0) {
            const uint32_t vt = smem_u32(places + sv * kCaTile);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t vr[4];  // keys 0-7 and 8-15 of dims 16 j .. + 7, then of dims 16 j + 8 ..
              ldsm_x4_t(vr, vt + (j >> 2) * kCaHalf + sw128(vrow, 2 * (j & 3) + (mi >> 1)));
              if (keys < 16) cut_v(vr, keys);
              mma_bf16(o[2 * j], pa[0], vr[0], vr[1]);
              mma_bf16(o[2 * j + 1], pa[0], vr[2], vr[3]);
            }
          }
          release(sv);
        }
      }
      if (!ok) break;
      // ---- the end of the item: the warps' sums meet in shared memory; each warp joins and writes two rows ----
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        const int row = g8 + 8 * h;
        if (t4 == 0) ml[warp * 16 + row] = make_float2(m[h], l[h]);
        // (the row's 64-byte pieces permuted: eight rows, eight banks)
        float* to = sums + (warp * 16 + row) * kDim;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if constexpr (kFp8) {
            *reinterpret_cast<float4*>(to + 16 * (c ^ g8) + 4 * t4) =
                make_float4(o[2 * c][2 * h], o[2 * c + 1][2 * h], o[2 * c][2 * h + 1], o[2 * c + 1][2 * h + 1]);
          } else {
            *reinterpret_cast<float2*>(to + 16 * (c ^ g8) + 2 * t4) = make_float2(o[2 * c][2 * h], o[2 * c][2 * h + 1]);
            *reinterpret_cast<float2*>(to + 16 * (c ^ g8) + 8 + 2 * t4) =
                make_float2(o[2 * c + 1][2 * h], o[2 * c + 1][2 * h + 1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.one_x_full);
      if (!ca_wait(&sm.one_x_full, xcount & 1, err, 846)) break;
#pragma unroll 1
      for (int row = 2 * warp; row < 2 * warp + 2; ++row) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) top = fmaxf(top, ml[w * 16 + row].x);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float2 c = ml[w * 16 + row];
          const float f = c.x == -INFINITY ? 0.f : ex2(c.x - top);
          sum = fmaf(f, c.y, sum);
          const float4 x = *reinterpret_cast<const float4*>(sums + (w * 16 + row) * kDim +
                                                            16 * ((lane >> 2) ^ (row & 7)) + 4 * (lane & 3));
          v.x = fmaf(f, x.x, v.x);
          v.y = fmaf(f, x.y, v.y);
          v.z = fmaf(f, x.z, v.z);
          v.w = fmaf(f, x.w, v.w);
        }
        if (it.slot >= 0) {
          const long long rows = kFp8 ? kGroup : a.rows;
          (kFp8 ? a.part1_o : a.part_o)[(static_cast<long long>(it.slot) * (kDim / 4) + lane) * rows + row] = v;
          if (lane == 0) (kFp8 ? a.part1_ml : a.part_ml)[it.slot * rows + row] = make_float2(top, sum);
        } else {
          const long long orow = static_cast<long long>(it.t0) * kHeads + it.g * kGroup + row;
          const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
          reinterpret_cast<uint2*>(a.out + orow * kDim)[lane] =
              make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
          if (a.lse && lane == 0) a.lse[orow] = sum == 0.f ? -INFINITY : top + log2f(sum);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.one_x_done);
      if (!ca_wait(&sm.one_x_done, xcount & 1, err, 847)) break;
      ++xcount;
    }
  }
}

// kOne: one-token items may be computed apart (over an E4M3 cache always)
template <bool kFp8, bool kOne>
__global__ void __launch_bounds__(CaShape<kFp8>::kThreads, 1) chunk_attend_kernel(
    const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
    const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CaArgs a) {
  using Shape = CaShape<kFp8>;
  constexpr int kTiles = Shape::kTiles, kThreads = Shape::kThreads;
  constexpr int kRing = kFp8 ? Shape::kRaw : kTiles;  // places that tiles are copied into
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  CaSmem<kFp8>& sm = *reinterpret_cast<CaSmem<kFp8>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  DevError* err = a.err;

  if (smem_u32(smem_raw) & 1023) {  // the swizzled tiles need it; with no static shared memory it holds
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
      record_error(err, MSA_DEVERR_TIMEOUT, 899);
      a.cuts[blockIdx.x] = a.cuts1[blockIdx.x] = CaCut{0, 0, 0, 0};
    }
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_ready[i], 4);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.o_full[i], 1);
    }
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&sm.kv_full[i], kFp8 ? 4 : 1);
      mbar_init(&sm.kv_empty[i], 1);
    }
    for (int i = 0; i < Shape::kRaw; ++i) {
      mbar_init(&sm.raw_full[i], 1);
      mbar_init(&sm.raw_empty[i], 4);
    }
    mbar_init(&sm.x_full, 8);
    mbar_init(&sm.x_done, 8);
    mbar_init(&sm.done, 1);
    for (int i = 0; i < kCaInfo; ++i) {
      mbar_init(&sm.info_full[i], 1);
      mbar_init(&sm.info_empty[i], 9 + Shape::kWiden);  // the softmax, MMA and widening warps
    }
    for (int i = 0; i < kCaOnePlaces; ++i) {
      mbar_init(&sm.one_full[i], 1);
      mbar_init(&sm.one_empty[i], 8);
    }
    for (int i = 0; i < kCaInfo; ++i) {
      mbar_init(&sm.one_info_full[i], 1);
      mbar_init(&sm.one_info_empty[i], 8);
    }
    mbar_init(&sm.one_x_full, 8);
    mbar_init(&sm.one_x_done, 8);
    fence_mbar_init();
  }
  if (warp == kCaMmaWarp) {
    tc::alloc(&sm.tmem_base, 512);
    tc::relinquish();
  }
  if (tid == 32 * kCaProducerWarp) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  // the kernel before has completed; the joining kernel may be launched behind this one
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  ca_find_shares<kFp8, kOne>(a, sm);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem_base, 0);

  // (where all items are one-token items computed apart, the tiles' roles have nothing to do: 0.2 us less)
  const bool tiles = !kOne || sm.share[0].total > 0;
  // All roles of all warps are done: tensor memory may be released, and the tiles' places copied into again.
  auto roles_done = [&] {
    if (!tiles) return;
    tc::fence_before();
    if (kFp8) fence_proxy_async_smem();  // (bf16: either there are other items, or one-token items)
    __syncwarp();
    asm volatile("barrier.sync 1, %0;" ::"n"(kThreads) : "memory");
  };
  // A wait that gives up (recorded in the error word) ends its role, so a broken pipeline ends after one bounded wait
  // per role.
  if (warp >= 8 && warp < kCaWidenWarp) ca_regs_down<Shape::kRegsIssue>();
  if (warp == kCaProducerWarp) {
    // ---------------- the share's items, and their copies ----------------
    const long long total = sm.share[0].total, ctas = sm.share[0].ctas, u0 = sm.share[0].u0, u1 = sm.share[0].u1;
    CaCut cut{0, 0, 0, 0};
    int nitem = 0, nq = 0, nload = 0, nblk = 0;  // descriptors, Q tiles, K / V tiles and blocks issued
    bool ok = true;
    if (u0 < u1) {
      const int extra = sm.extra;
      int r = sm.start[0].r;
      CaReq rq = sm.start[0].q;
      long long per = rq.per_head();
      int g = (sm.start[0].unit >= per) + (sm.start[0].unit >= 2 * per) + (sm.start[0].unit >= 3 * per);
      const long long rem = sm.start[0].unit - g * per;
      int i = 0;  // the last item that begins at or before unit rem of the head
      for (int lo = 0, hi = rq.items() - 1; lo <= hi;) {
        const int mid = (lo + hi) >> 1;
        if (rq.before(mid) <= rem) {
          i = mid;
          lo = mid + 1;
        } else {
          hi = mid - 1;
        }
      }
      long long at = u0, item0 = u0 - (rem - rq.before(i));  // where the share goes on, where the item begins
      while (ok) {
        const int blocks = rq.blocks(i);
        const bool dual = rq.dual(i);
        const long long end = item0 + rq.units(i);
        // blocks that begin before unit x of the item: the first at 0, the others after the item's own units
        auto begun = [&](long long x) {
          const int units = x <= 0 ? 0 : 1 + static_cast<int>(max(0LL, x - 1 - rq.extra));
          return min(blocks, dual ? units : 2 * units);
        };
        CaItem it;
        it.t0 = rq.t0 + kCaTok * i;
        it.ntok = min(kCaTok, rq.n - kCaTok * i);
        it.g = g;
        it.pos0 = rq.len - rq.n + kCaTok * i;
        it.len = rq.len;
        it.b0 = begun(at - item0);
        it.nb = begun(min(end, u1) - item0) - it.b0;
        const int b = it.b0;
        const bool to_end = b + it.nb == blocks;
        it.slot = b == 0 && to_end ? -1 : static_cast<int>(2 * blockIdx.x + (b == 0));
        at = end;
        item0 = end;
        if (it.nb > 0) {
        // publish
        const int is = nitem % kCaInfo;
        if (!(ok = ca_wait(&sm.info_empty[is], ((nitem / kCaInfo) & 1) ^ 1, err, 800))) break;
        if (lane == 0) {
          sm.info[is] = it;
          mbar_arrive(&sm.info_full[is]);
        }
        ++nitem;
        const int tiles = it.ntok > 8 ? 2 : 1;
        const int32_t* row = a.page_table + static_cast<long long>(r) * a.max_blocks;
        int ids = 0, ids_next = lane < it.nb ? row[b + lane] : 0;  // 32 page ids, and the next 32
        int last = 0, before = 0;  // pages of the last block that K was loaded of, and of the one before
        for (int j = 0; j < 2 * it.nb && ok; ++j) {  // tile j: K of block (j + 1) / 2 and V in turn
          const bool is_v = ca_is_v(j, it.nb);
          int page;
          if (!is_v) {
            const int k = (j + 1) >> 1;
            if ((k & 31) == 0) {
              ids = ids_next;
              ids_next = k + 32 + lane < it.nb ? row[b + k + 32 + lane] : 0;
            }
            page = __shfl_sync(0xffffffffu, ids, k & 31);
            const bool bad = page < 0 || page >= a.num_pages;
            if (bad) {
              if (lane == 0) record_error(err, MSA_DEVERR_PAGE, static_cast<long long>(r) * a.max_blocks + b + k);
              page = 0;
            }
            if (lane == 0) sm.bad[nblk % kCaBad] = bad;
            ++nblk;
          }
          // V of the block before the last K (the last tile: V of the last block itself)
          const int from = is_v && j < 2 * it.nb - 1 ? before : is_v ? last : page;
          if (!is_v) {
            before = last;
            last = page;
          }
          const CUtensorMap* map = is_v ? &vmap : &kmap;
          const int s = nload % kRing, turn = nload / kRing;
          if (!(ok = ca_wait(kFp8 ? &sm.raw_empty[s] : &sm.kv_empty[s], (turn & 1) ^ 1, err, 801))) break;
          if (lane == 0) {
            if (kFp8) {
              mbar_expect_tx(&sm.raw_full[s], kCaHalf);
              tma_load_3d(sm.raw[kFp8 ? s : 0], map, 0, g, from * kBlock, &sm.raw_full[s]);
            } else {
              mbar_expect_tx(&sm.kv_full[s], kCaTile);
              tma_load_3d(sm.kv[s], map, 0, g, from * kBlock, &sm.kv_full[s]);
              tma_load_3d(sm.kv[s] + kCaHalf, map, 64, g, from * kBlock, &sm.kv_full[s]);
            }
          }
          ++nload;
          // The item's Q follows its first K tile: that tile's place was freed by the items before, but Q's may have to
          // wait for their last S products.
          if (j == 0) {
            for (int q = 0; q < tiles; ++q) {
              const int qs = nq & 1, n = min(8, it.ntok - 8 * q);
              if (!(ok = ca_wait(&sm.q_empty[qs], ((nq >> 1) & 1) ^ 1, err, 803))) break;
              if (lane == 0) mbar_expect_tx(&sm.q_full[qs], n * kCaQEntry);
              __syncwarp();
              if (lane < n)
                tma_load_5d(sm.q[qs] + lane * kCaQEntry, &qmap, 0, 0, 0, 2 * g, it.t0 + 8 * q + lane, &sm.q_full[qs]);
              ++nq;
            }
          }
        }
        }
        // (here, not before the copies: a division) the share that holds the item's last unit
        if (b == 0 && !to_end) cut = CaCut{it.t0, it.ntok, g, static_cast<int>((end * ctas - 1) / total)};
        if (!ok || at >= u1) break;
        // the next item (the share goes on, so there is one)
        if (++i == rq.items()) {
          i = 0;
          if (++g == kKvHeads) {
            g = 0;
            do {
              rq = ca_req(a, ++r, kOne && sm.apart, extra);
            } while (rq.items() == 0);
          }
        }
      }
    }
    if (lane == 0) a.cuts[blockIdx.x] = cut;
    if (tiles && ok && ca_wait(&sm.info_empty[nitem % kCaInfo], ((nitem / kCaInfo) & 1) ^ 1, err, 804) && lane == 0) {
      sm.info[nitem % kCaInfo] = CaItem{0, 0, 0, 0, 0, 0, 0, 0};
      mbar_arrive(&sm.info_full[nitem % kCaInfo]);
    }
    // no copy may still be landing when the CTA exits: wait for the last fill of every place
    __syncwarp();
    if (lane == 0) {
      for (int s = 0; s < kRing; ++s) {
        const int ring = kRing, fills = (nload - s + ring - 1) / ring;
        if (fills > 0) mbar_wait(kFp8 ? &sm.raw_full[s] : &sm.kv_full[s], (fills - 1) & 1, err, 805);
      }
      for (int s = 0; s < 2; ++s) {
        const int fills = (nq - s + 1) / 2;
        if (fills > 0) mbar_wait(&sm.q_full[s], (fills - 1) & 1, err, 806);
      }
    }
    __syncwarp();
    roles_done();
    if constexpr (kOne)
      if (sm.apart) ca_one_produce<kFp8>(kmap, vmap, a, sm.share[1], sm);
  } else if (warp == kCaMmaWarp) {
    // ---------------- S and O products ----------------
    // One thread issues them all, and they execute in the order in which they are issued: an S product that overwrites P
    // follows the O product that reads it, and the two warpgroups' products alternate, so that one's softmax runs beside
    // the other's products.  (With a thread for each warpgroup's they fell into step, both softmaxes and then both
    // products at once: 1.59 ms instead of 1.34 ms for 2048 tokens over 32k keys.)  The thread holds few products
    // ahead of the tensor cores, so it looks for what the next ones need before it issues a group, not between groups.
    constexpr uint32_t idesc_s = ca_idesc(kFp8), idesc_o = ca_idesc(kFp8) | (1u << 16);
    const bool leader = ca_elect();
    int base = 0, nq = 0;         // blocks and Q tiles of the items before
    uint32_t pcount[2] = {0, 0};  // P tiles taken
    bool ok = tiles;
    for (int n = 0; ok; ++n) {
      const int is = n % kCaInfo;
      if (!(ok = ca_wait(&sm.info_full[is], (n / kCaInfo) & 1, err, 810))) break;
      const int nb = sm.info[is].nb, b0 = sm.info[is].b0, len = sm.info[is].len;
      const bool dual = sm.info[is].ntok > 8;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.info_empty[is]);
      if (nb == 0) break;
      bool more[2] = {false, false};  // O holds sums of this item
      // keys of a block that count for the last token: all, but in the request's last block and in a bad page
      auto keys_of = [&](int blk) {
        return sm.bad[(base + blk) % kCaBad] ? 0 : min(kBlock, len - (b0 + blk) * kBlock);
      };
      // O += P V of block `bo` (-1: none), then S of block `bs` (-1: none), for warpgroup w; one thread.  The tiles of
      // a block that both warpgroups read are waited for by the first and given back by the second.
      auto issue = [&](auto w_tag, int bo, int bs) {
        constexpr int w = decltype(w_tag)::value;
        const uint32_t s_col = tmem + 128 * w, o_col = tmem + kCaOCol + 128 * w;
        const bool first = !dual || w == 0, last = !dual || w == 1;
        const int lk = 2 * base + ca_load_k(max(bs, 0)), sk = lk % kTiles;
        bool k_here = bs < 0 || !first;
        if (!k_here) k_here = mbar_try_wait(&sm.kv_full[sk], (lk / kTiles) & 1);
        if (bo >= 0) {
          const int lv = 2 * base + ca_load_v(bo, nb), sv = lv % kTiles;
          if (first && !mbar_wait(&sm.kv_full[sv], (lv / kTiles) & 1, err, 813)) return false;
          const int ks = (keys_of(bo) + 15) / 16;  // the 16-key steps behind the last key are left out
          const uint64_t vd = tc::desc_v_mn_sw128(smem_u32(sm.kv[sv]));
          if (!mbar_wait(&sm.p_full[w], pcount[w] & 1, err, 814)) return false;
          ++pcount[w];
          tc::fence_after();
          if (ks == 8) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // (descriptor addresses count 16 bytes)
              tc::mma_bf16_ts(o_col, s_col + kk * 8, vd + kk * (2048 / 16), idesc_o, more[w] || kk > 0);
          } else {
            for (int kk = 0; kk < ks; ++kk)
              tc::mma_bf16_ts(o_col, s_col + kk * 8, vd + kk * (2048 / 16), idesc_o, more[w] || kk > 0);
          }
          more[w] = more[w] || ks > 0;
          if (last) tc::commit(&sm.kv_empty[sv]);
          if (bs < 0) tc::commit(&sm.o_full[w]);  // the item's last of this warpgroup
        }
        if (bs >= 0) {
          const int qs = (dual ? nq + w : nq) & 1;
          const uint64_t qd = tc::desc_k_sw128_sbo(smem_u32(sm.q[qs]), 2048),
                         kd = tc::desc_k_sw128(smem_u32(sm.kv[sk]));
          if (!k_here) {
            if (!mbar_wait(&sm.kv_full[sk], (lk / kTiles) & 1, err, 812)) return false;
            tc::fence_after();
          }
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::mma_bf16(s_col, qd + (kk >> 2) * (1024 / 16) + (kk & 3) * 2,
                         kd + (kk >> 2) * (kCaHalf / 16) + (kk & 3) * 2, idesc_s, kk > 0);
          tc::commit(&sm.s_full[w]);
          if (last) tc::commit(&sm.kv_empty[sk]);
          if (bs == nb - 1) tc::commit(&sm.q_empty[qs]);
        }
        return true;
      };
      const std::integral_constant<int, 0> w0;
      const std::integral_constant<int, 1> w1;
      if (leader) {
        // everything but the O products of the last block
        for (int q = 0; q < (dual ? 2 : 1) && ok; ++q) {
          const int t = nq + q;
          ok = mbar_wait(kFp8 ? &sm.q_ready[t & 1] : &sm.q_full[t & 1], (t >> 1) & 1, err, 811);
        }
        tc::fence_after();
        if (dual) {
          ok = ok && issue(w0, -1, 0) && issue(w1, -1, 0);
          for (int b = 0; b < nb - 1 && ok; ++b) ok = issue(w0, b, b + 1) && issue(w1, b, b + 1);
        } else {
          ok = ok && issue(w0, -1, 0) && (nb == 1 || issue(w1, -1, 1));
          for (int b = 0; b < nb - 1 && ok; b += 2) {
            ok = issue(w0, b, b + 2 < nb ? b + 2 : -1);
            if (ok && b + 1 < nb - 1) ok = issue(w1, b + 1, b + 3 < nb ? b + 3 : -1);
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      const int lv = 2 * base + 2 * nb - 1, sv = lv % kTiles;
      ok = ok && ca_wait(&sm.kv_full[sv], (lv / kTiles) & 1, err, 816);
      const int keys = keys_of(nb - 1);  // (the block's flag, written before its copies were asked for: behind the wait)
      if (!kFp8 && ok && (keys & 15)) {
        // V rows behind the last key, up to the end of their 16-row step: their weight is zero, but they may hold
        // anything, so they become zero too (the whole warp)
        const uint32_t va = smem_u32(sm.kv[sv]);
        for (int j = lane; j < (16 - (keys & 15)) * 16; j += 32) {
          const int vr = keys + (j >> 4);
          sts128(va + ((j >> 3) & 1) * kCaHalf + vr * 128 + (j & 7) * 16, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (leader && ok) {
        if (dual) ok = issue(w0, nb - 1, -1) && issue(w1, nb - 1, -1);
        else ok = (nb & 1) ? issue(w0, nb - 1, -1) : issue(w1, nb - 1, -1);
      }
      ok = __all_sync(0xffffffffu, ok);
      base += nb;
      nq += dual ? 2 : 1;
    }
    // every product has finished before tensor memory is released
    if (leader && tiles) {
      tc::commit(&sm.done);
      mbar_wait(&sm.done, 0, err, 815);
    }
    __syncwarp();
  } else if (warp == kCaMmaWarp + 1) {
    // ---------------- requests with bad lengths ----------------
    ca_refuse_bad(a, lane);
  } else if (warp < 8) {
    // ---------------- softmax, one row per thread; the end of an item ----------------
    ca_regs_up<Shape::kRegsSoftmax>();
    const int wg = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t scol = lanes + 128 * wg, ocol = lanes + kCaOCol + 128 * wg;
    int base = 0;
    uint32_t scount = 0, ocount = 0, xcount = 0;
    bool ok = tiles;
    for (int n = 0; ok; ++n) {
      const int is = n % kCaInfo;
      if (!(ok = ca_wait(&sm.info_full[is], (n / kCaInfo) & 1, err, 820))) break;
      const CaItem it = sm.info[is];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.info_empty[is]);
      if (it.nb == 0) break;
      const bool dual = it.ntok > 8;
      const int steps = dual ? it.nb : (it.nb + 1 - wg) / 2;
      const int tok = (dual ? 8 * wg : 0) + (row >> 4);
      const bool valid = tok < it.ntok;
      const bool active = __any_sync(0xffffffffu, valid);  // a warp without a row only keeps the barriers
      float m = -INFINITY, l = 0.f;  // reference (lowered by kLift), sum of the weights
      for (int s = 0; s < steps; ++s) {
        const int blk = dual ? s : 2 * s + wg;
        if (!(ok = ca_wait(&sm.s_full[wg], scount & 1, err, 821))) break;
        ++scount;
        tc::fence_after();
        if (active) {
          const int keys = !valid ? kBlock
                                  : sm.bad[(base + blk) % kCaBad]
                                        ? 0
                                        : min(kBlock, it.pos0 + tok + 1 - (it.b0 + blk) * kBlock);
          const bool masked = !__all_sync(0xffffffffu, keys >= kBlock);
          auto block = [&](auto mask_tag) {
            constexpr bool kMask = decltype(mask_tag)::value;
            // raises the reference to mx where it passes it by kCaSlack (so for the row's first key: m is -inf), with the
            // sums so far; before an item's first O product there is nothing in O
            auto raise_to = [&](float mx) {
              const bool raise = mx > m + kCaSlack;
              if (!__any_sync(0xffffffffu, raise)) return false;
              const float f = raise && m != -INFINITY ? ex2(m - mx) : 1.f;  // (no key yet: the sums are zero)
              if (raise) m = mx;
              l *= f;
              __syncwarp();  // (what follows wants the warp together)
              if (s > 0) {
#pragma unroll 1
                for (int ch = 0; ch < 8; ++ch) {
                  uint32_t o[16];
                  tc::ld_32x32b_x16(ocol + ch * 16, o);
                  tc::wait_ld();
#pragma unroll
                  for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
                  tc::st_32x32b_x16(ocol + ch * 16, o);
                }
              }
              return true;
            };
            uint32_t x[4][32] = {};  // the row of S, in four chunks of 32 columns
            auto score = [&](int ch, int i) {
              const float v = __uint_as_float(x[ch][i]);
              return kMask && ch * 32 + i >= keys ? -INFINITY : v;
            };
            auto load = [&](int ch) { tc::ld_32x32b_x32(scol + ch * 32, x[ch]); };
            auto top_of = [&](int ch, float (&top)[4]) {
#pragma unroll
              for (int q = 0; q < 16; ++q) top[q & 3] = fmax3(top[q & 3], score(ch, 2 * q), score(ch, 2 * q + 1));
            };
            auto scaled = [&](const float (&top)[4]) {
              return fmaxf(fmax3(top[0], top[1], top[2]), top[3]) * a.scale_log2 - Shape::kLift;
            };
            // P of the row against m, and the weights' sum; returns the row's maximum.  P's chunk goes over S columns that
            // are in registers by then.
            float sum;
            auto weights = [&](auto load_tag) {
              constexpr bool kLoad = decltype(load_tag)::value;
              const float mu = m == -INFINITY ? 0.f : m;
              float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
              float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
              if (kLoad) load(0);
#pragma unroll
              for (int ch = 0; ch < 4; ++ch) {
                if (kLoad) tc::wait_ld();
                if (kLoad && ch < 3) load(ch + 1);
                uint32_t pk[16];
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                  const float xa = score(ch, 2 * q), xb = score(ch, 2 * q + 1);
                  if (kLoad) top[q & 3] = fmax3(top[q & 3], xa, xb);
                  const float2 y = fma2(xa, xb, a.scale_log2, a.scale_log2, -mu, -mu);
                  const float pa = ex2(y.x), pb = ex2(y.y);
                  pk[q] = kFp8 ? pack_f16(pa, pb) : pack_bf16(pa, pb);
                  add[q & 1] = add2(add[q & 1].x, add[q & 1].y, pa, pb);
                }
                tc::st_32x32b_x16(scol + ch * 16, pk);
              }
              sum = (add[0].x + add[0].y) + (add[1].x + add[1].y);
              return scaled(top);
            };
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (s == 0) {
              // the item's first block: its maximum is the reference
              load(0);
#pragma unroll
              for (int ch = 0; ch < 4; ++ch) {
                tc::wait_ld();
                if (ch < 3) load(ch + 1);
                top_of(ch, top);
              }
              m = scaled(top);
              weights(std::false_type{});
            } else if (raise_to(weights(std::true_type{}))) {
              // the weights against the reference so far, and again only where the block's maximum turned out to raise it
              weights(std::false_type{});
            }
            l += sum;
          };
          if (!masked) block(std::false_type{});
          else block(std::true_type{});
          tc::wait_st();
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[wg]);
      }
      if (!ok) break;
      base += it.nb;

      // ---- the end of the item: its rows, or its partial ----
      if (steps > 0 && !(ok = ca_wait(&sm.o_full[wg], ocount & 1, err, 822))) break;
      ocount += steps > 0;
      const int h = it.g * kGroup + (row & 15);
      const long long orow = (static_cast<long long>(it.t0) + tok) * kHeads + h;
      const long long prow = tok * kGroup + (row & 15);
      // f0, f1: what the two warpgroups' sums are multiplied by; l: the row's denominator; dims d0 ..
      float f0 = m == -INFINITY ? 0.f : 1.f, f1 = 0.f;
      uint32_t c0 = ocol, c1 = ocol;
      int d0 = 0, nd = kDim;
      const bool shared = !dual && it.nb > 1;  // both warpgroups hold sums of the same rows: each writes half of their dims
      if (shared) {
        sm.ml[wg][row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.x_full);
        if (!(ok = ca_wait(&sm.x_full, xcount & 1, err, 823))) break;
        const float2 x0 = sm.ml[0][row], x1 = sm.ml[1][row];
        m = fmaxf(x0.x, x1.x);
        f0 = x0.x == -INFINITY ? 0.f : ex2(x0.x - m);
        f1 = x1.x == -INFINITY ? 0.f : ex2(x1.x - m);
        l = f0 * x0.y + f1 * x1.y;
        c0 = lanes + kCaOCol;
        c1 = lanes + kCaOCol + 128;
        d0 = 64 * wg;
        nd = 64;
      }
      __syncwarp();
      tc::fence_after();
      if (active && (steps > 0 || shared)) {
        const float inv = it.slot >= 0 ? 1.f : l == 0.f ? 0.f : a.v_scale / l;
        f0 *= inv;
        f1 *= inv;
#pragma unroll 1
        for (int d = d0; d < d0 + nd; d += 16) {
          uint32_t u[16], v[16];
          tc::ld_32x32b_x16(c0 + d, u);
          if (shared) tc::ld_32x32b_x16(c1 + d, v);
          tc::wait_ld();
          float o[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            // a factor of zero stands for sums that hold nothing: they are not read as numbers
            o[q] = f0 != 0.f ? __uint_as_float(u[q]) * f0 : 0.f;
            if (shared && f1 != 0.f) o[q] = fmaf(__uint_as_float(v[q]), f1, o[q]);
          }
          if (valid && it.slot >= 0) {
            float4* p = a.part_o + (static_cast<long long>(it.slot) * (kDim / 4) + d / 4) * a.rows + prow;
#pragma unroll
            for (int q = 0; q < 4; ++q) p[q * a.rows] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          } else if (valid) {
            uint32_t y[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] = pack_bf16(o[2 * q], o[2 * q + 1]);
            ca_store32(a.out + orow * kDim + d, y, (reinterpret_cast<uintptr_t>(a.out) & 31) == 0);
          }
          __syncwarp();
        }
        if (valid && d0 == 0) {
          if (it.slot >= 0) a.part_ml[static_cast<long long>(it.slot) * a.rows + prow] = make_float2(m, l);
          else if (a.lse) a.lse[orow] = l == 0.f ? -INFINITY : m + log2f(l);
        }
      }
      if (shared) {
        // neither goes on to its next O while the other still reads it
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.x_done);
        if (!(ok = ca_wait(&sm.x_done, xcount & 1, err, 824))) break;
        ++xcount;
      }
    }
    roles_done();
    if constexpr (kOne)
      if (sm.apart) ca_one_attend<kFp8>(a, sm, warp);
  } else if (kFp8 && warp >= kCaWidenWarp) {
    // ---------------- E4M3 pages and bf16 queries to fp16 ----------------
    ca_regs_down<Shape::kRegsWiden>();
    constexpr int kLanes = 128, kStep = kLanes / 8;  // kStep: rows at once
    const int wt = tid - 32 * kCaWidenWarp;
    // Eight lanes take 16-byte pieces of two neighbouring rows, the odd row's from the other half: they read and write
    // eight different 16-byte banks of the swizzled tiles.
    const int i8 = wt & 7, odd = i8 >> 2, piece = (i8 & 3) + 4 * (((wt >> 3) & 1) ^ odd), row0 = 2 * (wt >> 4) + odd;
    int base = 0, nq = 0;
    bool ok = tiles;
    // the item's queries
    auto widen_q = [&](int ntok) {
      for (int q = 0; q < (ntok > 8 ? 2 : 1) && ok; ++q, ++nq) {
        const int s = nq & 1, bytes = min(8, ntok - 8 * q) * kCaQEntry;
        if (!(ok = ca_wait(&sm.q_full[s], (nq >> 1) & 1, err, 833))) break;
        const uint32_t at = smem_u32(sm.q[s]);
        for (int o = wt * 16; o < bytes; o += kLanes * 16) {
          const uint4 v = lds128(at + o);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[i] = pack_f16(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
          sts128(at + o, y[0], y[1], y[2], y[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_ready[s]);
      }
    };
    for (int n = 0; ok; ++n) {
      const int is = n % kCaInfo;
      if (!(ok = ca_wait(&sm.info_full[is], (n / kCaInfo) & 1, err, 830))) break;
      const int nb = sm.info[is].nb, b0 = sm.info[is].b0, len = sm.info[is].len, ntok = sm.info[is].ntok;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.info_empty[is]);
      if (nb == 0) break;
      for (int j = 0; j < 2 * nb && ok; ++j) {
        const int load = 2 * base + j, rs = load % Shape::kRaw, st = load % kTiles;
        const bool is_v = ca_is_v(j, nb);
        if (!(ok = ca_wait(&sm.raw_full[rs], (load / Shape::kRaw) & 1, err, 831))) break;
        // V rows behind the last key become zero: their weight is zero, but they may hold anything
        int keys = kBlock;
        if (is_v) {
          const int k = ca_block_v(j, nb);
          keys = sm.bad[(base + k) % kCaBad] ? 0 : min(kBlock, len - (b0 + k) * kBlock);
        }
        const uint32_t src = smem_u32(sm.raw[kFp8 ? rs : 0]) + sw128(row0, piece);
        const uint32_t dst = smem_u32(sm.kv[st]) + (piece >> 2) * kCaHalf;
        const uint32_t dst0 = dst + sw128(row0, 2 * (piece & 3)), dst1 = dst + sw128(row0, 2 * (piece & 3) + 1);
        // two rows at a time, the next two asked for before
        constexpr int kBatches = kBlock / kStep / 2;
        uint4 x[2][2];
#pragma unroll
        for (int q = 0; q < 2; ++q) x[0][q] = lds128(src + q * kStep * 128);
        if (!(ok = ca_wait(&sm.kv_empty[st], ((load / kTiles) & 1) ^ 1, err, 832))) break;
#pragma unroll
        for (int n = 0; n < kBatches; ++n) {
          if (n + 1 < kBatches)
#pragma unroll
            for (int q = 0; q < 2; ++q) x[(n + 1) & 1][q] = lds128(src + (2 * n + 2 + q) * kStep * 128);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int down = (2 * n + q) * kStep;  // rows below row0, a multiple of the swizzle's eight
            uint4 v = x[n & 1][q];
            if (keys < kBlock && row0 + down >= keys) v = make_uint4(0u, 0u, 0u, 0u);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              y[2 * i] = ca_widen2(w[i]);
              y[2 * i + 1] = ca_widen2(w[i] >> 16);
            }
            sts128(dst0 + down * 128, y[0], y[1], y[2], y[3]);
            sts128(dst1 + down * 128, y[4], y[5], y[6], y[7]);
          }
          if (n + 2 == kBatches) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.raw_empty[rs]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.kv_full[st]);
        if (j == 0) widen_q(ntok);
      }
      base += nb;
    }
  }
  // (the roles' register counts end with their branches, so the one-token items are taken inside them)
  if (warp >= 8 && warp != kCaProducerWarp) roles_done();
  if (warp == kCaMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

// Joins the pieces of the items that were cut.  CTA (c, e) takes token e of the item that begins in share c, 16 rows (the
// token's heads); behind those, one CTA per share the one-token item that begins there.  The pieces' (m, l) go to shared
// memory; a warp per row turns them into factors; then thread (row, four dims) adds up its values, the loads of
// eight pieces in flight at once.  Bound by the latency of those rounds, so the rows are spread over as many CTAs as
// there are tokens.  (With four tokens to a CTA, and the factors in each thread, the whole call took 20 us instead of
// 14 for four short requests; with 256 threads, two values each, 20 instead of 16 for one of 63 blocks.)
constexpr int kCaJoinThreads = kGroup * kDim / 4;
__global__ void __launch_bounds__(kCaJoinThreads) chunk_join_kernel(const __grid_constant__ CaArgs a) {
  __shared__ float2 ml[kNumSMs][kGroup];  // then .x: the piece's factor
  __shared__ float inv[kGroup];
  __shared__ __align__(16) uint2 out[kGroup][kDim / 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int e = blockIdx.x / kNumSMs, c = blockIdx.x % kNumSMs;
  const bool one = e * kGroup >= a.rows;  // a one-token item over an E4M3 cache
  const int e0 = one ? 0 : e * kGroup;    // first row in the item
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float2* part_ml = one ? a.part1_ml : a.part_ml;
  const float4* part_o = one ? a.part1_o : a.part_o;
  const long long rows = one ? kGroup : a.rows;
  // the pieces lie in slots 2 c + 1, 2 (c + 1), 2 (c + 2), ..
  auto slot = [&](int s) { return s == 0 ? 2 * c + 1 : 2 * (c + s); };
  // asked for with the cut, not after it: the first 32 pieces' (m, l)
  const float2 first = part_ml[slot(min(tid / kGroup, kNumSMs - 1 - c)) * rows + e0 + tid % kGroup];
  const CaCut cut = (one ? a.cuts1 : a.cuts)[c];
  if (e0 >= cut.ntok * kGroup) return;
  const int parts = cut.last - c + 1;
  if (tid < parts * kGroup) ml[tid / kGroup][tid % kGroup] = first;
  for (int i = tid + kCaJoinThreads; i < parts * kGroup; i += kCaJoinThreads)
    ml[i / kGroup][i % kGroup] = part_ml[slot(i / kGroup) * rows + e0 + i % kGroup];
  __syncthreads();
  const long long row0 = (static_cast<long long>(cut.t0) + e0 / kGroup) * kHeads + cut.g * kGroup;  // the token's first row
  float m = -INFINITY, l = 0.f;  // of row `warp`
  for (int s = lane; s < parts; s += 32) m = fmaxf(m, ml[s][warp].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  for (int s = lane; s < parts; s += 32) {
    const float f = ml[s][warp].x == -INFINITY ? 0.f : ex2(ml[s][warp].x - m);
    ml[s][warp].x = f;
    l = fmaf(f, ml[s][warp].y, l);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if (lane == 0) {
    inv[warp] = l == 0.f ? 0.f : a.v_scale / l;
    if (a.lse) a.lse[row0 + warp] = l == 0.f ? -INFINITY : m + log2f(l);
  }
  __syncthreads();
  const int row = tid % kGroup, d4 = tid / kGroup;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = 0; s < parts; ++s) {
    const float4 x = part_o[(slot(s) * static_cast<long long>(kDim / 4) + d4) * rows + e0 + row];
    const float f = ml[s][row].x;
    o.x = fmaf(f, x.x, o.x);
    o.y = fmaf(f, x.y, o.y);
    o.z = fmaf(f, x.z, o.z);
    o.w = fmaf(f, x.w, o.w);
  }
  const float r = inv[row];
  out[row][d4] = make_uint2(pack_bf16(o.x * r, o.y * r), pack_bf16(o.z * r, o.w * r));
  __syncthreads();
  if (tid < kGroup * kDim / 8)
    reinterpret_cast<uint4*>(a.out + row0 * kDim)[tid] = reinterpret_cast<const uint4*>(&out[0][0])[tid];
}

// ---- host side ----------------------------------------------------------------------

static size_t ca_up(size_t x) { return (x + 255) / 256 * 256; }
static int ca_rows(long long tokens) { return kGroup * static_cast<int>(tokens < kCaTok ? tokens : kCaTok); }

// Scratch of a call: the cuts, then the two partials of every CTA, and of every CTA's one-token items.
constexpr size_t kCaRows1 = 2 * static_cast<size_t>(kNumSMs) * kGroup;
size_t attend_chunk_bytes(long long tokens, int) {
  const size_t rows = 2 * static_cast<size_t>(kNumSMs) * ca_rows(tokens);
  return ca_up(2 * kNumSMs * sizeof(CaCut)) + ca_up(rows * sizeof(float2)) + rows * kDim * sizeof(float) +
         ca_up(kCaRows1 * sizeof(float2)) + kCaRows1 * kDim * sizeof(float);
}

// q [T, 64, 128] bf16 as (dims 0-63, head % 8, dims / 64, head / 8, token): a token's 16 heads of a KV head in one box of
// four 8-row swizzle atoms.
static bool ca_encode_q(CUtensorMap* map, const void* base, cuuint64_t T) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[5] = {64, 8, 2, kHeads / 8, T};
  const cuuint64_t strides[4] = {kDim * 2, 128, 8 * kDim * 2, kHeads * kDim * 2};
  const cuuint32_t box[5] = {64, 8, 2, 2, 1}, step[5] = {1, 1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A cache [slots, 4, 128]: boxes of one head's 128 slots, 64 dims of bf16 or all 128 of E4M3.  A head's row is 256 bytes, or
// 128: promoted to 256 there, L2 fetched the neighbouring head's with it (16 tokens over 128k keys: 3.2 GB read for
// 2.1, 0.45 ms instead of 0.32).
static bool ca_encode_kv(CUtensorMap* map, const void* base, cuuint64_t slots, bool fp8) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  const cuuint64_t size = fp8 ? 1 : 2;
  const cuuint64_t dims[3] = {kDim, kKvHeads, slots}, strides[2] = {kDim * size, kKvHeads * kDim * size};
  const cuuint32_t box[3] = {fp8 ? 128u : 64u, 1, kBlock}, step[3] = {1, 1, 1};
  return enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B,
             fp8 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kFp8, bool kOne>
static cudaError_t ca_launch(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap, const CaArgs& a,
                             cudaStream_t stream) {
  constexpr size_t bytes = sizeof(CaSmem<kFp8>);
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
  if (const cudaError_t e = cudaFuncSetAttribute(chunk_attend_kernel<kFp8, kOne>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(bytes));
      e != cudaSuccess)
    return e;
  return launch_dependent(chunk_attend_kernel<kFp8, kOne>, dim3(kNumSMs), CaShape<kFp8>::kThreads, bytes, stream, qmap, kmap,
                             vmap, a);
}

cudaError_t launch_attend_chunk(const ChunkLaunch& L, cudaStream_t stream) {
  if (const cudaError_t e0 = launch_prologue(); e0 != cudaSuccess) return e0;
  CUtensorMap qmap, kmap, vmap;
  if (!ca_encode_q(&qmap, L.q, L.tokens) || !ca_encode_kv(&kmap, L.k, L.num_slots, L.kv_fp8) ||
      !ca_encode_kv(&vmap, L.v, L.num_slots, L.kv_fp8))
    return cudaErrorInvalidValue;
  CaArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(L.q);
  a.seq_lens = L.seq_lens;
  a.page_table = L.page_table;
  a.cu = L.cu;
  a.batch = L.batch;
  a.max_blocks = L.max_blocks;
  a.num_pages = static_cast<int>(L.num_slots / kBlock);
  a.tokens = L.tokens;
  a.scale_log2 = chunk_scale_log2(L.scale, L.k_scale);
  a.v_scale = L.v_scale;
  a.out = static_cast<__nv_bfloat16*>(L.out);
  a.lse = L.lse;
  a.rows = ca_rows(L.tokens);
  const size_t rows = 2 * static_cast<size_t>(kNumSMs) * a.rows;
  uint8_t* p = L.scratch;
  a.cuts = reinterpret_cast<CaCut*>(p);
  a.cuts1 = a.cuts + kNumSMs;
  p += ca_up(2 * kNumSMs * sizeof(CaCut));
  a.part_ml = reinterpret_cast<float2*>(p);
  p += ca_up(rows * sizeof(float2));
  a.part_o = reinterpret_cast<float4*>(p);
  p += rows * kDim * sizeof(float);
  a.part1_ml = reinterpret_cast<float2*>(p);
  p += ca_up(kCaRows1 * sizeof(float2));
  a.part1_o = reinterpret_cast<float4*>(p);
  a.err = L.err;
  // A batch of single tokens has no more of them than requests.  (The code for such batches cost others 0.4 us a call, and
  // 16 tokens over 32k keys 3.)
  if (const cudaError_t e = L.kv_fp8 ? ca_launch<true, true>(qmap, kmap, vmap, a, stream)
                            : L.tokens <= L.batch ? ca_launch<false, true>(qmap, kmap, vmap, a, stream)
                                                  : ca_launch<false, false>(qmap, kmap, vmap, a, stream);
      e != cudaSuccess)
    return e;
  return launch_dependent(chunk_join_kernel, dim3(kNumSMs * (a.rows / kGroup + (L.kv_fp8 ? 1 : 0))), kCaJoinThreads, 0,
                             stream, a);
}

}  // namespace msa
