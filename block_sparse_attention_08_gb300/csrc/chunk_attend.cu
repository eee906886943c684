// chunk_attend.cu -- causal attention of each request's new tokens over all its
// keys in the paged cache (bf16, E4M3 or int8), and the same where requests share
// the first pages of their contexts.
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
// has a third warpgroup that widens each page to fp16 (exactly) in shared memory;
// an int8 one has it write n s as bf16, each row by its scale (exactly, where
// scales are powers of two), so that Q and P stay bf16.
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
// int8: 2682 tokens in chunks over 3k to 13k keys take 0.587 ms (E4M3 0.51, bf16
// 0.475: its widening is 8 instructions for four values where E4M3's is 2; with one
// instead of four for a pair of values it would be 0.49), 16 single tokens over 128k keys
// (2.18 GB) 0.339 ms, 6.4 TB/s.
//
// Shared prefixes: sum_j p_j v_j and sum_j p_j over all keys are those over the
// shared and over a request's own keys, brought to one m.  The groups' shared blocks
// are items of their own, 16 tokens of any of the group's requests without a mask,
// listed before the requests', whose items leave these blocks out: pages that n
// requests share are read n / 16 times instead of n.  The pieces of both are
// joined by shared_join_kernel.  64 tokens over 16k shared keys, bf16: 63 us
// (194 unshared; 168 MB, 26 us); 256 over 32k, E4M3: 249 us (1200; 145), two thirds of it
// the shared items' tiles; four over 2k: 14 us, computed per request.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "int8_attend.cuh"
#include "launch.h"

namespace msa {

constexpr int kCaTok = 16;            // new tokens per item
constexpr int kCaTile = 128 * 256;    // 128 rows x 128 dims of 16 bits
constexpr int kCaHalf = kCaTile / 2;  // one 64-dim half
constexpr int kCaQEntry = 4096;       // one token's 16 heads x 128 dims
constexpr int kCaInfo = 4;            // item descriptors in flight
constexpr int kCaOnePlaces = 5;       // blocks in flight of one-token items (32 KB each)
constexpr int kCaBad = 8;             // block flags in flight (at most 5 blocks are)
// warps 0-7 softmax, 8 producer, 9 MMA, 10 bad requests (11 fills their warpgroup; int8: both widen too), 12-15 widening
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
  int slot;         // partial slot, or -1: the piece is the whole item (kCaOwn, kCaShared: to be joined with other items)
  int row;          // row of the page table
};
// Whole items of a token's own keys, and of those that its group shares: their sums go to the token's place.
constexpr int kCaOwn = -2, kCaShared = -3;
// For the joining kernel: an item that begins in CTA c and ends in CTA `last`.
struct CaCut {
  int t0, ntok, g, last;
};

// The sums of whole items, and where a token's pieces are (CaPieces).
struct CaTokens {
  float4* o;    // [tokens][4][32][16]
  float2* ml;   // [tokens][4][16]
  int32_t* at;  // [tokens][4]
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
  // int8: the rows' scales
  const __nv_bfloat16 *k_scales, *v_scales;
  // shared prefixes: groups of requests, and what each token's items left, by (token, KV head)
  const int32_t *group_offsets, *shared_lens;
  int groups;
  CaTokens own, shared;
};

// The caches' types (the template parameter kKv below).
constexpr int kCaBf16 = 0, kCaE4m3 = 1, kCaI8 = 2;

template <int kKv>
struct CaShape {
  static constexpr bool kFp8 = kKv != kCaBf16;  // 8-bit values (int8 as well): copied as they are, then widened
  static constexpr bool kF16 = kKv == kCaE4m3;  // Q, K, V and P enter the products as fp16
  // (int8: the scales lie in the fifth's place, and an even number leaves each place to the same four warps)
  static constexpr int kOnePlaces = kKv == kCaI8 ? 4 : kCaOnePlaces;
  // 16-bit K / V tiles.  (E4M3: with 3 of them and 4 copied ones, the places of widened tiles came free too late: 0.63 ms
  // instead of 0.60 for 2548 tokens in chunks over 4k to 12k keys.)
  static constexpr int kTiles = kFp8 ? 4 : 5;
  static constexpr int kRaw = kFp8 ? 2 : 1;    // 8-bit tiles as copied
  static constexpr int kWiden = kFp8 ? 4 : 0;  // widening warps
  // and beside the issuing warps: int8 tiles wait for their widening (2682 tokens in chunks over 3k to 13k keys 631 us without,
  // 587 with them; E4M3 511 either way)
  static constexpr int kHelp = kKv == kCaI8 ? 2 : 0;
  static constexpr int kThreads = 32 * (kCaWidenWarp + kWiden);
  // registers per thread of the roles, out of the launch's 168 (384 threads) or 128 (512 threads) a thread:
  // 256 * 216 + 128 * 72 = 384 * 168, and 256 * 208 + 128 * 56 + 128 * 40 = 512 * 128.  (With 184 for the softmax, E4M3
  // chunks took 6% more.
  // Two widening warps in the issuing warps' group leave it 216: chunks 1% faster, but items of few tokens, bound by the
  // widening, made 17 mixed requests 126 us instead of 115.  int8: 256 * 200 + 256 * 56; the widening in 40 registers 688 us,
  // in 48 599, in 64, which leave the softmax 192, 580, but 3 groups of 40 requests 138 instead of 137.)
  static constexpr int kRegsSoftmax = kKv == kCaI8 ? 200 : kFp8 ? 208 : 216, kRegsIssue = kFp8 ? 56 : 72;
  static constexpr int kRegsWiden = kKv == kCaI8 ? 56 : 40;
  // fp16 weights are kept near the top of their range (at most 2^(kLift + kCaSlack) = 2^15), so that small ones
  // stay normal down to 2^-21 of the largest
  static constexpr float kLift = kF16 ? 7.f : 0.f;
};

// A CTA's part [u0, u1) of all units of a kind.  The shares are equal parts of `total`, to which a unit of this kind adds
// `weight`, behind the `before` of the other (shared prefixes: both kinds are shared out in one row, else each by itself).
struct CaShareOf {
  long long total, ctas, u0, u1, before;
  int weight;
  // the share that holds the last unit before unit x
  __device__ __forceinline__ int holder(long long x) const {
    return static_cast<int>(((before + weight * x) * ctas - 1) / total);
  }
};
// ---- the units of a request --------------------------------------------------------

// sum of floor(y / 8) over 0 <= y < x
__device__ __forceinline__ long long ca_eighths(long long x) {
  const long long q = x >> 3;
  return 4 * q * (q - 1) + q * (x & 7);
}
// A request's n new tokens at positions len - n .. len - 1, as ceil(n / 16) items per KV head; item i sees the
// blocks up to its last token's, without the first `skip` ones (which its group shares).  With `whole`: the n tokens of a
// group's requests, which all see the blocks of the `len` shared keys.
struct CaReqOf {
  int t0, n, len;
  bool apart;  // a last item of one token is not counted (it is shared out apart)
  int extra;   // units of an item besides its blocks
  int skip, row;  // (with shared prefixes alone) row: of the page table
  bool whole;
};
template <bool kShared>
struct CaReq : CaReqOf {
  __device__ __forceinline__ bool one() const { return !(kShared && whole) && n % kCaTok == 1; }  // the last item has one token
  __device__ __forceinline__ int items() const { return (n + kCaTok - 1) / kCaTok - (apart && one()); }
  __device__ __forceinline__ int blocks(int i) const {
    if (kShared && whole) return len / kBlock;
    return (len - n + min(n, kCaTok * (i + 1)) - 1) / kBlock + 1 - (kShared ? skip : 0);
  }
  __device__ __forceinline__ bool dual(int i) const { return n - kCaTok * i > kCaTok / 2; }  // both tiles
  // units of the items before item i (all of 16 tokens)
  __device__ __forceinline__ long long before(int i) const {
    if (kShared && whole) return static_cast<long long>(len / kBlock + extra) * i;
    const long long a = (static_cast<long long>(len) - n + kCaTok - 1) / kCaTok;
    return ca_eighths(a + i) - ca_eighths(a) + i + static_cast<long long>(extra - (kShared ? skip : 0)) * i;
  }
  // units of item i
  __device__ __forceinline__ int units(int i) const { return extra + (dual(i) ? blocks(i) : (blocks(i) + 1) / 2); }
  __device__ __forceinline__ long long per_head() const {
    const int i = items() - 1;
    if (i < 0) return 0;
    return before(i) + units(i);
  }
  // units of the last item where that has one token and is shared out apart, and its blocks that begin before its unit x: the
  // first two at 0, the others after the item's own units
  __device__ __forceinline__ int one_blocks() const { return (len - 1) / kBlock + 1 - (kShared ? skip : 0); }
  __device__ __forceinline__ int one_units() const { return one() ? (one_blocks() + 1) / 2 + (kShared ? extra : 0) : 0; }
  __device__ __forceinline__ int one_begun(int x) const {
    if (kShared) x = x <= 0 ? 0 : 1 + max(0, x - 1 - extra);
    return min(one_blocks(), 2 * x);
  }
  // the items' sums are joined with others'
  __device__ __forceinline__ bool joined() const { return kShared && (whole || skip > 0); }
};
__device__ __forceinline__ bool ca_good(const CaArgs& a, long long c0, long long c1, int len) {
  return c0 >= 0 && c0 <= c1 && c1 <= a.tokens && c1 - c0 <= len && (len + kBlock - 1LL) / kBlock <= a.max_blocks;
}
// The requests of group g, the blocks that they share, the blocks that are attended to once for all of them (all or none), and
// their tokens.  Nothing is shared by a group with offsets that are no range, and nothing attended to once where that does not pay: for
// requests that bring 16 tokens or more on average, which fill their items by themselves; for two tokens (26 us instead of 21
// over 16k shared keys, 64 instead of 68 over 128k, and over E4M3 59 instead of 51); and for less than 8 over few pages (4 over 8k 20 us
// instead of 19, over 32k 35 and 34, over 64k 42 instead of 55; 5 over 16k 27 instead of 29; 8 over 1k 15 instead of 17).
constexpr int kCaFewTokens = 8, kCaFewBlocks = 400;
struct CaGroup {
  int r0, blocks, once, t0, n;
};
__device__ __forceinline__ CaGroup ca_group(const CaArgs& a, int g) {
  const int r0 = a.group_offsets[g], r1 = a.group_offsets[g + 1], blocks = a.shared_lens[g] / kBlock;
  if (r0 < 0 || r1 > a.batch || r1 <= r0 || blocks < 1) return CaGroup{r0, 0, 0, 0, 0};
  const int some = min(blocks, a.max_blocks);
  const long long c0 = a.cu[r0], c1 = a.cu[r1], n = c1 - c0;
  if (c0 < 0 || n < 3 || c1 > a.tokens || r1 - r0 < 2 || n >= static_cast<long long>(kCaTok) * (r1 - r0) ||
      (n < kCaFewTokens && (n - 1) * some < kCaFewBlocks))
    return CaGroup{r0, some, 0, 0, 0};
  return CaGroup{r0, some, some, static_cast<int>(c0), static_cast<int>(n)};
}
// The group of request r (no blocks: none).
__device__ __forceinline__ CaGroup ca_group_of(const CaArgs& a, int r) {
  int lo = 0, hi = a.groups;  // the first group that ends behind r
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (a.group_offsets[mid + 1] > r) hi = mid;
    else lo = mid + 1;
  }
  if (lo == a.groups) return CaGroup{0, 0, 0, 0, 0};
  const CaGroup g = ca_group(a, lo);
  return g.r0 <= r ? g : CaGroup{0, 0, 0, 0, 0};
}
// Whether request r is good, and the blocks that its group attends to for it.
template <bool kShared>
__device__ __forceinline__ bool ca_good_request(const CaArgs& a, int r, int c0, int c1, int len, int& skip) {
  skip = 0;
  if (!ca_good(a, c0, c1, len)) return false;
  if (!kShared) return true;
  const CaGroup g = ca_group_of(a, r);
  skip = g.once;
  return c0 == c1 || len - (c1 - c0) >= g.blocks * kBlock;
}
// Entry r of the list of work: a request, with shared prefixes the groups before them; one with bad lengths has no tokens.
template <bool kShared>
__device__ __forceinline__ CaReq<kShared> ca_req(const CaArgs& a, int r, bool apart, int extra = 0) {
  CaReq<kShared> q{CaReqOf{0, 0, 0, apart, extra, 0, 0, false}};
  if (kShared) {
    if (r < a.groups) {
      const CaGroup g = ca_group(a, r);
      if (g.once) q.t0 = g.t0, q.n = g.n, q.len = g.once * kBlock, q.row = g.r0, q.whole = true;
      return q;
    }
    r -= a.groups;
  }
  const int c0 = a.cu[r], c1 = a.cu[r + 1], len = a.seq_lens[r];
  int skip;
  if (ca_good_request<kShared>(a, r, c0, c1, len, skip)) q.t0 = c0, q.n = c1 - c0, q.len = len, q.skip = skip, q.row = r;
  return q;
}
// For the joining kernel where prefixes are shared: the pieces of a token's own item, and of its group's.
struct CaPieces {
  // join: there is something to join; shared: so is a part of the group's; cut: pieces of CTAs first .. last, else the token's
  // place; one: of one-token items; e: the token's number in its item
  bool join, shared, cut, one;
  int first, last, e;
  __device__ __forceinline__ int32_t code() const {
    return join | shared << 1 | cut << 2 | one << 3 | e << 4 | first << 8 | last << 16;
  }
  __device__ static __forceinline__ CaPieces of(int32_t x) {
    return CaPieces{(x & 1) != 0, (x & 2) != 0, (x & 4) != 0, (x & 8) != 0, min(x >> 8 & 255, kNumSMs - 1),
                    min(x >> 16 & 255, kNumSMs - 1), x >> 4 & 15};
  }
};
static_assert(kNumSMs <= 256 && kCaTok <= 16, "the fields of a CaPieces code");
// Zeros for the rows of a request with bad lengths (the whole warp).
template <bool kShared>
__device__ __noinline__ void ca_refuse(const CaArgs& a, int r, int lane) {
  if (lane == 0) record_error(a.err, MSA_DEVERR_LENGTH, r);
  const long long c0 = max(0, a.cu[r]), c1 = min(a.tokens, static_cast<long long>(a.cu[r + 1]));
  uint4* out = reinterpret_cast<uint4*>(a.out);
  for (long long i = c0 * (kHeads * kDim / 8) + lane; i < c1 * (kHeads * kDim / 8); i += 32)
    out[i] = make_uint4(0u, 0u, 0u, 0u);
  if (a.lse)
    for (long long i = c0 * kHeads + lane; i < c1 * kHeads; i += 32) a.lse[i] = -INFINITY;
  if (kShared)
    for (long long i = c0 * kKvHeads + lane; i < c1 * kKvHeads; i += 32) a.own.at[i] = 0;
}

// This CTA's part of the requests with bad lengths (one warp).
template <bool kShared>
__device__ __forceinline__ void ca_refuse_bad(const CaArgs& a, int lane) {
  for (long long r0 = blockIdx.x; r0 < a.batch; r0 += 32LL * gridDim.x) {
    const long long r = r0 + static_cast<long long>(lane) * gridDim.x;
    int skip;
    const bool bad = r < a.batch && !ca_good_request<kShared>(a, static_cast<int>(r), a.cu[r], a.cu[r + 1], a.seq_lens[r], skip);
    for (unsigned m = __ballot_sync(0xffffffffu, bad); m; m &= m - 1)
      ca_refuse<kShared>(a, static_cast<int>(r0 + static_cast<long long>(__ffs(m) - 1) * gridDim.x), lane);
  }
}

// The request (and the unit in it) where a share begins.
struct CaStart {
  long long unit;
  int r;
  CaReqOf q;
};

template <int kKv>
struct CaSmem {
  static constexpr bool kFp8 = kKv != kCaBf16;
  uint8_t q[2][kCaTile];
  uint8_t kv[CaShape<kKv>::kTiles][kCaTile];
  uint8_t raw[CaShape<kKv>::kRaw][kFp8 ? kCaHalf : 16];
  float2 ml[2][128];  // before the roles begin: the warps' sums
  uint64_t q_full[2], q_ready[2], q_empty[2];  // q_ready: as fp16 (E4M3 cache)
  uint64_t kv_full[CaShape<kKv>::kTiles], kv_empty[CaShape<kKv>::kTiles];
  uint64_t raw_full[CaShape<kKv>::kRaw], raw_empty[CaShape<kKv>::kRaw];
  uint64_t s_full[2], p_full[2], o_full[2], x_full, x_done, done;
  uint64_t info_full[kCaInfo], info_empty[kCaInfo];
  // one-token items: K and V bytes of a block per place (over kv and raw), descriptors, the warps' meeting
  uint64_t one_full[kCaOnePlaces], one_empty[kCaOnePlaces], one_info_full[kCaInfo], one_info_empty[kCaInfo];
  uint64_t one_x_full, one_x_done;
  CaItem info[kCaInfo];
  int bad[kCaBad];
  CaStart start[2];  // of the items, and of the one-token items
  CaShareOf share[2];
  int extra, extra1;  // units of an item besides its blocks, and of a one-token item
  bool apart;  // the one-token items are shared out apart, after the others
  uint32_t tmem_base;
};

// The whole CTA: sums up the requests' units and finds this CTA's share of each kind, and where it begins.  The units that an
// item counts besides its blocks depend on the total, so the items are summed up beside their blocks.  (The caller's barrier
// follows.)
template <int kKv, bool kOne, bool kShared>
__device__ __forceinline__ void ca_find_shares(const CaArgs& a, CaSmem<kKv>& sm) {
  constexpr bool kFp8 = CaShape<kKv>::kFp8;
  const int entries = a.batch + (kShared ? a.groups : 0);
  constexpr int kThreads = CaShape<kKv>::kThreads, kWarps = kThreads / 32, kKinds = kOne ? 2 : 1;
  constexpr int kN = kShared ? 4 : kOne ? 3 : 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // all KV heads' units without the items' own, items (bf16: the one-token ones too), and units of one-token items: of this
  // thread's request, and of the warp's requests up to and with it (the warps' own sums in wsum); shared prefixes: one-token
  // items
  long long (*wsum)[kWarps] = reinterpret_cast<long long (*)[kWarps]>(&sm.ml[0][0]);
  static_assert(kN * kWarps * sizeof(long long) <= sizeof(sm.ml), "wsum lies over ml");
  CaReq<kShared> q{};
  long long u[kN], incl[kN], base[kN] = {};
  auto pass = [&](int r0) {
    const int r = r0 + tid;
    q = r < entries ? ca_req<kShared>(a, r, kOne) : CaReq<kShared>{};
    u[0] = kKvHeads * q.per_head();
    u[1] = kKvHeads * static_cast<long long>(q.items() + (kOne && !kFp8 && !kShared && q.one()));
    if constexpr (kOne) u[2] = kKvHeads * static_cast<long long>(q.one_units());
    if constexpr (kShared) u[3] = kKvHeads * static_cast<long long>(q.one());
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
  int extra = 0, extra1 = 0;
  bool apart = kOne;
  // the units of either kind, out of the sums
  auto units = [&](const long long (&x)[kN], int k) {
    if (!kOne) return x[0] + extra * x[1];
    if constexpr (kShared) return k ? x[2] + extra1 * x[3] : x[0] + extra * x[1];
    if (kFp8 || apart) return k ? x[kN - 1] : x[0] + extra * x[1];
    return k ? 0LL : x[0] + x[kN - 1] + extra * x[1];
  };
  auto split = [&](const long long (&total)[kN]) {
    apart = kOne && (kFp8 || kShared || total[0] == 0);  // (bf16: only where there are no others)
    extra = 0;
    // (a share is long enough to hold some block's beginning)
    auto ctas = [&](long long n, int e) { return min(static_cast<long long>(gridDim.x), max(n / (1 + e), 1LL)); };
    bool row = false;
    if constexpr (kShared) {
      // The end of a one-token item is worth a unit (256 requests over 32k shared keys 0.264 ms without, 0.249 with).
      extra = ca_item_units(total[0] + total[2]);
      extra1 = min(extra, 1);
      // Both kinds in one row, so that all but one CTA have items of one kind, and the one's start, end and waits for HBM pass
      // beside the other's products: 64 requests over 16k keys, bf16, 63 us instead of 76, four over 2k 15 instead of 17.  In time a unit
      // of one-token items (two blocks) is 1.2 units of tiles over a bf16 cache, and 1.4 in shares of 32 units on (256 requests
      // over 32k 233 us instead of 244, 128 over 16k 86.6 instead of 89.2, but 64 over 16k 65 instead of 63).  Over 8-bit ones a unit
      // of either kind keeps an SM busy, and the one-token items' ends fall to few of them: in long shares the kinds take no less
      // side by side, whatever a unit counts (256 requests over 32k, E4M3, 0.29 ms instead of 0.25), so there each CTA takes the one
      // after the other.
      row = !kFp8 || extra < 2;
    }
    if (row) {
      const bool far = total[0] + total[2] >= 32LL * gridDim.x;
      const int tile = kFp8 || extra == 0 ? 1 : 5, token = kFp8 || extra == 0 ? 1 : far ? 7 : 6;
      const long long n0 = units(total, 0), n1 = units(total, 1), sum = tile * n0 + token * n1;
      const long long c = ctas(sum / token, extra);
      const long long p0 = sum * min(static_cast<long long>(blockIdx.x), c) / c, p1 = sum * min(blockIdx.x + 1LL, c) / c;
      auto part = [&](long long p) { return max(p - tile * n0, 0LL) / token; };
      share[0] = CaShareOf{sum, c, min(p0 / tile, n0), min(p1 / tile, n0), 0, tile};
      share[kKinds - 1] = CaShareOf{sum, c, part(p0), part(p1), tile * n0, token};
      return;
    }
    if (!kShared) extra = ca_item_units(units(total, 0));
#pragma unroll
    for (int k = 0; k < kKinds; ++k) {
      CaShareOf& s = share[k];
      s.total = units(total, k);
      s.ctas = ctas(s.total, k ? extra1 : extra);
      s.u0 = min(s.total, s.total * blockIdx.x / s.ctas);
      s.u1 = min(s.total, s.total * (blockIdx.x + 1) / s.ctas);
      s.before = 0;
      s.weight = 1;
    }
  };
  const bool once = entries <= kThreads;
  if (!once) {
    for (int r0 = 0; r0 < entries; r0 += kThreads) {
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
  for (int r0 = 0; r0 < entries; r0 += kThreads) {
    pass(r0);
    const int warps = min(kWarps, (entries - r0 + 31) / 32);  // that hold requests
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
        q.extra = k ? extra1 : extra;
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
    sm.extra1 = extra1;
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

// Two int8 values (bytes 0 and 1 of w, or 2 and 3) times a power of two s, as bf16, exactly.  at: the bits of 128 s in both halves,
// step: the bits in which those of 256 s differ.  With its low seven bits m a byte makes (128 + m) s, with its sign 128 s, or
// 256 s for a negative one (the byte permutation has the sign in all the upper bits); their difference is n s.  (Decoded
// first and multiplied then, one more instruction of four: 648 us instead of 625 for 2682 tokens in chunks.)
template <bool kUpper>
__device__ __forceinline__ uint32_t ca_i8_scaled(uint32_t w, uint32_t at, uint32_t step) {
  uint32_t t, d;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(t) : "r"(w), "n"(kUpper ? 0xb3a2 : 0x9180));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"((t & 0x007f007fu) | at), "r"((t & step) ^ at));
  return d;
}
// at (upper half) and step (lower) for the scale with bits s; not ok: it is no power of two for which 128 s and 256 s are normal
// numbers (and its code is that of 1).
__device__ __forceinline__ uint32_t ca_i8_code(uint32_t s, bool& ok) {
  const uint32_t field = s >> 7;  // (with the sign)
  ok = field ? (s & 0x7fu) == 0 && field <= 246 : s != 0 && (s & (s - 1)) == 0;
  const uint32_t at = !ok ? 0x4300u : field ? s + 0x380 : (32 - __clz(s)) << 7;
  return at << 16 | (at ^ (at + 0x80));
}

// Products of m16n8k16, the 16 query heads their rows, from the copied pages.  E4M3: warps 0 to 3 take the even blocks, 32
// keys each, warps 4 to 7 the odd ones.  S = Q K^T: a 16-bit ldmatrix of K gives a lane four consecutive bytes of one key,
// dims 16 s + 4 t .. + 3 of k-step s, so Q's fragments hold those dims in the same slots.  O += P V: a transposing ldmatrix
// gives a lane two dims of two keys, which make one value pair for each of two products, one for the even dims and one for the
// odd.  bf16: each warp takes 16 keys of every block, K and V in places of their own.  Bound by HBM: each page is copied in
// and read once.  (16 tokens over 128k keys, E4M3, 2.15 GB: 0.32 ms, 6.7 TB/s.)

// A CTA's share of the one-token items, piece by piece: units u .. of KV head g's item of entry r.
template <bool kShared>
struct CaOneWalk {
  int r;
  CaReq<kShared> q;
  int per, g, u;
  long long at;  // of all units
  __device__ __forceinline__ CaOneWalk(const CaStart& s, long long u0) : r(s.r), q{s.q}, per(q.one_units()), at(u0) {
    g = (s.unit >= per) + (s.unit >= 2LL * per) + (s.unit >= 3LL * per);
    u = static_cast<int>(s.unit - static_cast<long long>(g) * per);
  }
  // where the piece ends
  __device__ __forceinline__ int to(long long u1) const { return static_cast<int>(min(static_cast<long long>(per), u + u1 - at)); }
  // the piece's first block (of the request's), and its place in the page table
  __device__ __forceinline__ int block() const { return q.one_begun(u) + (kShared ? q.skip : 0); }
  __device__ __forceinline__ long long row(const CaArgs& a) const {
    return static_cast<long long>(kShared ? q.row : r) * a.max_blocks + block();
  }
  // goes on behind the piece, which ended before the share did
  __device__ __forceinline__ void next(const CaArgs& a, int extra1) {
    u = 0;
    if (++g < kKvHeads) return;
    g = 0;
    do {
      q = ca_req<kShared>(a, ++r, true, extra1);
      per = q.one_units();
    } while (per == 0);
  }
};

// The copies (the producer warp).
template <int kKv, bool kShared>
__device__ __forceinline__ void ca_one_produce(const CUtensorMap& kmap, const CUtensorMap& vmap, const CaArgs& a,
                                               const CaShareOf& share, CaSmem<kKv>& sm) {
  constexpr bool kFp8 = CaShape<kKv>::kFp8;
  constexpr int kPlaces = CaShape<kKv>::kOnePlaces;
  const int lane = threadIdx.x & 31, c = static_cast<int>(blockIdx.x);
  DevError* err = a.err;
  uint8_t* places = &sm.kv[0][0];
  static_assert(sizeof(sm.kv) + sizeof(sm.raw) >= kCaOnePlaces * kCaTile, "the places lie over kv and raw");
  {
    CaCut cut{0, 0, 0, 0};
    int nitem = 0, nplace = 0;  // descriptors and places filled
    bool ok = true;
    if (share.u0 < share.u1) {
      CaOneWalk<kShared> w(sm.start[1], share.u0);
      while (true) {
        const CaReq<kShared>& q = w.q;
        const int to = w.to(share.u1), g = w.g;
        CaItem it{q.t0 + q.n - 1, 1, g, q.len - 1, q.len, w.block(), q.one_begun(to) - q.one_begun(w.u), 0, 0};
        const bool begins = w.u == 0, whole = begins && it.nb == q.one_blocks();
        it.slot = whole ? (q.joined() ? kCaOwn : -1) : 2 * c + begins;
        if (begins) {
          const int last = whole ? 0 : share.holder(w.at + w.per);  // the share that holds the item's last unit
          if (kShared) {
            if (lane == 0)
              a.own.at[static_cast<long long>(it.t0) * kKvHeads + g] =
                  CaPieces{!whole || q.joined(), q.joined(), !whole, true, c, last, 0}.code();
          } else if (!whole) {
            cut = CaCut{it.t0, 1, g, last};
          }
        }
        w.at += to - w.u;
        if (it.nb > 0) {
        const int is = nitem % kCaInfo;
        if (!(ok = ca_wait(&sm.one_info_empty[is], ((nitem / kCaInfo) & 1) ^ 1, err, 840))) break;
        if (lane == 0) {
          sm.info[is] = it;
          mbar_arrive(&sm.one_info_full[is]);
        }
        ++nitem;
        const long long row0 = w.row(a);
        const int32_t* row = a.page_table + row0;
        int ids = 0, ids_next = lane < it.nb ? row[lane] : 0;
        for (int k = 0; k < it.nb && ok; ++k) {
          if ((k & 31) == 0) {
            ids = ids_next;
            ids_next = k + 32 + lane < it.nb ? row[k + 32 + lane] : 0;
          }
          int page = __shfl_sync(0xffffffffu, ids, k & 31);
          const bool bad = page < 0 || page >= a.num_pages;
          if (bad) {
            if (lane == 0) record_error(err, MSA_DEVERR_PAGE, row0 + k);
            page = 0;
          }
          // 8 bits: K and V to one place; bf16: to one each
#pragma unroll
          for (int kv = 0; kv < (kFp8 ? 1 : 2); ++kv, ++nplace) {
            const int s = nplace % kPlaces;
            if (!(ok = ca_wait(&sm.one_empty[s], ((nplace / kPlaces) & 1) ^ 1, err, 841))) break;
            if (lane == 0) {
              sm.bad[s] = bad;
              uint8_t* st = places + s * kCaTile;
              mbar_expect_tx(&sm.one_full[s], kCaTile + (kKv == kCaI8 ? 4 * kBlock : 0));
              tma_load_3d(st, kv ? &vmap : &kmap, 0, g, page * kBlock, &sm.one_full[s]);
              tma_load_3d(st + kCaHalf, kFp8 || kv ? &vmap : &kmap, kFp8 ? 0 : 64, g, page * kBlock, &sm.one_full[s]);
              if constexpr (kKv == kCaI8) {
                uint8_t* sc = places + kPlaces * kCaTile + s * 4 * kBlock;
                const long long from = (static_cast<long long>(page) * kKvHeads + g) * kBlock;
                tma_bulk_g2s(sc, a.k_scales + from, 2 * kBlock, &sm.one_full[s]);
                tma_bulk_g2s(sc + 2 * kBlock, a.v_scales + from, 2 * kBlock, &sm.one_full[s]);
              }
            }
          }
        }
        }
        if (!ok || w.at >= share.u1) break;
        w.next(a, sm.extra1);
      }
    }
    if (!kShared && lane == 0) (kFp8 ? a.cuts1 : a.cuts)[blockIdx.x] = cut;
    if (ok && ca_wait(&sm.one_info_empty[nitem % kCaInfo], ((nitem / kCaInfo) & 1) ^ 1, err, 842) && lane == 0) {
      sm.info[nitem % kCaInfo] = CaItem{0, 0, 0, 0, 0, 0, 0, 0, 0};
      mbar_arrive(&sm.one_info_full[nitem % kCaInfo]);
    }
    __syncwarp();
    if (lane == 0)  // no copy may still be landing when the CTA exits
      for (int s = 0; s < kPlaces; ++s) {
        const int fills = (nplace - s + kPlaces - 1) / kPlaces;
        if (fills > 0) mbar_wait(&sm.one_full[s], (fills - 1) & 1, err, 843);
      }
  }
}

// The sums (warps 0 to 7).
template <int kKv, bool kShared>
__device__ __forceinline__ void ca_one_attend(const CaArgs& a, CaSmem<kKv>& sm, int warp) {
  constexpr bool kFp8 = CaShape<kKv>::kFp8, kI8 = kKv == kCaI8;
  constexpr int kPlaces = CaShape<kKv>::kOnePlaces;
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
      // Q rows g8 and g8 + 8, the A operand.  bf16: k-step s holds dims 16 s + 2t, + 1, + 8, + 9.  E4M3 (as fp16), int8: dims
      // 16 s + 4 t .. + 3 in the same slots, which is where a lane's four bytes of K go.
      uint32_t qa[8][4];
      {
        const __nv_bfloat16* q0 = a.q + (static_cast<long long>(it.t0) * kHeads + it.g * kGroup + g8) * kDim;
        const __nv_bfloat16* q1 = q0 + 8 * kDim;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          if constexpr (kFp8) {
            const uint2 x = reinterpret_cast<const uint2*>(q0 + 4 * t4)[4 * s], y = reinterpret_cast<const uint2*>(q1 + 4 * t4)[4 * s];
            if constexpr (kI8) {
              i8_queries(qa[s], x, y);
            } else {
              qa[s][0] = pack_f16(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u));
              qa[s][1] = pack_f16(__uint_as_float(y.x << 16), __uint_as_float(y.x & 0xffff0000u));
              qa[s][2] = pack_f16(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
              qa[s][3] = pack_f16(__uint_as_float(y.y << 16), __uint_as_float(y.y & 0xffff0000u));
            }
          } else {
            qa[s][0] = *reinterpret_cast<const uint32_t*>(q0 + 16 * s + 2 * t4);
            qa[s][1] = *reinterpret_cast<const uint32_t*>(q1 + 16 * s + 2 * t4);
            qa[s][2] = *reinterpret_cast<const uint32_t*>(q0 + 16 * s + 2 * t4 + 8);
            qa[s][3] = *reinterpret_cast<const uint32_t*>(q1 + 16 * s + 2 * t4 + 8);
          }
        }
      }
      constexpr float kLift = CaShape<kKv>::kLift;
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
        // (int8: four warps have read the place, and arrive for the other four)
        if (lane < (kI8 ? 2 : 1)) mbar_arrive(&sm.one_empty[s]);
      };
      auto q_of = [&](int c, uint32_t(&x)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = qa[c][i];
      };
      I8State st;  // (an int8 cache's sums, until the item's end)
      if constexpr (kI8) i8_clear(st);
      uint32_t at8[4];
      if constexpr (kI8) i8_offsets(at8, 32 * (warp & 3), lane);
      bool ok = true;
      for (int k = 0; k < it.nb; ++k) {
        const int s = nplace % kPlaces;
        if (kI8 && (nplace & 1) != (warp >> 2)) {  // the other four warps' block
          ++nplace;
          continue;
        }
        if (!(ok = ca_wait(&sm.one_full[s], (nplace / kPlaces) & 1, err, 845))) break;
        const int block_keys = sm.bad[s] ? 0 : min(kBlock, it.len - (it.b0 + k) * kBlock);
        const uint32_t kt = smem_u32(places + s * kCaTile);
        if constexpr (kI8) {
          ++nplace;
          const int row0 = 32 * (warp & 3), keys = block_keys - row0;  // of this warp's 32
          const uint32_t* sc = reinterpret_cast<const uint32_t*>(places + kPlaces * kCaTile + s * 4 * kBlock) + row0 / 2 + t4;
          if (keys > 0) i8_attend32(st, q_of, kt, kt + kCaHalf, at8, sc, sc + kBlock / 2, keys, a.scale_log2, t4);
          release(s);
        } else if constexpr (kFp8) {
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
          const int sv = nplace % kPlaces;
          if (!(ok = ca_wait(&sm.one_full[sv], (nplace / kPlaces) & 1, err, 848))) break;
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
      if constexpr (kI8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m[h] = st.m[h];
          l[h] = st.l[h];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] = st.o[i][e];
      }
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
          constexpr bool kApart = kFp8 || kShared;  // pieces of their own
          const long long rows = kApart ? kGroup : a.rows;
          (kApart ? a.part1_o : a.part_o)[(static_cast<long long>(it.slot) * (kDim / 4) + lane) * rows + row] = v;
          if (lane == 0) (kApart ? a.part1_ml : a.part_ml)[it.slot * rows + row] = make_float2(top, sum);
        } else if (kShared && it.slot == kCaOwn) {
          const long long at = static_cast<long long>(it.t0) * kKvHeads + it.g;
          a.own.o[(at * (kDim / 4) + lane) * kGroup + row] = v;
          if (lane == 0) a.own.ml[at * kGroup + row] = make_float2(top, sum);
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
// kShared: the requests' entries begin with those of the groups, and sums that belong together are joined by
// shared_join_kernel
template <int kKv, bool kOne, bool kShared>
__global__ void __launch_bounds__(CaShape<kKv>::kThreads, 1) chunk_attend_kernel(
    const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
    const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CaArgs a) {
  using Shape = CaShape<kKv>;
  constexpr bool kFp8 = Shape::kFp8, kI8 = kKv == kCaI8;
  constexpr int kTiles = Shape::kTiles, kThreads = Shape::kThreads;
  constexpr int kRing = kFp8 ? Shape::kRaw : kTiles;  // places that tiles are copied into
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  CaSmem<kKv>& sm = *reinterpret_cast<CaSmem<kKv>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  DevError* err = a.err;

  if (smem_u32(smem_raw) & 1023) {  // the swizzled tiles need it; with no static shared memory it holds
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
      record_error(err, MSA_DEVERR_TIMEOUT, 899);
      if (!kShared) a.cuts[blockIdx.x] = a.cuts1[blockIdx.x] = CaCut{0, 0, 0, 0};
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
      if (!Shape::kHelp) mbar_init(&sm.kv_full[i], kFp8 ? 4 : 1);
      else mbar_init(&sm.kv_full[i], 4 + Shape::kHelp);
      mbar_init(&sm.kv_empty[i], 1);
    }
    for (int i = 0; i < Shape::kRaw; ++i) {
      mbar_init(&sm.raw_full[i], 1);
      if (!Shape::kHelp) mbar_init(&sm.raw_empty[i], 4);
      else mbar_init(&sm.raw_empty[i], 4 + Shape::kHelp);
    }
    mbar_init(&sm.x_full, 8);
    mbar_init(&sm.x_done, 8);
    mbar_init(&sm.done, 1);
    for (int i = 0; i < kCaInfo; ++i) {
      mbar_init(&sm.info_full[i], 1);
      if (!Shape::kHelp) mbar_init(&sm.info_empty[i], 9 + Shape::kWiden);  // the softmax, MMA and widening warps
      else mbar_init(&sm.info_empty[i], 9 + Shape::kWiden + Shape::kHelp);
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

  ca_find_shares<kKv, kOne, kShared>(a, sm);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem_base, 0);

  // (where all items are one-token items computed apart, the tiles' roles have nothing to do: 0.2 us less)
  const bool tiles = !kOne || (kShared ? sm.share[0].u0 < sm.share[0].u1 : sm.share[0].total > 0);
  // All roles of all warps are done: tensor memory may be released, and the tiles' places copied into again.
  auto roles_done = [&] {
    if (!tiles) return;
    tc::fence_before();
    if (kFp8 || kShared) fence_proxy_async_smem();  // (bf16 else: either there are other items, or one-token items)
    __syncwarp();
    asm volatile("barrier.sync 1, %0;" ::"n"(kThreads) : "memory");
  };
  // A wait that gives up (recorded in the error word) ends its role, so a broken pipeline ends after one bounded wait
  // per role.
  if (warp >= 8 && warp < kCaWidenWarp) ca_regs_down<Shape::kRegsIssue>();
  if (Shape::kHelp && warp >= kCaWidenWarp) ca_regs_down<Shape::kRegsWiden>();
  if (warp == kCaProducerWarp) {
    // ---------------- the share's items, and their copies ----------------
    const long long u0 = sm.share[0].u0, u1 = sm.share[0].u1;
    CaCut cut{0, 0, 0, 0};
    int nitem = 0, nq = 0, nload = 0, nblk = 0;  // descriptors, Q tiles, K / V tiles and blocks issued
    bool ok = true;
    if (u0 < u1) {
      const int extra = sm.extra;
      int r = sm.start[0].r;
      CaReq<kShared> rq{sm.start[0].q};
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
        it.row = kShared ? rq.row : r;
        if (kShared && rq.whole) it.pos0 = rq.len - 1;  // (all tokens see all keys)
        it.b0 = begun(at - item0);
        it.nb = begun(min(end, u1) - item0) - it.b0;
        const int b = it.b0;
        const bool to_end = b + it.nb == blocks;
        it.slot = b == 0 && to_end ? (!rq.joined() ? -1 : rq.whole ? kCaShared : kCaOwn)
                                   : static_cast<int>(2 * blockIdx.x + (b == 0));
        if (kShared && !rq.whole) it.b0 += rq.skip;  // (of the request's blocks)
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
        const long long row0 = static_cast<long long>(it.row) * a.max_blocks + it.b0;
        const int32_t* row = a.page_table + row0;
        int ids = 0, ids_next = lane < it.nb ? row[lane] : 0;  // 32 page ids, and the next 32
        int last = 0, before = 0;  // pages of the last block that K was loaded of, and of the one before
        for (int j = 0; j < 2 * it.nb && ok; ++j) {  // tile j: K of block (j + 1) / 2 and V in turn
          const bool is_v = ca_is_v(j, it.nb);
          int page;
          if (!is_v) {
            const int k = (j + 1) >> 1;
            if ((k & 31) == 0) {
              ids = ids_next;
              ids_next = k + 32 + lane < it.nb ? row[k + 32 + lane] : 0;
            }
            page = __shfl_sync(0xffffffffu, ids, k & 31);
            const bool bad = page < 0 || page >= a.num_pages;
            if (bad) {
              if (lane == 0) record_error(err, MSA_DEVERR_PAGE, row0 + k);
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
        if (kShared) {
          if (b == 0 && lane < it.ntok)
            (rq.whole ? a.shared : a.own).at[(static_cast<long long>(it.t0) + lane) * kKvHeads + g] =
                CaPieces{!to_end || rq.joined(), rq.joined(), !to_end, false, static_cast<int>(blockIdx.x),
                         to_end ? 0 : sm.share[0].holder(end), lane}.code();
        } else if (b == 0 && !to_end) {
          cut = CaCut{it.t0, it.ntok, g, sm.share[0].holder(end)};
        }
        if (!ok || at >= u1) break;
        // the next item (the share goes on, so there is one)
        if (++i == rq.items()) {
          i = 0;
          if (++g == kKvHeads) {
            g = 0;
            do {
              rq = ca_req<kShared>(a, ++r, kOne && sm.apart, extra);
            } while (rq.items() == 0);
          }
        }
      }
    }
    if (!kShared && lane == 0) a.cuts[blockIdx.x] = cut;
    if (tiles && ok && ca_wait(&sm.info_empty[nitem % kCaInfo], ((nitem / kCaInfo) & 1) ^ 1, err, 804) && lane == 0) {
      sm.info[nitem % kCaInfo] = CaItem{0, 0, 0, 0, 0, 0, 0, 0, 0};
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
      if (sm.apart) ca_one_produce<kKv, kShared>(kmap, vmap, a, sm.share[1], sm);
  } else if (warp == kCaMmaWarp) {
    // ---------------- S and O products ----------------
    // One thread issues them all, and they execute in the order in which they are issued: an S product that overwrites P
    // follows the O product that reads it, and the two warpgroups' products alternate, so that one's softmax runs beside
    // the other's products.  (With a thread for each warpgroup's they fell into step, both softmaxes and then both
    // products at once: 1.59 ms instead of 1.34 ms for 2048 tokens over 32k keys.)  The thread holds few products
    // ahead of the tensor cores, so it looks for what the next ones need before it issues a group, not between groups.
    constexpr uint32_t idesc_s = ca_idesc(Shape::kF16), idesc_o = ca_idesc(Shape::kF16) | (1u << 16);
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
          ok = mbar_wait(Shape::kF16 ? &sm.q_ready[t & 1] : &sm.q_full[t & 1], (t >> 1) & 1, err, 811);
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
  } else if (!Shape::kHelp && warp == kCaMmaWarp + 1) {
    // ---------------- requests with bad lengths ----------------
    ca_refuse_bad<kShared>(a, lane);
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
                  pk[q] = Shape::kF16 ? pack_f16(pa, pb) : pack_bf16(pa, pb);
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
        const bool part = kShared ? it.slot != -1 : it.slot >= 0;
        // where the sums go: a piece's place, or the token's
        float4* po = a.part_o + static_cast<long long>(it.slot) * (kDim / 4) * a.rows + prow;
        float2* pml = a.part_ml + static_cast<long long>(it.slot) * a.rows + prow;
        int rows = a.rows;
        if (kShared && it.slot < 0) {
          const CaTokens& to = it.slot == kCaOwn ? a.own : a.shared;
          const long long at = (static_cast<long long>(it.t0) + tok) * kKvHeads + it.g;
          rows = kGroup;
          po = to.o + at * (kDim / 4) * kGroup + (row & 15);
          pml = to.ml + at * kGroup + (row & 15);
        }
        const float inv = part ? 1.f : l == 0.f ? 0.f : a.v_scale / l;
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
          if (valid && part) {
            float4* p = po + static_cast<long long>(d / 4) * rows;
#pragma unroll
            for (int q = 0; q < 4; ++q) p[q * rows] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          } else if (valid) {
            uint32_t y[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] = pack_bf16(o[2 * q], o[2 * q + 1]);
            ca_store32(a.out + orow * kDim + d, y, (reinterpret_cast<uintptr_t>(a.out) & 31) == 0);
          }
          __syncwarp();
        }
        if (valid && d0 == 0) {
          if (part) *pml = make_float2(m, l);
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
      if (sm.apart) ca_one_attend<kKv, kShared>(a, sm, warp);
  } else if (kFp8 && (Shape::kHelp || warp >= kCaWidenWarp)) {
    // ---------------- E4M3 pages and bf16 queries to fp16; int8 pages, with their rows' scales, to bf16 ----------------
    if (!Shape::kHelp) ca_regs_down<Shape::kRegsWiden>();
    constexpr int kLanes = 32 * (kFp8 ? Shape::kWiden + Shape::kHelp : 4), kStep = kLanes / 8;  // kStep: rows at once
    constexpr int kSteps = (kBlock + kStep - 1) / kStep;                            // the last one by some warps alone
    const int ww = warp >= kCaWidenWarp ? warp - kCaWidenWarp : warp - (kCaWidenWarp - Shape::kHelp) + Shape::kWiden, wt = 32 * ww + lane;
    const bool all_steps = kBlock % kStep == 0 || 4 * ww + (kSteps - 1) * kStep < kBlock;
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
      // int8: each lane has the scale of one of the warp's 32 rows, asked for a tile ahead, from the pages as the producer
      // finds them
      const int i_row = 4 * ww + (lane & 3) + kStep * (lane >> 2);
      const int32_t* table = a.page_table + static_cast<long long>(sm.info[is].row) * a.max_blocks + b0;
      const int at_g = sm.info[is].g * kBlock + min(i_row, kBlock - 1);
      int ids = 0, ids_next = 0, last = 0, before = 0;
      uint32_t next_scale = 0;
      if (kI8 && nb > 0) ids_next = lane < nb ? table[lane] : 0;
      auto ask = [&](int j) {
        if (j >= 2 * nb) return;
        const bool is_v = ca_is_v(j, nb);
        if (!is_v) {
          const int k = (j + 1) >> 1;
          if ((k & 31) == 0) {
            ids = ids_next;
            ids_next = k + 32 + lane < nb ? table[k + 32 + lane] : 0;
          }
          const int page = __shfl_sync(0xffffffffu, ids, k & 31);
          before = last;
          last = page < 0 || page >= a.num_pages ? 0 : page;
        }
        const int from = is_v && j < 2 * nb - 1 ? before : last;
        next_scale = reinterpret_cast<const uint16_t*>(is_v ? a.v_scales : a.k_scales)[static_cast<long long>(from) * (kKvHeads * kBlock) + at_g];
      };
      if constexpr (kI8) ask(0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.info_empty[is]);
      if (nb == 0) break;
      for (int j = 0; j < 2 * nb && ok; ++j) {
        const int load = 2 * base + j, rs = load % Shape::kRaw, st = load % kTiles;
        const bool is_v = ca_is_v(j, nb);
        const uint32_t scale = next_scale;
        bool powers = true;
        uint32_t code = 0;
        if constexpr (kI8) {
          code = ca_i8_code(scale, powers);
          ask(j + 1);
        }
        if (!(ok = ca_wait(&sm.raw_full[rs], (load / Shape::kRaw) & 1, err, 831))) break;
        // V rows behind the last key become zero: their weight is zero, but they may hold anything
        int keys = kBlock;
        if (is_v) {
          const int k = ca_block_v(j, nb);
          keys = sm.bad[(base + k) % kCaBad] ? 0 : min(kBlock, len - (b0 + k) * kBlock);
        }
        // int8: tiles of powers of two, as rows are written, take no multiplication
        if constexpr (kI8)
          if (!(powers = __all_sync(0xffffffffu, powers || i_row >= keys))) code = (i_row < keys ? scale : 0x3f80u) * 0x10001u;
        const uint32_t src = smem_u32(sm.raw[kFp8 ? rs : 0]) + sw128(row0, piece);
        const uint32_t dst = smem_u32(sm.kv[st]) + (piece >> 2) * kCaHalf;
        const uint32_t dst0 = dst + sw128(row0, 2 * (piece & 3)), dst1 = dst + sw128(row0, 2 * (piece & 3) + 1);
        // two rows at a time, the next two asked for before
        constexpr int kBatches = kSteps / 2;
        uint4 x[2][2];
#pragma unroll
        for (int q = 0; q < 2; ++q) x[0][q] = lds128(src + q * kStep * 128);
        if (!(ok = ca_wait(&sm.kv_empty[st], ((load / kTiles) & 1) ^ 1, err, 832))) break;
        auto widen = [&](auto fast) {
#pragma unroll
          for (int n = 0; n < kBatches; ++n) {
            if (n + 1 < kBatches)
#pragma unroll
              for (int q = 0; q < 2; ++q)
                if (2 * n + 3 + q < kSteps || all_steps) x[(n + 1) & 1][q] = lds128(src + (2 * n + 2 + q) * kStep * 128);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              if (2 * n + q + 1 == kSteps && !all_steps) break;
              const int down = (2 * n + q) * kStep;  // rows below row0, a multiple of the swizzle's eight
              uint4 v = x[n & 1][q];
              if (keys < kBlock && row0 + down >= keys) v = make_uint4(0u, 0u, 0u, 0u);
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
              const uint32_t ss = kI8 ? __shfl_sync(0xffffffffu, code, (row0 & 3) + 4 * (2 * n + q)) : 0u;
              const uint32_t at = __byte_perm(ss, 0, 0x3232), step = __byte_perm(ss, 0, 0x1010);
              uint32_t y[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if constexpr (!kI8) {
                  y[2 * i] = ca_widen2(w[i]);
                  y[2 * i + 1] = ca_widen2(w[i] >> 16);
                } else if constexpr (decltype(fast)::value) {
                  y[2 * i] = ca_i8_scaled<false>(w[i], at, step);
                  y[2 * i + 1] = ca_i8_scaled<true>(w[i], at, step);
                } else {
                  y[2 * i] = mul_bf16x2(i8_lo2(w[i]), ss);
                  y[2 * i + 1] = mul_bf16x2(i8_hi2(w[i]), ss);
                }
              }
              sts128(dst0 + down * 128, y[0], y[1], y[2], y[3]);
              sts128(dst1 + down * 128, y[4], y[5], y[6], y[7]);
            }
            if (n + 1 == kBatches) {  // (once the last rows have been stored: a load that is only asked for may still read the place)
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.raw_empty[rs]);
            }
          }
        };
        if (!kI8 || powers) widen(std::true_type{});
        else widen(std::false_type{});
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.kv_full[st]);
        if (!kI8 && j == 0) widen_q(ntok);
      }
      base += nb;
    }
    if (Shape::kHelp && warp == kCaMmaWarp + 1) ca_refuse_bad<kShared>(a, lane);
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

// The same where prefixes are shared: a CTA takes (token, KV head) pairs, and joins the pieces of the token's own item with
// those of its group's.  A thread has four dims of a row, and reads the row's (m, l) of each piece beside its sums, so the only
// loads that follow each other are a pair's code and its pieces, kCaJoinBatch of them at a time.  (With the factors
// worked out once per row in shared memory, as above, four tokens took 28 us instead of 17.)  Few tokens over a long
// prefix have many pieces, one from each CTA that had a part of their group's item, and leave most SMs idle: kSplit > 1 gives a
// pair to kSplit CTAs, a part of the dims each, whose threads share out the pieces (4 tokens over 16k keys: 36 us without; two
// CTAs each for 64 tokens over 16k: 66.6 us instead of 64.1).
constexpr int kCaJoinBatch = 4, kCaJoinSplit = 4;
template <int kSplit>
__global__ void __launch_bounds__(kCaJoinThreads, 2) shared_join_kernel(const __grid_constant__ CaArgs a) {
  constexpr int kLanes = kCaJoinThreads / kSplit;  // threads that share out nothing: 16 rows, and dims in fours
  __shared__ float2 part_ml[kSplit][kGroup];
  __shared__ float4 part_o[kSplit][kSplit > 1 ? kLanes : 1];
  const int tid = threadIdx.x, lane = tid & 31, share = tid / kLanes, row = tid % kGroup;
  const int d4 = static_cast<int>(blockIdx.x % kSplit) * (kLanes / kGroup) + tid % kLanes / kGroup;
  const int cta = blockIdx.x / kSplit, ctas = gridDim.x / kSplit;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // (read beside the first codes, not before them)
  const long long from = static_cast<long long>(max(a.cu[0], 0)) * kKvHeads, all = a.tokens * kKvHeads;
  const long long to = min(all, static_cast<long long>(a.cu[a.batch]) * kKvHeads);
  // one source of n pieces, of which piece 0 lies one slot behind the pointers and piece q > 0 2 q slots (a slot has as many rows; a
  // token's place none)
  struct Source {
    const float4* o;
    const float2* ml;
    int rows, n;
  };
  auto source = [&](const CaPieces& c, const CaTokens& t, long long at) {
    if (!c.cut) return Source{t.o + (at * (kDim / 4) + d4) * kGroup + row, t.ml + at * kGroup + row, 0, 1};
    const int rows = c.one ? kGroup : a.rows, in = (c.one ? 0 : c.e * kGroup) + row, from = 2 * c.first * rows;
    return Source{(c.one ? a.part1_o : a.part_o) + (from * (kDim / 4) + d4 * rows + in),
                  (c.one ? a.part1_ml : a.part_ml) + (from + in), rows, max(c.last - c.first, 0) + 1};
  };
  // 32 pairs' codes at once: most of a long batch's have nothing to join
  for (long long base = cta; base < all; base += 32LL * ctas) {
    const long long mine = base + static_cast<long long>(lane) * ctas;
    const int32_t own_code = mine < all ? a.own.at[mine] : 0, with_code = mine < all ? a.shared.at[mine] : 0;  // (may be anything)
    if (base >= to) break;
    const bool in = mine >= from && mine < to;
    for (unsigned left = __ballot_sync(0xffffffffu, in && CaPieces::of(own_code).join); left; left &= left - 1) {
      const int k = __ffs(left) - 1;
      const long long at = base + static_cast<long long>(k) * ctas;
      const CaPieces own = CaPieces::of(__shfl_sync(0xffffffffu, own_code, k));
      const CaPieces with = CaPieces::of(__shfl_sync(0xffffffffu, with_code, k));
      const Source x = source(own, a.own, at), y = source(with, a.shared, at);
      const int n = x.n + (own.shared ? y.n : 0);
      float m = -INFINITY, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      // (m is at least the piece's.  A maximum passes over what is no number, so a piece without one may still have a sum that is
      // none: it is added, by a factor that keeps it so.)
      auto add = [&](float2 ml, float4 v) {
        const float g = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
        l = fmaf(g, ml.y, l);
        o.x = fmaf(g, v.x, o.x);
        o.y = fmaf(g, v.y, o.y);
        o.z = fmaf(g, v.z, o.z);
        o.w = fmaf(g, v.w, o.w);
      };
      for (int s0 = share; s0 < n; s0 += kSplit * kCaJoinBatch) {
        float4 v[kCaJoinBatch];
        float2 ml[kCaJoinBatch];
#pragma unroll
        for (int i = 0; i < kCaJoinBatch; ++i) {
          const int s = min(s0 + kSplit * i, n - 1);
          const bool first = s < x.n;
          const int q = first ? s : s - x.n, off = (2 * q + (q == 0)) * (first ? x.rows : y.rows);
          ml[i] = (first ? x.ml : y.ml)[off];
          v[i] = (first ? x.o : y.o)[off * (kDim / 4)];
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < kCaJoinBatch; ++i)
          if (s0 + kSplit * i < n) top = fmaxf(top, ml[i].x);
        const float f = m == -INFINITY ? 0.f : ex2(m - top);
        m = top;
        l *= f;
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
        for (int i = 0; i < kCaJoinBatch; ++i)
          if (s0 + kSplit * i < n) add(ml[i], v[i]);
      }
      if constexpr (kSplit > 1) {
        part_o[share][tid % kLanes] = o;
        if (tid % kLanes < kGroup) part_ml[share][row] = make_float2(m, l);
        __syncthreads();
        if (share == 0) {
          const float mine_m = m;
          float top = m;
#pragma unroll
          for (int i = 1; i < kSplit; ++i) top = fmaxf(top, part_ml[i][row].x);
          const float f = mine_m == -INFINITY ? 0.f : ex2(mine_m - top);
          m = top;
          l *= f;
          o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
          for (int i = 1; i < kSplit; ++i) add(part_ml[i][row], part_o[i][tid % kLanes]);
        }
      }
      if (share == 0) {
        const long long orow = at / kKvHeads * kHeads + at % kKvHeads * kGroup + row;
        const float inv = l == 0.f ? 0.f : a.v_scale / l;
        if (a.lse && d4 == 0) a.lse[orow] = l == 0.f ? -INFINITY : m + log2f(l);
        // the lanes of 16 rows have dims 4 d4 .. and, in the warp's other half, the next four: one 16-byte store for both
        const uint2 lo = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        const uint2 hi = make_uint2(__shfl_xor_sync(0xffffffffu, lo.x, 16), __shfl_xor_sync(0xffffffffu, lo.y, 16));
        if (lane < 16) stg128(a.out + orow * kDim + 4 * d4, lo.x, lo.y, hi.x, hi.y);
      }
      if (kSplit > 1) __syncthreads();
    }
  }
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

// With shared prefixes behind that: the sums of whole items and the codes of their pieces, of the tokens' own items and of
// their groups'.
static size_t ca_tokens_bytes(long long tokens) {
  const size_t pairs = static_cast<size_t>(tokens) * kKvHeads;
  return ca_up(pairs * sizeof(int32_t)) + ca_up(pairs * kGroup * sizeof(float2)) + pairs * kGroup * kDim * sizeof(float);
}
size_t attend_shared_bytes(long long tokens) { return attend_chunk_bytes(tokens, 0) + 2 * ca_tokens_bytes(tokens); }

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

template <int kKv, bool kOne, bool kShared>
static cudaError_t ca_launch(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap, const CaArgs& a,
                             cudaStream_t stream) {
  constexpr size_t bytes = sizeof(CaSmem<kKv>);
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
  if (const cudaError_t e = cudaFuncSetAttribute(chunk_attend_kernel<kKv, kOne, kShared>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
      e != cudaSuccess)
    return e;
  return launch_dependent(chunk_attend_kernel<kKv, kOne, kShared>, dim3(kNumSMs), CaShape<kKv>::kThreads, bytes, stream, qmap,
                          kmap, vmap, a);
}

cudaError_t launch_attend_chunk(const ChunkLaunch& L, cudaStream_t stream) {
  if (const cudaError_t e0 = launch_prologue(); e0 != cudaSuccess) return e0;
  CUtensorMap qmap, kmap, vmap;
  if (!ca_encode_q(&qmap, L.q, L.tokens) || !ca_encode_kv(&kmap, L.k, L.num_slots, L.kv != kCaBf16) ||
      !ca_encode_kv(&vmap, L.v, L.num_slots, L.kv != kCaBf16))
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
  p += kCaRows1 * kDim * sizeof(float);
  a.err = L.err;
  a.k_scales = static_cast<const __nv_bfloat16*>(L.k_scales);
  a.v_scales = static_cast<const __nv_bfloat16*>(L.v_scales);
  if (L.groups > 0) {
    a.group_offsets = L.group_offsets;
    a.shared_lens = L.shared_lens;
    a.groups = L.groups;
    const size_t pairs = static_cast<size_t>(L.tokens) * kKvHeads;
    for (CaTokens* t : {&a.own, &a.shared}) {
      t->at = reinterpret_cast<int32_t*>(p);
      p += ca_up(pairs * sizeof(int32_t));
      t->ml = reinterpret_cast<float2*>(p);
      p += ca_up(pairs * kGroup * sizeof(float2));
      t->o = reinterpret_cast<float4*>(p);
      p += pairs * kGroup * kDim * sizeof(float);
    }
    if (const cudaError_t e = L.kv == kCaBf16   ? ca_launch<kCaBf16, true, true>(qmap, kmap, vmap, a, stream)
                              : L.kv == kCaE4m3 ? ca_launch<kCaE4m3, true, true>(qmap, kmap, vmap, a, stream)
                                                : ca_launch<kCaI8, true, true>(qmap, kmap, vmap, a, stream);
        e != cudaSuccess)
      return e;
    // as many CTAs as are resident at once: two an SM
    constexpr size_t kCtas = 2 * kNumSMs;
    if (pairs * kCaJoinSplit <= 2 * kCtas)
      return launch_dependent(shared_join_kernel<kCaJoinSplit>, dim3(static_cast<unsigned>(pairs * kCaJoinSplit)),
                              kCaJoinThreads, 0, stream, a);
    return launch_dependent(shared_join_kernel<1>, dim3(static_cast<unsigned>(std::min(pairs, kCtas))), kCaJoinThreads, 0,
                            stream, a);
  }
  // A batch of single tokens has no more of them than requests.  (The code for such batches cost others 0.4 us a call, and
  // 16 tokens over 32k keys 3.)
  if (const cudaError_t e = L.kv == kCaI8     ? ca_launch<kCaI8, true, false>(qmap, kmap, vmap, a, stream)
                            : L.kv == kCaE4m3 ? ca_launch<kCaE4m3, true, false>(qmap, kmap, vmap, a, stream)
                            : L.tokens <= L.batch ? ca_launch<kCaBf16, true, false>(qmap, kmap, vmap, a, stream)
                                                  : ca_launch<kCaBf16, false, false>(qmap, kmap, vmap, a, stream);
      e != cudaSuccess)
    return e;
  return launch_dependent(chunk_join_kernel, dim3(kNumSMs * (a.rows / kGroup + (L.kv != kCaBf16 ? 1 : 0))), kCaJoinThreads, 0,
                             stream, a);
}

}  // namespace msa
