// tree_attn_decode: attention of a tree of drafted tokens over the FP4 cache.
//
// Token t of a sequence sees the prefix rows (all of them, or a selection) and the drafted rows of
// its mask: o = sum_j softmax_j(sm_scale q . v_j) v_j over those rows, lse = ln of the sum. All T * H
// query rows of a sequence meet the same cache rows, so this is two matrix products (4 * 512 flops
// per query row and cache row, tensor-core bound from about 64 query rows on).
//
// Item: 128 query rows (rows of [T * H] in order) of one sequence. The items' tiles of 64 cache rows,
// laid end to end, are cut into equal ranges, one per cluster of two CTAs, so that sequences of any
// lengths fill the GPU evenly. A cluster that has all tiles of an item writes its output; else
// it leaves (O, reference, sum) in the workspace and k_tree_merge joins them in a fixed order.
//
// Split in a cluster: O of 128 x 512 in fp32 is all of an SM's TMEM, so one CTA makes S = Q V^T and the
// softmax (Q in TMEM, four slots of S beside it) and the other one O += P V, with P in two parts of fp16. P goes
// over as it is made, 32 KiB a tile, in one direction only: no round trip is on the path of a tile. Both
// dequantize the tile's rows for themselves. Tensor work is 1,024 cycles a tile for the scores, 2,048 for the values.
// (Splitting the channels instead, each CTA with half of q, V and O, needs S summed over the two CTAs:
// 24 KiB a tile each way and a round trip, and took 2,850 cycles a tile, with P in one part. P in one part took
// 2,100 cycles a tile in this form, in two it takes 2,465.)
// 4 x 1,024 query rows over 32,784 rows each: 348 to 372 us (1.84 to 1.6 GHz: the power limit), bound by the value
// CTA: its tensor core works 83 % of a tile's cycles, and reads 1,536 wavefronts of operands a tile beside the
// dequantization's stores. 8 x 512 over 2,056: 51 us, 32 x 320 over 517: 45 us, bound by an item's start and end.
//
// A CTA (28 warps):
//  * warps 16-23 dequantize a tile's 64 rows to fp16 (exact) in 128-byte-swizzled 64-channel chunks,
//    the K-major B operand of S and the MN-major B operand of O; loads run a tile ahead;
//  * warp 24 issues the MMAs: S(t) with A = Q in TMEM, or O += P(t) V(t) with A = P in shared memory;
//  * warps 0-15 own TMEM lane quarter w % 4 (query rows); warps 0-7 work on the even tiles, 8-15 on
//    the odd ones. Scores: reference and sum in registers (lane = query row, 32 columns a thread);
//    the reference is handed from set to set. Values: P's arrival, O's rescaling, the output.
// Numerics: q as fp16 times a power of two per row (exact down to 2^-28 of the row's maximum), v exact
// in fp16, S and O in fp32. A row's logits are c S (log2 domain). The reference m, a value of S, moves only when a
// logit passes it by 2^8, to the maximum; p = 2^(c (S - m) + 7). The difference comes first: c S and c m rounded
// apart, a row's largest p could be anything once a logit has no bits left below 1 (from 2^24 on). c is cut off at
// 2^90 there, where it multiplies the least difference of two S (2^-34) to 2^56: one row has it all either way.
// A row's largest p is at least 2^7 and at most 2^15. p goes as two fp16, its upper 11 bits and the rest rounded
// to 11 bits: together off by at most 2^-21 of p, or by 2^-24, which is 2^-31 of the largest. One fp16 alone, 2^-11,
// shows where rows cancel, and breaks the library's bound on its attention (5e-3 in every value) where some rows
// are a hundred times louder. The sums are fp32.
// Every wait is bounded; on timeout a status bit is set and the kernel winds down.
#include <atomic>

#include "fp4kv_common.cuh"
#include "fp4kv_launch.h"
#include "fp4kv_quant.cuh"
#include "fp4kv_sm100.cuh"

namespace fp4kv {
namespace {

constexpr int kD = 512;
constexpr int kRows = 128;  // query rows of an item
constexpr int kTile = 64;   // cache rows of a tile
constexpr int kCols = kTile / 2;  // columns of S per softmax warp
constexpr int kSoftWarps = 16, kDeqWarps = 8, kMmaWarp = 24;
constexpr int kThreads = 32 * (kMmaWarp + 4);  // (whole warpgroups: registers move between them)
constexpr int kStages = 2;  // tiles of V
constexpr int kSlots = 4;   // tiles of S
constexpr int kPSlots = 2;  // tiles of P: tile m's in slot m & 1
// Tiles that are added up in TMEM at most. The tensor core's fp32 sums are cut off, not rounded: each of the 8
// steps of a tile loses half an ulp of O on average, always towards zero (2^-14 after 256 tiles; 2^-8 after 16,384).
// After kFlush tiles of an item O goes to the workspace, where it is added with rounding, and starts again from zero;
// a row's sum is kept in as many parts. Costs 3 % from 512 tiles on (661 against 643 us for 8,192 query rows over
// 32,832; 64 tiles instead of 256 cost 16 %); without it a prefix of 1,000,000 rows came out 0.4 to 0.8 % too small.
constexpr uint32_t kFlush = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMoveLog2 = 8.0f, kPLog2 = 7.0f;  // a reference moves past 2^8; p = 2^7 at it
constexpr float kMostC = 0x1p90f;  // (S stays below 2^37)

constexpr uint32_t kVChunk = kTile * 128;         // [64 rows][64 channels]
constexpr uint32_t kVBytes = 8 * kVChunk;         // 64 KiB
constexpr uint32_t kPHalf = kRows * 128;          // [16 groups of 8 query rows][high, low part][8][64 B] fp16
constexpr uint32_t kPBytes = 2 * kPHalf;          // two halves of 32 columns
constexpr uint32_t kOffV = 0;                     // (scores: first Q's way into TMEM)
constexpr uint32_t kOffP = kOffV + kStages * kVBytes;  // slots of P: as it is made, and as it arrives
constexpr uint32_t kOffBar = kOffP + kPSlots * kPBytes;
constexpr uint32_t kOffMisc = kOffBar + 320;
constexpr uint32_t kOffIter = kOffBar + 336;      // the cluster's range (a SegIter)
constexpr uint32_t kOffC = kOffBar + 448;         // scores: [128] power of two of the query rows
constexpr uint32_t kOffPair = kOffC + 512;        // scores: [4][128] exchange between a row's four threads
constexpr uint32_t kOffRef = kOffPair + 2048;     // scores: [2][128] reference after the last tile of either parity
constexpr uint32_t kOffFlushed = kOffRef + 1024;  // scores: [128] reference of what has been flushed
constexpr uint32_t kOffSum = kOffFlushed + 512;   // scores: [512] a thread's share of its row's sum, without the last tiles'
constexpr uint32_t kOffA = kOffSum + 2048;        // values: [2 slots][128] factors of O
constexpr uint32_t kOffML = kOffA + 1024;         // values: [2 slots][4][128] with an item's last tile: reference, sum, c, factor of what lies aside
constexpr uint32_t kSmem = kOffML + 4096;
static_assert(kSmem <= 232448, "shared memory");

// TMEM columns. Scores: Q [0, 256), S slots [256, 512). Values: O [0, 512).
constexpr uint32_t kColS = 256;

// Barriers. V's have two halves of 32 rows. Of S's slots: SFULL, SFREE (scores). Of P's: PXFULL, PREADY (values) and,
// for either half, PFREE (O has it, in both). SEG: the last product of an item is complete. A wait goes by parity, so
// nobody may wait for a use of a barrier before the use before it is known to be over.
enum { B_VFULL = 0, B_VFREE = 6, B_SFULL = 12, B_SFREE = 16, B_PFREE = 20, B_PXFULL = 24, B_PREADY = 26, B_REF = 32,
       B_QREADY = 34, B_SEG = 35, B_DONE = 36, B_COUNT = 37 };
static_assert(8 * B_COUNT <= 320, "barriers");

// ---------------------------------------------------------------------------------------
// cluster shared memory
// ---------------------------------------------------------------------------------------
FP4KV_DEV uint32_t map_peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
FP4KV_DEV void mbar_arrive_peer(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
FP4KV_DEV void st_peer_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
FP4KV_DEV bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
// Bounded waits by all lanes of a warp; the same value in every lane.
FP4KV_DEV bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait_timed(bar, parity));
}
FP4KV_DEV bool warp_wait_cluster(uint64_t* bar, uint32_t parity) {
  bool ok = mbar_try_wait_cluster(bar, parity);
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1; !ok; ++i) {
      ok = mbar_try_wait_cluster(bar, parity);
      if ((i & 255u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}
// To the other CTA's shared memory, completing on a barrier there: a copy (16-byte units) and a store.
FP4KV_DEV void bulk_peer(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "r"(src), "r"(bytes), "r"(bar) : "memory");
}
FP4KV_DEV void st_async_f32(uint32_t dst, float v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(dst), "f"(v), "r"(bar) : "memory");
}

FP4KV_DEV void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

FP4KV_DEV void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }

// One lane of a converged warp.
FP4KV_DEV uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r;
}
// The MMA and commit wrappers below are called by the whole warp; the lane with `go` issues. The
// operands stay warp-uniform that way: inside a branch of one lane each MMA took 100 cycles to issue.
// Descriptors go as their low word (address, leading offset) and a constant high one.
// D[tmem] (+)= A * B^T, fp16, A from TMEM, B from shared memory
template <uint32_t kBHigh>
FP4KV_DEV void umma_ts(uint32_t go, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, g;\n .reg .b64 bd;\n mov.b64 bd, {%2, %6};\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 g, %5, 0;\n"
      " @g tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %3, p;\n}"
      ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(go), "n"(kBHigh) : "memory");
}
// the same, A from shared memory
template <uint32_t kAHigh, uint32_t kBHigh>
FP4KV_DEV void umma_ss(uint32_t go, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, g;\n .reg .b64 ad, bd;\n mov.b64 ad, {%1, %6};\n mov.b64 bd, {%2, %7};\n setp.ne.b32 p, %4, 0;\n"
      " setp.ne.b32 g, %5, 0;\n @g tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %3, p;\n}"
      ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(go), "n"(kAHigh), "n"(kBHigh) : "memory");
}
// High words of the 128-byte and 64-byte swizzled layouts: 1024 bytes between 8-row groups (of P's, high and low
// parts alternate).
constexpr uint32_t kHigh128 = (1024u >> 4) | (1u << 14) | (2u << 29), kHigh64 = (1024u >> 4) | (1u << 14) | (4u << 29);
FP4KV_DEV void commit_if(uint32_t go, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred g;\n setp.ne.b32 g, %1, 0;\n"
      " @g tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
      ::"r"(smem_u32(bar)), "r"(go) : "memory");
}
// Arrive on the mbarrier at this offset in the CTAs of `mask`.
FP4KV_DEV void commit_to_if(uint32_t go, uint64_t* bar, uint16_t mask) {
  asm volatile(
      "{\n .reg .pred g;\n setp.ne.b32 g, %2, 0;\n"
      " @g tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}"
      ::"r"(smem_u32(bar)), "h"(mask), "r"(go) : "memory");
}
FP4KV_DEV float ex2(float x) {  // a few units in the last place; results below 2^-126 flushed to zero
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The two warps (column halves) of a lane quarter in one set.
FP4KV_DEV void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(2 + id) : "memory"); }
FP4KV_DEV bool pair_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n bar.red.or.pred po, %2, 64, pi;\n selp.u32 %0, 1, 0, po;\n}"
      : "=r"(r) : "r"(v ? 1u : 0u), "r"(2 + id) : "memory");
  return r != 0;
}
// The four warps of a lane quarter.
FP4KV_DEV void quad_sync(int q) { asm volatile("bar.sync %0, 128;" ::"r"(10 + q) : "memory"); }
// Registers move between warpgroups: 896 threads are launched with 72 each, the softmax warps keep
// theirs, the idle ones' go to the dequantizing ones (16 x 72 + 8 x 80 + 4 x 56 = 28 x 72 per lane).
template <int N>
FP4KV_DEV void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
FP4KV_DEV void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// ---------------------------------------------------------------------------------------
// what a sequence has to do
// ---------------------------------------------------------------------------------------
struct Seq {
  int nd;          // drafted tokens
  uint32_t pre;    // rows of the prefix (cap < 2^31)
  uint32_t n_sel;  // entries before the drafts: the prefix, or the selection
  uint32_t tiles, groups;
  // what the clusters share out: tiles, or whole items
  FP4KV_DEV uint32_t work(bool whole) const { return whole ? (tiles ? groups : 0) : tiles * groups; }
};
FP4KV_DEV Seq seq_of(const TreeAttnParams& p, int b) {
  Seq s;
  s.nd = p.n_draft ? max(0, min(p.n_draft[b], p.T)) : p.T;
  s.pre = static_cast<uint32_t>(max(int64_t(0), min(int64_t(p.prefix_lens[b]), p.cap)));
  s.n_sel = p.idx && s.pre > 0 ? p.top_k : s.pre;
  s.tiles = (s.n_sel + s.nd + kTile - 1) / kTile;
  s.groups = (static_cast<uint32_t>(s.nd) * p.H + kRows - 1) / kRows;
  return s;
}
// All tile counts fit 32 bits (the host refuses more): a 64-bit division is a call of 100 instructions.
// Clusters in use for `total` tiles of `items` items, whose tiles are `tiles` each (0: not all the same):
// at least min_tiles each. Where whole fractions of an item to a cluster cost no more than the parts
// that begin and end anywhere, they are taken: a cluster then has one segment, not two, and a segment costs
// about as much as 6 tiles (Q, the pipeline's start, the output). With fractions and without: 32 items of 33
// tiles 51.2 and 56.3 us, 16 of 63 50.6 and 54.3, 32 of 63 72.8 and 75.5, 8 of 313 83.6 and 85.3; where they are
// not taken, 16 of 200 100.3 and 98.0, 20 of 100 76.0 and 74.5, 30 of 150 133 and 123.
FP4KV_DEV uint32_t clusters_used(uint32_t total, uint32_t items, uint32_t tiles, uint32_t n_clusters, uint32_t min_tiles) {
  const uint32_t n = max(1u, min(n_clusters, total / min_tiles + (total % min_tiles != 0)));
  if (tiles == 0 || items > n) return n;
  const uint32_t k = n / items;  // clusters an item
  return (tiles + k - 1) / k <= total / n + 6 ? k * items : n;
}
// floor(total * i / used): where cluster i's range starts.
FP4KV_DEV uint32_t range_start(uint32_t total, uint32_t used, uint32_t i) {
  const uint32_t per = total / used;
  return per * i + (total - per * used) * i / used;
}
// The cluster of tile x: the largest i whose range starts at x or before.
FP4KV_DEV uint32_t cluster_of(uint32_t total, uint32_t used, uint32_t x) {
  uint32_t i = min(used - 1, static_cast<uint32_t>(static_cast<float>(x) / static_cast<float>(total) * static_cast<float>(used)));
  while (i > 0 && range_start(total, used, i) > x) --i;
  while (i + 1 < used && range_start(total, used, i + 1) <= x) ++i;
  return i;
}

// A cluster's range of tiles, segment by segment (a segment: consecutive tiles of one item).
struct alignas(16) SegIter {
  uint32_t off, rem;  // tiles of sequence b already passed; tiles still to do
  int b;
  bool ready;         // the segment below is still to be done
  uint32_t g, tile0, nt;
  Seq s;
  FP4KV_DEV void cut(bool whole) {
    if (whole) {
      g = off++;
      tile0 = 0;
      nt = s.tiles;
      --rem;
      return;
    }
    g = off / s.tiles;
    tile0 = off - g * s.tiles;
    nt = min(s.tiles - tile0, rem);
    off += nt;
    rem -= nt;
  }
  FP4KV_DEV bool next(const TreeAttnParams& p) {
    if (ready) {
      ready = false;
      return true;
    }
    if (rem == 0) return false;
    while (off >= s.work(p.whole)) {
      off -= s.work(p.whole);
      s = seq_of(p, ++b);
    }
    cut(p.whole);
    return true;
  }
};
static_assert(sizeof(SegIter) <= 448 - 336 && kOffIter % 16 == 0, "the range's place");

// One thread's share of a tile: chunks j and j + 4 of a row (64 channels each: 32 code bytes, 4 scales).
struct RawRow {
  uint32_t c[2][8];
  uint32_t s[2];
};
FP4KV_DEV void ld_nc_32b(uint32_t (&r)[8], const uint8_t* p, bool al32) {
  if (al32) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "l"(p));
  } else {
    const uint4 a = ld_nc_v4(p), b = ld_nc_v4(p + 16);
    r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w; r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
  }
}
// Four E4M3 scales, a NaN (all bits but the sign) as 1.875.
FP4KV_DEV uint32_t finite_scales(uint32_t s) {
  return s & ~((((s & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 1);
}
// A chunk's row in shared memory, by lane j = 0 .. 3 of the four that share a row: unit k of 16 bytes goes to
// position k ^ (row & 7) (the swizzle), and the lane writes its units in the order k ^ 2 j. That way a
// row's 128 code bytes are read by neighbouring lanes (one line per eight lanes; eight rows to eight lanes
// took four times the wavefronts), and eight lanes still write to distinct banks.
// at: the row's address, with (row & 7) ^ 2 j in its unit bits.
FP4KV_DEV void dequant_chunk(uint32_t at, uint32_t j, const uint32_t (&c)[8], uint32_t s) {
  uint32_t v[8], w[8], sc[4];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = j & 1 ? c[k ^ 2] : c[k];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = j & 2 ? v[k ^ 4] : v[k];
  s = __byte_perm(s, 0, 0x3210u ^ (0x1111u * j));
  const uint32_t s01 = e4m3x2_to_f16x2(static_cast<uint16_t>(s & 0xffffu)), s23 = e4m3x2_to_f16x2(static_cast<uint16_t>(s >> 16));
  sc[0] = __byte_perm(s01, 0, 0x1010);
  sc[1] = __byte_perm(s01, 0, 0x3232);
  sc[2] = __byte_perm(s23, 0, 0x1010);
  sc[3] = __byte_perm(s23, 0, 0x3232);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t h[4];
    e2m1x8_to_f16(w[k], h);
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                 ::"r"(at ^ (16u * k)), "r"(hmul2_f16(h[0], sc[k >> 1])), "r"(hmul2_f16(h[1], sc[k >> 1])),
                   "r"(hmul2_f16(h[2], sc[k >> 1])), "r"(hmul2_f16(h[3], sc[k >> 1])) : "memory");
  }
}

// kCols of this thread's O (its TMEM lane) plus a times what the workspace has of them (first: nothing yet): to there,
// or with kBack to TMEM. 16 columns at a time: with 32 the loop's registers cost the kernel 200 bytes of spills.
template <int kCols, bool kBack>
FP4KV_DEV void flush_o(uint32_t addr, float4* w, float a, bool first, bool live) {
#pragma unroll 1
  for (int c = 0; c < kCols / 16; ++c) {
    uint32_t r[16];
    tmem_ld16(addr + 16 * c, r);
    tmem_ld_wait();
    if (live) {
      if (!first) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 v = __ldcg(w + k * kRows);
          r[4 * k] = __float_as_uint(fmaf(v.x, a, __uint_as_float(r[4 * k])));
          r[4 * k + 1] = __float_as_uint(fmaf(v.y, a, __uint_as_float(r[4 * k + 1])));
          r[4 * k + 2] = __float_as_uint(fmaf(v.z, a, __uint_as_float(r[4 * k + 2])));
          r[4 * k + 3] = __float_as_uint(fmaf(v.w, a, __uint_as_float(r[4 * k + 3])));
        }
      }
      if (!kBack) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          __stcg(w + k * kRows, make_float4(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]),
                                            __uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3])));
      }
    }
    w += 4 * kRows;
    __syncwarp();
    if (kBack) tmem_st16(addr + 16 * c, r);
  }
  if (kBack) tmem_st_wait();
}

FP4KV_DEV float lse_of(float ref, float l, float c) {
  return l == 0.0f ? -INFINITY : fmaf(ref, c, -kPLog2) * kLn2 + logf(l);
}

// this thread's TMEM lane, 256 of its O columns, times a
FP4KV_DEV void rescale_o(uint32_t addr, float a) {
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {
    uint32_t r[32];
    tmem_ld32(addr + 32 * c, r);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * a);
    tmem_st32(addr + 32 * c, r);
  }
  tmem_st_wait();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) k_tree_attn(const TreeAttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  int* sLow = reinterpret_cast<int*>(smem + kOffC);
  float* sPair = reinterpret_cast<float*>(smem + kOffPair);
  float* sRef = reinterpret_cast<float*>(smem + kOffRef);
  float* sFlushed = reinterpret_cast<float*>(smem + kOffFlushed);
  float* sSum = reinterpret_cast<float*>(smem + kOffSum);
  const float* sA = reinterpret_cast<const float*>(smem + kOffA);
  const float* sML = reinterpret_cast<const float*>(smem + kOffML);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile uint32_t* s_abort = s_tmem + 1;
  SegIter* s_it = reinterpret_cast<SegIter*>(smem + kOffIter);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool values = cluster_ctarank() != 0;  // the CTA that makes O
  const uint32_t cl = blockIdx.x >> 1;
  // k_tree_merge waits for this grid before it reads anything; with whole items it isn't launched, and the kernel
  // that then comes next may read what this one writes before its own wait (sparse_attn_decode its query)
  if (!p.whole) griddep_launch_dependents();
  griddep_wait();

  // the smem alignment that the swizzled operands need (the same in both CTAs of a launch)
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) atomicOr(p.status, 2u);
    return;
  }
  // ---- this cluster's range of tiles, and its first segment ----
  if (warp == kMmaWarp) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  if (warp == 0) {
    Seq mine{};  // of sequence lane, then of the 32 at hand
    if (lane < p.B) mine = seq_of(p, lane);
    uint32_t total = mine.work(p.whole), items = mine.groups;
    uint32_t most = total ? mine.tiles : 0, least = total ? mine.tiles : 0xffffffffu;
#pragma unroll 1
    for (int b = lane + 32; b < p.B; b += 32) {
      const Seq s = seq_of(p, b);
      total += s.work(p.whole);
      items += s.groups;
      if (s.work(p.whole)) {
        most = max(most, s.tiles);
        least = min(least, s.tiles);
      }
    }
    total = __reduce_add_sync(0xffffffffu, total);
    items = __reduce_add_sync(0xffffffffu, items);
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    const uint32_t used = p.whole ? max(1u, min(uint32_t(p.n_clusters), total))
                                  : clusters_used(total, items, most == least ? most : 0, p.n_clusters, p.min_tiles);
    const uint32_t x0 = cl < used ? range_start(total, used, cl) : total;
    const uint32_t x1 = cl < used ? range_start(total, used, cl + 1) : total;
    // where x0 lies, and (cluster 0) each sequence's first tile for the merge
    uint32_t at = 0;
    bool found = x1 <= x0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B && (!found || cl == 0); b0 += 32) {
      const int b = b0 + lane;
      if (b0 > 0) {
        mine = Seq{};
        if (b < p.B) mine = seq_of(p, b);
      }
      const uint32_t n = mine.work(p.whole);
      uint32_t incl = n;
#pragma unroll 1
      for (int o = 1; o < 32 && o < p.B; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (cl == 0 && !values && b < p.B) p.first_tile[b] = at + incl - n;
      const uint32_t hit = __ballot_sync(0xffffffffu, at + incl > x0);
      if (!found && hit) {
        if (lane == __ffs(hit) - 1) {
          SegIter first;
          first.b = b;
          first.off = x0 - (at + incl - n);
          first.rem = x1 - x0;
          first.s = mine;
          first.cut(p.whole);
          first.ready = true;
          *s_it = first;
        }
        found = true;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      if (x1 <= x0) s_it->ready = false;
      *s_abort = 0;
      if (cl == 0 && !values) {
        p.first_tile[p.B] = total;
        p.first_tile[p.B + 1] = used;
      }
    }
  }
  if (tid == 32) {
    for (int i = 0; i < 2 * kStages; ++i) {
      mbar_init(&bars[B_VFULL + i], kDeqWarps / 2);
      mbar_init(&bars[B_VFREE + i], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bars[B_SFULL + i], 1);
      mbar_init(&bars[B_SFREE + i], kSoftWarps / 2);
    }
    for (int i = 0; i < 2 * kPSlots; ++i) mbar_init(&bars[B_PFREE + i], 1);
    for (int i = 0; i < kPSlots; ++i) {
      mbar_init(&bars[B_PXFULL + i], 1);
      mbar_init(&bars[B_PREADY + i], kSoftWarps / 2);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&bars[B_REF + i], 4);
    mbar_init(&bars[B_QREADY], kSoftWarps);
    mbar_init(&bars[B_SEG], 1);
    mbar_init(&bars[B_DONE], 1);
    fence_mbar_init();
  }
  __syncthreads();
  SegIter it = *s_it;
  if (!it.ready) {  // nothing to do, for both CTAs of the cluster
    if (warp == kMmaWarp) tmem_dealloc(*s_tmem, 512);
    return;
  }
  cluster_arrive_relaxed();  // (the barriers' initialisation has been released by its own fence)
  // Each role waits where it first needs the other CTA's barriers or TMEM; its first loads come before.
  uint32_t tmem = 0;
  auto join = [&]() {
    cluster_wait();
    tc_fence_after();
    tmem = *s_tmem;
  };
  uint32_t n = 0;    // tiles so far, over all segments: slot n % 4
  uint32_t seg = 0;  // segments so far

  auto aborted = [&]() { return __any_sync(0xffffffffu, *s_abort != 0) != 0; };
  // (in both CTAs: neither may leave while the other's copies may still be on their way)
  auto give_up = [&]() {
    if (lane == 0) {
      atomicOr(p.status, kFlagWaitTimeout);
      *s_abort = 1;
      st_peer_u32(map_peer(smem_u32(smem) + kOffMisc + 4, values ? 0 : 1), 1);
    }
  };

  uint32_t st = 0, sph = 0;  // the next tile's stage, and the parity of that stage's use
  auto next_stage = [&]() {
    if (++st == kStages) {
      st = 0;
      sph ^= 1;
    }
  };

  if (warp >= kSoftWarps && warp < kMmaWarp) {
    // ------------------------------ load and dequantize ------------------------------
    more_registers<80>();
    // Four lanes share a row, two chunks each.
    const int row = 8 * (warp - kSoftWarps) + (lane >> 2), half = (warp - kSoftWarps) >> 2;
    const uint32_t j = lane & 3;
    const uint32_t unit0 = smem_u32(smem) + kOffV + j * kVChunk + row * 128 + (((row & 7) ^ (2 * j)) << 4);
    const bool al32 = (reinterpret_cast<uintptr_t>(p.packed) & 31) == 0;
    bool ok = true;
    while (it.next(p)) {
      const Seq& s = it.s;
      // a drafted row that no token sees counts as absent
      uint64_t seen = 0;
      {
        const uint64_t* tm = p.tree_mask + int64_t(it.b) * p.T;
        if (lane < s.nd) seen = tm[lane];
        if (lane + 32 < s.nd) seen |= tm[lane + 32];
      }
      const int32_t* idx = p.idx ? p.idx + int64_t(it.b) * p.top_k : nullptr;
      const uint8_t* packed = p.packed + int64_t(it.b) * p.cap * (kD / 2) + 32 * j;
      const uint8_t* scales = p.scales + int64_t(it.b) * p.cap * (kD / kGroup) + 4 * j;
      // This thread's row of tile i: the entry, which is turned into a position only when it is used (it may
      // still be on its way from the selection).
      auto entry = [&](uint32_t i) -> int32_t {
        const uint32_t e = (it.tile0 + i) * kTile + row;
        return i < it.nt && idx && e < s.n_sel ? idx[e] : static_cast<int32_t>(e);
      };
      // Where this thread's row of tile i lies (-1: absent), and a chunk of it.
      auto place = [&](uint32_t i, int32_t ent) -> int64_t {
        const uint32_t e = (it.tile0 + i) * kTile + row;
        int64_t pos = static_cast<uint32_t>(ent);
        bool there = i < it.nt;
        if (e < s.n_sel) {
          there = there && static_cast<uint32_t>(ent) < s.pre;
        } else {
          const uint32_t d = e - s.n_sel;
          pos = int64_t(s.pre) + d;
          there = there && d < uint32_t(s.nd) && ((seen >> d) & 1) && pos < p.cap;
        }
        return there ? pos : -1;
      };
      auto load = [&](uint32_t (&c)[8], uint32_t& sc, int64_t pos, int k) {
        if (pos >= 0) {
          ld_nc_32b(c, packed + pos * (kD / 2) + 128 * k, al32);
          sc = *reinterpret_cast<const uint32_t*>(scales + pos * (kD / kGroup) + 16 * k);
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u) c[u] = 0;
          sc = 0;
        }
      };
      const int32_t e0 = entry(0);
      int32_t ent = entry(1);
      seen = uint64_t(__reduce_or_sync(0xffffffffu, uint32_t(seen))) |
             (uint64_t(__reduce_or_sync(0xffffffffu, uint32_t(seen >> 32))) << 32);
      // The next tile's, loaded over the one that has just been converted. (Two tiles ahead
      // in two buffers, the loop written out twice, took 302 against 280 us for 4 x 1,024 query rows over 32,784:
      // 3 % more instructions, 53 times the spill stores, and more waiting for instructions. Written out once more,
      // for either kind of CTA: 368, with 6 times that waiting. A loop over the two chunks: 348.)
      RawRow r;
      {
        const int64_t pos = place(0, e0);
        load(r.c[0], r.s[0], pos, 0);
        load(r.c[1], r.s[1], pos, 1);
      }
      if (seg == 0) join();
      // (Q comes through the stages, but for a first item of up to 64 rows: then this wait comes at the end)
      const bool q_apart = seg == 0 && s.nd * p.H - static_cast<int>(it.g) * kRows <= 64;
      if (!values && !q_apart) ok = ok && !aborted() && warp_wait(&bars[B_QREADY], seg & 1);
      for (uint32_t i = 0; ok && i < it.nt; ++i) {
        // (eight warps that wait most of the time: sparing polls leave shared memory to the others)
        ok = __all_sync(0xffffffffu, mbar_wait_sleepy(&bars[B_VFREE + 2 * st + half], sph ^ 1, 32));
        if (!ok) break;
        const uint32_t at = unit0 + st * kVBytes;
        // A row with a NaN scale makes its logits NaN, so p is NaN for those who see it and 0 for the others; as a
        // value it is read as finite, since 0 * NaN would reach the others too.
        if (values) {
          r.s[0] = finite_scales(r.s[0]);
          r.s[1] = finite_scales(r.s[1]);
        }
        dequant_chunk(at, j, r.c[0], r.s[0]);
        dequant_chunk(at + 4 * kVChunk, j, r.c[1], r.s[1]);
        const int64_t pos = place(i + 1, ent);
        load(r.c[0], r.s[0], pos, 0);
        load(r.c[1], r.s[1], pos, 1);
        ent = entry(i + 2);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_VFULL + 2 * st + half]);
        next_stage();
      }
      if (!values && q_apart) ok = ok && warp_wait(&bars[B_QREADY], seg & 1);
      if (!ok) give_up();
      ++seg;
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------ MMA issue (one warp; its warpgroup's others idle) ------------------------------
    fewer_registers<56>();
    join();
    if (warp == kMmaWarp) {
      const uint32_t go = elect_lane();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      bool ok = true;
      while (ok && it.next(p)) {
        if (!values) {
          constexpr uint32_t kIdesc = umma_idesc(0u, kRows, kTile, 0u, 0u);
          const uint32_t dv = static_cast<uint32_t>(sw128_kmajor_desc(smem_u32(smem + kOffV)));
          ok = warp_wait(&bars[B_QREADY], seg & 1);
          for (uint32_t i = 0; ok && i < it.nt; ++i) {
            const uint32_t m = n + i, sl = m & (kSlots - 1);
            ok = warp_wait(&bars[B_SFREE + sl], ((m >> 2) & 1) ^ 1) && warp_wait(&bars[B_VFULL + 2 * st], sph) &&
                 warp_wait(&bars[B_VFULL + 2 * st + 1], sph);
            if (!ok) break;
            tc_fence_after();
            const uint32_t b0 = dv + ((st * kVBytes) >> 4);
            const uint32_t d = tm + kColS + kTile * sl;
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_ts<kHigh128>(go, d, tm + 32 * c + 8 * k, b0 + ((c * kVChunk) >> 4) + 2 * k, kIdesc, (c | k) != 0);
            commit_if(go, &bars[B_SFULL + sl]);
            commit_if(go, &bars[B_VFREE + 2 * st]);
            commit_if(go, &bars[B_VFREE + 2 * st + 1]);
            if (i + 1 == it.nt) commit_if(go, &bars[B_SEG]);
            next_stage();
          }
        } else {
          constexpr uint32_t kIdesc = umma_idesc(0u, kRows, 256, 0u, 1u);
          const uint32_t dv = static_cast<uint32_t>(sw128_mnmajor_desc(smem_u32(smem + kOffV), kVChunk));
          const uint32_t dp = static_cast<uint32_t>(sw64_kmajor_desc(smem_u32(smem + kOffP)));
          for (uint32_t i = 0; ok && i < it.nt; ++i) {
            const uint32_t m = n + i, ps = m & 1;
            ok = warp_wait(&bars[B_PREADY + ps], (m >> 1) & 1);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {  // 32 cache rows: two steps of 16, two halves of the channels
              ok = ok && warp_wait(&bars[B_VFULL + 2 * st + hf], sph);
              if (ok) {
                tc_fence_after();
                const uint32_t a0 = dp + ((ps * kPBytes + hf * kPHalf) >> 4);
                const uint32_t b0 = dv + ((st * kVBytes + hf * 4096) >> 4);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                  for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int part = 0; part < 2; ++part)
                      umma_ss<kHigh64, kHigh128>(go, tm + 256 * c, a0 + 2 * k + 32 * part, b0 + ((2048 * k + 4 * c * kVChunk) >> 4), kIdesc,
                                                 (i & (kFlush - 1)) != 0 || (hf | k | part) != 0);
                commit_if(go, &bars[B_VFREE + 2 * st + hf]);
                // (an item's last slot is given back after its reference and sum have been read)
                commit_to_if(go, &bars[B_PFREE + 2 * ps + hf], i + 1 < it.nt ? 3 : 2);
              }
            }
            if (ok && i + 1 == it.nt) commit_if(go, &bars[B_SEG]);
            next_stage();
          }
        }
        n += it.nt;
        ++seg;
      }
      if (!ok) give_up();
      commit_if(go, &bars[B_DONE]);  // nothing is in flight when TMEM is released
      __syncwarp();
      if (!warp_wait(&bars[B_DONE], 0)) give_up();
    }
  } else {
    more_registers<72>();  // (as launched: said so, the allocator spills less)
    const int q = warp & 3, h4 = warp >> 2, h = h4 & 1;
    const uint32_t set = warp >> 3;
    const int pair = 4 * static_cast<int>(set) + q;
    const int R = 32 * q + lane;  // query row of the item
    uint32_t lane_addr = 0;
    const uint32_t peer_smem = map_peer(smem_u32(smem), values ? 0 : 1);
    while (it.next(p)) {
      const Seq& s = it.s;
      const int live_rows = s.nd * p.H - static_cast<int>(it.g) * kRows;  // of this item (and behind)
      const int64_t row0 = int64_t(it.b) * p.T * p.H + int64_t(it.g) * kRows;
      const uint32_t last = n + it.nt - 1;
      const uint32_t i0 = (n ^ set) & 1;  // this set's first tile
      bool ok = !aborted();
      if (!values) {
        // ------------------------------ scores and softmax ------------------------------
        // ---- Q: through shared memory into TMEM, bf16 -> fp16 times a power of two ----
        // (The last item's products are complete: its stages and Q's place are free. Before the first item the
        // slots of P are too, and hold 64 rows: then V need not wait.) Rows behind the last are not staged:
        // what TMEM has in their place stays in their rows of S, which count as masked.
        const uint32_t q_at = smem_u32(smem) + (seg == 0 && live_rows <= 64 ? kOffP : kOffV);
        const int rows = min(live_rows, kRows);
#pragma unroll 1
        for (int r = warp; r < rows; r += kSoftWarps) {
          const uint16_t* src = p.q + (row0 + r) * kD + 8 * lane;
          const uint32_t dst = q_at + r * 1024 + ((lane ^ (r & 7)) << 4);
          cp_async_16(dst, src);
          cp_async_16(dst + 512, src + kD / 2);
        }
        uint64_t rmask = 0;  // the drafts that this row's token sees
        if (R < live_rows) {
          rmask = p.tree_mask[int64_t(it.b) * p.T + (it.g * kRows + R) / uint32_t(p.H)];
          const int64_t nv = min(int64_t(s.nd), p.cap - int64_t(s.pre));
          if (nv < 64) rmask &= (uint64_t(1) << nv) - 1;
        }
        if (seg == 0) {
          join();
          lane_addr = tmem + (uint32_t(32 * q) << 16);
        }
        cp_async_wait_all();
#pragma unroll 1
        for (int r = warp; r < rows; r += kSoftWarps) {  // a row's maximum (each lane of what it has copied itself)
          const uint32_t at = q_at + r * 1024 + ((lane ^ (r & 7)) << 4);
          const uint4 v0 = lds_v4(at), v1 = lds_v4(at + 512);
          uint32_t m2 = __vmaxu2(__vmaxu2(v0.x & 0x7fff7fffu, v0.y & 0x7fff7fffu), __vmaxu2(v0.z & 0x7fff7fffu, v0.w & 0x7fff7fffu));
          m2 = __vmaxu2(m2, __vmaxu2(v1.x & 0x7fff7fffu, v1.y & 0x7fff7fffu));
          m2 = __vmaxu2(m2, __vmaxu2(v1.z & 0x7fff7fffu, v1.w & 0x7fff7fffu));
          const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
          // The power of two that brings the row's maximum into [2^14, 2^15), whose fp16 exponent is 29:
          // an exponent field x of bf16 becomes x - low (values of field low or less, below 2^-28 of the
          // maximum, come out wrong by up to 2^-29 of it).
          if (lane == 0) sLow[r] = max(int(m >> 7), 29) - 29;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory");
        const int low = R < rows ? sLow[R] : 0;
        {
          const uint32_t low2 = static_cast<uint32_t>(low) * 0x00800080u;
          // (a negative scale goes into q's sign: the factor of the logits is positive)
          const uint32_t flip = p.sm_scale < 0.0f ? 0x80008000u : 0u;
          // (an infinity has no fp16 here, and no softmax: with it, or NaN, in the row all of q is NaN)
          const uint32_t nan2 = low == 255 - 29 ? 0x7fff7fffu : 0u;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 f = lds_v4(q_at + R % (q_at == smem_u32(smem) + kOffP ? 64 : kRows) * 1024 + (((16 * h4 + 4 * c + k) ^ (R & 7)) << 4));
              w[4 * k] = f.x; w[4 * k + 1] = f.y; w[4 * k + 2] = f.z; w[4 * k + 3] = f.w;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)  // (field and mantissa three bits up, the sign beside them)
              w[k] = ((__vmaxu2(w[k] & 0x7fff7fffu, low2) - low2) << 3) | ((w[k] ^ flip) & 0x80008000u) | nan2;
            tmem_st16(lane_addr + 64 * h4 + 16 * c, w);
          }
        }
        tmem_st_wait();
        // q = fp16 * 2^(low - 112)
        const int up = low - 112;
        const float c = fminf(fmaxf(fabsf(p.sm_scale) * __uint_as_float(uint32_t(127 + up / 2) << 23) *
                                        __uint_as_float(uint32_t(127 + (up - up / 2)) << 23) * kLog2e,
                                    2e-38f),       // (above zero: a masked -inf stays -inf)
                              3.4028235e38f);      // (finite: times a reference of 0 it is 0)
        const float cc = fminf(c, kMostC);
        // the same bytes are written by the dequantizing warps next and read by the tensor cores
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_QREADY]);

        const int32_t* idx = p.idx ? p.idx + int64_t(it.b) * p.top_k : nullptr;
        auto entry_ok = [&](uint32_t i) -> bool {  // entry 32 h + lane of tile i lies in the prefix
          const uint32_t e = (it.tile0 + i) * kTile + kCols * h + lane;
          if (i >= it.nt || e >= s.n_sel) return false;
          return !idx || static_cast<uint32_t>(idx[e]) < s.pre;
        };
        bool e_ok = entry_ok(i0);
        float ref = -INFINITY;  // the reference that l2 is relative to
        uint64_t l2 = 0;        // the row's sum over even and odd columns, of at most kFlush tiles
        sSum[tid] = 0.0f;       // and over the tiles before
        if (i0 == 0 && h == 0) sFlushed[R] = -INFINITY;  // the reference of what the workspace has of O
        const uint64_t c2 = pack2(cc, cc);
        // a wait that ran out ends the loop of both warps of a row at the next vote
        bool dead = !ok;
        for (uint32_t i = i0; i < it.nt; i += 2) {
          const uint32_t m = n + i, sl = m & (kSlots - 1), ph = (m >> 2) & 1;
          uint32_t vis = __ballot_sync(0xffffffffu, e_ok);
          e_ok = entry_ok(i + 2);
          const uint32_t e0 = (it.tile0 + i) * kTile + kCols * h;
          if (e0 + kCols > s.n_sel)  // drafts among the columns
            vis |= e0 >= s.n_sel ? (e0 - s.n_sel < 64 ? uint32_t(rmask >> (e0 - s.n_sel)) : 0u) : uint32_t(rmask << (s.n_sel - e0));
          if (R >= live_rows) vis = 0;
          dead = dead || !warp_wait(&bars[B_SFULL + sl], ph);
          tc_fence_after();
          uint32_t r[32];
          tmem_ld32(lane_addr + kColS + kTile * sl + kCols * h, r);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_SFREE + sl]);
          if (!__all_sync(0xffffffffu, vis == 0xffffffffu)) {
#pragma unroll
            for (int k = 0; k < 32; ++k) r[k] = (vis >> k) & 1 ? r[k] : 0xff800000u;
          }
          float mx = __uint_as_float(r[0]);
#pragma unroll
          for (int k = 1; k < 32; ++k) mx = fmaxf(mx, __uint_as_float(r[k]));
          // the reference after the tile before, from the other set
          float old = -INFINITY;
          if (i > 0) {
            dead = dead || !warp_wait(&bars[B_REF + (set ^ 1)], ((m - 1) >> 1) & 1);
            old = sRef[128 * (set ^ 1) + R];
          }
          float to = old, a = 1.0f;
          const bool moves = pair_any(pair, (mx - old) * cc > kMoveLog2 || dead);
          if (moves) {  // a reference of these 32 rows moves
            if (pair_any(pair, dead)) {
              dead = true;
              break;
            }
            sPair[128 * (2 * set + h) + R] = mx;
            pair_sync(pair);
            mx = fmaxf(mx, sPair[128 * (2 * set + (h ^ 1)) + R]);
            if ((mx - old) * cc > kMoveLog2) {
              to = mx;
              if (i > 0) a = ex2((old - to) * cc);  // (O starts with the first tile; no reference so far: 0)
            }
          }
          if (h == 0) {
            sRef[128 * set + R] = to;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_REF + set]);
          }
          if (to != ref) {
            const float f = ex2((ref - to) * cc);
            l2 = fma2(l2, pack2(f, f), 0);
            sSum[tid] *= f;
            ref = to;
          }
          if (i > 1 && (i & (kFlush - 2)) == 0) {  // (either set's first tile of the next kFlush)
            float l0, l1;
            unpack2(l2, l0, l1);
            sSum[tid] += l0 + l1;
            l2 = 0;
            if ((i & 1) == 0 && h == 0) {  // O goes to the workspace: the factor is that of what lies there
              a = sFlushed[R] == -INFINITY ? 0.0f : ex2((sFlushed[R] - old) * cc);
              sFlushed[R] = old;
            }
          }
          const float base = ref == -INFINITY ? 0.0f : -ref;
          const uint64_t base2 = pack2(base, base), k2 = pack2(kPLog2, kPLog2), kMinus1 = pack2(-1.0f, -1.0f);
#pragma unroll
          for (int u = 0; u < 4; ++u) {  // eight columns: their high parts, then their low parts, in the scores' place
            uint32_t w[4], v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float z0, z1;
              unpack2(fma2(add2(pack2(__uint_as_float(r[8 * u + 2 * k]), __uint_as_float(r[8 * u + 2 * k + 1])), base2), c2, k2), z0, z1);
              const float e0 = ex2(z0), e1 = ex2(z1);
              l2 = add2(l2, pack2(e0, e1));
              // the high part's 11 bits by truncation, so that the rest is exact
              const float t0 = __uint_as_float(__float_as_uint(e0) & 0xffffe000u), t1 = __uint_as_float(__float_as_uint(e1) & 0xffffe000u);
              w[k] = pack_f16x2(t0, t1);
              float d0, d1;
              unpack2(fma2(pack2(t0, t1), kMinus1, pack2(e0, e1)), d0, d1);
              v[k] = pack_f16x2(d0, d1);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              r[8 * u + k] = w[k];
              r[8 * u + 4 + k] = v[k];
            }
          }
          // (the slot of this set's tiles)
          dead = dead || !warp_wait_cluster(&bars[B_PFREE + 2 * set + h], ((m >> 1) & 1) ^ 1);
          const uint32_t px_bar = peer_smem + kOffBar + 8 * (B_PXFULL + set);
          if (h == 0) st_async_f32(peer_smem + kOffA + 4 * (128 * set + R), a, px_bar);
          const uint32_t pw = kOffP + set * kPBytes + h * kPHalf + q * (kPHalf / 4);  // this warp's 4 KiB
          uint8_t* prow = smem + pw + (lane >> 3) * 1024 + (lane & 7) * 64;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint8_t* at = prow + ((u ^ ((lane >> 1) & 3)) << 4);
            *reinterpret_cast<uint4*>(at) = make_uint4(r[8 * u], r[8 * u + 1], r[8 * u + 2], r[8 * u + 3]);
            *reinterpret_cast<uint4*>(at + 512) = make_uint4(r[8 * u + 4], r[8 * u + 5], r[8 * u + 6], r[8 * u + 7]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) bulk_peer(peer_smem + pw, smem_u32(smem) + pw, kPHalf / 4, px_bar);
        }
        ok = !dead;
        // the row's sum over its four threads; reference and sum go with the last tile's P
        quad_sync(q);
        const float fin = sRef[128 * (last & 1) + R];
        float l0, l1;
        unpack2(l2, l0, l1);
        float l = sSum[tid] + (l0 + l1);
        if (l > 0.0f) l *= ex2((ref - fin) * cc);
        if (h4 != 0) sPair[128 * h4 + R] = l;
        quad_sync(q);
        const uint32_t ml = peer_smem + kOffML + 4 * (512 * (last & 1) + R), ml_bar = peer_smem + kOffBar + 8 * (B_PXFULL + (last & 1));
        if (h4 == 0) {
          l += sPair[128 + R] + sPair[256 + R] + sPair[384 + R];
          st_async_f32(ml, fin, ml_bar);
          st_async_f32(ml + 512, l, ml_bar);
          st_async_f32(ml + 1024, c, ml_bar);
        }
        if (i0 == 0 && h == 0)  // the set that flushes
          st_async_f32(ml + 1536, sFlushed[R] == -INFINITY ? 0.0f : ex2((sFlushed[R] - fin) * cc), ml_bar);
        // the last product is complete: the stages may take the next item's Q, and Q's place too
        if (ok) ok = warp_wait(&bars[B_SEG], seg & 1);
        quad_sync(q);  // (the sums have been read)
      } else {
        // ------------------------------ O: arrivals, rescaling ------------------------------
        if (seg == 0) {
          join();
          lane_addr = tmem + (uint32_t(32 * q) << 16);
        }
        const bool arms = h == 0 && q == 0 && lane == 0;
        // this thread's row in the workspace (a whole item's slot is free: the one that another would begin in)
        auto part = [&]() { return reinterpret_cast<float4*>(p.part_o) + int64_t(2 * cl + (it.tile0 == 0 ? 1 : 0)) * (kD / 4) * kRows + R; };
        for (uint32_t i = i0; ok && i < it.nt; i += 2) {
          const uint32_t m = n + i;
          if (arms) mbar_arrive_expect_tx(&bars[B_PXFULL + set], kPBytes + 512 + (i + 1 == it.nt ? 2048 : 0));
          ok = warp_wait_cluster(&bars[B_PXFULL + set], (m >> 1) & 1);
          const float a = sA[128 * set + R];
          const bool flush = i > 0 && (i & (kFlush - 1)) == 0;
          if (flush || __any_sync(0xffffffffu, a != 1.0f)) {  // O(m - 1) is complete, O(m) waits for this warp
            ok = ok && warp_wait(&bars[B_PFREE + 2 * (set ^ 1) + 1], ((m - 1) >> 1) & 1);
            tc_fence_after();
            if (flush)
              flush_o<256, false>(lane_addr + 256 * h, part() + 64 * h * kRows, a, i == kFlush, R < live_rows);
            else
              rescale_o(lane_addr + 256 * h, a);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_PREADY + set]);
        }
        if (ok) ok = warp_wait(&bars[B_SEG], seg & 1);
        // ------------------------------ out ------------------------------
        const uint32_t ps = last & 1;
        if (ok) ok = warp_wait_cluster(&bars[B_PXFULL + ps], (last >> 1) & 1);
        tc_fence_after();
        const float ref = sML[512 * ps + R], l = sML[512 * ps + 128 + R], c = sML[512 * ps + 256 + R];
        const bool whole = it.tile0 == 0 && it.nt == s.tiles;
        if (it.nt > kFlush) {
          asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory");  // (what others have flushed)
          flush_o<128, true>(lane_addr + 128 * h4, part() + 32 * h4 * kRows, sML[512 * ps + 384 + R], false, R < live_rows);
        }
        const bool live = R < live_rows;
        const int slot = 2 * cl + (it.tile0 == 0 ? 1 : 0);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // (NaN stays NaN)
        const bool al32 = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
          const int ch = 128 * h4 + 32 * u;
          uint32_t r[32];
          tmem_ld32(lane_addr + ch, r);
          tmem_ld_wait();
          if (live && whole) {
            uint16_t* dst = p.out + (row0 + R) * kD + ch;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t w[8];
#pragma unroll
              for (int v = 0; v < 8; ++v)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                    : "=r"(w[v])
                    : "f"(__uint_as_float(r[16 * k + 2 * v + 1]) * inv), "f"(__uint_as_float(r[16 * k + 2 * v]) * inv));
              if (al32) {
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 16 * k), "r"(w[0]), "r"(w[1]),
                             "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
              } else {
                reinterpret_cast<uint4*>(dst + 16 * k)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(dst + 16 * k)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          } else if (live) {  // [slot][128 fours of channels][128 rows][4]: a warp's stores are contiguous
            float4* dst = reinterpret_cast<float4*>(p.part_o) + (int64_t(slot) * (kD / 4) + ch / 4) * kRows + R;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              __stcg(dst + kRows * k, make_float4(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]),
                                                  __uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3])));
          }
          __syncwarp();
        }
        if (live && h4 == 0) {
          if (!whole)
            __stcg(reinterpret_cast<float4*>(p.part_ml) + slot * kRows + R, make_float4(ref, l, c, 0.0f));
          else if (p.lse)
            p.lse[row0 + R] = lse_of(ref, l, c);
        }
        tc_fence_before();
        // every warp has read O, the reference and the sum: the next item may start, the slot is free
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory");
        if (tid < 2) mbar_arrive_peer(peer_smem + kOffBar + 8 * (B_PFREE + 2 * ps + tid));
      }
      if (!ok) give_up();
      n += it.nt;
      ++seg;
      __syncwarp();
    }
  }
  tc_fence_before();
  cluster_sync_all();  // (no arrival or store is on its way to a CTA that has left)
  // In a range that ran to its end every copy of P has been waited for. After a wait that ran out nobody may have: the
  // last ones, sent before the barrier, get 1 ms (they take microseconds) before either end's shared memory goes.
  if (*s_abort != 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000) __nanosleep(1000);
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of items that several clusters worked on: o = sum_i 2^(c (m_i - M)) O_i / sum_i 2^(c (m_i - M)) l_i.
// A block takes 32 query rows and 128 channels: lanes along the rows as the parts lie, then through shared
// memory to lanes along the channels.
constexpr int kMergeCh = 128;
__global__ void __launch_bounds__(256) k_tree_merge(const TreeAttnParams p) {
  griddep_wait();
  __shared__ float tile[32][kMergeCh + 1];
  const int blocks = (p.T * p.H + 31) / 32;
  const int b = blockIdx.x / blocks, r0 = 32 * (blockIdx.x % blocks), ch0 = kMergeCh * blockIdx.y;
  const uint32_t total = p.first_tile[p.B], used = p.first_tile[p.B + 1], first = p.first_tile[b];
  const Seq s = seq_of(p, b);
  const int n_rows = s.nd * p.H;
  if (r0 >= n_rows) return;
  const uint32_t x = first + (r0 / kRows) * s.tiles;
  const uint32_t c0 = cluster_of(total, used, x), c1 = cluster_of(total, used, x + s.tiles - 1);
  if (c0 == c1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = r0 % kRows + lane, n = static_cast<int>(c1 - c0 + 1);
  const bool live = r0 + lane < n_rows;
  auto slot = [&](int i) { return int64_t(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)); };
  const float4* ml = reinterpret_cast<const float4*>(p.part_ml) + R;
  const float4* po = reinterpret_cast<const float4*>(p.part_o) + (ch0 / 4 + warp) * kRows + R;
  float m = -INFINITY, l = 0.0f, c = 1.0f;
  float4 o[4] = {};  // fours warp, warp + 8, ... of the block's channels
  if (live) {
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const float4 v = __ldcg(ml + slot(i) * kRows);  // reference, sum, c (the same in every part)
      float4 f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = __ldcg(po + slot(i) * (kD / 4) * kRows + 8 * k * kRows);
      const float to = v.y > 0.0f ? fmaxf(m, v.x) : m;
      const float cc = fminf(v.z, kMostC);
      const float w0 = m == to ? 1.0f : ex2((m - to) * cc), w1 = v.y > 0.0f ? ex2((v.x - to) * cc) : 0.0f;
      m = to;
      c = v.z;
      l = fmaf(w1, v.y, l * w0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[k].x = fmaf(w1, f[k].x, o[k].x * w0);
        o[k].y = fmaf(w1, f[k].y, o[k].y * w0);
        o[k].z = fmaf(w1, f[k].z, o[k].z * w0);
        o[k].w = fmaf(w1, f[k].w, o[k].w * w0);
      }
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // (NaN stays NaN)
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float* t = &tile[lane][4 * (warp + 8 * k)];
    t[0] = o[k].x * inv; t[1] = o[k].y * inv; t[2] = o[k].z * inv; t[3] = o[k].w * inv;
  }
  const int64_t row0 = int64_t(b) * p.T * p.H + r0;
  if (p.lse && blockIdx.y == 0 && warp == 0 && live) p.lse[row0 + lane] = lse_of(m, l, c);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = warp + 8 * k;
    if (r0 + r >= n_rows) continue;
    uint2 w;
    const float* t = &tile[r][4 * lane];
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(t[1]), "f"(t[0]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(t[3]), "f"(t[2]));
    *reinterpret_cast<uint2*>(p.out + (row0 + r) * kD + ch0 + 4 * lane) = w;
  }
}

}  // namespace

int tree_min_tiles() { return 2; }

// Items go whole to a cluster where sharing them would save less than it costs. All of them at once (up to one
// a cluster): an item shared by k clusters is done t - t / k tiles sooner, and the kernel that joins the parts takes
// as long as kJoin tiles. In several turns: a segment costs what kSegment tiles do beside its own, so whole items
// take ceil(items / clusters) (t + kSegment); sharing levels that to items / clusters, for one more segment per
// cluster and the second launch, kSharing tiles together. t counts the cache's rows, or the selection's, and 64
// drafts. Items of more than 20 tiles are always shared (their real lengths, which the host doesn't know, may
// differ). With 64 heads and 2 drafts (so of one tile less than t), whole against shared: 4 items of 5 tiles 23.9
// against 26.1 us, of 8 28.7 against 26.3, of 15 39.6 against 29.1; 16 of 5 25.3 against 28.4, of 8 29.2 against
// 28.3; 37 of 9 32.6 against 32.9, of 18 46.0 against 40.6; 45 of 20 49.0 against 52.3; 75 of 9 49.8 against 53.3,
// of 15 69.1 against 62.8; 96 of 9 53.6 against 63.1, of 15 71.9 against 76.9, of 22 91.2 against 90.2; 128 of 8
// 52.2 against 69.3; 225 of 12 112 against 118.
constexpr int64_t kJoin = 5, kSegment = 6, kSharing = 19, kMostWhole = 20;
static_assert(kMostWhole < int64_t(kFlush) && kFlush % 2 == 0, "whole items have no workspace; one set flushes");
static_assert(kJoin + 1 + kSegment <= kSharing, "items of kJoin + 1 tiles are whole in several turns too");
static int64_t tree_item_tiles(int64_t cap, int64_t top_k) { return ((top_k ? top_k : cap) + 64 + kTile - 1) / kTile; }

bool tree_always_whole(int64_t cap, int64_t top_k) { return tree_item_tiles(cap, top_k) - 1 <= kJoin; }

bool tree_whole_items(int64_t B, int64_t rows, int64_t cap, int64_t top_k, int num_sms) {
  const int64_t t = tree_item_tiles(cap, top_k), items = B * ((rows + kRows - 1) / kRows), most = num_sms / 2;
  if (t > kMostWhole) return false;
  if (items <= most) {
    const int64_t k = most / items;
    return t - (t + k - 1) / k <= kJoin;
  }
  const int64_t idle = (most - items % most) % most;  // clusters without an item in the last turn
  return idle * (t + kSegment) <= kSharing * most;
}

int64_t tree_tiles(int64_t B, int64_t rows, int64_t cap, int64_t top_k) {
  return B * ((rows + kRows - 1) / kRows) * tree_item_tiles(cap, top_k);
}

int tree_clusters(int64_t B, int64_t rows, int64_t cap, int64_t top_k, int num_sms) {
  const int64_t most = tree_always_whole(cap, top_k)
                           ? B * ((rows + kRows - 1) / kRows)
                           : (tree_tiles(B, rows, cap, top_k) + tree_min_tiles() - 1) / tree_min_tiles();
  return static_cast<int>(most < num_sms / 2 ? most : num_sms / 2);
}

cudaError_t launch_tree_attn(const TreeAttnParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> set[4];  // devices whose kernel has its shared-memory limit (calls of any thread)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev >= 256 || !(set[dev >> 6].load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k_tree_attn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    if (dev < 256) set[dev >> 6].fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.n_clusters);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_tree_attn, p);
  if (e != cudaSuccess || p.whole) return e;
  return launch_pdl(k_tree_merge, dim3(static_cast<unsigned>(p.B * ((p.T * p.H + 31) / 32)), kD / kMergeCh), dim3(256), stream, p);
}

}  // namespace fp4kv
