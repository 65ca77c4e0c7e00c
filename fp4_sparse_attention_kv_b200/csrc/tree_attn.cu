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
// Split in a cluster: O of 128 x 512 in fp32 would fill TMEM, so CTA r holds channels [256 r, +256)
// of q, V and O. S = Q V^T then is a sum over the CTAs: each forms its part with the tensor cores,
// CTA r finishes the rows [64 r, +64) of the item (it gets the other part through distributed
// shared memory), and P goes back to both. That way each cache row is dequantized once per cluster and
// half row of V feeds N = 64 and N = 256 products whose other operand is 128 rows deep. (The transposed
// form with all channels in one CTA, O^T of 512 x 64, reads shared memory 1.6 times as much per flop.)
//
// A CTA (25 warps):
//  * warps 16-23 dequantize: a tile's 64 half rows to fp16 (exact) in 128-byte-swizzled 64-channel
//    chunks, K-major B operand of S and MN-major B operand of O; four stages, loads two tiles ahead;
//  * warp 24 issues S(t + 2) (A = Q in TMEM), then O += P(t) V(t) (A = P in shared memory);
//  * warps 0-15 own TMEM lane quarter w % 4 (query rows) and column quarter w / 4. Those of the CTA's
//    own rows add the two parts of S, keep reference and sum in registers (lane = query row), and
//    write P; the others send their part of S over and take P's arrival.
// What crosses over goes by bulk copies that complete on the receiver's barrier: 2 KiB of S per warp
// and tile, 1 KiB of P. (Stores to the other CTA's memory, followed by a releasing arrival, held up the
// SM's other shared-memory instructions: 6,300 cycles a tile. The link moves 20 bytes a cycle each way.)
// Numerics: q as fp16 times a power of two per row (exact within 2^29 of the row's maximum), v exact
// in fp16, S and O in fp32. The reference m moves only when a logit passes it by 2^9 (log2 domain),
// to 2^3 above the maximum; p is stored as p * 2^6 in fp16, so the row's largest is at least 2^3 and at
// most 2^15: 11 bits each, and below 2^-14 a step of 2^-24, 2^-27 of the largest. The sums are fp32.
// Every wait is bounded; on timeout a status bit is set and the kernel winds down.
#include "fp4kv_common.cuh"
#include "fp4kv_launch.h"
#include "fp4kv_quant.cuh"
#include "fp4kv_sm100.cuh"

namespace fp4kv {
namespace {

constexpr int kD = 512, kHalf = 256;
constexpr int kRows = 128;  // query rows of an item
constexpr int kTile = 64;   // cache rows of a tile
constexpr int kStages = 4;
constexpr int kSoftWarps = 16, kDeqWarps = 8, kMmaWarp = 24;
constexpr int kThreads = 32 * (kMmaWarp + 4);  // (whole warpgroups: registers move between them)
constexpr int kCols = kTile / 2;  // columns of S per softmax warp
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMoveLog2 = 9.0f, kHeadroomLog2 = 3.0f, kPLog2 = 6.0f;

constexpr uint32_t kVBytes = kTile * kHalf * 2;   // 32 KiB: 4 chunks of [64 rows][128 B]
constexpr uint32_t kVChunk = kTile * 128;
constexpr uint32_t kPBytes = kRows * 128;         // [2 column halves][128 query rows][64 B] fp16
constexpr uint32_t kSxBytes = 64 * kTile * 4;     // [4 warps][8 column fours][32 query rows][4] fp32
constexpr uint32_t kOffV = 0;
constexpr uint32_t kOffP = kOffV + kStages * kVBytes;
constexpr uint32_t kOffSx = kOffP + 2 * kPBytes;
constexpr uint32_t kOffSt = kOffSx + 2 * kSxBytes;  // S on its way out, [2 tiles], 4 KiB per warp
constexpr uint32_t kOffQ = kOffP;                 // Q's way into TMEM: [128 rows][512 B] over P and Sx
static_assert(2 * kPBytes + 2 * kSxBytes == kRows * kHalf * 2, "Q staging");
constexpr uint32_t kOffBar = kOffSt + 2 * kSxBytes;
constexpr uint32_t kOffMisc = kOffBar + 208;
constexpr uint32_t kOffC = kOffBar + 256;         // [128] logit scale (log2 domain) per query row
constexpr uint32_t kOffMLx = kOffC;               // [2][64] (C is read before the start): the other CTA's rows' reference, sum
constexpr uint32_t kOffAx = kOffC + 512;          // [2][64] rescale factors of the other CTA's rows
constexpr uint32_t kOffPair = kOffAx + 512;       // [4][64] exchange between a row's four threads
constexpr uint32_t kOffRef = kOffPair + 1024;     // [2][64] reference after the last tile of either parity
constexpr uint32_t kSmem = kOffRef + 512;
static_assert(kSmem <= 232448, "shared memory");

// TMEM columns: O [0, 256), Q [256, 384), S slots [384, 448) and [448, 512)
constexpr uint32_t kColQ = 256, kColS = 384;

constexpr uint32_t kAhead = 2;  // S runs so many tiles ahead of O

enum { B_VFULL = 0, B_VFREE = 4, B_SFULL = 8, B_SFREE = 10, B_SXFULL = 12, B_PXFULL = 14, B_PREADY = 16, B_PFREE = 18,
       B_SXFREE = 20, B_REF = 22, B_DONE = 24 };

// ---------------------------------------------------------------------------------------
// cluster shared memory
// ---------------------------------------------------------------------------------------
FP4KV_DEV uint32_t map_peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
FP4KV_DEV void st_peer_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// An arrival that only says "my loads have returned" (a releasing one would first wait for every
// outstanding access of the thread: 1,000 cycles and more here).
FP4KV_DEV void mbar_arrive_peer_relaxed(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
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
// This CTA's shared memory to the other's, completing on a barrier there; 16-byte units.
FP4KV_DEV void bulk_peer(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "r"(src), "r"(bytes), "r"(bar) : "memory");
}
FP4KV_DEV void st_async_f32(uint32_t dst, float v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(dst), "f"(v), "r"(bar) : "memory");
}

// two fp32 at once
FP4KV_DEV uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
FP4KV_DEV void unpack2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
FP4KV_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
FP4KV_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// One lane of a converged warp.
FP4KV_DEV uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r;
}
// The MMA and commit wrappers below are called by the whole warp; the lane with `go` issues. The
// operands stay warp-uniform that way: inside a branch of one lane each MMA took 100 cycles to issue.
// D[tmem] (+)= A * B^T, fp16, A from TMEM, B from shared memory
FP4KV_DEV void umma_ts(uint32_t go, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, g;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 g, %5, 0;\n"
      " @g tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(go) : "memory");
}
// the same, A from shared memory
FP4KV_DEV void umma_ss(uint32_t go, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, g;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 g, %5, 0;\n"
      " @g tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(go) : "memory");
}
FP4KV_DEV void commit_if(uint32_t go, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred g;\n setp.ne.b32 g, %1, 0;\n"
      " @g tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
      ::"r"(smem_u32(bar)), "r"(go) : "memory");
}
// Arrive on the mbarrier at this offset in both CTAs of the cluster.
FP4KV_DEV void commit_pair_if(uint32_t go, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred g;\n setp.ne.b32 g, %2, 0;\n"
      " @g tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}"
      ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3)), "r"(go) : "memory");
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
// Registers move between warpgroups: 896 threads are launched with 72 each (16 x 88 + 8 x 48 + 4 x 56
// = 28 x 72 registers per lane).
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
  FP4KV_DEV int64_t work() const { return int64_t(tiles) * groups; }
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
// Clusters in use for `total` tiles: at least min_tiles each.
FP4KV_DEV int64_t clusters_used(int64_t total, int n_clusters, int min_tiles) {
  return max(int64_t(1), min(int64_t(n_clusters), (total + min_tiles - 1) / min_tiles));
}

// A cluster's range of tiles, segment by segment (a segment: consecutive tiles of one item).
struct SegIter {
  int b;
  int64_t off, rem;  // tiles of sequence b already passed; tiles still to do
  Seq s;
  uint32_t g, tile0, nt;
  FP4KV_DEV bool next(const TreeAttnParams& p) {
    if (rem <= 0) return false;
    s = seq_of(p, b);
    while (off >= s.work()) {
      off -= s.work();
      s = seq_of(p, ++b);
    }
    g = static_cast<uint32_t>(off / s.tiles);
    tile0 = static_cast<uint32_t>(off - int64_t(g) * s.tiles);
    nt = static_cast<uint32_t>(min(int64_t(s.tiles - tile0), rem));
    off += nt;
    rem -= nt;
    return true;
  }
};

// One thread's share of a tile's half rows: 16-byte units u and u + 4 of a row (32 channels each).
struct RawRow {
  uint4 c0, c1;
  uint32_t s0, s1;
};
FP4KV_DEV void dequant_unit(uint8_t* stage, int row, int u, const uint4& c, uint32_t s) {
  const uint32_t sa = e4m3x2_to_f16x2(static_cast<uint16_t>((s & 0xffu) * 0x101u));
  const uint32_t sb = e4m3x2_to_f16x2(static_cast<uint16_t>((s >> 8) * 0x101u));
  uint8_t* base = stage + (u >> 1) * kVChunk + row * 128;
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t s2 = k < 2 ? sa : sb;
    uint4 o;
    o.x = hmul2_f16(e2m1x2_to_f16x2(w[k] & 0xffu), s2);
    o.y = hmul2_f16(e2m1x2_to_f16x2((w[k] >> 8) & 0xffu), s2);
    o.z = hmul2_f16(e2m1x2_to_f16x2((w[k] >> 16) & 0xffu), s2);
    o.w = hmul2_f16(e2m1x2_to_f16x2(w[k] >> 24), s2);
    *reinterpret_cast<uint4*>(base + (((4 * (u & 1) + k) ^ (row & 7)) << 4)) = o;
  }
}

// this thread's TMEM lane, 128 of its O columns, times a
FP4KV_DEV void rescale_o(uint32_t addr, float a) {
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {  // (16 at a time: the caller holds a tile's logits)
    uint32_t r[16];
    tmem_ld16(addr + 16 * c, r);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * a);
    tmem_st16(addr + 16 * c, r);
  }
  tmem_st_wait();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) k_tree_attn(const TreeAttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  float* sC = reinterpret_cast<float*>(smem + kOffC);
  float* sAx = reinterpret_cast<float*>(smem + kOffAx);
  const float* sMLx = reinterpret_cast<const float*>(smem + kOffMLx);
  float* sPair = reinterpret_cast<float*>(smem + kOffPair);
  float* sRef = reinterpret_cast<float*>(smem + kOffRef);
  int64_t* s_off = reinterpret_cast<int64_t*>(smem + kOffMisc);  // the range's start: tiles into sequence s_b
  int64_t* s_rem = s_off + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc + 16);
  volatile uint32_t* s_abort = s_tmem + 1;
  int* s_b = reinterpret_cast<int*>(s_tmem + 2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank(), peer = rank ^ 1u;
  const int cl = blockIdx.x >> 1;
  griddep_wait();

  // the smem alignment that the swizzled operands need (the same in both CTAs of a launch)
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) atomicOr(p.status, 2u);
    return;
  }
  // ---- this cluster's range of tiles ----
  if (warp == 0) {
    int64_t total = 0;
    for (int b = lane; b < p.B; b += 32) {
      const Seq s = seq_of(p, b);
      total += s.work();
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int64_t used = clusters_used(total, p.n_clusters, p.min_tiles);
    const int64_t x0 = cl < used ? total * cl / used : total;
    const int64_t x1 = cl < used ? total * (cl + 1) / used : total;
    // where x0 lies, and (cluster 0) each sequence's first tile for the merge
    int64_t at = 0;
    bool found = x1 <= x0;
    for (int b0 = 0; b0 < p.B && (!found || cl == 0); b0 += 32) {
      const int b = b0 + lane;
      int64_t n = 0;
      if (b < p.B) {
        const Seq s = seq_of(p, b);
        n = s.work();
      }
      int64_t incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (cl == 0 && rank == 0 && b < p.B) p.first_tile[b] = at + incl - n;
      const uint32_t hit = __ballot_sync(0xffffffffu, at + incl > x0);
      if (!found && hit) {
        if (lane == __ffs(hit) - 1) {
          *s_b = b;
          *s_off = x0 - (at + incl - n);
        }
        found = true;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      *s_rem = x1 - x0;
      *s_abort = 0;
      if (cl == 0 && rank == 0) p.first_tile[p.B] = total;
    }
  }
  if (tid == 32) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars[B_VFULL + i], kDeqWarps);
      mbar_init(&bars[B_VFREE + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[B_SFULL + i], 1);
      mbar_init(&bars[B_SFREE + i], kSoftWarps / 2);
      mbar_init(&bars[B_SXFULL + i], 1);
      mbar_init(&bars[B_SXFREE + i], kSoftWarps / 4);
      mbar_init(&bars[B_PXFULL + i], 1);
      mbar_init(&bars[B_PREADY + i], kSoftWarps / 2);
      mbar_init(&bars[B_REF + i], 2);
      mbar_init(&bars[B_PFREE + i], 2);
    }
    mbar_init(&bars[B_DONE], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (*s_rem <= 0) return;  // (both CTAs of the cluster)
  if (warp == kMmaWarp) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  SegIter it;
  it.b = *s_b;
  it.off = *s_off;
  it.rem = *s_rem;
  uint32_t n = 0;  // tiles so far, over all segments: stage n % 4, slot n % 2

  auto aborted = [&]() { return __any_sync(0xffffffffu, *s_abort != 0) != 0; };
  auto give_up = [&]() {
    if (lane == 0) {
      atomicOr(p.status, kFlagWaitTimeout);
      *s_abort = 1;
    }
  };

  if (warp >= kSoftWarps && warp < kMmaWarp) {
    // ------------------------------ load and dequantize ------------------------------
    fewer_registers<48>();
    // Eight lanes take eight rows (distinct swizzle phases: no store conflicts), four units each.
    const int row = 8 * (warp - kSoftWarps) + (lane & 7), u0 = lane >> 3;
    while (it.next(p)) {
      const Seq& s = it.s;
      // a drafted row that no token sees counts as absent
      uint64_t seen = 0;
      for (int t = lane; t < s.nd; t += 32) seen |= p.tree_mask[int64_t(it.b) * p.T + t];
      seen = uint64_t(__reduce_or_sync(0xffffffffu, uint32_t(seen))) |
             (uint64_t(__reduce_or_sync(0xffffffffu, uint32_t(seen >> 32))) << 32);
      const int32_t* idx = p.idx ? p.idx + int64_t(it.b) * p.top_k : nullptr;
      const uint8_t* packed = p.packed + int64_t(it.b) * p.cap * (kD / 2) + 128 * rank;
      const uint8_t* scales = p.scales + int64_t(it.b) * p.cap * (kD / kGroup) + 16 * rank;
      // this thread's row of tile i: a position, which is checked only when it is used (it may still be
      // on its way from the selection)
      auto pos_of = [&](uint32_t i) -> int32_t {
        const uint32_t e = (it.tile0 + i) * kTile + row;
        if (i >= it.nt) return -1;
        if (e < s.n_sel) return idx ? idx[e] : static_cast<int32_t>(e);
        const uint32_t j = e - s.n_sel;
        return j < uint32_t(s.nd) && ((seen >> j) & 1) && int64_t(s.pre) + j < p.cap ? static_cast<int32_t>(s.pre + j) : -1;
      };
      auto load = [&](RawRow& r, uint32_t i, int32_t pos) {
        const bool sel = (it.tile0 + i) * kTile + row < s.n_sel;
        r.c0 = r.c1 = make_uint4(0, 0, 0, 0);
        r.s0 = r.s1 = 0;
        if (static_cast<uint32_t>(pos) < (sel ? s.pre : 0x80000000u)) {
          const uint8_t* c = packed + int64_t(pos) * (kD / 2) + 16 * u0;
          const uint8_t* f = scales + int64_t(pos) * (kD / kGroup) + 2 * u0;
          r.c0 = ld_nc_v4(c);
          r.c1 = ld_nc_v4(c + 64);
          r.s0 = *reinterpret_cast<const uint16_t*>(f);
          r.s1 = *reinterpret_cast<const uint16_t*>(f + 8);
        }
      };
      RawRow ra, rb, rc;  // tiles i, i + 1, i + 2 (each reloaded in place: a copy would wait for its loads)
      load(ra, 0, pos_of(0));
      load(rb, 1, pos_of(1));
      load(rc, 2, pos_of(2));
      int32_t pos = pos_of(3);
      bool ok = !aborted();
      cluster_sync_all();  // start of the segment
      auto tile = [&](RawRow& r, uint32_t i) {
        if (!ok || i >= it.nt) return;
        const uint32_t m = n + i, st = m & (kStages - 1);
        // (eight warps that wait most of the time: sparing polls leave shared memory to the others)
        ok = __all_sync(0xffffffffu, mbar_wait_sleepy(&bars[B_VFREE + st], ((m >> 2) & 1) ^ 1, 64));
        if (!ok) return;
        uint8_t* stage = smem + kOffV + st * kVBytes;
        dequant_unit(stage, row, u0, r.c0, r.s0);
        dequant_unit(stage, row, u0 + 4, r.c1, r.s1);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_VFULL + st]);
        load(r, i + 3, pos);
        pos = pos_of(i + 4);
      };
      for (uint32_t i = 0; ok && i < it.nt; i += 3) {
        tile(ra, i);
        tile(rb, i + 1);
        tile(rc, i + 2);
      }
      if (!ok) give_up();
      n += it.nt;
      __syncwarp();
      cluster_sync_all();  // end of the segment
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------ MMA issue (one warp; its warpgroup's others idle) ------------------------------
    fewer_registers<56>();
    constexpr uint32_t kIdescS = umma_idesc(0u, kRows, kTile, 0u, 0u);
    constexpr uint32_t kIdescO = umma_idesc(0u, kRows, kHalf, 0u, 1u);
    const uint64_t dvk = sw128_kmajor_desc(smem_u32(smem + kOffV));
    const uint64_t dvm = sw128_mnmajor_desc(smem_u32(smem + kOffV), kVChunk);
    const uint64_t dp = sw64_kmajor_desc(smem_u32(smem + kOffP));
    const uint32_t go = elect_lane();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto scores = [&](uint32_t m) -> bool {
      const uint32_t st = m & (kStages - 1), sl = m & 1;
      if (!warp_wait(&bars[B_VFULL + st], (m >> 2) & 1) || !warp_wait(&bars[B_SFREE + sl], ((m >> 1) & 1) ^ 1)) return false;
      tc_fence_after();
      const uint64_t b0 = dvk + ((st * kVBytes) >> 4);
      const uint32_t d = tm + kColS + kTile * sl;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_ts(go, d, tm + kColQ + 32 * c + 8 * k, b0 + ((c * kVChunk) >> 4) + 2 * k, kIdescS, (c | k) != 0);
      commit_if(go, &bars[B_SFULL + sl]);
      return true;
    };
    while (it.next(p)) {
      cluster_sync_all();  // start
      tc_fence_after();
      if (warp != kMmaWarp) {
        cluster_sync_all();
        continue;
      }
      bool ok = !aborted();
      for (uint32_t i = 0; ok && i < kAhead && i < it.nt; ++i) ok = scores(n + i);
      for (uint32_t i = 0; ok && i < it.nt; ++i) {
        const uint32_t m = n + i, st = m & (kStages - 1), sl = m & 1;
        if (i + kAhead < it.nt && !scores(m + kAhead)) ok = false;
        if (ok && !warp_wait(&bars[B_PREADY + sl], (m >> 1) & 1)) ok = false;
        if (ok) {
          tc_fence_after();
          const uint64_t a0 = dp + ((sl * kPBytes) >> 4), b0 = dvm + ((st * kVBytes) >> 4);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            umma_ss(go, tm, a0 + ((kPBytes / 2 * (k >> 1)) >> 4) + 2 * (k & 1), b0 + ((2048 * k) >> 4), kIdescO, i > 0 || k > 0);
          commit_if(go, &bars[B_VFREE + st]);
          commit_pair_if(go, &bars[B_PFREE + sl]);
        }
      }
      if (!ok) give_up();
      n += it.nt;
      __syncwarp();
      cluster_sync_all();  // end
    }
    if (warp == kMmaWarp) {
      commit_if(go, &bars[B_DONE]);  // nothing is in flight when TMEM is released
      __syncwarp();
      if (!warp_wait(&bars[B_DONE], 0)) give_up();
    }
  } else {
    // ------------------------------ softmax ------------------------------
    // Own rows: warps 0-7 take the even tiles (of all that the cluster works on), 8-15 the odd ones:
    // every slot that a set uses is its own, and one set's waits overlap the other's arithmetic.
    more_registers<88>();
    const int q = warp & 3, h4 = warp >> 2, h = h4 & 1;
    const uint32_t sl = warp >> 3;
    const int pair = 4 * static_cast<int>(sl) + q;
    const int R = 32 * q + lane, rl = R & 63;  // query row of the item, and within its half
    const bool own = static_cast<uint32_t>(q >> 1) == rank;
    const uint32_t lane_addr = tmem + (uint32_t(32 * q) << 16);
    const uint32_t o_addr = lane_addr + 128 * h;
    const uint32_t peer_smem = map_peer(smem_u32(smem), peer);
    while (it.next(p)) {
      const Seq& s = it.s;
      const int live_rows = s.nd * p.H - static_cast<int>(it.g) * kRows;  // of this item (and behind)
      const int64_t row0 = int64_t(it.b) * p.T * p.H + int64_t(it.g) * kRows;
      // ---- Q: bf16 -> fp16 times a power of two, through shared memory into TMEM ----
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        uint4 v[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = warp + kSoftWarps * (4 * part + k);
          v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
          if (r < live_rows) {
            const uint16_t* src = p.q + (row0 + r) * kD + 8 * lane;
            v[k][0] = *reinterpret_cast<const uint4*>(src);
            v[k][1] = *reinterpret_cast<const uint4*>(src + kHalf);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = warp + kSoftWarps * (4 * part + k);
          uint32_t m2 = 0;
          m2 = __vmaxu2(v[k][0].x & 0x7fff7fffu, v[k][0].y & 0x7fff7fffu);
          m2 = __vmaxu2(m2, __vmaxu2(v[k][0].z & 0x7fff7fffu, v[k][0].w & 0x7fff7fffu));
          m2 = __vmaxu2(m2, __vmaxu2(v[k][1].x & 0x7fff7fffu, v[k][1].y & 0x7fff7fffu));
          m2 = __vmaxu2(m2, __vmaxu2(v[k][1].z & 0x7fff7fffu, v[k][1].w & 0x7fff7fffu));
          const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
          int e = 0;  // the power of two that brings the row's maximum into [2^14, 2^15)
          if (m != 0) e = max(-126, min(127, 14 - max(-126, int(m >> 7) - 127)));
          // (a negative scale goes into q's sign: the factor of the logits is positive)
          const float up = copysignf(__uint_as_float(uint32_t(127 + e) << 23), p.sm_scale);
          const uint4 own_half = rank ? v[k][1] : v[k][0];
          const uint32_t w[4] = {own_half.x, own_half.y, own_half.z, own_half.w};
          uint32_t f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            f[j] = pack_f16x2(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up);
          *reinterpret_cast<uint4*>(smem + kOffQ + r * 512 + ((lane ^ (r & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
          if (lane == 0)
            sC[r] = fmaxf(fabsf(p.sm_scale) * kLog2e * __uint_as_float(uint32_t(127 - e / 2) << 23) *
                              __uint_as_float(uint32_t(127 - (e - e / 2)) << 23),
                          2e-38f);  // (above zero: a masked -inf stays -inf)
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory");
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 f = *reinterpret_cast<const uint4*>(smem + kOffQ + R * 512 + (((8 * h4 + 4 * c + k) ^ (R & 7)) << 4));
          w[4 * k] = f.x; w[4 * k + 1] = f.y; w[4 * k + 2] = f.z; w[4 * k + 3] = f.w;
        }
        tmem_st16(lane_addr + kColQ + 32 * h4 + 16 * c, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      const float c = sC[R];
      cluster_sync_all();  // start: Q is in TMEM, its staging (P, Sx) is free, in both CTAs
      tc_fence_after();

      bool ok = !aborted();
      const uint32_t last = n + it.nt - 1;
      const uint32_t i0 = (n ^ sl) & 1;  // this set's first tile
      if (own) {
        uint64_t rmask = 0;  // the drafts that this row's token sees
        if (R < live_rows) {
          rmask = p.tree_mask[int64_t(it.b) * p.T + (it.g * kRows + R) / uint32_t(p.H)];
          const int64_t nv = min(int64_t(s.nd), p.cap - int64_t(s.pre));
          if (nv < 64) rmask &= (uint64_t(1) << nv) - 1;
        }
        const int32_t* idx = p.idx ? p.idx + int64_t(it.b) * p.top_k : nullptr;
        auto entry_ok = [&](uint32_t i) -> bool {  // entry 32 h + lane of tile i lies in the prefix
          const uint32_t e = (it.tile0 + i) * kTile + kCols * h + lane;
          if (i >= it.nt || e >= s.n_sel) return false;
          return !idx || static_cast<uint32_t>(idx[e]) < s.pre;
        };
        bool e_ok = entry_ok(i0);
        float ref = -INFINITY;  // the reference that l2 is relative to
        uint64_t l2 = 0;        // the row's sum over even and odd columns
        const uint64_t c2 = pack2(c, c);
        const bool arms = h == 0 && (q & 1) == 0 && lane == 0;
        // a wait that ran out ends the loop of both warps of a row at the next vote
        bool dead = !ok;
        for (uint32_t i = i0; i < it.nt; i += 2) {
          const uint32_t m = n + i, ph = (m >> 1) & 1;
          if (arms) mbar_arrive_expect_tx(&bars[B_SXFULL + sl], kSxBytes);
          uint32_t vis = __ballot_sync(0xffffffffu, e_ok);
          e_ok = entry_ok(i + 2);
          const uint32_t e0 = (it.tile0 + i) * kTile + kCols * h;
          if (e0 + kCols > s.n_sel)  // drafts among the columns
            vis |= e0 >= s.n_sel ? (e0 - s.n_sel < 64 ? uint32_t(rmask >> (e0 - s.n_sel)) : 0u) : uint32_t(rmask << (s.n_sel - e0));
          dead = dead || !warp_wait(&bars[B_SFULL + sl], ph);
          tc_fence_after();
          uint32_t r[32];
          tmem_ld32(lane_addr + kColS + kTile * sl + kCols * h, r);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_SFREE + sl]);
          dead = dead || !warp_wait_cluster(&bars[B_SXFULL + sl], ph);
          const float4* sx = reinterpret_cast<const float4*>(smem + kOffSx + sl * kSxBytes + 4096 * (2 * (q & 1) + h)) + lane;
          uint64_t z[16];  // logits over c
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 f = sx[32 * k];
            z[2 * k] = add2(pack2(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1])), pack2(f.x, f.y));
            z[2 * k + 1] = add2(pack2(__uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3])), pack2(f.z, f.w));
          }
          float mx = -INFINITY;
          if (__all_sync(0xffffffffu, vis == 0xffffffffu)) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float z0, z1;
              unpack2(z[k], z0, z1);
              mx = fmaxf(mx, fmaxf(z0, z1));
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float z0, z1;
              unpack2(z[k], z0, z1);
              z0 = (vis >> (2 * k)) & 1 ? z0 : -INFINITY;
              z1 = (vis >> (2 * k + 1)) & 1 ? z1 : -INFINITY;
              z[k] = pack2(z0, z1);
              mx = fmaxf(mx, fmaxf(z0, z1));
            }
          }
          mx *= c;
          // the reference after the tile before, from the other set
          float old = -INFINITY;
          if (i > 0) {
            dead = dead || !warp_wait(&bars[B_REF + (sl ^ 1)], ((m - 1) >> 1) & 1);
            old = sRef[64 * (sl ^ 1) + rl];
          }
          float to = old, a = 1.0f;
          const bool moves = pair_any(pair, mx > old + kMoveLog2 || dead);
          // (the vote needs the loaded values, so every lane's loads from the slot have returned)
          if (lane == 0) mbar_arrive_peer_relaxed(peer_smem + kOffBar + 8 * (B_SXFREE + sl));
          if (moves) {  // a reference of these 32 rows moves
            if (pair_any(pair, dead)) {
              dead = true;
              break;
            }
            sPair[64 * (2 * sl + h) + rl] = mx;
            pair_sync(pair);
            mx = fmaxf(mx, sPair[64 * (2 * sl + (h ^ 1)) + rl]);
            if (mx > old + kMoveLog2) {
              to = mx + kHeadroomLog2;
              if (i > 0) a = ex2(old - to);  // (O starts with the first tile; no reference so far: 0)
            }
          }
          if (h == 0) {
            sRef[64 * sl + rl] = to;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_REF + sl]);
          }
          if (to != ref) {
            const float f = ex2(ref - to);
            l2 = fma2(l2, pack2(f, f), 0);
            ref = to;
          }
          if (moves && __any_sync(0xffffffffu, a != 1.0f)) {
            dead = !warp_wait(&bars[B_VFREE + ((m - 1) & (kStages - 1))], ((m - 1) >> 2) & 1);
            tc_fence_after();
            rescale_o(o_addr, a);
          }
          // P's slot is free in both CTAs
          dead = dead || !warp_wait_cluster(&bars[B_PFREE + sl], ph ^ 1);
          const uint32_t px_bar = peer_smem + kOffBar + 8 * (B_PXFULL + sl);
          if (h == 0) st_async_f32(peer_smem + kOffAx + 4 * (64 * sl + rl), a, px_bar);
          const uint32_t pw = kOffP + sl * kPBytes + h * (kPBytes / 2) + 32 * q * 64;  // this warp's 2 KiB
          uint8_t* prow = smem + pw + lane * 64;
          const float m6 = ref == -INFINITY ? -INFINITY : kPLog2 - ref;
          const uint64_t m62 = pack2(m6, m6);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float z0, z1;
              unpack2(fma2(z[4 * u + k], c2, m62), z0, z1);
              const float e0 = ex2(z0), e1 = ex2(z1);
              l2 = add2(l2, pack2(e0, e1));
              w[k] = pack_f16x2(e0, e1);
            }
            *reinterpret_cast<uint4*>(prow + ((u ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            bulk_peer(peer_smem + pw, smem_u32(smem) + pw, kPBytes / 8, px_bar);
            mbar_arrive(&bars[B_PREADY + sl]);
          }
        }
        ok = !dead;
        // the row's sum over its four threads; reference and sum to both CTAs
        quad_sync(q);
        const float fin = sRef[64 * (last & 1) + rl];
        float l, l1;
        unpack2(l2, l, l1);
        l += l1;
        if (l > 0.0f) l *= ex2(ref - fin);
        if (h4 != 0) sPair[64 * h4 + rl] = l;
        quad_sync(q);
        if (h4 == 0) {
          l += sPair[64 + rl] + sPair[128 + rl] + sPair[192 + rl];
          sPair[rl] = l;
          st_peer_f32(peer_smem + kOffMLx + 4 * rl, fin);
          st_peer_f32(peer_smem + kOffMLx + 4 * (64 + rl), l);
        }
      } else if (sl == 0) {
        // send S's rows over: warps 0-7, every tile
        for (uint32_t i = 0; ok && i < it.nt; ++i) {
          const uint32_t m = n + i, to = m & 1, ph = (m >> 1) & 1;
          ok = warp_wait(&bars[B_SFULL + to], ph);
          tc_fence_after();
          uint32_t r[32];
          tmem_ld32(lane_addr + kColS + kTile * to + kCols * h, r);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_SFREE + to]);
          // (the receiver has read S(m - 2): its slot and its staging here are free)
          ok = ok && warp_wait_cluster(&bars[B_SXFREE + to], ph ^ 1);
          const uint32_t wo = to * kSxBytes + 4096 * (2 * (q & 1) + h);
          uint4* st = reinterpret_cast<uint4*>(smem + kOffSt + wo) + lane;
#pragma unroll
          for (int k = 0; k < 8; ++k) st[32 * k] = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0)
            bulk_peer(peer_smem + kOffSx + wo, smem_u32(smem + kOffSt) + wo, 4096, peer_smem + kOffBar + 8 * (B_SXFULL + to));
        }
      } else {
        // take P's arrival: warps 8-15, every tile; O's rows follow a moved reference
        const bool arms = h == 0 && (q & 1) == 0 && lane == 0;
        for (uint32_t i = 0; ok && i < it.nt; ++i) {
          const uint32_t m = n + i, at = m & 1;
          if (arms) mbar_arrive_expect_tx(&bars[B_PXFULL + at], kPBytes / 2 + 256);
          ok = warp_wait_cluster(&bars[B_PXFULL + at], (m >> 1) & 1);
          const float a = sAx[64 * at + rl];
          if (__any_sync(0xffffffffu, a != 1.0f)) {
            ok = ok && warp_wait(&bars[B_VFREE + ((m - 1) & (kStages - 1))], ((m - 1) >> 2) & 1);
            tc_fence_after();
            rescale_o(o_addr, a);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_PREADY + at]);
        }
      }
      n += it.nt;
      if (ok) ok = warp_wait(&bars[B_VFREE + (last & (kStages - 1))], (last >> 2) & 1);
      if (!ok) give_up();
      __syncwarp();
      cluster_sync_all();  // end: O, references and sums are complete in both CTAs
      tc_fence_after();
      // ---- out ----
      const float ref = own ? sRef[64 * (last & 1) + rl] : sMLx[rl], l = own ? sPair[rl] : sMLx[64 + rl];
      const bool whole = it.tile0 == 0 && it.nt == s.tiles;
      const bool live = R < live_rows;
      const int slot = 2 * cl + (it.tile0 == 0 ? 1 : 0);
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t r[32];
        tmem_ld32(lane_addr + 64 * h4 + 32 * c, r);
        tmem_ld_wait();
        const int ch = kHalf * rank + 64 * h4 + 32 * c;
        if (live && whole) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + (row0 + R) * kD + ch);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                  : "=r"(w[j])
                  : "f"(__uint_as_float(r[8 * k + 2 * j + 1]) * inv), "f"(__uint_as_float(r[8 * k + 2 * j]) * inv));
            dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (live) {
          uint4* dst = reinterpret_cast<uint4*>(p.part_o + int64_t(slot * kRows + R) * kD + ch);
#pragma unroll
          for (int k = 0; k < 8; ++k) __stcg(dst + k, make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]));
        }
        __syncwarp();
      }
      if (live && rank == 0 && h4 == 0) {
        if (!whole)
          __stcg(reinterpret_cast<float2*>(p.part_ml) + slot * kRows + R, make_float2(ref, l));
        else if (p.lse)
          p.lse[row0 + R] = l > 0.0f ? (ref - kPLog2) * kLn2 + logf(l) : -INFINITY;
      }
      tc_fence_before();
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of items that several clusters worked on: o = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c.
// One block per query row, four channels per thread; the parts are read once from L2.
__global__ void __launch_bounds__(kD / 4) k_tree_merge(const TreeAttnParams p) {
  griddep_wait();
  const int64_t row = blockIdx.x;
  const int b = static_cast<int>(row / (p.T * p.H));
  const int rr = static_cast<int>(row - int64_t(b) * p.T * p.H);
  const Seq s = seq_of(p, b);
  if (rr >= s.nd * p.H) return;
  const int64_t total = p.first_tile[p.B], used = clusters_used(total, p.n_clusters, p.min_tiles);
  const int64_t x = p.first_tile[b] + int64_t(rr / kRows) * s.tiles;
  // the cluster of tile x: the largest i with floor(total i / used) <= x
  const int64_t c0 = ((x + 1) * used - 1) / total, c1 = ((x + s.tiles) * used - 1) / total;
  if (c0 == c1) return;
  const int R = rr % kRows, n = static_cast<int>(c1 - c0 + 1);
  auto slot = [&](int i) { return i == 0 ? 2 * c0 + 1 : 2 * (c0 + i); };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float m = -INFINITY;
  for (int i = 0; i < n; ++i) {
    const float2 v = __ldcg(ml + slot(i) * kRows + R);
    if (v.y > 0.0f) m = fmaxf(m, v.x);
  }
  float l = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = 0; i < n; ++i) {
    const float2 v = __ldcg(ml + slot(i) * kRows + R);
    const float4 f = __ldcg(reinterpret_cast<const float4*>(p.part_o + (slot(i) * kRows + R) * kD) + threadIdx.x);
    const float w = v.y > 0.0f ? ex2(v.x - m) : 0.0f;
    l = fmaf(w, v.y, l);
    o.x = fmaf(w, f.x, o.x);
    o.y = fmaf(w, f.y, o.y);
    o.z = fmaf(w, f.z, o.z);
    o.w = fmaf(w, f.w, o.w);
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  uint2 w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(o.y * inv), "f"(o.x * inv));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(o.w * inv), "f"(o.z * inv));
  *reinterpret_cast<uint2*>(p.out + row * kD + 4 * threadIdx.x) = w;
  if (p.lse && threadIdx.x == 0) p.lse[row] = l > 0.0f ? (m - kPLog2) * kLn2 + logf(l) : -INFINITY;
}

}  // namespace

int tree_min_tiles() { return 2; }

int tree_clusters(int64_t B, int64_t rows, int64_t cap, int64_t top_k, int num_sms) {
  const int64_t tiles = ((top_k ? top_k : cap) + 64 + kTile - 1) / kTile;
  const int64_t total = B * ((rows + kRows - 1) / kRows) * tiles;
  const int64_t most = (total + tree_min_tiles() - 1) / tree_min_tiles();
  return static_cast<int>(most < num_sms / 2 ? most : num_sms / 2);
}

cudaError_t launch_tree_attn(const TreeAttnParams& p, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(k_tree_attn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
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
  if (e != cudaSuccess) return e;
  return launch_pdl(k_tree_merge, dim3(static_cast<unsigned>(int64_t(p.B) * p.T * p.H)), dim3(kD / 4), stream, p);
}

}  // namespace fp4kv
