// qkv_norm_rope_fp4: RMS norm and position rotation of every query head and of the token's KV row
// in one launch; the KV row is quantised into the FP4 cache as it is made.
//
// For a row x of d channels with weight w (or 1):  r = 1 / sqrt(sum x^2 / d + eps),  u = x w;
// y_i = u_i r for the first d - rope_dim channels; the last rope_dim are rotated in pairs (a, b) by
// the token's angles: y_a = (u_a c - u_b s) r, y_b = (u_b c + u_a s) r. Pairs are neighbours
// (2j, 2j + 1), or (j, j + rope_dim / 2).
//
// Bound by memory: 2 d bytes in and out per query row, 2 d in and 9/16 d out per KV row; a row is read
// once. LPR lanes share a row, each with GPL groups of 16 channels (two 16-byte loads a group).
//
// Queries: a warp takes several heads of one token. With P = w c and Q = -+ w_partner s, formed once per
// token, every channel is y = (x P + x_partner Q) r, two at a time in packed fp32 (outside the rotated
// channels P = w, Q = 0), so no lane waits for the rotated ones. fp32, rounded once to bf16. Rows come
// through a ring in shared memory, four passes ahead (in registers one ahead fitted: 241 us for 8,192
// tokens of 64 heads with their KV rows and a read table of positions; now 185 us, 5.9 TB/s; the queries alone 170).
//
// The KV row: y's nearest fp32 value is rounded to bf16 and that is quantised, so the cache holds
// exactly what kv_quant_fp4 makes of kv_out. A code is decided by which side of a border a value
// falls on, so y must not be off by even an fp32 step: sum x^2 and r are held in fp64. A quick fp32 form
// v of y is off by at most 4 x 2^-24 of mag, the sum of the magnitudes of its two terms (the product and
// the sum rounded, r rounded, one product; one term and 2 x 2^-24 outside the rotated channels). Where v
// lies nearer than that (6, or 3 units) to a bf16 rounding border, y is formed in fp64: one value in
// thousands. The rotated groups of a warp's rows are done together, one to a lane, after the others
// (beside the others four lanes in 32 worked on them: 1,150 instructions a row, 172 us for 131,072 rows;
// now 532 and 98 us, bound by issuing them).
#include "fp4kv_common.cuh"
#include "fp4kv_launch.h"
#include "fp4kv_quant.cuh"
#include "fp4kv_sm100.cuh"

namespace fp4kv {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kOnes = 0x3f803f80u;  // two bf16 ones
enum { kNone = 0, kNeighbours = 1, kHalves = 2 };  // the rotation's pairs

FP4KV_DEV uint32_t f32_to_bf16(float f) {  // round to nearest even
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
  return r;
}
FP4KV_DEV uint32_t f32x2_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// (fp64 to fp32 to bf16, each to nearest even)
FP4KV_DEV uint32_t f64_to_bf16(double y) { return f32_to_bf16(__double2float_rn(y)); }
FP4KV_DEV float half_of(uint32_t w, int k) {  // channel k (0 low, 1 high) of a bf16 pair
  return __uint_as_float(k ? (w & 0xffff0000u) : (w << 16));
}
FP4KV_DEV uint4 ld_v4(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

FP4KV_DEV uint64_t widen2(uint32_t w) { return pack2(half_of(w, 0), half_of(w, 1)); }

// The 8-channel unit that holds the partners of the unit at channel c0 (pairs of halves), and whether c0's
// unit is the second half.
FP4KV_DEV int partner_unit(const NormRopeParams& p, int c0, bool& second) {
  const int hr = p.rope_dim / 2;
  second = c0 - (p.d - p.rope_dim) >= hr;
  return second ? c0 - hr : c0 + hr;
}

// ---------------------------------------------------------------------------------------
// queries
// ---------------------------------------------------------------------------------------
FP4KV_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
FP4KV_DEV void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int LPR, int GPL, int kPairs>
FP4KV_DEV void query_heads(const NormRopeParams& p, uint32_t ring, int64_t tok, int h0, int h1) {
  constexpr int kDepth = 4 / GPL;             // passes in flight
  constexpr uint32_t kSlot = 1024 * GPL;       // bytes of one: the rows at once, LPR * GPL groups of 32 each
  constexpr int kRows = 32 / LPR;  // heads at once
  const int l = threadIdx.x & (LPR - 1), sub = (threadIdx.x & 31) / LPR;
  if (kPairs != kNone && (p.positions[tok] < 0 || p.positions[tok] >= p.max_pos)) return;
  // P and Q of this lane's channels
  uint64_t P[GPL][8], Q[GPL][8];
  bool there[GPL], rot[GPL];
#pragma unroll
  for (int g = 0; g < GPL; ++g) {
    const int c0 = (l + LPR * g) * kGroup;
    there[g] = c0 < p.d;
    // (rope_dim is a multiple of 16: a group is rotated as a whole)
    rot[g] = kPairs != kNone && there[g] && c0 >= p.d - p.rope_dim;
    uint4 wa = make_uint4(kOnes, kOnes, kOnes, kOnes), wb = wa;
    if (p.q_weight && there[g]) {
      wa = ld_v4(p.q_weight + c0);
      wb = ld_v4(p.q_weight + c0 + 8);
    }
    const uint32_t w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      P[g][k] = widen2(w[k]);
      Q[g][k] = 0;
    }
    if (kPairs != kNone && rot[g]) {
      const float* cs = p.cos_sin + p.positions[tok] * p.rope_dim;
      const int hr = p.rope_dim / 2, j0 = c0 - (p.d - p.rope_dim);
      if (kPairs == kNeighbours) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float co = cs[j0 / 2 + k], si = cs[hr + j0 / 2 + k];
          const float w0 = half_of(w[k], 0), w1 = half_of(w[k], 1);
          P[g][k] = pack2(w0 * co, w1 * co);
          Q[g][k] = pack2(-w1 * si, w0 * si);
        }
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          bool second;
          const int cp = partner_unit(p, c0 + 8 * u, second);
          const int jj = j0 + 8 * u - (second ? hr : 0);
          const uint4 pw = p.q_weight ? ld_v4(p.q_weight + cp) : make_uint4(kOnes, kOnes, kOnes, kOnes);
          const uint32_t wp[4] = {pw.x, pw.y, pw.z, pw.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float c_0 = cs[jj + 2 * k], c_1 = cs[jj + 2 * k + 1];
            float s_0 = cs[hr + jj + 2 * k], s_1 = cs[hr + jj + 2 * k + 1];
            if (!second) s_0 = -s_0, s_1 = -s_1;
            P[g][4 * u + k] = pack2(half_of(w[4 * u + k], 0) * c_0, half_of(w[4 * u + k], 1) * c_1);
            Q[g][4 * u + k] = pack2(half_of(wp[k], 0) * s_0, half_of(wp[k], 1) * s_1);
          }
        }
      }
    }
  }
  const uint16_t* xt = p.q + tok * p.q_tok_stride;
  uint16_t* yt = p.q_out + tok * p.H * p.d;
  const float eps = static_cast<float>(p.eps), inv_d = 1.0f / static_cast<float>(p.d);
  const int lane = threadIdx.x & 31;
  // A pass's rows into a slot: each lane a unit of 16 bytes of each 512, wherever its row is.
  auto fetch = [&](int h, uint32_t slot) {
#pragma unroll
    for (int i = 0; i < 2 * GPL; ++i) {
      const int u = lane + 32 * i, row = u / (2 * LPR * GPL), at = u - row * (2 * LPR * GPL);
      if (h + row < h1 && 8 * at < p.d) cp_async_16(slot + 16 * u, xt + (h + row) * p.q_head_stride + 8 * at);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) fetch(h0 + i * kRows, ring + i * kSlot);  // (none behind h1)
  uint32_t slot = ring;
#pragma unroll 1
  for (int hb = h0; hb < h1; hb += kRows) {
    cp_async_wait<kDepth - 1>();
    __syncwarp();
    const uint32_t row = slot + sub * (32 * LPR * GPL);
    uint32_t x[GPL][8], xp[GPL][8];
#pragma unroll
    for (int g = 0; g < GPL; ++g) {
      const int c0 = (l + LPR * g) * kGroup;
      uint4 a = make_uint4(0, 0, 0, 0), b = a, e = a, f = a;
      if (there[g]) {
        a = lds_v4(row + 2 * c0);
        b = lds_v4(row + 2 * c0 + 16);
      }
      if (kPairs == kHalves && rot[g]) {
        bool second;
        e = lds_v4(row + 2 * partner_unit(p, c0, second));
        f = lds_v4(row + 2 * partner_unit(p, c0 + 8, second));
      }
      x[g][0] = a.x; x[g][1] = a.y; x[g][2] = a.z; x[g][3] = a.w;
      x[g][4] = b.x; x[g][5] = b.y; x[g][6] = b.z; x[g][7] = b.w;
      xp[g][0] = e.x; xp[g][1] = e.y; xp[g][2] = e.z; xp[g][3] = e.w;
      xp[g][4] = f.x; xp[g][5] = f.y; xp[g][6] = f.z; xp[g][7] = f.w;
    }
    uint64_t s2 = 0;
#pragma unroll
    for (int g = 0; g < GPL; ++g)
#pragma unroll
      for (int k = 0; k < 8; ++k) s2 = fma2(widen2(x[g][k]), widen2(x[g][k]), s2);
    float ss, s1;
    unpack2(s2, ss, s1);
    ss += s1;
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(fmaf(ss, inv_d, eps));
    const uint64_t r2 = pack2(r, r);
    __syncwarp();  // (every lane has read the slot; a row may be written over itself: it is here already)
    fetch(hb + kDepth * kRows, slot);
    slot = slot + kSlot == ring + kDepth * kSlot ? ring : slot + kSlot;
    const int h = hb + sub;
#pragma unroll
    for (int g = 0; g < GPL; ++g) {
      if (!there[g] || h >= h1) continue;
      // (outside the rotated channels Q is 0, but 0 times an infinite neighbour would be NaN: two zeros instead)
      const uint32_t swap = rot[g] ? 0x1032u : 0x4444u;
      uint32_t y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint64_t t = mul2(widen2(x[g][k]), P[g][k]);
        if (kPairs == kNeighbours) t = fma2(widen2(__byte_perm(x[g][k], 0, swap)), Q[g][k], t);
        if (kPairs == kHalves) t = fma2(widen2(xp[g][k]), Q[g][k], t);
        float y0, y1;
        unpack2(mul2(t, r2), y0, y1);
        y[k] = f32x2_to_bf16x2(y0, y1);
      }
      uint16_t* out = yt + static_cast<int64_t>(h) * p.d + (l + LPR * g) * kGroup;
      *reinterpret_cast<uint4*>(out) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(out + 8) = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------------------
// KV rows
// ---------------------------------------------------------------------------------------
constexpr float kLeastR = 0x1p-120f;  // below it r as fp32 loses bits that the quick forms count on
// v: the quick form of a rotated channel; mag_r: the magnitudes of its two terms
FP4KV_DEV bool near_border(float v, float mag_r, float units) {
  const int off = static_cast<int>(__float_as_uint(v) & 0xffffu) - 0x8000;
  return !(static_cast<float>(abs(off)) * fabsf(v) > units * mag_r);  // (also where v is NaN, as of two infinite terms)
}
FP4KV_DEV uint32_t add_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A finished group to where it goes.
FP4KV_DEV void store_group(const NormRopeParams& p, int64_t tok, int64_t dst, int gi, const uint32_t (&y)[8]) {
  if (p.kv_out) {
    uint16_t* out = p.kv_out + tok * p.d + gi * kGroup;
    *reinterpret_cast<uint4*>(out) = make_uint4(y[0], y[1], y[2], y[3]);
    *reinterpret_cast<uint4*>(out + 8) = make_uint4(y[4], y[5], y[6], y[7]);
  }
  if (dst >= 0) {
    uint2 pk;
    uint32_t sc;
    quant_group(y, pk, sc);
    *reinterpret_cast<uint2*>(p.packed + dst * (p.d / 2) + gi * 8) = pk;
    p.scales[dst * (p.d / kGroup) + gi] = static_cast<uint8_t>(sc);
  }
}
// A rotated group of channels [c0, +16) of a row; the whole warp calls it (lanes with nothing to do: !on).
template <int kPairs>
FP4KV_DEV void rotated_group(const NormRopeParams& p, bool on, int64_t tok, int64_t dst, int64_t pos, int c0, double rd) {
  const uint16_t* xr = p.kv + tok * p.kv_stride;
  const int hr = p.rope_dim / 2, j0 = c0 - (p.d - p.rope_dim);
  uint32_t x[8], w[8], xp[8], wp[8];
  float co[16], si[16];  // kNeighbours: of pair k; kHalves: of channel k
  bool second[2] = {false, false};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint4 a = make_uint4(0, 0, 0, 0), b = make_uint4(kOnes, kOnes, kOnes, kOnes), e = a, f = b;
    float4 c[2] = {}, s[2] = {};
    if (on) {
      a = ld_v4(xr + c0 + 8 * u);
      if (p.kv_weight) b = ld_v4(p.kv_weight + c0 + 8 * u);
      int jj = j0 / 2 + 4 * u;
      if (kPairs == kHalves) {
        const int cp = partner_unit(p, c0 + 8 * u, second[u]);
        e = ld_v4(xr + cp);
        if (p.kv_weight) f = ld_v4(p.kv_weight + cp);
        jj = j0 + 8 * u - (second[u] ? hr : 0);
      }
      const float4* cs = reinterpret_cast<const float4*>(p.cos_sin + pos * p.rope_dim + jj);
      const float4* sn = reinterpret_cast<const float4*>(p.cos_sin + pos * p.rope_dim + hr + jj);
      c[0] = cs[0];
      s[0] = sn[0];
      if (kPairs == kHalves) {
        c[1] = cs[1];
        s[1] = sn[1];
      }
    }
    x[4 * u] = a.x; x[4 * u + 1] = a.y; x[4 * u + 2] = a.z; x[4 * u + 3] = a.w;
    w[4 * u] = b.x; w[4 * u + 1] = b.y; w[4 * u + 2] = b.z; w[4 * u + 3] = b.w;
    xp[4 * u] = e.x; xp[4 * u + 1] = e.y; xp[4 * u + 2] = e.z; xp[4 * u + 3] = e.w;
    wp[4 * u] = f.x; wp[4 * u + 1] = f.y; wp[4 * u + 2] = f.z; wp[4 * u + 3] = f.w;
    constexpr int n = kPairs == kHalves ? 8 : 4;
#pragma unroll
    for (int i = 0; i < n / 4; ++i) {
      co[n * u + 4 * i] = c[i].x; co[n * u + 4 * i + 1] = c[i].y; co[n * u + 4 * i + 2] = c[i].z; co[n * u + 4 * i + 3] = c[i].w;
      si[n * u + 4 * i] = s[i].x; si[n * u + 4 * i + 1] = s[i].y; si[n * u + 4 * i + 2] = s[i].z; si[n * u + 4 * i + 3] = s[i].w;
    }
  }
  __syncwarp();  // every lane has its partners: a row may be written over itself
  if (!on) return;
  const float rf = static_cast<float>(rd), wide = rf < kLeastR ? INFINITY : 6.0f;
  // me c + other s (s with its sign)
  auto turn = [&](float me, float other, float c, float s) -> uint32_t {
    const float os = other * s;
    const float v = fmaf(me, c, os) * rf;
    if (near_border(v, (fabsf(me * c) + fabsf(os)) * rf, wide))
      return f64_to_bf16(fma(static_cast<double>(me), static_cast<double>(c), static_cast<double>(other) * s) * rd);
    return f32_to_bf16(v);
  };
  uint32_t y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float a = half_of(x[k], 0) * half_of(w[k], 0), b = half_of(x[k], 1) * half_of(w[k], 1);
    if (kPairs == kNeighbours) {
      y[k] = turn(a, b, co[k], -si[k]) | (turn(b, a, co[k], si[k]) << 16);
    } else {
      const float ap = half_of(xp[k], 0) * half_of(wp[k], 0), bp = half_of(xp[k], 1) * half_of(wp[k], 1);
      const bool sec = second[k >> 2];
      y[k] = turn(a, ap, co[2 * k], sec ? si[2 * k] : -si[2 * k]) |
             (turn(b, bp, co[2 * k + 1], sec ? si[2 * k + 1] : -si[2 * k + 1]) << 16);
    }
  }
  store_group(p, tok, dst, c0 / kGroup, y);
}

// kPasses passes of 32 / LPR rows by one warp, from row row0 on.
template <int LPR, int GPL, int kPairs, int kPasses>
FP4KV_DEV void kv_rows(const NormRopeParams& p, int64_t row0) {
  constexpr int kRows = 32 / LPR, kBatch = kRows * kPasses;
  static_assert(kBatch <= 32, "a lane per row");
  const int lane = threadIdx.x & 31, l = lane & (LPR - 1), sub = lane / LPR;
  const int groups = p.d / kGroup, plain = (p.d - p.rope_dim) / kGroup;
  // lane i: row i's place, position and r
  int64_t my_dst = -1, my_pos = 0;
  bool my_live = false;
  if (lane < kBatch && row0 + lane < p.n_tokens) {
    my_live = true;
    if (kPairs != kNone) {
      my_pos = p.positions[row0 + lane];
      my_live = my_pos >= 0 && my_pos < p.max_pos;
    }
    if (my_live && p.packed) {
      my_dst = p.dst_row ? p.dst_row[row0 + lane] : row0 + lane;
      if (my_dst >= p.cap_rows) my_dst = -1;
    }
  }
  const uint32_t live_rows = __ballot_sync(0xffffffffu, my_live);
  uint32_t x[kPasses][GPL][8];
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
#pragma unroll
    for (int g = 0; g < GPL; ++g) {
      const int r = i * kRows + sub, c0 = (l + LPR * g) * kGroup;
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (((live_rows >> r) & 1) && c0 < p.d) {
        const uint16_t* xr = p.kv + (row0 + r) * p.kv_stride + c0;
        a = ld_v4(xr);
        b = ld_v4(xr + 8);
      }
      x[i][g][0] = a.x; x[i][g][1] = a.y; x[i][g][2] = a.z; x[i][g][3] = a.w;
      x[i][g][4] = b.x; x[i][g][5] = b.y; x[i][g][6] = b.z; x[i][g][7] = b.w;
    }
  double my_r = 0.0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    double s0 = 0.0, s1 = 0.0;
#pragma unroll
    for (int g = 0; g < GPL; ++g)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // |x| as fp64 by its bits (a zero becomes 2^-127, whose square is nothing beside eps; an
        // infinity or NaN at least 2^128: below)
        const double a = __hiloint2double(static_cast<int>(((x[i][g][k] & 0x7fffu) << 13) + (896u << 20)), 0);
        const double b = __hiloint2double(static_cast<int>(((x[i][g][k] >> 3) & 0x0fffe000u) + (896u << 20)), 0);
        s0 = fma(a, a, s0);
        s1 = fma(b, b, s1);
      }
    double ss = s0 + s1;
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // (row i * kRows + k's sum lies in the lanes from k * LPR on)
    ss = __shfl_sync(0xffffffffu, ss, (lane & (kRows - 1)) * LPR);
    if (lane / kRows == i) my_r = ss;
  }
  if (__any_sync(0xffffffffu, my_r >= 0x1p255)) {  // a row that isn't finite, or one near the type's end
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int g = 0; g < GPL; ++g)
#pragma unroll
        for (int k = 0; k < 8; ++k) m = __vmaxu2(m, x[i][g][k] & 0x7fff7fffu);
      m = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = __shfl_sync(0xffffffffu, m, (lane & (kRows - 1)) * LPR);
      if (lane / kRows == i && m >= 0x7f80u) my_r = __hiloint2double(m == 0x7f80u ? 0x7ff00000 : 0x7ff80000, 0);
    }
  }
  my_r = rsqrt(my_r / p.d + p.eps);
  uint32_t w[GPL][8];
#pragma unroll
  for (int g = 0; g < GPL; ++g) {
    const int c0 = (l + LPR * g) * kGroup;
    uint4 a = make_uint4(kOnes, kOnes, kOnes, kOnes), b = a;
    if (p.kv_weight && c0 < p.d) {
      a = ld_v4(p.kv_weight + c0);
      b = ld_v4(p.kv_weight + c0 + 8);
    }
    w[g][0] = a.x; w[g][1] = a.y; w[g][2] = a.z; w[g][3] = a.w;
    w[g][4] = b.x; w[g][5] = b.y; w[g][6] = b.z; w[g][7] = b.w;
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + sub;
    const double rd = __shfl_sync(0xffffffffu, my_r, r);
    const int64_t dst = __shfl_sync(0xffffffffu, my_dst, r);
    const float rf = static_cast<float>(rd);
#pragma unroll
    for (int g = 0; g < GPL; ++g) {
      const int gi = l + LPR * g;
      if (!((live_rows >> r) & 1) || gi >= plain) continue;
      uint32_t y[8], near = rf < kLeastR ? 0 : 0xffffffffu;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v0 = half_of(x[i][g][k], 0) * half_of(w[g][k], 0) * rf, v1 = half_of(x[i][g][k], 1) * half_of(w[g][k], 1) * rf;
        y[k] = f32x2_to_bf16x2(v0, v1);
        // the low halves, 0 .. 6 where within 3 units of a rounding border (0x8000)
        near = __vminu2(near, add_u16x2(__byte_perm(__float_as_uint(v0), __float_as_uint(v1), 0x5410), 0x80038003u));
      }
      if (min(near & 0xffffu, near >> 16) <= 6u) {  // too near for fp32 to tell
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float u0 = half_of(x[i][g][k], 0) * half_of(w[g][k], 0), u1 = half_of(x[i][g][k], 1) * half_of(w[g][k], 1);
          y[k] = f64_to_bf16(static_cast<double>(u0) * rd) | (f64_to_bf16(static_cast<double>(u1) * rd) << 16);
        }
      }
      store_group(p, row0 + r, dst, gi, y);
    }
  }
  if (kPairs != kNone) {
    // the rotated groups, one to a lane; a row's are all done in one step
    const int rg = groups - plain, rows = 32 / rg;
#pragma unroll 1
    for (int first = 0; first < kBatch; first += rows) {
      const int q = lane / rg, r = first + q;
      const bool mine = q < rows && r < kBatch;
      const int from = mine ? r : 0;
      const double rd = __shfl_sync(0xffffffffu, my_r, from);
      const int64_t dst = __shfl_sync(0xffffffffu, my_dst, from), pos = __shfl_sync(0xffffffffu, my_pos, from);
      rotated_group<kPairs>(p, mine && ((live_rows >> from) & 1), row0 + from, dst, pos, (plain + lane - q * rg) * kGroup, rd);
    }
  }
}

// Rows of a KV warp: eight (four of more than 512 channels), whose rotated groups share the lanes and whose
// loads overlap; where that leaves SMs without a warp or two, as few as a pass has. Rows of 512 (not in L2, calls
// replayed from a graph), one pass against eight: 1,024 rows 5.1 against 9.7 us, 4,096 12.6 against 11.6, 9,472
// 23.2 against 12.0, 131,072 286 against 98.
template <int LPR, int GPL>
constexpr int kKvPasses = (GPL == 1 ? 8 : 4) * LPR / 32;

template <int LPR, int GPL, int kPairs, int kPasses>
__global__ void __launch_bounds__(kThreads) k_kv_norm_rope(const NormRopeParams p) {
  griddep_wait();
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * (kPasses * 32 / LPR);
  if (row0 < p.n_tokens) kv_rows<LPR, GPL, kPairs, kPasses>(p, row0);
}

// The KV rows' blocks (more arithmetic each) come first, then the query heads', `heads` of a token per warp.
template <int LPR, int GPL, int kPairs>
__global__ void __launch_bounds__(kThreads, GPL == 1 ? 2 : 1) k_qkv_norm_rope(const NormRopeParams p, uint32_t kv_blocks, int heads) {
  __shared__ __align__(128) uint8_t ring[kThreads / 32][4096];
  griddep_wait();
  if (blockIdx.x < kv_blocks) {
    const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * (32 / LPR);
    if (row0 < p.n_tokens) kv_rows<LPR, GPL, kPairs, 1>(p, row0);
    return;
  }
  const int64_t unit = static_cast<int64_t>(blockIdx.x - kv_blocks) * (kThreads / 32) + (threadIdx.x >> 5);
  const int parts = (p.H + heads - 1) / heads;
  const int64_t tok = unit / parts;
  if (tok >= p.n_tokens) return;
  const int h0 = static_cast<int>(unit - tok * parts) * heads;
  query_heads<LPR, GPL, kPairs>(p, smem_u32(ring[threadIdx.x >> 5]), tok, h0, min(h0 + heads, p.H));
}

// (what takes the GPU no longer than the host is launched plainly)
bool few_rows(int64_t rows, int num_sms) { return rows < int64_t(num_sms) * 64; }

template <int LPR, int GPL, int kPairs, int kPasses>
cudaError_t launch_kv(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
  const int64_t per_block = kPasses * (32 / LPR) * (kThreads / 32);
  const int64_t blocks = (p.n_tokens + per_block - 1) / per_block;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_sized(few_rows(p.n_tokens, num_sms), k_kv_norm_rope<LPR, GPL, kPairs, kPasses>, dim3(static_cast<unsigned>(blocks)),
                      dim3(kThreads), stream, p);
}

template <int LPR, int GPL, int kPairs>
cudaError_t launch(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kRows = 32 / LPR;
  const int64_t per_block = kRows * (kThreads / 32);
  const int64_t kv_blocks = p.kv ? (p.n_tokens + per_block - 1) / per_block : 0;
  if (!p.q) {
    constexpr int kMany = kKvPasses<LPR, GPL>;
    return p.n_tokens >= int64_t(num_sms) * 2 * kMany * kRows ? launch_kv<LPR, GPL, kPairs, kMany>(p, num_sms, stream)
                                                              : launch_kv<LPR, GPL, kPairs, 1>(p, num_sms, stream);
  }
  // Heads per warp: one pass (kRows) where there are few rows, up to 16 passes where that leaves every SM
  // 8 warps (as many as its ring of rows needs, and the coefficients are formed once for all of them). 64
  // heads of 512 without KV rows (not in L2, calls replayed from a graph), 1, 4 and 16 a warp: 32 tokens 4.3, 5.1,
  // 8.9 us, 128 tokens 12.0, 7.1, 9.6, 512 tokens 37.3, 18.7, 14.9, 8,192 tokens 554, 237, 170.
  int heads = kRows;
  while (heads < 16 * kRows && heads < p.H && p.n_tokens * p.H >= int64_t(2) * heads * 8 * num_sms) heads *= 2;
  const int64_t units = p.n_tokens * ((p.H + heads - 1) / heads);
  const int64_t blocks = kv_blocks + (units + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_sized(few_rows(p.n_tokens * (p.H + 1) / kRows, num_sms), k_qkv_norm_rope<LPR, GPL, kPairs>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), stream,
                      p, static_cast<uint32_t>(kv_blocks), heads);
}

template <int kPairs>
cudaError_t launch_width(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
  if (p.d <= 128) return launch<8, 1, kPairs>(p, num_sms, stream);
  if (p.d <= 256) return launch<16, 1, kPairs>(p, num_sms, stream);
  if (p.d <= 512) return launch<32, 1, kPairs>(p, num_sms, stream);
  return launch<32, 2, kPairs>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_qkv_norm_rope(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
  if (p.n_tokens == 0 || (!p.q && !p.kv)) return cudaSuccess;
  if (p.rope_dim == 0) return launch_width<kNone>(p, num_sms, stream);
  return p.rope_half ? launch_width<kHalves>(p, num_sms, stream) : launch_width<kNeighbours>(p, num_sms, stream);
}

}  // namespace fp4kv
