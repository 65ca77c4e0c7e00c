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
// channels P = w, Q = 0), so no lane waits for the rotated ones. fp32, rounded once to bf16. The next
// head's row is on its way while one is computed.
//
// The KV row: y's nearest fp32 value is rounded to bf16 and that is quantised, so the cache holds
// exactly what kv_quant_fp4 makes of kv_out. A code is decided by which side of a border a value
// falls on, so y must not be off by even an fp32 step: sum x^2 and r are held in fp64. A quick fp32 form
// v of y is off by at most 4 x 2^-24 of mag, the sum of the magnitudes of its two terms (the product and
// the sum rounded, r rounded, one product; one term and 2 x 2^-24 outside the rotated channels). Where v
// lies nearer than that (6, or 3 units) to a bf16 rounding border, y is formed in fp64: one value in
// thousands. (All rotated channels in fp64: 145 us instead of the figure below for 131,072 rows.)
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

// two fp32 at once
FP4KV_DEV uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
FP4KV_DEV void unpack2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
FP4KV_DEV uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
FP4KV_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
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
// One group's x (words 0-7) and, for pairs of halves, its partners (8-15).
template <int kPairs>
FP4KV_DEV void load_group(const NormRopeParams& p, const uint16_t* xr, int c0, bool rot, uint32_t (&x)[8], uint32_t (&xp)[8]) {
  const uint4 a = ld_v4(xr + c0), b = ld_v4(xr + c0 + 8);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  if (kPairs == kHalves) {
    uint4 e = make_uint4(0, 0, 0, 0), f = e;
    if (rot) {
      bool second;
      e = ld_v4(xr + partner_unit(p, c0, second));
      f = ld_v4(xr + partner_unit(p, c0 + 8, second));
    }
    xp[0] = e.x; xp[1] = e.y; xp[2] = e.z; xp[3] = e.w;
    xp[4] = f.x; xp[5] = f.y; xp[6] = f.z; xp[7] = f.w;
  }
}

template <int LPR, int GPL, int kPairs>
FP4KV_DEV void query_heads(const NormRopeParams& p, int64_t tok, int h0, int h1) {
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
  uint32_t x[GPL][8] = {}, xp[GPL][8] = {};
  if (h0 + sub < h1)
#pragma unroll
    for (int g = 0; g < GPL; ++g)
      if (there[g]) load_group<kPairs>(p, xt + (h0 + sub) * p.q_head_stride, (l + LPR * g) * kGroup, rot[g], x[g], xp[g]);
#pragma unroll 1
  for (int h = h0 + sub; h - sub < h1; h += kRows) {
    uint32_t nx[GPL][8] = {}, np[GPL][8] = {};  // the next head's
    if (h + kRows < h1)
#pragma unroll
      for (int g = 0; g < GPL; ++g)
        if (there[g]) load_group<kPairs>(p, xt + (h + kRows) * p.q_head_stride, (l + LPR * g) * kGroup, rot[g], nx[g], np[g]);
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
    __syncwarp();  // every lane has its row's partners: a row may be written over itself
#pragma unroll
    for (int g = 0; g < GPL; ++g) {
      if (!there[g] || h >= h1) continue;
      uint32_t y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint64_t t = mul2(widen2(x[g][k]), P[g][k]);
        if (kPairs == kNeighbours) t = fma2(widen2(__byte_perm(x[g][k], 0, 0x1032)), Q[g][k], t);
        if (kPairs == kHalves) t = fma2(widen2(xp[g][k]), Q[g][k], t);
        float y0, y1;
        unpack2(mul2(t, r2), y0, y1);
        y[k] = f32x2_to_bf16x2(y0, y1);
      }
      uint16_t* out = yt + static_cast<int64_t>(h) * p.d + (l + LPR * g) * kGroup;
      *reinterpret_cast<uint4*>(out) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(out + 8) = make_uint4(y[4], y[5], y[6], y[7]);
    }
#pragma unroll
    for (int g = 0; g < GPL; ++g)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[g][k] = nx[g][k];
        xp[g][k] = np[g][k];
      }
  }
}

// ---------------------------------------------------------------------------------------
// KV rows
// ---------------------------------------------------------------------------------------
// u: the channel's value over r, mag: the sum of its terms' magnitudes (at least |u|)
FP4KV_DEV bool near_border(float v, float mag_r) {
  const int off = static_cast<int>(__float_as_uint(v) & 0xffffu) - 0x8000;
  return static_cast<float>(abs(off)) * fabsf(v) <= 6.0f * mag_r;
}

template <int LPR, int GPL, int kPairs>
FP4KV_DEV void kv_row(const NormRopeParams& p, int64_t tok) {
  const int l = threadIdx.x & (LPR - 1);
  const int groups = p.d / kGroup;
  bool live = tok < p.n_tokens;
  int64_t pos = 0;
  if (kPairs != kNone && live) {
    pos = p.positions[tok];
    live = pos >= 0 && pos < p.max_pos;
  }
  int64_t dst = -1;
  if (live && p.packed) {
    dst = p.dst_row ? p.dst_row[tok] : tok;
    if (dst >= p.cap_rows) dst = -1;
  }
  const uint16_t* xr = p.kv + tok * p.kv_stride;
  uint32_t x[GPL][8], xp[GPL][8];
  double s0 = 0.0, s1 = 0.0;
#pragma unroll
  for (int g = 0; g < GPL; ++g) {
    const int c0 = (l + LPR * g) * kGroup;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[g][k] = xp[g][k] = 0;
    if (live && c0 < p.d) load_group<kPairs>(p, xr, c0, kPairs != kNone && c0 >= p.d - p.rope_dim, x[g], xp[g]);
  }
#pragma unroll
  for (int g = 0; g < GPL; ++g)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // |x| as fp64 by its bits (a zero becomes 2^-127, whose square is nothing beside eps)
      const double a = __hiloint2double(static_cast<int>(((x[g][k] & 0x7fffu) << 13) + (896u << 20)), 0);
      const double b = __hiloint2double(static_cast<int>(((x[g][k] >> 3) & 0x0fffe000u) + (896u << 20)), 0);
      s0 = fma(a, a, s0);
      s1 = fma(b, b, s1);
    }
  double ss = s0 + s1;
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const double rd = rsqrt(ss / p.d + p.eps);
  const float rf = static_cast<float>(rd);
  __syncwarp();  // every lane has its row's partners: a row may be written over itself
#pragma unroll
  for (int g = 0; g < GPL; ++g) {
    const int gi = l + LPR * g, c0 = gi * kGroup;
    if (!live || gi >= groups) continue;
    uint32_t y[8];
    uint32_t w[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint4 wv = p.kv_weight ? ld_v4(p.kv_weight + c0 + 8 * u) : make_uint4(kOnes, kOnes, kOnes, kOnes);
      w[4 * u] = wv.x; w[4 * u + 1] = wv.y; w[4 * u + 2] = wv.z; w[4 * u + 3] = wv.w;
    }
    if (kPairs != kNone && c0 >= p.d - p.rope_dim) {
      const float* cs = p.cos_sin + pos * p.rope_dim;
      const int hr = p.rope_dim / 2, j0 = c0 - (p.d - p.rope_dim);
      // me c + other s (s with its sign)
      auto turn = [&](float me, float other, float co, float si) -> uint32_t {
        const float os = other * si;
        const float v = fmaf(me, co, os) * rf;
        if (near_border(v, (fabsf(me * co) + fabsf(os)) * rf))
          return f64_to_bf16(fma(static_cast<double>(me), static_cast<double>(co), static_cast<double>(other) * si) * rd);
        return f32_to_bf16(v);
      };
      if (kPairs == kNeighbours) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float co = cs[j0 / 2 + k], si = cs[hr + j0 / 2 + k];
          const float a = half_of(x[g][k], 0) * half_of(w[k], 0), b = half_of(x[g][k], 1) * half_of(w[k], 1);
          y[k] = turn(a, b, co, -si) | (turn(b, a, co, si) << 16);
        }
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          bool second;
          const int cp = partner_unit(p, c0 + 8 * u, second);
          const int jj = j0 + 8 * u - (second ? hr : 0);
          const uint4 pw = p.kv_weight ? ld_v4(p.kv_weight + cp) : make_uint4(kOnes, kOnes, kOnes, kOnes);
          const uint32_t wp[4] = {pw.x, pw.y, pw.z, pw.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t e[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float si = cs[hr + jj + 2 * k + i];
              e[i] = turn(half_of(x[g][4 * u + k], i) * half_of(w[4 * u + k], i), half_of(xp[g][4 * u + k], i) * half_of(wp[k], i),
                          cs[jj + 2 * k + i], second ? si : -si);
            }
            y[4 * u + k] = e[0] | (e[1] << 16);
          }
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float u0 = half_of(x[g][k], 0) * half_of(w[k], 0), u1 = half_of(x[g][k], 1) * half_of(w[k], 1);
        const float v0 = u0 * rf, v1 = u1 * rf;
        y[k] = f32x2_to_bf16x2(v0, v1);
        // too near a rounding border for fp32 to tell
        const bool n0 = (__float_as_uint(v0) & 0xffffu) - 0x7ffdu <= 6u, n1 = (__float_as_uint(v1) & 0xffffu) - 0x7ffdu <= 6u;
        if (n0 || n1) {
          if (n0) y[k] = (y[k] & 0xffff0000u) | f64_to_bf16(static_cast<double>(u0) * rd);
          if (n1) y[k] = (y[k] & 0xffffu) | (f64_to_bf16(static_cast<double>(u1) * rd) << 16);
        }
      }
    }
    if (p.kv_out) {
      uint16_t* out = p.kv_out + tok * p.d + c0;
      *reinterpret_cast<uint4*>(out) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(out + 8) = make_uint4(y[4], y[5], y[6], y[7]);
    }
    if (dst >= 0) {
      uint2 pk;
      uint32_t sc;
      quant_group(y, pk, sc);
      *reinterpret_cast<uint2*>(p.packed + dst * (p.d / 2) + gi * 8) = pk;
      p.scales[dst * groups + gi] = static_cast<uint8_t>(sc);
    }
  }
}

template <int LPR, int GPL, int kPairs>
__global__ void __launch_bounds__(kThreads) k_kv_norm_rope(const NormRopeParams p) {
  constexpr int kRows = 32 / LPR;  // rows of a warp
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  kv_row<LPR, GPL, kPairs>(p, warp * kRows + (threadIdx.x & 31) / LPR);
}

// The KV rows' blocks (more arithmetic each) come first, then the query heads', `heads` of a token per warp.
template <int LPR, int GPL, int kPairs>
__global__ void __launch_bounds__(kThreads, GPL == 1 ? 2 : 1) k_qkv_norm_rope(const NormRopeParams p, uint32_t kv_blocks, int heads) {
  constexpr int kRows = 32 / LPR;
  if (blockIdx.x < kv_blocks) {
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (warp * kRows < p.n_tokens) kv_row<LPR, GPL, kPairs>(p, warp * kRows + (threadIdx.x & 31) / LPR);
    return;
  }
  const int64_t unit = static_cast<int64_t>(blockIdx.x - kv_blocks) * (kThreads / 32) + (threadIdx.x >> 5);
  const int parts = (p.H + heads - 1) / heads;
  const int64_t tok = unit / parts;
  if (tok >= p.n_tokens) return;
  const int h0 = static_cast<int>(unit - tok * parts) * heads;
  query_heads<LPR, GPL, kPairs>(p, tok, h0, min(h0 + heads, p.H));
}

template <int LPR, int GPL, int kPairs>
cudaError_t launch(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kRows = 32 / LPR;
  const int64_t per_block = kRows * (kThreads / 32);
  const int64_t kv_blocks = p.kv ? (p.n_tokens + per_block - 1) / per_block : 0;
  if (!p.q) {
    if (kv_blocks > 0x7fffffff) return cudaErrorInvalidValue;
    k_kv_norm_rope<LPR, GPL, kPairs><<<static_cast<unsigned>(kv_blocks), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  // heads per warp: one pass (kRows) where there are few rows, up to 16 passes where that leaves every SM
  // 32 warps to run
  int heads = kRows;
  while (heads < 16 * kRows && heads < p.H && p.n_tokens * p.H >= int64_t(2) * heads * 32 * num_sms) heads *= 2;
  const int64_t units = p.n_tokens * ((p.H + heads - 1) / heads);
  const int64_t blocks = kv_blocks + (units + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  k_qkv_norm_rope<LPR, GPL, kPairs>
      <<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p, static_cast<uint32_t>(kv_blocks), heads);
  return cudaGetLastError();
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
