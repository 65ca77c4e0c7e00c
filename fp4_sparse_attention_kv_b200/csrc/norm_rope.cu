// qkv_norm_rope_fp4: RMS norm and position rotation of every query head and of the token's KV row
// in one launch; the KV row is quantised into the FP4 cache as it is made.
//
// For a row x of d channels with weight w (or 1):  r = 1 / sqrt(sum x^2 / d + eps),  u = x w;
// y_i = u_i r for the first d - rope_dim channels; the last rope_dim are rotated in pairs (a, b) by
// the token's angles: y_a = (u_a c - u_b s) r, y_b = (u_b c + u_a s) r. Pairs are neighbours
// (2j, 2j + 1), or (j, j + rope_dim / 2).
//
// Numerics:
//  * queries: fp32, rounded once to bf16. u = x w is exact in fp32 (two 8-bit significands).
//  * the KV row: y's nearest fp32 value is rounded to bf16 and that is quantised, so the cache holds
//    exactly what kv_quant_fp4 makes of kv_out. A code is decided by which side of a border a value
//    falls on, so y must not be off by even an fp32 step: sum x^2 and r are held in fp64, and y is
//    formed in fp64 where a quick fp32 form of it lies within 3 units in the last place of a bf16
//    rounding border (r rounded, 2^-24, and one product, 2^-24: at most 2 units), and for the
//    rotated channels, whose difference can cancel.
// Memory: LPR lanes share a row, each with GPL groups of 16 channels (two 16-byte loads a group).
#include "fp4kv_common.cuh"
#include "fp4kv_launch.h"
#include "fp4kv_quant.cuh"
#include "fp4kv_sm100.cuh"

namespace fp4kv {
namespace {

constexpr int kThreads = 256;

FP4KV_DEV uint32_t f32_to_bf16(float f) {  // round to nearest even
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
  return r;
}
// (fp64 to fp32 to bf16, each to nearest even)
FP4KV_DEV uint32_t f64_to_bf16(double y) { return f32_to_bf16(__double2float_rn(y)); }
FP4KV_DEV float half_of(uint32_t w, int k) {  // channel k (0 low, 1 high) of a bf16 pair
  return __uint_as_float(k ? (w & 0xffff0000u) : (w << 16));
}
FP4KV_DEV uint4 ld_v4(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// The 8 channels [c0, c0 + 8) of a rotated row, in the product's type: calls f(k, t) with the
// rotated, not yet normed value t of channel c0 + k.
template <typename Real, typename F>
FP4KV_DEV void rotate8(const NormRopeParams& p, const uint16_t* xr, const uint16_t* w, const float* cs, int c0,
                       const uint32_t (&x)[4], const uint32_t (&wt)[4], F f) {
  const int j0 = c0 - (p.d - p.rope_dim), hr = p.rope_dim / 2;
  if (!p.rope_half) {
    const float4 c4 = *reinterpret_cast<const float4*>(cs + j0 / 2);
    const float4 s4 = *reinterpret_cast<const float4*>(cs + hr + j0 / 2);
    const float co[4] = {c4.x, c4.y, c4.z, c4.w}, si[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Real a = half_of(x[k], 0) * half_of(wt[k], 0), b = half_of(x[k], 1) * half_of(wt[k], 1);
      f(2 * k, fma(a, static_cast<Real>(co[k]), -(b * static_cast<Real>(si[k]))));
      f(2 * k + 1, fma(b, static_cast<Real>(co[k]), a * static_cast<Real>(si[k])));
    }
  } else {
    const bool second = j0 >= hr;
    const int jj = second ? j0 - hr : j0, cp = second ? c0 - hr : c0 + hr;  // the partners' channels
    const uint4 px = ld_v4(xr + cp);
    const uint4 pw = w ? ld_v4(w + cp) : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    const uint32_t xp[4] = {px.x, px.y, px.z, px.w}, wp[4] = {pw.x, pw.y, pw.z, pw.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const Real me = half_of(x[k >> 1], k & 1) * half_of(wt[k >> 1], k & 1);
      const Real other = half_of(xp[k >> 1], k & 1) * half_of(wp[k >> 1], k & 1);
      const Real co = cs[jj + k], si = cs[hr + jj + k];
      f(k, second ? fma(me, co, other * si) : fma(me, co, -(other * si)));
    }
  }
}

// One row: LPR lanes (lane l of the row: groups l, l + LPR, ...). kKv: the fp64 rules, the bf16
// row nullable, and the FP4 row at cache row `dst` (or none).
template <int LPR, int GPL, bool kKv>
FP4KV_DEV void row_pass(const NormRopeParams& p, const uint16_t* xr, const uint16_t* w, int64_t tok, bool live,
                        uint16_t* out, int64_t dst) {
  const int l = threadIdx.x & (LPR - 1);
  const int groups = p.d / kGroup;
  uint32_t x[GPL][8];
#pragma unroll
  for (int g = 0; g < GPL; ++g) {
    const int gi = l + LPR * g;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (live && gi < groups) {
      a = ld_v4(xr + gi * kGroup);
      b = ld_v4(xr + gi * kGroup + 8);
    }
    x[g][0] = a.x; x[g][1] = a.y; x[g][2] = a.z; x[g][3] = a.w;
    x[g][4] = b.x; x[g][5] = b.y; x[g][6] = b.z; x[g][7] = b.w;
  }
  double rd = 0.0;
  float rf;
  if (kKv) {
    double s0 = 0.0, s1 = 0.0;
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
    rd = rsqrt(ss / p.d + p.eps);
    rf = static_cast<float>(rd);
  } else {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int g = 0; g < GPL; ++g)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s0 = fmaf(half_of(x[g][k], 0), half_of(x[g][k], 0), s0);
        s1 = fmaf(half_of(x[g][k], 1), half_of(x[g][k], 1), s1);
      }
    float ss = s0 + s1;
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    rf = rsqrtf(ss / static_cast<float>(p.d) + static_cast<float>(p.eps));
  }
  const float* cs = p.rope_dim && live ? p.cos_sin + p.positions[tok] * p.rope_dim : nullptr;
  uint32_t y[GPL][8];
#pragma unroll
  for (int g = 0; g < GPL; ++g) {
    const int gi = l + LPR * g;
    if (!live || gi >= groups) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c0 = gi * kGroup + 8 * h;
      const uint4 wv = w ? ld_v4(w + c0) : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
      const uint32_t wt[4] = {wv.x, wv.y, wv.z, wv.w};
      const uint32_t xx[4] = {x[g][4 * h], x[g][4 * h + 1], x[g][4 * h + 2], x[g][4 * h + 3]};
      uint32_t e[8];
      if (c0 >= p.d - p.rope_dim) {
        if (kKv)
          rotate8<double>(p, xr, w, cs, c0, xx, wt, [&](int k, double t) { e[k] = f64_to_bf16(t * rd); });
        else
          rotate8<float>(p, xr, w, cs, c0, xx, wt, [&](int k, float t) { e[k] = f32_to_bf16(t * rf); });
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float u = half_of(xx[k >> 1], k & 1) * half_of(wt[k >> 1], k & 1);
          const float v = u * rf;
          e[k] = f32_to_bf16(v);
          if (kKv) {  // too near a rounding border for fp32 to tell
            const uint32_t off = (__float_as_uint(v) & 0xffffu) - 0x7ffdu;
            if (off <= 6u) e[k] = f64_to_bf16(static_cast<double>(u) * rd);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) y[g][4 * h + k] = e[2 * k] | (e[2 * k + 1] << 16);
    }
  }
  __syncwarp();  // every lane has read its partners: a row may be written over itself
#pragma unroll
  for (int g = 0; g < GPL; ++g) {
    const int gi = l + LPR * g;
    if (!live || gi >= groups) continue;
    if (out) {
      *reinterpret_cast<uint4*>(out + gi * kGroup) = make_uint4(y[g][0], y[g][1], y[g][2], y[g][3]);
      *reinterpret_cast<uint4*>(out + gi * kGroup + 8) = make_uint4(y[g][4], y[g][5], y[g][6], y[g][7]);
    }
    if (kKv && dst >= 0) {
      uint2 pk;
      uint32_t sc;
      quant_group(y[g], pk, sc);
      *reinterpret_cast<uint2*>(p.packed + dst * (p.d / 2) + gi * 8) = pk;
      p.scales[dst * groups + gi] = static_cast<uint8_t>(sc);
    }
  }
}

template <int LPR, int GPL>
__global__ void __launch_bounds__(kThreads) k_qkv_norm_rope(const NormRopeParams p, int64_t kv_warps, int64_t q_warps) {
  griddep_wait();
  constexpr int kRows = 32 / LPR;  // rows of a warp
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int sub = (threadIdx.x & 31) / LPR;
  // the KV rows (more arithmetic each) come first
  if (warp < kv_warps) {
    const int64_t tok = warp * kRows + sub;
    bool live = tok < p.n_tokens;
    if (live && p.rope_dim) live = p.positions[tok] >= 0 && p.positions[tok] < p.max_pos;
    int64_t dst = -1;
    if (live && p.packed) {
      dst = p.dst_row ? p.dst_row[tok] : tok;
      if (dst >= p.cap_rows) dst = -1;
    }
    row_pass<LPR, GPL, true>(p, p.kv + tok * p.kv_stride, p.kv_weight, tok, live,
                             p.kv_out ? p.kv_out + tok * p.d : nullptr, dst);
  } else if (warp < kv_warps + q_warps) {
    const int64_t row = (warp - kv_warps) * kRows + sub;
    const int64_t tok = row / p.H;
    const int64_t h = row - tok * p.H;
    bool live = tok < p.n_tokens;
    if (live && p.rope_dim) live = p.positions[tok] >= 0 && p.positions[tok] < p.max_pos;
    row_pass<LPR, GPL, false>(p, p.q + tok * p.q_tok_stride + h * p.q_head_stride, p.q_weight, tok, live,
                              p.q_out + row * p.d, -1);
  }
}

template <int LPR, int GPL>
cudaError_t launch(const NormRopeParams& p, cudaStream_t stream) {
  constexpr int kRows = 32 / LPR;
  const int64_t kv_warps = p.kv ? (p.n_tokens + kRows - 1) / kRows : 0;
  const int64_t q_warps = p.q ? (p.n_tokens * p.H + kRows - 1) / kRows : 0;
  const int64_t blocks = (kv_warps + q_warps + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(k_qkv_norm_rope<LPR, GPL>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), stream, p, kv_warps,
                    q_warps);
}

}  // namespace

cudaError_t launch_qkv_norm_rope(const NormRopeParams& p, cudaStream_t stream) {
  if (p.n_tokens == 0 || (!p.q && !p.kv)) return cudaSuccess;
  if (p.d <= 128) return launch<8, 1>(p, stream);
  if (p.d <= 256) return launch<16, 1>(p, stream);
  if (p.d <= 512) return launch<32, 1>(p, stream);
  return launch<32, 2>(p, stream);
}

}  // namespace fp4kv
