// tree_attn_decode: attention of a tree of drafted tokens over the FP4 cache.
//
// Token t of a sequence sees the prefix rows (all of them, or a selection) and the drafted rows of
// its mask: o = sum_j softmax_j(sm_scale q . v_j) v_j over those rows, lse = ln of the sum.
//
// One warp per query row (token, head), 16 channels per lane; a block dequantizes 16 rows at a
// time to fp32 in shared memory for its 8 query rows, each with a running maximum and sum.
#include "fp4kv_common.cuh"
#include "fp4kv_launch.h"
#include "fp4kv_quant.cuh"
#include "fp4kv_sm100.cuh"

namespace fp4kv {
namespace {

constexpr int kD = 512;
constexpr int kTileRows = 16;

__global__ void __launch_bounds__(256) k_tree_attn(const TreeAttnParams p) {
  __shared__ float tile[kTileRows][kD];
  __shared__ int64_t pos_s[kTileRows];
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  const int r = blockIdx.x * 8 + warp;
  const int nd = p.n_draft ? max(0, min(p.n_draft[b], p.T)) : p.T;
  const int t = r / p.H;
  const bool live = t < nd;
  const int64_t pre = max(int64_t(0), min(int64_t(p.prefix_lens[b]), p.cap));
  const int64_t n_sel = p.idx ? p.top_k : pre;
  const int64_t row = int64_t(b) * p.T * p.H + r;
  const uint64_t mask = live ? p.tree_mask[int64_t(b) * p.T + t] : 0;
  float q[16], o[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    q[k] = live ? bf16_bits_to_f32(p.q[row * kD + 128 * (k >> 2) + 4 * lane + (k & 3)]) * p.sm_scale : 0.0f;
    o[k] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t e0 = 0; e0 < n_sel + nd; e0 += kTileRows) {
    __syncthreads();
    if (threadIdx.x < kTileRows) {
      const int64_t e = e0 + threadIdx.x;
      int64_t pos = -1;
      if (e < n_sel) {
        pos = p.idx ? p.idx[int64_t(b) * p.top_k + e] : e;
        if (pos >= pre) pos = -1;
      } else if (e < n_sel + nd && pre + (e - n_sel) < p.cap) {
        pos = pre + (e - n_sel);
      }
      pos_s[threadIdx.x] = pos < 0 ? -1 : pos;
    }
    __syncthreads();
    for (int u = threadIdx.x; u < kTileRows * (kD / 8); u += 256) {
      const int tr = u / (kD / 8), c = u % (kD / 8);
      const int64_t pos = pos_s[tr];
      uint32_t code = 0, sc = 0;
      if (pos >= 0) {
        const int64_t cr = int64_t(b) * p.cap + pos;
        code = *reinterpret_cast<const uint32_t*>(p.packed + cr * (kD / 2) + 4 * c);
        sc = p.scales[cr * (kD / kGroup) + c / 2];
      }
      const uint32_t s2 = e4m3x2_to_f16x2(static_cast<uint16_t>(sc * 0x101u));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t h = hmul2_f16(e2m1x2_to_f16x2((code >> (8 * k)) & 0xffu), s2);
        tile[tr][8 * c + 2 * k] = f16_lo_to_f32(h);
        tile[tr][8 * c + 2 * k + 1] = f16_hi_to_f32(h);
      }
    }
    __syncthreads();
    for (int tr = 0; tr < kTileRows; ++tr) {
      const int64_t e = e0 + tr;
      const bool see = live && pos_s[tr] >= 0 && (e < n_sel || ((mask >> (e - n_sel)) & 1));
      if (!see) continue;  // (uniform in the warp)
      float v[16], s = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 f = *reinterpret_cast<const float4*>(&tile[tr][128 * k + 4 * lane]);
        v[4 * k] = f.x; v[4 * k + 1] = f.y; v[4 * k + 2] = f.z; v[4 * k + 3] = f.w;
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) s = fmaf(q[k], v[k], s);
      s = warp_sum(s);
      const float mn = fmaxf(m, s), a = expf(m - mn), pr = expf(s - mn);
      m = mn;
      l = l * a + pr;
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] = fmaf(pr, v[k], o[k] * a);
    }
  }
  if (!live) return;
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(o[4 * k + 1] * inv), "f"(o[4 * k] * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(o[4 * k + 3] * inv), "f"(o[4 * k + 2] * inv));
    *reinterpret_cast<uint2*>(p.out + row * kD + 128 * k + 4 * lane) = w;
  }
  if (p.lse && lane == 0) p.lse[row] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_tree_attn(const TreeAttnParams& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  return launch_pdl(k_tree_attn, dim3((p.T * p.H + 7) / 8, p.B), dim3(256), stream, p);
}

}  // namespace fp4kv
