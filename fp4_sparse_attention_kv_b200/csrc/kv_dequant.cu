// kv_dequant_fp4: rows of the FP4 cache read back by row number, to bf16 or fp32.
//
// value = e2m1(code) * e4m3(scale). A code has at most 2 significant bits and a scale 4, so a
// value has at most 6 and lies in [2^-10, 2688] (or is a signed zero): exact in fp16, in bf16 and
// in fp32. The product is formed in fp16 (one packed multiply for two channels) and widened.
//
// Memory: a warp reads consecutive codes and writes consecutive 16-byte units: 8 channels per
// thread for bf16, 4 for fp32. A block owns whole rows, so that the row of a unit comes from a
// 32-bit division by a small number (a multiply and a shift).
#include "fp4kv_common.cuh"
#include "fp4kv_launch.h"
#include "fp4kv_quant.cuh"
#include "fp4kv_sm100.cuh"

namespace fp4kv {
namespace {

constexpr int kThreads = 256;

// kF32: 4 channels (2 code bytes) to a 16-byte unit, else 8 channels (4 code bytes). kIter units
// per thread, their loads issued before the first is converted.
template <bool kF32, int kIter>
__global__ void __launch_bounds__(kThreads) k_kv_dequant_fp4(const uint8_t* __restrict__ packed,
                                                             const uint8_t* __restrict__ scales, int64_t cap_rows,
                                                             int d, const int64_t* __restrict__ src_row,
                                                             int64_t n_rows, uint8_t* __restrict__ out,
                                                             int64_t out_row_bytes, int rows_per_block, int upr,
                                                             uint32_t magic) {
  constexpr int kCh = kF32 ? 4 : 8;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_per_block;
  const int n_units = static_cast<int>(min(static_cast<int64_t>(rows_per_block), n_rows - row0)) * upr;
  uint32_t code[kIter], sc[kIter];
  int64_t dst[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const uint32_t u = i * kThreads + threadIdx.x;
    dst[i] = -1;
    code[i] = sc[i] = 0;
    if (static_cast<int>(u) < n_units) {
      const uint32_t lr = __umulhi(u, magic);  // u / upr (u < 2^16, upr <= 256)
      const uint32_t c = u - lr * upr;
      const int64_t r = row0 + lr;
      const int64_t src = src_row ? src_row[r] : r;
      dst[i] = r * out_row_bytes + 16 * static_cast<int64_t>(c);
      if (src >= 0 && src < cap_rows) {  // absent rows read as zeros
        const uint8_t* p = packed + src * (d / 2);
        if (kF32)
          code[i] = *reinterpret_cast<const uint16_t*>(p + 2 * c);
        else
          code[i] = *reinterpret_cast<const uint32_t*>(p + 4 * c);
        sc[i] = scales[src * (d / kGroup) + (c * kCh) / kGroup];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    if (dst[i] < 0) continue;
    const uint32_t s2 = e4m3x2_to_f16x2(static_cast<uint16_t>(sc[i] * 0x101u));
    uint32_t h[kCh / 2];
#pragma unroll
    for (int k = 0; k < kCh / 2; ++k) h[k] = hmul2_f16(e2m1x2_to_f16x2((code[i] >> (8 * k)) & 0xffu), s2);
    uint4 o;
    if (kF32) {
      o.x = __float_as_uint(f16_lo_to_f32(h[0]));
      o.y = __float_as_uint(f16_hi_to_f32(h[0]));
      o.z = __float_as_uint(f16_lo_to_f32(h[1]));
      o.w = __float_as_uint(f16_hi_to_f32(h[1]));
    } else {  // (exact: the upper half of the fp32 bits)
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < kCh / 2; ++k)
        w[k] = __byte_perm(__float_as_uint(f16_lo_to_f32(h[k])), __float_as_uint(f16_hi_to_f32(h[k])), 0x7632);
      o = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4*>(out + dst[i]) = o;
  }
}

template <bool kF32, int kIter>
cudaError_t launch(const uint8_t* packed, const uint8_t* scales, int64_t cap_rows, int d, const int64_t* src_row,
                   int64_t n_rows, void* out, int64_t out_row_stride, cudaStream_t stream) {
  const int upr = d / (kF32 ? 4 : 8);  // units per row: 4 .. 256
  const int rows = kThreads * kIter / upr;
  const uint32_t magic = static_cast<uint32_t>((uint64_t(1) << 32) / upr + 1);
  const int64_t blocks = (n_rows + rows - 1) / rows;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  k_kv_dequant_fp4<kF32, kIter><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
      packed, scales, cap_rows, d, src_row, n_rows, static_cast<uint8_t*>(out), out_row_stride * (kF32 ? 4 : 2), rows, upr,
      magic);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_dequant_fp4(const uint8_t* packed, const uint8_t* scales, int64_t cap_rows, int d,
                                  const int64_t* src_row, int64_t n_rows, void* out, bool f32, int64_t out_row_stride,
                                  int num_sms, cudaStream_t stream) {
  if (n_rows == 0) return cudaSuccess;
  // four units per thread where that still fills the GPU twice over, one where latency counts
  const int64_t units = n_rows * (d / (f32 ? 4 : 8));
  const bool big = units >= int64_t(num_sms) * 2 * 8 * kThreads * 4;
  if (f32)
    return big ? launch<true, 4>(packed, scales, cap_rows, d, src_row, n_rows, out, out_row_stride, stream)
               : launch<true, 1>(packed, scales, cap_rows, d, src_row, n_rows, out, out_row_stride, stream);
  return big ? launch<false, 4>(packed, scales, cap_rows, d, src_row, n_rows, out, out_row_stride, stream)
             : launch<false, 1>(packed, scales, cap_rows, d, src_row, n_rows, out, out_row_stride, stream);
}

}  // namespace fp4kv
