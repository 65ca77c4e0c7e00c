// kv_dequant_fp4: rows of the FP4 cache read back by row number, to bf16 or fp32.
//
// value = e2m1(code) * e4m3(scale). A code has at most 2 significant bits and a scale 4, so a
// value has at most 6 and lies in [2^-10, 2688] (or is a signed zero): exact in fp16, in bf16 and
// in fp32. The product is formed in fp16 (one packed multiply for two channels) and widened.
//
// Bound by memory: 9/16 d bytes in, 2 d or 4 d out per row. A thread makes 64 consecutive bytes (32
// channels in bf16, 16 in fp32) from one load of codes, written as two 32-byte sectors: addresses
// and row numbers cost more instructions than the values where it makes 16 bytes (65,536 rows of 512 to
// bf16 out of a cache of 1,048,576: 20 us that way, 16 us
// this way, 5.5 TB/s; 400,000 rows in order to fp32: 142 us, 6.6 TB/s). A block owns whole rows, so that the row of a unit
// comes from a 32-bit division by a small number (a multiply and a shift).
#include "fp4kv_common.cuh"
#include "fp4kv_launch.h"
#include "fp4kv_quant.cuh"
#include "fp4kv_sm100.cuh"

namespace fp4kv {
namespace {

constexpr int kThreads = 256;

FP4KV_DEV void store_32b(uint8_t* at, const uint32_t* w, bool al32) {
  if (al32) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
  } else {
    reinterpret_cast<uint4*>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// Eight codes times a scale -> four f16x2.
FP4KV_DEV void values8(uint32_t codes, uint32_t s2, uint32_t (&h)[4]) {
  e2m1x8_to_f16(codes, h);
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = hmul2_f16(h[k], s2);
}

// kIter units per thread, their loads issued before the first is converted. flags: bit 0: stores of 32
// bytes are aligned, bit 1: pairs of scales are.
template <bool kF32, int kIter>
__global__ void __launch_bounds__(kThreads) k_kv_dequant_fp4(const uint8_t* __restrict__ packed,
                                                             const uint8_t* __restrict__ scales, int64_t cap_rows,
                                                             int d, const int64_t* __restrict__ src_row,
                                                             int64_t n_rows, uint8_t* __restrict__ out,
                                                             int64_t out_row_bytes, int rows_per_block, int upr,
                                                             uint32_t magic, int flags) {
  griddep_wait();  // the rows may come from the kernel before this one on the stream
  constexpr int kWords = kF32 ? 2 : 4;  // of codes to a unit
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_per_block;
  const int n_units = static_cast<int>(min(static_cast<int64_t>(rows_per_block), n_rows - row0)) * upr;
  uint32_t code[kIter][kWords], sc[kIter];
  int lr[kIter], col[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const uint32_t u = i * kThreads + threadIdx.x;
    lr[i] = upr == 1 ? u : __umulhi(u, magic);  // u / upr (u < 2^16, 2 <= upr <= 64)
    col[i] = u - lr[i] * upr;
#pragma unroll
    for (int k = 0; k < kWords; ++k) code[i][k] = 0;
    sc[i] = 0;
    if (static_cast<int>(u) < n_units) {
      const int64_t r = row0 + lr[i];
      const int64_t src = src_row ? src_row[r] : r;
      if (src >= 0 && src < cap_rows) {  // absent rows read as zeros
        const uint8_t* c = packed + src * (d / 2) + 4 * kWords * col[i];
        const uint8_t* f = scales + src * (d / kGroup) + kWords / 2 * col[i];
        if (kF32) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(c));
          code[i][0] = v.x;
          code[i][1] = v.y;
          sc[i] = *f;
        } else {
          const uint4 v = ld_nc_v4(c);
          code[i][0] = v.x; code[i][1] = v.y; code[i][kWords - 2] = v.z; code[i][kWords - 1] = v.w;
          sc[i] = flags & 2 ? *reinterpret_cast<const uint16_t*>(f) : f[0] | (uint32_t(f[1]) << 8);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    if (static_cast<int>(i * kThreads + threadIdx.x) >= n_units) continue;
    uint8_t* at = out + (row0 + lr[i]) * out_row_bytes + 64 * col[i];
    const uint32_t s = e4m3x2_to_f16x2(static_cast<uint16_t>(sc[i]));
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // 32 bytes
      uint32_t w[8];
      if (kF32) {
        uint32_t h[4];
        values8(code[i][j], __byte_perm(s, 0, 0x1010), h);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[2 * k] = __float_as_uint(f16_lo_to_f32(h[k]));
          w[2 * k + 1] = __float_as_uint(f16_hi_to_f32(h[k]));
        }
      } else {
        const uint32_t s2 = __byte_perm(s, 0, j ? 0x3232 : 0x1010);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          uint32_t h[4];
          values8(code[i][2 * j + v < kWords ? 2 * j + v : 0], s2, h);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // (exact: the upper half of the fp32 bits)
            w[4 * v + k] = __byte_perm(__float_as_uint(f16_lo_to_f32(h[k])), __float_as_uint(f16_hi_to_f32(h[k])), 0x7632);
        }
      }
      store_32b(at + 32 * j, w, flags & 1);
    }
  }
}

template <bool kF32, int kIter>
cudaError_t launch(const uint8_t* packed, const uint8_t* scales, int64_t cap_rows, int d, const int64_t* src_row,
                   int64_t n_rows, void* out, int64_t out_row_stride, cudaStream_t stream) {
  const int upr = d / (kF32 ? 16 : 32);  // units per row: 1 .. 64
  const int rows = kThreads * kIter / upr;
  const uint32_t magic = upr == 1 ? 0 : static_cast<uint32_t>((uint64_t(1) << 32) / upr + 1);
  const int64_t blocks = (n_rows + rows - 1) / rows, row_bytes = out_row_stride * (kF32 ? 4 : 2);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const int flags = ((reinterpret_cast<uintptr_t>(out) | static_cast<uintptr_t>(row_bytes)) % 32 == 0 ? 1 : 0) |
                    (reinterpret_cast<uintptr_t>(scales) % 2 == 0 ? 2 : 0);
  return launch_sized(kIter == 1, k_kv_dequant_fp4<kF32, kIter>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), stream,
                      packed, scales, cap_rows, d, src_row, n_rows, static_cast<uint8_t*>(out), row_bytes, rows, upr, magic,
                      flags);
}

}  // namespace

cudaError_t launch_kv_dequant_fp4(const uint8_t* packed, const uint8_t* scales, int64_t cap_rows, int d,
                                  const int64_t* src_row, int64_t n_rows, void* out, bool f32, int64_t out_row_stride,
                                  int num_sms, cudaStream_t stream) {
  if (n_rows == 0) return cudaSuccess;
  // Two units per thread, whose loads overlap, and a dependent launch where one unit each would be more than the
  // threads that fit; one, launched plainly, below: there the host's 6 to 7 us a call are what counts. Rows of 512
  // gathered from 1,048,576 (neither they nor the output in L2, calls replayed from a graph), one unit launched plainly
  // against two: 9,472 to bf16 4.5 against 4.2 us, to fp32 5.9 against 5.4, 18,944 to bf16 6.5 against 5.9, to fp32 9.9
  // against 8.8, 37,888 to bf16 10.8 against 9.7, 65,536 16.8 against 15.7.
  const int64_t units = n_rows * (d / (f32 ? 16 : 32));
  const bool big = units > int64_t(num_sms) * 8 * kThreads;
  if (f32)
    return big ? launch<true, 2>(packed, scales, cap_rows, d, src_row, n_rows, out, out_row_stride, stream)
               : launch<true, 1>(packed, scales, cap_rows, d, src_row, n_rows, out, out_row_stride, stream);
  return big ? launch<false, 2>(packed, scales, cap_rows, d, src_row, n_rows, out, out_row_stride, stream)
             : launch<false, 1>(packed, scales, cap_rows, d, src_row, n_rows, out, out_row_stride, stream);
}

}  // namespace fp4kv
