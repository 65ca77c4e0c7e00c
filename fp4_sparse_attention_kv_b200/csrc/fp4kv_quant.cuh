// Quantising one 16-channel group to E2M1 codes and an E4M3 scale, reading groups back, and small helpers:
// shared by the cache writes and reads and the operators beside them. The rounding rules and their exactness argument are
// stated in kv_quant.cu.
#pragma once

#include "fp4kv_common.cuh"

namespace fp4kv {

// RN(a * inv + 128) - 128: the ratio a * inv rounded once to a multiple of 2^-16 (for
// a * inv < 128; larger ratios saturate the code either way)
FP4KV_DEV float snap_ratio(float a, float inv) {
  return __fadd_rn(__fmaf_rn(a, inv, 128.0f), -128.0f);
}

// Quantize one group of 16 bf16 values held as 8 words (2 values per word, low half first).
// Returns the 8 packed bytes (low nibble = even channel) and the scale code.
FP4KV_DEV void quant_group(const uint32_t (&w)[8], uint2& packed, uint32_t& scale_code) {
  uint32_t m2 = 0;  // per-half maxima of the 15-bit magnitudes
#pragma unroll
  for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7fff7fffu);
  const uint32_t m = max(m2 & 0xffffu, m2 >> 16);
  const float amax = bf16_bits_to_f32(m);
  const uint32_t sc = f32_to_e4m3_satfinite(__fdiv_rn(amax, 6.0f));
  const float S = f16_lo_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(sc)));
  uint32_t bytes[8];
  if (S > 0.0f) {
    const float inv = __frcp_rn(S);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t e = w[i] << 16, o = w[i] & 0xffff0000u;  // the two channels as f32 bits
      const float r0 = snap_ratio(__uint_as_float(e & 0x7fffffffu), inv);
      const float r1 = snap_ratio(__uint_as_float(o & 0x7fffffffu), inv);
      // the sign goes back on before the rounding to E2M1, which is symmetric; a negative
      // value that rounds to zero keeps its sign (code 0x8)
      bytes[i] = f32x2_to_e2m1x2_satfinite(__uint_as_float(__float_as_uint(r0) | (e & 0x80000000u)),
                                           __uint_as_float(__float_as_uint(r1) | (o & 0x80000000u)));
    }
  } else {  // an all-zero group: sign-only codes
#pragma unroll
    for (int i = 0; i < 8; ++i) bytes[i] = ((w[i] >> 12) & 0x8u) | ((w[i] >> 24) & 0x80u);
  }
  packed.x = bytes[0] | (bytes[1] << 8) | (bytes[2] << 16) | (bytes[3] << 24);
  packed.y = bytes[4] | (bytes[5] << 8) | (bytes[6] << 16) | (bytes[7] << 24);
  scale_code = sc;
}

// Eight codes -> four f16x2 (the byte registers spare the shifts).
FP4KV_DEV void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
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

// 16 bytes from global to shared memory, asynchronously, and from shared memory
FP4KV_DEV void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
FP4KV_DEV uint4 lds_v4(uint32_t at) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
  return r;
}

// A launch that may begin while the kernel before it on the stream finishes (programmatic
// dependent launch); the kernel orders itself with griddep_wait().
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// The same kernel (it calls griddep_wait(), which returns at once in a plain launch), launched plainly
// where `small`: a plain launch costs the host 1 us less, and the host is what bounds small calls; a
// dependent one follows the kernel before it 2.5 us sooner, which counts for the large ones.
template <typename... KArgs, typename... Args>
cudaError_t launch_sized(bool small, void (*kern)(KArgs...), dim3 grid, dim3 block, cudaStream_t stream, Args... args) {
  if (!small) return launch_pdl(kern, grid, block, stream, args...);
  kern<<<grid, block, 0, stream>>>(static_cast<KArgs>(args)...);
  return cudaGetLastError();
}

}  // namespace fp4kv
