// e2m1 codes to BF16, shared by the kernels that take NVFP4 weights.
#pragma once

#include <stdint.h>

namespace gb300 {

// W4A16 weights ("gemm_dense.rs", w4a16_gemm: C = A @ dequant(B), NVFP4
// weights dequantised to BF16): 16 packed bytes of one weight row (32 e2m1
// codes, element 2j in the low nibble of byte j) and the row's two e4m3
// block scales for those elements (low byte: elements 0..15) ->
//   w = e2m1 * e4m3
// as 16 bf16x2 words in element order.  The product has at most six
// significant bits and lies in [2^-10, 2688], so BF16 holds it exactly and
// the BF16 multiply below rounds nothing (the per-tensor scale is applied
// to the FP32 sum in the epilogue).
//
// The e2m1 code -> BF16 step is a byte-permute table lookup (integer pipe):
// the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 of codes 0..7 are the BF16
// patterns 0x0000 3F00 3F80 3FC0 4000 4040 4080 40C0; one PRMT looks up the
// low bytes of four codes, one the high bytes, and the code's sign bit
// (bit 3) becomes bit 15 of its BF16 value.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// Four e2m1 codes (the low 16 bits of g, code i in bits 4i..4i+3) -> two
// bf16x2 words (codes 0, 1 and codes 2, 3).
__device__ __forceinline__ void e2m1x4_to_bf16(uint32_t g, uint32_t& w01, uint32_t& w23) {
  constexpr uint32_t kLo0 = 0xC0800000u, kLo1 = 0xC0804000u;  // low bytes, codes 0..3 / 4..7
  constexpr uint32_t kHi0 = 0x3F3F3F00u, kHi1 = 0x40404040u;  // high bytes
  const uint32_t sel = g & 0x7777u;
  const uint32_t lo = prmt(kLo0, kLo1, sel);
  uint32_t hi = prmt(kHi0, kHi1, sel);
  // sign: a negative code selects byte 4 (0x80) in sign-replicate mode
  // (0xFF), a positive one byte 4 as is (0x80); bit 6 then says which
  const uint32_t sg = prmt(0u, 0x80u, (g & 0x8888u) | 0x4444u);
  hi |= (sg << 1) & 0x80808080u;  // bit 7 of a byte: bit 6 of its sg byte
  w01 = prmt(lo, hi, 0x5140u);
  w23 = prmt(lo, hi, 0x7362u);
}

}  // namespace gb300
