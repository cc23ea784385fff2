// Geometry and conversions of the 8-bit K/V cache: a page holds 128 token rows of one head as 128
// OCP E4M3 bytes each ("vllm.models.minimax_m3.amd.mono.dispatch", _config_refusal: the fp8 K/V
// cache), and every 32 tokens of a page and head share one e8m0 scale, kept beside the pool
// ([pages, heads, 4] bytes).
#pragma once

#include "common.cuh"

namespace mx4 {

constexpr int kFp8Row = kHeadDim;                // bytes of a token row
constexpr int kFp8Page = kPageTokens * kFp8Row;  // 16384
constexpr int kSub = 32;                         // tokens that share a scale
constexpr int kPageSubs = kPageTokens / kSub;    // scales of a page and head
static_assert(kFp8Page == MX4_FP8_PAGE_BYTES, "fp8 page geometry");

// Two E4M3 pairs of w -> two f16x2, exact (the low byte of a pair -> the low half).
__device__ __forceinline__ void e4m3x4_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 h0, h1;\n mov.b32 {h0, h1}, %2;\n"
      " cvt.rn.f16x2.e4m3x2 %0, h0;\n cvt.rn.f16x2.e4m3x2 %1, h1;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

}  // namespace mx4
