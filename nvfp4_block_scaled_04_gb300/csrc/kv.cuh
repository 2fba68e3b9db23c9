// Shared pieces of the paged key-value cache kernels: which sequences a call
// deals with, and where a sequence's new rows lie.
#pragma once

#include "kv_line.h"
#include "launch.h"
#include "tc_util.cuh"

namespace nvfp4 {

// First new-token row of sequence b (b == batch: one past the last), clamped
// to the rows the caller's arrays hold.
NVFP4_DEV int kv_row0(const KvSeqs& s, int b) {
  const int64_t r = s.start ? static_cast<int64_t>(s.start[b]) : static_cast<int64_t>(b) * s.max_new;
  return static_cast<int>(r < 0 ? 0 : (r > s.tokens ? s.tokens : r));
}

// Length of sequence b, inside what position arithmetic in 32 bits can hold.
NVFP4_DEV int kv_len(const KvSeqs& s, int b) { return min(max(s.lens[b], 0), 1 << 30); }

NVFP4_DEV void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// The scale of softmax weights: p = 2^(x - m + LIFT) with m the maximum that the
// sums are kept relative to, which moves only where p would exceed 2^(SLACK +
// LIFT). The lift is the same in l and o, so it leaves no trace in the output.
// E4M3 caches take p as one f16: lifted, and with less slack, a row's heaviest
// weight lies in [2^11, 2^15.9], so that weights keep f16's 11 bits down to 2^-25
// of it (131,072 tokens of that weight hold 2^-8 together) and lose 2^-36 of it at
// most below. Scores so large that x - m is off by 0.1 (2^20) could pass f16's
// 65504: the conversion saturates. (2,048 new tokens on 6,144, 32 heads on 8: a
// slack of 4 took 4% longer; one of 8 with a lift of 7, which keeps 11 bits down to
// 2^-21 only, 4% less.) Weights in bf16 have fp32's range and need no lift.
template <bool E4M3>
struct KvWeights {
  static constexpr float SLACK = E4M3 ? 4.9f : 8.0f;
  static constexpr float LIFT = E4M3 ? 11.0f : 0.0f;
};

// Two weights as f16, lo in the low half: to nearest even, saturating.
NVFP4_DEV uint32_t kv_weights_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// Non-finite elements of value rows that some rows of a block see and others do
// not. As an operand they would reach the others too (0 * inf is NaN), so the
// kernels put zeros in their place and keep a bit for the token; at the end they
// read its values again and add those elements to the rows that see them.

// The four consecutive value elements at `at` of a pool where they are not
// finite (E4M3: its one NaN), zeros where they are.
template <bool E4M3>
NVFP4_DEV float4 kv_not_finite(const void* v, int64_t at) {
  float x[4];
  if (E4M3) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(v) + at);
#pragma unroll
    for (int z = 0; z < 4; ++z) x[z] = ((w >> (8 * z)) & 0x7Fu) == 0x7Fu ? __int_as_float(0x7FFFFFFF) : 0.0f;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(v) + at);
    const uint32_t h[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
    for (int z = 0; z < 4; ++z) x[z] = (h[z] & 0x7F80u) == 0x7F80u ? bf16_bits_to_f32(h[z]) : 0.0f;
  }
  return make_float4(x[0], x[1], x[2], x[3]);
}

// Whether a row at position pos sees position j.
NVFP4_DEV bool kv_sees(int pos, int j, int window, int sinks) {
  return j <= pos && (window <= 0 || pos - j < window || j < sinks);
}

// 2^x (2 ulp), zero for -inf.
NVFP4_DEV float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace nvfp4
