// The draw's arithmetic: keys and bins of logits, weights, products with a fraction. Plain code, the same on
// the device and on the host (any C++17 compiler that does not contract).
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

#ifndef NVFP4_HD
#ifdef __CUDACC__
#define NVFP4_HD __host__ __device__ __forceinline__
#else
#define NVFP4_HD inline
#endif
#endif

namespace nvfp4 {

// ---- fp32 operations, each rounded by itself
#ifdef __CUDA_ARCH__
NVFP4_HD float f32_add(float a, float b) { return __fadd_rn(a, b); }
NVFP4_HD float f32_sub(float a, float b) { return __fsub_rn(a, b); }
NVFP4_HD float f32_mul(float a, float b) { return __fmul_rn(a, b); }
NVFP4_HD float f32_div(float a, float b) { return __fdiv_rn(a, b); }
NVFP4_HD float f32_fma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
NVFP4_HD float f32_of_bits(uint32_t b) { return __uint_as_float(b); }
NVFP4_HD uint32_t bits_of_f32(float f) { return __float_as_uint(f); }
NVFP4_HD int int_of_f32(float f) { return __float2int_rn(f); }
NVFP4_HD unsigned long long high_half(unsigned long long a, unsigned long long b) { return __umul64hi(a, b); }
#else
NVFP4_HD float f32_add(float a, float b) { return a + b; }
NVFP4_HD float f32_sub(float a, float b) { return a - b; }
NVFP4_HD float f32_mul(float a, float b) { return a * b; }
NVFP4_HD float f32_div(float a, float b) { return a / b; }
NVFP4_HD float f32_fma(float a, float b, float c) { return std::fmaf(a, b, c); }
NVFP4_HD float f32_of_bits(uint32_t b) {
  float f;
  std::memcpy(&f, &b, 4);
  return f;
}
NVFP4_HD uint32_t bits_of_f32(float f) {
  uint32_t b;
  std::memcpy(&b, &f, 4);
  return b;
}
NVFP4_HD int int_of_f32(float f) { return static_cast<int>(std::nearbyint(f)); }
NVFP4_HD unsigned long long high_half(unsigned long long a, unsigned long long b) {
  const unsigned long long a0 = a & 0xFFFFFFFFu, a1 = a >> 32, b0 = b & 0xFFFFFFFFu, b1 = b >> 32;
  const unsigned long long mid = a1 * b0 + (a0 * b0 >> 32), low = a0 * b1 + (mid & 0xFFFFFFFFu);
  return a1 * b1 + (mid >> 32) + (low >> 32);
}
#endif

// ---- keys

template <bool F32>
struct Key {
  static constexpr int GROUP = F32 ? 4 : 8;                      // logits in 16 bytes
  static constexpr uint32_t SIGN = F32 ? 0x80000000u : 0x8000u;
  static constexpr uint32_t ALL = F32 ? 0xFFFFFFFFu : 0xFFFFu;
  static constexpr uint32_t PINF = F32 ? 0xFF800000u : 0xFF80u;  // key of +inf
  static constexpr uint32_t LOWEST = F32 ? 0x00800000u : 0x80u;  // key of the lowest finite value
  static constexpr int LOW = F32 ? 16 : 0;                       // bits of a key below the bins'
};

// 0 for what is never drawn (-inf, NaN); -0 is 0.
template <bool F32>
NVFP4_HD uint32_t key_of(uint32_t b) {
  using K = Key<F32>;
  if (b == K::SIGN) b = 0;
  const uint32_t k = (b & K::SIGN) ? (~b & K::ALL) : (b | K::SIGN);
  return k - K::LOWEST <= K::PINF - K::LOWEST ? k : 0u;
}

template <bool F32>
NVFP4_HD float value_of(uint32_t k) {
  using K = Key<F32>;
  const uint32_t b = (k & K::SIGN) ? (k & ~K::SIGN) : (~k & K::ALL);
  return f32_of_bits(F32 ? b : b << 16);
}

// ---- bins of the upper 16 bits h of a key, in falling order
constexpr int E_LO = 117, E_HI = 134;                      // exponent fields: 2^-10 .. 2^7
constexpr int OUTER = (E_HI - E_LO) * 128;
constexpr uint32_t POS_TOP = 0x8000u + (E_HI << 7);        // from here up: bin 0
constexpr uint32_t POS_LOW = 0x8000u + (E_LO << 7);        // the lowest positive h with a bin of its own
constexpr uint32_t NEG_TOP = 0x7FFFu - (E_LO << 7);        // the highest negative one
constexpr uint32_t NEG_LOW = 0x7FFFu - (E_HI << 7) + 1;    // the lowest
constexpr int B_MID = OUTER + 1, B_LAST = 2 * OUTER + 3, NB = 2 * OUTER + 4;   // B_MID: 0 and up, B_MID + 1: below 0

NVFP4_HD int bin_of(uint32_t h) {
  if (h & 0x8000u) {
    const int b = static_cast<int>(POS_TOP) - static_cast<int>(h);
    return b < 0 ? 0 : b > B_MID ? B_MID : b;
  }
  const int b = B_MID + 2 + static_cast<int>(NEG_TOP) - static_cast<int>(h);
  return b < B_MID + 1 ? B_MID + 1 : b > B_LAST ? B_LAST : b;
}

// The four bins of many values, by number, and -1 for the others.
NVFP4_HD int wide_bin(int b) { return b == 0 ? 0 : b == B_MID ? 1 : b == B_MID + 1 ? 2 : b == B_LAST ? 3 : -1; }

// The upper halves of the keys of a bin.
NVFP4_HD void bin_range(int b, uint32_t& lo, uint32_t& hi) {
  if (b == 0) lo = POS_TOP, hi = 0xFF80u;
  else if (b == B_MID) lo = 0x8000u, hi = POS_LOW - 1;
  else if (b == B_MID + 1) lo = NEG_TOP + 1, hi = 0x7FFFu;
  else if (b == B_LAST) lo = 0x80u, hi = NEG_LOW - 1;
  else lo = hi = b < B_MID ? POS_TOP - b : NEG_TOP + B_MID + 2 - b;
}

// Two bf16 logits of one word: (bin of each) = B_MID - (its signed half of what is returned), for magnitudes of
// 2^-10 and more (infinities and NaN fall into the first and the last bin). sign: 0xFFFF where negative.
constexpr uint32_t MAG_LOW = E_LO << 7, MAG_TOP = E_HI << 7;
NVFP4_HD uint32_t bin_steps(uint32_t clamped_magnitudes, uint32_t sign) {
  return (clamped_magnitudes - (MAG_LOW - 1) * 0x10001u) ^ sign;
}

// ---- weights

constexpr int W_BITS = 44;
constexpr unsigned long long ONE = 1ull << W_BITS;

// round(2^44 * 2^(-i/64))
#ifdef __CUDACC__
__device__
#endif
const unsigned long long EXP2_TABLE[64] = {
    0x100000000000ull, 0xfd3e0c0cf48ull, 0xfa83b2db723ull, 0xf7d0df730adull, 0xf5257d15248ull, 0xf281773c5a0ull, 0xefe4b99bdceull, 0xed4f301ed99ull,
    0xeac0c6e7dd2ull, 0xe8396a503c5ull, 0xe5b906e77c8ull, 0xe33f8972be9ull, 0xe0ccdeec2a9ull, 0xde60f4825e1ull, 0xdbfbb797dafull, 0xd99d15c278bull,
    0xd744fccad6aull, 0xd4f35aabcffull, 0xd2a81d91f13ull, 0xd06333daef3ull, 0xce248c151f8ull, 0xcbec14fef27ull, 0xc9b9bd866e3ull, 0xc78d74c8abcull,
    0xc5672a11550ull, 0xc346ccda249ull, 0xc12c4cca667ull, 0xbf1799b67a7ull, 0xbd08a39f581ull, 0xbaff5ab2134ull, 0xb8fbaf47630ull, 0xb6fd91e328dull,
    0xb504f333f9eull, 0xb311c412a91ull, 0xb123f581d2bull, 0xaf3b78ad691ull, 0xad583eea42aull, 0xab7a39b5a94ull, 0xa9a15ab4ea8ull, 0xa7cd93b4e96ull,
    0xa5fed6a9b15ull, 0xa43515ae09eull, 0xa27043030c5ull, 0xa0b0510fb97ull, 0x9ef5326091aull, 0x9d3ed9a72d0ull, 0x9b8d39b9d55ull, 0x99e0459320bull,
    0x9837f0518dcull, 0x96942d37202ull, 0x94f4efa8fefull, 0x935a2b2f13eull, 0x91c3d373ab1ull, 0x9031dc43146ull, 0x8ea4398b45dull, 0x8d1adf5b7e6ull,
    0x8b95c1e3ea9ull, 0x8a14d575497ull, 0x88980e8092eull, 0x871f61969e9ull, 0x85aac367cc5ull, 0x843a28c3aceull, 0x82cd8698ac3ull, 0x8164d1f3bc0ull,
};

// log2(e) / T in two floats (the remainder of the division is exact), and the power of two that T and the logits are taken
// times first: one, but for a T at which log2(e) / T or a difference of two logits may have no fp32 value. (Logits that
// lose bits by it are small beside such a T; those that overflow differ by more than 46 T or not at all.)
struct Slope {
  float hi, lo, scale;
};

NVFP4_HD Slope slope_of(float t) {
  const float l_hi = 1.44269502e+00f, l_lo = 1.92596303e-08f;   // log2(e) = l_hi + l_lo to 2^-50
  Slope s;
  s.scale = t >= 0x1p64f ? 0x1p-64f : t < 0x1p-64f ? 0x1p64f : 1.0f;
  t = f32_mul(t, s.scale);
  s.hi = f32_div(l_hi, t);
  s.lo = f32_div(f32_add(f32_fma(-s.hi, t, l_hi), l_lo), t);
  return s;
}

// exp((x - ref) / T) for x <= ref as 2^(-44 - n) times what is returned, to 2^-35 of itself: 2^-y by a table of 64
// steps and a short series (Tang, 1989), with y = (ref - x) log2(e) / T carried in two floats. Equal values weigh
// one, also infinite ones; 0 where y >= 46 and for a NaN. (|l| < 0.0055: the series' second term is rounded three
// times by 2^-25 of 2^-16, q twice by 2^-38, the table's factor by 2^-31 of l, the term left out is 2^-44: 2^-36
// together.) Written for one value (F = float, float operations) or a pair (the pair's operations).
constexpr float W_MAGIC = 12582912.0f;   // 1.5 * 2^23: a sum with it is rounded to a whole number

template <class F>
struct WeightParts {
  F y, t, l, tail;   // 2^-y = 2^(-k/64) (1 - l + tail), k in the lower bits of t
};

template <class F, class S>
NVFP4_HD WeightParts<F> weight_parts(F ref, F nx, F hi, F lo, S) {
  const F minus1 = S::all(-1.0f);
  const F d = S::add(ref, nx);                                   // d + dl = ref - x exactly
  const F b = S::fma(ref, minus1, d);
  const F dl = S::add(S::fma(S::fma(b, minus1, d), minus1, ref), S::fma(b, minus1, nx));
  WeightParts<F> p;
  p.y = S::mul(d, hi);
  p.t = S::fma(p.y, S::all(64.0f), S::all(W_MAGIC));
  const F r0 = S::fma(S::add(p.t, S::all(-W_MAGIC)), S::all(-0.015625f), p.y);   // exact, at most 2^-7
  const F yl = S::fma(d, lo, S::fma(dl, hi, S::fma(d, hi, S::mul(p.y, minus1))));
  const F r = S::add(r0, yl), rl = S::fma(S::fma(r0, minus1, r), minus1, yl);
  const F ln2 = S::all(6.93147182e-01f);
  p.l = S::mul(r, ln2);
  const F nl = S::mul(p.l, minus1);
  const F ll = S::add(S::fma(r, ln2, nl), S::fma(r, S::all(-1.90465421e-09f), S::mul(rl, ln2)));
  // e^-(l + ll) = 1 - l + tail
  const F h = S::fma(nl, S::fma(nl, S::all(0.0416666667f), S::all(0.166666667f)), S::all(0.5f));
  p.tail = S::fma(S::mul(p.l, p.l), h, S::mul(S::fma(nl, ll, ll), minus1));
  return p;
}

struct OneFloat {
  static NVFP4_HD float all(float v) { return v; }
  static NVFP4_HD float add(float a, float b) { return f32_add(a, b); }
  static NVFP4_HD float mul(float a, float b) { return f32_mul(a, b); }
  static NVFP4_HD float fma(float a, float b, float c) { return f32_fma(a, b, c); }
};

NVFP4_HD unsigned long long weight_of_parts(float y, float t, float l, float tail, const unsigned long long* table, int& n) {
  const int k = static_cast<int>(bits_of_f32(t) - bits_of_f32(W_MAGIC));
  const int q = int_of_f32(l * -0x1p37f) + int_of_f32(tail * 0x1p37f);   // below 2^30
  const unsigned long long e = table[k & 63];
  n = (k >> 6) & 63;
  const long long add = static_cast<long long>(static_cast<int>((e + 8192) >> 14)) * q;
  return y < 46.f ? e + static_cast<unsigned long long>(add >> 23) : 0ull;
}

NVFP4_HD unsigned long long weight_and_scale(float ref, float x, const Slope& c, const unsigned long long* table, int& n) {
  const WeightParts<float> p = weight_parts(f32_mul(ref, c.scale), f32_mul(-x, c.scale), c.hi, c.lo, OneFloat());
  const bool some = p.y < 46.f;
  const unsigned long long w = some ? weight_of_parts(p.y, p.t, p.l, p.tail, table, n) : 0ull;
  // (an infinite temperature: all finite logits)
  const bool even = x == ref || (c.hi == 0.f && ref - ref == 0.f && x - x == 0.f);
  if (even || !some) n = 0;
  return even ? ONE : w;
}

NVFP4_HD unsigned long long rounded_weight(unsigned long long w, int n) { return (((w << 1) >> n) + 1) >> 1; }

// round(2^44 exp((x - ref) / T))
NVFP4_HD unsigned long long weight(float ref, float x, const Slope& c, const unsigned long long* table) {
  int n;
  const unsigned long long w = weight_and_scale(ref, x, c, table, n);
  return rounded_weight(w, n);
}

// ceil(x / w) where that is below 2^21 (w = 0: 0).
NVFP4_HD uint32_t few_times(unsigned long long x, unsigned long long w) {
  if (w == 0) return 0;
  uint32_t n = static_cast<uint32_t>(f32_div(static_cast<float>(x), static_cast<float>(w)));   // off by one at most
  if (n > 0 && (n - 1) * w >= x) --n;
  while (n * w < x) ++n;
  return n;
}

// floor(v * x) for 0 <= v < 1, and whether something was cut off.
NVFP4_HD unsigned long long times(unsigned long long x, float v, bool& cut) {
  const uint32_t b = bits_of_f32(v);
  const int e = static_cast<int>(b >> 23);
  const unsigned long long m = e ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
  const int shift = 150 - (e ? e : 1);                          // v = m 2^-shift, shift > 23
  const unsigned long long lo = m * x, hi = high_half(m, x);
  if (shift < 64) {
    cut = (lo << (64 - shift)) != 0;
    return hi << (64 - shift) | lo >> shift;
  }
  if (shift == 64) {
    cut = lo != 0;
    return hi;
  }
  const int s = shift - 64;
  if (s >= 64) {
    cut = lo != 0 || hi != 0;
    return 0ull;
  }
  cut = lo != 0 || (hi << (64 - s)) != 0;
  return hi >> s;
}

}  // namespace nvfp4
