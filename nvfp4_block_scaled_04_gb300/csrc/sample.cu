// The draw of a token from each row of logits: temperature, top-k, top-p, min-p, one given random number.
//
// The order. A row's tokens are ordered by falling logit, equal logits by index. Every filter keeps a first
// part of that order (the k first; the shortest part whose mass reaches p of that; the tokens of at least
// min_p times the first one's weight), so what is kept is a first part too, and all that remains of it is its
// mass W. The draw is the first token whose cumulated mass exceeds u * W. With weights
// w_j = exp((l_j - l_max) / T), each step asks for a position in cumulated counts or masses.
//
// No sort. Keys (the logits' bits, turned so that they order as unsigned numbers) are counted in a histogram
// whose bins follow the upper 16 bits: one bin for each bf16 value of magnitude 2^-10 to 2^7, one for all
// smaller magnitudes, one for everything above and one for everything below. For bf16 logits a bin is one
// value, so its mass is its count times one weight, and a position inside it is a division. Where a bin holds
// several values (fp32 logits; the three wide bins), it is counted again by finer parts of the key until a part
// is one value. What is left is the m-th token of one key in index order: a scan of one CTA's slice.
//
// Exactness. The token has to be the one that the definition names, so masses are 64-bit integers: a weight is
// round(2^44 w) with a relative error below 2^-35 (sample_math.h), sums of up to 2^19 of them are exact and
// do not depend on order, and u * W and p * W are compared exactly. The result is the same from call to call.
//
// Work. A cluster of 1 to 16 CTAs takes a row, each a slice of it; counts are joined through distributed
// shared memory, and the cluster's first CTA searches. HBM sees each logit once.
#include <atomic>

#include "common.cuh"
#include "launch.h"
#include "sample_math.h"
#include "tc_util.cuh"

namespace nvfp4 {

namespace {

constexpr int S_THREADS = 512;
constexpr int S_WARPS = S_THREADS / 32;

// (for the places that few tokens reach)
__device__ __noinline__ unsigned long long rare_weight(float ref, float x, const Slope& c, const unsigned long long* table) {
  return weight(ref, x, c, table);
}

// ---- distributed shared memory

template <typename T>
NVFP4_DEV T* in_cta(T* p, uint32_t rank) {
  T* r;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
  return r;
}

// ---- the kernel

struct SampleArgs {
  const void* logits;
  int64_t stride;        // elements between rows
  int vocab;
  int rows_each;         // rows that share one entry of the settings
  nvfp4_sampling_t set;
  const float* uniform;
  int32_t* ids;
  float* probs;
};

enum { CMD_FIND = 0, CMD_REFINE = 1 };

struct Command {
  int what;
  uint32_t lo, hi;       // REFINE: keys lo .. hi by parts of 2^shift
  int shift;
  uint32_t key;          // FIND: the nth of CTA `owner`'s tokens with this key, from 1
  uint32_t nth;
  int owner;
};

// A position in cumulated counts and masses: a bin, and what lies before and in it.
struct Place {
  int bin;
  uint32_t count_before, count;
  unsigned long long mass_before, mass;
};

enum { BY_COUNT = 0, BY_MASS = 1, BY_BIN = 2 };

struct Shared {
  unsigned long long table[64];
  unsigned long long wide_mass[3];   // bf16: masses of the wide bins (B_MID relative to 2^-10 in regular rows)
  unsigned long long scan_mass[S_WARPS];
  uint32_t scan_count[S_WARPS];
  Place place;
  Command cmd;
  uint32_t max_key;                  // of this CTA's slice
  uint32_t row_max;
  int irregular;
  uint32_t found;
  uint32_t warp_count[S_WARPS];
};

template <bool F32>
struct Layout {
  using K = Key<F32>;
  // bytes of dynamic shared memory, masses first
  static constexpr int MASS = 0;                                          // F32: masses of the slice's bins
  static constexpr int MERGED_MASS = MASS + (F32 ? NB * 8 : 0);           // of the row's (first CTA)
  static constexpr int MASS2 = MERGED_MASS + NB * 8 + 8 * (NB & 1);       // finer counts: the slice's (F32: in place of MASS)
  static constexpr int MERGED_MASS2 = MASS2 + (F32 ? 0 : K::NB2 * 8);
  static constexpr int COUNT = MERGED_MASS2 + K::NB2 * 8;
  static constexpr int MERGED = COUNT + NB * 4;
  static constexpr int COUNT2 = MERGED + NB * 4;
  static constexpr int MERGED2 = COUNT2 + (F32 ? 0 : K::NB2 * 4);
  static constexpr int BYTES = MERGED2 + K::NB2 * 4;
};

// This CTA's part of a row: 16-byte groups g0 .. g1 - 1, group g holding logits g * GROUP - shift onwards
// (groups lie on 16-byte boundaries wherever the row starts; logits outside the row read as -inf).
template <bool F32>
struct Slice {
  using K = Key<F32>;
  const char* base;   // of group 0
  int shift, vocab, g0, g1;

  NVFP4_DEV uint4 load(int g) const {
    const int first = g * K::GROUP - shift;
    if (first >= 0 && first + K::GROUP <= vocab) return __ldg(reinterpret_cast<const uint4*>(base) + g);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (F32) {
        const int j = first + i;
        w[i] = j >= 0 && j < vocab ? __ldg(reinterpret_cast<const uint32_t*>(base) + g * 4 + i) : 0xFF800000u;
      } else {
        uint32_t h[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = first + 2 * i + e;
          h[e] = j >= 0 && j < vocab ? __ldg(reinterpret_cast<const unsigned short*>(base) + g * 8 + 2 * i + e) : 0xFF80u;
        }
        w[i] = h[0] | h[1] << 16;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }

  static NVFP4_DEV uint32_t bits(const uint4& u, int e) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    return F32 ? w[e] : (e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu;
  }

  // f(key) for every logit of the slice that can be drawn.
  template <typename F>
  NVFP4_DEV void each(F f) const {
    int g = g0 + threadIdx.x;
    for (; g + 3 * S_THREADS < g1; g += 4 * S_THREADS) {
      uint4 u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = load(g + i * S_THREADS);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < K::GROUP; ++e)
          if (const uint32_t k = key_of<F32>(bits(u[i], e))) f(k);
    }
    for (; g < g1; g += S_THREADS) {
      const uint4 u = load(g);
#pragma unroll
      for (int e = 0; e < K::GROUP; ++e)
        if (const uint32_t k = key_of<F32>(bits(u, e))) f(k);
    }
  }
};

// Cumulated counts and masses of n bins, and the search in them (a whole CTA).
struct Cumulated {
  const uint32_t* count;
  const unsigned long long* mass;
  int first, last;                 // this thread's bins
  uint32_t count_before, count_sum;
  unsigned long long mass_before, mass_sum, total;

  // afterwards total counts and masses are in sh.place
  NVFP4_DEV void build(Shared& sh, const uint32_t* c, const unsigned long long* m, int n) {
    count = c;
    mass = m;
    const int per = (n + S_THREADS - 1) / S_THREADS, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    first = min(static_cast<int>(threadIdx.x) * per, n);
    last = min(first + per, n);
    count_sum = 0;
    mass_sum = 0;
    for (int b = first; b < last; ++b) {
      count_sum += c[b];
      mass_sum += m[b];
    }
    uint32_t cs = count_sum;
    unsigned long long ms = mass_sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t cu = __shfl_up_sync(0xffffffffu, cs, o);
      const unsigned long long mu = __shfl_up_sync(0xffffffffu, ms, o);
      if (lane >= o) cs += cu, ms += mu;
    }
    if (lane == 31) sh.scan_count[warp] = cs, sh.scan_mass[warp] = ms;
    __syncthreads();
    uint32_t c0 = 0;
    unsigned long long m0 = 0;
    for (int w = 0; w < warp; ++w) c0 += sh.scan_count[w], m0 += sh.scan_mass[w];
    count_before = c0 + cs - count_sum;
    mass_before = m0 + ms - mass_sum;
    if (threadIdx.x == S_THREADS - 1) sh.place.count = c0 + cs, sh.place.mass = m0 + ms;
    __syncthreads();
    total = sh.place.mass;
  }

  // The bin in which the cumulated count (or mass) reaches `target`, or bin `target` itself.
  NVFP4_DEV Place find(Shared& sh, int how, unsigned long long target) const {
    // (the middle bin's mass is that of its parts up to a rounding)
    if (how == BY_MASS) target = min(target, total);
    if (how == BY_MASS && total == 0) how = BY_COUNT, target = 1;
    __syncthreads();   // the last place has been read
    const bool mine = how == BY_BIN     ? static_cast<int>(target) >= first && static_cast<int>(target) < last
                      : how == BY_COUNT ? count_before < target && target <= count_before + count_sum
                                        : mass_before < target && target <= mass_before + mass_sum;
    if (mine) {
      uint32_t c = count_before;
      unsigned long long m = mass_before;
      int b = first;
      for (; b < last - 1; ++b) {
        if (how == BY_BIN ? b == static_cast<int>(target) : how == BY_COUNT ? target <= c + count[b] : target <= m + mass[b]) break;
        c += count[b];
        m += mass[b];
      }
      sh.place = {b, c, count[b], m, mass[b]};
    }
    __syncthreads();
    return sh.place;
  }
};

template <bool F32>
__global__ void __launch_bounds__(S_THREADS, 2) sample_kernel(const SampleArgs a, int ctas) {
  using K = Key<F32>;
  using L = Layout<F32>;
  extern __shared__ __align__(16) char smem[];
  __shared__ Shared sh;
  auto at_mass = [&](int o) { return reinterpret_cast<unsigned long long*>(smem + o); };
  auto at_count = [&](int o) { return reinterpret_cast<uint32_t*>(smem + o); };
  unsigned long long* const mass = at_mass(L::MASS);
  unsigned long long* const merged_mass = at_mass(L::MERGED_MASS);
  unsigned long long* const mass2 = at_mass(F32 ? L::MASS : L::MASS2);
  unsigned long long* const merged_mass2 = at_mass(L::MERGED_MASS2);
  uint32_t* const count = at_count(L::COUNT);
  uint32_t* const merged = at_count(L::MERGED);
  uint32_t* const count2 = at_count(F32 ? L::COUNT : L::COUNT2);
  uint32_t* const merged2 = at_count(L::MERGED2);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x) % ctas, row = static_cast<int>(blockIdx.x) / ctas;
  const bool first_cta = rank == 0;

  if (tid < 64) sh.table[tid] = EXP2_TABLE[tid];
  if (tid < 3) sh.wide_mass[tid] = 0;
  if (tid == 0) sh.max_key = 0;
  for (int b = tid; b < NB; b += S_THREADS) {
    count[b] = 0;
    if (F32) mass[b] = 0;
  }
  pdl_wait();
  pdl_launch_dependents();

  const int entry = row / a.rows_each;
  const float temperature = a.set.temperature ? a.set.temperature[entry] : a.set.temperature_all;
  const bool greedy = !(temperature > 0.f);
  const Slope slope = slope_of(greedy ? 1.f : temperature);

  Slice<F32> slice;
  {
    const char* p = static_cast<const char*>(a.logits) + static_cast<int64_t>(row) * a.stride * (F32 ? 4 : 2);
    slice.shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) / (F32 ? 4 : 2);
    slice.base = p - slice.shift * (F32 ? 4 : 2);
    slice.vocab = a.vocab;
    const int groups = (a.vocab + slice.shift + K::GROUP - 1) / K::GROUP, per = (groups + ctas - 1) / ctas;
    slice.g0 = min(rank * per, groups);
    slice.g1 = min(slice.g0 + per, groups);
  }
  __syncthreads();

  // the slice's largest key, and its counts
  {
    uint32_t most = 0;
    if (greedy || F32) {
      slice.each([&](uint32_t k) { most = max(most, k); });
    } else {
      const float edge = 0x1p-10f;
      unsigned long long mid = 0;
      slice.each([&](uint32_t k) {
        most = max(most, k);
        const int b = bin_of(k);
        atomicAdd(count + b, 1u);
        if (b == B_MID) mid += rare_weight(edge, value_of<false>(k), slope, sh.table);
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mid += __shfl_xor_sync(0xffffffffu, mid, o);
      if (lane == 0 && mid) atomicAdd(&sh.wide_mass[1], mid);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&sh.max_key, most);
  }
  cluster_sync_all();
  // the row's, and (greedy) the first CTA that has it; whether the wide bins' masses have to be taken token by token
  if (warp == 0) {
    const uint32_t most = lane < ctas ? *in_cta(&sh.max_key, lane) : 0u;
    const uint32_t row_max = __reduce_max_sync(0xffffffffu, most);
    const unsigned holders = __ballot_sync(0xffffffffu, lane < ctas && most == row_max);
    int irregular = 0;
    if (!F32 && !greedy && row_max) {
      uint32_t top = lane < ctas ? *in_cta(count, lane) : 0u, mid = lane < ctas ? *in_cta(count + B_MID, lane) : 0u;
      uint32_t low = lane < ctas ? *in_cta(count + B_LAST, lane) : 0u;
      top = __reduce_add_sync(0xffffffffu, top);
      mid = __reduce_add_sync(0xffffffffu, mid);
      low = __reduce_add_sync(0xffffffffu, low);
      const float best = value_of<F32>(row_max);
      const bool above = row_max >= POS_LOW;   // the middle bin's masses are relative to 2^-10
      irregular = top > 0 || (mid > 0 && (!above || (slope.hi > 739.f && weight(best, 0x1p-10f, slope, sh.table) > 0))) ||
                  (low > 0 && (best < -128.f || weight(best, -128.f, slope, sh.table) > 0));
    }
    if (lane == 0) {
      sh.row_max = row_max;
      sh.irregular = irregular;
      sh.cmd = {CMD_FIND, 0u, 0u, 0, row_max, 1u, __ffs(holders) - 1};
    }
  }
  __syncthreads();
  const uint32_t row_max = sh.row_max;
  const float best = value_of<F32>(row_max);
  const bool drawn = row_max != 0 && !greedy;    // the same in every CTA of the cluster
  float prob = row_max ? 1.f : 0.f;

  // Counts (and masses) of the keys lo .. hi by parts of 2^shift, joined in the first CTA.
  auto refine = [&](uint32_t lo, uint32_t hi, int shift) {
    for (int b = tid; b < K::NB2; b += S_THREADS) count2[b] = 0, mass2[b] = 0;
    __syncthreads();
    slice.each([&](uint32_t k) {
      if (k < lo || k > hi) return;
      const uint32_t b = (hi - k) >> shift;
      atomicAdd(count2 + b, 1u);
      if (shift > 0)
        if (const unsigned long long w = rare_weight(best, value_of<F32>(k), slope, sh.table)) atomicAdd(mass2 + b, w);
    });
    cluster_sync_all();
    const int per = (K::NB2 + ctas - 1) / ctas;
    for (int b = rank * per + tid; b < min((rank + 1) * per, K::NB2); b += S_THREADS) {
      uint32_t c = 0;
      unsigned long long m = 0;
      for (int r = 0; r < ctas; ++r) c += *in_cta(count2 + b, r);
      if (shift == 0) {
        if (c) m = c * weight(best, value_of<F32>(hi - b), slope, sh.table);
      } else if (c) {
        for (int r = 0; r < ctas; ++r) m += *in_cta(mass2 + b, r);
      }
      *in_cta(merged2 + b, 0) = c;
      *in_cta(merged_mass2 + b, 0) = m;
    }
    cluster_sync_all();
  };

  if (drawn) {
    if (F32 || sh.irregular) {
      if (!F32 && tid < 3) sh.wide_mass[tid] = 0;
      __syncthreads();
      slice.each([&](uint32_t k) {
        const int b = bin_of(k >> K::LOW);
        if (F32) {
          atomicAdd(count + b, 1u);
          if (const unsigned long long w = weight(best, value_of<F32>(k), slope, sh.table)) atomicAdd(mass + b, w);
        } else if (wide_bin(b)) {
          const unsigned long long w = rare_weight(best, value_of<F32>(k), slope, sh.table);
          if (w) atomicAdd(&sh.wide_mass[b == 0 ? 0 : b == B_MID ? 1 : 2], w);
        }
      });
      cluster_sync_all();
    }
    // each CTA joins its share of the bins
    const int per = (NB + ctas - 1) / ctas;
    for (int b = rank * per + tid; b < min((rank + 1) * per, NB); b += S_THREADS) {
      uint32_t c = 0;
      unsigned long long m = 0;
      for (int r = 0; r < ctas; ++r) c += *in_cta(count + b, r);
      if (c) {
        if (F32) {
          for (int r = 0; r < ctas; ++r) m += *in_cta(mass + b, r);
        } else if (!wide_bin(b)) {
          uint32_t h, same;
          bin_range(b, h, same);
          m = c * weight(best, value_of<false>(h), slope, sh.table);
        } else {
          for (int r = 0; r < ctas; ++r) m += *in_cta(&sh.wide_mass[b == 0 ? 0 : b == B_MID ? 1 : 2], r);
          if (!sh.irregular) {   // a regular row: the middle bin's, relative to 2^-10 so far; nothing in the others
            const unsigned long long w = b == B_MID ? weight(best, 0x1p-10f, slope, sh.table) : 0ull;
            m = __umul64hi(m, w) << (64 - W_BITS) | (m * w) >> W_BITS;
          }
        }
      }
      *in_cta(merged + b, 0) = c;
      *in_cta(merged_mass + b, 0) = m;
    }
    cluster_sync_all();
  }

  if (drawn && first_cta) {
    Cumulated all;
    all.build(sh, merged, merged_mass, NB);
    const uint32_t tokens = sh.place.count;
    unsigned long long W = sh.place.mass;
    Command next = {};
    bool from_refined = false;

    auto send = [&](const Command& c) {
      __syncthreads();
      if (tid < ctas) *in_cta(&sh.cmd, tid) = c;
      cluster_sync_all();
    };
    // The key at a position, its weight, and what lies before it; counts of the last, finest step stay in
    // count2 and merged2 when the position needed one (`refined`).
    auto resolve = [&](int how, unsigned long long target, uint32_t target_key, uint32_t& key, unsigned long long& w, bool& refined) {
      Place p = all.find(sh, how, how == BY_BIN ? bin_of(target_key >> K::LOW) : target);
      refined = p.count > 0 && (F32 || wide_bin(p.bin));
      uint32_t lo, hi;
      bin_range(p.bin, lo, hi);
      lo <<= K::LOW;
      hi = (hi << K::LOW) | ((1u << K::LOW) - 1u);
      if (p.bin == 0) hi = K::PINF;
      if (refined) {
        uint32_t c0 = p.count_before;
        unsigned long long m0 = p.mass_before;
        for (;;) {
          int shift = 0;
          while (((hi - lo) >> shift) >= static_cast<uint32_t>(K::NB2)) ++shift;
          send({CMD_REFINE, lo, hi, shift, 0u, 0u, 0});
          refine(lo, hi, shift);
          Cumulated part;
          part.build(sh, merged2, merged_mass2, K::NB2);
          p = part.find(sh, how, how == BY_BIN ? (hi - target_key) >> shift : how == BY_COUNT ? target - c0 : target - m0);
          p.count_before += c0;
          p.mass_before += m0;
          c0 = p.count_before;
          m0 = p.mass_before;
          const uint32_t top = hi - (static_cast<uint32_t>(p.bin) << shift);
          hi = top;
          if (shift == 0) break;
          const uint32_t bottom = top - ((1u << shift) - 1u);
          lo = bottom > lo && bottom <= top ? bottom : lo;
        }
      }
      key = hi;
      w = weight(best, value_of<F32>(key), slope, sh.table);
      return p;
    };

    uint32_t key;
    unsigned long long w;
    const int k = a.set.top_k ? a.set.top_k[entry] : a.set.top_k_all;
    if (k > 0 && static_cast<uint32_t>(k) < tokens) {
      const Place p = resolve(BY_COUNT, k, 0u, key, w, from_refined);
      W = p.mass_before + (k - p.count_before) * w;
    }
    const float top_p = a.set.top_p ? a.set.top_p[entry] : a.set.top_p_all;
    if (top_p < 1.f) {
      bool cut = false;
      unsigned long long t = top_p > 0.f ? times(W, top_p, cut) : 0ull;
      t = max(t + cut, 1ull);
      const Place p = resolve(BY_MASS, t, 0u, key, w, from_refined);
      W = p.mass_before + (t - p.mass_before + w - 1) / max(w, 1ull) * w;
    }
    const float min_p = a.set.min_p ? a.set.min_p[entry] : a.set.min_p_all;
    if (min_p > 0.f) {
      // the lowest key that weighs enough, 32 keys at a time
      bool cut = false;
      const unsigned long long least = min_p < 1.f ? max(times(ONE, min_p, cut) + cut, 1ull) : ONE;
      uint32_t good = row_max, bad = 0;   // good weighs enough, bad does not (or is no token)
      while (good - bad > 1) {
        const uint32_t step = (good - bad + 31) / 32;
        const uint32_t probe = static_cast<uint32_t>(lane + 1) * step < good - bad ? good - (lane + 1) * step : bad;
        const bool ok = probe > bad && probe >= K::LOWEST && weight(best, value_of<F32>(probe), slope, sh.table) >= least;
        const int n = __ffs(~__ballot_sync(0xffffffffu, ok)) - 1;   // the first n probes; the last never is one
        bad = __shfl_sync(0xffffffffu, probe, n);
        good -= n * step;
      }
      const Place p = resolve(BY_BIN, 0, good, key, w, from_refined);
      W = min(W, p.mass_before + p.mass);
    }
    const float u = a.uniform[row];
    bool cut;
    const unsigned long long t = 1ull + (u > 0.f ? u < 1.f ? times(W, u, cut) : W - 1 : 0ull);
    const Place p = resolve(BY_MASS, t, 0u, key, w, from_refined);
    const unsigned long long n = (t - p.mass_before + w - 1) / max(w, 1ull);
    const uint32_t nth = n < 1 ? 1u : n > p.count ? p.count : static_cast<uint32_t>(n);
    int scale;   // (a light token's probability has more bits than its rounded weight)
    const float exact_w = __ull2float_rn(weight_and_scale(best, value_of<F32>(key), slope, sh.table, scale));
    prob = exact_w * __uint_as_float((127u - scale) << 23) / __ull2float_rn(W);
    // the CTA that holds the nth token of this key
    if (warp == 0) {
      const uint32_t mine = lane < ctas ? *in_cta((from_refined ? count2 : count) + p.bin, lane) : 0u;
      uint32_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const unsigned has = __ballot_sync(0xffffffffu, lane < ctas && upto >= nth);
      const int owner = has ? __ffs(has) - 1 : 0;
      next = {CMD_FIND, 0u, 0u, 0, key, nth - __shfl_sync(0xffffffffu, upto - mine, owner), owner};
    }
    send(next);   // (made and sent by the first warp)
    if (tid == 0 && a.probs) a.probs[row] = prob;
  } else if (drawn) {
    for (;;) {
      cluster_sync_all();
      const Command c = sh.cmd;
      __syncthreads();
      if (c.what == CMD_FIND) break;
      refine(c.lo, c.hi, c.shift);
    }
  } else if (first_cta && tid == 0 && a.probs) {
    a.probs[row] = prob;
  }

  if (row_max == 0) {
    if (first_cta && tid == 0) a.ids[row] = -1;
  } else if (sh.cmd.owner == rank) {
    // the nth token with the key: each warp counts a run of groups, the one that holds it counts again
    const uint32_t key = sh.cmd.key, nth = sh.cmd.nth;
    const int n = slice.g1 - slice.g0, per = (n + S_WARPS - 1) / S_WARPS;
    const int w0 = slice.g0 + min(warp * per, n), w1 = slice.g0 + min(warp * per + per, n);
    uint32_t mine = 0;
    for (int g = w0 + lane; g < w1; g += 32) {
      const uint4 u = slice.load(g);
#pragma unroll
      for (int e = 0; e < K::GROUP; ++e) mine += key_of<F32>(Slice<F32>::bits(u, e)) == key;
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) sh.warp_count[warp] = mine;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += sh.warp_count[w];
    if (before < nth && nth <= before + mine) {
      for (int g = w0; g < w1; g += 32) {
        const uint4 u = g + lane < w1 ? slice.load(g + lane) : make_uint4(~0u, ~0u, ~0u, ~0u);   // (NaN)
        uint32_t hits = 0;
#pragma unroll
        for (int e = 0; e < K::GROUP; ++e) hits += key_of<F32>(Slice<F32>::bits(u, e)) == key;
        uint32_t upto = hits;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        const uint32_t sum = __shfl_sync(0xffffffffu, upto, 31);
        if (before + sum >= nth) {
          uint32_t c = before + upto - hits;
          if (c < nth && nth <= c + hits) {
            for (int e = 0; e < K::GROUP; ++e)
              if (key_of<F32>(Slice<F32>::bits(u, e)) == key && ++c == nth) a.ids[row] = (g + lane) * K::GROUP - slice.shift + e;
          }
          break;
        }
        before += sum;
      }
    }
  }
  cluster_sync_all();   // no CTA leaves while another may read its shared memory
}

// Accepted drafts: the leading ones that are the token drawn at their position.
__global__ void accept_kernel(const int32_t* tokens, const int32_t* drafts, int64_t batch, int n_draft, int32_t* accepted) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t b = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (b >= batch) return;
  int n = 0;
  while (n < n_draft && tokens[b * (n_draft + 1) + n] == drafts[b * n_draft + n]) ++n;
  accepted[b] = n;
}

// Clusters of 16 CTAs have to be allowed for a kernel, once on each device.
int allow_wide_clusters(const void* kernel, int which) {
  static std::atomic<unsigned long long> done[2];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done[which].load() & bit) return NVFP4_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return NVFP4_ERR_CUDA;
  done[which].fetch_or(bit);
  return NVFP4_OK;
}

template <bool F32>
int launch_sample_type(const SampleArgs& a, int64_t rows, cudaStream_t stream) {
  const auto kernel = sample_kernel<F32>;
  if (int rc = ensure_smem(kernel, Layout<F32>::BYTES)) return rc;
  // as many CTAs for a row as the rows leave room for, none with less than 4096 logits
  int ctas = 1;
  while (ctas < 16 && rows * ctas <= sm_count() && a.vocab > 4096 * ctas) ctas *= 2;
  if (ctas > 8)
    if (int rc = allow_wide_clusters(reinterpret_cast<const void*>(kernel), F32)) return rc;
  return launch_ex(kernel, dim3(static_cast<unsigned>(rows * ctas)), dim3(S_THREADS), Layout<F32>::BYTES, ctas, true, stream, a, ctas);
}

}  // namespace

int launch_sample(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t stride, const nvfp4_sampling_t& set,
                  int rows_each, const float* uniform, int32_t* ids, float* probs, cudaStream_t stream) {
  const SampleArgs a = {logits, stride, static_cast<int>(vocab), rows_each, set, uniform, ids, probs};
  return dtype == NVFP4_DTYPE_F32 ? launch_sample_type<true>(a, rows, stream) : launch_sample_type<false>(a, rows, stream);
}

int launch_accept(const int32_t* tokens, const int32_t* drafts, int64_t batch, int n_draft, int32_t* accepted, cudaStream_t stream) {
  return launch_ex(accept_kernel, dim3(static_cast<unsigned>(ceil_div(batch, 128))), dim3(128), 0, 1, true, stream, tokens, drafts, batch,
                   n_draft, accepted);
}

}  // namespace nvfp4
