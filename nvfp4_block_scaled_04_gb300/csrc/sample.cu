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

// The sum of *p over the CTAs of the cluster, eight loads at a time.
template <typename T>
NVFP4_DEV T cluster_sum(T* p, int ctas) {
  T sum = 0;
  for (int r0 = 0; r0 < ctas; r0 += 8) {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r0 + i < ctas ? *in_cta(p, r0 + i) : T(0);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += v[i];
  }
  return sum;
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

constexpr int NB2 = 1024;         // parts of a finer count
constexpr int LIST = S_THREADS;   // tokens that the first CTA puts in order at once

enum { CMD_FIND = 0, CMD_REFINE = 1, CMD_GATHER = 2, CMD_END = 3 };

struct Command {
  int what;
  uint32_t lo, hi;       // REFINE: count keys lo .. hi by parts of 2^shift; GATHER: hand their tokens to the first CTA
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
  unsigned long long wide_mass[4];   // bf16: masses of the wide bins (the middle ones' relative to 2^-10 in regular rows)
  unsigned long long scan_mass[S_WARPS];
  uint32_t scan_count[S_WARPS];
  Place place;
  Command cmd;
  uint32_t max_key;                  // of this CTA's slice
  int min_bin;                       // bf16: its first bin that is not empty
  uint32_t row_max;
  int row_bin;
  int irregular;
  uint32_t list_n;
};

// Bytes of dynamic shared memory. `count`, `mass`: of this CTA's slice. `merged`: of the row (first CTA's). The finer
// counts lie over the slice's masses (F32), which have been joined by then.
template <bool F32>
struct Layout {
  static constexpr int FINE = NB2 * 24;                       // masses, joined masses, counts, joined counts
  static constexpr int MASS = 0;                              // F32: lower words, then upper words
  static constexpr int SLICE = F32 ? NB * 8 : FINE;
  static_assert(!F32 || NB * 8 >= FINE, "finer counts");
  static constexpr int MERGED_MASS = SLICE;
  static constexpr int COUNT = MERGED_MASS + NB * 8;
  static constexpr int MERGED = COUNT + NB * 4;
  static constexpr int ORDER = MERGED + NB * 4;               // the list: key and index, then cumulated masses
  static constexpr int BYTES = ORDER + LIST * 16;
};

// This CTA's part of a row: 16-byte groups g0 .. g1 - 1, group g holding logits g * GROUP - shift onwards
// (groups lie on 16-byte boundaries wherever the row starts; logits outside the row read as -inf).
template <bool F32>
struct Slice {
  using K = Key<F32>;
  static constexpr uint32_t NONE = F32 ? 0xFF800000u : 0xFF80FF80u;   // -inf
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
        w[i] = j >= 0 && j < vocab ? __ldg(reinterpret_cast<const uint32_t*>(base) + g * 4 + i) : NONE;
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

  // f(group's words, g) for every group of the slice, four loads at a time.
  template <typename F>
  NVFP4_DEV void groups(F f) const {
    for (int g = g0 + threadIdx.x; g < g1; g += 4 * S_THREADS) {
      uint4 u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (g + i * S_THREADS < g1) u[i] = load(g + i * S_THREADS);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (g + i * S_THREADS < g1) f(u[i], g + i * S_THREADS);
    }
  }

  // f(key, index) for every logit of the slice that can be drawn.
  template <typename F>
  NVFP4_DEV void each(F f) const {
    groups([&](const uint4& u, int g) {
#pragma unroll
      for (int e = 0; e < K::GROUP; ++e)
        if (const uint32_t k = key_of<F32>(bits(u, e))) f(k, g * K::GROUP - shift + e);
    });
  }
};

// Cumulated counts and masses of N bins, and the search in them (a whole CTA).
template <int N>
struct Cumulated {
  static constexpr int PER = (N + S_THREADS - 1) / S_THREADS;
  const uint32_t* count;
  const unsigned long long* mass;
  uint32_t count_before, count_sum, tokens;
  unsigned long long mass_before, mass_sum, total;

  NVFP4_DEV void build(Shared& sh, const uint32_t* c, const unsigned long long* m) {
    count = c;
    mass = m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = threadIdx.x * PER;
    count_sum = 0;
    mass_sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (first + i < N) {
        count_sum += c[first + i];
        mass_sum += m[first + i];
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
    tokens = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < S_WARPS; ++w) {
      if (w == warp) c0 = tokens, m0 = total;
      tokens += sh.scan_count[w];
      total += sh.scan_mass[w];
    }
    count_before = c0 + cs - count_sum;
    mass_before = m0 + ms - mass_sum;
  }

  // The bin in which the cumulated count (or mass) reaches `target`, or bin `target` itself.
  NVFP4_DEV Place find(Shared& sh, int how, unsigned long long target) const {
    // (a middle bin's mass is that of its parts up to a rounding)
    if (how == BY_MASS) target = min(target, total);
    if (how == BY_MASS && total == 0) how = BY_COUNT, target = 1;
    __syncthreads();   // the last place has been read, and the sums
    // (logits that another stream changes during the call may not be found again: the search still ends)
    if (threadIdx.x == 0) sh.place = {0, 0u, 0u, 0ull, 0ull};
    __syncthreads();
    const int first = threadIdx.x * PER;
    const bool mine = how == BY_BIN     ? static_cast<int>(target) / PER == threadIdx.x
                      : how == BY_COUNT ? count_before < target && target <= count_before + count_sum
                                        : mass_before < target && target <= mass_before + mass_sum;
    if (mine) {
      uint32_t c = count_before;
      unsigned long long m = mass_before;
      bool found = false;
      Place p = {0, 0u, 0u, 0ull, 0ull};
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = first + i;
        const uint32_t cb = b < N ? count[b] : 0u;
        const unsigned long long mb = b < N ? mass[b] : 0ull;
        const bool here = how == BY_BIN ? b == static_cast<int>(target) : how == BY_COUNT ? target <= c + cb : target <= m + mb;
        if (here && !found) {
          p = {b, c, cb, m, mb};
          found = true;
        }
        c += cb;
        m += mb;
      }
      sh.place = p;
    }
    __syncthreads();
    return sh.place;
  }
};

NVFP4_DEV uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// 0xFFFF in each half of w that is negative
NVFP4_DEV uint32_t signs(uint32_t w) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %1, 0xBB99;" : "=r"(d) : "r"(w));   // (a selector's upper bit spreads the byte's sign)
  return d;
}

// Adds to a 64-bit sum in two words (most weights fit into the lower one).
NVFP4_DEV void add_mass(uint32_t* lower, uint32_t* upper, unsigned long long w) {
  const uint32_t lo = static_cast<uint32_t>(w);
  const uint32_t old = atomicAdd(lower, lo);
  const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old ? 1u : 0u);
  if (hi) atomicAdd(upper, hi);
}

// The list's entry at this thread's place once 2^ceil entries (all of them in the first `n` threads) are in rising order.
NVFP4_DEV unsigned long long sort_list(unsigned long long v, int n, unsigned long long* room) {
  const int t = threadIdx.x;
  for (int k = 2; k < 2 * n; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      unsigned long long other;
      if (j >= 32) {
        __syncthreads();
        room[t] = v;
        __syncthreads();
        other = room[t ^ j];
      } else {
        other = __shfl_xor_sync(0xffffffffu, v, j);
      }
      const bool low = (t & j) == 0, up = (t & k) == 0;
      v = (v < other) == (low == up) ? v : other;
    }
  }
  return v;
}

template <bool F32>
__global__ void __launch_bounds__(S_THREADS, 2) sample_kernel(const SampleArgs a, int ctas) {
  using K = Key<F32>;
  using L = Layout<F32>;
  extern __shared__ __align__(16) char smem[];
  __shared__ Shared sh;
  uint32_t* const mass_lo = reinterpret_cast<uint32_t*>(smem + L::MASS);
  uint32_t* const mass_hi = mass_lo + NB;
  unsigned long long* const mass2 = reinterpret_cast<unsigned long long*>(smem + L::MASS);
  unsigned long long* const merged_mass2 = mass2 + NB2;
  uint32_t* const count2 = reinterpret_cast<uint32_t*>(merged_mass2 + NB2);
  uint32_t* const merged2 = count2 + NB2;
  unsigned long long* const merged_mass = reinterpret_cast<unsigned long long*>(smem + L::MERGED_MASS);
  uint32_t* const count = reinterpret_cast<uint32_t*>(smem + L::COUNT);
  uint32_t* const merged = reinterpret_cast<uint32_t*>(smem + L::MERGED);
  unsigned long long* const order = reinterpret_cast<unsigned long long*>(smem + L::ORDER);
  unsigned long long* const upto = order + LIST;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x) % ctas, row = static_cast<int>(blockIdx.x) / ctas;
  const bool first_cta = rank == 0;

  if (tid < 64) sh.table[tid] = EXP2_TABLE[tid];
  if (tid < 4) sh.wide_mass[tid] = 0;
  if (tid == 0) sh.max_key = 0, sh.min_bin = NB, sh.list_n = 0;
  for (int b = tid; b < NB; b += S_THREADS) {
    count[b] = 0;
    if (F32) mass_lo[b] = 0, mass_hi[b] = 0;
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

  // The slice's largest key (into sh.max_key; the caller synchronises).
  auto find_max = [&]() {
    uint32_t most = 0;
    slice.each([&](uint32_t k, int) { most = max(most, k); });
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&sh.max_key, most);
  };
  // The row's largest key, and which of the cluster's CTAs has it first, after a cluster barrier (the first warp's answer).
  auto row_max_of = [&](int& holder) {
    const uint32_t most = lane < ctas ? *in_cta(&sh.max_key, lane) : 0u;
    const uint32_t row = __reduce_max_sync(0xffffffffu, most);
    holder = __ffs(__ballot_sync(0xffffffffu, lane < ctas && most == row)) - 1;
    return row;
  };

  if (F32 || greedy) {
    find_max();
    cluster_sync_all();
    if (warp == 0) {
      int holder;
      const uint32_t most = row_max_of(holder);
      if (lane == 0) {
        sh.row_max = most;
        sh.irregular = 0;
        sh.cmd = {CMD_FIND, 0u, 0u, 0, most, 1u, holder};
      }
    }
    __syncthreads();
  } else {
    // Counts. Two logits of a word at a time: clamped magnitudes give the bins; groups with a magnitude below 2^-10
    // go logit by logit, and what lies in the middle bins is weighed on the way (relative to 2^-10).
    unsigned long long mid[2] = {0ull, 0ull};
    uint32_t* const middle = count + B_MID;
    slice.groups([&](const uint4& u, int) {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = w[i] & 0x7FFF7FFFu;
      const uint32_t least = min_u16x2(min_u16x2(m[0], m[1]), min_u16x2(m[2], m[3]));
      if (min_u16x2(least, MAG_LOW * 0x10001u) == MAG_LOW * 0x10001u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t s = bin_steps(min_u16x2(m[i], MAG_TOP * 0x10001u), signs(w[i]));
          atomicAdd(middle - static_cast<int16_t>(s & 0xFFFFu), 1u);
          atomicAdd(middle - (static_cast<int32_t>(s) >> 16), 1u);
        }
      } else {
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
          const uint32_t word = e < 4 ? (e < 2 ? u.x : u.y) : (e < 6 ? u.z : u.w);
          const uint32_t k = key_of<false>((e & 1) ? word >> 16 : word & 0xFFFFu);
          if (k == 0) continue;
          const int b = bin_of(k);
          atomicAdd(count + b, 1u);
          if (b == B_MID || b == B_MID + 1) {
            const unsigned long long v = weight(0x1p-10f, value_of<false>(k), slope, sh.table);
            if (b == B_MID) mid[0] += v;
            else mid[1] += v;
          }
        }
      }
    });
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (__any_sync(0xffffffffu, mid[i] != 0)) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mid[i] += __shfl_xor_sync(0xffffffffu, mid[i], o);
        if (lane == 0) atomicAdd(&sh.wide_mass[1 + i], mid[i]);
      }
    }
    __syncthreads();
    // the first bin that is not empty: the largest logit, where it is a bin of one value
    int first = NB;
    for (int b = tid; b < NB; b += S_THREADS)
      if (count[b]) {
        first = b;
        break;
      }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) atomicMin(&sh.min_bin, first);
    cluster_sync_all();
    if (warp == 0) {
      int bin = lane < ctas ? *in_cta(&sh.min_bin, lane) : NB;
      const uint32_t mid_any = lane < ctas ? *in_cta(count + B_MID, lane) + *in_cta(count + B_MID + 1, lane) : 0u;
      const uint32_t low_any = lane < ctas ? *in_cta(count + B_LAST, lane) : 0u;
      bin = __reduce_min_sync(0xffffffffu, bin);
      const bool mids = __any_sync(0xffffffffu, mid_any != 0), lows = __any_sync(0xffffffffu, low_any != 0);
      uint32_t key = 0, same;
      int irregular = bin == NB || wide_bin(bin) >= 0;
      if (!irregular) {
        bin_range(bin, key, same);
        const float best = value_of<false>(key);
        irregular = (mids && bin < B_MID && slope.hi > 739.f && weight(best, 0x1p-10f, slope, sh.table) > 0) ||
                    (lows && weight(best, -128.f, slope, sh.table) > 0);
      }
      if (lane == 0) {
        sh.row_max = key;
        sh.irregular = irregular;
      }
    }
    __syncthreads();
    if (sh.irregular) {
      // Largest logits in a wide bin, weights that a wide bin's figures do not serve: these bins logit by logit.
      find_max();
      cluster_sync_all();
      if (warp == 0) {
        int holder;
        const uint32_t most = row_max_of(holder);
        if (lane == 0) sh.row_max = most;
      }
      if (tid < 4) {
        sh.wide_mass[tid] = 0;
        count[tid == 0 ? 0 : tid == 3 ? B_LAST : B_MID + tid - 1] = 0;
      }
      __syncthreads();
      const float best = value_of<false>(sh.row_max);
      slice.each([&](uint32_t k, int) {
        const int b = bin_of(k), n = wide_bin(b);
        if (n < 0) return;
        atomicAdd(count + b, 1u);
        if (const unsigned long long w = rare_weight(best, value_of<false>(k), slope, sh.table)) atomicAdd(&sh.wide_mass[n], w);
      });
      cluster_sync_all();
    }
  }
  const uint32_t row_max = sh.row_max;
  const float best = value_of<F32>(row_max);
  const bool drawn = row_max != 0 && !greedy;    // the same in every CTA of the cluster

  // Counts (and masses) of the keys lo .. hi by parts of 2^shift, joined in the first CTA.
  auto refine = [&](uint32_t lo, uint32_t hi, int shift) {
    for (int b = tid; b < NB2; b += S_THREADS) count2[b] = 0, mass2[b] = 0;
    __syncthreads();
    slice.each([&](uint32_t k, int) {
      if (k < lo || k > hi) return;
      const uint32_t b = (hi - k) >> shift;
      atomicAdd(count2 + b, 1u);
      if (shift > 0)
        if (const unsigned long long w = rare_weight(best, value_of<F32>(k), slope, sh.table)) atomicAdd(mass2 + b, w);
    });
    cluster_sync_all();
    const int per = (NB2 + ctas - 1) / ctas;
    for (int b = rank * per + tid; b < min((rank + 1) * per, NB2); b += S_THREADS) {
      const uint32_t c = cluster_sum(count2 + b, ctas);
      unsigned long long m = 0;
      if (shift == 0) {
        if (c) m = c * weight(best, value_of<F32>(hi - b), slope, sh.table);
      } else if (c) {
        m = cluster_sum(mass2 + b, ctas);
      }
      *in_cta(merged2 + b, 0) = c;
      *in_cta(merged_mass2 + b, 0) = m;
    }
    cluster_sync_all();
  };
  // The tokens with keys lo .. hi into the first CTA's list (in no order yet).
  auto gather = [&](uint32_t lo, uint32_t hi) {
    slice.each([&](uint32_t k, int index) {
      if (k < lo || k > hi) return;
      const uint32_t at = atomicAdd(in_cta(&sh.list_n, 0), 1u);
      if (at < LIST) *in_cta(order + at, 0) = static_cast<unsigned long long>(~k) << 32 | static_cast<uint32_t>(index);
    });
    cluster_sync_all();
  };

  if (drawn) {
    if (F32) {
      slice.each([&](uint32_t k, int) {
        const int b = bin_of(k >> K::LOW);
        atomicAdd(count + b, 1u);
        if (const unsigned long long w = weight(best, value_of<F32>(k), slope, sh.table)) add_mass(mass_lo + b, mass_hi + b, w);
      });
      cluster_sync_all();
    }
    // each CTA joins its share of the bins
    const int per = (NB + ctas - 1) / ctas;
    for (int b = rank * per + tid; b < min((rank + 1) * per, NB); b += S_THREADS) {
      uint32_t c = cluster_sum(count + b, ctas);
      unsigned long long m = 0;
      if (c) {
        const int wide = wide_bin(b);
        if (F32) {
          for (int r = 0; r < ctas; ++r)
            m += static_cast<unsigned long long>(*in_cta(mass_hi + b, r)) << 32 | *in_cta(mass_lo + b, r);
        } else if (wide < 0) {
          uint32_t h, same;
          bin_range(b, h, same);
          m = c * weight(best, value_of<false>(h), slope, sh.table);
        } else if (sh.irregular) {
          m = cluster_sum(&sh.wide_mass[wide], ctas);
        } else if (wide == 3) {
          c = 0;   // nothing in it weighs anything (and -inf and NaN were counted too)
        } else {   // a middle bin, relative to 2^-10 so far
          m = cluster_sum(&sh.wide_mass[wide], ctas);
          const unsigned long long w = weight(best, 0x1p-10f, slope, sh.table);
          m = __umul64hi(m, w) << (64 - W_BITS) | (m * w) >> W_BITS;
        }
      }
      *in_cta(merged + b, 0) = c;
      *in_cta(merged_mass + b, 0) = m;
    }
    cluster_sync_all();
  }

  float prob = row_max ? 1.f : 0.f;
  if (drawn && first_cta) {
    Cumulated<NB> all;
    all.build(sh, merged, merged_mass);
    unsigned long long W = all.total;

    auto send = [&](const Command& c) {
      __syncthreads();
      if (tid < ctas) *in_cta(&sh.cmd, tid) = c;
      cluster_sync_all();
    };
    // the list in order: tokens with keys of list_lo and up, of which list_n are there, from count list_c0 and mass list_m0 on
    int list_n = 0;
    uint32_t list_lo = 0, list_hi = 0, list_c0 = 0;
    unsigned long long list_m0 = 0, list_mass = 0;
    auto make_list = [&](uint32_t lo, uint32_t hi, uint32_t c0, unsigned long long m0) {
      __syncthreads();
      if (tid == 0) sh.list_n = 0;
      send({CMD_GATHER, lo, hi, 0, 0u, 0u, 0});
      gather(lo, hi);
      list_n = min(sh.list_n, static_cast<uint32_t>(LIST));
      list_lo = lo;
      list_hi = hi;
      list_c0 = c0;
      list_m0 = m0;
      const unsigned long long v = sort_list(tid < list_n ? order[tid] : ~0ull, list_n, upto);
      unsigned long long m = tid < list_n ? weight(best, value_of<F32>(~static_cast<uint32_t>(v >> 32) & K::ALL), slope, sh.table) : 0ull;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long mu = __shfl_up_sync(0xffffffffu, m, o);
        if (lane >= o) m += mu;
      }
      __syncthreads();
      if (lane == 31) sh.scan_mass[warp] = m;
      order[tid] = v;
      __syncthreads();
      for (int i = 0; i < warp; ++i) m += sh.scan_mass[i];
      upto[tid] = m;
      __syncthreads();
      list_mass = list_n ? upto[list_n - 1] : 0ull;
    };
    // What a search found: how many tokens lie before the one at the position, their mass, the token's weight, the mass
    // through it; its key, and its index (-1: the nth of its key, a bin of the slices' counts `where`).
    struct Found {
      uint32_t key, nth;
      int index;
      const uint32_t* where;
      unsigned long long through;
    };
    // The position where the cumulated count or mass reaches target, or (BY_BIN) the last token with a key of target or more.
    auto resolve = [&](int how, unsigned long long target) {
      Found f = {0u, 0u, -1, nullptr, 0ull};
      auto in_list = [&]() {
        return list_n > 0 && (how == BY_BIN     ? target >= list_lo && target <= list_hi
                              : how == BY_COUNT ? target > list_c0 && target - list_c0 <= static_cast<unsigned>(list_n)
                                                : target > list_m0 && target - list_m0 <= list_mass);
      };
      auto from_list = [&]() {
        int i;
        if (how == BY_COUNT) {
          i = static_cast<int>(target - list_c0) - 1;
        } else if (how == BY_MASS) {
          i = __syncthreads_count(tid < list_n && list_m0 + upto[tid] < target);
          i = min(i, list_n - 1);
        } else {
          i = __syncthreads_count(tid < list_n && (~static_cast<uint32_t>(order[tid] >> 32) & K::ALL) >= target) - 1;
        }
        f.through = list_m0 + (i >= 0 ? upto[i] : 0ull);
        f.key = i >= 0 ? ~static_cast<uint32_t>(order[i] >> 32) & K::ALL : 0u;
        f.index = i >= 0 ? static_cast<int>(static_cast<uint32_t>(order[i])) : -1;
      };
      if (in_list()) {
        from_list();
        return f;
      }
      Place p = all.find(sh, how, how == BY_BIN ? bin_of(static_cast<uint32_t>(target) >> K::LOW) : target);
      uint32_t lo, hi;
      bin_range(p.bin, lo, hi);
      lo <<= K::LOW;
      hi = (hi << K::LOW) | ((1u << K::LOW) - 1u);
      if (p.bin == 0) hi = K::PINF;
      f.where = count + p.bin;
      if (F32 || wide_bin(p.bin) >= 0) {
        uint32_t c0 = p.count_before;
        unsigned long long m0 = p.mass_before;
        while (p.count > 0 && hi >= lo) {
          if (p.count <= LIST) {
            // few tokens: in order, with all before them where these are few as well
            if (c0 + p.count <= LIST) make_list(lo, K::PINF, 0u, 0ull);
            else make_list(lo, hi, c0, m0);
            if (list_n == 0) break;   // (they are gone)
            if (how == BY_MASS) target = min(target, list_m0 + list_mass);
            from_list();
            return f;
          }
          int shift = 0;
          while (((hi - lo) >> shift) >= static_cast<uint32_t>(NB2)) ++shift;
          send({CMD_REFINE, lo, hi, shift, 0u, 0u, 0});
          refine(lo, hi, shift);
          Cumulated<NB2> part;
          part.build(sh, merged2, merged_mass2);
          p = part.find(sh, how, how == BY_BIN ? (hi - static_cast<uint32_t>(target)) >> shift : how == BY_COUNT ? target - c0 : target - m0);
          f.where = count2 + p.bin;
          p.count_before += c0;
          p.mass_before += m0;
          c0 = p.count_before;
          m0 = p.mass_before;
          hi -= static_cast<uint32_t>(p.bin) << shift;
          if (shift == 0) break;
          const uint32_t bottom = hi - ((1u << shift) - 1u);
          lo = bottom > lo && bottom <= hi ? bottom : lo;
        }
      }
      // one key
      f.key = hi;
      const unsigned long long w = weight(best, value_of<F32>(hi), slope, sh.table);
      f.nth = how == BY_BIN     ? p.count
              : how == BY_COUNT ? static_cast<uint32_t>(target) - p.count_before
                                : few_times(target - p.mass_before, w);
      f.nth = max(1u, min(f.nth, p.count));
      f.through = p.mass_before + min(f.nth, p.count) * w;
      return f;
    };

    const int k = a.set.top_k ? a.set.top_k[entry] : a.set.top_k_all;
    const float top_p = a.set.top_p ? a.set.top_p[entry] : a.set.top_p_all;
    const float min_p = a.set.min_p ? a.set.min_p[entry] : a.set.min_p_all;
    const float u = a.uniform[row];
    if (k > 0 && static_cast<uint32_t>(k) < all.tokens) W = resolve(BY_COUNT, k).through;
    if (top_p < 1.f) {
      bool cut = false;
      const unsigned long long t = top_p > 0.f ? times(W, top_p, cut) : 0ull;
      W = resolve(BY_MASS, max(t + cut, 1ull)).through;
    }
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
      W = min(W, resolve(BY_BIN, good).through);
    }
    bool cut;
    const Found f = resolve(BY_MASS, 1ull + (u > 0.f ? u < 1.f ? times(W, u, cut) : W - 1 : 0ull));
    int scale;   // (a light token's probability has more bits than its rounded weight)
    const float w = __ull2float_rn(weight_and_scale(best, value_of<F32>(f.key), slope, sh.table, scale));
    prob = w * __uint_as_float((127u - scale) << 23) / __ull2float_rn(W);
    Command next = {CMD_END, 0u, 0u, 0, 0u, 0u, 0};
    if (f.index < 0 && warp == 0) {
      // the CTA that holds the nth token of this key
      const uint32_t mine = lane < ctas ? *in_cta(f.where, lane) : 0u;
      uint32_t sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const unsigned has = __ballot_sync(0xffffffffu, lane < ctas && sum >= f.nth);
      const int owner = has ? __ffs(has) - 1 : 0;
      next = {CMD_FIND, 0u, 0u, 0, f.key, f.nth - __shfl_sync(0xffffffffu, sum - mine, owner), owner};
    }
    send(next);   // (made and sent by the first warp)
    if (tid == 0 && f.index >= 0) a.ids[row] = f.index;
  } else if (drawn) {
    for (;;) {
      cluster_sync_all();
      const Command c = sh.cmd;
      __syncthreads();
      if (c.what == CMD_REFINE) refine(c.lo, c.hi, c.shift);
      else if (c.what == CMD_GATHER) gather(c.lo, c.hi);
      else break;
    }
  }
  if (first_cta && tid == 0) {
    if (a.probs) a.probs[row] = prob;
    if (row_max == 0) a.ids[row] = -1;
  }

  if (row_max != 0 && sh.cmd.what == CMD_FIND && sh.cmd.owner == rank) {
    // the nth token with the key: the warps count equal runs of groups, and again inside the run that holds it
    const float value = value_of<F32>(sh.cmd.key);
    const uint32_t zero = value == 0.f ? (F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu) : ~0u;   // (0 is -0 too)
    const uint32_t raw = F32 ? __float_as_uint(value) : (__float_as_uint(value) >> 16) * 0x10001u;
    auto hits_of = [&](const uint4& u) {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      uint32_t misses = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) misses += F32 ? ((w[i] & zero) != raw) : min_u16x2((w[i] & zero) ^ raw, 0x10001u);
      return F32 ? 4u - misses : 8u - (misses & 0xFFFFu) - (misses >> 16);
    };
    uint32_t nth = sh.cmd.nth;
    int lo = slice.g0, hi = slice.g1;
    while (hi - lo > 32) {
      const int per = (hi - lo + S_WARPS - 1) / S_WARPS;
      const int w0 = min(lo + warp * per, hi), w1 = min(w0 + per, hi);
      uint32_t mine = 0;
      for (int g = w0 + lane; g < w1; g += 8 * 32) {
        uint4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = g + i * 32 < w1 ? slice.load(g + i * 32) : make_uint4(~0u, ~0u, ~0u, ~0u);   // (NaN)
#pragma unroll
        for (int i = 0; i < 8; ++i) mine += hits_of(u[i]);
      }
      mine = __reduce_add_sync(0xffffffffu, mine);
      __syncthreads();
      if (lane == 0) sh.scan_count[warp] = mine;
      __syncthreads();
      int w = 0;
      for (; w < S_WARPS - 1 && sh.scan_count[w] < nth; ++w) nth -= sh.scan_count[w];
      lo = min(lo + w * per, hi);
      hi = min(lo + per, hi);
    }
    if (warp == 0) {
      const uint4 u = lo + lane < hi ? slice.load(lo + lane) : make_uint4(~0u, ~0u, ~0u, ~0u);
      const uint32_t hits = hits_of(u);
      uint32_t sum = hits;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      uint32_t c = sum - hits;
      if (c < nth && nth <= sum) {
        int at = -1;
#pragma unroll
        for (int e = 0; e < K::GROUP; ++e)
          if ((Slice<F32>::bits(u, e) & (F32 ? zero : zero & 0xFFFFu)) == (F32 ? raw : raw & 0xFFFFu) && ++c == nth) at = e;
        a.ids[row] = (lo + lane) * K::GROUP - slice.shift + at;
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
