// The draw of a token from each row of logits: temperature, top-k, top-p, min-p, one given random number.
//
// The order. A row's tokens are ordered by falling logit, equal logits by index. Every filter keeps a first
// part of that order (the k first; the shortest part whose mass reaches p of that; the tokens of at least
// min_p times the first one's weight), so what is kept is a first part too, and all that remains of it is its
// mass W. The draw is the first token whose cumulated mass exceeds u * W. With weights
// w_j = exp((l_j - l_max) / T), each step asks for a position in cumulated counts or masses.
//
// No sort. Keys (the logits' bits, turned so that they order as unsigned numbers) are counted in a histogram
// whose bins follow the upper 16 bits: one bin for each bf16 value of magnitude 2^-10 to 2^7, and four wide ones
// for what is above, below, and on either side of zero. For bf16 logits a bin is one value, so its mass is its
// count times one weight, and a position inside it is a division. Where a bin holds several values (fp32 logits;
// the wide bins), its tokens are put in order if they are few (with all before them, so that later searches
// find their places there too), or counted again by finer parts of the key until they are few or one value. What
// is left of a position in a bin of one value is the nth token of that key in index order; the runs of the slice
// whose largest key is smaller are not read again for it.
//
// Exactness. The token has to be the one that the definition names, so masses are 64-bit integers: a weight is
// round(2^44 w), off by 2^-35 of itself (sample_math.h) and half a unit, sums of up to 2^19 of them are exact and
// do not depend on order, and u * W and p * W are compared exactly. A border between two tokens is then within
// 2^-34 + vocab * 2^-45 of its place (many light tokens below one heavy one are what the second term is for: 2^-27 for
// 248,320, where an fp32 sum is off by 2^-24 and more). The result is the same from call to call.
//
// Work. A cluster of 1 to 16 CTAs takes a row, each a slice of it; counts are joined through distributed
// shared memory, and the first warp of the cluster's first CTA searches and hands out commands. Every bf16 logit is read
// once for the counts, every fp32 one twice (masses need the row's maximum first); each list and finer count reads the
// slice again, and the token's search the runs that may hold it (fp32: all), from L2 where the logits fit.
// Times in a graph of calls on changing inputs (one card; others differ by up to 3%):
//   few rows: latency, 30 thousand clocks of dependent steps, a third of them waits at the four cluster barriers and a
//     quarter the searches (248,320 bf16 logits without a filter: 1 row 15.7 us, 64 rows 25.6; top-k 20 and top-p 0.8: 17.2
//     and 25.4)
//   many rows: atomics in shared memory, one for each logit, 3.3 to 4.8 clocks for a warp's (256 rows: 64 us, of which
//     the pass that counts takes 36 where an SM has two rows; HBM alone would take 18.7)
//   fp32: the instructions of the weights, 60% of the issue slots (24 rows of 151,937, top-p 0.95: 52 us; 128 of 248,320
//     without a filter: 198 us)
// Steps that carried it: bins of two logits at a time from clamped magnitudes; one warp searching by ballots in
// place of the CTA; one copy of each rare piece of code (instruction fetches bound the single pass); masses
// in two 32-bit words (a 64-bit atomic is a loop: 11 to 1700 clocks); two weights to an instruction.
#include <atomic>

#include "common.cuh"
#include "launch.h"
#include "sample_math.h"
#include "tc_util.cuh"

namespace nvfp4 {

namespace {

constexpr int S_THREADS = 512;
constexpr int S_WARPS = S_THREADS / 32;
constexpr int NB2 = S_THREADS;    // parts of a finer count
constexpr int LIST = S_THREADS;   // tokens that the first CTA puts in order at once

// What weights need beside a slope (in shared memory).
struct Weigher {
  unsigned long long table[64];
  float scale;
};

// (one copy of the code: a call runs most of its code once, and waits for instructions more than for data)
__device__ __noinline__ unsigned long long weight_copy(float ref, float x, float hi, float lo, const Weigher* by) {
  int n;
  const unsigned long long w = weight_and_scale(ref, x, Slope{hi, lo, by->scale}, by->table, n);
  return w | static_cast<unsigned long long>(n) << 48;   // (w <= 2^44)
}
NVFP4_DEV unsigned long long weight_call(float ref, float x, const Slope& c, const Weigher& by) {
  const unsigned long long v = weight_copy(ref, x, c.hi, c.lo, &by), w = v & ((1ull << 48) - 1);
  return rounded_weight(w, static_cast<int>(v >> 48));
}

// Operations on two floats at once.
struct TwoFloats {
  static NVFP4_DEV uint64_t pair(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
  }
  static NVFP4_DEV void split(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
  static NVFP4_DEV uint64_t all(float v) { return pair(v, v); }
  static NVFP4_DEV uint64_t add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
  }
  static NVFP4_DEV uint64_t mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
  }
  static NVFP4_DEV uint64_t fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
  }
};

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

// The same of masses in two words.
NVFP4_DEV unsigned long long mass_sum(uint32_t* lower, uint32_t* upper, int ctas) {
  unsigned long long sum = 0;
  for (int r0 = 0; r0 < ctas; r0 += 8) {
    uint32_t lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = r0 + i < ctas ? *in_cta(lower, r0 + i) : 0u;
      hi[i] = r0 + i < ctas ? *in_cta(upper, r0 + i) : 0u;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += static_cast<unsigned long long>(hi[i]) << 32 | lo[i];
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

enum { CMD_FIND = 0, CMD_END = 1, CMD_REFINE = 2, CMD_GATHER = 3 };

struct Command {
  int what;
  uint32_t lo, hi;       // REFINE: count keys lo .. hi by parts of 2^shift; GATHER: hand their tokens to the first CTA
  int shift;
  uint32_t key;          // FIND: the nth of CTA `owner`'s tokens with this key, from 1
  uint32_t nth;
  int owner;
};

enum { BY_COUNT = 0, BY_MASS = 1, BY_KEY = 2 };

struct Shared {
  uint4 edge[2];
  Weigher by;
  uint32_t wide[4][3];   // bf16: masses of the wide bins, of the row, in the first CTA: sums of 22 bits, 22 and the rest
  unsigned long long scan_mass[S_WARPS];
  uint32_t scan_count[S_WARPS];
  Command cmd;
  uint32_t max_key;                  // of this CTA's slice
  int min_bin;                       // bf16: its first bin that is not empty
  uint32_t zeros[2];                 // bf16: how many logits are 0, and -0
  uint32_t list_n, noted_n, base;
  uint32_t hits[4 * S_WARPS];
};

// Cumulated counts and masses through entry i.
struct Upto {
  unsigned long long mass[S_THREADS];
  uint32_t count[S_THREADS];
};

// Dynamic shared memory. `count`, `lower`, `upper`: of this CTA's slice (F32: masses in two words). `merged`: of the row,
// in the first CTA, with what is cumulated through each thread's bins.
struct Finer {
  union {
    Upto part;                          // of a finer count, cumulated
    unsigned long long mine[LIST];      // the slice's part of a list
  };
  uint32_t noted[LIST];                 // logits or keys that wait to be weighed
  uint32_t fine_lower[NB2], fine_upper[NB2];
  unsigned long long order[LIST];       // the list: key and index,
  unsigned long long order_mass[LIST];  // and masses through each entry
  uint32_t fine_count[NB2];
};
// Runs of 32 groups, in the order of the row: run r is of warp r % 16's turn r / 64.
constexpr int RUNS = (524288 / 8 + 1) / 32 + 2 * S_WARPS;
struct SliceMass {
  uint32_t lower[NB], upper[NB];
};
template <bool F32>
struct Room;
template <>
struct Room<false> : Finer {
  unsigned long long merged_mass[NB];
  Upto all;
  uint32_t count[NB], merged[NB];
  uint32_t lower[1], upper[1];   // (none)
  uint16_t most[RUNS / 4 + S_WARPS];   // the largest key (or more) of each warp's turns of four runs
  uint16_t runs[RUNS];           // (while the token is looked for) the runs that may hold it
};
template <>
struct Room<true> {
  union {   // the slices' masses have been joined before the first finer count
    SliceMass slice;
    Finer finer;
  };
  unsigned long long merged_mass[NB];
  Upto all;
  uint32_t count[NB], merged[NB];
};
NVFP4_DEV Finer& finer_of(Room<false>& r) { return r; }
NVFP4_DEV Finer& finer_of(Room<true>& r) { return r.finer; }
NVFP4_DEV uint16_t* most_of(Room<false>& r) { return r.most; }
NVFP4_DEV uint16_t* most_of(Room<true>&) { return nullptr; }
NVFP4_DEV uint16_t* runs_of(Room<false>& r) { return r.runs; }
NVFP4_DEV uint16_t* runs_of(Room<true>&) { return nullptr; }
NVFP4_DEV uint32_t* lower_of(Room<false>& r) { return r.lower; }
NVFP4_DEV uint32_t* lower_of(Room<true>& r) { return r.slice.lower; }
NVFP4_DEV uint32_t* upper_of(Room<false>& r) { return r.upper; }
NVFP4_DEV uint32_t* upper_of(Room<true>& r) { return r.slice.upper; }

// This CTA's part of a row: 16-byte groups g0 .. g1 - 1, group g holding logits g * GROUP - shift onwards
// (groups lie on 16-byte boundaries wherever the row starts; logits outside the row read as -inf). Ordinary loads: the
// grid ahead may still be writing the logits when this one starts, so they are not constant for the kernel's life.
template <bool F32>
struct Slice {
  using K = Key<F32>;
  static constexpr uint32_t NONE = F32 ? 0xFF800000u : 0xFF80FF80u;   // -inf
  const char* base;   // of group 0
  const uint4* edge;  // the first and the last group, where the row does not fill them (in shared memory)
  int shift, vocab, g0, g1;

  NVFP4_DEV bool whole(int g) const {
    const int first = g * K::GROUP - shift;
    return first >= 0 && first + K::GROUP <= vocab;
  }
  // A group that the row does not fill: logit by logit.
  NVFP4_DEV uint4 load_part(int g) const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = NONE;
#pragma unroll
    for (int e = 0; e < K::GROUP; ++e) {
      const int j = g * K::GROUP - shift + e;
      if (j < 0 || j >= vocab) continue;
      if (F32) {
        w[e] = reinterpret_cast<const uint32_t*>(base)[g * 4 + e];
      } else {
        const uint32_t h = reinterpret_cast<const unsigned short*>(base)[g * 8 + e];
        w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xFFFFu) | h << 16 : (w[e >> 1] & 0xFFFF0000u) | h;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  NVFP4_DEV uint4 load(int g) const { return whole(g) ? reinterpret_cast<const uint4*>(base)[g] : edge[g != 0]; }

  static NVFP4_DEV uint32_t bits(const uint4& u, int e) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    return F32 ? w[e] : (e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu;
  }

  // f(logit, its bits, index) for every logit of the slice. (Four loads at a time; the code for one group.)
  template <typename F>
  NVFP4_DEV void each(F f) const {
#pragma unroll 1
    for (int g = g0 + threadIdx.x; g < g1; g += 4 * S_THREADS) {
      uint4 u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = g + i * S_THREADS < g1 ? load(g + i * S_THREADS) : make_uint4(NONE, NONE, NONE, NONE);
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < K::GROUP; ++e) {
          const uint32_t b = bits(u[0], e);
          f(__uint_as_float(F32 ? b : b << 16), b, (g + i * S_THREADS) * K::GROUP - shift + e);
        }
        u[0] = u[1];
        u[1] = u[2];
        u[2] = u[3];
      }
    }
  }
  // f(key, index) for every logit with a key of lo .. hi.
  template <typename F>
  NVFP4_DEV void each_of(uint32_t lo, uint32_t hi, F f) const {
    const float least = value_of<F32>(lo), most = value_of<F32>(hi);
    each([&](float x, uint32_t b, int i) {
      if (!(x >= least && x <= most)) return;   // (also a NaN)
      const uint32_t k = key_of<F32>(b);
      if (k >= lo && k <= hi) f(k, i);          // (the highest key below 0 is that of no value, and compares as 0)
    });
  }
};

NVFP4_DEV uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
NVFP4_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
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

// Adds each thread's mass to the row's of a wide bin (whole warps; 256 of them at most, so that no part runs over, and no
// add waits for a carry from the first CTA: 1 row of 248,320 1% faster).
NVFP4_DEV void add_wide(Shared& sh, int wide, unsigned long long m) {
  if (!__any_sync(0xffffffffu, m != 0)) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
  if ((threadIdx.x & 31) == 0) {
    uint32_t* const to = in_cta(sh.wide[wide], 0);
    atomicAdd(to, static_cast<uint32_t>(m) & 0x3FFFFFu);
    atomicAdd(to + 1, static_cast<uint32_t>(m >> 22) & 0x3FFFFFu);
    atomicAdd(to + 2, static_cast<uint32_t>(m >> 44));
  }
}

// The sum over this and all earlier threads of the CTA (every thread calls it; ends behind a barrier).
NVFP4_DEV void scan_block(Shared& sh, uint32_t& c, unsigned long long& m) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t cu = __shfl_up_sync(0xffffffffu, c, o);
    const unsigned long long mu = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) c += cu, m += mu;
  }
  if (lane == 31) sh.scan_count[warp] = c, sh.scan_mass[warp] = m;
  __syncthreads();
  uint32_t cb = lane < warp ? sh.scan_count[lane] : 0u;
  unsigned long long mb = lane < warp ? sh.scan_mass[lane] : 0ull;
#pragma unroll
  for (int o = 1; o < S_WARPS; o <<= 1) {
    cb += __shfl_xor_sync(0xffffffffu, cb, o);
    mb += __shfl_xor_sync(0xffffffffu, mb, o);
  }
  c += __shfl_sync(0xffffffffu, cb, 0);
  m += __shfl_sync(0xffffffffu, mb, 0);
  __syncthreads();
}

// The first of 512 rising entries for which `reached` holds, 512 if none does (one warp).
template <typename F>
NVFP4_DEV int first_of(F reached) {
  const int lane = threadIdx.x & 31;
  const unsigned b = __ballot_sync(0xffffffffu, reached(lane * 16 + 15));
  if (b == 0) return S_THREADS;
  const int j = (__ffs(b) - 1) * 16;
  const unsigned c = __ballot_sync(0xffffffffu, lane < 16 && reached(j + (lane & 15)));
  return j + (c ? __ffs(c) - 1 : 15);
}

// The list's entry at this thread's place once its first n entries (one in each thread, the others ~0) are in rising order.
NVFP4_DEV unsigned long long sort_list(unsigned long long v, int n, unsigned long long* room) {
  const int t = threadIdx.x;
#pragma unroll 1
  for (int k = 2; k < 2 * n; k <<= 1) {
#pragma unroll 1
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
  extern __shared__ __align__(16) char smem[];
  __shared__ Shared sh;
  Room<F32>& room = *reinterpret_cast<Room<F32>*>(smem);
  Finer& fine_room = finer_of(room);
  uint32_t *const lower = lower_of(room), *const upper = upper_of(room);
  uint16_t* const room_most = most_of(room);
  constexpr int PER = (NB + S_THREADS - 1) / S_THREADS;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x) % ctas, row = static_cast<int>(blockIdx.x) / ctas;
  const bool first_cta = rank == 0;

  if (tid < 64) sh.by.table[tid] = EXP2_TABLE[tid];
  if (tid < 12) sh.wide[tid / 3][tid % 3] = 0;
  if (tid == 0) sh.max_key = 0, sh.min_bin = NB, sh.list_n = 0, sh.zeros[0] = sh.zeros[1] = 0;
  for (int b = tid; b < NB; b += S_THREADS) {
    room.count[b] = 0;
    if (F32) lower[b] = 0, upper[b] = 0;
  }
  pdl_wait();
  pdl_launch_dependents();

  const int entry = row / a.rows_each;
  const float temperature = a.set.temperature ? a.set.temperature[entry] : a.set.temperature_all;
  const bool searcher = first_cta && warp == 0;   // (its lanes hold the row's settings)
  float setting = 0.f;
  if (searcher && lane < 4) {
    const float* p = lane == 0   ? reinterpret_cast<const float*>(a.set.top_k)
                     : lane == 1 ? a.set.top_p
                     : lane == 2 ? a.set.min_p
                                 : a.uniform;
    setting = lane == 0 ? __int_as_float(a.set.top_k_all) : lane == 1 ? a.set.top_p_all : a.set.min_p_all;
    if (p) setting = p[lane == 3 ? row : entry];
  }

  Slice<F32> slice;
  {
    const char* p = static_cast<const char*>(a.logits) + static_cast<int64_t>(row) * a.stride * (F32 ? 4 : 2);
    slice.shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) / (F32 ? 4 : 2);
    slice.base = p - slice.shift * (F32 ? 4 : 2);
    slice.vocab = a.vocab;
    const int groups = (a.vocab + slice.shift + K::GROUP - 1) / K::GROUP, per = (groups + ctas - 1) / ctas;
    slice.g0 = min(rank * per, groups);
    slice.g1 = min(slice.g0 + per, groups);
    slice.edge = sh.edge;
    if (lane == 0 && warp < 2) {
      const int g = warp == 0 ? 0 : groups - 1;
      if (!slice.whole(g)) sh.edge[g != 0] = slice.load_part(g);
    }
  }
  __syncthreads();

  // Largest key of the row, and the first CTA that holds it (behind a cluster barrier).
  auto row_max_of = [&](int& holder) {
    float largest = __int_as_float(0xFF800000);
    slice.each([&](float x, uint32_t, int) { largest = fmaxf(largest, x); });   // (which passes over NaN)
    uint32_t most = key_of<F32>(F32 ? __float_as_uint(largest) : __float_as_uint(largest) >> 16);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&sh.max_key, most);
    cluster_sync_all();
    most = lane < ctas ? *in_cta(&sh.max_key, lane) : 0u;   // (each warp for itself)
    const uint32_t row = __reduce_max_sync(0xffffffffu, most);
    holder = __ffs(__ballot_sync(0xffffffffu, lane < ctas && most == row)) - 1;
    return row;
  };

  uint32_t row_max;
  bool irregular = false, mids = false;
  // (the temperature is looked at behind the pass over the logits: its load takes as long as theirs; a barrier behind it)
  bool greedy;
  Slope slope;
  auto look_at_temperature = [&]() {
    greedy = !(temperature > 0.f);
    slope = slope_of(greedy ? 1.f : temperature);
    if (tid == 0) sh.by.scale = slope.scale;
  };
  if (F32) {
    int holder;
    row_max = row_max_of(holder);
    look_at_temperature();
    if (tid == 0) sh.cmd = {CMD_FIND, 0u, 0u, 0, row_max, 1u, holder};
    __syncthreads();
  } else {
    // Counts. Two logits of a word at a time: clamped magnitudes give the bins. Logits of magnitudes below 2^-10
    // are noted: what lies in the middle bins is weighed afterwards, one by one.
    uint32_t* const middle = room.count + B_MID;
#pragma unroll 1
    for (int g = slice.g0 + tid, turn = 0; g - lane < slice.g1; g += 4 * S_THREADS, ++turn) {   // (a warp's turns together)
      uint4 u[4];
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (g + i * S_THREADS < slice.g1) u[i] = slice.load(g + i * S_THREADS);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (g + i * S_THREADS >= slice.g1) continue;
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        uint32_t m[4], sign[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          m[j] = max_u16x2(w[j] & 0x7FFF7FFFu, (MAG_LOW - 1) * 0x10001u);
          sign[j] = signs(w[j]);
          most = max_u16x2(most, w[j] ^ (sign[j] | 0x80008000u));   // (keys, but for -0, infinities and NaN)
        }
        const uint32_t least = min_u16x2(min_u16x2(m[0], m[1]), min_u16x2(m[2], m[3]));
        if (min_u16x2(least, MAG_LOW * 0x10001u) != MAG_LOW * 0x10001u) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t half = (e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu;
            if ((half & 0x7FFFu) >= MAG_LOW) continue;
            if ((half & 0x7FFFu) == 0) {   // a padded vocabulary has many
              atomicAdd(&sh.zeros[half >> 15], 1u);
              continue;
            }
            if (*static_cast<volatile uint32_t*>(&sh.list_n) > LIST) continue;
            const uint32_t at = atomicAdd(&sh.list_n, 1u);   // (more than LIST: no list, an irregular row)
            if (at < LIST) fine_room.noted[at] = half;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t s = bin_steps(min_u16x2(m[j], MAG_TOP * 0x10001u), sign[j]);
          atomicAdd(middle - static_cast<int16_t>(s & 0xFFFFu), 1u);
          atomicAdd(middle - (static_cast<int32_t>(s) >> 16), 1u);
        }
      }
      most = __reduce_max_sync(0xffffffffu, max(most & 0xFFFFu, most >> 16));
      if (lane == 0) room_most[turn * S_WARPS + warp] = static_cast<uint16_t>(most);
    }
    look_at_temperature();
    __syncthreads();
    if (sh.zeros[1] > 0) {   // -0 is 0
      if (tid == 0) {
        middle[1] -= sh.zeros[1];
        middle[0] += sh.zeros[1];
      }
      __syncthreads();
    }
    // the first bin that is not empty: the largest logit, where it is a bin of one value
    int bin = NB;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) {
      const int b = tid + i * S_THREADS;
      if (b < NB && room.count[b]) bin = b;
    }
    bin = __reduce_min_sync(0xffffffffu, bin);
    if (lane == 0 && bin < NB) atomicMin(&sh.min_bin, bin);
    cluster_sync_all();
    // (each warp for itself)
    const int my_bin = lane < ctas ? *in_cta(&sh.min_bin, lane) : NB;
    const uint32_t mid_any = lane < ctas ? *in_cta(room.count + B_MID, lane) | *in_cta(room.count + B_MID + 1, lane) : 0u;
    const bool many = __any_sync(0xffffffffu, lane < ctas && *in_cta(&sh.list_n, lane) > LIST);
    const uint32_t low_any = lane < ctas ? *in_cta(room.count + B_LAST, lane) : 0u;
    bin = __reduce_min_sync(0xffffffffu, my_bin);
    int holder = __ffs(__ballot_sync(0xffffffffu, my_bin == bin)) - 1;   // (greedy: the first CTA that has it)
    const bool lows = __any_sync(0xffffffffu, low_any != 0);
    mids = __any_sync(0xffffffffu, mid_any != 0) && bin < B_MID;
    uint32_t same;
    row_max = 0;
    irregular = bin == NB || wide_bin(bin) >= 0;
    if (!irregular) {
      bin_range(bin, row_max, same);
      const float best = value_of<false>(row_max);
      // (middle: their list has run over)
      irregular = !greedy && ((mids && many && weight_call(best, 0x1p-10f, slope, sh.by) > 0) ||
                              (lows && weight_call(best, -128.f, slope, sh.by) > 0));
    }
    if (irregular) {
      // Largest logits in a wide bin, weights that a wide bin's figures do not serve: these bins logit by logit.
      row_max = row_max_of(holder);
      if (tid < 4) room.count[tid == 0 ? 0 : tid == 3 ? B_LAST : B_MID + tid - 1] = 0;
      __syncthreads();
      const float best = value_of<false>(row_max);
      unsigned long long masses[4] = {0ull, 0ull, 0ull, 0ull};
      uint32_t last = 0;   // (runs of one value are common: a mask, a padded vocabulary)
      unsigned long long last_w = 0;
      slice.each([&](float, uint32_t bits, int) {
        const uint32_t k = key_of<false>(bits);
        const int b = bin_of(k), n = k ? wide_bin(b) : -1;
        if (n < 0) return;
        atomicAdd(room.count + b, 1u);
        if (k != last) last = k, last_w = weight_call(best, value_of<false>(k), slope, sh.by);
#pragma unroll
        for (int i = 0; i < 4; ++i) masses[i] += n == i ? last_w : 0ull;
      });
#pragma unroll
      for (int i = 0; i < 4; ++i) add_wide(sh, i, masses[i]);
      cluster_sync_all();
    }
    if (tid == 0) sh.cmd = {CMD_FIND, 0u, 0u, 0, row_max, 1u, holder};
    __syncthreads();
  }
  const float best = value_of<F32>(row_max);
  const bool drawn = row_max != 0 && !greedy;    // the same in every CTA of the cluster
  auto weigh = [&](uint32_t key) { return weight_call(best, value_of<F32>(key), slope, sh.by); };

  if (drawn) {
    if (F32) {
      // (the four weights of a group side by side, two to an instruction: their instructions bound this)
      const bool ordinary = slope.scale == 1.f && best < __int_as_float(0x7F800000);
      uint4 ahead = slice.g0 + tid < slice.g1 ? slice.load(slice.g0 + tid) : uint4{};
#pragma unroll 1
      for (int g = slice.g0 + tid; g < slice.g1; g += S_THREADS) {
        const uint4 u = ahead;
        if (g + S_THREADS < slice.g1) ahead = slice.load(g + S_THREADS);
        const uint32_t raw[4] = {u.x, u.y, u.z, u.w};
        unsigned long long w[4];
        if (ordinary) {
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const uint64_t minus = TwoFloats::pair(-__uint_as_float(raw[e]), -__uint_as_float(raw[e + 1]));
            const auto parts =
                weight_parts(TwoFloats::all(best), minus, TwoFloats::all(slope.hi), TwoFloats::all(slope.lo), TwoFloats());
            float y[2], t[2], l[2], tail[2];
            TwoFloats::split(parts.y, y[0], y[1]);
            TwoFloats::split(parts.t, t[0], t[1]);
            TwoFloats::split(parts.l, l[0], l[1]);
            TwoFloats::split(parts.tail, tail[0], tail[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              int n;
              const unsigned long long v = weight_of_parts(y[i], t[i], l[i], tail[i], sh.by.table, n);
              w[e + i] = rounded_weight(v, n);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = weight_call(best, __uint_as_float(raw[e]), slope, sh.by);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = __uint_as_float(raw[e]) + 0.f;   // (-0 is 0)
          if (!(x >= -3.402823466e+38f)) continue;
          // bin_of, from the magnitude
          const int m = static_cast<int>(__float_as_uint(x) >> 16 & 0x7FFFu);
          const int sign = static_cast<int>(__float_as_uint(x)) >> 31;
          constexpr int below = static_cast<int>(MAG_LOW) - 1;
          const int b = B_MID - ((min(max(m, below), static_cast<int>(MAG_TOP)) - below) ^ sign);
          atomicAdd(room.count + b, 1u);
          if (w[e]) add_mass(lower + b, upper + b, w[e]);   // (a mask's many equal logits weigh nothing)
        }
      }
      cluster_sync_all();
    }
    // each CTA joins its share of the bins
    const int per = (NB + ctas - 1) / ctas;
    for (int b = rank * per + tid; b < min((rank + 1) * per, NB); b += S_THREADS) {
      uint32_t c = cluster_sum(room.count + b, ctas);
      unsigned long long m = 0;
      if (c) {
        const int wide = wide_bin(b);
        if (F32) {
          m = mass_sum(lower + b, upper + b, ctas);
        } else if (wide < 0) {
          uint32_t h, same;
          bin_range(b, h, same);
          m = c * weight(best, value_of<false>(h), Slope{slope.hi, slope.lo, sh.by.scale}, sh.by.table);
        } else if (wide == 3 && !irregular) {
          c = 0;   // nothing in it weighs anything (and -inf and NaN were counted too)
        }
      }
      *in_cta(room.merged + b, 0) = c;
      *in_cta(room.merged_mass + b, 0) = m;
    }
    if (!F32 && mids && !irregular) {   // the middle bins' masses are those of their tokens, as lists and finer counts have them
      const int at = S_THREADS - 1 - tid;   // (the last warps had the fewest bins to join: 1 row of 248,320 2% faster)
      uint32_t half = 0;
      unsigned long long w = 0;
      if (at < min(sh.list_n, static_cast<uint32_t>(LIST))) {
        half = fine_room.noted[at];
        w = weigh(key_of<false>(half));
      }
      add_wide(sh, 2, half > 0x8000u ? w : 0ull);
      if (half > 0x8000u) w = 0;
      if (at == 0 && sh.zeros[0] + sh.zeros[1] > 0) w += (sh.zeros[0] + sh.zeros[1]) * weigh(key_of<false>(0u));
      add_wide(sh, 1, w);
    }
    cluster_sync_all();

    if (first_cta) {
      uint32_t c = 0;
      unsigned long long m = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        if (b < NB) {
          const int wide = F32 ? -1 : wide_bin(b);
          if (wide >= 0) room.merged_mass[b] = sh.wide[wide][0] + (static_cast<unsigned long long>(sh.wide[wide][1]) << 22) +
                                                (static_cast<unsigned long long>(sh.wide[wide][2]) << 44);
          c += room.merged[b];
          m += room.merged_mass[b];
        }
      }
      scan_block(sh, c, m);
      room.all.count[tid] = c;
      room.all.mass[tid] = m;
      __syncthreads();
    }

    // The first CTA's first warp searches; the others, and it, do what its commands say.
    int step = 0, phase = 0, how = BY_COUNT;
    unsigned long long target = 0, W = 0;
    uint32_t lo = 0, hi = 0, c0 = 0;                       // a range of keys, and what lies before it
    unsigned long long m0 = 0;
    const uint32_t* where = nullptr;                       // the slices' counts of the part that was found
    int list_n = 0;                                        // the list: tokens with keys list_lo .. list_hi, from
    uint32_t list_lo = 0, list_hi = 0, list_c0 = 0;        // count list_c0 and mass list_m0 on
    unsigned long long list_m0 = 0, list_mass = 0;
    if (searcher) W = room.all.mass[S_THREADS - 1];

    for (;;) {
      if (searcher) {
        Command next;
        for (;;) {
          // phase 0: a step begins (0: top-k, 1: top-p, 2: min-p, 3: the draw); 1: a finer count, 2: a list has come
          int index = -1;
          uint32_t key = 0, nth = 1;
          unsigned long long through = 0;
          bool done = false, listed = false;
          if (phase == 0) {
            bool off = false;
            if (step == 0) {
              const int k = __float_as_int(__shfl_sync(0xffffffffu, setting, 0));
              how = BY_COUNT;
              target = static_cast<unsigned long long>(k);
              off = k <= 0 || static_cast<uint32_t>(k) >= room.all.count[S_THREADS - 1];
            } else if (step == 2) {
              const float p = __shfl_sync(0xffffffffu, setting, 2);
              how = BY_KEY;
              off = !(p > 0.f);
              if (!off) {
                // the lowest key that weighs enough, 32 keys at a time
                bool cut = false;
                const unsigned long long least = p < 1.f ? max(times(ONE, p, cut) + cut, 1ull) : ONE;
                uint32_t good = row_max, bad = 0;   // good weighs enough, bad does not (or is no token)
                while (good - bad > 1) {
                  const uint32_t by = (good - bad + 31) / 32;
                  const uint32_t probe = static_cast<uint32_t>(lane + 1) * by < good - bad ? good - (lane + 1) * by : bad;
                  const bool ok = probe > bad && probe >= K::LOWEST && weigh(probe) >= least;
                  const int n = __ffs(~__ballot_sync(0xffffffffu, ok)) - 1;   // the first n probes; the last never is one
                  bad = __shfl_sync(0xffffffffu, probe, n);
                  good -= n * by;
                }
                target = good;
              }
            } else {
              const float v = __shfl_sync(0xffffffffu, setting, step);
              how = BY_MASS;
              bool cut = false;
              target = v > 0.f ? v < 1.f ? times(W, v, cut) : W - 1 : 0ull;
              if (step == 1) {   // at least v of the mass, and one token
                off = !(v < 1.f);
                target = max(target + cut, 1ull);
              } else {           // more than v of it
                target += 1;
              }
            }
            if (off) {
              ++step;
              continue;
            }
            listed = list_n > 0 && (how == BY_KEY     ? target >= list_lo && target <= list_hi
                                    : how == BY_COUNT ? target > list_c0 && target - list_c0 <= static_cast<unsigned>(list_n)
                                                      : target > list_m0 && target - list_m0 <= list_mass);
          }
          if (phase == 2) {
            list_n = min(sh.list_n, static_cast<uint32_t>(LIST));
            list_mass = fine_room.order_mass[LIST - 1];
            listed = true;
            if (how == BY_MASS) target = min(target, list_m0 + list_mass);
          }
          if (listed) {
            int i = how == BY_COUNT  ? static_cast<int>(target - list_c0) - 1
                    : how == BY_MASS ? first_of([&](int t) { return list_m0 + fine_room.order_mass[t] >= target; })
                                     : first_of([&](int t) {
                                         return t >= list_n || (~static_cast<uint32_t>(fine_room.order[t] >> 32) & K::ALL) < target;
                                       }) - 1;
            i = min(i, list_n - 1);   // (tokens that are gone: logits changed during the call)
            through = list_m0 + (i >= 0 ? fine_room.order_mass[i] : 0ull);
            key = i >= 0 ? ~static_cast<uint32_t>(fine_room.order[i] >> 32) & K::ALL : row_max;
            index = i >= 0 ? static_cast<int>(static_cast<uint32_t>(fine_room.order[i])) : 0;
            done = true;
          } else {
            // the bin or part that holds the position
            const bool fine = phase == 1;
            const Upto& upto = fine ? fine_room.part : room.all;
            const int n = fine ? 1 : PER;
            uint32_t cb = fine ? c0 : 0u;                        // what lies before the thread's bins that hold it
            unsigned long long mb = fine ? m0 : 0ull;
            const uint32_t part_of_target = fine ? (hi - static_cast<uint32_t>(target)) >> sh.cmd.shift
                                                 : static_cast<uint32_t>(bin_of(static_cast<uint32_t>(target) >> K::LOW));
            const unsigned long long aim = how == BY_COUNT  ? target - cb
                                           : how == BY_MASS ? min(target - mb, upto.mass[S_THREADS - 1])
                                                            : 0ull;
            int t = how == BY_KEY     ? static_cast<int>(part_of_target) / n
                    : how == BY_COUNT ? first_of([&](int i) { return upto.count[i] >= aim; })
                                      : first_of([&](int i) { return upto.mass[i] >= aim && upto.mass[i] > 0; });
            t = min(t, S_THREADS - 1);
            const uint32_t c_at = t ? upto.count[t - 1] : 0u;
            const unsigned long long m_at = t ? upto.mass[t - 1] : 0ull;
            cb += c_at;
            mb += m_at;
            // its bins, one in a lane
            const int b = t * n + lane;
            uint32_t c = 0;
            unsigned long long m = 0;
            if (lane < n && (fine || b < NB)) {
              c = fine ? upto.count[t] - c_at : room.merged[b];
              m = fine ? upto.mass[t] - m_at : room.merged_mass[b];
            }
            uint32_t cs = c;
            unsigned long long ms = m;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) {
              const uint32_t cu = __shfl_up_sync(0xffffffffu, cs, o);
              const unsigned long long mu = __shfl_up_sync(0xffffffffu, ms, o);
              if (lane >= o) cs += cu, ms += mu;
            }
            const bool here = lane < n && (how == BY_KEY     ? b == static_cast<int>(part_of_target)
                                           : how == BY_COUNT ? c_at + cs >= aim
                                                             : m_at + ms >= aim && ms > 0);
            const unsigned all_here = __ballot_sync(0xffffffffu, here);
            const int at = all_here ? __ffs(all_here) - 1 : 0;
            c0 = cb + __shfl_sync(0xffffffffu, cs - c, at);
            m0 = mb + __shfl_sync(0xffffffffu, ms - m, at);
            c = __shfl_sync(0xffffffffu, c, at);
            m = __shfl_sync(0xffffffffu, m, at);
            const int bin = t * n + at;
            bool single;
            if (fine) {
              const int shift = sh.cmd.shift;
              hi -= static_cast<uint32_t>(bin) << shift;
              const uint32_t bottom = hi - ((1u << shift) - 1u);
              lo = bottom > lo && bottom <= hi ? bottom : lo;
              single = shift == 0;
              where = fine_room.fine_count + bin;
            } else {
              bin_range(bin, lo, hi);
              lo <<= K::LOW;
              hi = (hi << K::LOW) | ((1u << K::LOW) - 1u);
              if (bin == 0) hi = K::PINF;
              single = !F32 && wide_bin(bin) < 0;
              where = room.count + bin;
            }
            if (single || c == 0 || hi < lo) {
              key = hi;
              const unsigned long long w = c == 1 ? m : weigh(key);   // (a call and a division less for most drawn tokens)
              if (c > 1) {
                nth = how == BY_KEY     ? c
                      : how == BY_COUNT ? static_cast<uint32_t>(target) - c0
                                        : few_times(target - m0, w);
                nth = max(1u, min(nth, c));
              }
              through = m0 + min(nth, c) * w;
              done = true;
            } else if (c <= LIST) {
              // few tokens: in order, with all before them where these are few as well
              if (c0 + c <= LIST) hi = K::PINF, c0 = 0, m0 = 0;
              list_lo = lo;
              list_hi = hi;
              list_c0 = c0;
              list_m0 = m0;
              next = {CMD_GATHER, lo, hi, 0, 0u, 0u, 0};
              phase = 2;
            } else {
              int shift = 0;
              while (((hi - lo) >> shift) >= static_cast<uint32_t>(NB2)) ++shift;
              next = {CMD_REFINE, lo, hi, shift, 0u, 0u, 0};
              phase = 1;
            }
          }
          if (!done) break;
          phase = 0;
          if (step < 3) {
            W = step == 2 ? min(W, through) : through;
            ++step;
            continue;
          }
          // (a light token's probability has more bits than its rounded weight)
          const unsigned long long v = weight_copy(best, value_of<F32>(key), slope.hi, slope.lo, &sh.by);
          const float w = __ull2float_rn(v & ((1ull << 48) - 1)) * __uint_as_float((127u - static_cast<uint32_t>(v >> 48)) << 23);
          if (lane == 0 && a.probs) a.probs[row] = w / __ull2float_rn(W);
          next = {CMD_END, 0u, 0u, 0, 0u, 0u, 0};
          if (index >= 0) {
            if (lane == 0) a.ids[row] = index;
          } else {
            // the CTA that holds the nth token of this key
            const uint32_t mine = lane < ctas ? *in_cta(where, lane) : 0u;
            uint32_t sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
              if (lane >= o) sum += v;
            }
            const unsigned has = __ballot_sync(0xffffffffu, lane < ctas && sum >= nth);
            const int owner = has ? __ffs(has) - 1 : 0;
            next = {CMD_FIND, 0u, 0u, 0, key, nth - __shfl_sync(0xffffffffu, sum - mine, owner), owner};
          }
          break;
        }
        if (lane == 0 && next.what == CMD_GATHER) sh.list_n = 0;
        __syncwarp();
        if (lane < ctas) *in_cta(&sh.cmd, lane) = next;
        __syncwarp();
      }
      cluster_sync_all();
      const Command c = sh.cmd;
      if (c.what == CMD_FIND || c.what == CMD_END) break;
      if (c.what == CMD_GATHER) {
        // the tokens with keys lo .. hi into the first CTA's list
        if (tid == 0) sh.noted_n = 0;
        __syncthreads();
        slice.each_of(c.lo, c.hi, [&](uint32_t k, int i) {
          const uint32_t at = atomicAdd(&sh.noted_n, 1u);
          if (at < LIST) fine_room.mine[at] = static_cast<unsigned long long>(~k) << 32 | static_cast<uint32_t>(i);
        });
        __syncthreads();
        const int n_mine = min(sh.noted_n, static_cast<uint32_t>(LIST));
        if (tid == 0 && n_mine > 0) sh.base = atomicAdd(in_cta(&sh.list_n, 0), static_cast<uint32_t>(n_mine));
        __syncthreads();
        if (tid < n_mine && sh.base + tid < LIST) *in_cta(fine_room.order + sh.base + tid, 0) = fine_room.mine[tid];
        cluster_sync_all();
        if (first_cta) {
          const int n = min(sh.list_n, static_cast<uint32_t>(LIST));
          const unsigned long long v = sort_list(tid < n ? fine_room.order[tid] : ~0ull, n, fine_room.order_mass);
          unsigned long long m = tid < n ? weigh(~static_cast<uint32_t>(v >> 32) & K::ALL) : 0ull;
          uint32_t none = 0;
          scan_block(sh, none, m);
          fine_room.order[tid] = v;
          fine_room.order_mass[tid] = m;
          __syncthreads();
        }
      } else {
        // counts (and masses) of the keys lo .. hi by parts of 2^shift, cumulated in the first CTA
        fine_room.fine_count[tid] = 0;
        fine_room.fine_lower[tid] = fine_room.fine_upper[tid] = 0;
        if (tid == 0) sh.noted_n = 0;
        __syncthreads();
        slice.each_of(c.lo, c.hi, [&](uint32_t k, int) {
          const uint32_t b = (c.hi - k) >> c.shift;
          atomicAdd(fine_room.fine_count + b, 1u);
          if (c.shift == 0) return;   // (one key: its count and weight are its mass)
          const uint32_t at = atomicAdd(&sh.noted_n, 1u);
          if (at < LIST) fine_room.noted[at] = k;
          else if (const unsigned long long w = weigh(k)) add_mass(fine_room.fine_lower + b, fine_room.fine_upper + b, w);
        });
        __syncthreads();
        if (tid < min(sh.noted_n, static_cast<uint32_t>(LIST))) {
          const uint32_t k = fine_room.noted[tid], b = (c.hi - k) >> c.shift;
          if (const unsigned long long w = weigh(k)) add_mass(fine_room.fine_lower + b, fine_room.fine_upper + b, w);
        }
        cluster_sync_all();
        const int each = NB2 / ctas, b = rank * each + tid;
        if (tid < each) {
          const uint32_t n = cluster_sum(fine_room.fine_count + b, ctas);
          *in_cta(fine_room.part.count + b, 0) = n;
          *in_cta(fine_room.part.mass + b, 0) = n == 0    ? 0ull
                                                : c.shift ? mass_sum(fine_room.fine_lower + b, fine_room.fine_upper + b, ctas)
                                                          : n * weigh(c.hi - b);
        }
        cluster_sync_all();
        if (first_cta) {
          uint32_t n = fine_room.part.count[tid];
          unsigned long long m = fine_room.part.mass[tid];
          scan_block(sh, n, m);
          fine_room.part.count[tid] = n;
          fine_room.part.mass[tid] = m;
          __syncthreads();
        }
      }
    }
  } else if (first_cta && tid == 0) {
    if (a.probs) a.probs[row] = row_max ? 1.f : 0.f;
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
    // the runs of 32 groups that may hold it, in order (all of them where their largest keys were not kept)
    const int all_runs = (slice.g1 - slice.g0 + 31) / 32;
    uint16_t* const runs = runs_of(room);
    int n_runs = all_runs;
    if (!F32) {
      n_runs = 0;
      for (int r0 = 0; r0 < all_runs; r0 += S_THREADS) {
        const int r = r0 + tid, turn = r / (4 * S_WARPS) * S_WARPS + r % S_WARPS;
        const bool may = r < all_runs && room_most[turn] >= (value == 0.f ? 0x7FFFu : sh.cmd.key);   // (-0 is one key lower)
        const unsigned any = __ballot_sync(0xffffffffu, may);
        if (lane == 0) sh.scan_count[warp] = __popc(any);
        __syncthreads();
        uint32_t before = lane < S_WARPS ? sh.scan_count[lane] : 0u, sum = before;
#pragma unroll
        for (int o = 1; o < S_WARPS; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += v;
        }
        before = __shfl_sync(0xffffffffu, sum - before, warp);
        if (may) runs[n_runs + before + __popc(any & ((1u << lane) - 1u))] = static_cast<uint16_t>(r0 + tid);
        n_runs += __shfl_sync(0xffffffffu, sum, S_WARPS - 1);
        __syncthreads();
      }
    }
    // group g of the runs, as far as the slice goes
    const bool direct = n_runs == all_runs;
    auto group_at = [&](int g) { return slice.g0 + (direct ? g : runs[g >> 5] * 32 + (g & 31)); };
    auto load_at = [&](int g, int end) {
      const int at = g < end ? group_at(g) : slice.g1;
      return at < slice.g1 ? slice.load(at) : make_uint4(~0u, ~0u, ~0u, ~0u);   // (NaN)
    };
    uint32_t nth = sh.cmd.nth;
    int lo = 0, hi = n_runs * 32;
#pragma unroll 1
    while (hi - lo > 4 * S_THREADS) {
      const int per = (hi - lo + S_WARPS - 1) / S_WARPS;
      const int w0 = min(lo + warp * per, hi), w1 = min(w0 + per, hi);
      uint32_t mine = 0;
#pragma unroll 1
      for (int g = w0 + lane; g < w1; g += 8 * 32) {
        uint4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = load_at(g + i * 32, w1);
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
    // four groups a thread: the i-th of all threads, warp by warp, before the next
    uint4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = load_at(lo + i * S_THREADS + tid, hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t n = __reduce_add_sync(0xffffffffu, hits_of(u[i]));
      if (lane == 0) sh.hits[i * S_WARPS + warp] = n;
    }
    __syncthreads();
    const uint32_t first = sh.hits[2 * lane], second = sh.hits[2 * lane + 1];
    uint32_t sum = first + second;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned reached = __ballot_sync(0xffffffffu, sum >= nth);
    if (reached) {
      const int at = __ffs(reached) - 1;
      uint32_t before = __shfl_sync(0xffffffffu, sum - first - second, at);
      const uint32_t half = __shfl_sync(0xffffffffu, first, at);
      const bool later = before + half < nth;
      if (later) before += half;
      const int run = 2 * at + (later ? 1 : 0), i = run / S_WARPS;
      if (run % S_WARPS == warp) {
        const uint4 v = i == 0 ? u[0] : i == 1 ? u[1] : i == 2 ? u[2] : u[3];
        const uint32_t n = hits_of(v);
        uint32_t upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
        uint32_t c = before + upto - n;
        if (c < nth && nth <= c + n) {
          constexpr uint32_t one = F32 ? 0xFFFFFFFFu : 0xFFFFu;
          int e_at = 0;
#pragma unroll
          for (int e = 0; e < K::GROUP; ++e)
            if ((Slice<F32>::bits(v, e) & zero & one) == (raw & one) && ++c == nth) e_at = e;
          a.ids[row] = group_at(lo + i * S_THREADS + tid) * K::GROUP - slice.shift + e_at;
        }
      }
    }
  }
  cluster_sync_all();   // no CTA leaves while another may read its shared memory
}

// Accepted drafts: the leading ones that are the token drawn at their position (-1, in a row without a token, is none).
__global__ void accept_kernel(const int32_t* tokens, const int32_t* drafts, int64_t batch, int n_draft, int32_t* accepted) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t b = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (b >= batch) return;
  int n = 0;
  for (; n < n_draft; ++n) {
    const int32_t token = tokens[b * (n_draft + 1) + n];
    if (token < 0 || token != drafts[b * n_draft + n]) break;
  }
  accepted[b] = n;
}

// Whether clusters of 16 CTAs of a kernel find a place: they have to be allowed, and the device has to have the SMs
// together. Asked once on each device.
bool wide_clusters(const void* kernel, int smem, int which) {
  static std::atomic<unsigned long long> asked[2], found[2];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
  const unsigned long long bit = 1ull << dev;
  if (!(asked[which].load() & bit)) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 16;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(S_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
    if (ok) found[which].fetch_or(bit);
    else cudaGetLastError();   // (an answer, not an error of the call)
    asked[which].fetch_or(bit);
  }
  return found[which].load() & bit;
}

template <bool F32>
int launch_sample_type(const SampleArgs& a, int64_t rows, cudaStream_t stream) {
  const auto kernel = sample_kernel<F32>;
  constexpr int smem = static_cast<int>(sizeof(Room<F32>));
  if (int rc = ensure_smem(kernel, smem)) return rc;
  // as many CTAs for a row as the rows leave room for, none with less than 4096 logits
  int ctas = 1;
  while (ctas < 16 && rows * ctas <= sm_count() && a.vocab > 4096 * ctas) ctas *= 2;
  if (ctas > 8 && !wide_clusters(reinterpret_cast<const void*>(kernel), smem, F32)) ctas = 8;
  return launch_ex(kernel, dim3(static_cast<unsigned>(rows * ctas)), dim3(S_THREADS), smem, ctas, true, stream, a, ctas);
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
