// Attention of many new rows over a paged key-value cache on the
// 5th-generation tensor cores: prompts and chunks of prompts, causal, with an
// optional sliding window and sinks.
//
// The mathematics is attention_rows.cuh's: per row a running maximum m, l =
// sum 2^(x - m) and o = sum 2^(x - m) v over the tiles that the row sees, with
// x the score in powers of two. The rows of one kv head share its keys and
// values, so a 128-row tile packs (token, query head) pairs: 128 / G tokens of
// all G heads. The running maximum that o is kept relative to moves only when
// it would grow by more than 2^8 (E4M3 caches: 2^4.9; p stays below 2^16), so o is
// rescaled in tensor memory a few times per row, not per tile.
//
// What bounds it: 4 * 128 * 128 * D flops per (row tile, 128 positions); K and
// V come from L2 mostly. Per SM 1024 tensor clocks a tile at D = 128, against
// 16384 exponentials. So two row tiles (A, B) share every K and V tile and
// take turns: while one warpgroup turns S_A into P_A the tensor cores do
// O_B += P_B V and the next S_B = Q_B K^T.
//   warps 0..3, 4..7  softmax of row tile A, B: a thread owns a row (a
//                     tensor-memory lane), reads S, writes P over it (bf16
//                     pairs), and at the end reads O, divides and writes out
//   warp 8            producer: hands out work items, loads Q, K and V (a box
//                     per page and 64 d's) by TMA
//   warp 9            tensor-memory allocation; issues the MMAs
//   warps 10, 11      (bf16 caches) zero value rows that no row of the item sees
//                     (they may hold anything, and 0 * NaN is not 0), and take
//                     elements that are not finite out of rows that only some
//                     rows see (kv.cuh); the softmax warps add them at the end
//   warps 10..15      (E4M3 caches) 10 loads V, 11 takes such elements out, 12, 13
//                     turn K's codes and 14, 15 V's, copied in chunks of 32
//                     rows, into f16 tiles; the MMAs are f16 then, and the
//                     softmax warps bring each item's Q to f16
// S and P of a tile share 128 columns: S(j + 1) is issued after O += P(j) V(j),
// and the tensor cores run one thread's MMAs in order. For the same reason a
// finished S(j + 1) says that O += P(j) V(j) is finished, so the softmax warps
// may rescale O before they publish P(j + 1).
//
// Roundings. bf16 caches: q, k, v as they are, products exact, sums fp32; p is
// rounded to one bf16 (2^-8) for the second product, as the tensor cores take it:
// about as much error as the output's own rounding. Two halves, as the token
// kernel takes, would be half as much tensor time again. E4M3 caches: k and v are
// exact in f16, q is scaled by a power of two into f16, p is one f16 (2^-11) in
// f16's upper range (kv.cuh).
//
// Few items (a short chunk on a long context) are split over the positions:
// each part leaves (m, l, o) in the workspace and the last part of a row tile
// to arrive joins them in order.
//
// Measured, bf16, D = 128: 1500 and 2048 new tokens of two sequences, 32 heads on
// 8, on up to 14k positions, 594-607 us (75% of the bf16 burst rate that a large
// matrix product reaches; under the power cap); an 8k prompt, 40 heads on 8, with
// a window of 1024, 176-197 us (84 us of MMAs, 111 in whole tiles); 2,048 new
// tokens on 6,144, 186 us, over E4M3 259 us (124 of MMAs; every item converts the
// codes again; 4 bytes of registers spill). Two row tiles rather than
// one: a tile's exponentials hide behind the other's MMAs. A warpgroup of its own
// for the output was slower (2k on 8k: 188 -> 211 us).
//
// Every wait is bounded; one that gives up raises the CTA's abort flag, every
// role leaves its loop, and nothing more is written.
#pragma once

#include "kv.cuh"
#include "tcgen05.cuh"

namespace nvfp4 {
namespace {

constexpr int AT_ROWS = 128;                 // rows of a row tile
constexpr int AT_TILE = 128;                 // positions of a key tile
constexpr int AT_SLOTS = 4;                  // ring slots of K and V tiles
constexpr int AT_CHUNK = 32;                 // rows of a chunk of 8-bit codes
constexpr int AT_CHUNKS = 4;                 // chunks of K, and of V, in flight: a tile's
constexpr int AT_ITEMS = 2;                  // items announced ahead
constexpr int AT_OKS = 8;                    // announced page masks of tiles
// Tokens of an item whose values had elements taken out: bit n for position p0 +
// 1 + n, bit 256 + n for the n-th position of the first row's window (at most
// 255 of either are seen by some rows of an item and not by others). A role can
// be two items ahead of the softmax warps, so four items' bits are kept; each
// checking warp has its own.
constexpr int AT_CUTS = 4, AT_CUT_WORDS = 16;
constexpr int AT_SOFTMAX_WARPS = 8;
constexpr int AT_PROD_WARP = 8, AT_MMA_WARP = 9, AT_CLEAN_WARP = 10;   // 10, 11: half a tile each
constexpr int AT_V_PROD_WARP = 10, AT_CHECK_WARP = 11;   // (E4M3 caches)
constexpr int AT_CONVERT_WARP = 12;          // 12, 13: K's codes, 14, 15: V's (E4M3 caches)
// slot full / empty / clean, item full / empty, q full / empty, s full, p full,
// o full, join, q ready (each for A and B), chunk full / empty (K's, V's), chunk
// checked (V's), drain
constexpr int AT_BARS = 3 * AT_SLOTS + 2 * AT_ITEMS + 2 + 10 + 5 * AT_CHUNKS + 1;

struct AtItem {
  int done;
  int h;                 // kv head
  int b;                 // sequence
  int row0, n_tok;       // first new-token row, tokens
  int p0;                // first position
  int key_end;           // positions at or past it hold nothing
  int st, w0, i0, i1;    // tiles (KvTiles) and the part of them that is this item's
  int item, part, parts; // index of the unsplit item, part of it, its parts
};

struct AtParams {
  KvSeqs s;
  uint16_t* out;
  int64_t pages;
  int heads, group;
  int page_size, page_log2;
  int window, sinks;
  float scale;           // softmax scale * log2 e, > 0
  int parts;             // parts of an item (1: no split)
  int64_t units;         // work items that the launch and the workspace were sized for
  const void* v;         // the value pool
  const float* k_scale;  // E4M3 only
  const float* v_scale;
  unsigned* arrived;     // [items][2], zero between calls (split only)
  float* part;           // [items][parts][2] of o [D / 4][128] float4 (a warp's rows next to each other), (m, l) [128]
  int* status;
};

template <bool E4M3, int D>
struct AtShape {
  static constexpr int HALVES = D / 64;
  static constexpr int MAT_BYTES = AT_TILE * D * 2;       // Q row tile, K tile or V tile
  static constexpr int K_SLOTS = 2, V_SLOTS = 2;          // rings: K's slots, then V's
  static constexpr int CHUNK_BYTES = E4M3 ? AT_CHUNK * D : 0;
  // beside the tiles: E4M3 chunks of K and V, or each softmax warp's staging of
  // 32 output rows x 64 d's
  static constexpr int STAGING = E4M3 ? 0 : AT_SOFTMAX_WARPS * 32 * 128;
  static constexpr int DATA = (2 + K_SLOTS + V_SLOTS) * MAT_BYTES + 2 * AT_CHUNKS * CHUNK_BYTES + STAGING;
  static constexpr int SMEM = DATA + AT_ITEMS * static_cast<int>(sizeof(AtItem)) + AT_OKS * 4 + AT_BARS * 8 +
                              AT_CUTS * 2 * (AT_CUT_WORDS + 1) * 4 + 64 + 1024;
  static constexpr int O_COL0 = 256;                       // tensor memory: S_A, S_B, O_A, O_B
  // Registers a thread, moved from the other warpgroups to the two softmax
  // ones: 384 x 168 = 64512 at launch, 256 x 208 + 128 x 80 = 63488 after; with
  // converters 512 x 128 = 65536, 256 x 192 + 256 x 64 = 65536.
  static constexpr int THREADS = E4M3 ? 16 * 32 : 12 * 32;
  static constexpr int REGS_SOFTMAX = E4M3 ? 192 : 208, REGS_OTHER = E4M3 ? 64 : 80;
  static_assert(256 * REGS_SOFTMAX + (THREADS - 256) * REGS_OTHER <= THREADS * (E4M3 ? 128 : 168), "register split");
};
static_assert(AtShape<false, 128>::SMEM <= 227 * 1024 && AtShape<true, 128>::SMEM <= 227 * 1024, "shared memory");

// 1 in one lane of the (converged) warp, 0 in the others.
NVFP4_DEV uint32_t elect_one() {
  uint32_t x;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
  return x;
}

// D (+)= A * B, both from shared memory, by the lane whose `lead` is set.
NVFP4_DEV void tc_mma_bf16_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// The same with A from tensor memory.
NVFP4_DEV void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
NVFP4_DEV void tc_st_32cols(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

NVFP4_DEV void fma2(float& a, float& b, float c, float d) {   // (a, b) = (a, b) * c + d
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}
NVFP4_DEV void add2(float& a, float& b, float c, float d) {   // (a, b) += (c, d)
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}

NVFP4_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

NVFP4_DEV void sts128(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// A word with its lowest n bits set (none for n <= 0).
NVFP4_DEV uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// Whether the tile at position j0 has positions that no row of p0..p1 sees.
NVFP4_DEV bool at_unclean(int j0, int p0, int p1, int window, int sinks) {
  if (j0 + AT_TILE - 1 > p1) return true;
  return window > 0 && p0 - window >= max(j0, sinks) && sinks < j0 + AT_TILE;
}

template <bool E4M3, int D>
__global__ void __launch_bounds__(AtShape<E4M3, D>::THREADS, 1)
    attention_tiles_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v, const AtParams p) {
  using S = AtShape<E4M3, D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* at = smem_raw + (base - raw) + S::DATA;
  uint64_t* bars = reinterpret_cast<uint64_t*>(at);
  AtItem* items = reinterpret_cast<AtItem*>(bars + AT_BARS);
  unsigned* oks = reinterpret_cast<unsigned*>(items + AT_ITEMS);
  uint32_t* tmem_slot = oks + AT_OKS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  unsigned* last_flag = tmem_slot + 2;   // [2]
  volatile unsigned* cut_any = tmem_slot + 4;               // [AT_CUTS][2]: 1 where a bit is set in
  unsigned* cuts = tmem_slot + 4 + 2 * AT_CUTS;             // [AT_CUTS][2][AT_CUT_WORDS]
  const uint32_t bar0 = smem_addr(bars);
  auto kv_full = [&](int s) { return bar0 + 8u * s; };
  auto kv_empty = [&](int s) { return bar0 + 8u * (AT_SLOTS + s); };
  auto kv_clean = [&](int s) { return bar0 + 8u * (2 * AT_SLOTS + s); };
  auto item_full = [&](int s) { return bar0 + 8u * (3 * AT_SLOTS + s); };
  auto item_empty = [&](int s) { return bar0 + 8u * (3 * AT_SLOTS + AT_ITEMS + s); };
  constexpr int B1 = 3 * AT_SLOTS + 2 * AT_ITEMS;
  const uint32_t q_full = bar0 + 8u * B1, q_empty = bar0 + 8u * (B1 + 1);
  auto s_full = [&](int x) { return bar0 + 8u * (B1 + 2 + x); };
  auto p_full = [&](int x) { return bar0 + 8u * (B1 + 4 + x); };
  auto o_full = [&](int x) { return bar0 + 8u * (B1 + 6 + x); };
  auto join_bar = [&](int x) { return bar0 + 8u * (B1 + 8 + x); };
  auto q_ready = [&](int x) { return bar0 + 8u * (B1 + 10 + x); };
  auto chunk_full = [&](int kv, int s) { return bar0 + 8u * (B1 + 12 + 2 * AT_CHUNKS * kv + s); };
  auto chunk_empty = [&](int kv, int s) { return bar0 + 8u * (B1 + 12 + 2 * AT_CHUNKS * kv + AT_CHUNKS + s); };
  auto chunk_ok = [&](int s) { return bar0 + 8u * (B1 + 12 + 4 * AT_CHUNKS + s); };
  const uint32_t drain_bar = bar0 + 8u * (B1 + 12 + 5 * AT_CHUNKS);
  auto q_tile = [&](int x) { return base + x * S::MAT_BYTES; };
  auto slot = [&](int s) { return base + (2 + s) * S::MAT_BYTES; };
  auto chunk = [&](int kv, int s) { return base + (2 + S::K_SLOTS + S::V_SLOTS) * S::MAT_BYTES + (kv * AT_CHUNKS + s) * S::CHUNK_BYTES; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < AT_SLOTS; ++s) {
      mbar_init(kv_full(s), E4M3 ? 2 : 1);
      mbar_init(kv_empty(s), 1);
      mbar_init(kv_clean(s), 2);
    }
    for (int s = 0; s < AT_ITEMS; ++s) {
      mbar_init(item_full(s), 1);
      mbar_init(item_empty(s), AT_SOFTMAX_WARPS + (E4M3 ? 6 : 3));
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full(x), 1);
      mbar_init(p_full(x), AT_SOFTMAX_WARPS / 2);
      mbar_init(o_full(x), 1);
      mbar_init(join_bar(x), AT_SOFTMAX_WARPS / 2);
      mbar_init(q_ready(x), AT_SOFTMAX_WARPS / 2);
      for (int s = 0; s < AT_CHUNKS; ++s) {
        mbar_init(chunk_full(x, s), 1);
        mbar_init(chunk_empty(x, s), 1);
        if (x == 0) mbar_init(chunk_ok(s), 1);
      }
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    for (int n = 0; n < 2 * AT_CUTS; ++n) cut_any[n] = 0;
    for (int n = 0; n < 2 * AT_CUTS * AT_CUT_WORDS; ++n) cuts[n] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_q) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v) : "memory");
  }
  if (warp == AT_MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_launch_dependents();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const int tile_tok = AT_ROWS / p.group;      // tokens of a row tile
  const int item_tok = 2 * tile_tok;
  constexpr int BOX = E4M3 ? AT_CHUNK : AT_TILE;   // most rows of a copied box
  const int box = p.page_size < BOX ? p.page_size : BOX;
  const int boxes = AT_TILE / box;

  // waits of a whole warp
  auto wait = [&](uint32_t bar, int parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, static_cast<uint32_t>(parity), abort_flag, p.status)) != 0;
  };
  // the k-th announced item, for the roles that read it; false: no more
  auto get_item = [&](int k, AtItem& g) {
    const int s = k % AT_ITEMS;
    if (!wait(item_full(s), (k / AT_ITEMS) & 1)) return false;
    g = items[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(item_empty(s));
    return g.done == 0;
  };
  // the ring slot of the n-th K (or V) tile and the parity of that use
  auto k_slot = [&](int n) { return n % S::K_SLOTS; };
  auto v_slot = [&](int n) { return S::K_SLOTS + n % S::V_SLOTS; };
  auto k_par = [&](int n) { return (n / S::K_SLOTS) & 1; };
  auto v_par = [&](int n) { return (n / S::V_SLOTS) & 1; };
  // a checking warp's words for item k, cleared
  auto clear_cuts = [&](int k, int half) {
    const int at = (k % AT_CUTS) * 2 + half;
    if (cut_any[at]) {
      __syncwarp();
      if (lane < AT_CUT_WORDS) cuts[at * AT_CUT_WORDS + lane] = 0;
      if (lane == 0) cut_any[at] = 0;
      __syncwarp();
    }
  };
  auto mark_cut = [&](int k, int half, int bit) {
    const int at = (k % AT_CUTS) * 2 + half;
    atomicOr(cuts + at * AT_CUT_WORDS + (bit >> 5), 1u << (bit & 31));
    cut_any[at] = 1;
  };
  auto tile_pos = [&](const AtItem& g, int i) { return (i < g.st ? i : g.w0 + (i - g.st)) * AT_TILE; };

  if (warp < AT_SOFTMAX_WARPS) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::REGS_SOFTMAX));
    // ----------------------------------------------------------------- softmax
    const int x = warp >> 2;                                       // row tile
    const int r = (warp & 3) * 32 + lane;                          // row: tensor-memory lane
    const int my_tok = r / p.group, my_head = r - my_tok * p.group;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_cols = lane_base + AT_TILE * x, o_cols = lane_base + S::O_COL0 + D * x;
    const unsigned all_boxes = (1u << boxes) - 1u;
    float c = p.scale;                                             // of this row, with E4M3 its powers of two
    int tiles = 0, used = 0, outs = 0, joins = 0, q_seen = 0;   // tiles of the CTA, of this row tile, finished items, meetings
    auto meet = [&]() {   // of the row tile's four warps
      __syncwarp();
      if (lane == 0) mbar_arrive(join_bar(x));
      return wait(join_bar(x), joins++ & 1);
    };
    AtItem g;
    for (int k = 0; get_item(k, g); ++k) {
      const int nt = g.i1 - g.i0;
      const bool active = x == 0 || g.n_tok > tile_tok;
      if (!active) {
        tiles += max(nt, 0);
        if constexpr (E4M3) {
          // in step with the other row tile, whether it has rows or not
          if (nt > 0) {
            if (!wait(q_full, q_seen++ & 1)) break;
            if (lane == 0) mbar_arrive(q_ready(x));
          }
        }
        continue;
      }
      const int tok = x * tile_tok + my_tok;                       // token of the item
      const bool live = my_tok < tile_tok && tok < g.n_tok;
      const int pos = g.p0 + min(tok, g.n_tok - 1);
      float m = -INFINITY, l[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // l in four chains
      bool ok = true;
      if constexpr (E4M3) {
        if (nt > 0) {
          // this thread's row of Q to f16 in place, scaled by a power of two that
          // brings its largest element into [2^14, 2^15): exact for elements above
          // 2^-29 of it. c takes the power back.
          ok = wait(q_full, q_seen++ & 1);
          if (!ok) break;
          auto at_chunk = [&](int e) {   // 16-byte chunk e of the row, 128B swizzle
            return q_tile(x) + (e >> 3) * (AT_ROWS * 128) + r * 128 + (((e & 7) ^ (r & 7)) << 4);
          };
          uint32_t top = 0;              // largest magnitude, bf16 bits of either half
#pragma unroll
          for (int e = 0; e < D / 8; ++e) {
            const uint4 w = lds128(at_chunk(e));
            top = __vmaxu2(top, w.x & 0x7FFF7FFFu);
            top = __vmaxu2(top, w.y & 0x7FFF7FFFu);
            top = __vmaxu2(top, w.z & 0x7FFF7FFFu);
            top = __vmaxu2(top, w.w & 0x7FFF7FFFu);
          }
          const float amax = bf16_bits_to_f32(max(top & 0xFFFFu, top >> 16));
          const int e2 = amax > 0.0f && amax < INFINITY ? ilogbf(amax) - 14 : 0;
          // in two factors: 2^-e2 alone may lie outside fp32
          const int e1 = min(max(-e2, -100), 100);
          const float down = scalbnf(1.0f, e1), rest = scalbnf(1.0f, -e2 - e1);
#pragma unroll
          for (int e = 0; e < D / 8; ++e) {
            const uint4 w = lds128(at_chunk(e));
            const uint32_t y[4] = {w.x, w.y, w.z, w.w};
            uint32_t h[4];
#pragma unroll
            for (int z = 0; z < 4; ++z)
              h[z] = f32x2_to_f16x2(bf16_bits_to_f32(y[z] & 0xFFFFu) * down * rest, bf16_bits_to_f32(y[z] >> 16) * down * rest);
            sts128(at_chunk(e), h);
          }
          c = fmaxf(p.scale * p.k_scale[g.h] * scalbnf(1.0f, e2), 1e-44f);   // not zero: a masked score times it is -inf
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(q_ready(x));
        }
      }
      for (int i = g.i0; i < g.i1; ++i, ++tiles, ++used) {
        ok = wait(s_full(x), used & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t v[4][32];
        tc_ld_32cols(s_cols, v[0]);
        tc_ld_32cols(s_cols + 32, v[1]);
        const int j0 = tile_pos(g, i);
        const unsigned there = oks[tiles % AT_OKS];
        // this row sees columns 0..hi of the tile but for sk..lo - 1
        const int hi = min(pos, g.key_end - 1) - j0;
        const int lo = p.window > 0 ? pos - p.window + 1 - j0 : 0, sk = p.window > 0 ? p.sinks - j0 : 0;
        const bool whole = hi >= AT_TILE - 1 && (lo <= 0 || sk >= AT_TILE) && there == all_boxes;
        const bool masked = !__all_sync(0xffffffffu, whole);
        const int box_log2 = 31 - __clz(box);
        // scores of a row that are masked, and its maximum in four chains; the
        // second half arrives meanwhile
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if ((q & 1) == 0) tc_wait_ld();
          if (q == 0) {
            tc_ld_32cols(s_cols + 64, v[2]);
            tc_ld_32cols(s_cols + 96, v[3]);
          }
          if (masked) {
            // bit e: this row sees column 32 q + e
            const uint32_t page_bits = (((there >> ((32 * q) >> box_log2)) & 1u) ? 0x0000FFFFu : 0u) |
                                       (((there >> ((32 * q + 16) >> box_log2)) & 1u) ? 0xFFFF0000u : 0u);
            const uint32_t sees = low_bits(hi + 1 - 32 * q) & (~low_bits(lo - 32 * q) | low_bits(sk - 32 * q)) & page_bits;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(sees & (1u << e))) v[q][e] = 0xFF800000u;   // -inf
          }
          mx[q] = fmaxf(__uint_as_float(v[q][0]), __uint_as_float(v[q][1]));
#pragma unroll
          for (int e = 2; e < 32; e += 2) mx[q] = max3(mx[q], __uint_as_float(v[q][e]), __uint_as_float(v[q][e + 1]));
        }
        const float mn = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), m);
        const bool grows = (mn - m) * c > KvWeights<E4M3>::SLACK;
        const bool rescale = __any_sync(0xffffffffu, grows);
        float alpha = 1.0f;
        if (rescale) {
          // (a row's steps depend on its own scores alone: its bits must not on the warp's other rows)
          if (grows) {
            alpha = exp2_approx((m - mn) * c);
            m = mn;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) l[e] *= alpha;
          if (!E4M3 && i > g.i0) {
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tc_ld_16cols(o_cols + 16 * q, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tc_st_16cols(o_cols + 16 * q, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.0f : KvWeights<E4M3>::LIFT - m * c;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a = __uint_as_float(v[q][2 * e]), b = __uint_as_float(v[q][2 * e + 1]);
            fma2(a, b, c, neg);
            a = exp2_approx(a);
            b = exp2_approx(b);
            add2(l[2 * (e & 1)], l[2 * (e & 1) + 1], a, b);
            w[e] = E4M3 ? kv_weights_f16x2(a, b) : f32x2_to_bf16x2(a, b);
          }
          tc_st_16cols(s_cols + 16 * q, w);
        }
        if (E4M3 && rescale && i > g.i0) {
          // the scores' registers are free here (2,048 new tokens on 6,144, 32 heads on
          // 8: 314 -> 282 us at a slack of 4; bf16 caches, which come here less often,
          // lost 3%). Rolled: this kernel's time goes with its code's size (unrolled
          // 272 us, rolled 260)
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tc_ld_32cols(o_cols + 32 * q, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc_st_32cols(o_cols + 32 * q, o);
          }
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(x));
      }
      if (!ok) break;
      const float sum_l = (l[0] + l[1]) + (l[2] + l[3]);
      const float v_mult = E4M3 ? p.v_scale[g.h] : 1.0f;
      if (nt > 0) {
        ok = wait(o_full(x), outs & 1);
        if (!ok) break;
        ++outs;
        tc_fence_after();
      }
      // whether elements were taken out of the item's values; give_back(add) calls
      // add(d, v) for those that this row sees, v four elements from d on
      const int cut_at = (k % AT_CUTS) * 2;
      const bool cut = nt > 0 && (cut_any[cut_at] | cut_any[cut_at + 1]) != 0;
      auto give_back = [&](auto add) {
        const int32_t* row = p.s.table + static_cast<int64_t>(g.b) * p.s.table_stride;
#pragma unroll 1
        for (int w = 0; w < 2 * AT_CUT_WORDS; ++w) {
#pragma unroll 1
          for (unsigned bits = *reinterpret_cast<volatile unsigned*>(cuts + cut_at * AT_CUT_WORDS + w); bits; bits &= bits - 1) {
            const int n = (w % AT_CUT_WORDS) * 32 + __ffs(static_cast<int>(bits)) - 1;
            const int j = n < 256 ? g.p0 + 1 + n : max(g.p0 - p.window + 1, p.sinks) + (n - 256);
            if (!live || !kv_sees(pos, j, p.window, p.sinks)) continue;
            const int64_t at = ((static_cast<int64_t>(row[j >> p.page_log2]) * p.heads + g.h) * p.page_size + (j & (p.page_size - 1))) * D;
#pragma unroll 1
            for (int d = 0; d < D; d += 4) {
              const float4 v = kv_not_finite<E4M3>(p.v, at + d);
              if (v.x != 0.0f || v.y != 0.0f || v.z != 0.0f || v.w != 0.0f) add(d, v);
            }
          }
        }
      };
      uint16_t* dst = p.out + (static_cast<int64_t>(g.row0 + tok) * p.heads * p.group + static_cast<int64_t>(g.h) * p.group + my_head) * D;
      if (g.parts == 1) {
        const float inv = sum_l > 0.0f ? v_mult / sum_l : (sum_l == 0.0f ? 0.0f : sum_l);   // a NaN stays one
        // bf16 rows through shared memory, 64 d's at a time, so that a store
        // writes four rows' 128 bytes: from one row per thread it would write 32
        // rows' 16 (E4M3 caches leave no room for that)
        const uint32_t my_off = live ? static_cast<uint32_t>((tok * p.heads * p.group + my_head) * D) : 0xFFFFFFFFu;
        uint16_t* out0 = p.out + (static_cast<int64_t>(g.row0) * p.heads * p.group + static_cast<int64_t>(g.h) * p.group) * D;
        const uint32_t stage = slot(S::K_SLOTS + S::V_SLOTS) + warp * (32 * 128);
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {
          uint32_t o[2][32];
          if (nt > 0) {
            tc_ld_32cols(o_cols + 64 * hf, o[0]);
            tc_ld_32cols(o_cols + 64 * hf + 32, o[1]);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[0][e] = o[1][e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t y[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const int q = 8 * (e & 3) + 2 * z;
              y[z] = f32x2_to_bf16x2(__uint_as_float(o[e >> 2][q]) * inv, __uint_as_float(o[e >> 2][q + 1]) * inv);
            }
            if constexpr (E4M3) {
              if (live) *reinterpret_cast<uint4*>(out0 + my_off + 64 * hf + 8 * e) = make_uint4(y[0], y[1], y[2], y[3]);
            } else {
              sts128(stage + lane * 128 + ((e ^ (lane & 7)) << 4), y);
            }
          }
          if constexpr (!E4M3) {
            __syncwarp();
#pragma unroll
            for (int it = 0; it < 8; ++it) {
              const int rr = 4 * it + (lane >> 3), e = lane & 7;
              const uint32_t off = __shfl_sync(0xffffffffu, my_off, rr);
              const uint4 y = lds128(stage + rr * 128 + ((e ^ (rr & 7)) << 4));
              if (off != 0xFFFFFFFFu) *reinterpret_cast<uint4*>(out0 + off + 64 * hf + 8 * e) = y;
            }
            __syncwarp();
          }
        }
        if (cut) {
          // (the row was written by this warp's lanes: they have met since)
          __syncwarp();
          give_back([&](int d, float4 v) {
            const uint2 y = __ldcg(reinterpret_cast<const uint2*>(dst + d));
            *reinterpret_cast<uint2*>(dst + d) =
                make_uint2(f32x2_to_bf16x2(bf16_bits_to_f32(y.x & 0xFFFFu) + v.x, bf16_bits_to_f32(y.x >> 16) + v.y),
                           f32x2_to_bf16x2(bf16_bits_to_f32(y.y & 0xFFFFu) + v.z, bf16_bits_to_f32(y.y >> 16) + v.w));
          });
        }
        tc_fence_before();
        continue;
      }
      // this part's (m, l, o); the last part of the row tile to arrive joins them in order
      auto part = [&](int i) {
        return p.part + ((static_cast<int64_t>(g.item) * p.parts + i) * 2 + x) * (AT_ROWS * (D + 2));
      };
      {
        float* mine = part(g.part);
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          if (nt > 0) {
            tc_ld_32cols(o_cols + 32 * q, o);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            __stcg(reinterpret_cast<float4*>(mine) + (8 * q + e / 4) * AT_ROWS + r,
                   make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                               __uint_as_float(o[e + 3])));
        }
        __stcg(reinterpret_cast<float2*>(mine + AT_ROWS * D + 2 * r), make_float2(m * c, sum_l));
        if (cut)
          give_back([&](int d, float4 v) {
            float4* y = reinterpret_cast<float4*>(mine) + (d / 4) * AT_ROWS + r;
            const float4 x = __ldcg(y);
            __stcg(y, make_float4(x.x + v.x, x.y + v.y, x.z + v.z, x.w + v.w));
          });
        tc_fence_before();
      }
      if (!meet()) break;   // the four warps' shares are written: the release below covers them
      if ((threadIdx.x & 127) == 0) {
        unsigned* counter = p.arrived + g.item * 2 + x;
        unsigned before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
        last_flag[x] = before + 1 == static_cast<unsigned>(g.parts);
        if (before + 1 == static_cast<unsigned>(g.parts)) *counter = 0;   // ready for the next call
      }
      if (!meet()) break;
      if (last_flag[x] && live) {
        float mx = -INFINITY;
        for (int i = 0; i < g.parts; ++i) mx = fmaxf(mx, __ldcg(part(i) + AT_ROWS * D + 2 * r));
        const float use = mx == -INFINITY ? 0.0f : mx;
        float sum = 0.0f;
        for (int i = 0; i < g.parts; ++i) {
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(part(i) + AT_ROWS * D + 2 * r));
          sum += ml.y * exp2_approx(ml.x - use);
        }
        const float inv = sum > 0.0f ? v_mult / sum : (sum == 0.0f ? 0.0f : sum);
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
          float acc[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
#pragma unroll 4
          for (int i = 0; i < g.parts; ++i) {
            const float f = exp2_approx(__ldcg(part(i) + AT_ROWS * D + 2 * r) - use) * inv;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 y = __ldcg(reinterpret_cast<const float4*>(part(i)) + (4 * q + e / 4) * AT_ROWS + r);
              acc[e] += y.x * f;
              acc[e + 1] += y.y * f;
              acc[e + 2] += y.z * f;
              acc[e + 3] += y.w * f;
            }
          }
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            *reinterpret_cast<uint4*>(dst + 16 * q + e) =
                make_uint4(f32x2_to_bf16x2(acc[e], acc[e + 1]), f32x2_to_bf16x2(acc[e + 2], acc[e + 3]),
                           f32x2_to_bf16x2(acc[e + 4], acc[e + 5]), f32x2_to_bf16x2(acc[e + 6], acc[e + 7]));
        }
      }
      if (!meet()) break;   // the flag may be written again
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_OTHER));
    if (warp == AT_PROD_WARP || (E4M3 && warp == AT_V_PROD_WARP)) {
      // ---------------------------------------------------------------- producer
      // (with E4M3 a second one for V, so that K's codes need not wait for it)
      const bool first = warp == AT_PROD_WARP;   // announces items, brings Q
      const int64_t table_end = static_cast<int64_t>(p.s.max_pages) * p.page_size;
      int tiles = 0, asked[2] = {0, 0}, q_used = 0;   // tiles done, K and V tiles requested, items whose Q was
      bool ok = true;
      int k = -1, b_from = 0;                  // items announced
      int64_t run_from = 0;
      for (int64_t w = blockIdx.x; ok; w += gridDim.x) {
        // work item w: (sequence, block of its rows, kv head, part), the parts of
        // a block next to each other, then its heads; late blocks, which see
        // more, come first
        const int64_t flat = w / (p.parts * p.heads);
        const int rest = static_cast<int>(w - flat * (p.parts * p.heads));
        AtItem g = {};
        g.done = 1;
        g.h = rest / p.parts;
        g.part = rest - g.h * p.parts;
        g.item = static_cast<int>(w / p.parts);
        const int32_t* row = p.s.table;
        int64_t run = run_from;
        for (int b0 = b_from; b0 < p.s.batch && g.done; b0 += 32) {
          const int b = b0 + lane;
          const int r0 = b < p.s.batch ? kv_row0(p.s, b) : 0;
          const int n = b < p.s.batch ? max(kv_row0(p.s, b + 1) - r0, 0) : 0;
          const int blocks = (n + item_tok - 1) / item_tok;
          int x = blocks;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, run + x > flat);
          if (hit) {
            b_from = b0;   // items come in order: the next one's search begins here
            run_from = run;
            const int src = __ffs(hit) - 1;
            const int n_b = __shfl_sync(0xffffffffu, n, src), r0_b = __shfl_sync(0xffffffffu, r0, src);
            const int nb = __shfl_sync(0xffffffffu, blocks, src), before = __shfl_sync(0xffffffffu, x, src) - nb;
            const int blk = nb - 1 - static_cast<int>(flat - run - before);
            const int len = kv_len(p.s, b0 + src);
            g.done = 0;
            g.b = b0 + src;
            g.row0 = r0_b + blk * item_tok;
            g.n_tok = min(item_tok, n_b - blk * item_tok);
            g.p0 = len - n_b + blk * item_tok;
            g.key_end = static_cast<int>(min(table_end, static_cast<int64_t>(len)));
            const KvTiles tl = kv_tiles<AT_TILE>(g.p0, g.p0 + g.n_tok - 1, p.window, p.sinks, g.key_end);
            g.st = tl.st;
            g.w0 = tl.w0;
            // parts of two tiles at least
            g.parts = max(1, min(p.parts, tl.count / 2));
            g.i0 = static_cast<int>(static_cast<int64_t>(tl.count) * g.part / g.parts);
            g.i1 = static_cast<int>(static_cast<int64_t>(tl.count) * (g.part + 1) / g.parts);
            row = p.s.table + static_cast<int64_t>(b0 + src) * p.s.table_stride;
          }
          run += __shfl_sync(0xffffffffu, x, 31);
        }
        if (!g.done && w >= p.units) {
          // more blocks than `tokens` rows can hold: offsets that fall. The workspace has no room for them.
          if (lane == 0) atomicExch(p.status, NVFP4_ERR_INVALID_ARG);
          g.done = 1;
        }
        if (!g.done && g.part >= g.parts) continue;   // fewer parts than the launch has room for
        ++k;
        const int slot_i = k % AT_ITEMS;
        if (first && k >= AT_ITEMS && !(ok = wait(item_empty(slot_i), ((k / AT_ITEMS) - 1) & 1))) break;
        if (first && lane == 0) {
          items[slot_i] = g;
          mbar_arrive(item_full(slot_i));
        }
        if (g.done) break;
        if (g.i1 <= g.i0) continue;
        auto page_of = [&](int i) {   // lane's box of tile i: its page, -1 where there is none
          const int j = tile_pos(g, i) + (lane & (boxes - 1)) * box;
          const int e = j >> p.page_log2;
          const int page = j < g.key_end && e < p.s.max_pages ? row[e] : -1;
          return page >= 0 && page < p.pages ? page : -1;
        };
        int page = page_of(g.i0);
        // both row tiles of Q, once the last item's MMAs have read theirs
        if (first && q_used > 0 && !(ok = wait(q_empty, (q_used - 1) & 1))) break;
        if (first && lane == 0) {
          const int n_x = g.n_tok > tile_tok ? 2 : 1;
          mbar_arrive_expect_tx(q_full, n_x * S::HALVES * tile_tok * p.group * 128);
          for (int x = 0; x < n_x; ++x)
            for (int hf = 0; hf < S::HALVES; ++hf)
              tma_load_4d(q_tile(x) + hf * (AT_ROWS * 128), &map_q, 0, g.h * p.group, g.row0 + x * tile_tok, hf, q_full);
        }
        ++q_used;
        for (int i = g.i0; i < g.i1 && ok; ++i, ++tiles) {
          const unsigned there = __ballot_sync(0xffffffffu, lane < boxes && page >= 0);
          // a page that is not there: a box past the pool's end, which the copy fills with zeros
          const int64_t block = page >= 0 ? static_cast<int64_t>(page) * p.heads + g.h : p.pages * p.heads;
          const int y = (tile_pos(g, i) + (lane & (boxes - 1)) * box) & (p.page_size - 1);
          if (i + 1 < g.i1) page = page_of(i + 1);
          if constexpr (E4M3) {
            // codes in chunks of 32 rows; the converters read them
            const int kv = first ? 0 : 1;
            if (first && lane == 0) oks[tiles % AT_OKS] = there;
            const int per = boxes / AT_CHUNKS;   // boxes of a chunk: those of lanes cu * per .. + per - 1
            for (int cu = 0; cu < AT_CHUNKS; ++cu) {
              if (tiles > 0 && !(ok = wait(chunk_empty(kv, cu), (tiles - 1) & 1))) break;
              if (lane == 0) mbar_arrive_expect_tx(chunk_full(kv, cu), S::CHUNK_BYTES);
              __syncwarp();
              if (lane < boxes && lane / per == cu)
                tma_load_4d(chunk(kv, cu) + (lane - cu * per) * box * D, kv ? &map_v : &map_k, 0, y, 0, static_cast<int>(block),
                            chunk_full(kv, cu));
              asked[kv] = tiles * AT_CHUNKS + cu + 1;
            }
          } else {
            for (int kv = 0; kv < 2; ++kv) {
              const int s = kv ? v_slot(tiles) : k_slot(tiles);
              if (tiles >= (kv ? S::V_SLOTS : S::K_SLOTS) &&
                  !(ok = wait(kv_empty(s), kv ? v_par(tiles - S::V_SLOTS) : k_par(tiles - S::K_SLOTS))))
                break;
              if (lane == 0) {
                if (kv == 0) oks[tiles % AT_OKS] = there;
                mbar_arrive_expect_tx(kv_full(s), S::MAT_BYTES);
              }
              __syncwarp();
              if (lane < boxes)
                for (int hf = 0; hf < S::HALVES; ++hf)
                  tma_load_4d(slot(s) + hf * (AT_TILE * 128) + lane * box * 128, kv ? &map_v : &map_k, 0, y, hf,
                              static_cast<int>(block), kv_full(s));
              ++asked[kv];
            }
          }
          if (!ok) break;
        }
      }
      if (!ok) {
        // the copies in flight land before this CTA's shared memory goes
        for (int kv = 0; kv < 2; ++kv)
          for (int n = max(asked[kv] - (E4M3 ? AT_CHUNKS : kv ? S::V_SLOTS : S::K_SLOTS), 0); n < asked[kv]; ++n) {
            const uint32_t bar = E4M3 ? chunk_full(kv, n % AT_CHUNKS) : kv_full(kv ? v_slot(n) : k_slot(n));
            mbar_wait_bounded(bar, E4M3 ? (n / AT_CHUNKS) & 1 : kv ? v_par(n) : k_par(n), nullptr, p.status);
          }
        if (first && q_used > 0) mbar_wait_bounded(q_full, (q_used - 1) & 1, nullptr, p.status);
      }
    } else if (warp == AT_MMA_WARP) {
      // -------------------------------------------------------------- MMA issue
      // kind::f16, bf16 (E4M3 caches: f16) A and B, fp32 D, M = 128; S = Q K^T: both K-major, N =
      // 128; O = P V: V's d's are contiguous, so B is N-major (bit 16), N = D.
      // The whole warp walks the loops and one lane's MMAs take effect, by a
      // predicate and not a branch, with loop bounds from warp reductions: so
      // descriptors stay in uniform registers. Issued from a one-lane branch a
      // MMA took about 100 clocks to issue, more than its 64 on the tensor
      // cores (2k rows on 8k positions: 231 -> 188 us). One warp for each row
      // tile was slower (267 us): their MMAs interleave, so both tiles' scores
      // come late together instead of in turns.
      constexpr uint32_t ab = E4M3 ? 0u : (1u << 7) | (1u << 10);   // f16 or bf16 A and B
      constexpr uint32_t idesc_s = (1u << 4) | ab | ((AT_TILE >> 3) << 17) | ((AT_ROWS >> 4) << 24);
      constexpr uint32_t idesc_o = (1u << 4) | ab | (1u << 16) | ((D >> 3) << 17) | ((AT_ROWS >> 4) << 24);
      const uint64_t desc_q = smem_desc(q_tile(0), 16, 1024, 2), desc_k = smem_desc(slot(0), 16, 1024, 2);
      const uint64_t desc_v = smem_desc(slot(S::K_SLOTS), AT_TILE * 128, 1024, 2);
      const uint32_t lead = elect_one();
      int tiles = 0, q_used = 0;   // tiles done, items with tiles
      int p_used[2] = {0, 0};
      bool ok = true;
      AtItem g;
      for (int k = 0; ok && get_item(k, g); ++k) {
        const int nt = __reduce_max_sync(0xffffffffu, g.i1 - g.i0);
        if (nt <= 0) continue;
        const int n_x = __reduce_max_sync(0xffffffffu, g.n_tok > tile_tok ? 2 : 1);
        auto issue_s = [&](int x, int n) {   // S_x = Q_x K^T with the n-th K tile
          const uint64_t q0 = desc_q + static_cast<uint64_t>(x) * (S::MAT_BYTES >> 4);
          const uint64_t k0 = desc_k + static_cast<uint64_t>(k_slot(n)) * (S::MAT_BYTES >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            // the descriptors' address field counts 16 bytes
            const uint64_t off = ((ks >> 2) * (AT_TILE * 128) + (ks & 3) * 32) >> 4;
            tc_mma_bf16_ss(tmem + AT_TILE * x, q0 + off, k0 + off, idesc_s, ks > 0, lead);
          }
          if (lead) {
            tc_commit(s_full(x));
            if (x + 1 == n_x) tc_commit(kv_empty(k_slot(n)));
          }
          __syncwarp();
        };
        if constexpr (E4M3) {
          // the softmax warps convert each row tile's Q
          ok = wait(q_ready(0), q_used & 1) && wait(q_ready(1), q_used & 1);
        } else {
          ok = wait(q_full, q_used & 1);
        }
        if (!ok || !(ok = wait(kv_full(k_slot(tiles)), k_par(tiles)))) break;
        ++q_used;
        tc_fence_after();
        for (int x = 0; x < n_x; ++x) issue_s(x, tiles);
        if (nt == 1 && lead) tc_commit(q_empty);
        __syncwarp();
        for (int i = 0; i < nt && ok; ++i, ++tiles) {
          const int sv = v_slot(tiles);
          const bool more = i + 1 < nt;
          if (!(ok = wait(kv_clean(sv), v_par(tiles)))) break;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (x >= n_x) break;
            if (!(ok = wait(p_full(x), p_used[x] & 1))) break;
            ++p_used[x];
            tc_fence_after();
            const uint32_t d = tmem + S::O_COL0 + D * x, a = tmem + AT_TILE * x;
            const uint64_t v0 = desc_v + static_cast<uint64_t>(sv - S::K_SLOTS) * (S::MAT_BYTES >> 4);
            tc_mma_bf16_ts(d, a, v0, idesc_o, i > 0, lead);
#pragma unroll
            for (int ks = 1; ks < AT_TILE / 16; ++ks)   // 16 positions of V, 8 columns of P
              tc_mma_bf16_ts(d, a + 8 * ks, v0 + ((ks * 16 * 128) >> 4), idesc_o, 1, lead);
            if (lead) {
              if (x + 1 == n_x) tc_commit(kv_empty(sv));
              if (!more) tc_commit(o_full(x));
            }
            __syncwarp();
            if (!more) continue;
            if (x == 0 && !(ok = wait(kv_full(k_slot(tiles + 1)), k_par(tiles + 1)))) break;
            issue_s(x, tiles + 1);
          }
          if (ok && lead && i + 2 == nt) tc_commit(q_empty);
          __syncwarp();
        }
      }
      // every MMA issued so far has completed before the CTA's memory goes
      if (lead) tc_commit(drain_bar);
      mbar_wait_bounded(drain_bar, 0, nullptr, p.status);
      __syncwarp();
    } else if constexpr (E4M3) {
      if (warp == AT_CHECK_WARP) {
        // ----------------------------- V's codes on their way to the converters
        int tiles = 0;
        bool ok = true;
        AtItem g;
        for (int k = 0; ok && get_item(k, g); ++k) {
          clear_cuts(k, 0);
          const int p1 = g.p0 + g.n_tok - 1;
          for (int i = g.i0; i < g.i1 && ok; ++i, ++tiles) {
            // tile rows that later rows of the item see and earlier ones do not, and the other way round
            const int j0 = tile_pos(g, i), a0 = g.p0 + 1 - j0, a1 = p1 + 1 - j0;
            const int b0 = max(g.p0 - p.window + 1, p.sinks) - j0, b1 = p.window > 0 ? min(p1 - p.window, g.p0) + 1 - j0 : b0;
            for (int cu = 0; cu < AT_CHUNKS; ++cu) {
              if (!(ok = wait(chunk_full(1, cu), tiles & 1))) break;
              const int c0 = cu * AT_CHUNK, c1 = c0 + AT_CHUNK;
              if ((max(a0, c0) < min(a1, c1)) || (max(b0, c0) < min(b1, c1))) {
#pragma unroll 2
                for (int u = 0; u < D / 16; ++u) {
                  const int row = c0 + (u * 32 + lane) / (D / 16), piece = lane % (D / 16);
                  if (!((row >= a0 && row < a1) || (row >= b0 && row < b1))) continue;
                  const uint32_t addr = chunk(1, cu) + (u * 32 + lane) * 16;
                  const uint4 w = lds128(addr);
                  uint32_t y[4] = {w.x, w.y, w.z, w.w}, any = 0;
#pragma unroll
                  for (int z = 0; z < 4; ++z) {
                    const uint32_t top = ((y[z] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;   // bit 7 of a NaN's byte
                    any |= top;
                    y[z] &= ~((top >> 7) * 0xFFu);
                  }
                  if (!any) continue;
                  mark_cut(k, 0, row >= a0 && row < a1 ? row - a0 : 256 + row - b0);
                  sts128(addr, y);
                  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the chunk's next copy comes after
                }
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(chunk_ok(cu));
            }
          }
        }
      }
      if (warp >= AT_CONVERT_WARP) {
        // ---------------- codes to f16 tiles: two warps for K, two for V, which
        // also do the clean warp's work; each takes every second chunk
        const int kv = (warp - AT_CONVERT_WARP) >> 1, sub = warp & 1;
        constexpr int UNITS = D / 16;       // 16-byte pieces of a code row; pieces of a lane in a chunk
        constexpr int BATCH = 4;            // pieces in registers at once
        int tiles = 0;
        bool ok = true;
        AtItem g;
        for (int k = 0; ok && get_item(k, g); ++k) {
          const int p1 = g.p0 + g.n_tok - 1;
          for (int i = g.i0; i < g.i1 && ok; ++i, ++tiles) {
            const int j0 = tile_pos(g, i), s = kv ? v_slot(tiles) : k_slot(tiles);
            if (tiles >= (kv ? S::V_SLOTS : S::K_SLOTS) &&
                !(ok = wait(kv_empty(s), kv ? v_par(tiles - S::V_SLOTS) : k_par(tiles - S::K_SLOTS))))
              break;
            const bool unclean = kv && at_unclean(j0, g.p0, p1, p.window, p.sinks);
            for (int cu = sub; cu < AT_CHUNKS; cu += 2) {
              if (!(ok = wait(kv ? chunk_ok(cu) : chunk_full(0, cu), tiles & 1))) break;
#pragma unroll 1
              for (int u0 = 0; u0 < UNITS; u0 += BATCH) {
                uint4 w[BATCH];
#pragma unroll
                for (int u = 0; u < BATCH; ++u) w[u] = lds128(chunk(kv, cu) + ((u0 + u) * 32 + lane) * 16);
                if (u0 + BATCH == UNITS) {
                  __syncwarp();
                  if (lane == 0) mbar_arrive(chunk_empty(kv, cu));
                }
#pragma unroll
                for (int u = 0; u < BATCH; ++u) {
                  const int row = cu * AT_CHUNK + ((u0 + u) * 32 + lane) / UNITS, piece = lane % UNITS;
                  if (unclean) {
                    // value rows no row of the item sees become zeros: they may hold anything, and 0 * NaN is not 0
                    const int j = j0 + row;
                    if (j > p1 || (p.window > 0 && j >= p.sinks && g.p0 - j >= p.window)) w[u] = make_uint4(0u, 0u, 0u, 0u);
                  }
                  uint32_t y[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf) {
                    uint32_t h[4];
                    e4m3x4_to_f16x2(y[2 * hf], h[0], h[1]);
                    e4m3x4_to_f16x2(y[2 * hf + 1], h[2], h[3]);
                    const int c8 = 2 * piece + hf;   // 16-byte chunk of the f16 row
                    sts128(slot(s) + (c8 >> 3) * (AT_TILE * 128) + row * 128 + (((c8 & 7) ^ (row & 7)) << 4), h);
                  }
                }
              }
            }
            if (!ok) break;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(kv ? kv_clean(s) : kv_full(s));
          }
        }
      }
    } else if (warp == AT_CLEAN_WARP || warp == AT_CLEAN_WARP + 1) {
      // --------------------------------------- value rows that no row may take in
      // every V tile passes here, so these warps and the rings stay in step
      const int half = warp - AT_CLEAN_WARP;
      int tiles = 0;
      bool ok = true;
      AtItem g;
      for (int k = 0; ok && get_item(k, g); ++k) {
        clear_cuts(k, half);
        const int p1 = g.p0 + g.n_tok - 1;
        for (int i = g.i0; i < g.i1; ++i, ++tiles) {
          const int j0 = tile_pos(g, i), s = v_slot(tiles);
          ok = wait(kv_full(s), v_par(tiles));
          if (!ok) break;
          bool wrote = false;
          // tile rows c0 .. c1 - 1, 16 bytes a step, shared by the two warps
          auto each = [&](int c0, int c1, auto f) {
            c0 = max(c0, 0);
            c1 = min(c1, AT_TILE);
            for (int e = c0 * 8 + half * 32 + lane; e < c1 * 8; e += 64)
#pragma unroll
              for (int hf = 0; hf < S::HALVES; ++hf) f(slot(s) + hf * (AT_TILE * 128) + e * 16, e >> 3);
            wrote = wrote || c0 < c1;
          };
          // rows past the item's last position, and rows between the sinks and its first window
          auto zero = [&](uint32_t addr, int) { sts128(addr, {0u, 0u, 0u, 0u}); };
          each(p1 + 1 - j0, AT_TILE, zero);
          if (p.window > 0) each(p.sinks - j0, g.p0 - p.window + 1 - j0, zero);
          // rows that later rows of the item see and earlier ones do not, and the other way round
          // (bit0: the bit of tile row 0)
          auto check = [&](int bit0) {
            return [&, bit0](uint32_t addr, int row) {
              const uint4 w = lds128(addr);
              uint32_t y[4] = {w.x, w.y, w.z, w.w}, any = 0;
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const uint32_t top = ((y[z] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;   // bit 15 of a half whose exponent is all ones
                any |= top;
                y[z] &= ~((top >> 15) * 0xFFFFu);
              }
              if (!any) return;
              mark_cut(k, half, bit0 + row);
              sts128(addr, y);
            };
          };
          each(g.p0 + 1 - j0, p1 + 1 - j0, check(j0 - (g.p0 + 1)));
          if (p.window > 0) {
            const int lo_b = max(g.p0 - p.window + 1, p.sinks);
            each(lo_b - j0, min(p1 - p.window, g.p0) + 1 - j0, check(256 + j0 - lo_b));
          }
          if (wrote) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(kv_clean(s));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == AT_MMA_WARP)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

}  // namespace
}  // namespace nvfp4
