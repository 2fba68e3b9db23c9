// Attention of few new rows over a paged key-value cache, split over the
// cache's length and joined in the same launch.
//
// The mathematics. Row r (one query head at one new token) sees the positions
// V(r) of its mask; out_r = sum_j exp(x_rj - m_r) v_j / sum_j exp(x_rj - m_r)
// with x_rj = scale q_r.k_j and m_r = max x_rj. A pass over any part of V(r)
// keeps (m, l = sum exp(x - m), o = sum exp(x - m) v), the online softmax of
// Milakov and Gimelshein (2018), and two parts join as
// m = max(m1, m2), l = l1 e^(m1-m) + l2 e^(m2-m), o likewise. All of it is
// fp32, in powers of two (log2 e folded into the scale).
//
// What bounds it: each key and value byte is used by the rows of one kv head
// only (G query heads of 1..8 tokens), so it is bound by streaming K and V.
// Tokens are the M side of mma.sync m16n8k16 (S^T = K Q^T, then O^T = V^T P^T)
// and rows its N side, eight at a time, so four rows cost half of what they
// would as a 16-row M side: 16 MMAs for 16 tokens, 8 rows and D = 128, an
// eighth of the time that the bytes take to arrive.
//
// Work is cut by device-side lengths: the (sequence, kv head, block of 8 NT
// rows) items, each of as many 64-token tiles as its rows see, lie on one line
// that is cut into equal pieces, one per CTA. A CTA whose piece ends inside an
// item leaves (m, l, o) in the workspace; the last of an item's CTAs to arrive
// joins them in CTA order, so results do not depend on which one it is.
//
// One producer warp keeps a ring of tiles full (a page's rows are one 4-D box;
// pages shorter than 64 tokens give several boxes), another one brings the next
// item and its query rows as fragments. Four consumer warps take 16 tokens of a
// tile each, with an online softmax of their own, and meet at the end of an
// item. A key or value fragment is loaded (and from E4M3 converted) once for all
// rows of an item.
//
// Roundings. Products are exact in fp32 sums. bf16 caches: q and k as they
// are; p is split into two bf16 halves (p = hi + lo to 2^-16), since one bf16
// would cost as much error as the output's own rounding and the second MMA
// costs no time here. E4M3 caches: k and v are exact in f16, q is scaled by a
// power of two into f16 (exact for elements above amax 2^-29), p is one f16
// (2^-11, an eighth of the output's rounding) in f16's upper range (kv.cuh): that
// much down to 2^-25 of the heaviest weight so far, and an absolute 2^-36 of it
// below.
//
// Measured, 8 kv heads, D = 128: 64 sequences of 9k..22k positions, bf16, 578 us
// (the copy rate); 8 sequences of 517..24k, 20 rows, E4M3, 63.8 us against 29.7
// for the bytes (bound by instruction latency); 8 of 22k, single tokens, E4M3,
// 64.2 us against 53.2; one sequence of 2k positions, 8.6 us on the device.
//
// Masked places: scores are replaced, not added to; a token no row of the item
// sees has its value row replaced by zeros (stale page contents may be NaN),
// elements that are not finite in tokens that some rows see and others do not are
// taken out by the producer and given back at the output (kv.cuh), and pages that
// are not there are filled with zeros by the copy engine (their boxes lie past the
// pool's last page).
#pragma once

#include "kv.cuh"
#include "tcgen05.cuh"

namespace nvfp4 {
namespace {

constexpr int AR_WARPS = 4;                  // consumer warps, 16 tokens of a tile each
constexpr int AR_MAX_STAGES = 8;
constexpr int AR_ITEMS = 2;                  // items announced ahead
constexpr int AR_KEPT = 128;                 // sequences whose lengths are kept in shared memory
constexpr int AR_PAD = 4;                    // fp32 words between rows of the merge buffer: no bank conflicts
constexpr unsigned AR_ALL = 0xffffffffu;

struct ArParams {
  KvSeqs s;
  const uint16_t* q;
  const void* v;          // the value pool
  int64_t q_stride;
  uint16_t* out;
  const float* k_scale;
  const float* v_scale;
  int64_t pages;
  int heads, group;       // kv heads, query heads per kv head
  int page_size, page_log2;
  int window, sinks;
  float scale;            // softmax scale * log2 e
  unsigned* arrived;      // [CTAs], zero between calls
  float* part;            // [CTAs][2][rows of an item][D + 2]
  int stages;             // of the ring
  int* status;
};

// A shape of the kernel for NT eight-row tiles of queries. Up to three, two CTAs
// fit an SM's registers; four need 255 a thread (8 sequences of 22k positions,
// E4M3, 20 rows: eight warps of one CTA 120 us, four of two CTAs 100 us; bf16,
// 32 rows: eight warps 183 us, spilling, four warps of one CTA 151 us).
template <bool E4M3, int D, int NT>
struct ArShape {
  static constexpr int TILE = 16 * AR_WARPS;                        // tokens of a tile
  static constexpr int ROWS = 8 * NT;
  static constexpr int THREADS = (AR_WARPS + 2) * 32;               // consumers, the producer, the item warp
  static constexpr int CTAS = NT <= 3 ? 2 : 1;                   // per SM
  static constexpr int EXTRA = 3;                                // tiles' time that an item costs beside its tiles
  static constexpr int BUFS = NT <= 3 ? 2 : 4;                   // merge buffers
  static constexpr bool Q_REGS = NT <= 2;                        // query fragments in registers, else read per tile
  static constexpr int ROW_BYTES = D * (E4M3 ? 1 : 2);
  static constexpr int SEG = ROW_BYTES >= 128 ? 128 : 64;        // bytes of a swizzled row of a box
  static constexpr int HALVES = ROW_BYTES / SEG;
  static constexpr int MAT_BYTES = TILE * ROW_BYTES;             // K or V of a tile
  static constexpr int STAGE_BYTES = 2 * MAT_BYTES;
  static constexpr int KS = D / 16;                              // 16-d steps
  static constexpr int OSTR = D + AR_PAD;
  static constexpr int QFRAGS = KS * NT * 32;
  // shared memory without the ring: merge buffers, fragments, multipliers and
  // positions of the announced items, each warp's m and l, barriers
  static constexpr int FIXED_BYTES = 1024 + BUFS * ROWS * OSTR * 4 + AR_ITEMS * (QFRAGS * 8 + ROWS * 8) + 2 * AR_WARPS * ROWS * 4 +
                                     8 * (2 * AR_MAX_STAGES + 2 * AR_ITEMS + 1) + 12 * AR_MAX_STAGES + AR_ITEMS * 64 + 64;
};

NVFP4_DEV void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
NVFP4_DEV void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 8x8 16-bit transpose across the warp
NVFP4_DEV uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
NVFP4_DEV void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// AND of `pred` over the N consumer threads.
template <int N>
NVFP4_DEV bool ar_all(bool pred) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(static_cast<uint32_t>(pred)), "n"(N)
      : "memory");
  return out != 0;
}
template <int N>
NVFP4_DEV void ar_consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

static_assert(sizeof(ArItem) <= 64, "announced items");

// A CTA's piece of the line (kv_line.h), item by item.
template <class S>
struct ArWalk {
  const ArParams& p;
  const ArLine& line;
  const uint64_t* pre;   // the line before each sequence (shared memory)
  const int* rows;       // first new-token rows [batch + 1] and lengths [batch], for batches up to AR_KEPT
  ArPiece<S::TILE, S::ROWS, S::EXTRA> piece;

  NVFP4_DEV bool next(ArItem& g) {
    auto seq = [&](int b) {
      const bool kept = line.batch <= AR_KEPT;
      const int r0 = kept ? rows[b] : kv_row0(p.s, b);
      return ArSeq{r0, (kept ? rows[b + 1] : kv_row0(p.s, b + 1)) - r0, kept ? rows[line.batch + 1 + b] : kv_len(p.s, b)};
    };
    return piece.next(line, pre, seq, g);
  }
};

template <bool E4M3, int D, int NT>
__global__ void __launch_bounds__(ArShape<E4M3, D, NT>::THREADS, ArShape<E4M3, D, NT>::CTAS)
    attention_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                          const ArParams p) {
  using S = ArShape<E4M3, D, NT>;
  constexpr int WARPS = AR_WARPS;
  constexpr int ROWS = S::ROWS, KS = S::KS, BUFS = S::BUFS, OSTR = S::OSTR, TILE = S::TILE, CONSUMERS = WARPS * 32;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const int stages = p.stages;
  uint8_t* at = smem_raw + (base - raw) + stages * S::STAGE_BYTES;
  float* merge = reinterpret_cast<float*>(at);                     // [BUFS][ROWS][OSTR]
  at += BUFS * ROWS * OSTR * 4;
  uint2* qfrag = reinterpret_cast<uint2*>(at);                     // [AR_ITEMS][KS][NT][32]
  at += AR_ITEMS * S::QFRAGS * 8;
  ArItem* items = reinterpret_cast<ArItem*>(at);                   // [AR_ITEMS]
  at += AR_ITEMS * 64;
  uint64_t* bars = reinterpret_cast<uint64_t*>(at);
  float* row_mult = reinterpret_cast<float*>(bars + 2 * AR_MAX_STAGES + 2 * AR_ITEMS + 1);   // [AR_ITEMS][ROWS]
  int* row_pos = reinterpret_cast<int*>(row_mult + AR_ITEMS * ROWS);                     // [AR_ITEMS][ROWS]
  float* warp_m = reinterpret_cast<float*>(row_pos + AR_ITEMS * ROWS);                   // [WARPS][ROWS]
  float* warp_l = warp_m + WARPS * ROWS;
  unsigned* stage_ok = reinterpret_cast<unsigned*>(warp_l + WARPS * ROWS);               // which boxes hold pages
  unsigned* stage_cut = stage_ok + AR_MAX_STAGES;                                        // [2]: tokens that elements were taken out of
  volatile int* abort_flag = reinterpret_cast<volatile int*>(stage_cut + 2 * AR_MAX_STAGES);
  unsigned* last_flag = stage_cut + 2 * AR_MAX_STAGES + 1;
  uint64_t* pre = reinterpret_cast<uint64_t*>((reinterpret_cast<uintptr_t>(last_flag + 1) + 7u) & ~static_cast<uintptr_t>(7));   // [batch + 1]
  int* rows = reinterpret_cast<int*>(pre + p.s.batch + 1);                               // [2 batch + 1]
  const uint32_t bar0 = smem_addr(bars);
  auto full_bar = [&](int st) { return bar0 + 8u * st; };
  auto empty_bar = [&](int st) { return bar0 + 8u * (AR_MAX_STAGES + st); };
  auto item_full = [&](int i) { return bar0 + 8u * (2 * AR_MAX_STAGES + i); };
  auto item_empty = [&](int i) { return bar0 + 8u * (2 * AR_MAX_STAGES + AR_ITEMS + i); };
  const uint32_t check_bar = bar0 + 8u * (2 * AR_MAX_STAGES + 2 * AR_ITEMS);
  auto stage_k = [&](int st) { return base + st * S::STAGE_BYTES; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int st = 0; st < stages; ++st) {
      mbar_init(full_bar(st), 1);
      mbar_init(empty_bar(st), WARPS);
    }
    for (int i = 0; i < AR_ITEMS; ++i) {
      mbar_init(item_full(i), 1);
      mbar_init(item_empty(i), WARPS);
    }
    mbar_init(check_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v) : "memory");
  }
  pdl_launch_dependents();
  pdl_wait();
  // the line of work: prefix sums over the sequences
  const ArLine line = {p.s.batch, p.heads, p.group, p.window, p.sinks, static_cast<int64_t>(p.s.max_pages) * p.page_size};
  for (int b = threadIdx.x; b < p.s.batch; b += S::THREADS) {
    const int r0 = kv_row0(p.s, b), r1 = kv_row0(p.s, b + 1), len = kv_len(p.s, b);
    pre[b + 1] = ar_seq_units<S::TILE, S::ROWS, S::EXTRA>(line, {r0, r1 - r0, len});
    if (p.s.batch <= AR_KEPT) {
      rows[b] = r0;
      rows[b + 1] = r1;   // the next thread writes the same
      rows[p.s.batch + 1 + b] = len;
    }
  }
  __syncthreads();
  if (warp == 0) {
    uint64_t run = 0;
    for (int b0 = 0; b0 < p.s.batch; b0 += 32) {
      uint64_t x = b0 + lane < p.s.batch ? pre[b0 + lane + 1] : 0u;
      if (__any_sync(AR_ALL, (x >> 26) != 0)) {
#pragma unroll 1
        for (int d = 1; d < 32; d <<= 1) {
          const uint64_t y = __shfl_up_sync(AR_ALL, x, d);
          if (lane >= d) x += y;
        }
      } else {
        unsigned w = static_cast<unsigned>(x);   // 32 of them fit 32 bits
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const unsigned y = __shfl_up_sync(AR_ALL, w, d);
          if (lane >= d) w += y;
        }
        x = w;
      }
      if (b0 + lane < p.s.batch) pre[b0 + lane + 1] = run + x;
      run += __shfl_sync(AR_ALL, x, 31);
    }
    if (lane == 0) pre[0] = 0;
  }
  __syncthreads();
  ArWalk<S> walk{p, line, pre, rows, {line, pre[p.s.batch], gridDim.x, blockIdx.x}};
  if (walk.piece.u >= walk.piece.end) return;
  ArItem g;
  const int box = p.page_size < TILE ? p.page_size : TILE;   // tokens of one copied box
  const int box_log2 = 31 - __clz(box), boxes = TILE >> box_log2, boxes_log2 = 31 - __clz(boxes);

  if (warp == WARPS) {
    // ------------------------------------------------------------ producer
    int st = 0, par = 1, used = 0;   // ring slot, parity of its last release, slots used
    int checks = 0;                  // tiles looked at
    bool ok = true;
    while (ok && walk.next(g)) {
      const int32_t* row = p.s.table + static_cast<int64_t>(g.b) * p.s.table_stride;
      // page ids of 32 boxes at a time, one per lane
      int page = -1;
      for (int i = g.i0; i < g.i1; ++i) {
        const int k = (i - g.i0) << boxes_log2;   // this tile's first box since the piece began
        if ((k & 31) == 0) {
          const int j = g.tiles.tile(min(i + (lane >> boxes_log2), g.i1 - 1)) * TILE + ((lane & (boxes - 1)) << box_log2);
          const int e = j >> p.page_log2;
          page = j < g.key_end && e < p.s.max_pages ? row[e] : -1;
          if (page < 0 || page >= p.pages) page = -1;
        }
        if (used >= stages) ok = __all_sync(AR_ALL, mbar_wait_bounded(empty_bar(st), par, abort_flag, p.status));
        if (!ok) break;
        const int mine = __shfl_sync(AR_ALL, page, (k & 31) + (lane & (boxes - 1)));
        const unsigned there = __ballot_sync(AR_ALL, lane < boxes && mine >= 0);
        // tokens that later rows of the item see and earlier ones do not, and the
        // other way round at a window's edge: the tile is looked at before the
        // consumers get it
        const int j0 = g.tiles.tile(i) * TILE;
        const KvPartly part = kv_partly(g.p0, g.p1, p.window, p.sinks);
        const bool mixed = part.meets(j0, TILE);
        const uint32_t landed = mixed ? check_bar : full_bar(st);
        if (lane == 0) {
          stage_ok[st] = there;
          stage_cut[2 * st] = stage_cut[2 * st + 1] = 0;
          mbar_arrive_expect_tx(landed, S::STAGE_BYTES);
        }
        __syncwarp();
        if (lane < boxes) {
          const int j = j0 + (lane << box_log2);
          // a page that is not there: a box past the pool's end, which the copy fills with zeros
          const int64_t block = mine >= 0 ? static_cast<int64_t>(mine) * p.heads + g.h : p.pages * p.heads;
          const int y = j & (p.page_size - 1);
          const uint32_t dst = stage_k(st) + (lane << box_log2) * S::ROW_BYTES;
          tma_load_4d(dst, &map_k, 0, y, 0, static_cast<int>(block), landed);
          tma_load_4d(dst + S::MAT_BYTES, &map_v, 0, y, 0, static_cast<int>(block), landed);
        }
        if (mixed) {
          // value elements that are not finite are taken out and added at the
          // end to the rows that see them (kv.cuh): a bit for each of the up to
          // 31 tokens from part.a0 on, and of those from part.b0 on, that had any
          ok = __all_sync(AR_ALL, mbar_wait_bounded(check_bar, checks++ & 1, abort_flag, p.status));
          if (!ok) break;
          constexpr int CHUNKS = S::ROW_BYTES / 16;
          unsigned cut_a = 0, cut_b = 0;
#pragma unroll 2
          for (int u = lane; u < TILE * CHUNKS; u += 32) {
            const int row = u / CHUNKS, chunk = u % CHUNKS, jj = j0 + row;
            if (!((jj >= part.a0 && jj < part.a1) || (jj >= part.b0 && jj < part.b1))) continue;
            const int r = row & (box - 1), half = S::SEG == 128 ? chunk >> 3 : 0;
            const int c16 = S::SEG == 128 ? (chunk & 7) ^ (r & 7) : chunk ^ ((r >> 1) & 3);
            const uint32_t addr = stage_k(st) + S::MAT_BYTES + (row - r) * S::ROW_BYTES + ((half << box_log2) + r) * S::SEG + (c16 << 4);
            const uint4 w = lds128(addr);
            uint32_t y[4] = {w.x, w.y, w.z, w.w}, any = 0;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              // the top bit of each element whose exponent (E4M3: code) is all ones
              const uint32_t top = E4M3 ? ((y[z] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u
                                        : ((y[z] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
              any |= top;
              y[z] &= ~(E4M3 ? (top >> 7) * 0xFFu : (top >> 15) * 0xFFFFu);
            }
            if (!any) continue;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the slot's next copy comes after
            if (jj >= part.a0)
              cut_a |= 1u << (jj - part.a0);
            else
              cut_b |= 1u << (jj - part.b0);
          }
          cut_a = __reduce_or_sync(AR_ALL, cut_a);
          cut_b = __reduce_or_sync(AR_ALL, cut_b);
          if (lane == 0) {
            stage_cut[2 * st] = cut_a;   // read with the slot, before the slot is released
            stage_cut[2 * st + 1] = cut_b;
            mbar_arrive(full_bar(st));
          }
        }
        ++used;
        if (++st == stages) {
          st = 0;
          par ^= 1;
        }
      }
    }
    if (!ok) {
      // the copies in flight land before this CTA's shared memory goes
      for (int k = used > stages ? used - stages : 0; k < used; ++k)
        mbar_wait_bounded(full_bar(k % stages), (k / stages) & 1, nullptr, p.status);
    }
    return;
  }

  if (warp == WARPS + 1) {
    // ------------------------------------------ items and their query rows
    const int quad = lane & 3, oct = lane >> 2;
    for (int k = 0;; ++k) {
      const int buf = k % AR_ITEMS;
      const bool more = walk.next(g);
      uint32_t w[NT][KS][2];
      int tok[NT];
      if (more) {
        // fragments (B of m16n8k16: k = d, n = row), requested before the wait
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = g.r0 + nt * 8 + oct;
          const bool live = nt * 8 + oct < g.n_rows;
          const int i = r / p.group;
          tok[nt] = live ? i : -1;
          const uint16_t* src = p.q + static_cast<int64_t>(g.row0 + i) * p.q_stride +
                                (static_cast<int64_t>(g.h) * p.group + (r - i * p.group)) * D;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            if (E4M3) {
              // an 8-bit ldmatrix hands a lane four consecutive d's: the same order here
              const uint2 x = live ? *reinterpret_cast<const uint2*>(src + 16 * ks + 4 * quad) : make_uint2(0u, 0u);
              w[nt][ks][0] = x.x;
              w[nt][ks][1] = x.y;
            } else {
              w[nt][ks][0] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * quad) : 0u;
              w[nt][ks][1] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 8 + 2 * quad) : 0u;
            }
          }
        }
      }
      if (k >= AR_ITEMS &&
          !__all_sync(AR_ALL, mbar_wait_bounded(item_empty(buf), ((k / AR_ITEMS) - 1) & 1, abort_flag, p.status)))
        return;
      if (more) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float mult = p.scale;
          if (E4M3) {
            float amax = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                amax = fmaxf(amax, fmaxf(fabsf(bf16_bits_to_f32(w[nt][ks][c] & 0xFFFFu)), fabsf(bf16_bits_to_f32(w[nt][ks][c] >> 16))));
            amax = fmaxf(amax, __shfl_xor_sync(AR_ALL, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(AR_ALL, amax, 2));
            // 2^-e brings amax into [2^14, 2^15)
            const int e = amax > 0.0f && amax < INFINITY ? ilogbf(amax) - 14 : 0;
            // in two factors: 2^-e alone may lie outside fp32
            const int e1 = min(max(-e, -100), 100);
            const float down = scalbnf(1.0f, e1), rest = scalbnf(1.0f, -e - e1);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                w[nt][ks][c] = f32x2_to_f16x2(bf16_bits_to_f32(w[nt][ks][c] & 0xFFFFu) * down * rest,
                                              bf16_bits_to_f32(w[nt][ks][c] >> 16) * down * rest);
            mult = p.scale * p.k_scale[g.h] * scalbnf(1.0f, e);
          }
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            qfrag[buf * S::QFRAGS + (ks * NT + nt) * 32 + lane] = make_uint2(w[nt][ks][0], w[nt][ks][1]);
          if (quad == 0) {
            row_mult[buf * ROWS + nt * 8 + oct] = mult;
            // the position, from the item's first row's
            row_pos[buf * ROWS + nt * 8 + oct] = tok[nt] >= 0 ? g.p0 + (tok[nt] - g.r0 / p.group) : -1;
          }
        }
      } else {
        g.done = 1;
      }
      if (lane == 0) items[buf] = g;
      __syncwarp();
      if (lane == 0) mbar_arrive(item_full(buf));
      if (!more) return;
    }
  }

  // -------------------------------------------------------------- consumers
  const int quad = lane & 3, oct = lane >> 2;
  const int tok0 = warp * 16;                                  // this warp's tokens of a tile
  const int my_box = tok0 >> box_log2;
  // byte offsets of this lane's ldmatrix rows inside a tile
  const int k_row = (tok0 & (box - 1)) + (lane & 15);
  const int v_row = (tok0 & (box - 1)) + (lane & 7) +
                    (E4M3 ? ((lane >> 3) & 1) * 8 : ((lane >> 4) & 1) * 8);
  const uint32_t box_off = static_cast<uint32_t>((my_box << box_log2) * S::ROW_BYTES);
  auto swz = [&](int row, int chunk) {                         // 16-byte chunk of a box row
    const int half = S::SEG == 128 ? chunk >> 3 : 0;
    const int c = S::SEG == 128 ? (chunk & 7) ^ (row & 7) : chunk ^ ((row >> 1) & 3);
    return static_cast<uint32_t>(((half << box_log2) + row) * S::SEG + (c << 4));
  };

  int st = 0, par = 0;                                         // ring slot, parity of its next filling
  bool ok = true;
  float o[KS][NT][4];
  float m[NT][2], l[NT][2];
  for (int k = 0;; ++k) {
    const int buf = k % AR_ITEMS;
    // a wait that gives up ends every consumer here: they agree on `ok` at the end of each item
    if (!ar_all<CONSUMERS>(ok && mbar_wait_bounded(item_full(buf), (k / AR_ITEMS) & 1, abort_flag, p.status))) return;
    g = items[buf];
    if (g.done) return;
    const uint2* qf = qfrag + buf * S::QFRAGS + lane;
    uint2 qreg[S::Q_REGS ? KS : 1][S::Q_REGS ? NT : 1];
    if constexpr (S::Q_REGS) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) qreg[ks][nt] = qf[(ks * NT + nt) * 32];
    }
    auto q_at = [&](int ks, int nt) {
      if constexpr (S::Q_REGS)
        return qreg[ks][nt];
      else
        return qf[(ks * NT + nt) * 32];
    };
    float mult[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mult[nt][c] = row_mult[buf * ROWS + nt * 8 + 2 * quad + c];
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.0f;
      }
#pragma unroll
    for (int mt = 0; mt < KS; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[mt][nt][c] = 0.0f;

    unsigned cut_a = 0, cut_b = 0;   // tokens that elements were taken out of: every warp reads every tile's words, so all agree
    for (int i = g.i0; i < g.i1; ++i) {
      if (ok) ok = __all_sync(AR_ALL, mbar_wait_bounded(full_bar(st), par, abort_flag, p.status));
      if (!ok) break;
      const int j0 = g.tiles.tile(i) * TILE;                     // the tile's first position
      const bool box_ok = (stage_ok[st] >> my_box) & 1u;
      const uint32_t kb = stage_k(st) + box_off, vb = kb + S::MAT_BYTES;
      // S^T = K Q^T
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[nt][c] = 0.0f;
      float s2[NT][4];   // (two tiles leave room for a second chain of products)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s2[nt][c] = 0.0f;
      if constexpr (E4M3) {
#pragma unroll
        for (int k2 = 0; k2 < KS / 2; ++k2) {
          uint32_t r[4];
          ldsm_x4(kb + swz(k_row, 2 * k2 + (lane >> 4)), r);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t a[4];
            e4m3x4_to_f16x2(r[2 * hf], a[0], a[2]);
            e4m3x4_to_f16x2(r[2 * hf + 1], a[1], a[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16_16816(hf && NT == 2 ? s2[nt] : s[nt], a, q_at(2 * k2 + hf, nt).x, q_at(2 * k2 + hf, nt).y);
          }
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t a[4];
          ldsm_x4(kb + swz(k_row, 2 * ks + (lane >> 4)), a);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_bf16_16816((ks & 1) && NT == 2 ? s2[nt] : s[nt], a, q_at(ks, nt).x, q_at(ks, nt).y);
        }
      }
      // scores in powers of two; masked ones replaced
      const bool all_seen = stage_ok[st] == (1u << boxes) - 1u && j0 + TILE - 1 <= g.p0 &&
                            j0 + TILE <= g.key_end &&
                            (p.window <= 0 || g.p1 - j0 < p.window || j0 + TILE <= p.sinks);
      uint32_t keep[2] = {AR_ALL, AR_ALL};                     // value rows of tokens 2 quad, +1 (and + 8)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[nt][c] = (s[nt][c] + s2[nt][c]) * mult[nt][c & 1];
      if (!all_seen) {   // (a tile that the producer looked at is one of these)
        cut_a |= stage_cut[2 * st];
        cut_b |= stage_cut[2 * st + 1];
        auto none_sees = [&](int j) {
          return !box_ok || j > g.p1 || j >= g.key_end || (p.window > 0 && j >= p.sinks && g.p0 - j >= p.window);
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int j = j0 + tok0 + oct + (c >> 1) * 8;
            const int at_pos = row_pos[buf * ROWS + nt * 8 + 2 * quad + (c & 1)];
            const bool sees = box_ok && j <= at_pos && j < g.key_end &&
                              (p.window <= 0 || at_pos - j < p.window || j < p.sinks);
            if (!sees) s[nt][c] = -INFINITY;
          }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int j = j0 + tok0 + 8 * hf + 2 * quad;
          keep[hf] = (none_sees(j) ? 0u : 0xFFFFu) | (none_sees(j + 1) ? 0u : 0xFFFF0000u);
        }
      }
      // online softmax over this warp's 16 tokens
      uint32_t hi[NT][2], lo[NT][2];
      float alpha[NT][2];
      bool moved = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(s[nt][c], s[nt][c + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(AR_ALL, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(AR_ALL, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(AR_ALL, mx, 16));
          // m moves, and o with it, only where p would exceed 2^SLACK
          const bool grows = mx - m[nt][c] > KvWeights<E4M3>::SLACK;
          alpha[nt][c] = grows ? exp2_approx(m[nt][c] - mx) : 1.0f;
          moved = moved || grows;
          if (grows) m[nt][c] = mx;
          const float use = (m[nt][c] == -INFINITY ? 0.0f : m[nt][c]) - KvWeights<E4M3>::LIFT;
          s[nt][c] = exp2_approx(s[nt][c] - use);
          s[nt][c + 2] = exp2_approx(s[nt][c + 2] - use);
          l[nt][c] = l[nt][c] * alpha[nt][c] + (s[nt][c] + s[nt][c + 2]);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float a = s[nt][2 * hf], b = s[nt][2 * hf + 1];
          if (E4M3) {
            hi[nt][hf] = movmatrix_t(kv_weights_f16x2(a, b));
          } else {
            const uint32_t w = f32x2_to_bf16x2(a, b);
            hi[nt][hf] = movmatrix_t(w);
            lo[nt][hf] = movmatrix_t(f32x2_to_bf16x2(a - bf16_bits_to_f32(w & 0xFFFFu), b - __uint_as_float(w & 0xFFFF0000u)));
          }
        }
      }
      if (__any_sync(AR_ALL, moved)) {
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[mt][nt][c] *= alpha[nt][c & 1];
      }
      // O^T += V^T P^T
      if constexpr (E4M3) {
#pragma unroll
        for (int m2 = 0; m2 < KS / 2; ++m2) {
          uint32_t r[4];
          ldsm_x4_t(vb + swz(v_row, 2 * m2 + (lane >> 4)), r);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            // a word holds two tokens' codes of two d's: (token, d), (token, d + 1), (token + 1, d), ...
            uint32_t a[4];
            r[2 * hf] &= keep[0];
            r[2 * hf + 1] &= keep[1];
            e4m3x4_to_f16x2(__byte_perm(r[2 * hf], 0, 0x3120), a[0], a[1]);
            e4m3x4_to_f16x2(__byte_perm(r[2 * hf + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[2 * m2 + hf][nt], a, hi[nt][0], hi[nt][1]);
          }
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          uint32_t a[4];
          ldsm_x4_t(vb + swz(v_row, 2 * mt + ((lane >> 3) & 1)), a);
          a[0] &= keep[0];
          a[1] &= keep[0];
          a[2] &= keep[1];
          a[3] &= keep[1];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(o[mt][nt], a, hi[nt][0], hi[nt][1]);
            mma_bf16_16816(o[mt][nt], a, lo[nt][0], lo[nt][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(st));
      if (++st == stages) {
        st = 0;
        par ^= 1;
      }
    }

    // the item's rows and fragments have been read; the warps' parts meet
    __syncwarp();
    if (lane == 0) mbar_arrive(item_empty(buf));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[nt][c] += __shfl_xor_sync(AR_ALL, l[nt][c], 4);
        l[nt][c] += __shfl_xor_sync(AR_ALL, l[nt][c], 8);
        l[nt][c] += __shfl_xor_sync(AR_ALL, l[nt][c], 16);
        if (oct == 0) {
          warp_m[warp * ROWS + nt * 8 + 2 * quad + c] = m[nt][c];
          warp_l[warp * ROWS + nt * 8 + 2 * quad + c] = l[nt][c];
        }
      }
    ok = ar_all<CONSUMERS>(ok);
    if (!ok) continue;   // a wait gave up: nothing more is written
    auto row_max = [&](int r) {
      float x = warp_m[r];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) x = fmaxf(x, warp_m[w * ROWS + r]);
      return x;
    };
    float f[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float x = row_max(nt * 8 + 2 * quad + c);
        f[nt][c] = exp2_approx(m[nt][c] - (x == -INFINITY ? 0.0f : x));
      }
    constexpr int TURNS = WARPS / BUFS;
#pragma unroll 1
    for (int turn = 0; turn < TURNS; ++turn) {
      if (warp / BUFS == turn) {
        float* mbuf = merge + (warp % BUFS) * ROWS * OSTR;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int d = 16 * mt + (E4M3 ? 2 * oct + (c >> 1) : oct + 8 * (c >> 1));
              float* x = mbuf + (nt * 8 + 2 * quad + (c & 1)) * OSTR + d;
              const float y = o[mt][nt][c] * f[nt][c & 1];
              *x = turn == 0 ? y : *x + y;
            }
      }
      ar_consumer_sync<CONSUMERS>();
    }
    auto merged = [&](int r, int d) {
      float4 x = *reinterpret_cast<const float4*>(merge + r * OSTR + d);
#pragma unroll
      for (int w = 1; w < BUFS; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(merge + (w * ROWS + r) * OSTR + d);
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
      }
      if (cut_a | cut_b) {
        // what was taken out of the values that this row sees, from the pool itself
        const int pos = g.p0 + ((g.r0 + r) / p.group - g.r0 / p.group);
        const int32_t* row = p.s.table + static_cast<int64_t>(g.b) * p.s.table_stride;
        const KvPartly part = kv_partly(g.p0, g.p1, p.window, p.sinks);
#pragma unroll 1
        for (uint64_t bits = cut_a | (static_cast<uint64_t>(cut_b) << 32); bits; bits &= bits - 1) {
          const int n = __ffsll(static_cast<long long>(bits)) - 1;
          const int j = n < 32 ? part.a0 + n : part.b0 + (n - 32);
          if (!kv_sees(pos, j, p.window, p.sinks)) continue;
          const int64_t at = ((static_cast<int64_t>(row[j >> p.page_log2]) * p.heads + g.h) * p.page_size + (j & (p.page_size - 1))) * D + d;
          const float4 v = kv_not_finite<E4M3>(p.v, at);
          x = make_float4(x.x + v.x, x.y + v.y, x.z + v.z, x.w + v.w);
        }
      }
      return x;
    };
    auto row_sum = [&](int r, float mx) {
      const float use = mx == -INFINITY ? 0.0f : mx;
      float x = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) x += warp_l[w * ROWS + r] * exp2_approx(warp_m[w * ROWS + r] - use);
      return x;
    };
    const float v_mult = E4M3 ? p.v_scale[g.h] : 1.0f;
    auto store = [&](int r, int d, float4 x, float sum) {
      const float inv = sum > 0.0f ? v_mult / sum : (sum == 0.0f ? 0.0f : sum);   // a NaN stays one
      const int i = (g.r0 + r) / p.group;
      const int64_t head = static_cast<int64_t>(g.h) * p.group + (g.r0 + r - i * p.group);
      uint16_t* dst = p.out + (static_cast<int64_t>(g.row0 + i) * p.heads * p.group + head) * D + d;
      *reinterpret_cast<uint2*>(dst) = make_uint2(f32x2_to_bf16x2(x.x * inv, x.y * inv), f32x2_to_bf16x2(x.z * inv, x.w * inv));
    };
    const unsigned first_cta = g.first_cta, last_cta = g.last_cta;
    if (first_cta == last_cta) {
      for (int x = threadIdx.x; x < g.n_rows * (D / 4); x += CONSUMERS) {
        const int r = x / (D / 4), d = (x % (D / 4)) * 4;
        store(r, d, merged(r, d), row_sum(r, row_max(r)));
      }
      continue;
    }
    // this CTA's part, then the join by the last one to arrive
    auto part = [&](unsigned cta) {
      return p.part + (static_cast<int64_t>(cta) * 2 + (cta == first_cta ? 1 : 0)) * (ROWS * (D + 2));
    };
    float* mine = part(blockIdx.x);
    for (int x = threadIdx.x; x < g.n_rows * (D / 4); x += CONSUMERS) {
      const int r = x / (D / 4), d = (x % (D / 4)) * 4;
      __stcg(reinterpret_cast<float4*>(mine + r * D + d), merged(r, d));
    }
    for (int r = threadIdx.x; r < g.n_rows; r += CONSUMERS) {
      const float mx = row_max(r);
      __stcg(reinterpret_cast<float2*>(mine + ROWS * D + 2 * r), make_float2(mx, row_sum(r, mx)));
    }
    ar_consumer_sync<CONSUMERS>();   // every warp's share is written: thread 0's release below covers it
    if (threadIdx.x == 0) {
      unsigned before;
      asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.arrived + first_cta) : "memory");
      const bool last = before == last_cta - first_cta;
      if (last) p.arrived[first_cta] = 0;    // ready for the next call
      *last_flag = last;
    }
    ar_consumer_sync<CONSUMERS>();
    if (*last_flag) {
      // each row's maximum over the parts: a thread takes every STEP-th part of
      // a row, then the row's threads meet in shared memory
      constexpr int STEP = CONSUMERS / ROWS;
      const int n_parts = static_cast<int>(last_cta - first_cta) + 1;
      {
        const int r = threadIdx.x % ROWS;
        float mx = -INFINITY;
        if (r < g.n_rows)
#pragma unroll 4
          for (int c = threadIdx.x / ROWS; c < n_parts; c += STEP)
            mx = fmaxf(mx, __ldcg(part(first_cta + c) + ROWS * D + 2 * r));
        merge[threadIdx.x] = mx;
      }
      ar_consumer_sync<CONSUMERS>();
      for (int x = threadIdx.x; x < g.n_rows * (D / 4); x += CONSUMERS) {
        const int r = x / (D / 4), d = (x % (D / 4)) * 4;
        float mx = merge[r];
#pragma unroll
        for (int c = 1; c < STEP; ++c) mx = fmaxf(mx, merge[c * ROWS + r]);
        const float use = mx == -INFINITY ? 0.0f : mx;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float sum = 0.0f;
        // sixteen parts' loads in flight
        for (int c0 = 0; c0 < n_parts; c0 += 16) {
          float2 ml[16];
          float4 y[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float* src = part(first_cta + min(c0 + c, n_parts - 1));
            ml[c] = __ldcg(reinterpret_cast<const float2*>(src + ROWS * D + 2 * r));
            y[c] = __ldcg(reinterpret_cast<const float4*>(src + r * D + d));
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            if (c0 + c >= n_parts) continue;
            const float w = exp2_approx(ml[c].x - use);
            sum += ml[c].y * w;
            acc.x += y[c].x * w;
            acc.y += y[c].y * w;
            acc.z += y[c].z * w;
            acc.w += y[c].w * w;
          }
        }
        store(r, d, acc, sum);
      }
    }
  }
}

}  // namespace
}  // namespace nvfp4
