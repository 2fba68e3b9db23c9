// Attention of few new rows over a paged key-value cache, split over the
// cache's length and joined in the same launch.
//
// The mathematics. Row r (one query head at one new token) sees the positions
// V(r) of its mask; out_r = sum_j exp(x_rj - m_r) v_j / sum_j exp(x_rj - m_r)
// with x_rj = scale q_r.k_j and m_r = max x_rj. A pass over any part of V(r)
// keeps (m, l = sum exp(x - m), o = sum exp(x - m) v), and two parts join as
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
// pages shorter than 64 tokens give several boxes), four consumer warps take
// 16 tokens each with an online softmax of their own and meet at the end of an
// item.
//
// Roundings. Products are exact in fp32 sums. bf16 caches: q and k as they
// are; p is split into two bf16 halves (p = hi + lo to 2^-17), since one bf16
// would cost as much error as the output's own rounding and the second MMA
// costs no time here. E4M3 caches: k and v are exact in f16, q is scaled by a
// power of two into f16 (exact for elements above amax 2^-29), p is one f16
// (2^-12, a sixteenth of the output's rounding).
//
// Masked places: scores are replaced, not added to; a token no row of the item
// sees has its value row replaced by zeros (stale page contents may be NaN),
// and pages that are not there are filled with zeros by the copy engine
// (their boxes lie past the pool's last page).
#pragma once

#include "kv.cuh"

namespace nvfp4 {
namespace {

constexpr int AR_TILE = 64;                  // tokens of one tile
constexpr int AR_WARPS = 4;                  // consumer warps, 16 tokens of a tile each
constexpr int AR_THREADS = (AR_WARPS + 1) * 32;
constexpr int AR_RING_BYTES = 96 * 1024;     // two CTAs per SM
constexpr int AR_MAX_BATCH = 4096;
constexpr int AR_PAD = 4;                    // fp32 words between rows of the merge buffer: no bank conflicts
constexpr unsigned AR_ALL = 0xffffffffu;

template <bool E4M3, int D>
struct ArShape {
  static constexpr int ROW_BYTES = D * (E4M3 ? 1 : 2);
  static constexpr int SEG = ROW_BYTES >= 128 ? 128 : 64;       // bytes of a swizzled row of a box
  static constexpr int HALVES = ROW_BYTES / SEG;
  static constexpr int MAT_BYTES = AR_TILE * ROW_BYTES;          // K or V of a tile
  static constexpr int STAGE_BYTES = 2 * MAT_BYTES;
  static constexpr int STAGES = AR_RING_BYTES / STAGE_BYTES < 8 ? AR_RING_BYTES / STAGE_BYTES : 8;
  static constexpr int KS = D / 16;                              // 16-d steps
};

struct ArParams {
  KvSeqs s;
  const uint16_t* q;
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
  float* part;            // [CTAs][2][8 NT][D + 2]
  int min_tiles;          // least tiles of a CTA's piece
  int* status;
};

template <bool E4M3, int D, int NT>
constexpr int ar_smem_bytes(int batch) {
  using S = ArShape<E4M3, D>;
  const int merge = (NT <= 2 ? 2 : 1) * 8 * NT * (D + AR_PAD) * 4;
  const int qfrag = S::KS * NT * 32 * 8;
  const int small = 8 * NT * 4 * (2 + 2 * AR_WARPS);             // row positions, multipliers, each warp's m and l
  return 1024 + S::STAGES * S::STAGE_BYTES + merge + qfrag + small + 8 * (2 * S::STAGES + 1) + 4 * S::STAGES + 64 +
         4 * (batch + 2);
}

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

// AND of `pred` over the consumer warps.
NVFP4_DEV bool ar_all(bool pred) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(static_cast<uint32_t>(pred)), "n"(AR_WARPS * 32)
      : "memory");
  return out != 0;
}
NVFP4_DEV void ar_consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(AR_WARPS * 32) : "memory"); }

// A piece of the line of tiles that lies inside one item.
struct ArSeg {
  int b, h, rb;          // sequence, kv head, block of rows
  int n, len, row0;      // new tokens, length, first new-token row
  int i0, i1;            // its tiles
  int per_item;          // tiles of the whole item
  unsigned item_u0;      // where the item starts on the line
};

template <int NT>
struct ArWalk {
  const ArParams& p;
  const unsigned* pre;   // tiles of the sequences before (shared memory)
  unsigned u, end;

  NVFP4_DEV bool next(ArSeg& g) {
    if (u >= end) return false;
    int lo = 0, hi = p.s.batch;             // last b with pre[b] <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= u)
        lo = mid;
      else
        hi = mid;
    }
    g.b = lo;
    g.row0 = kv_row0(p.s, lo);
    g.n = kv_row0(p.s, lo + 1) - g.row0;
    g.len = kv_len(p.s, lo);
    const int blocks = (g.n * p.group + 8 * NT - 1) / (8 * NT);
    g.per_item = static_cast<int>((pre[lo + 1] - pre[lo]) / static_cast<unsigned>(blocks * p.heads));
    const unsigned in = u - pre[lo], item = in / static_cast<unsigned>(g.per_item);
    g.h = static_cast<int>(item) % p.heads;
    g.rb = static_cast<int>(item) / p.heads;
    g.i0 = static_cast<int>(in - item * static_cast<unsigned>(g.per_item));
    g.item_u0 = u - static_cast<unsigned>(g.i0);
    const unsigned left = end - u;
    g.i1 = left < static_cast<unsigned>(g.per_item - g.i0) ? g.i0 + static_cast<int>(left) : g.per_item;
    u += static_cast<unsigned>(g.i1 - g.i0);
    return true;
  }
};

// Tiles that each block of sequence b's rows is given (the most any sees, at least one).
template <int NT>
NVFP4_DEV unsigned ar_seq_tiles(const ArParams& p, int b) {
  const int n = kv_row0(p.s, b + 1) - kv_row0(p.s, b);
  if (n <= 0) return 0;
  const int len = kv_len(p.s, b);
  const int64_t cap = static_cast<int64_t>(p.s.max_pages) * p.page_size;
  const int key_end = static_cast<int>(cap < len ? cap : len);
  const int blocks = (n * p.group + 8 * NT - 1) / (8 * NT);
  const int span = (8 * NT - 1 + p.group - 1) / p.group;   // positions between a block's first and last row, at most
  int most;
  if (p.window > 0 && blocks > 1) {
    // a block whose rows lie as late as any: two more tiles than its widest range of positions can touch
    const int64_t st = (min(p.sinks, max(key_end, 0)) + AR_TILE - 1) / AR_TILE;
    const int64_t w = (static_cast<int64_t>(p.window) + span) / AR_TILE + 2;
    const int64_t all = (max(key_end, 0) + AR_TILE - 1) / AR_TILE;
    most = static_cast<int>(st + w < all ? st + w : all);
  } else {
    most = kv_tiles<AR_TILE>(len - n, len - 1, p.window, p.sinks, key_end).count;
  }
  return static_cast<unsigned>(max(most, 1)) * static_cast<unsigned>(blocks * p.heads);
}

template <bool E4M3, int D, int NT>
__global__ void __launch_bounds__(AR_THREADS, NT <= 2 ? 2 : 1)
    attention_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                          const ArParams p) {
  using S = ArShape<E4M3, D>;
  constexpr int ROWS = 8 * NT;
  constexpr int MERGE_BUFS = NT <= 2 ? 2 : 1;
  constexpr int OSTR = D + AR_PAD;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* at = smem_raw + (base - raw) + S::STAGES * S::STAGE_BYTES;
  float* merge = reinterpret_cast<float*>(at);                     // [bufs][ROWS][OSTR]
  at += MERGE_BUFS * ROWS * OSTR * 4;
  uint2* qfrag = reinterpret_cast<uint2*>(at);                     // [KS][NT][32]
  at += S::KS * NT * 32 * 8;
  float* row_mult = reinterpret_cast<float*>(at);                  // [ROWS]
  int* row_pos = reinterpret_cast<int*>(row_mult + ROWS);          // [ROWS]
  float* warp_m = reinterpret_cast<float*>(row_pos + ROWS);        // [AR_WARPS][ROWS]
  float* warp_l = warp_m + AR_WARPS * ROWS;
  at = reinterpret_cast<uint8_t*>(warp_l + AR_WARPS * ROWS);
  at = smem_raw + ((at - smem_raw + 7) & ~7);
  uint64_t* bars = reinterpret_cast<uint64_t*>(at);
  unsigned* stage_ok = reinterpret_cast<unsigned*>(bars + 2 * S::STAGES);   // which boxes hold pages
  volatile int* abort_flag = reinterpret_cast<volatile int*>(stage_ok + S::STAGES);
  unsigned* last_flag = stage_ok + S::STAGES + 1;
  unsigned* pre = last_flag + 1;                                   // [batch + 1]
  const uint32_t bar0 = smem_addr(bars);
  auto full_bar = [&](int st) { return bar0 + 8u * st; };
  auto empty_bar = [&](int st) { return bar0 + 8u * (S::STAGES + st); };
  auto stage_k = [&](int st) { return base + st * S::STAGE_BYTES; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int st = 0; st < S::STAGES; ++st) {
      mbar_init(full_bar(st), 1);
      mbar_init(empty_bar(st), AR_WARPS);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v) : "memory");
  }
  pdl_launch_dependents();
  pdl_wait();
  // the line of tiles: prefix sums over the sequences, by the first warp
  for (int b = threadIdx.x; b < p.s.batch; b += AR_THREADS) pre[b + 1] = ar_seq_tiles<NT>(p, b);
  __syncthreads();
  if (warp == 0) {
    unsigned run = 0;
    for (int b0 = 0; b0 < p.s.batch; b0 += 32) {
      unsigned x = b0 + lane < p.s.batch ? pre[b0 + lane + 1] : 0u;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned y = __shfl_up_sync(AR_ALL, x, d);
        if (lane >= d) x += y;
      }
      if (b0 + lane < p.s.batch) pre[b0 + lane + 1] = run + x;
      run += __shfl_sync(AR_ALL, x, 31);
    }
    if (lane == 0) pre[0] = 0;
  }
  __syncthreads();
  const unsigned total = pre[p.s.batch];
  unsigned per = (total + gridDim.x - 1) / gridDim.x;
  if (per < static_cast<unsigned>(p.min_tiles)) per = static_cast<unsigned>(p.min_tiles);
  const uint64_t u0 = static_cast<uint64_t>(blockIdx.x) * per;
  if (u0 >= total) return;
  ArWalk<NT> walk{p, pre, static_cast<unsigned>(u0), static_cast<unsigned>(u0 + per < total ? u0 + per : total)};
  ArSeg g;
  const int box = p.page_size < AR_TILE ? p.page_size : AR_TILE;   // tokens of one copied box
  const int boxes = AR_TILE / box;
  const int64_t cap = static_cast<int64_t>(p.s.max_pages) * p.page_size;

  if (warp == AR_WARPS) {
    // ------------------------------------------------------------ producer
    int it = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      const int key_end = static_cast<int>(cap < g.len ? cap : g.len);
      const int r0 = g.rb * ROWS, r1 = min(r0 + ROWS, g.n * p.group) - 1;
      const KvTiles tl = kv_tiles<AR_TILE>(g.len - g.n + r0 / p.group, g.len - g.n + r1 / p.group, p.window, p.sinks, key_end);
      const int i1 = min(g.i1, tl.count);
      const int32_t* row = p.s.table + static_cast<int64_t>(g.b) * p.s.table_stride;
      // page ids of 32 boxes at a time, one per lane
      const int boxes_log2 = boxes == 4 ? 2 : boxes - 1;
      int page = -1;
      for (int i = g.i0; i < i1; ++i, ++it) {
        const int k = (i - g.i0) << boxes_log2;   // this tile's first box since the piece began
        if ((k & 31) == 0) {
          const int j = tl.tile(min(i + (lane >> boxes_log2), i1 - 1)) * AR_TILE + (lane & (boxes - 1)) * box;
          const int e = j >> p.page_log2;
          page = j < key_end && e < p.s.max_pages ? row[e] : -1;
          if (page < 0 || page >= p.pages) page = -1;
        }
        const int st = it % S::STAGES;
        if (it >= S::STAGES)
          ok = __all_sync(AR_ALL, mbar_wait_bounded(empty_bar(st), ((it / S::STAGES) - 1) & 1, abort_flag, p.status));
        if (!ok) break;
        const int mine = __shfl_sync(AR_ALL, page, (k & 31) + (lane & (boxes - 1)));
        const unsigned there = __ballot_sync(AR_ALL, lane < boxes && mine >= 0);
        if (lane == 0) {
          stage_ok[st] = there;
          mbar_arrive_expect_tx(full_bar(st), S::STAGE_BYTES);
        }
        __syncwarp();
        if (lane < boxes) {
          const int j = tl.tile(i) * AR_TILE + lane * box;
          // a page that is not there: a box past the pool's end, which the copy fills with zeros
          const int64_t block = mine >= 0 ? static_cast<int64_t>(mine) * p.heads + g.h : p.pages * p.heads;
          const int y = j & (p.page_size - 1);
          const uint32_t dst = stage_k(st) + lane * box * S::ROW_BYTES;
          tma_load_4d(dst, &map_k, 0, y, 0, static_cast<int>(block), full_bar(st));
          tma_load_4d(dst + S::MAT_BYTES, &map_v, 0, y, 0, static_cast<int>(block), full_bar(st));
        }
      }
    }
    if (!ok) {
      // the copies in flight land before this CTA's shared memory goes
      for (int k = it > S::STAGES ? it - S::STAGES : 0; k < it; ++k)
        mbar_wait_bounded(full_bar(k % S::STAGES), (k / S::STAGES) & 1, nullptr, p.status);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int quad = lane & 3, oct = lane >> 2;
  const int tok0 = warp * 16;                                  // this warp's tokens of a tile
  const int my_box = tok0 / box;
  // byte offsets of this lane's ldmatrix rows inside a tile
  const int k_row = (tok0 & (box - 1)) + (lane & 15);
  const int v_row = (tok0 & (box - 1)) + (lane & 7) +
                    (E4M3 ? ((lane >> 3) & 1) * 8 : ((lane >> 4) & 1) * 8);
  const uint32_t box_off = static_cast<uint32_t>(my_box * box * S::ROW_BYTES);
  auto swz = [&](int row, int chunk) {                         // 16-byte chunk of a box row
    const int half = S::SEG == 128 ? chunk >> 3 : 0;
    const int c = S::SEG == 128 ? (chunk & 7) ^ (row & 7) : chunk ^ ((row >> 1) & 3);
    return static_cast<uint32_t>(half * box * S::SEG + row * S::SEG + (c << 4));
  };

  int it = 0;
  bool ok = true;
  float o[S::KS][NT][4];
  float m[NT][2], l[NT][2];
  while (walk.next(g)) {
    const int key_end = static_cast<int>(cap < g.len ? cap : g.len);
    const int r0 = g.rb * ROWS, n_rows = min(ROWS, g.n * p.group - r0);
    const int p0 = g.len - g.n + r0 / p.group, p1 = g.len - g.n + (r0 + n_rows - 1) / p.group;
    const KvTiles tl = kv_tiles<AR_TILE>(p0, p1, p.window, p.sinks, key_end);
    const int i1 = min(g.i1, tl.count);
    // query fragments (B of m16n8k16: k = d, n = row), one eight-row tile per warp
    if (warp < NT) {
      const int r = r0 + warp * 8 + oct;
      const bool live = warp * 8 + oct < n_rows;
      const int i = r / p.group;
      const uint16_t* src = p.q + static_cast<int64_t>(g.row0 + i) * p.q_stride +
                            (static_cast<int64_t>(g.h) * p.group + (r - i * p.group)) * D;
      uint32_t w[S::KS][2];
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) {
        if (E4M3) {
          // an 8-bit ldmatrix hands a lane four consecutive d's: the same order here
          const uint2 x = live ? *reinterpret_cast<const uint2*>(src + 16 * ks + 4 * quad) : make_uint2(0u, 0u);
          w[ks][0] = x.x;
          w[ks][1] = x.y;
        } else {
          w[ks][0] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * quad) : 0u;
          w[ks][1] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 8 + 2 * quad) : 0u;
        }
      }
      float mult = p.scale;
      if (E4M3) {
        float amax = 0.0f;
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            amax = fmaxf(amax, fmaxf(fabsf(bf16_bits_to_f32(w[ks][c] & 0xFFFFu)), fabsf(bf16_bits_to_f32(w[ks][c] >> 16))));
        amax = fmaxf(amax, __shfl_xor_sync(AR_ALL, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(AR_ALL, amax, 2));
        // 2^-e brings amax into [2^14, 2^15)
        const int e = amax > 0.0f && amax < INFINITY ? ilogbf(amax) - 14 : 0;
        // in two factors: 2^-e alone may lie outside fp32
        const int e1 = min(max(-e, -100), 100);
        const float down = scalbnf(1.0f, e1), rest = scalbnf(1.0f, -e - e1);
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            w[ks][c] = f32x2_to_f16x2(bf16_bits_to_f32(w[ks][c] & 0xFFFFu) * down * rest,
                                      bf16_bits_to_f32(w[ks][c] >> 16) * down * rest);
        mult = p.scale * p.k_scale[g.h] * scalbnf(1.0f, e);
      }
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) qfrag[(ks * NT + warp) * 32 + lane] = make_uint2(w[ks][0], w[ks][1]);
      if (quad == 0) {
        row_mult[warp * 8 + oct] = mult;
        row_pos[warp * 8 + oct] = live ? g.len - g.n + i : -1;
      }
    }
    ar_consumer_sync();
    uint2 qreg[NT <= 2 ? S::KS : 1][NT <= 2 ? NT : 1];
    if constexpr (NT <= 2) {
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) qreg[ks][nt] = qfrag[(ks * NT + nt) * 32 + lane];
    }
    float mult[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mult[nt][c] = row_mult[nt * 8 + 2 * quad + c];
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.0f;
      }
#pragma unroll
    for (int mt = 0; mt < S::KS; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[mt][nt][c] = 0.0f;

    for (int i = g.i0; i < i1; ++i, ++it) {
      const int st = it % S::STAGES;
      if (ok) ok = __all_sync(AR_ALL, mbar_wait_bounded(full_bar(st), (it / S::STAGES) & 1, abort_flag, p.status));
      if (!ok) continue;
      const int j0 = tl.tile(i) * AR_TILE;                     // the tile's first position
      const bool box_ok = (stage_ok[st] >> my_box) & 1u;
      const uint32_t kb = stage_k(st) + box_off, vb = kb + S::MAT_BYTES;
      // S^T = K Q^T
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[nt][c] = 0.0f;
      if constexpr (E4M3) {
#pragma unroll
        for (int k2 = 0; k2 < S::KS / 2; ++k2) {
          uint32_t r[4];
          ldsm_x4(kb + swz(k_row, 2 * k2 + (lane >> 4)), r);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t a[4] = {e4m3x2_to_f16x2(r[2 * hf] & 0xFFFFu), e4m3x2_to_f16x2(r[2 * hf + 1] & 0xFFFFu),
                                   e4m3x2_to_f16x2(r[2 * hf] >> 16), e4m3x2_to_f16x2(r[2 * hf + 1] >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 qb = NT <= 2 ? qreg[NT <= 2 ? 2 * k2 + hf : 0][NT <= 2 ? nt : 0]
                                       : qfrag[((2 * k2 + hf) * NT + nt) * 32 + lane];
              mma_f16_16816(s[nt], a, qb.x, qb.y);
            }
          }
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks) {
          uint32_t a[4];
          ldsm_x4(kb + swz(k_row, 2 * ks + (lane >> 4)), a);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 qb = NT <= 2 ? qreg[NT <= 2 ? ks : 0][NT <= 2 ? nt : 0] : qfrag[(ks * NT + nt) * 32 + lane];
            mma_bf16_16816(s[nt], a, qb.x, qb.y);
          }
        }
      }
      // scores in powers of two; masked ones replaced
      const bool all_seen = stage_ok[st] == (1u << boxes) - 1u && j0 + AR_TILE - 1 <= p0 &&
                            j0 + AR_TILE <= key_end &&
                            (p.window <= 0 || p1 - j0 < p.window || j0 + AR_TILE <= p.sinks);
      uint32_t keep[2] = {AR_ALL, AR_ALL};                     // value rows of tokens 2 quad, +1 (and + 8)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[nt][c] *= mult[nt][c & 1];
      if (!all_seen) {
        auto none_sees = [&](int j) {
          return !box_ok || j > p1 || j >= key_end || (p.window > 0 && j >= p.sinks && p0 - j >= p.window);
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int j = j0 + tok0 + oct + (c >> 1) * 8;
            const int pos = row_pos[nt * 8 + 2 * quad + (c & 1)];
            const bool sees = box_ok && j <= pos && j < key_end &&
                              (p.window <= 0 || pos - j < p.window || j < p.sinks);
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
          const float mn = fmaxf(m[nt][c], mx);
          const float use = mn == -INFINITY ? 0.0f : mn;
          alpha[nt][c] = exp2_approx(m[nt][c] - use);
          moved = moved || mn != m[nt][c];
          m[nt][c] = mn;
          s[nt][c] = exp2_approx(s[nt][c] - use);
          s[nt][c + 2] = exp2_approx(s[nt][c + 2] - use);
          l[nt][c] = l[nt][c] * alpha[nt][c] + (s[nt][c] + s[nt][c + 2]);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float a = s[nt][2 * hf], b = s[nt][2 * hf + 1];
          if (E4M3) {
            hi[nt][hf] = movmatrix_t(f32x2_to_f16x2(a, b));
          } else {
            const uint32_t w = f32x2_to_bf16x2(a, b);
            hi[nt][hf] = movmatrix_t(w);
            lo[nt][hf] = movmatrix_t(f32x2_to_bf16x2(a - bf16_bits_to_f32(w & 0xFFFFu), b - __uint_as_float(w & 0xFFFF0000u)));
          }
        }
      }
      if (__any_sync(AR_ALL, moved)) {
#pragma unroll
        for (int mt = 0; mt < S::KS; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[mt][nt][c] *= alpha[nt][c & 1];
      }
      // O^T += V^T P^T
      if constexpr (E4M3) {
#pragma unroll
        for (int m2 = 0; m2 < S::KS / 2; ++m2) {
          uint32_t r[4];
          ldsm_x4_t(vb + swz(v_row, 2 * m2 + (lane >> 4)), r);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t x = __byte_perm(r[2 * hf], 0, 0x3120), y = __byte_perm(r[2 * hf + 1], 0, 0x3120);
            const uint32_t a[4] = {e4m3x2_to_f16x2(x & 0xFFFFu) & keep[0], e4m3x2_to_f16x2(x >> 16) & keep[0],
                                   e4m3x2_to_f16x2(y & 0xFFFFu) & keep[1], e4m3x2_to_f16x2(y >> 16) & keep[1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[2 * m2 + hf][nt], a, hi[nt][0], hi[nt][1]);
          }
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < S::KS; ++mt) {
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
    }

    // the four warps' parts meet
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
    ar_consumer_sync();
    auto row_max = [&](int r) {
      float x = warp_m[r];
#pragma unroll
      for (int w = 1; w < AR_WARPS; ++w) x = fmaxf(x, warp_m[w * ROWS + r]);
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
    constexpr int TURNS = AR_WARPS / MERGE_BUFS;
#pragma unroll 1
    for (int turn = 0; turn < TURNS; ++turn) {
      if (warp / MERGE_BUFS == turn) {
        float* buf = merge + (warp % MERGE_BUFS) * ROWS * OSTR;
#pragma unroll
        for (int mt = 0; mt < S::KS; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int d = 16 * mt + (E4M3 ? 2 * oct + (c >> 1) : oct + 8 * (c >> 1));
              float* x = buf + (nt * 8 + 2 * quad + (c & 1)) * OSTR + d;
              const float y = o[mt][nt][c] * f[nt][c & 1];
              *x = turn == 0 ? y : *x + y;
            }
      }
      ar_consumer_sync();
    }
    auto merged = [&](int r, int d) {
      float4 x = *reinterpret_cast<const float4*>(merge + r * OSTR + d);
      if constexpr (MERGE_BUFS == 2) {
        const float4 y = *reinterpret_cast<const float4*>(merge + (ROWS + r) * OSTR + d);
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
      }
      return x;
    };
    auto row_sum = [&](int r, float mx) {
      const float use = mx == -INFINITY ? 0.0f : mx;
      float x = 0.0f;
#pragma unroll
      for (int w = 0; w < AR_WARPS; ++w) x += warp_l[w * ROWS + r] * exp2_approx(warp_m[w * ROWS + r] - use);
      return x;
    };
    const float v_mult = E4M3 ? p.v_scale[g.h] : 1.0f;
    auto store = [&](int r, int d, float4 x, float sum) {
      const float inv = sum > 0.0f ? v_mult / sum : (sum == 0.0f ? 0.0f : sum);   // a NaN stays one
      const int i = (r0 + r) / p.group;
      const int64_t head = static_cast<int64_t>(g.h) * p.group + (r0 + r - i * p.group);
      uint16_t* dst = p.out + (static_cast<int64_t>(g.row0 + i) * p.heads * p.group + head) * D + d;
      *reinterpret_cast<uint2*>(dst) = make_uint2(f32x2_to_bf16x2(x.x * inv, x.y * inv), f32x2_to_bf16x2(x.z * inv, x.w * inv));
    };
    const unsigned first_cta = g.item_u0 / per, last_cta = (g.item_u0 + static_cast<unsigned>(g.per_item) - 1u) / per;
    ok = ar_all(ok);
    if (!ok) continue;   // a wait gave up: nothing more is written
    if (first_cta == last_cta) {
      for (int x = threadIdx.x; x < n_rows * (D / 4); x += AR_WARPS * 32) {
        const int r = x / (D / 4), d = (x % (D / 4)) * 4;
        store(r, d, merged(r, d), row_sum(r, row_max(r)));
      }
      ar_consumer_sync();   // the merge buffers may be written again
      continue;
    }
    // this CTA's part, then the join by the last one to arrive
    auto part = [&](unsigned cta) {
      return p.part + (static_cast<int64_t>(cta) * 2 + (cta == first_cta ? 1 : 0)) * (ROWS * (D + 2));
    };
    float* mine = part(blockIdx.x);
    for (int x = threadIdx.x; x < n_rows * (D / 4); x += AR_WARPS * 32) {
      const int r = x / (D / 4), d = (x % (D / 4)) * 4;
      __stcg(reinterpret_cast<float4*>(mine + r * D + d), merged(r, d));
    }
    for (int r = threadIdx.x; r < n_rows; r += AR_WARPS * 32) {
      const float mx = row_max(r);
      __stcg(reinterpret_cast<float2*>(mine + ROWS * D + 2 * r), make_float2(mx, row_sum(r, mx)));
    }
    fence_acq_rel_gpu();
    ar_consumer_sync();
    if (threadIdx.x == 0) {
      const unsigned n_parts = last_cta - first_cta + 1;
      const unsigned before = atomicAdd(p.arrived + first_cta, 1u);
      *last_flag = before + 1 == n_parts;
      if (before + 1 == n_parts) p.arrived[first_cta] = 0;    // ready for the next call
      fence_acq_rel_gpu();
    }
    ar_consumer_sync();
    if (*last_flag) {
      fence_acq_rel_gpu();
      for (int x = threadIdx.x; x < n_rows * (D / 4); x += AR_WARPS * 32) {
        const int r = x / (D / 4), d = (x % (D / 4)) * 4;
        float mx = -INFINITY;
        for (unsigned c = first_cta; c <= last_cta; ++c)
          mx = fmaxf(mx, __ldcg(part(c) + ROWS * D + 2 * r));
        const float use = mx == -INFINITY ? 0.0f : mx;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float sum = 0.0f;
#pragma unroll 4
        for (unsigned c = first_cta; c <= last_cta; ++c) {
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(part(c) + ROWS * D + 2 * r));
          const float4 y = __ldcg(reinterpret_cast<const float4*>(part(c) + r * D + d));
          const float w = exp2_approx(ml.x - use);
          sum += ml.y * w;
          acc.x += y.x * w;
          acc.y += y.y * w;
          acc.z += y.z * w;
          acc.w += y.w * w;
        }
        store(r, d, acc, sum);
      }
    }
    ar_consumer_sync();   // the merge buffers and the flag may be written again
  }
}

}  // namespace
}  // namespace nvfp4
