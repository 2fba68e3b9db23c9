// How the token attention kernel's work is cut: plain arithmetic on the call's
// sizes, the same on the device and on the host (any C++17 compiler).
//
// The (sequence, block of rows, kv head) items, each of as many tiles of
// positions as its rows see and EXTRA more, lie one after another on a line,
// which is cut into equal pieces, one per CTA. The line is counted in 64 bits:
// two prompts of 131,072 tokens in blocks of eight rows are 2^32 long.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define NVFP4_HD __host__ __device__ __forceinline__
#else
#define NVFP4_HD inline
#endif

namespace nvfp4 {

template <class T>
NVFP4_HD T least(T a, T b) {
  return a < b ? a : b;
}
template <class T>
NVFP4_HD T most_of(T a, T b) {
  return a > b ? a : b;
}

// The tiles that a block of rows sees: [0, st) (sinks) and [w0, end).
struct KvTiles {
  int st, w0, count;
  NVFP4_HD int tile(int i) const { return i < st ? i : w0 + (i - st); }
};

// Tiles of the rows at positions p0..p1 (p1 < 0: none).
template <int TILE>
NVFP4_HD KvTiles kv_tiles(int p0, int p1, int window, int sinks, int key_end) {
  KvTiles t;
  const int end = (least(p1 + 1, key_end) + TILE - 1) / TILE;   // one past the last
  t.st = 0;
  t.w0 = 0;
  if (window > 0) {
    const int lo = p0 - window + 1;                                  // first position in a window
    const int w0 = lo > 0 ? lo / TILE : 0;
    const int st = least((least(sinks, key_end) + TILE - 1) / TILE, end);
    if (w0 > st) {
      t.st = st;
      t.w0 = w0;
    }
  }
  t.count = end > t.w0 ? t.st + end - t.w0 : t.st;
  if (end <= 0) t.count = 0;
  return t;
}

// The positions that some of the rows at positions p0..p1 see and others do not:
// [a0, a1), seen by the later rows only, and [b0, b1), which the later rows'
// windows have left behind. Either may be empty; neither holds more than p1 - p0.
struct KvPartly {
  int a0, a1, b0, b1;
  NVFP4_HD bool meets(int j0, int tile) const {   // whether the tile at j0 has any
    return most_of(a0, j0) < least(a1, j0 + tile) || most_of(b0, j0) < least(b1, j0 + tile);
  }
};
NVFP4_HD KvPartly kv_partly(int p0, int p1, int window, int sinks) {
  KvPartly x = {p0 + 1, p1 + 1, 0, 0};
  if (window > 0) {
    x.b0 = most_of(p0 - window + 1, sinks);
    x.b1 = least(p1 - window, p0) + 1;
  }
  return x;
}

// What the line depends on beside the sequences.
struct ArLine {
  int batch, heads, group;   // sequences, kv heads, query heads of each
  int window, sinks;
  int64_t cap;               // positions that a table row has pages for
};

// A sequence: its first new-token row, new tokens (below zero: none), length.
// Rows times query heads fit 31 bits (the call's entry sees to that).
struct ArSeq {
  int row0, n, len;
};

// A piece of the line that lies inside one item.
struct ArItem {
  int done;
  int h;                  // kv head
  int r0, n_rows;         // rows of the sequence's (token, head) pairs
  int row0;               // the sequence's first new-token row
  int p0, p1;             // positions of the first and the last row
  int key_end;            // positions at or past it hold nothing
  KvTiles tiles;
  int i0, i1;             // the piece's tiles
  int b;                  // sequence
  unsigned first_cta, last_cta;   // CTAs that share the item
};

// Length on the line of all items of a sequence: each block of rows is given
// the most tiles that any sees, and EXTRA more that stand for what an item costs
// beside them (its parts' meeting and the output).
template <int TILE, int ROWS, int EXTRA>
NVFP4_HD uint64_t ar_seq_units(const ArLine& a, const ArSeq& s) {
  if (s.n <= 0) return 0;
  const int key_end = static_cast<int>(least<int64_t>(a.cap, s.len));
  const int blocks = (s.n * a.group + ROWS - 1) / ROWS;
  const int span = (ROWS - 1 + a.group - 1) / a.group;   // positions between a block's first and last row, at most
  int most;
  if (a.window > 0 && blocks > 1) {
    // a block whose rows lie as late as any: two more tiles than its widest range of positions can touch
    const int64_t st = (least(a.sinks, key_end) + TILE - 1) / TILE;
    const int64_t w = (static_cast<int64_t>(a.window) + span) / TILE + 2;
    most = static_cast<int>(least<int64_t>(st + w, (key_end + TILE - 1) / TILE));
  } else {
    most = kv_tiles<TILE>(s.len - s.n, s.len - 1, a.window, a.sinks, key_end).count;
  }
  return static_cast<uint64_t>(most_of(most, 1) + EXTRA) * (static_cast<uint64_t>(blocks) * static_cast<unsigned>(a.heads));
}

// Length of a CTA's piece, of lines that U (uint32_t or uint64_t) can hold.
template <int EXTRA, class U>
NVFP4_HD U ar_piece(const ArLine& a, U total, unsigned ctas) {
  const U per = (total + (ctas - 1)) / ctas;
  // where a CTA's piece would be one tile of long items, two: half the parts to
  // join (one sequence of 2,000 positions: 8.9 -> 8.6 us)
  return per == 1 && total / (16u + EXTRA) >= static_cast<unsigned>(a.batch) * static_cast<unsigned>(a.heads) ? 2 : per;
}

// The item at u, up to the piece's end, and u behind it; false once the piece is
// done. pre[b]: the line before sequence b; seq(b) gives an ArSeq.
template <int TILE, int ROWS, class U, class Seqs>
NVFP4_HD bool ar_next(const ArLine& a, const uint64_t* pre, const Seqs& seq, U per, U& u, U end, ArItem& g) {
  while (u < end) {
    int lo = 0, hi = a.batch;             // last b with pre[b] <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (static_cast<U>(pre[mid]) <= u)
        lo = mid;
      else
        hi = mid;
    }
    g.b = lo;
    g.done = 0;
    const ArSeq s = seq(lo);
    g.row0 = s.row0;
    const U items = static_cast<U>((s.n * a.group + ROWS - 1) / ROWS) * static_cast<unsigned>(a.heads);
    const U before = static_cast<U>(pre[lo]), per_item = (static_cast<U>(pre[lo + 1]) - before) / items;
    const U in = u - before, item = in / per_item;
    const U rb = item / static_cast<unsigned>(a.heads);
    g.h = static_cast<int>(item - rb * static_cast<unsigned>(a.heads));
    g.i0 = static_cast<int>(in - item * per_item);
    const U u0 = u - static_cast<unsigned>(g.i0);
    const int i1 = static_cast<int>(least(static_cast<U>(end - u0), per_item));
    u = u0 + static_cast<unsigned>(i1);
    g.r0 = static_cast<int>(rb) * ROWS;
    g.n_rows = least(ROWS, s.n * a.group - g.r0);
    g.p0 = s.len - s.n + g.r0 / a.group;
    g.p1 = s.len - s.n + (g.r0 + g.n_rows - 1) / a.group;
    g.key_end = static_cast<int>(least<int64_t>(a.cap, s.len));
    g.tiles = kv_tiles<TILE>(g.p0, g.p1, a.window, a.sinks, g.key_end);
    // what follows the item's tiles on the line is nobody's work
    const int real = most_of(g.tiles.count, 1);
    if (g.i0 >= real) continue;
    g.i1 = least(i1, g.tiles.count);
    g.first_cta = static_cast<unsigned>(u0 / per);
    g.last_cta = static_cast<unsigned>((u0 + static_cast<unsigned>(real) - 1u) / per);
    return true;
  }
  return false;
}

// A CTA's piece of a line, walked in 32 bits where its length is below 2^31: the
// GPU has no 64-bit division (all in 64 bits, one sequence of 2,000 positions took
// 9.0 us, in both ways 8.5-8.6).
template <int TILE, int ROWS, int EXTRA>
struct ArPiece {
  uint64_t per, u, end;
  bool wide;

  NVFP4_HD ArPiece(const ArLine& a, uint64_t total, unsigned ctas, unsigned cta) : wide((total >> 31) != 0) {
    if (wide) {
      per = ar_piece<EXTRA, uint64_t>(a, total, ctas);
      u = least(cta * per, total);
      end = least(u + per, total);
    } else {
      // cta * n is below 2^31 + 2 ctas
      const uint32_t t = static_cast<uint32_t>(total), n = ar_piece<EXTRA, uint32_t>(a, t, ctas), at = least(cta * n, t);
      per = n;
      u = at;
      end = least(at + n, t);
    }
  }
  template <class Seqs>
  NVFP4_HD bool next(const ArLine& a, const uint64_t* pre, const Seqs& seq, ArItem& g) {
    if (wide) return ar_next<TILE, ROWS, uint64_t>(a, pre, seq, per, u, end, g);
    uint32_t at = static_cast<uint32_t>(u);
    const bool more = ar_next<TILE, ROWS, uint32_t>(a, pre, seq, static_cast<uint32_t>(per), at, static_cast<uint32_t>(end), g);
    u = at;
    return more;
  }
};

}  // namespace nvfp4
