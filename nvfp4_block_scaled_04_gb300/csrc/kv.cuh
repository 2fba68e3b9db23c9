// Shared pieces of the paged key-value cache kernels: which sequences a call
// deals with, and where a sequence's new rows lie.
#pragma once

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

// The tiles that a block of rows sees: [0, st) (sinks) and [w0, end).
struct KvTiles {
  int st, w0, count;
  NVFP4_DEV int tile(int i) const { return i < st ? i : w0 + (i - st); }
};

// Tiles of the rows at positions p0..p1 (p1 < 0: none).
template <int TILE>
NVFP4_DEV KvTiles kv_tiles(int p0, int p1, int window, int sinks, int key_end) {
  KvTiles t;
  const int end = (min(p1 + 1, key_end) + TILE - 1) / TILE;   // one past the last
  t.st = 0;
  t.w0 = 0;
  if (window > 0) {
    const int lo = p0 - window + 1;                                  // first position in a window
    const int w0 = lo > 0 ? lo / TILE : 0;
    const int st = min((min(sinks, key_end) + TILE - 1) / TILE, end);
    if (w0 > st) {
      t.st = st;
      t.w0 = w0;
    }
  }
  t.count = end > t.w0 ? t.st + end - t.w0 : t.st;
  if (end <= 0) t.count = 0;
  return t;
}

NVFP4_DEV void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// Non-finite elements of value rows that some rows of a block see and others do
// not. As an operand they would reach the others too (0 * inf is NaN), so the
// kernels put zeros in their place and add them, at the end, to the rows that
// see them. A CTA remembers KV_BAD of them; further ones stay where they are.
constexpr int KV_BAD = 16;
struct KvBad {
  int item, j, d;      // item of the CTA, position, element
  float v;
};
// Remembers one; false if there is no room left. Other threads may be reading
// the list for other items meanwhile: `item`, which no reader looks for yet, is
// written last (it is -1 in entries that were never written).
NVFP4_DEV bool kv_remember(int* count, KvBad* list, int item, int j, int d, float v) {
  const int n = atomicAdd(count, 1);
  if (n >= KV_BAD) return false;
  list[n].j = j;
  list[n].d = d;
  list[n].v = v;
  __threadfence_block();
  *reinterpret_cast<volatile int*>(&list[n].item) = item;
  return true;
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
