// Keeping a paged key-value cache on the device: new rows appended, pages
// reserved, sequences forked and released, the pool compacted. Lengths, page
// tables and reference counts stay in device memory, so a decode loop needs
// no host round trip (and can be captured in a CUDA graph).
//
// Pages are handed out lowest id first, in the order of the call's sequences,
// so results do not depend on scheduling. The kernels that decide (which
// pages, which moves) run in one CTA and leave a plan in the workspace; the
// kernels that move data read it.
//
// Cost. Append and the copies are bound by memory; the planning CTA reads the
// reference counts 16 to a thread (64 KB per round) and stops as soon as it
// has the pages it needs. Measured: 16k tokens appended in 26.3 us (19.8 at the
// copy rate), 64 single tokens in 2.8 us on the device; a half full pool of
// 24k pages compacted in 273 us (237.6 at the copy rate, 8 of them planning); a
// reserve in which no sequence lacks a page 2.7 us in a pool of 8 pages (one
// sequence) and 5.4 us in one of 24k (64 sequences).
#include "kv.cuh"
#include "launch.h"

namespace nvfp4 {

namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_PER_THREAD = 16;

// ------------------------------------------------------------------ append

// Eight bf16 values over sc as E4M3 codes of the IEEE quotients. With r =
// RN(1 / sc), rl = RN(r (1 - 2^-20)) lies below 1 / sc and rh = RN(r (1 + 2^-20))
// above it, and rounding is monotone: where the codes of RN(x rl) and RN(x rh)
// agree, they are the quotient's. Otherwise (a midpoint close by) the division
// decides. (60,000 tokens: 82.6 -> 72.0 us, 5.1 TB/s.)
NVFP4_DEV uint2 e4m3_of_quotients(const uint4& x, float sc) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const float r = __frcp_rn(sc), rl = r * 0.99999904632568359375f, rh = r * 1.00000095367431640625f;
  uint32_t o[4], differ = 0;
#pragma unroll
  for (int z = 0; z < 4; ++z) {
    const float a = bf16_bits_to_f32(w[z] & 0xFFFFu), b = bf16_bits_to_f32(w[z] >> 16);
    o[z] = f32x2_to_e4m3x2(a * rl, b * rl);
    differ |= o[z] ^ f32x2_to_e4m3x2(a * rh, b * rh);
  }
  if (differ || !(sc > 0x1p-100f && sc < 0x1p100f)) {
#pragma unroll
    for (int z = 0; z < 4; ++z)
      o[z] = f32x2_to_e4m3x2(__fdiv_rn(bf16_bits_to_f32(w[z] & 0xFFFFu), sc), __fdiv_rn(bf16_bits_to_f32(w[z] >> 16), sc));
  }
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

// One warp per (TOKENS consecutive tokens, K or V): their rows of every head.
// The lanes look up the tokens' places side by side. bf16 rows are copied, E4M3
// rows are x / scale[head] (IEEE division), rounded to nearest even and
// saturated at 448: the cache's 8 bits are the one rounding of the append.
// TOKENS is 8 for long appends, which share one chain of dependent lookups
// among 16 KB of rows, and 1 for short ones, which need all the warps.
template <bool E4M3, int TOKENS>
__global__ void __launch_bounds__(256) kv_append_kernel(const nvfp4_kv_cache_t c, const KvSeqs s, const uint16_t* K,
                                                        const uint16_t* V, int64_t k_stride, int64_t v_stride,
                                                        int* status) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int64_t t0 = (unit >> 1) * TOKENS;
  const bool is_v = unit & 1;
  if (t0 >= s.tokens) return;
  const int64_t head_elems = static_cast<int64_t>(c.page_size) * c.head_dim;
  int64_t place = -1;   // of lane's token's row of head 0, in elements of the pool
  const int64_t t = t0 + lane;
  if (lane < TOKENS && t < s.tokens) {
    // its sequence: the last one whose rows start at or before t
    int lo = 0, hi = s.batch;
    if (s.start) {
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.start[mid] <= t)
          lo = mid;
        else
          hi = mid;
      }
    } else {
      lo = static_cast<int>(t / s.max_new);
    }
    const int64_t r0 = kv_row0(s, lo), r1 = kv_row0(s, lo + 1);
    if (t >= r0 && t < r1) {
      const int64_t pos = static_cast<int64_t>(s.lens[lo]) - (r1 - t);
      const int64_t entry = pos / c.page_size;
      const int page = pos >= 0 && entry < s.max_pages ? s.table[lo * s.table_stride + entry] : -1;
      if (page >= 0 && page < c.pages)
        place = static_cast<int64_t>(page) * c.heads * head_elems + (pos % c.page_size) * c.head_dim;
      else if (!is_v)
        atomicExch(status, NVFP4_ERR_INVALID_ARG);
    }
  }
  __syncwarp();
  const int n8 = c.heads * c.head_dim / 8, d8_log2 = c.head_dim == 128 ? 4 : 3;
  const int64_t stride = is_v ? v_stride : k_stride;
  const uint16_t* src0 = (is_v ? V : K) + t0 * stride;
  uint8_t* pool = static_cast<uint8_t*>(is_v ? c.v : c.k);
  const float* scale = is_v ? c.v_scale : c.k_scale;
  for (int tt = 0; tt < TOKENS; ++tt) {
    const int64_t row0 = __shfl_sync(0xffffffffu, place, tt);
    if (row0 < 0) continue;
    const uint16_t* src = src0 + tt * stride;
    for (int i0 = lane; i0 < n8; i0 += 128) {
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + 32 * j < n8) x[j] = *reinterpret_cast<const uint4*>(src + (i0 + 32 * j) * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + 32 * j;
        if (i >= n8) break;
        const int h = i >> d8_log2;
        const int64_t at = row0 + h * head_elems + (i - (h << d8_log2)) * 8;
        if (E4M3) {
          *reinterpret_cast<uint2*>(pool + at) = e4m3_of_quotients(x[j], scale[h]);
        } else {
          *reinterpret_cast<uint4*>(pool + 2 * at) = x[j];
        }
      }
    }
  }
}

template <bool E4M3>
int launch_append(const nvfp4_kv_cache_t& c, const KvSeqs& s, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                  int64_t v_stride, int* status, cudaStream_t stream) {
  // 8 tokens a warp once that still gives every SM 16 warps
  const bool many = s.tokens >= 64 * static_cast<int64_t>(sm_count());
  const int64_t units = 2 * ceil_div(s.tokens, many ? 8 : 1);
  // few rows spread over more CTAs, one warp each
  const int threads = units <= 8 * sm_count() ? 32 : 256;
  const dim3 grid(static_cast<unsigned>(ceil_div(units, threads / 32)));
  return many ? launch_ex(kv_append_kernel<E4M3, 8>, grid, dim3(threads), 0, 1, true, stream, c, s, k, v, k_stride, v_stride, status)
              : launch_ex(kv_append_kernel<E4M3, 1>, grid, dim3(threads), 0, 1, true, stream, c, s, k, v, k_stride, v_stride, status);
}

// ------------------------------------------------------------ planning CTA

// Exclusive prefix sum of v over the PLAN_THREADS threads; *total gets the sum.
NVFP4_DEV int plan_scan(int v, int* total) {
  __shared__ int warp_sum[PLAN_THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();   // the previous scan's sums have been read
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int w = warp_sum[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
  return before + x - v;
}

// This thread's PLAN_PER_THREAD consecutive reference counts from page p0 on
// (1 past the pool's end: taken).
NVFP4_DEV void load_refs(const int32_t* refs, int64_t pages, int64_t p0, int (&r)[PLAN_PER_THREAD]) {
  if (p0 + PLAN_PER_THREAD <= pages && (reinterpret_cast<uintptr_t>(refs) & 15u) == 0) {
#pragma unroll
    for (int j = 0; j < PLAN_PER_THREAD / 4; ++j) {
      const int4 x = *reinterpret_cast<const int4*>(refs + p0 + 4 * j);
      r[4 * j] = x.x;
      r[4 * j + 1] = x.y;
      r[4 * j + 2] = x.z;
      r[4 * j + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < PLAN_PER_THREAD; ++j) r[j] = p0 + j < pages ? refs[p0 + j] : 1;
  }
}

// The `need` lowest free pages, in order, into list; returns how many there are.
NVFP4_DEV int lowest_free(const int32_t* refs, int64_t pages, int need, int32_t* list) {
  int have = 0;
  for (int64_t base = 0; base < pages && have < need; base += PLAN_THREADS * PLAN_PER_THREAD) {
    const int64_t p0 = base + static_cast<int64_t>(threadIdx.x) * PLAN_PER_THREAD;
    int r[PLAN_PER_THREAD], n = 0, total;
    load_refs(refs, pages, p0, r);
#pragma unroll
    for (int j = 0; j < PLAN_PER_THREAD; ++j) n += r[j] <= 0;
    int at = have + plan_scan(n, &total);
#pragma unroll
    for (int j = 0; j < PLAN_PER_THREAD; ++j)
      if (r[j] <= 0) {
        if (at < need) list[at] = static_cast<int32_t>(p0 + j);
        ++at;
      }
    have += total;
  }
  __syncthreads();   // the list is written
  return have < need ? have : need;
}

// ----------------------------------------------------------------- reserve

// Pages for the positions of each sequence's new tokens: every table entry
// there that holds no page (an id outside the pool) gets one, in (sequence, position) order. One warp
// counts and fills a sequence's entries.
// ws: free pages [pages], then entries needed by the sequences before each [batch].
__global__ void __launch_bounds__(PLAN_THREADS) kv_reserve_kernel(const KvSeqs s, int page_size, int32_t* table,
                                                                  int32_t* refs, int64_t pages, int32_t* ws,
                                                                  int* status) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t* list = ws;              // [pages]
  int32_t* first = ws + pages;     // [batch] entries needed by the sequences before
  auto range = [&](int b, int* e0, int* e1) {
    const int n = kv_row0(s, b + 1) - kv_row0(s, b);
    const int64_t len = s.lens[b], p0 = len - n > 0 ? len - n : 0;
    *e0 = static_cast<int>(p0 / page_size);
    const int64_t end = n > 0 && len > 0 ? (len + page_size - 1) / page_size : 0;
    if (lane == 0 && end > s.max_pages) atomicExch(status, NVFP4_ERR_INVALID_ARG);
    *e1 = static_cast<int>(end < s.max_pages ? end : s.max_pages);
  };
  auto holds_none = [&](int page) { return page < 0 || page >= pages; };
  for (int b = warp; b < s.batch; b += PLAN_THREADS / 32) {
    int e0, e1, n = 0;
    range(b, &e0, &e1);
    const int32_t* row = table + b * s.table_stride;
    for (int e = e0 + lane; e < e1; e += 32) n += holds_none(row[e]);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) first[b] = n;
  }
  __syncthreads();
  int need = 0;
  for (int b0 = 0; b0 < s.batch; b0 += PLAN_THREADS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int total;
    const int n = b < s.batch ? first[b] : 0;
    const int at = need + plan_scan(n, &total);
    if (b < s.batch) first[b] = at;
    need += total;
  }
  const int want = need < pages ? need : static_cast<int>(pages);
  const int have = lowest_free(refs, pages, want, list);
  if (threadIdx.x == 0 && have < need) atomicExch(status, NVFP4_ERR_NO_PAGES);
  for (int b = warp; b < s.batch; b += PLAN_THREADS / 32) {
    int e0, e1;
    range(b, &e0, &e1);
    int32_t* row = table + b * s.table_stride;
    int at = first[b];
    for (int e = e0; e < e1; e += 32) {
      const bool lacks = e + lane < e1 && holds_none(row[e + lane]);
      const unsigned m = __ballot_sync(0xffffffffu, lacks);
      const int k = at + __popc(m & ((1u << lane) - 1u));
      if (lacks && k < have) {
        row[e + lane] = list[k];
        refs[list[k]] = 1;
      }
      at += __popc(m);
    }
  }
}

// -------------------------------------------------------------------- fork

// Gives each fork's partly filled last page a fresh page (-1 where there is
// none left or none is needed): its id goes into the fork's table row, and the
// page is taken. PLAN_THREADS forks at a time.
__global__ void __launch_bounds__(PLAN_THREADS) kv_fork_plan_kernel(int32_t* table, int64_t table_stride, int max_pages,
                                                                    const int32_t* lens, int rows, int32_t* refs,
                                                                    int64_t pages, int page_size, const int32_t* src,
                                                                    const int32_t* dst, int n, int* status) {
  __shared__ int32_t list[PLAN_THREADS];
  pdl_launch_dependents();
  pdl_wait();
  for (int f0 = 0; f0 < n; f0 += PLAN_THREADS) {
    const int f = f0 + static_cast<int>(threadIdx.x);
    bool wants = false;
    int32_t* entry = nullptr;   // of the fork's last page, where it is partly filled
    if (f < n) {
      const int a = src[f], d = dst[f];
      if (a >= 0 && a < rows && d >= 0 && d < rows && a != d) {
        const int len = lens[a];
        if (len > 0 && len % page_size != 0 && len / page_size < max_pages) {
          const int p = table[a * table_stride + len / page_size];
          wants = p >= 0 && p < pages;
          entry = table + d * table_stride + len / page_size;
        }
      } else {
        atomicExch(status, NVFP4_ERR_INVALID_ARG);
      }
    }
    int need;
    const int at = plan_scan(wants, &need);
    const int have = lowest_free(refs, pages, need, list);
    if (threadIdx.x == 0 && have < need) atomicExch(status, NVFP4_ERR_NO_PAGES);
    const int p = wants && at < have ? list[at] : -1;
    if (entry) *entry = p;
    if (p >= 0) refs[p] = 1;
    __syncthreads();   // the list has been read, and these pages are taken for the next forks
  }
}

// Block (f, y): y < 2 heads: the rows in use of one head of fork f's last
// page (K, then V); y == 2 heads: its table row, length and reference counts.
__global__ void __launch_bounds__(128) kv_fork_copy_kernel(const nvfp4_kv_cache_t c, int32_t* table,
                                                           int64_t table_stride, int max_pages, int32_t* lens,
                                                           int rows, int32_t* refs, const int32_t* src,
                                                           const int32_t* dst, int elem_bytes) {
  pdl_launch_dependents();
  pdl_wait();
  const int f = blockIdx.x, y = blockIdx.y;
  const int a = src[f], d = dst[f];
  if (a < 0 || a >= rows || d < 0 || d >= rows || a == d) return;
  const int len = lens[a] > 0 ? lens[a] : 0;
  const int full = len / c.page_size, tail = len % c.page_size;
  // the plan wrote it; the block that writes the row writes it again as it is
  const int fresh = tail && full < max_pages ? table[d * table_stride + full] : -1;
  const int32_t* from = table + a * table_stride;
  if (y < 2 * c.heads) {
    // (in orderly lists the plan has seen the source's page; where a source is also a
    // fork, its row is being written meanwhile)
    const int last = fresh >= 0 ? from[full] : -1;
    if (last < 0 || last >= c.pages || fresh >= c.pages) return;
    const int64_t block = static_cast<int64_t>(c.page_size) * c.head_dim * elem_bytes;
    const int64_t h = y >> 1;
    uint8_t* pool = static_cast<uint8_t*>((y & 1) ? c.v : c.k);
    const uint4* x = reinterpret_cast<const uint4*>(pool + (last * static_cast<int64_t>(c.heads) + h) * block);
    uint4* o = reinterpret_cast<uint4*>(pool + (fresh * static_cast<int64_t>(c.heads) + h) * block);
    const int n16 = tail * c.head_dim * elem_bytes / 16;
#pragma unroll 4
    for (int i = threadIdx.x; i < n16; i += 128) o[i] = x[i];
    return;
  }
  int32_t* to = table + d * table_stride;
  for (int e = threadIdx.x; e < max_pages; e += 128) {
    int p = -1;
    if (e < full) {
      p = from[e];
      if (p >= 0 && p < c.pages)
        atomicAdd(refs + p, 1);
      else
        p = -1;
    } else if (e == full && tail) {
      p = fresh;
    }
    to[e] = p;
  }
  if (threadIdx.x == 0) lens[d] = len;
}

// ----------------------------------------------------------------- release

__global__ void __launch_bounds__(128) kv_release_kernel(int32_t* table, int64_t table_stride, int max_pages,
                                                         int32_t* lens, int rows, int32_t* refs, int64_t pages,
                                                         const int32_t* seqs, int* status) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = seqs[blockIdx.x];
  if (b < 0 || b >= rows) {
    if (threadIdx.x == 0) atomicExch(status, NVFP4_ERR_INVALID_ARG);
    return;
  }
  int32_t* row = table + b * table_stride;
  for (int e = threadIdx.x; e < max_pages; e += 128) {
    const int p = row[e];
    if (p >= 0 && p < pages) atomicSub(refs + p, 1);
    row[e] = -1;
  }
  if (threadIdx.x == 0) lens[b] = 0;
}

// ----------------------------------------------------------------- compact

// The plan: live pages whose id is at or past the number n of live pages go to
// the free ids below n, the i-th to the i-th. Sources and destinations are
// disjoint, so the moves need no order, and no page moves that need not.
// ws: the moved pages in order [pages], where each goes [pages], the number of
// moves and n.
__global__ void __launch_bounds__(PLAN_THREADS) kv_compact_plan_kernel(const int32_t* refs, int64_t pages,
                                                                       int32_t* live, int32_t* ws) {
  pdl_launch_dependents();
  pdl_wait();
  int32_t* from = ws;
  int32_t* to = ws + pages;
  int32_t* counts = ws + 2 * pages;
  int n = 0;
  for (int64_t base = 0; base < pages; base += PLAN_THREADS * PLAN_PER_THREAD) {
    int r[PLAN_PER_THREAD], k = 0, total;
    const int64_t p0 = base + static_cast<int64_t>(threadIdx.x) * PLAN_PER_THREAD;
    load_refs(refs, pages, p0, r);
#pragma unroll
    for (int j = 0; j < PLAN_PER_THREAD; ++j) k += r[j] > 0 && p0 + j < pages;
    plan_scan(k, &total);
    n += total;
  }
  int movers = 0, holes = 0;
  for (int64_t base = 0; base < pages; base += PLAN_THREADS * PLAN_PER_THREAD) {
    int r[PLAN_PER_THREAD], k = 0, total;
    const int64_t p0 = base + static_cast<int64_t>(threadIdx.x) * PLAN_PER_THREAD;
    load_refs(refs, pages, p0, r);
    // a thread's pages may lie on both sides of n: movers in the high half of the scanned word, holes in the low
#pragma unroll
    for (int j = 0; j < PLAN_PER_THREAD; ++j) {
      const int64_t p = p0 + j;
      if (p < pages) k += p < n ? (r[j] <= 0) : (r[j] > 0) << 16;
    }
    const int before = plan_scan(k, &total);
    int m = movers + (before >> 16), h = holes + (before & 0xFFFF);
#pragma unroll
    for (int j = 0; j < PLAN_PER_THREAD; ++j) {
      const int64_t p = p0 + j;
      if (p >= pages) break;
      if (p < n && r[j] <= 0) to[h++] = static_cast<int32_t>(p);
      if (p >= n && r[j] > 0) from[m++] = static_cast<int32_t>(p);
    }
    movers += total >> 16;
    holes += total & 0xFFFF;
  }
  if (threadIdx.x == 0) {
    counts[0] = movers;
    counts[1] = n;
    *live = n;
  }
}

constexpr int COMPACT_CHUNK = 16384;   // bytes of one CTA's step

// Copies the moved pages (chunks of K, then of V), moves their reference
// counts and renames their table entries.
__global__ void __launch_bounds__(256) kv_compact_move_kernel(const nvfp4_kv_cache_t c, int32_t* table,
                                                              int64_t table_stride, int max_pages, int rows,
                                                              int32_t* refs, const int32_t* ws, int64_t page_bytes) {
  pdl_launch_dependents();
  pdl_wait();
  const int32_t* from = ws;
  const int32_t* to = ws + c.pages;
  const int moves = ws[2 * c.pages], n = ws[2 * c.pages + 1];
  const int chunks = static_cast<int>((page_bytes + COMPACT_CHUNK - 1) / COMPACT_CHUNK);
  const int64_t units = static_cast<int64_t>(moves) * 2 * chunks;
  // a step's loads are in flight while the last step's stores go out, and its
  // page ids are read a step earlier still
  struct Step {
    const uint4* x;
    uint4* o;
    int n16;
  };
  auto step = [&](int64_t u) {
    Step t = {nullptr, nullptr, 0};
    if (u < units) {
      const int m = static_cast<int>(u / (2 * chunks)), part = static_cast<int>(u - static_cast<int64_t>(m) * 2 * chunks);
      uint8_t* pool = static_cast<uint8_t*>(part < chunks ? c.k : c.v);
      const int64_t off = static_cast<int64_t>(part < chunks ? part : part - chunks) * COMPACT_CHUNK;
      t.x = reinterpret_cast<const uint4*>(pool + from[m] * page_bytes + off) + threadIdx.x;
      t.o = reinterpret_cast<uint4*>(pool + to[m] * page_bytes + off) + threadIdx.x;
      t.n16 = static_cast<int>((page_bytes - off < COMPACT_CHUNK ? page_bytes - off : COMPACT_CHUNK) / 16) - static_cast<int>(threadIdx.x);
    }
    return t;
  };
  constexpr int PER = COMPACT_CHUNK / 16 / 256;
  Step now = step(blockIdx.x), then = step(static_cast<int64_t>(blockIdx.x) + gridDim.x);
  uint4 x[PER], y[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (256 * j < now.n16) x[j] = now.x[256 * j];
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (256 * j < then.n16) y[j] = then.x[256 * j];
    const Step next = step(u + 2 * static_cast<int64_t>(gridDim.x));
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (256 * j < now.n16) now.o[256 * j] = x[j];
#pragma unroll
    for (int j = 0; j < PER; ++j) x[j] = y[j];
    now = then;
    then = next;
  }
  const int64_t gtid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t gthreads = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t m = gtid; m < moves; m += gthreads) {
    refs[to[m]] = refs[from[m]];
    refs[from[m]] = 0;
  }
  const int64_t entries = static_cast<int64_t>(rows) * max_pages;
  for (int64_t i = gtid; i < entries; i += gthreads) {
    int32_t* e = table + (i / max_pages) * table_stride + i % max_pages;
    const int p = *e;
    if (p < n || p >= c.pages) continue;
    // moved ids are sorted: its place among them
    int lo = 0, hi = moves;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (from[mid] < p)
        lo = mid + 1;
      else
        hi = mid;
    }
    if (lo < moves && from[lo] == p) *e = to[lo];
  }
}

int elem_bytes_of(const nvfp4_kv_cache_t& c) { return c.dtype == NVFP4_DTYPE_BF16 ? 2 : 1; }

}  // namespace

int launch_kv_append(const nvfp4_kv_cache_t& c, const KvSeqs& s, const void* K, const void* V, int64_t k_stride,
                     int64_t v_stride, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return NVFP4_ERR_CUDA;
  auto* k = static_cast<const uint16_t*>(K);
  auto* v = static_cast<const uint16_t*>(V);
  return c.dtype == NVFP4_DTYPE_E4M3 ? launch_append<true>(c, s, k, v, k_stride, v_stride, status, stream)
                                     : launch_append<false>(c, s, k, v, k_stride, v_stride, status, stream);
}

size_t kv_pages_workspace_bytes(int64_t pages, int64_t n) { return static_cast<size_t>(4 * (2 * pages + n + 4)); }

int launch_kv_reserve(const KvSeqs& s, int page_size, int32_t* table, int32_t* refs, int64_t pages, void* ws,
                      cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return NVFP4_ERR_CUDA;
  return launch_ex(kv_reserve_kernel, dim3(1), dim3(PLAN_THREADS), 0, 1, true, stream, s, page_size, table, refs, pages,
                   static_cast<int32_t*>(ws), status);
}

int launch_kv_fork(const nvfp4_kv_cache_t& c, int32_t* table, int64_t table_stride, int max_pages, int32_t* lens,
                   int rows, int32_t* refs, const int32_t* src, const int32_t* dst, int n, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return NVFP4_ERR_CUDA;
  int rc = launch_ex(kv_fork_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, 1, true, stream, table, table_stride, max_pages,
                     static_cast<const int32_t*>(lens), rows, refs, static_cast<int64_t>(c.pages),
                     static_cast<int>(c.page_size), src, dst, n, status);
  if (rc) return rc;
  return launch_ex(kv_fork_copy_kernel, dim3(n, 2 * c.heads + 1), dim3(128), 0, 1, true, stream, c, table, table_stride,
                   max_pages, lens, rows, refs, src, dst, elem_bytes_of(c));
}

int launch_kv_release(int32_t* table, int64_t table_stride, int max_pages, int32_t* lens, int rows, int32_t* refs,
                      int64_t pages, const int32_t* seqs, int n, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return NVFP4_ERR_CUDA;
  return launch_ex(kv_release_kernel, dim3(n), dim3(128), 0, 1, true, stream, table, table_stride, max_pages, lens, rows,
                   refs, pages, seqs, status);
}

int launch_kv_compact(const nvfp4_kv_cache_t& c, int32_t* table, int64_t table_stride, int max_pages, int rows,
                      int32_t* refs, int32_t* live, void* ws, cudaStream_t stream) {
  int32_t* w = static_cast<int32_t*>(ws);
  int rc = launch_ex(kv_compact_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, 1, true, stream,
                     static_cast<const int32_t*>(refs), static_cast<int64_t>(c.pages), live, w);
  if (rc) return rc;
  const int64_t page_bytes = static_cast<int64_t>(c.heads) * c.page_size * c.head_dim * elem_bytes_of(c);
  return launch_ex(kv_compact_move_kernel, dim3(8 * sm_count()), dim3(256), 0, 1, true, stream, c, table, table_stride,
                   max_pages, rows, refs, static_cast<const int32_t*>(w), page_bytes);
}

}  // namespace nvfp4
