// Attention over a paged key-value cache: which kernel a call takes.
#include "attention_rows.cuh"
#include "attention_tiles.cuh"
#include "kv.cuh"
#include "launch.h"

#include <algorithm>

namespace nvfp4 {

namespace {

constexpr float LOG2_E = 1.4426950408889634f;

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

// Eight-row tiles of an item of the split kernel (more than 32 rows: several items).
int rows_nt(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4; }

// Its CTAs: two per SM while the accumulators leave room (ArShape::CTAS).
int rows_grid(int nt) { return (nt <= 3 ? 2 : 1) * sm_count(); }

constexpr int64_t COUNTER_BYTES = 4096;   // arrival counters at the front of the workspace
constexpr int SMEM_SM = 227 * 1024;       // dynamic shared memory of the CTAs of an SM (1 KB each is reserved beside it)

// One page of one head as [halves][rows][seg bytes], a copy box of `box` rows of `box_halves` halves.
int kv_map(CUtensorMap* map, const void* pool, const nvfp4_kv_cache_t& c, int box, int box_halves, bool swizzled = true) {
  const int64_t row = static_cast<int64_t>(c.head_dim) * (c.dtype == NVFP4_DTYPE_BF16 ? 2 : 1);
  const int64_t seg = row >= 128 ? 128 : 64, halves = row / seg;
  const int64_t dims[4] = {seg, c.page_size, halves, c.pages * c.heads};
  const int64_t strides[3] = {row, halves > 1 ? seg : row * c.page_size, row * c.page_size};
  const int boxes[4] = {static_cast<int>(seg), box, box_halves, 1};
  return make_tmap_4d_u8(map, pool, dims, strides, boxes,
                         !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : seg == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <bool E4M3, int D, int NT>
int launch_rows(ArParams p, const nvfp4_kv_cache_t& c, cudaStream_t stream) {
  using S = ArShape<E4M3, D, NT>;
  CUtensorMap mk, mv;
  const int box = c.page_size < S::TILE ? c.page_size : S::TILE;
  if (int rc = kv_map(&mk, c.k, c, box, S::HALVES)) return rc;
  if (int rc = kv_map(&mv, c.v, c, box, S::HALVES)) return rc;
  const int fixed = S::FIXED_BYTES + 8 * (p.s.batch + 2) + (p.s.batch <= AR_KEPT ? 4 * (2 * p.s.batch + 2) : 0);
  const int room = (SMEM_SM - (S::CTAS - 1) * 1024) / S::CTAS - fixed;
  p.stages = std::max(2, std::min(AR_MAX_STAGES, room / S::STAGE_BYTES));
  const int smem = fixed + p.stages * S::STAGE_BYTES;
  const int rc = ensure_smem(attention_rows_kernel<E4M3, D, NT>, smem);
  if (rc) return rc;
  return launch_ex(attention_rows_kernel<E4M3, D, NT>, dim3(rows_grid(NT)), dim3(S::THREADS), smem, 1, true, stream,
                   mk, mv, p);
}

template <bool E4M3, int D>
int launch_rows_nt(int nt, const ArParams& p, const nvfp4_kv_cache_t& c, cudaStream_t stream) {
  switch (nt) {
    case 1: return launch_rows<E4M3, D, 1>(p, c, stream);
    case 2: return launch_rows<E4M3, D, 2>(p, c, stream);
    case 3: return launch_rows<E4M3, D, 3>(p, c, stream);
    default: return launch_rows<E4M3, D, 4>(p, c, stream);
  }
}

// Blocks of rows (256 at most, whole tokens) times kv heads of a call of the tile kernel, at most
// (where `start` does not fall: the sequences' rows add up to `tokens` or fewer).
int64_t tiles_items(int64_t tokens, int64_t batch, int64_t heads, int group) {
  const int64_t block = 2 * (AT_ROWS / group);
  return heads * ((tokens + batch * (block - 1)) / block);
}

template <bool E4M3, int D>
int launch_tiles(const uint16_t* Q, int64_t q_stride, int q_heads, const nvfp4_kv_cache_t& c, AtParams& p,
                 cudaStream_t stream) {
  CUtensorMap mq, mk, mv;
  const int64_t q_dims[4] = {128, q_heads, p.s.tokens, D / 64};
  const int64_t q_strides[3] = {D * 2, q_stride * 2, 128};
  const int q_box[4] = {128, p.group, AT_ROWS / p.group, 1};
  if (int rc = make_tmap_4d_u8(&mq, Q, q_dims, q_strides, q_box, CU_TENSOR_MAP_SWIZZLE_128B)) return rc;
  // E4M3 codes are copied as they lie, in boxes of up to a chunk's rows
  constexpr int most = E4M3 ? AT_CHUNK : AT_TILE;
  const int box = c.page_size < most ? c.page_size : most;
  if (int rc = kv_map(&mk, c.k, c, box, 1, !E4M3)) return rc;
  if (int rc = kv_map(&mv, c.v, c, box, 1, !E4M3)) return rc;
  const int64_t items = tiles_items(p.s.tokens, p.s.batch, c.heads, p.group);
  const int ctas = sm_count();
  // fewer items than half the SMs: each is split over its positions
  p.parts = items < ctas ? static_cast<int>(ctas / items) : 1;
  p.units = items * p.parts;
  const int rc = ensure_smem(attention_tiles_kernel<E4M3, D>, AtShape<E4M3, D>::SMEM);
  if (rc) return rc;
  return launch_ex(attention_tiles_kernel<E4M3, D>, dim3(static_cast<unsigned>(p.units < ctas ? p.units : ctas)), dim3(AtShape<E4M3, D>::THREADS),
                   AtShape<E4M3, D>::SMEM, 1, true, stream, mq, mk, mv, p);
}

// Rows of a kv head from which the tile kernel takes a call.
bool takes_tiles(int64_t rows) { return rows > 32; }

}  // namespace

size_t attention_workspace_bytes(int64_t batch, int64_t max_new, int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  if (batch <= 0 || max_new <= 0 || kv_heads <= 0 || q_heads <= 0 || head_dim <= 0) return 0;
  const int64_t rows = max_new * (q_heads / kv_heads);
  // rows of partial sums, the most of any call with as many rows or fewer (an
  // item of 24 rows has more than one of 32, whose CTAs are half as many)
  int64_t parts = 0;
  for (int nt = 1; nt <= rows_nt(rows); ++nt) parts = std::max(parts, static_cast<int64_t>(rows_grid(nt)) * 2 * 8 * nt);
  if (takes_tiles(rows)) parts = std::max(parts, static_cast<int64_t>(sm_count()) * 2 * AT_ROWS);
  return static_cast<size_t>(COUNTER_BYTES + parts * (head_dim + 2) * 4);
}

int launch_paged_attention(const uint16_t* Q, int64_t q_stride, int q_heads, const nvfp4_kv_cache_t& c,
                           const KvSeqs& s, int window, int sinks, float scale, uint16_t* out, void* ws,
                           cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return NVFP4_ERR_CUDA;
  const int group = q_heads / c.heads;
  const int64_t rows = static_cast<int64_t>(s.max_new) * group;
  const bool e4m3 = c.dtype == NVFP4_DTYPE_E4M3;
  if (takes_tiles(rows) && group <= AT_ROWS / 2 && scale > 0.0f) {
    AtParams p;
    p.s = s;
    p.out = out;
    p.pages = c.pages;
    p.heads = c.heads;
    p.group = group;
    p.page_size = c.page_size;
    p.page_log2 = log2_of(c.page_size);
    p.window = window;
    p.sinks = sinks;
    p.scale = scale * LOG2_E;
    p.arrived = static_cast<unsigned*>(ws);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + COUNTER_BYTES);
    p.status = status;
    p.v = c.v;
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    if (c.head_dim == 128)
      return e4m3 ? launch_tiles<true, 128>(Q, q_stride, q_heads, c, p, stream)
                  : launch_tiles<false, 128>(Q, q_stride, q_heads, c, p, stream);
    return e4m3 ? launch_tiles<true, 64>(Q, q_stride, q_heads, c, p, stream)
                : launch_tiles<false, 64>(Q, q_stride, q_heads, c, p, stream);
  }
  const int nt = rows_nt(rows);
  if (4 * rows_grid(nt) > COUNTER_BYTES) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  ArParams p;
  p.s = s;
  p.q = Q;
  p.v = c.v;
  p.q_stride = q_stride;
  p.out = out;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.pages = c.pages;
  p.heads = c.heads;
  p.group = group;
  p.page_size = c.page_size;
  p.page_log2 = log2_of(c.page_size);
  p.window = window;
  p.sinks = sinks;
  p.scale = scale * LOG2_E;
  p.arrived = static_cast<unsigned*>(ws);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + COUNTER_BYTES);
  p.status = status;
  if (c.head_dim == 128)
    return e4m3 ? launch_rows_nt<true, 128>(nt, p, c, stream) : launch_rows_nt<false, 128>(nt, p, c, stream);
  return e4m3 ? launch_rows_nt<true, 64>(nt, p, c, stream) : launch_rows_nt<false, 64>(nt, p, c, stream);
}

}  // namespace nvfp4
