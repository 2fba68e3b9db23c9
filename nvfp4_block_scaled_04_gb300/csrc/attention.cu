// Attention over a paged key-value cache: which kernel a call takes.
#include "attention_rows.cuh"
#include "kv.cuh"
#include "launch.h"

namespace nvfp4 {

namespace {

constexpr float LOG2_E = 1.4426950408889634f;

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

// Eight-row tiles of a call of the split kernel.
int rows_nt(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4; }

// CTAs of the split kernel: two per SM while the accumulators leave room.
int rows_grid(int nt) { return (nt <= 2 ? 2 : 1) * sm_count(); }

constexpr int64_t COUNTER_BYTES = 4096;   // arrival counters at the front of the workspace

template <bool E4M3, int D, int NT>
int launch_rows(const ArParams& p, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  const int smem = ar_smem_bytes<E4M3, D, NT>(p.s.batch);
  const int rc = ensure_smem(attention_rows_kernel<E4M3, D, NT>, smem);
  if (rc) return rc;
  return launch_ex(attention_rows_kernel<E4M3, D, NT>, dim3(rows_grid(NT)), dim3(AR_THREADS), smem, 1, true, stream, mk, mv,
                   p);
}

template <bool E4M3, int D>
int launch_rows_nt(int nt, const ArParams& p, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  switch (nt) {
    case 1: return launch_rows<E4M3, D, 1>(p, mk, mv, stream);
    case 2: return launch_rows<E4M3, D, 2>(p, mk, mv, stream);
    case 3: return launch_rows<E4M3, D, 3>(p, mk, mv, stream);
    default: return launch_rows<E4M3, D, 4>(p, mk, mv, stream);
  }
}

// One page of one head as [halves][rows][seg bytes], a copy box of `box` rows of it.
int kv_map(CUtensorMap* map, const void* pool, const nvfp4_kv_cache_t& c, int box) {
  const int64_t row = static_cast<int64_t>(c.head_dim) * (c.dtype == NVFP4_DTYPE_BF16 ? 2 : 1);
  const int64_t seg = row >= 128 ? 128 : 64, halves = row / seg;
  const int64_t dims[4] = {seg, c.page_size, halves, c.pages * c.heads};
  const int64_t strides[3] = {row, halves > 1 ? seg : row * c.page_size, row * c.page_size};
  const int boxes[4] = {static_cast<int>(seg), box, static_cast<int>(halves), 1};
  return make_tmap_4d_u8(map, pool, dims, strides, boxes,
                         seg == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace

size_t attention_workspace_bytes(int64_t batch, int64_t max_new, int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  if (batch <= 0 || max_new <= 0 || kv_heads <= 0 || q_heads <= 0 || head_dim <= 0) return 0;
  const int nt = rows_nt(max_new * (q_heads / kv_heads));
  return static_cast<size_t>(COUNTER_BYTES + static_cast<int64_t>(rows_grid(nt)) * 2 * 8 * nt * (head_dim + 2) * 4);
}

int launch_paged_attention(const uint16_t* Q, int64_t q_stride, int q_heads, const nvfp4_kv_cache_t& c,
                           const KvSeqs& s, int window, int sinks, float scale, uint16_t* out, void* ws,
                           cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return NVFP4_ERR_CUDA;
  const int group = q_heads / c.heads;
  const int nt = rows_nt(static_cast<int64_t>(s.max_new) * group);
  if (4 * rows_grid(nt) > COUNTER_BYTES) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  CUtensorMap mk, mv;
  const int box = c.page_size < AR_TILE ? c.page_size : AR_TILE;
  if (int rc = kv_map(&mk, c.k, c, box)) return rc;
  if (int rc = kv_map(&mv, c.v, c, box)) return rc;
  ArParams p;
  p.s = s;
  p.q = Q;
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
  p.min_tiles = 1;
  p.status = status;
  const bool e4m3 = c.dtype == NVFP4_DTYPE_E4M3;
  if (c.head_dim == 128)
    return e4m3 ? launch_rows_nt<true, 128>(nt, p, mk, mv, stream) : launch_rows_nt<false, 128>(nt, p, mk, mv, stream);
  return e4m3 ? launch_rows_nt<true, 64>(nt, p, mk, mv, stream) : launch_rows_nt<false, 64>(nt, p, mk, mv, stream);
}

}  // namespace nvfp4
