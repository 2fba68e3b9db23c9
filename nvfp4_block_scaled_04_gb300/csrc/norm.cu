// Root-mean-square norm of bf16 rows, with the residual's addition in front and
// the conversion to what the next linear takes behind:
//   s = x + residual          (rounded to the residual's type and stored; s = x without one)
//   t = s * (w + offset),  r = 1 / sqrt(mean(s^2) + eps),  y = t * r
//   out: bf16 y | E4M3 codes of y / a with a = max|y| / 448 of the row | NVFP4 of y
//
// The gain goes in before the row's r, so the sum of squares and the largest
// |t| come out of one reduction: rounding is monotone, so fl(max|t| * r) is
// max|y| exactly, for a row (E4M3), a block of 16 (NVFP4) and the tensor.
// Sums and all arithmetic are fp32; s is rounded because it is the stream that
// the next layer reads, and the norm is that of the stored stream.
//
// Bound by HBM for many rows, by latency (one load, one reduction, one store)
// for few. One row stays in registers between its only read and its only
// write; what is read once is loaded evict-first (2048 x 2048: 7.8 -> 7.1 us,
// 2048 x 16384 with an fp32 stream 71 -> 69), and a CTA's next row while its last
// one is summed and stored (7.1 -> 6.3, 69 -> 64). Measured in graphs of calls on
// changing inputs, bf16 stream and output: 1 x 5120 2.4 us, 512 x 5120 5.7,
// 8192 x 5120 52 (6.4 TB/s); E4M3 output, fp32 stream, 8192 x 5120 70.4 (6.5 TB/s).
// Rows of up to 1024 elements (heads of 64 or 128 among them) belong to 8, 16 or
// 32 lanes of a warp and need no block-wide step; longer rows to a CTA.
#include "common.cuh"
#include "launch.h"
#include "quant_core.cuh"
#include "tc_util.cuh"

namespace nvfp4 {

namespace {

enum { OUT_BF16 = 0, OUT_E4M3 = 1, OUT_NVFP4 = 2, OUT_STATS = 3 };
enum { RES_NONE = 0, RES_BF16 = 1, RES_F32 = 2 };

struct NormArgs {
  const uint16_t* x;
  const uint16_t* weight;
  const void* residual;
  void* residual_out;
  int64_t x_stride;    // elements between tokens
  int64_t y_stride;
  int rows;            // tokens * heads
  int heads;
  int K;
  float eps;
  float offset;
  void* out;           // bf16 rows, or codes
  void* scales;        // fp32 [rows] (E4M3), block scales (NVFP4)
  const float* s_t;    // NVFP4 with a given tensor scale
  float* row_r;        // OUT_STATS: r of each row
  unsigned int* partial;  // OUT_STATS: largest |y| (fp32 bits) of each CTA's rows
  int64_t cols4;       // block-scale columns with their padding (MMA layout)
  int rows_p;          // rows with their padding (MMA layout; else rows)
  int mma;             // block scales in the MMA layout
};

// Byte of (row, 0) in the block scales, and the step from one column tile of four to the next.
NVFP4_DEV int64_t mma_row_offset(int row, int64_t cols4) {
  return static_cast<int64_t>(row >> 7) * (cols4 >> 2) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

NVFP4_DEV void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(w[e] << 16);
    v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

NVFP4_DEV uint4 pack8(const float (&v)[8]) {
  return make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                    f32x2_to_bf16x2(v[6], v[7]));
}

// The raw words of eight elements of a row: x, and the residual's.
template <int RES>
struct Raw {
  uint4 x;
  uint4 r[RES == RES_F32 ? 2 : 1];
};

template <int RES>
NVFP4_DEV void load_raw(const uint16_t* x, const void* residual, int64_t at, Raw<RES>& raw) {
  raw.x = __ldcs(reinterpret_cast<const uint4*>(x));
  if (RES == RES_BF16) raw.r[0] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(residual) + at));
  if (RES == RES_F32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(residual) + at);
    raw.r[0] = __ldcs(p);
    raw.r[RES == RES_F32 ? 1 : 0] = __ldcs(p + 1);
  }
}

// s of eight elements, stored to residual_out on the way.
template <int RES>
NVFP4_DEV void stream8(const Raw<RES>& raw, void* residual_out, int64_t at, float (&s)[8]) {
  unpack8(raw.x, s);
  if (RES == RES_BF16) {
    float r[8];
    unpack8(raw.r[0], r);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += r[e];
    const uint4 u = pack8(s);   // 24 bits hold the sum of two bf16 well enough for one rounding to be exact
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(residual_out) + at) = u;
    unpack8(u, s);
  }
  if (RES == RES_F32) {
    const uint32_t w[8] = {raw.r[0].x, raw.r[0].y, raw.r[0].z, raw.r[0].w, raw.r[RES == RES_F32 ? 1 : 0].x,
                           raw.r[RES == RES_F32 ? 1 : 0].y, raw.r[RES == RES_F32 ? 1 : 0].z,
                           raw.r[RES == RES_F32 ? 1 : 0].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += __uint_as_float(w[e]);
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(residual_out) + at);
    p[0] = make_float4(s[0], s[1], s[2], s[3]);
    p[1] = make_float4(s[4], s[5], s[6], s[7]);
  }
}

// t = s * gain
NVFP4_DEV void gain8(const uint16_t* weight, float offset, int k, float (&s)[8]) {
  if (weight) {
    float w[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(weight + k)), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] *= w[e] + offset;
  }
}

NVFP4_DEV float amax8(const float (&t)[8]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(t[e]));
  return m;
}

// The gain of eight columns, and t from it.
NVFP4_DEV void gain_of(const uint16_t* weight, float offset, int k, float (&g)[8]) {
  if (weight) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(weight + k)), g);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] += offset;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = 1.f;
  }
}

// Codes and block scale of eight elements of a block whose other eight are in
// the neighbouring lane (lanes 2j, 2j + 1; both run this): the decisions of
// the quantiser on y.
struct TensorScale {
  float st, d, rdh, rdl;
};

NVFP4_DEV TensorScale tensor_scale(float st) {
  TensorScale ts;
  ts.st = st;
  ts.d = __fmul_rn(st, 6.0f);
  recip_brackets(ts.d, ts.rdh, ts.rdl);
  return ts;
}

NVFP4_DEV uint32_t quant8(const float (&y)[8], const TensorScale& ts, uint32_t& scale) {
  float ab = amax8(y);
  ab = fmaxf(ab, __shfl_xor_sync(3u << (threadIdx.x & 30), ab, 1));
  scale = block_scale_code(ab, ts.d, ts.rdh, ts.rdl);
  if (scale == 0) return 0u;
  return e2m1x8(y, __fmul_rn(e4m3_to_f32(scale), ts.st));
}

// The E4M3 scale a of a row. Codes come from y * lift, den = a * lift and 1 / den.
struct RowScale {
  float a, lift, den, inv;
};

// Writes eight elements of y = t * r (k: their first column).
template <int OUT>
NVFP4_DEV void store8(const NormArgs& a, int row, int64_t y_at, int k, float (&t)[8], float r, const RowScale& rs, const TensorScale* ts) {
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] *= r;
  if (OUT == OUT_BF16) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + y_at + k) = pack8(t);
  if (OUT == OUT_E4M3) {
    if (rs.lift != 1.0f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] *= rs.lift;
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + static_cast<int64_t>(row) * a.K + k) = e4m3x8(t, rs.den, rs.inv);
  }
  if (OUT == OUT_NVFP4) {
    uint32_t sc;
    const uint32_t codes = quant8(t, *ts, sc);
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + (static_cast<int64_t>(row) * a.K + k) / 2) = codes;
    const int b = k >> 4;
    if ((k & 8) == 0)
      static_cast<uint8_t*>(a.scales)[a.mma ? mma_row_offset(row, a.cols4) + (b >> 2) * 512 + (b & 3)
                                            : static_cast<int64_t>(row) * (a.K >> 4) + b] = static_cast<uint8_t>(sc);
  }
}

// The scale columns behind the last block of a row, and the rows behind the last one, are zero (MMA layout).
NVFP4_DEV void pad_scales(const NormArgs& a, int row, int first, int lane, int lanes) {
  uint8_t* p = static_cast<uint8_t*>(a.scales) + mma_row_offset(row, a.cols4);
  for (int c = first + lane; c < a.cols4; c += lanes) p[static_cast<int64_t>(c >> 2) * 512 + (c & 3)] = 0;
}

// The row's E4M3 scale a = max|y| / 448 (1 for a row of zeros; 2^-120 at least, so that 1 / a is finite). Codes are those
// of the quotients y / a: a product with 1 / a alone gives a neighbour's where a quotient is next to a border
// between two, and rows of few different values (a bf16 stream without a gain) have many quotients exactly on one.
// Rows of small values are lifted by a power of two, so that the quotient's remainder has its bits above 2^-149.
NVFP4_DEV RowScale e4m3_row_scale(float most) {
  RowScale rs;
  rs.a = most > 0.f ? fmaxf(__fdiv_rn(most, 448.0f), 0x1p-120f) : 1.0f;
  rs.lift = rs.a < 0x1p-60f ? 0x1p64f : 1.0f;
  rs.den = rs.a * rs.lift;
  rs.inv = __frcp_rn(rs.den);
  if (rs.inv == 0.f) rs.den = 0.f;   // (an infinite scale: finite values are 0 beside it)
  return rs;
}

NVFP4_DEV float rms_r(float sum, const NormArgs& a) { return rsqrtf(sum / static_cast<float>(a.K) + a.eps); }

// ---- a row for TPR lanes of a warp: K <= 8 * TPR * VPT
// ROWS of them at a time, where a row is one load of a lane: more bytes in flight (4096 x 40 heads of 128: 18.6 -> 16.8 us)
template <int OUT, int RES, int TPR, int VPT, int ROWS>
__global__ void __launch_bounds__(256) norm_lanes_kernel(const NormArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & (TPR - 1);
  const int per_cta = 256 / TPR;
  const int nvec = a.K >> 3;
  const float st = OUT == OUT_NVFP4 ? *a.s_t : 1.0f;
  float most_all = 0.f;
  // a lane's columns are the same in every row: their gain stays in registers where a lane has few (15.9 -> 15.1)
  constexpr bool KEPT = VPT <= 2;
  float gain[KEPT ? VPT : 1][8];
  if (KEPT) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (lane + i * TPR < nvec) gain_of(a.weight, a.offset, (lane + i * TPR) * 8, gain[KEPT ? i : 0]);
  }
  // (all lanes of a warp walk the same number of rows: the reductions are warp-wide)
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * (per_cta * ROWS); row0 < a.rows_p; row0 += static_cast<int64_t>(gridDim.x) * (per_cta * ROWS)) {
    Raw<RES> raw[ROWS][VPT];
    int64_t y_at[ROWS];
    bool live[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int row = static_cast<int>(row0) + j * per_cta + threadIdx.x / TPR;
      live[j] = row < a.rows;
      const int token = live[j] ? row / a.heads : 0, head = live[j] ? row - token * a.heads : 0;
      const uint16_t* xr = a.x + token * a.x_stride + static_cast<int64_t>(head) * a.K;
      y_at[j] = token * a.y_stride + static_cast<int64_t>(head) * a.K;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = lane + i * TPR;
        if (live[j] && v < nvec) load_raw<RES>(xr + v * 8, a.residual, static_cast<int64_t>(row) * a.K + v * 8, raw[j][i]);
      }
    }
    const TensorScale ts = tensor_scale(st);   // (behind the rows' loads: st is a load too)
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int row = static_cast<int>(row0) + j * per_cta + threadIdx.x / TPR;
      const int64_t base = static_cast<int64_t>(row) * a.K;
      float t[VPT][8], sum = 0.f, most = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = lane + i * TPR;
        if (live[j] && v < nvec) {
          stream8<RES>(raw[j][i], a.residual_out, base + v * 8, t[i]);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(t[i][e], t[i][e], sum);
          if (KEPT) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[i][e] *= gain[KEPT ? i : 0][e];
          } else {
            gain8(a.weight, a.offset, v * 8, t[i]);
          }
          if (OUT == OUT_E4M3 || OUT == OUT_STATS) most = fmaxf(most, amax8(t[i]));
        }
      }
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (OUT == OUT_E4M3 || OUT == OUT_STATS) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      }
      const float r = rms_r(sum, a);
      RowScale rs = {};
      if (OUT == OUT_E4M3) {
        rs = e4m3_row_scale(most * r);
        if (live[j] && lane == 0) static_cast<float*>(a.scales)[row] = rs.a;
      }
      if (OUT == OUT_STATS) {
        if (live[j] && lane == 0) a.row_r[row] = r;
        if (live[j]) most_all = fmaxf(most_all, most * r);
        continue;
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = lane + i * TPR;
        if (live[j] && v < nvec) store8<OUT>(a, row, y_at[j], v * 8, t[i], r, rs, &ts);
      }
      if (OUT == OUT_NVFP4 && a.mma && row < a.rows_p) pad_scales(a, row, live[j] ? a.K >> 4 : 0, lane, TPR);
    }
  }
  if (OUT == OUT_STATS) {
    __shared__ unsigned int s_most;
    if (threadIdx.x == 0) s_most = 0u;
    __syncthreads();
    const unsigned int m = __reduce_max_sync(0xffffffffu, __float_as_uint(most_all));
    if ((threadIdx.x & 31) == 0) atomicMax(&s_most, m);
    __syncthreads();
    if (threadIdx.x == 0) a.partial[blockIdx.x] = s_most;
  }
}

// ---- a row for a CTA: K <= 8 * blockDim.x * VPT
template <int OUT, int RES, int VPT>
__global__ void __launch_bounds__(VPT > 1 ? 512 : 1024) norm_cta_kernel(const NormArgs a) {
  __shared__ float s_sum[2][32], s_most[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int nvec = a.K >> 3, warps = blockDim.x >> 5, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float st = OUT == OUT_NVFP4 ? *a.s_t : 1.0f;
  float most_all = 0.f;
  int turn = 0;
  // (rows of more than 16384 elements: the loads of two or four vectors at a time, as registers allow; else the next
  // row's loads are under way while this one is summed and stored)
  constexpr int AT_ONCE = VPT < 8 ? VPT : RES == RES_F32 ? 2 : 4;
  Raw<RES> raw[AT_ONCE];
  auto load_row = [&](int row, int i0) {
    const int token = row / a.heads, head = row - token * a.heads;
    const uint16_t* xr = a.x + token * a.x_stride + static_cast<int64_t>(head) * a.K;
    const int64_t base = static_cast<int64_t>(row) * a.K;
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int v = threadIdx.x + (i0 + i) * blockDim.x;
      if (v < nvec) load_raw<RES>(xr + v * 8, a.residual, base + v * 8, raw[i]);
    }
  };
  if (AT_ONCE == VPT && blockIdx.x < a.rows) load_row(blockIdx.x, 0);
  for (int row = blockIdx.x; row < a.rows_p; row += gridDim.x, turn ^= 1) {
    if (row >= a.rows) {   // padding rows of the block scales (whole CTAs)
      pad_scales(a, row, 0, threadIdx.x, blockDim.x);
      continue;
    }
    const int token = row / a.heads, head = row - token * a.heads;
    const int64_t base = static_cast<int64_t>(row) * a.K;
    float t[VPT][8], sum = 0.f, most = 0.f;
#pragma unroll
    for (int i0 = 0; i0 < VPT; i0 += AT_ONCE) {
      if (AT_ONCE < VPT) load_row(row, i0);
#pragma unroll
      for (int i = i0; i < i0 + AT_ONCE; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          stream8<RES>(raw[i - i0], a.residual_out, base + v * 8, t[i]);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(t[i][e], t[i][e], sum);
          gain8(a.weight, a.offset, v * 8, t[i]);
          if (OUT == OUT_E4M3 || OUT == OUT_STATS) most = fmaxf(most, amax8(t[i]));
        }
      }
    }
    if (AT_ONCE == VPT && row + gridDim.x < a.rows) load_row(row + gridDim.x, 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (OUT == OUT_E4M3 || OUT == OUT_STATS) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    const TensorScale ts = tensor_scale(st);   // (behind the row's loads: st is a load too)
    // (two sets of slots in turn: a warp that is a row ahead does not overwrite what a slower one still reads)
    if (lane == 0) {
      s_sum[turn][warp] = sum;
      s_most[turn][warp] = most;
    }
    __syncthreads();
    sum = lane < warps ? s_sum[turn][lane] : 0.f;
    most = lane < warps ? s_most[turn][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (OUT == OUT_E4M3 || OUT == OUT_STATS) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    const float r = rms_r(sum, a);
    RowScale rs = {};
    if (OUT == OUT_E4M3) {
      rs = e4m3_row_scale(most * r);
      if (threadIdx.x == 0) static_cast<float*>(a.scales)[row] = rs.a;
    }
    if (OUT == OUT_STATS) {
      if (threadIdx.x == 0) a.row_r[row] = r;
      most_all = fmaxf(most_all, most * r);
      continue;
    }
    const int64_t y_at = token * a.y_stride + static_cast<int64_t>(head) * a.K;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) store8<OUT>(a, row, y_at, v * 8, t[i], r, rs, &ts);
    }
    if (OUT == OUT_NVFP4 && a.mma) pad_scales(a, row, a.K >> 4, threadIdx.x, blockDim.x);
  }
  if (OUT == OUT_STATS && threadIdx.x == 0) a.partial[blockIdx.x] = __float_as_uint(most_all);
}

// ---- the codes of a tensor whose scale had to be found first: y = s * (w + offset) * r is formed again
// from the stream (or x) and each row's r, so both passes see the same y. A lane takes a block of 16, a warp 32
// blocks of a row at a time, two such chunks in flight; the block step's constants come from tables, as in
// the quantiser (4096 x 5120 from DRAM: rows of a CTA, halves of blocks and formed reciprocals 33.8 us; blocks 23.5; with
// the gain in registers 20.9).
template <bool F32>
struct RawBlock {
  uint4 w[F32 ? 4 : 2];
};

// (ordinary loads: the stream was written by the statistics pass, beside which this grid may start)
template <bool F32>
NVFP4_DEV void load_block(const void* s, int64_t at, RawBlock<F32>& r) {
  const uint4* p = F32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(s) + at)
                       : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(s) + at);
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 2); ++i) r.w[i] = p[i];
}

template <bool F32>
NVFP4_DEV void unpack_block(const RawBlock<F32>& r, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 2); ++i) {
    const uint32_t u[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (F32) {
        v[4 * i + e] = __uint_as_float(u[e]);
      } else {
        v[8 * i + 2 * e] = __uint_as_float(u[e] << 16);
        v[8 * i + 2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
      }
    }
  }
}

constexpr int encode_ctas(bool f32) { return f32 ? 3 : 4; }   // of an SM

template <bool F32>
__global__ void __launch_bounds__(256, encode_ctas(F32)) norm_encode_kernel(const NormArgs a, const void* s, int64_t s_stride, int n_partial,
                                                          float* s_t) {
  __shared__ unsigned int s_most;
  __shared__ QuantTables tab;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int bpr = a.K >> 4, cpr = (bpr + 31) >> 5;
  const int64_t chunks = static_cast<int64_t>(a.rows) * cpr, step = static_cast<int64_t>(gridDim.x) * 8;
  int64_t chunk = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  struct At {
    int row, block;
  };
  auto at_chunk = [&](int64_t c) {
    const int row = static_cast<int>(c / cpr);
    return At{row, static_cast<int>(c - static_cast<int64_t>(row) * cpr) * 32 + lane};
  };
  auto load = [&](const At& p, RawBlock<F32>& raw, float& r) {
    if (p.block >= bpr) return;
    const int token = p.row / a.heads, head = p.row - token * a.heads;
    load_block<F32>(s, token * s_stride + static_cast<int64_t>(head) * a.K + p.block * 16, raw);
    r = a.row_r[p.row];
  };
  RawBlock<F32> raw = {}, next = {};
  float r = 0.f, next_r = 0.f;
  At at = {0, bpr};
  if (chunk < chunks) load(at = at_chunk(chunk), raw, r);
  if (threadIdx.x == 0) s_most = 0u;
  __syncthreads();
  unsigned int m = 0u;
  for (int i = threadIdx.x; i < n_partial; i += blockDim.x) m = max(m, __ldcg(a.partial + i));
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) atomicMax(&s_most, m);
  __syncthreads();
  const float amax = __uint_as_float(s_most);
  const TensorScale ts = tensor_scale(amax > 0.f ? __fdiv_rn(amax, 2688.0f) : 1.0f);
  if (blockIdx.x == 0 && threadIdx.x == 0) *s_t = ts.st;
  quant_tables_init(tab, ts.st);
  // a warp's chunks all lie in the same columns (the grid's step is whole rows): their gain stays in registers
  uint64_t gain[8];
  {
    float g[16];
    if (a.weight && at.block < bpr) {
      RawBlock<false> w;
      load_block<false>(a.weight, at.block * 16, w);
      unpack_block<false>(w, g);
    }
#pragma unroll
    for (int e = 0; e < 16; e += 2) gain[e / 2] = a.weight ? f32_pair(g[e] + a.offset, g[e + 1] + a.offset) : f32_pair(1.f, 1.f);
  }
  __syncthreads();
  for (; chunk < chunks; chunk += step) {
    At then = {0, bpr};
    if (chunk + step < chunks) load(then = at_chunk(chunk + step), next, next_r);
    if (at.block < bpr) {
      float t[16], most = 0.f;
      unpack_block<F32>(raw, t);
      const uint64_t rr = f32_pair(r, r);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const uint64_t y = mul_f32x2(mul_f32x2(f32_pair(t[e], t[e + 1]), gain[e / 2]), rr);
        t[e] = __uint_as_float(static_cast<uint32_t>(y));
        t[e + 1] = __uint_as_float(static_cast<uint32_t>(y >> 32));
        most = fmaxf(most, fmaxf(fabsf(t[e]), fabsf(t[e + 1])));
      }
      uint2 codes;
      const uint32_t sc = quant_block16_tab(t, most, ts.d, ts.rdh, ts.rdl, tab, codes);
      reinterpret_cast<uint2*>(a.out)[static_cast<int64_t>(at.row) * bpr + at.block] = codes;
      static_cast<uint8_t*>(a.scales)[a.mma ? mma_row_offset(at.row, a.cols4) + (at.block >> 2) * 512 + (at.block & 3)
                                            : static_cast<int64_t>(at.row) * bpr + at.block] = static_cast<uint8_t>(sc);
    }
    at = then;
    raw = next;
    r = next_r;
  }
  if (a.mma)   // the layout's padding
    for (int row = blockIdx.x; row < a.rows_p; row += gridDim.x) pad_scales(a, row, row < a.rows ? bpr : 0, threadIdx.x, blockDim.x);
}

constexpr int PARTIALS = 2048;   // CTAs of a statistics pass at most

// Launches the kernel for the rows' length; `grid` says how many CTAs it had.
template <int OUT, int RES>
int launch_rows(const NormArgs& a, int* grid, cudaStream_t stream) {
  const int nvec = a.K / 8;
  if (a.K <= 1024) {
    const int most = OUT == OUT_STATS ? PARTIALS : 1 << 30;
    const int tpr = nvec <= 8 ? 8 : nvec <= 16 ? 16 : 32, vpt = static_cast<int>(ceil_div(nvec, tpr));
    // several rows at a time only where the CTAs fill the SMs all the same
    const bool many = vpt == 1 && a.rows_p >= static_cast<int64_t>(sm_count()) * 8 * (256 / tpr) * 4;
    const int64_t want = ceil_div(a.rows_p, 256 / tpr * (many ? 4 : 1));
    *grid = static_cast<int>(want < most ? want : most);
#define NVFP4_LANES(T, V, R) \
  return launch_ex(norm_lanes_kernel<OUT, RES, T, V, R>, dim3(*grid), dim3(256), 0, 1, true, stream, a)
    if (tpr == 8 && many) NVFP4_LANES(8, 1, 4);
    if (tpr == 8) NVFP4_LANES(8, 1, 1);
    if (tpr == 16 && many) NVFP4_LANES(16, 1, 4);
    if (tpr == 16) NVFP4_LANES(16, 1, 1);
    if (vpt == 1 && many) NVFP4_LANES(32, 1, 4);
    if (vpt == 1) NVFP4_LANES(32, 1, 1);
    if (vpt == 2) NVFP4_LANES(32, 2, 1);
    NVFP4_LANES(32, 4, 1);
#undef NVFP4_LANES
  }
  // fewer rows than SMs: as many threads as a row has vectors of eight (32 x 5120: 2.5 us; two vectors a thread
  // 2.6, four 3.0); more: two a thread (512 x 5120: 5.8 us; one 8.5, four 6.9; 8192 x 5120, a row for a CTA: 55; 108;
  // 57), and four for the statistics pass, whose CTAs take several rows
  const int vpt = nvec > 2048 ? 8 : nvec > 1024 ? 4 : a.rows >= sm_count() ? (OUT == OUT_STATS ? 4 : 2) : 1;
  const int threads = static_cast<int>(ceil_div(ceil_div(nvec, vpt), 32) * 32);
  // two rows to a CTA where that leaves eight CTAs an SM to start with (8192 x 5120: 54.5 -> 52.0 us; 2048 x 16384, fp32
  // stream: 67 -> 63.5); the statistics pass as many as four CTAs an SM take (4096 x 5120 with the rest: 66 -> 62.7)
  const int sms = sm_count();
  *grid = OUT == OUT_STATS ? (a.rows_p < 4 * sms ? a.rows_p : 4 * sms) : a.rows_p >= 8 * sms ? (a.rows_p + 1) / 2 : a.rows_p;
#define NVFP4_CTA(V) return launch_ex(norm_cta_kernel<OUT, RES, V>, dim3(*grid), dim3(threads), 0, 1, true, stream, a)
  if (vpt == 1) NVFP4_CTA(1);
  if (vpt == 2) NVFP4_CTA(2);
  if (vpt == 4) NVFP4_CTA(4);
  NVFP4_CTA(8);
#undef NVFP4_CTA
}

template <int OUT>
int launch_out(const NormArgs& a, int res, int* grid, cudaStream_t stream) {
  if (res == RES_NONE) return launch_rows<OUT, RES_NONE>(a, grid, stream);
  if (res == RES_BF16) return launch_rows<OUT, RES_BF16>(a, grid, stream);
  return launch_rows<OUT, RES_F32>(a, grid, stream);
}

int res_of(const nvfp4_norm_t& n) {
  return !n.residual ? RES_NONE : n.residual_dtype == NVFP4_DTYPE_F32 ? RES_F32 : RES_BF16;
}

NormArgs args_of(const nvfp4_norm_t& n) {
  NormArgs a = {};
  a.x = static_cast<const uint16_t*>(n.x);
  a.weight = static_cast<const uint16_t*>(n.weight);
  a.residual = n.residual;
  a.residual_out = n.residual_out;
  a.x_stride = n.x_stride;
  a.heads = n.heads;
  a.rows = static_cast<int>(n.tokens * n.heads);
  a.rows_p = a.rows;
  a.K = n.K;
  a.eps = n.eps;
  a.offset = n.weight_offset;
  return a;
}

}  // namespace

size_t norm_workspace_bytes(int64_t rows) { return PARTIALS * sizeof(unsigned int) + static_cast<size_t>(rows) * sizeof(float); }

int launch_rms_norm(const nvfp4_norm_t& n, void* y, int64_t y_stride, cudaStream_t stream) {
  NormArgs a = args_of(n);
  a.out = y;
  a.y_stride = y_stride;
  int grid;
  return launch_out<OUT_BF16>(a, res_of(n), &grid, stream);
}

int launch_rms_norm_e4m3(const nvfp4_norm_t& n, uint8_t* codes, float* scales, cudaStream_t stream) {
  NormArgs a = args_of(n);
  a.out = codes;
  a.scales = scales;
  int grid;
  return launch_out<OUT_E4M3>(a, res_of(n), &grid, stream);
}

int launch_rms_norm_quantize(const nvfp4_norm_t& n, uint8_t* codes, uint8_t* scales, float* s_t, int s_t_mode,
                             int scale_layout, void* workspace, cudaStream_t stream) {
  NormArgs a = args_of(n);
  a.out = codes;
  a.scales = scales;
  a.mma = scale_layout == NVFP4_SCALES_MMA;
  a.cols4 = mma_scale_cols(n.K);
  const int rows_p = a.mma ? static_cast<int>(mma_scale_rows(a.rows)) : a.rows;
  int grid;
  if (s_t_mode == NVFP4_ST_GIVEN) {
    a.s_t = s_t;
    a.rows_p = rows_p;
    return launch_out<OUT_NVFP4>(a, res_of(n), &grid, stream);
  }
  a.partial = static_cast<unsigned int*>(workspace);
  a.row_r = reinterpret_cast<float*>(a.partial + PARTIALS);
  grid = 0;
  if (a.rows > 0)
    if (int rc = launch_out<OUT_STATS>(a, res_of(n), &grid, stream)) return rc;
  a.rows_p = rows_p;
  const int res = res_of(n);
  const void* s = res == RES_NONE ? n.x : n.residual_out;
  const int64_t s_stride = res == RES_NONE ? n.x_stride : static_cast<int64_t>(n.heads) * n.K;
  const int cpr = static_cast<int>(ceil_div(n.K / 16, 32));   // a row's chunks of 32 blocks, one for a warp
  const int64_t chunks = static_cast<int64_t>(rows_p) * cpr;
  const int most = encode_ctas(res_of(n) == RES_F32) * sm_count();
  int ctas = static_cast<int>(chunks < 8 ? 1 : chunks < 8ll * most ? ceil_div(chunks, 8) : most);
  // where a warp takes several chunks, its step is whole rows (cpr is 64 at most)
  int unit = cpr;
  for (int i = 0; i < 3 && unit % 2 == 0; ++i) unit /= 2;
  if (chunks > 8ll * ctas) ctas -= ctas % unit;
  return res == RES_F32
             ? launch_ex(norm_encode_kernel<true>, dim3(ctas), dim3(256), 0, 1, true, stream, a, s, s_stride, grid, s_t)
             : launch_ex(norm_encode_kernel<false>, dim3(ctas), dim3(256), 0, 1, true, stream, a, s, s_stride, grid, s_t);
}

}  // namespace nvfp4
