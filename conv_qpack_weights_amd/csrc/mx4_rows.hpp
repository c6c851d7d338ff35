// mx4_rows.hpp -- the products with MXFP4 weights for few rows, operands straight from
// memory: of f32 rows, and of the 16-bit and MXFP4 rows that the direct loads of
// mx4_stream.hpp cannot take (rows at odd addresses, or too far apart).
//
//   y[r,n] = clamp(sum_k x[r,k] w[n,k] + bias[n], lo, hi)
//
// One pass over the weights is the floor (17/32 of a byte each).  A workgroup
// owns kTiles 16-channel tiles and 16 rows; its waves share out K in runs of
// 128-K blocks, everything straight from memory into registers, and their sums
// meet in LDS in a fixed order.  Lane l's 16 bytes of a block are channel l%16's
// values of 32-block l/16: one operand of the scaled 4-bit MFMA, or, word t of
// them with the rows' elements 32 (l/16) + 8t .. + 7, of four bf16 MFMAs (which
// of the block's K meet in which MFMA does not matter to the sum).
//
// A row's four scales of a block come in words, for four blocks at a time 16 bytes: a
// load of 16 rows looks up 16 lines, however few bytes of each it takes, and those
// look-ups bound the kernel (16 x 11008 x 4096 f32 19.6 us by 48 channels, 38 by 16).
// f32 rows are three bf16 pieces, each product of a piece exact.
#pragma once

#include "mx4.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

// One block's operands of a wave.
template <typename T, int kTiles>
struct MxStage {
  u32x4 q[kTiles];
  uint32_t s[kTiles];
  MxFrag<T> x[4];
};
template <int kTiles>
struct MxStage<mx4_t, kTiles> {
  u32x4 q[kTiles];
  uint32_t s[kTiles];
  u32x4 x;
  uint32_t xs;
};

// s, xs: the words of four scales, of which the lane's is byte `quad`
template <typename T, int kTiles>
__device__ __forceinline__ void mx_step(const MxStage<T, kTiles>& st, int quad,
                                        f32x4 (&acc)[kTiles]) {
  if constexpr (__is_same(T, mx4_t)) {
    const uint32_t xs = st.xs >> (8 * quad);
#pragma unroll
    for (int c = 0; c < kTiles; ++c)
      acc[c] = mx_mfma16(st.x, xs, st.q[c], st.s[c] >> (8 * quad), acc[c]);
  } else {
    constexpr int NP = MxFrag<T>::kPieces;
    float s[kTiles];
#pragma unroll
    for (int c = 0; c < kTiles; ++c) s[c] = mx_scale((st.s[c] >> (8 * quad)) & 0xffu);
    if constexpr (__is_same(T, f16_t)) {
      // f16 rows as they are where all the weights are f16 values (see mx_f16_scale)
      bool fit = true;
#pragma unroll
      for (int c = 0; c < kTiles; ++c) fit = fit && mx_f16_scale(s[c]);
      if (__all(fit)) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int c = 0; c < kTiles; ++c) {
            const f16x8 w = mx_unpack_f16(st.q[c][t], s[c]);
            acc[c] = mfma32(__builtin_bit_cast(f16x8, st.x[t].v), w, acc[c]);
          }
        return;
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      bf16x8 wv[kTiles];
#pragma unroll
      for (int c = 0; c < kTiles; ++c) wv[c] = mx_unpack(st.q[c][t], s[c]);
      bf16x8 xv[NP];
      st.x[t].split(xv);
#pragma unroll
      for (int c = 0; c < kTiles; ++c)
#pragma unroll
        for (int i = 0; i < NP; ++i) acc[c] = mfma32(xv[i], wv[c], acc[c]);
    }
  }
}

// Rows of no expert are stored as zeros; true where the tile is of them.
template <int kTiles, int kWaves>
__device__ __forceinline__ bool mx_rows_of_none(const MxArgs& a, const W4Tile& tile, int64_t n0) {
  if (!a.rows.offsets || tile.expert != a.rows.experts) return false;
  for (int64_t i = threadIdx.x; i < (tile.r1 - tile.r0) * 16 * kTiles; i += kWaves * 64) {
    const int64_t r = tile.r0 + i / (16 * kTiles), n = n0 + i % (16 * kTiles);
    if (n < a.w.rows) w4_store(a.Y, a.y_dtype, r * a.ldy + n, 0.0f);
  }
  return true;
}

// Where a lane's operands lie: rows past the tile's end repeat its last row, channels
// past the last one that one (their results are not stored).
template <typename T, int kTiles>
struct MxSources {
  static constexpr bool kA4 = __is_same(T, mx4_t);
  const uint8_t *wq[kTiles], *ws[kTiles], *xr, *xs;
  int quad;
  __device__ __forceinline__ MxSources(const MxArgs& a, const W4Tile& tile, int64_t n0) {
    const int ch = threadIdx.x & 15;
    quad = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      int64_t n = n0 + c * 16 + ch;
      n = n < a.w.rows ? n : a.w.rows - 1;
      wq[c] = a.w.codes + tile.expert * a.w.cstride + n * a.w.ldc + quad * 16;
      ws[c] = a.w.scales + tile.expert * a.w.sstride + n * a.w.lds;
    }
    int64_t r = tile.r0 + ch;
    r = r < tile.r1 ? r : tile.r1 - 1;
    int64_t x = w4_source_row(a.rows, r);
    x = x < 0 ? 0 : x;
    if constexpr (kA4) {
      xr = a.a.codes + x * a.a.ldc + quad * 16;
      xs = a.a.scales + x * a.a.lds;
    } else {
      xr = static_cast<const uint8_t*>(a.X) + (x * a.ldx + 32 * quad) * (int64_t)sizeof(T);
      xs = nullptr;
    }
  }
  // everything of the whole 128-K block b but its scales
  __device__ __forceinline__ void load(MxStage<T, kTiles>& st, int64_t b) const {
#pragma unroll
    for (int c = 0; c < kTiles; ++c) st.q[c] = *reinterpret_cast<const u32x4*>(wq[c] + b * 64);
    if constexpr (kA4) {
      st.x = *reinterpret_cast<const u32x4*>(xr + b * 64);
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        st.x[t].load(reinterpret_cast<const T*>(xr) + b * 128 + t * 8);
    }
  }
  __device__ __forceinline__ void load_scales(MxStage<T, kTiles>& st, int64_t b) const {
#pragma unroll
    for (int c = 0; c < kTiles; ++c)
      st.s[c] = *reinterpret_cast<const uint32_t*>(ws[c] + b * 4);
    if constexpr (kA4) st.xs = *reinterpret_cast<const uint32_t*>(xs + b * 4);
  }
  // the block that K cuts.  32-blocks past the row's last one: zero codes and scale (a
  // scale found there could be a NaN), read from the row's start
  __device__ __forceinline__ void load_cut(MxStage<T, kTiles>& st, int64_t full, int64_t K,
                                           int64_t G) const {
    const bool in = 4 * full + quad < G;
    const int64_t at = in ? full * 64 : -quad * 16;
    const u32x4 none = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      const u32x4 q = *reinterpret_cast<const u32x4*>(wq[c] + at);
      const uint32_t s = *reinterpret_cast<const uint32_t*>(ws[c] + full * 4);
      st.q[c] = in ? q : none;
      st.s[c] = in ? s : 0u;
    }
    if constexpr (kA4) {
      const u32x4 q = *reinterpret_cast<const u32x4*>(xr + at);
      const uint32_t s = *reinterpret_cast<const uint32_t*>(xs + full * 4);
      st.x = in ? q : none;
      st.xs = in ? s : 0u;
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int64_t left = K - (full * 128 + 32 * quad + 8 * t);
        const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
        const T* row = reinterpret_cast<const T*>(xr);
        st.x[t].load_n(n > 0 ? row + full * 128 + 8 * t : row - 32 * quad, n);
      }
    }
  }
};

// The blocks from `b` on, one at a time, and the one that K cuts.
template <typename T, int kTiles>
__device__ __forceinline__ void mx_rows_tail(const MxArgs& a, const W4Tile& tile, int64_t n0,
                                             int64_t b, f32x4 (&acc)[kTiles]) {
  const MxSources<T, kTiles> src(a, tile, n0);
  const int64_t full = a.w.K / 128;
  MxStage<T, kTiles> st;
#pragma unroll 1
  for (; b * 128 < a.w.K; ++b) {
    if (b < full) {
      src.load(st, b);
      src.load_scales(st, b);
    } else {
      src.load_cut(st, full, a.w.K, a.w.G);
    }
    mx_step<T, kTiles>(st, src.quad, acc);
  }
}

// The waves' sums added up in order, bias, clamp, out.  red: the workgroup's LDS.
template <int kTiles, int kWaves>
__device__ __forceinline__ void mx_rows_store(const f32x4 (&acc)[kTiles], const MxArgs& a,
                                              const W4Tile& tile, int64_t n0, f32x4* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int c = 0; c < kTiles; ++c) red[(wave * kTiles + c) * 64 + lane] = acc[c];
  __syncthreads();
  // thread: row m of 16, channel n of 16 of a tile
  for (int i = threadIdx.x; i < kTiles * 256; i += kWaves * 64) {
    const int c = i >> 8, m = (i >> 4) & 15, n = i & 15;
    const int64_t r = tile.r0 + m;
    const int64_t col = n0 + c * 16 + n;
    if (r >= tile.r1 || col >= a.w.rows) continue;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      y += red[(w * kTiles + c) * 64 + (m >> 2) * 16 + n][m & 3];
    if (w4_source_row(a.rows, r) < 0) y = 0.0f;
    if (a.bias) y += a.bias[tile.expert * a.w.rows + col];
    y = y < a.lo ? a.lo : y;
    y = y > a.hi ? a.hi : y;
    w4_store(a.Y, a.y_dtype, r * a.ldy + col, y);
  }
}

template <typename T, int kTiles, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void mx_rows_kernel(MxArgs a, uint32_t row_slots) {
  constexpr bool kA4 = __is_same(T, mx4_t);
  constexpr int kGroup = 4;  // blocks at a time, as many as a load of scales has words
  __shared__ f32x4 red[kWaves * kTiles * 64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the row tiles of a channel group next to each other, so that an expert's
  // weights cross the fabric once for all of them
  const uint32_t id = xcd_run(blockIdx.x, gridDim.x);
  const uint32_t group = id / row_slots, slot = id - group * row_slots;
  const W4Tile tile = w4_find_tile<16>(a.rows, slot);
  if (tile.expert < 0) return;
  const int64_t n0 = (int64_t)group * kTiles * 16;
  if (mx_rows_of_none<kTiles, kWaves>(a, tile, n0)) return;
  const MxSources<T, kTiles> src(a, tile, n0);

  f32x4 acc[kTiles];
#pragma unroll
  for (int c = 0; c < kTiles; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // whole blocks, a run per wave; the cut block at the end of K is the last wave's.
  // Four blocks at a time, with one load for a channel's scales of all four (a load of
  // four bytes of 16 rows costs as much as one of 16).
  using Stage = MxStage<T, kTiles>;
  const int64_t full = a.w.K / 128;
  const int64_t per = (full + kWaves - 1) / kWaves;
  const int64_t b0 = wave * per < full ? wave * per : full;
  const int64_t b1 = b0 + per < full ? b0 + per : full;
  int64_t b = b0;
  typedef uint32_t words __attribute__((ext_vector_type(4), aligned(4)));
  for (; b + kGroup <= b1; b += kGroup) {
    Stage st[kGroup];
    words s[kTiles], sx;
#pragma unroll
    for (int c = 0; c < kTiles; ++c) s[c] = *reinterpret_cast<const words*>(src.ws[c] + b * 4);
    if constexpr (kA4) sx = *reinterpret_cast<const words*>(src.xs + b * 4);
#pragma unroll
    for (int g = 0; g < kGroup; ++g) src.load(st[g], b + g);
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
#pragma unroll
      for (int c = 0; c < kTiles; ++c) st[g].s[c] = s[c][g];
      if constexpr (kA4) st[g].xs = sx[g];
      mx_step<T, kTiles>(st[g], src.quad, acc);
    }
  }
  for (; b < b1; ++b) {
    Stage st;
    src.load(st, b);
    src.load_scales(st, b);
    mx_step<T, kTiles>(st, src.quad, acc);
  }
  if (wave == kWaves - 1 && full * 128 < a.w.K) {
    Stage st;
    src.load_cut(st, full, a.w.K, a.w.G);
    mx_step<T, kTiles>(st, src.quad, acc);
  }
  mx_rows_store<kTiles, kWaves>(acc, a, tile, n0, red);
}

template <typename T, int kTiles, int kWaves>
qp_status mx_launch_rows(const MxArgs& a, hipStream_t stream) {
  const int64_t groups = ceil_div(a.w.rows, 16 * kTiles), slots = w4_tile_slots(a.rows, 16);
  QP_REQUIRE(slots * groups * kWaves * 64 < (INT64_C(1) << 32), QP_EUNSUPPORTED,
             "qgemm_mx: rows and channels for more than 2^32 threads");
  hipLaunchKernelGGL((mx_rows_kernel<T, kTiles, kWaves>),
                     dim3((unsigned)(slots * groups)), dim3(kWaves * 64), 0, stream, a,
                     (uint32_t)slots);
  return check_launch("qgemm_mx (few rows)");
}

}  // namespace
}  // namespace qp
