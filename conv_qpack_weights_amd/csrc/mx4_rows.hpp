// mx4_rows.hpp -- the products with MXFP4 weights for few rows: of float rows or
// MXFP4 rows, instantiated per row type.
//
//   y[r,n] = clamp(sum_k x[r,k] w[n,k] + bias[n], lo, hi)
//
// One pass over the weights is the floor (17/32 of a byte each).  A workgroup
// owns kTiles 16-channel tiles and 16 kFM rows; its waves share out K in runs of
// 128-K blocks, everything straight from memory into registers, and their sums
// meet in LDS in a fixed order.  Lane l's 16 bytes of a block are channel l%16's
// values of 32-block l/16: one operand of the scaled 4-bit MFMA, or, word t of
// them with the rows' elements 32 (l/16) + 8t .. + 7, of four bf16 MFMAs (which
// of the block's K meet in which MFMA does not matter to the sum).
#pragma once

#include "mx4.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

// One block's operands of a wave.
template <typename T, int kFM, int kTiles>
struct MxStage {
  u32x4 q[kTiles];
  uint32_t s[kTiles];
  MxFrag<T> x[kFM][4];
};
template <int kFM, int kTiles>
struct MxStage<mx4_t, kFM, kTiles> {
  u32x4 q[kTiles];
  uint32_t s[kTiles];
  u32x4 x[kFM];
  uint32_t xs[kFM];
};

// s, xs: the words of four scales, of which the lane's is byte `quad`
template <typename T, int kFM, int kTiles>
__device__ __forceinline__ void mx_step(const MxStage<T, kFM, kTiles>& st, int quad,
                                        f32x4 (&acc)[kFM][kTiles]) {
  if constexpr (__is_same(T, mx4_t)) {
    uint32_t xs[kFM];
#pragma unroll
    for (int f = 0; f < kFM; ++f) xs[f] = st.xs[f] >> (8 * quad);
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      const uint32_t s = st.s[c] >> (8 * quad);
#pragma unroll
      for (int f = 0; f < kFM; ++f)
        acc[f][c] = mx_mfma16(st.x[f], xs[f], st.q[c], s, acc[f][c]);
    }
  } else {
    constexpr int NP = MxFrag<T>::kPieces;
    float s[kTiles];
#pragma unroll
    for (int c = 0; c < kTiles; ++c) s[c] = mx_scale((st.s[c] >> (8 * quad)) & 0xffu);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      bf16x8 wv[kTiles];
#pragma unroll
      for (int c = 0; c < kTiles; ++c) wv[c] = mx_unpack(st.q[c][t], s[c]);
#pragma unroll
      for (int f = 0; f < kFM; ++f) {
        bf16x8 xv[NP];
        st.x[f][t].split(xv);
#pragma unroll
        for (int c = 0; c < kTiles; ++c)
#pragma unroll
          for (int i = 0; i < NP; ++i) acc[f][c] = mfma32(xv[i], wv[c], acc[f][c]);
      }
    }
  }
}

template <typename T, int kFM, int kTiles, int kWaves, int kAhead>
__global__ __launch_bounds__(kWaves * 64) void mx_rows_kernel(MxArgs a, uint32_t row_slots) {
  constexpr bool kA4 = __is_same(T, mx4_t);
  __shared__ f32x4 red[kWaves][kFM * kTiles][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the row tiles of a channel group next to each other, so that an expert's
  // weights cross the fabric once for all of them
  const uint32_t id = xcd_run(blockIdx.x, gridDim.x);
  const uint32_t group = id / row_slots, slot = id - group * row_slots;
  const W4Tile tile = w4_find_tile<16 * kFM>(a.rows, slot);
  if (tile.expert < 0) return;
  const int64_t n0 = (int64_t)group * kTiles * 16;
  const int64_t N = a.w.rows;
  if (a.rows.offsets && tile.expert == a.rows.experts) {  // rows of no expert
    for (int64_t i = threadIdx.x; i < (tile.r1 - tile.r0) * 16 * kTiles; i += kWaves * 64) {
      const int64_t r = tile.r0 + i / (16 * kTiles), n = n0 + i % (16 * kTiles);
      if (n < N) w4_store(a.Y, a.y_dtype, r * a.ldy + n, 0.0f);
    }
    return;
  }
  const int ch = lane & 15, quad = lane >> 4;

  // rows past the tile's end repeat its last row, channels past the last one that
  // one: their results are not stored
  const uint8_t *wq[kTiles], *ws[kTiles];
#pragma unroll
  for (int c = 0; c < kTiles; ++c) {
    int64_t n = n0 + c * 16 + ch;
    n = n < N ? n : N - 1;
    wq[c] = a.w.codes + tile.expert * a.w.cstride + n * a.w.ldc + quad * 16;
    ws[c] = a.w.scales + tile.expert * a.w.sstride + n * a.w.lds;
  }
  const uint8_t *xr[kFM], *xs[kFM];
#pragma unroll
  for (int f = 0; f < kFM; ++f) {
    int64_t r = tile.r0 + f * 16 + ch;
    r = r < tile.r1 ? r : tile.r1 - 1;
    int64_t x = w4_source_row(a.rows, r);
    x = x < 0 ? 0 : x;
    if constexpr (kA4) {
      xr[f] = a.a.codes + x * a.a.ldc + quad * 16;
      xs[f] = a.a.scales + x * a.a.lds;
    } else {
      xr[f] = static_cast<const uint8_t*>(a.X) + (x * a.ldx + 32 * quad) * (int64_t)sizeof(T);
      xs[f] = nullptr;
    }
  }

  f32x4 acc[kFM][kTiles];
#pragma unroll
  for (int f = 0; f < kFM; ++f)
#pragma unroll
    for (int c = 0; c < kTiles; ++c) acc[f][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  using Stage = MxStage<T, kFM, kTiles>;
  auto load = [&](Stage& st, int64_t b) {
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      st.q[c] = *reinterpret_cast<const u32x4*>(wq[c] + b * 64);
      st.s[c] = *reinterpret_cast<const uint32_t*>(ws[c] + b * 4);
    }
#pragma unroll
    for (int f = 0; f < kFM; ++f) {
      if constexpr (kA4) {
        st.x[f] = *reinterpret_cast<const u32x4*>(xr[f] + b * 64);
        st.xs[f] = *reinterpret_cast<const uint32_t*>(xs[f] + b * 4);
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
          st.x[f][t].load(reinterpret_cast<const T*>(xr[f]) + b * 128 + t * 8);
      }
    }
  };

  // whole blocks, a run per wave; the cut block at the end of K is the last wave's
  const int64_t full = a.w.K / 128;
  const int64_t per = (full + kWaves - 1) / kWaves;
  const int64_t b0 = wave * per < full ? wave * per : full;
  const int64_t b1 = b0 + per < full ? b0 + per : full;
  if (b0 < b1) {
    Stage st[kAhead];
#pragma unroll
    for (int p = 0; p < kAhead; ++p) load(st[p], b0 + p < b1 ? b0 + p : b1 - 1);
    int64_t b = b0;
    for (; b + kAhead < b1; b += kAhead) {
#pragma unroll
      for (int p = 0; p < kAhead; ++p) {
        mx_step<T, kFM, kTiles>(st[p], quad, acc);
        const int64_t nb = b + p + kAhead;
        load(st[p], nb < b1 ? nb : b1 - 1);
      }
    }
#pragma unroll
    for (int p = 0; p < kAhead; ++p)  // (no load behind a branch: its join would wait)
      if (b + p < b1) mx_step<T, kFM, kTiles>(st[p], quad, acc);
  }
  if (wave == kWaves - 1 && full * 128 < a.w.K) {
    // 32-blocks past the row's last one: zero codes and scale (a scale found there
    // could be a NaN), read from the row's start
    Stage st;
    const bool in = 4 * full + quad < a.w.G;
    const int64_t at = in ? full * 64 : -quad * 16;
    const u32x4 none = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      const u32x4 q = *reinterpret_cast<const u32x4*>(wq[c] + at);
      const uint32_t s = *reinterpret_cast<const uint32_t*>(ws[c] + full * 4);
      st.q[c] = in ? q : none;
      st.s[c] = in ? s : 0u;
    }
#pragma unroll
    for (int f = 0; f < kFM; ++f) {
      if constexpr (kA4) {
        const u32x4 q = *reinterpret_cast<const u32x4*>(xr[f] + at);
        const uint32_t s = *reinterpret_cast<const uint32_t*>(xs[f] + full * 4);
        st.x[f] = in ? q : none;
        st.xs[f] = in ? s : 0u;
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int64_t left = a.w.K - (full * 128 + 32 * quad + 8 * t);
          const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
          const T* row = reinterpret_cast<const T*>(xr[f]);
          st.x[f][t].load_n(n > 0 ? row + full * 128 + 8 * t : row - 32 * quad, n);
        }
      }
    }
    mx_step<T, kFM, kTiles>(st, quad, acc);
  }

#pragma unroll
  for (int f = 0; f < kFM; ++f)
#pragma unroll
    for (int c = 0; c < kTiles; ++c) red[wave][f * kTiles + c][lane] = acc[f][c];
  __syncthreads();
  // thread: row m of 16 in a fragment, channel n of 16
  for (int i = threadIdx.x; i < kFM * kTiles * 256; i += kWaves * 64) {
    const int frag = i >> 8, m = (i >> 4) & 15, n = i & 15;
    const int64_t r = tile.r0 + (frag / kTiles) * 16 + m;
    const int64_t col = n0 + (frag % kTiles) * 16 + n;
    if (r >= tile.r1 || col >= N) continue;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) y += red[w][frag][(m >> 2) * 16 + n][m & 3];
    if (w4_source_row(a.rows, r) < 0) y = 0.0f;
    if (a.bias) y += a.bias[tile.expert * N + col];
    y = y < a.lo ? a.lo : y;
    y = y > a.hi ? a.hi : y;
    w4_store(a.Y, a.y_dtype, r * a.ldy + col, y);
  }
}

template <typename T, int kFM, int kTiles, int kWaves, int kAhead>
qp_status mx_launch_rows(const MxArgs& a, hipStream_t stream) {
  const int64_t groups = ceil_div(a.w.rows, 16 * kTiles), slots = w4_tile_slots(a.rows, 16 * kFM);
  QP_REQUIRE(slots * groups * kWaves * 64 < (INT64_C(1) << 32), QP_EUNSUPPORTED,
             "qgemm_mx: rows and channels for more than 2^32 threads");
  hipLaunchKernelGGL((mx_rows_kernel<T, kFM, kTiles, kWaves, kAhead>),
                     dim3((unsigned)(slots * groups)), dim3(kWaves * 64), 0, stream, a,
                     (uint32_t)slots);
  return check_launch("qgemm_mx (few rows)");
}

}  // namespace
}  // namespace qp
