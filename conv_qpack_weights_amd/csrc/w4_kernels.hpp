// w4_kernels.hpp -- the kernels of the weight-only int4 products (the
// mathematics and the choice between them: w4.hip), instantiated per row type
// in w4_f32.hip, w4_bf16.hip and w4_f16.hip.
#pragma once

#include <type_traits>

#include "w4.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

// The four 32-K scales (or offsets) of a channel's 128-K block: groups of 32
// have one each; a group of 64 serves two; larger groups have one in all
// (kOne).  They are kept as they come from memory until a step needs them: the
// picking apart would wait for the load right behind it.
template <bool kBf16, bool kOne>
struct W4Scales {
  using Raw = std::conditional_t<kOne, uint32_t, std::conditional_t<kBf16, u32x2, u32x4>>;
  Raw v;

  // p: the channel tile's scales (the same for the whole wave), ch: the lane's
  // channel of 16
  __device__ __forceinline__ void load(const uint8_t* p, int64_t b, int32_t group, int ch) {
    constexpr uint32_t ES = kBf16 ? 2 : 4;
    if constexpr (kOne) {
      const int64_t g = (uint32_t)b / ((uint32_t)group / 128);
      const uint8_t* at = p + ((g / 4) * 64 + (g & 3)) * ES + (uint32_t)ch * (4 * ES);
      if constexpr (kBf16)
        v = *reinterpret_cast<const uint16_t*>(at);
      else
        v = *reinterpret_cast<const uint32_t*>(at);
    } else {
      // the quad that holds the block's scales
      v = *reinterpret_cast<const Raw*>(p + (group == 64 ? b >> 1 : b) * (64 * ES) +
                                        (uint32_t)ch * (4 * ES));
    }
  }
  // of block b: without a branch
  __device__ __forceinline__ void pick(int64_t b, int32_t group, float (&s)[kOne ? 1 : 4]) const {
    if constexpr (kOne) {
      s[0] = __builtin_bit_cast(float, kBf16 ? v << 16 : v);
    } else {
      f32x4 q;
      if constexpr (kBf16) {
        const uint32_t lo = v.x, hi = v.y;
        q[0] = __builtin_bit_cast(float, lo << 16);
        q[1] = __builtin_bit_cast(float, lo & 0xffff0000u);
        q[2] = __builtin_bit_cast(float, hi << 16);
        q[3] = __builtin_bit_cast(float, hi & 0xffff0000u);
      } else {
        q = __builtin_bit_cast(f32x4, v);
      }
      const bool wide = group == 64, odd = wide && (b & 1);
      s[0] = odd ? q[2] : q[0];
      s[1] = wide ? s[0] : q[1];
      s[2] = odd ? q[3] : wide ? q[1] : q[2];
      s[3] = wide ? s[2] : q[3];
    }
  }
};

// One block's operands of a wave: kTiles channel tiles, kFM row fragments.
template <typename T, int kKind, bool kOne, int kFM, int kTiles>
struct W4Stage {
  u32x4 q[kTiles];
  W4Scales<kKind == 1, kOne> s[kTiles];
  W4Scales<false, kOne> o[kKind == 2 ? kTiles : 1];
  XFrag<T> x[kFM][4];
};

template <typename T, int kKind, bool kOne, int kFM, int kTiles>
__device__ __forceinline__ void w4_step(const W4Stage<T, kKind, kOne, kFM, kTiles>& st,
                                        int64_t b, int32_t group, f32x4 (&acc)[kFM][kTiles]) {
  using V = typename XFrag<T>::vec;
  constexpr int NP = XFrag<T>::kPieces;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 p[kFM][kTiles], sum[kFM];
  float s[kTiles][kOne ? 1 : 4], o[kKind == 2 ? kTiles : 1][kOne ? 1 : 4];
#pragma unroll
  for (int c = 0; c < kTiles; ++c) {
    st.s[c].pick(b, group, s[c]);
    if constexpr (kKind == 2) st.o[c].pick(b, group, o[c]);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    V wv[kTiles];
#pragma unroll
    for (int c = 0; c < kTiles; ++c) wv[c] = w4_unpack<V>(st.q[c][t]);
#pragma unroll
    for (int f = 0; f < kFM; ++f) {
      V xv[NP];
      st.x[f][t].split(xv);
      const bool fresh = !kOne || t == 0;
#pragma unroll
      for (int c = 0; c < kTiles; ++c) {
        f32x4 d = fresh ? zero : p[f][c];
#pragma unroll
        for (int i = 0; i < NP; ++i) d = mfma32(xv[i], wv[c], d);
        p[f][c] = d;
      }
      if constexpr (kKind == 2) {
        V ones;
#pragma unroll
        for (int i = 0; i < 8; ++i) ones[i] = (decltype(ones[0] + ones[0]))0.0625f;
        f32x4 d = fresh ? zero : sum[f];
#pragma unroll
        for (int i = 0; i < NP; ++i) d = mfma32(xv[i], ones, d);
        sum[f] = d;
      }
      if (!kOne || t == 3) {
#pragma unroll
        for (int c = 0; c < kTiles; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float a = acc[f][c][i];
            a = __builtin_fmaf(s[c][kOne ? 0 : t], p[f][c][i], a);
            if constexpr (kKind == 2) a = __builtin_fmaf(o[c][kOne ? 0 : t], sum[f][i], a);
            acc[f][c][i] = a;
          }
      }
    }
  }
}

// ---- few rows: the waves of a workgroup share out K --------------------------
// A workgroup owns kTiles 16-channel tiles and 16*kFM rows; each wave takes a
// run of 128-K blocks with kAhead of them in flight in registers (weights,
// scales and the rows' pieces, all straight from memory: a wave's rows are
// nobody else's, so LDS would only add a hop), and the waves' sums meet in LDS
// in a fixed order.  Bound by the weights' way from memory and, above some eight
// rows, by the vector instructions (13 a word to unpack, 4 a group and tile to
// rescale): 1 x 4096 x 4096 5.0 us (10.5 MB; a read of the same bytes takes 3.4),
// 16 x 11008 x 4096 f16 10 us (24.5 MB), 64 tokens x 2 of 16 experts of
// 11008 x 4096 96-100 us (454 MB, 4.6 TB/s).  kAhead = 1: two and four blocks in
// flight cost waves a SIMD and measured 1-15% slower at every shape.
template <typename T, int kKind, bool kOne, int kFM, int kTiles, int kWaves, int kAhead>
__global__ __launch_bounds__(kWaves * 64) void w4_rows_kernel(W4Args a, uint32_t row_slots) {
  __shared__ f32x4 red[kWaves][kFM * kTiles][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups go round the 8 XCDs in launch order: give each XCD a run of
  // tiles with the row tiles of a channel group next to each other, so that an
  // expert's weights cross the fabric once for all its row tiles.
  uint32_t id = blockIdx.x;
  {
    const uint32_t n = gridDim.x, per = n / 8, rest = n % 8, x = id % 8;
    id = x * per + (x < rest ? x : rest) + id / 8;
  }
  const uint32_t group = id / row_slots, slot = id - group * row_slots;
  const W4Tile tile = w4_find_tile<16 * kFM>(a.rows, slot);
  if (tile.expert < 0) return;
  const int64_t n0 = (int64_t)group * kTiles * 16;
  if (a.rows.offsets && tile.expert == a.rows.experts) {  // rows of no expert
    for (int64_t i = threadIdx.x; i < (tile.r1 - tile.r0) * 16 * kTiles; i += kWaves * 64) {
      const int64_t r = tile.r0 + i / (16 * kTiles), n = n0 + i % (16 * kTiles);
      if (n < a.w.N) w4_store(a.Y, a.y_dtype, r * a.ldy + n, 0.0f);
    }
    return;
  }
  const uint8_t* blob = a.w.blob + tile.expert * a.w.expert_stride;
  const int ch = lane & 15, quad = lane >> 4;

  // rows past the tile's end repeat its last row: their results are not stored
  const T* xr[kFM];
#pragma unroll
  for (int f = 0; f < kFM; ++f) {
    int64_t r = tile.r0 + f * 16 + ch;
    r = r < tile.r1 ? r : tile.r1 - 1;
    const int64_t x = w4_source_row(a.rows, r);
    xr[f] = static_cast<const T*>(a.X) + (x < 0 ? 0 : x) * a.ldx + 8 * quad;
  }

  f32x4 acc[kFM][kTiles];
#pragma unroll
  for (int f = 0; f < kFM; ++f)
#pragma unroll
    for (int c = 0; c < kTiles; ++c) acc[f][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const int64_t t0 = n0 / 16;
  const int64_t last_tile = a.w.Npad / 16 - 1;
  using Stage = W4Stage<T, kKind, kOne, kFM, kTiles>;
  auto load_weights = [&](Stage& st, int64_t b) {
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      const int64_t tc = t0 + c < last_tile ? t0 + c : last_tile;
      st.q[c] = *reinterpret_cast<const u32x4*>(blob + a.w.data_off + (tc * a.w.nblk + b) * 1024 +
                                                (uint32_t)(ch * 64 + quad * 16));
      st.s[c].load(blob + a.w.scale_off + tc * a.w.G4 * (kKind == 1 ? 128 : 256), b, a.w.group, ch);
      if constexpr (kKind == 2)
        st.o[c].load(blob + a.w.offs_off + tc * a.w.G4 * 256, b, a.w.group, ch);
    }
  };
  auto load = [&](Stage& st, int64_t b) {
    load_weights(st, b);
#pragma unroll
    for (int f = 0; f < kFM; ++f)
#pragma unroll
      for (int t = 0; t < 4; ++t) st.x[f][t].load(xr[f] + b * 128 + t * 32);
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
        w4_step<T, kKind, kOne, kFM, kTiles>(st[p], b + p, a.w.group, acc);
        const int64_t nb = b + p + kAhead;
        load(st[p], nb < b1 ? nb : b1 - 1);
      }
    }
#pragma unroll
    for (int p = 0; p < kAhead; ++p)  // (no load behind a branch: its join would wait)
      if (b + p < b1) w4_step<T, kKind, kOne, kFM, kTiles>(st[p], b + p, a.w.group, acc);
  }
  if (wave == kWaves - 1 && full * 128 < a.w.K) {
    Stage st;
    load_weights(st, full);
#pragma unroll
    for (int f = 0; f < kFM; ++f)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int64_t left = a.w.K - (full * 128 + t * 32 + 8 * quad);
        const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
        st.x[f][t].load_n(xr[f] + (n > 0 ? full * 128 + t * 32 : -8 * quad), n);
      }
    w4_step<T, kKind, kOne, kFM, kTiles>(st, full, a.w.group, acc);
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
    if (r >= tile.r1 || col >= a.w.N) continue;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) y += red[w][frag][(m >> 2) * 16 + n][m & 3];
    y *= 16.0f;
    if (w4_source_row(a.rows, r) < 0) y = 0.0f;
    if (a.bias) y += a.bias[tile.expert * a.w.N + col];
    y = y < a.lo ? a.lo : y;
    y = y > a.hi ? a.hi : y;
    w4_store(a.Y, a.y_dtype, r * a.ldy + col, y);
  }
}

template <typename T, int kKind, bool kOne, int kFM, int kTiles, int kWaves, int kAhead>
qp_status launch_rows(const W4Args& a, hipStream_t stream) {
  const int64_t groups = ceil_div(a.w.Npad / 16, kTiles), slots = w4_tile_slots(a.rows, 16 * kFM);
  QP_REQUIRE(slots * groups * kWaves * 64 < (INT64_C(1) << 32), QP_EUNSUPPORTED,
             "qgemm_w4: rows and channels for more than 2^32 threads");
  hipLaunchKernelGGL((w4_rows_kernel<T, kKind, kOne, kFM, kTiles, kWaves, kAhead>),
                     dim3((unsigned)(slots * groups)), dim3(kWaves * 64), 0, stream, a,
                     (uint32_t)slots);
  return check_launch("qgemm_w4 (few rows)");
}

// ---- many rows: tiles of 16*kFM rows x 64*kFN channels -----------------------
// Four waves side by side on the channels, each 16*kFM x 16*kFN outputs in
// registers.  The rows go through LDS in operand order, 64 K at a time, double
// buffered, and serve all four waves; the weights come straight from memory,
// each wave its own, half a block ahead.
//
// What bounds it with groups of 32: per 16x16x32 MFMA (16 cycles of the matrix
// unit) the group's rescale is 4 fused multiply-adds and a weight word costs 13
// vector instructions to unpack, used kFM times; the two units hardly overlap
// on this part.  8192 rows x 11008 x 4096 over 8 experts: 920 us, 800 TFLOP/s;
// of the cycles the matrix unit is busy 38%, vector instructions issue 63%
// (a library product of bf16 matrices of 8192: 1275 TFLOP/s).  128 x 128 tiles
// at three waves a SIMD; 128 x 256 (spills), 64 x 256 and two waves a SIMD
// measured 1540, 1100 and 1130 us where this took 1050.  Every register counts
// (168 a lane at three waves): the weights' and scales' addresses are a scalar
// base and one lane offset, made anew each block so that they are not kept as
// 64-bit pointers (11 reloads of spilled registers a block without).  The loop over
// whole blocks then spills none; the prologue and the cut or half block at the end
// of K do (40 to 119 registers in all for bf16 and f16 rows without offsets), which
// a K off 128 pays once.  Groups of
// 128 on take one rescale per 64 K: 1024 x 11008 x 4096 f16 107 us (119 with
// those reloads); the MFMAs of a tile spread out between the other tile's changed
// nothing.
template <typename T, int kKind, bool kOne, int kFM, int kFN, int kOcc>
__global__ __launch_bounds__(256, kOcc) void w4_tile_kernel(W4Args a, uint32_t row_slots,
                                                         uint32_t col_groups) {
  using V = typename XFrag<T>::vec;
  constexpr int NP = XFrag<T>::kPieces;
  constexpr int kBlocks = kFM * 2;  // kilobytes of a piece plane a stage
  constexpr int kOutLd = 16 * kFN + 4;
  constexpr size_t kRing = 2 * kBlocks * NP * 1024, kOut = 4 * 16 * kOutLd * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRing > kOut ? kRing : kOut];
  u32x4* const xs = reinterpret_cast<u32x4*>(lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ch = lane & 15, quad = lane >> 4;

  // Workgroups go round the 8 XCDs in launch order: give each XCD a run of
  // tiles, eight row tiles by neighbouring channel groups, so that its L2 serves
  // rows and weights several times.
  uint32_t id = blockIdx.x;
  {
    const uint32_t n = gridDim.x, per = n / 8, rest = n % 8, x = id % 8;
    id = x * per + (x < rest ? x : rest) + id / 8;
  }
  const uint32_t band = id / (8 * col_groups);
  const uint32_t in_band = id - band * 8 * col_groups;
  const uint32_t band_rows = row_slots - band * 8 < 8 ? row_slots - band * 8 : 8;
  const uint32_t slot = band * 8 + in_band % band_rows;
  const int64_t n0 = ((int64_t)(in_band / band_rows) * 4 + wave) * 16 * kFN;

  const W4Tile tile = w4_find_tile<16 * kFM>(a.rows, slot);
  if (tile.expert < 0) return;
  if (a.rows.offsets && tile.expert == a.rows.experts) {  // rows of no expert
    for (int64_t r = tile.r0; r < tile.r1; ++r)
      for (int64_t n = n0 + lane; n < n0 + 16 * kFN; n += 64)
        if (n < a.w.N) w4_store(a.Y, a.y_dtype, r * a.ldy + n, 0.0f);
    return;
  }
  const uint8_t* blob = a.w.blob + tile.expert * a.w.expert_stride;

  // staging: a lane brings 8 K of a row, eight lanes a row's 64-K unit side by
  // side in memory (whole lines), a wave eight rows at a time.  In LDS piece c
  // (of 8) of row r sits in the operand order of fragment r/16 and 32-K number
  // c/4, but at place (r%16) ^ c of its 16: otherwise the eight lanes that write
  // one row would meet in the same banks.
  constexpr int kMine = kFM / 2;
  const uint8_t* xbase = static_cast<const uint8_t*>(a.X);
  if (!a.rows.map) xbase += tile.r0 * a.ldx * sizeof(T);
  const int piece_in = lane & 7, row8 = wave * 8 + (lane >> 3);
  const int k_in = piece_in * 8;
  int64_t xoff[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    int64_t r = tile.r0 + j * 32 + row8;
    r = r < tile.r1 ? r : tile.r1 - 1;
    int64_t x = a.rows.map ? w4_source_row(a.rows, r) : r - tile.r0;
    x = x < 0 ? 0 : x;
    xoff[j] = (x * a.ldx + k_in) * (int64_t)sizeof(T);
  }
  // (row8/16 and c/4 pick the kilobyte, fragments 2j and 2j + 1)
  const int place = ((row8 >> 4) * 2 + (piece_in >> 2)) * 64 + (piece_in & 3) * 16 +
                    ((row8 & 15) ^ piece_in);
  constexpr int kBatch = kMine / 2;  // fetched at a time, twice a unit
  auto fetch = [&](XFrag<T> (&x)[kBatch], int batch, int64_t u) {
    const uint8_t* base = xbase + u * (64 * sizeof(T));
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      x[j].load(reinterpret_cast<const T*>(base + xoff[batch * kBatch + j]));
  };
  // the unit that K cuts
  auto fetch_cut = [&](XFrag<T> (&x)[kBatch], int batch, int64_t u) {
    const int64_t left = a.w.K - (u * 64 + k_in);
    const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
    // (a lane with nothing left points at its row's first element)
    const uint8_t* base = xbase + (n > 0 ? u * (int64_t)(64 * sizeof(T)) : -k_in * (int64_t)sizeof(T));
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      x[j].load_n(reinterpret_cast<const T*>(base + xoff[batch * kBatch + j]), n);
  };
  auto stage = [&](const XFrag<T> (&x)[kBatch], int batch, int buf) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      V v[NP];
      x[j].split(v);
#pragma unroll
      for (int i = 0; i < NP; ++i)
        xs[((buf * NP + i) * kBlocks + (batch * kBatch + j) * 4) * 64 + place] =
            __builtin_bit_cast(u32x4, v[i]);
    }
  };

  const int64_t t0 = n0 / 16, last_tile = a.w.Npad / 16 - 1;
  struct Scales {
    float s[kFN][kOne ? 1 : 4];
    float o[kKind == 2 ? kFN : 1][kOne ? 1 : 4];
  };
  struct RawScales {
    W4Scales<kKind == 1, kOne> s[kFN];
    W4Scales<false, kOne> o[kKind == 2 ? kFN : 1];
  };
  auto load_q = [&](u32x4 (&q)[kFN], int64_t b) {
    uint32_t at = ch * 64 + quad * 16;
    asm volatile("" : "+v"(at));
#pragma unroll
    for (int c = 0; c < kFN; ++c) {
      const int64_t tc = t0 + c < last_tile ? t0 + c : last_tile;
      q[c] = *reinterpret_cast<const u32x4*>(blob + a.w.data_off + (tc * a.w.nblk + b) * 1024 + at);
    }
  };
  auto load_s = [&](RawScales& w, int64_t b) {
    int ch = lane & 15;
    asm volatile("" : "+v"(ch));
#pragma unroll
    for (int c = 0; c < kFN; ++c) {
      const int64_t tc = t0 + c < last_tile ? t0 + c : last_tile;
      w.s[c].load(blob + a.w.scale_off + tc * a.w.G4 * (kKind == 1 ? 128 : 256), b, a.w.group, ch);
      if constexpr (kKind == 2)
        w.o[c].load(blob + a.w.offs_off + tc * a.w.G4 * 256, b, a.w.group, ch);
    }
  };
  auto pick_s = [&](Scales& w, const RawScales& raw, int64_t b) {
#pragma unroll
    for (int c = 0; c < kFN; ++c) {
      raw.s[c].pick(b, a.w.group, w.s[c]);
      if constexpr (kKind == 2) raw.o[c].pick(b, a.w.group, w.o[c]);
    }
  };

  f32x4 acc[kFM][kFN];
#pragma unroll
  for (int f = 0; f < kFM; ++f)
#pragma unroll
    for (int c = 0; c < kFN; ++c) acc[f][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  V ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (decltype(ones[0] + ones[0]))0.0625f;

  struct Operand {
    V v[NP];
  };
  const int from[2] = {quad * 16 + (ch ^ quad), quad * 16 + (ch ^ (4 + quad))};
  auto operand = [&](Operand& x, int buf, int f, int t) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      x.v[i] = __builtin_bit_cast(V, xs[((buf * NP + i) * kBlocks + f * 2 + t) * 64 + from[t]]);
  };
  struct Sums {
    f32x4 p[kFN];
    f32x4 sum;
  };
  auto add_tile = [&](const Scales& w, int f, int t, const Sums& d, int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v = __builtin_fmaf(w.s[c][t], d.p[c][i], acc[f][c][i]);
      if constexpr (kKind == 2) v = __builtin_fmaf(w.o[c][t], d.sum[i], v);
      acc[f][c][i] = v;
    }
  };
  auto add = [&](const Scales& w, int f, int t, const Sums& d) {
#pragma unroll
    for (int c = 0; c < kFN; ++c) add_tile(w, f, t, d, c);
  };
  // A 64-K unit as a sequence of steps, each the MFMAs of one row fragment, the
  // rescale of the step before it (whose MFMAs are done by then), a share of
  // the next weights' unpacking and the operand read two steps ahead.  The
  // scheduler is kept from moving work between steps: left alone it gathers
  // the unpacking and the reads in front and spills.
  XFrag<T> x[kBatch];
  u32x4 q[kFN], qn[kFN];
  Scales w;
  RawScales wn;
  constexpr int kT = kOne ? 2 : 1;  // 32-K steps with one rescale
  V wv[2][kT][kFN];                 // the words of this step and the next
  auto unpack_first = [&](auto half) {
    constexpr int H = decltype(half)::value;
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int c = 0; c < kFN; ++c) wv[0][t][c] = w4_unpack<V>(q[c][2 * H + t]);
  };
  // The products of the unit in `buf`, words 2H and 2H+1 of the weights; kMore:
  // unit `next` goes into the other buffer meanwhile.
  auto unit = [&](auto half, auto more, int buf, int64_t next) {
    constexpr int H = decltype(half)::value;
    constexpr bool kMore = decltype(more)::value;
    constexpr int kRounds = 2 / kT, kSteps = kRounds * kFM;
    Sums d[2];
    constexpr int kReads = kOne ? 2 : 3;
    Operand ahead[kReads][kT];
    auto read = [&](int i) {
      if (i < kSteps) {
#pragma unroll
        for (int t = 0; t < kT; ++t)
          operand(ahead[i % kReads][t], buf, i % kFM, kOne ? t : i / kFM);
      }
    };
    if constexpr (kMore) fetch(x, 0, next);
    read(0);
    if (kReads > 2) read(1);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int round = i / kFM, f = i % kFM;
      // which unpacked words: rounds alternate; the whole unit for kOne
      const int now = kOne ? H : round & 1;
      __builtin_amdgcn_sched_barrier(0);
      read(i + kReads - 1);
      if (kMore && i == kSteps / 2) {
        stage(x, 0, buf ^ 1);
        fetch(x, 1, next);
      }
#pragma unroll
      for (int c = 0; c < kFN; ++c) {
        // an MFMA, then the rescale of a tile of the step before: MFMAs in a
        // row would hold the wave up for the matrix unit
        f32x4 p = zero;
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int n = 0; n < NP; ++n) p = mfma32(ahead[i % kReads][t].v[n], wv[now][t][c], p);
        d[i & 1].p[c] = p;
        if (kKind == 2 && c == 0) {
          f32x4 o = zero;
#pragma unroll
          for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int n = 0; n < NP; ++n) o = mfma32(ahead[i % kReads][t].v[n], ones, o);
          d[i & 1].sum = o;
        }
        __builtin_amdgcn_sched_barrier(0);
        if (i > 0)
          add_tile(w, (i - 1) % kFM, kOne ? 0 : 2 * H + (i - 1) / kFM, d[(i - 1) & 1], c);
        if (c + 1 < kFN) __builtin_amdgcn_sched_barrier(0);
      }
      // the next words, a channel tile at a time
#pragma unroll
      for (int c = 0; c < kFN; ++c)
        if (f == ((c + 1) * kFM + kFN - 1) / kFN - 1) {
          if constexpr (kOne) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if constexpr (H == 0)
                wv[1][t][c] = w4_unpack<V>(q[c][2 + t]);
              else if constexpr (kMore)
                wv[0][t][c] = w4_unpack<V>(qn[c][t]);
            }
          } else {
            if (round == 0)
              wv[1][0][c] = w4_unpack<V>(q[c][2 * H + 1]);
            else if constexpr (H == 0)
              wv[0][0][c] = w4_unpack<V>(q[c][2]);
            else if constexpr (kMore)
              wv[0][0][c] = w4_unpack<V>(qn[c][0]);
          }
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    add(w, kFM - 1, kOne ? 0 : 2 * H + kRounds - 1, d[(kSteps - 1) & 1]);
    if constexpr (kMore) stage(x, 1, buf ^ 1);
  };
  using std::false_type;
  using std::true_type;
  using Half0 = std::integral_constant<int, 0>;
  using Half1 = std::integral_constant<int, 1>;
  const int64_t units = a.w.K / 64, pairs = units / 2;
  if (pairs > 0) {
    load_q(q, 0);
    load_s(wn, 0);
    pick_s(w, wn, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fetch(x, i, 0);
      stage(x, i, 0);
    }
    unpack_first(Half0{});
    // (the last round fetches what is there once more; nobody reads that)
    for (int64_t b = 0; b < pairs; ++b) {
      const int64_t nb = b + 1 < pairs ? b + 1 : b;
      // everyone's pieces of the unit are in LDS, and everyone is done with the
      // unit whose buffer is filled next
      __syncthreads();
      unit(Half0{}, true_type{}, 0, 2 * b + 1);
      __syncthreads();
      load_q(qn, nb);
      load_s(wn, nb);
      unit(Half1{}, true_type{}, 1, 2 * nb);
      pick_s(w, wn, nb);
#pragma unroll
      for (int c = 0; c < kFN; ++c) q[c] = qn[c];
    }
  }
  if (units * 64 < a.w.K || (units & 1)) {  // the last, cut or half, block
    load_q(q, pairs);
    load_s(wn, pairs);
    pick_s(w, wn, pairs);
    unpack_first(Half0{});
    for (int64_t u = 2 * pairs; u * 64 < a.w.K; ++u) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (u < units)
          fetch(x, i, u);
        else
          fetch_cut(x, i, u);
        stage(x, i, 0);
      }
      __syncthreads();
      if (u & 1)
        unit(Half1{}, false_type{}, 0, 0);
      else
        unit(Half0{}, false_type{}, 0, 0);
    }
  }

  // out: 16 rows at a time through the wave's own LDS, so that a lane stores
  // eight neighbouring channels
  __syncthreads();
  float* const out = reinterpret_cast<float*>(lds) + wave * 16 * kOutLd;
  constexpr int kPieces8 = 2 * kFN;                // eight-channel pieces of a row
  constexpr int kRowsPass = 64 / kPieces8;         // rows stored at a time
  const int piece = lane % kPieces8, row_in = lane / kPieces8;
  const int64_t col = n0 + piece * 8;
  float bias[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    bias[j] = a.bias && col + j < a.w.N ? a.bias[tile.expert * a.w.N + col + j] : 0.0f;
#pragma unroll
  for (int f = 0; f < kFM; ++f) {
#pragma unroll
    for (int c = 0; c < kFN; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) out[(4 * quad + i) * kOutLd + c * 16 + ch] = acc[f][c][i];
    wave_sync();
#pragma unroll
    for (int h = 0; h < 16; h += kRowsPass) {
      const int64_t r = tile.r0 + f * 16 + h + row_in;
      if (r < tile.r1 && col < a.w.N) {
        const float* src = out + (h + row_in) * kOutLd + piece * 8;
        const float k16 = w4_source_row(a.rows, r) < 0 ? 0.0f : 16.0f;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v = src[j] * 16.0f;
          v = (k16 == 0.0f ? 0.0f : v) + bias[j];
          v = v < a.lo ? a.lo : v;
          y[j] = v > a.hi ? a.hi : v;
        }
        const int n = a.w.N - col < 8 ? (int)(a.w.N - col) : 8;
        w4_store8(a.Y, a.y_dtype, r * a.ldy + col, y, n);
      }
    }
    wave_sync();
  }
}

template <typename T, int kKind, bool kOne, int kFM, int kFN, int kOcc>
qp_status launch_tile(const W4Args& a, hipStream_t stream) {
  const int64_t slots = w4_tile_slots(a.rows, 16 * kFM);
  const int64_t groups = ceil_div(a.w.N, 64 * kFN);
  QP_REQUIRE(slots * groups * 256 < (INT64_C(1) << 32), QP_EUNSUPPORTED,
             "qgemm_w4: rows and channels for more than 2^32 threads");
  hipLaunchKernelGGL((w4_tile_kernel<T, kKind, kOne, kFM, kFN, kOcc>), dim3((unsigned)(slots * groups)),
                     dim3(256), 0, stream, a, (uint32_t)slots, (uint32_t)groups);
  return check_launch("qgemm_w4 (many rows)");
}

template <typename T, int kKind, bool kOne>
qp_status launch_shape(const W4Args& a, W4Shape shape, hipStream_t stream) {
  switch (shape) {
    case kRows1x1: return launch_rows<T, kKind, kOne, 1, 1, 8, 1>(a, stream);
    case kRows1x2: return launch_rows<T, kKind, kOne, 1, 2, 8, 1>(a, stream);
    case kRows1x3: return launch_rows<T, kKind, kOne, 1, 3, 8, 1>(a, stream);
    case kRows1x4: return launch_rows<T, kKind, kOne, 1, 4, 8, 1>(a, stream);
    case kRows2x3: return launch_rows<T, kKind, kOne, 2, 3, 8, 1>(a, stream);
    case kRows2x4: return launch_rows<T, kKind, kOne, 2, 4, 8, 1>(a, stream);
    case kTile4x8:
      // (three pieces a row and the asymmetric sums need the registers)
      return launch_tile<T, kKind, kOne, 4, 2, sizeof(T) == 4 || kKind == 2 ? 2 : 4>(a, stream);
    case kTile8x8: break;  // (for f32 rows 64 rows a workgroup here too, at about the same cost a row)
  }
  if constexpr (sizeof(T) == 4)
    return launch_tile<T, kKind, kOne, 4, 2, 2>(a, stream);  // (LDS holds three pieces of 64 rows)
  else
    return launch_tile<T, kKind, kOne, 8, 2, kKind == 2 ? 2 : 3>(a, stream);
}

template <typename T>
qp_status run_w4_type(const W4Args& a, int32_t format, W4Shape shape, hipStream_t stream) {
  const bool one = a.w.group >= 128;
  if (format == 2)
    return one ? launch_shape<T, 0, true>(a, shape, stream)
               : launch_shape<T, 0, false>(a, shape, stream);
  if (format == 3)
    return one ? launch_shape<T, 1, true>(a, shape, stream)
               : launch_shape<T, 1, false>(a, shape, stream);
  return one ? launch_shape<T, 2, true>(a, shape, stream)
             : launch_shape<T, 2, false>(a, shape, stream);
}

}  // namespace
}  // namespace qp
