// mx4_tile.hpp -- what the many-row kernels of the MXFP4 products share: direct
// loads into LDS, the order of the tiles, the way out.
#pragma once

#include <atomic>

#include "mx4.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// kBytes per lane from base + voff + soff straight into LDS, lane after lane from dst
// on; offsets of `range` bytes and more ask for nothing.  kOnce: data that no one reads
// again, which the caches need not keep.  (The caller waits.)
template <int kBytes, bool kOnce = false>
__device__ __forceinline__ void dma_to_lds(const void* base, int range, lds_u8* dst, uint32_t voff,
                                           uint32_t soff) {
#if defined(__HIP_DEVICE_COMPILE__)
  __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, range, 0x00020000);
  if constexpr (kBytes == 16)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)dst, 16, voff, soff, 0, kOnce ? 2 : 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)dst, 4, voff, soff, 0, kOnce ? 2 : 0);
#endif
}

// The same from an address of the lane's own, anywhere in memory.
template <int kBytes>
__device__ __forceinline__ void far_to_lds(const uint8_t* from, lds_u8* dst) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (kBytes == 16)
    __builtin_amdgcn_global_load_lds((const glb_void_t*)from, (lds_void_t*)dst, 16, 0, 0);
  else
    __builtin_amdgcn_global_load_lds((const glb_void_t*)from, (lds_void_t*)dst, 4, 0, 0);
#endif
}

// Rows of 128 bytes in LDS: the 16-byte piece c of row r lies at place c ^ mx_turn(r)
// of the row's eight, so that the 16 rows whose pieces are read at a time are at 16
// different places of the banks' 256 bytes.
__device__ __forceinline__ int mx_turn(int r) { return (r >> 1) & 7; }

__device__ __forceinline__ f32x16 mx_mfma_bf16(bf16x8 a, bf16x8 b, f32x16 d) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, d, 0, 0, 0);
}

__device__ __forceinline__ f32x16 mx_mfma_f16(f16x8 a, f16x8 b, f32x16 d) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, d, 0, 0, 0);
}

// Whether one of the blocks of `rows` rows, `blocks` from codes and scales on, is no block
// of f16 values; each of `threads` answers for its share.  (f16 rows and a block of zeros in
// every channel: 4096^3 126 us, begun again 382, without such blocks 112; 64 x 11008 x 4096
// 33, 83, 20; gradients 4096^3 137, 380, 124.  With the codes looked at in the main loops
// instead ordinary weights took 112 -> 113 and 20 -> 21 us, their gradients 124 -> 138.)
__device__ __forceinline__ bool mx_no_f16_among(const uint8_t* codes, int64_t ldc,
                                                const uint8_t* scales, int64_t lds, int64_t rows,
                                                int blocks, int threads) {
  const uint32_t words = (blocks + 3) / 4;
  bool out = false;
  for (uint32_t i = threadIdx.x; i < (uint32_t)rows * words; i += threads) {
    const int64_t row = i / words, w = i % words;
    const uint32_t four = *reinterpret_cast<const uint32_t*>(scales + row * lds + w * 4);
#pragma unroll 1
    for (int j = 0; j < 4 && w * 4 + j < blocks; ++j) {
      const float s = mx_scale(four >> (8 * j) & 0xffu);
      if (!mx_f16_scale(s))
        out |= !mx_f16_block(
            *reinterpret_cast<const u32x4*>(codes + row * ldc + (w * 4 + j) * 16), s);
    }
  }
  return out;
}

// Entry m of a map of rows (w4_source_row without branches: a lane's entries are loaded
// one after another and waited for once): the row it stands for, 0 where it is none.
__device__ __forceinline__ bool mx_has_source(const W4Rows& rows, int32_t m) {
  return m >= 0 && (uint32_t)m / (uint32_t)rows.map_div < rows.x_rows;
}
__device__ __forceinline__ int64_t mx_source(const W4Rows& rows, int32_t m) {
  return mx_has_source(rows, m) ? (uint32_t)m / (uint32_t)rows.map_div : 0;
}

// The rows of X that rows r0 + row(i), i < kN, of a tile read, from row `first` on: those
// past the tile's end repeat its last row.
template <int kN, typename Row>
__device__ __forceinline__ void mx_sources(const W4Rows& rows, const W4Tile& tile, int64_t first,
                                           Row row, int64_t (&x)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int64_t r = tile.r0 + row(i);
    x[i] = r < tile.r1 ? r : tile.r1 - 1;
  }
  if (rows.map) {
    int32_t m[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) m[i] = rows.map[x[i]];
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = mx_source(rows, m[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] -= first;
  }
}

// Which tile a workgroup takes: eight row tiles by neighbouring channel groups, in
// runs per XCD.
__device__ __forceinline__ void mx_place_of(uint32_t id, uint32_t row_slots, uint32_t col_groups,
                                            uint32_t& slot, uint32_t& group) {
  const uint32_t band = id / (8 * col_groups), in_band = id - band * 8 * col_groups;
  const uint32_t band_rows = row_slots - band * 8 < 8 ? row_slots - band * 8 : 8;
  slot = band * 8 + in_band % band_rows;
  group = in_band / band_rows;
}

// How many BM-row tiles the rows have.
template <int BM>
__device__ __forceinline__ uint32_t mx_count_tiles(const W4Rows& rows) {
  if (!rows.offsets) return (uint32_t)((rows.M + BM - 1) / BM);
  const int lane = threadIdx.x & 63;
  const int32_t M = (int32_t)rows.M;
  uint32_t n = 0;
  for (int e0 = 0; e0 <= rows.experts; e0 += 64) {  // (the clamps of w4_find_tile)
    const int e = e0 + lane;
    int32_t a = M, b = M;
    if (e <= rows.experts) {
      a = rows.offsets[e];
      if (e < rows.experts) b = rows.offsets[e + 1];
    }
    a = a < 0 ? 0 : a > M ? M : a;
    b = b < a ? a : b > M ? M : b;
    n += (uint32_t)((b - a + BM - 1) / BM);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) n += __shfl_xor(n, d);
  return __builtin_amdgcn_readfirstlane(n);
}

// Workgroups of BM-row tiles that are one to a CU: an XCD's tiles go by in rounds of its
// 32 CUs, and those of a last round that leaves half of them idle and more are split in
// two halves of the rows, which take 0.53 of the time.  (4096 tokens x 2 of 8 experts of
// 11008 x 4096: a4w4 334 -> 322 us, bf16 rows 764 -> 741, their gradient 957 -> 841.)
constexpr uint32_t kMxXcdCus = 32;

// The tile of workgroup blockIdx.x; false: none.
template <int BM, bool kHalves>
__device__ __forceinline__ bool mx_take_tile(const W4Rows& rows, uint32_t row_slots,
                                             uint32_t col_groups, W4Tile& tile, uint32_t& group) {
  uint32_t slot;
  if constexpr (!kHalves) {
    mx_place_of(xcd_run(blockIdx.x, gridDim.x), row_slots, col_groups, slot, group);
    tile = w4_find_tile<BM>(rows, slot);
    return tile.expert >= 0;
  } else {
    const uint32_t slots = mx_count_tiles<BM>(rows), n = slots * col_groups;
    const uint32_t x = blockIdx.x % 8, at = blockIdx.x / 8;
    const uint32_t per = n / 8, rest = n % 8;
    const uint32_t mine = per + (x < rest ? 1 : 0), first = x * per + (x < rest ? x : rest);
    const uint32_t last = mine % kMxXcdCus, whole = mine - last;
    const bool halved = last <= kMxXcdCus / 2 && at >= whole;
    const uint32_t id = halved ? whole + (at - whole) / 2 : at;
    if (id >= mine) return false;
    mx_place_of(first + id, slots, col_groups, slot, group);
    tile = w4_find_tile<BM>(rows, slot);
    if (halved) {
      const int64_t half = tile.r0 + BM / 2;
      if ((at - whole) % 2)
        tile.r0 = half;
      else
        tile.r1 = tile.r1 < half ? tile.r1 : half;
    }
    return tile.expert >= 0 && tile.r0 < tile.r1;
  }
}

// How many workgroups `slots` row tiles (at most) by `groups` take.
inline int64_t mx_tile_grid(int64_t slots, int64_t groups, bool halves) {
  return halves ? (ceil_div(slots * groups, 8) + kMxXcdCus / 2) * 8 : slots * groups;
}

// A kernel's LDS reserved once per device: `reserved` has a bit for each that it is for.
inline qp_status mx_reserve_lds(const char* what, const void* kern, int bytes,
                                std::atomic<uint64_t>& reserved) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) QP_FAIL(QP_EHIP, "%s: hipGetDevice failed", what);
  const uint64_t bit = dev >= 0 && dev < 64 ? UINT64_C(1) << dev : 0;
  if (bit && (reserved.load(std::memory_order_acquire) & bit)) return QP_OK;
  if (hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess)
    QP_FAIL(QP_EHIP, "%s: cannot reserve %d bytes of LDS", what, bytes);
  reserved.fetch_or(bit, std::memory_order_release);
  return QP_OK;
}

constexpr int mx_out_ld(int FN) { return 32 * FN + 4; }

// Eight neighbouring outputs to p.
template <typename T>
__device__ __forceinline__ void mx_store8(T* p, const float (&y)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float lo[4] = {y[0], y[1], y[2], y[3]}, hi[4] = {y[4], y[5], y[6], y[7]};
    store_piece(p, lo, 4);
    store_piece(p + 4, hi, 4);
  } else {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    u32x4_any v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 two = {y[2 * i], y[2 * i + 1]};
      if constexpr (__is_same(T, f16_t)) {
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, f16x2));
      } else {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2));
      }
    }
    *reinterpret_cast<u32x4_any*>(p) = v;
  }
}

// (Against the way through LDS below, 128 x 128 tiles: a4w4 2048 x 4096 x 4096 26.7 -> 24.9
// us, bf16 2048 tokens x 2 of 8 experts of 4096 x 4096 165 -> 159.  256 x 256 tiles, whose
// CUs all store at once, took 3 us longer with its 32 bytes of a row at a time.)
// A wave's sums to Y where all its channels are there: a lane holds one row and, of 16
// channels, runs of four 8 apart, the other half of the wave the runs between; halves
// swapped, each has eight neighbouring channels.
template <typename T, int FM, int FN>
__device__ __forceinline__ void mx_store_whole(const f32x16 (&acc)[FN][FM], const MxArgs& a,
                                               const W4Tile& tile, int row0, int64_t col0) {
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
  int64_t row[FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) row[j] = tile.r0 + row0 + j * 32 + l32;
  bool none[FM] = {};
  if (a.rows.map) {
    int32_t m[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) m[j] = a.rows.map[row[j] < tile.r1 ? row[j] : tile.r1 - 1];
#pragma unroll
    for (int j = 0; j < FM; ++j) none[j] = !mx_has_source(a.rows, m[j]);
  }
  const bool bounds = a.lo > -INFINITY || a.hi < INFINITY;
  T* const Y = static_cast<T*>(a.Y) + col0 + half * 8;
  const float* const bias = a.bias ? a.bias + tile.expert * a.w.rows + col0 + half * 8 : nullptr;
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      const int c = i * 32 + q * 8;
      float b[8] = {};
      if (bias) {
#pragma unroll
        for (int t = 0; t < 8; ++t) b[t] = bias[c + t];
      }
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        float y[8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float lo = acc[i][j][4 * q + t], hi = acc[i][j][4 * q + 4 + t];
          const auto two = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, lo),
                                                            __builtin_bit_cast(uint32_t, hi),
                                                            false, false);
          const uint32_t mine = two[0], other = two[1];
          y[t] = __builtin_bit_cast(float, mine);
          y[4 + t] = __builtin_bit_cast(float, other);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) y[t] = (none[j] ? 0.0f : y[t]) + b[t];
        if (bounds) {
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const float v = y[t] < a.lo ? a.lo : y[t];
            y[t] = v > a.hi ? a.hi : v;
          }
        }
        if (row[j] < tile.r1) mx_store8(Y + row[j] * a.ldy + c, y);
      }
    }
}

// A wave's sums (weights the first operand of its 32x32 MFMAs: a lane holds one row
// and runs of four channels) to Y: 32 rows at a time through `out`, the wave's own
// LDS of 32 mx_out_ld(FN) floats, so that a lane stores eight neighbouring channels.
// (The loops are kept rolled: unrolled with all the types' stores they are tens of
// kilobytes, and fetching those takes longer than a short product.)
template <int FM, int FN>
__device__ __forceinline__ void mx_store_tile(const f32x16 (&acc)[FN][FM], const MxArgs& a,
                                              const W4Tile& tile, int row0, int64_t col0,
                                              float* out) {
  constexpr int kLd = mx_out_ld(FN);
  constexpr int kPieces8 = 4 * FN, kRowsPass = 64 / kPieces8;
  if (FM <= 2 && col0 + 32 * FN <= a.w.rows) {
    if (a.y_dtype == QP_F32)
      mx_store_whole<float, FM, FN>(acc, a, tile, row0, col0);
    else if (a.y_dtype == QP_BF16)
      mx_store_whole<bf16_t, FM, FN>(acc, a, tile, row0, col0);
    else
      mx_store_whole<f16_t, FM, FN>(acc, a, tile, row0, col0);
    return;
  }
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
  const int p8 = lane % kPieces8, row_in = lane / kPieces8;
  const int64_t N = a.w.rows, col = col0 + p8 * 8;
  float bias[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    bias[j] = a.bias && col + j < N ? a.bias[tile.expert * N + col + j] : 0.0f;
  // which of the lane's rows have no source
  uint32_t none = 0;
  if (a.rows.map) {
    constexpr int kPasses = FM * (32 / kRowsPass);
    int32_t m[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int64_t r = tile.r0 + row0 + i * kRowsPass + row_in;
      m[i] = a.rows.map[r < tile.r1 ? r : tile.r1 - 1];
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) none |= mx_has_source(a.rows, m[i]) ? 0u : 1u << i;
  }
  // (no load is under way in the loop: waiting for one would be waiting for the stores
  // before it, a microsecond a pass)
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
#pragma unroll 1
  for (int f = 0; f < FM; ++f) {
#pragma unroll
    for (int j = 0; j < FM; ++j)
      if (j == f) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(out + l32 * kLd + i * 32 + q * 8 + half * 4) =
                f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                      acc[i][j][4 * q + 3]};
      }
    wave_sync();
#pragma unroll 1
    for (int h = 0; h < 32; h += kRowsPass) {
      const int64_t r = tile.r0 + row0 + f * 32 + h + row_in;
      if (r < tile.r1 && col < N) {
        const float* src = out + (h + row_in) * kLd + p8 * 8;
        const f32x4 lo = *reinterpret_cast<const f32x4*>(src);
        const f32x4 hi = *reinterpret_cast<const f32x4*>(src + 4);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v = (none & 1 ? 0.0f : j < 4 ? lo[j % 4] : hi[j % 4]) + bias[j];
          v = v < a.lo ? a.lo : v;
          y[j] = v > a.hi ? a.hi : v;
        }
        const int64_t at = r * a.ldy + col;
        if (N - col < 8)
          w4_store8(a.Y, a.y_dtype, at, y, (int)(N - col));
        else if (a.y_dtype == QP_F32)
          mx_store8(static_cast<float*>(a.Y) + at, y);
        else if (a.y_dtype == QP_BF16)
          mx_store8(static_cast<bf16_t*>(a.Y) + at, y);
        else
          mx_store8(static_cast<f16_t*>(a.Y) + at, y);
      }
      none >>= 1;
    }
    wave_sync();
  }
}

}  // namespace
}  // namespace qp
