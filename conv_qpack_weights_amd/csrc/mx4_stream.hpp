// mx4_stream.hpp -- up to 16 16-bit or MXFP4 rows times MXFP4 weights.
//
// As mx_rows_kernel (mx4_rows.hpp): a workgroup owns kTiles 16-channel tiles, its
// waves share out K.  What a wave needs of 256 K comes by direct loads into LDS that
// is its own, two buffers of it, with no barrier until the sums meet: a direct load
// takes 128 bytes of each of eight rows, where a load of an operand takes 64 or 32
// bytes of each of 16, and the card looks up a line at a time.
//
// Bound by the weights' way from memory where they are large: cold weights of 176128 x 4096
// (383 MB) times 1 / 8 bf16 rows 84 / 87 us, 4.6 / 4.4 TB/s.  Smaller ones take 1.6 times
// what a kernel that only reads as many bytes does, and for what is not known: 4096 x 4096
// (8.9 MB; reading 10.5 MB 3.4 us) times 1 / 16 rows 5.2 / 6.0 to 6.4 us, times MXFP4 rows
// 4.9; 11008 x 4096 (24 MB; reading 28 MB 5.9) 8.3 to 8.6 / 9.6 to 9.8.  With operands
// straight from memory (mx4_rows.hpp) 16 x 4096 x 4096 took 8.3.
#pragma once

#include "mx4_rows.hpp"
#include "mx4_tile.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

template <typename T, int kTiles, int kWaves>
struct MxStream {
  static constexpr bool kA4 = __is_same(T, mx4_t);
  static constexpr int kX = kA4 ? 2048 : 8192;             // 16 rows of 256 K
  static constexpr int kScaleLoads = (kTiles + 1) / 2;      // of 32 channels
  static constexpr int kBuf = kX + kTiles * 2048 + kScaleLoads * 256 + (kA4 ? 256 : 0);
  static constexpr int kLoads = kX / 1024 + 2 * kTiles + kScaleLoads + (kA4 ? 1 : 0);
  static constexpr int kRed = kWaves * kTiles * 1024;
  static constexpr int kLds = 2 * kBuf * kWaves > kRed ? 2 * kBuf * kWaves : kRed;
};

// kOnce: one row tile is to read the weights (of an expert).
template <typename T, int kTiles, int kWaves, bool kOnce>
__global__ __launch_bounds__(kWaves * 64) void mx_stream_kernel(MxArgs a, uint32_t row_slots) {
  using L = MxStream<T, kTiles, kWaves>;
  constexpr bool kA4 = L::kA4;
  constexpr int kParts = L::kX / 2048;  // of 128 bytes of a row
  extern __shared__ __attribute__((aligned(16))) uint8_t mx_lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  lds_u8* const mine = (lds_u8*)mx_lds + wave * 2 * L::kBuf;
  const uint32_t id = xcd_run(blockIdx.x, gridDim.x);
  const uint32_t group = id / row_slots, slot = id - group * row_slots;
  const W4Tile tile = w4_find_tile<16>(a.rows, slot);
  if (tile.expert < 0) return;
  const int64_t n0 = (int64_t)group * kTiles * 16, N = a.w.rows;
  if (mx_rows_of_none<kTiles, kWaves>(a, tile, n0)) return;

  // what a lane loads: a piece of row lane / 8 of eight; rows past the tile's end
  // repeat its last row
  const int lrow = lane >> 3;
  int64_t first = a.rows.map ? 0 : tile.r0;
  int64_t source[kA4 ? 3 : 2];
  mx_sources(a.rows, tile, first,
             [&](int i) { return i < 2 ? i * 8 + lrow : lane >> 1 & 15; }, source);
  auto piece = [&](int h) { return (lane & 7) ^ mx_turn(h * 8 + lrow); };
  const uint8_t* const wbase = a.w.codes + tile.expert * a.w.cstride + n0 * a.w.ldc;
  const uint8_t* const swbase = a.w.scales + tile.expert * a.w.sstride + n0 * a.w.lds;
  const int64_t last_n = N - 1 - n0;
  const uint8_t *xbase, *sxbase = nullptr;
  int64_t xld;
  if constexpr (kA4) {
    xld = a.a.ldc;
    xbase = a.a.codes + first * xld;
    sxbase = a.a.scales + first * a.a.lds;
  } else {
    xld = a.ldx * (int64_t)sizeof(T);
    xbase = static_cast<const uint8_t*>(a.X) + first * xld;
  }
  uint32_t vx[2], vw[kTiles][2], vs[L::kScaleLoads], vsx = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    vx[h] = (uint32_t)(source[h] * xld) + piece(h) * 16;
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      const int64_t n = c * 16 + h * 8 + lrow;
      vw[c][h] = (uint32_t)((n < last_n ? n : last_n) * a.w.ldc) + piece(h) * 16;
    }
  }
#pragma unroll
  for (int i = 0; i < L::kScaleLoads; ++i) {
    const int64_t n = i * 32 + (lane >> 1);
    vs[i] = (uint32_t)((n < last_n ? n : last_n) * a.w.lds) + (lane & 1) * 4;
  }
  if constexpr (kA4) vsx = (uint32_t)(source[2] * a.a.lds) + (lane & 1) * 4;

  // 256 K from 256 g on into buffer g & 1; past the wave's last nothing is asked for
  const int groups = (int)(a.w.K / 256), per = (groups + kWaves - 1) / kWaves;
  const int g0 = wave * per < groups ? wave * per : groups;
  const int g1 = g0 + per < groups ? g0 + per : groups;
  auto issue = [&](int g) {
    const int range = g < g1 ? 0x7fffffff : 0;
    lds_u8* to = mine + (g & 1) * L::kBuf;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int p = 0; p < kParts; ++p, to += 1024)
        dma_to_lds<16>(xbase, range, to, vx[h], g * (kParts * 128) + p * 128);
#pragma unroll
    for (int c = 0; c < kTiles; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h, to += 1024)
        dma_to_lds<16, kOnce>(wbase, range, to, vw[c][h], g * 128);
#pragma unroll
    for (int i = 0; i < L::kScaleLoads; ++i, to += 256)
      dma_to_lds<4>(swbase, range, to, vs[i], g * 8);
    if constexpr (kA4) dma_to_lds<4>(sxbase, range, to, vsx, g * 8);
  };

  const int ch = lane & 15, quad = lane >> 4;
  f32x4 acc[kTiles];
#pragma unroll
  for (int c = 0; c < kTiles; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  typedef MxStage<T, kTiles> Stage;
  auto at = [&](int c) { return (ch & 7) * 128 + (c ^ mx_turn(ch)) * 16; };
  auto read = [&](Stage (&st)[2], int g) {
    const lds_u8* from = mine + (g & 1) * L::kBuf + (ch >> 3) * kParts * 1024;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (kA4) {
        st[j].x = *(const __attribute__((address_space(3))) u32x4*)(from + at(4 * j + quad));
      } else {
        // elements 128 j + 32 quad + 8 t ..: piece 4 (quad & 1) + t of part 2 j + quad / 2
#pragma unroll
        for (int t = 0; t < 4; ++t)
          st[j].x[t].v = *(const __attribute__((address_space(3))) u32x4*)(
              from + (2 * j + (quad >> 1)) * 1024 + at(4 * (quad & 1) + t));
      }
    }
    const lds_u8* const w = mine + (g & 1) * L::kBuf + L::kX + (ch >> 3) * 1024;
    const lds_u8* const s = mine + (g & 1) * L::kBuf + L::kX + kTiles * 2048 + ch * 8;
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      const u32x2 v = *(const __attribute__((address_space(3))) u32x2*)(s + c * 128);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        st[j].q[c] =
            *(const __attribute__((address_space(3))) u32x4*)(w + c * 2048 + at(4 * j + quad));
        st[j].s[c] = v[j];
      }
    }
    if constexpr (kA4) {
      const u32x2 v =
          *(const __attribute__((address_space(3))) u32x2*)(s + L::kScaleLoads * 256);
      st[0].xs = v.x;
      st[1].xs = v.y;
    }
  };

  issue(g0);
  for (int g = g0; g < g1; ++g) {
    issue(g + 1);
    wait_vmcnt<L::kLoads>();
    asm volatile("" ::: "memory");
    Stage st[2];
    read(st, g);
    // (the next round loads into what is read here)
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    mx_step<T, kTiles>(st[0], quad, acc);
    mx_step<T, kTiles>(st[1], quad, acc);
  }
  if (wave == kWaves - 1 && (int64_t)groups * 256 < a.w.K)
    mx_rows_tail<T, kTiles>(a, tile, n0, (int64_t)groups * 2, acc);
  wait_vmcnt<0>();
  __syncthreads();
  mx_rows_store<kTiles, kWaves>(acc, a, tile, n0, reinterpret_cast<f32x4*>(mx_lds));
}

template <typename T, int kTiles, int kWaves, bool kOnce>
qp_status mx_launch_stream_of(const MxArgs& a, hipStream_t stream) {
  using L = MxStream<T, kTiles, kWaves>;
  const int64_t groups = ceil_div(a.w.rows, 16 * kTiles), slots = w4_tile_slots(a.rows, 16);
  QP_REQUIRE(slots * groups * kWaves * 64 < (INT64_C(1) << 32), QP_EUNSUPPORTED,
             "qgemm_mx: rows and channels for more than 2^32 threads");
  auto kern = mx_stream_kernel<T, kTiles, kWaves, kOnce>;
  static std::atomic<uint64_t> reserved{0};
  if (qp_status st =
          mx_reserve_lds("qgemm_mx", reinterpret_cast<const void*>(kern), L::kLds, reserved))
    return st;
  hipLaunchKernelGGL(kern, dim3((unsigned)(slots * groups)), dim3(kWaves * 64), L::kLds, stream, a,
                     (uint32_t)slots);
  return check_launch("qgemm_mx (few rows)");
}

// (Loads for once, cold weights: 1 x 11008 x 4096 bf16 8.9 -> 8.3 us, 16 x 4096 x 11008
// 13.0 -> 12.1, 16 tokens x 2 of 8 experts of 4096 x 4096 23.5 -> 21.9; with four row
// tiles, 64 x 4096 x 11008, 18.1 -> 19.5.)
template <typename T, int kTiles, int kWaves>
qp_status mx_launch_stream(const MxArgs& a, hipStream_t stream) {
  return mx_read_once(a, 16) ? mx_launch_stream_of<T, kTiles, kWaves, true>(a, stream)
                             : mx_launch_stream_of<T, kTiles, kWaves, false>(a, stream);
}

}  // namespace
}  // namespace qp
