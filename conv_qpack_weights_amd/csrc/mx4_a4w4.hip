// mx4_a4w4.hip -- MXFP4 rows times MXFP4 weights: both go into the scaled 4-bit
// MFMA as they are,
//   y[r,n] = clamp(sum_b 2^(sa[r,b] + sw[n,b] - 254) sum_{k in b} a[r,k] w[n,k] + bias[n], lo, hi)
// with every product and scaling exact and the sums in f32.  Few rows: the kernel
// of mx4_stream.hpp; many rows: tiles over LDS, below.
#include <type_traits>

#include "mx4_rows.hpp"
#include "mx4_scales.hpp"
#include "mx4_stream.hpp"
#include "mx4_tile.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

// d + a b^T over 64 K: lane l holds 32 values of row l%32 from 32 (l/32) on; their
// scale is byte kByte of sa / sb.
template <int kByte>
__device__ __forceinline__ f32x16 mx_mfma32(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x16 d) {
  const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, d, 4, 4, kByte, (int)sa, kByte,
                                                         (int)sb);
}

// ---- many rows -----------------------------------------------------------------
// A workgroup owns BM rows x BN channels, its WM x WN waves 32 FM rows x 32 FN
// channels each, in registers.  256 K of rows and channels at a time, a stage, come
// into one of D LDS buffers by direct loads, 128 bytes of a row side by side; the
// 16-byte piece c of row r lies at place c ^ mx_turn(r) of the row's eight, so that the
// rows an operand takes piece c of meet every bank alike.  The weights are the
// MFMA's first operand: a lane ends with one row and runs of four channels.
//
// 8192^3, 256 x 256 tiles, on random codes: 289 to 309 us on different cards, 3.7 PFLOP/s.
// Its matrix instructions alone, on random codes, took 177 us in one loop of nothing else
// and 217 in another (the card's clock gives way to them, by the operands), with the LDS
// reads 248; its loads alone 187.  Eight waves of 128 x 64 read 6 operands
// for 8 MFMAs; one workgroup fills a CU's LDS.  A step's operands are read ahead of the
// MFMAs of the step before, over the barrier too.
template <int BM, int BN, int WM, int WN, int D>
struct A4Tile {
  static constexpr int NW = WM * WN, FM = BM / (32 * WM), FN = BN / (32 * WN);
  static constexpr int kStage = (BM + BN) * 128, kScales = (BM + BN) * kMxScaleRow;
  static constexpr int kSpans = D == 2 ? 2 : 4;  // of 512 K: D / 2 + 1 are live
  static constexpr int kOutLd = mx_out_ld(FN);
  static constexpr int kOut = NW * 32 * kOutLd * 4;
  static constexpr int kRing = D * kStage + kSpans * kScales + kMxScaleRoom;
  static constexpr int kLds = kRing > kOut ? kRing : kOut;
};

// kWide (four words of scales a row and more): a row's scales of 512 K come by one
// lane's 16 bytes; those of the last 512 K end with the row's last word.
// kFar: rows further from each other, or from the first, than 32-bit offsets reach; each
// lane has addresses of its own for them.
template <int BM, int BN, int WM, int WN, int D, bool kWide, bool kFar>
__global__ __launch_bounds__(WM * WN * 64) void mx_a4w4_tile_kernel(MxArgs a, uint32_t row_slots,
                                                                   uint32_t col_groups) {
  using L = A4Tile<BM, BN, WM, WN, D>;
  constexpr int NW = L::NW, FM = L::FM, FN = L::FN;
  constexpr int kA = BM / 8 / NW, kB = BN / 8 / NW, kSRows = kWide ? 64 : 16,
                kSI = (BM + BN) / kSRows, kS = (kSI + NW - 1) / NW;
  static_assert(kA * 8 * NW == BM && kB * 8 * NW == BN && BM % kSRows == 0, "shares");
  static_assert(!kFar || D == 2, "waits of the far loads");
  extern __shared__ __attribute__((aligned(16))) uint8_t mx_lds[];
  lds_u8* const ring = (lds_u8*)mx_lds;
  lds_u8* const scales = ring + D * L::kStage;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  W4Tile tile;
  uint32_t group;
  if (!mx_take_tile<BM, (BM >= 256)>(a.rows, row_slots, col_groups, tile, group)) return;
  const int64_t n0 = (int64_t)group * BN;
  const int64_t N = a.w.rows;
  if (a.rows.offsets && tile.expert == a.rows.experts) {  // rows of no expert
    for (int64_t r = tile.r0 + wave; r < tile.r1; r += NW)
      for (int64_t n = n0 + lane; n < n0 + BN && n < N; n += 64)
        w4_store(a.Y, a.y_dtype, r * a.ldy + n, 0.0f);
    return;
  }

  // what a lane loads: a piece of row lane / 8 of eight; rows past the tile's end
  // repeat its last row
  const int lrow = lane >> 3;
  auto piece = [&](int j) { return (lane & 7) ^ mx_turn(j * 8 + lrow); };
  static_assert(kA % 2 == 0 && kB % 2 == 0, "turn of a wave's first row");
  const uint8_t *abase = a.a.codes, *sabase = a.a.scales;
  int64_t first = 0;
  if (!a.rows.map) {
    first = tile.r0;
    abase += first * a.a.ldc;
    sabase += first * a.a.lds;
  }
  const uint8_t* const wbase = a.w.codes + tile.expert * a.w.cstride + n0 * a.w.ldc;
  const uint8_t* const swbase = a.w.scales + tile.expert * a.w.sstride + n0 * a.w.lds;
  const int64_t last_n = N - 1 - n0;
  uint32_t va[kA], vb[kB], vs[kS];
  const uint8_t *pa[kFar ? kA : 1], *ps[kFar ? kS : 1];
#pragma unroll
  for (int j = 0; j < kB; ++j) {
    const int64_t n = (wave * kB + j) * 8 + lrow;
    vb[j] = (uint32_t)((n < last_n ? n : last_n) * a.w.ldc) + piece(j) * 16;
  }
  // which rows' scales a wave loads (the last ones twice where they do not go round)
  const int sdw = kWide ? 0 : lane & 3, srow = kWide ? lane : lane >> 2;
  auto scale_part = [&](int j) {
    const int i = wave * kS + j;
    return i < kSI ? i : kSI - 1;
  };
  int64_t x[kA + kS];
  mx_sources(a.rows, tile, first, [&](int i) {
    return i < kA ? (wave * kA + i) * 8 + lrow : scale_part(i - kA) * kSRows + srow;
  }, x);
#pragma unroll
  for (int j = 0; j < kA; ++j) {
    if constexpr (kFar)
      pa[j] = abase + x[j] * a.a.ldc + piece(j) * 16;
    else
      va[j] = (uint32_t)(x[j] * a.a.ldc) + piece(j) * 16;
  }
#pragma unroll
  for (int j = 0; j < kS; ++j) {
    const int i = scale_part(j);
    if (i * kSRows < BM) {
      if constexpr (kFar)
        ps[j] = sabase + x[kA + j] * a.a.lds + sdw * 4;
      else
        vs[j] = (uint32_t)(x[kA + j] * a.a.lds) + sdw * 4;
    } else {
      const int64_t n = i * kSRows + srow - BM;
      vs[j] = (uint32_t)((n < last_n ? n : last_n) * a.w.lds) + sdw * 4;
    }
  }

  // Stage s into buffer s % D, and with an even one the scales of it and the next.
  // Pieces past the row's last block and words past its last scale are read from the
  // stage's first (the cut stage puts them to zero).  A stage past the last one asks
  // for nothing: its buffers' range is empty, so that every round of the loop has the
  // same loads to wait for (far rows: for the first stage's, which no one reads there).
  const int G = (int)a.w.G, full = G / 8, stages = (G + 7) / 8, words = (G + 3) / 4;
  const int over = mx_scales_over(words);
  auto late = [&](int s) { return kWide && mx_scales_end(s) > words ? over : 0; };
  auto issue = [&](int s, auto with_scales) {
    lds_u8* const to = ring + (s % D) * L::kStage;
    const int range = s < stages ? 0x7fffffff : 0;
    const int from = kFar && s >= stages ? 0 : s;
    auto back = [&](int j) { return from * 8 + piece(j) < G ? 0u : piece(j) * 16u; };
#pragma unroll
    for (int j = 0; j < kA; ++j) {
      if constexpr (kFar)
        far_to_lds<16>(pa[j] + (from * 128 - (int)back(j)), to + (wave * kA + j) * 1024);
      else
        dma_to_lds<16>(abase, range, to + (wave * kA + j) * 1024, va[j] - back(j),
                       s * 128);
    }
#pragma unroll
    for (int j = 0; j < kB; ++j)
      dma_to_lds<16>(wbase, range, to + BM * 128 + (wave * kB + j) * 1024, vb[j] - back(j),
                     s * 128);
    if constexpr (decltype(with_scales)::value) {
      lds_u8* const st = scales + ((s >> 1) % L::kSpans) * L::kScales;
      const uint32_t sback = kWide || from * 2 + sdw < words ? 0u : sdw * 4u;
#pragma unroll
      for (int j = 0; j < kS; ++j) {
        const int i = scale_part(j);
        if constexpr (kFar) {
          if (i * kSRows < BM) {
            far_to_lds<kWide ? 16 : 4>(ps[j] + (from * 8 - late(from) - (int)sback),
                                       st + i * kSRows * 16);
            continue;
          }
        }
        dma_to_lds<kWide ? 16 : 4>(i * kSRows < BM ? sabase : swbase, range,
                                   st + i * kSRows * 16, vs[j] - sback, s * 8 - late(s));
      }
    }
  };

  // F x FN operands a wave
  auto run = [&](auto operands) {
    constexpr int F = decltype(operands)::value;
    f32x16 acc[FN][F];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    const int l32 = lane & 31, half = lane >> 5;
    const uint32_t sel = half ? 0x07050301u : 0x06040200u;  // the half's scale of each 64 K
    auto mine = [&](const lds_u8* at) {
      const u32x2 v = *(const __attribute__((address_space(3))) u32x2*)at;
      return __builtin_amdgcn_perm(v.y, v.x, sel);
    };
    const int arow = wm * 32 * F + l32, brow = wn * 32 * FN + l32;
    struct Operands {
      u32x4 x[F], w[FN];
    };
    struct Scales {
      uint32_t a[F], w[FN];
    };
    auto read = [&](Operands& o, int s, int step) {
      const lds_u8* const from = ring + (s % D) * L::kStage;
      const int at = ((2 * step + half) ^ mx_turn(l32)) * 16;
#pragma unroll
      for (int i = 0; i < FN; ++i)
        o.w[i] = *(const __attribute__((address_space(3))) u32x4*)(
            from + (BM + brow + i * 32) * 128 + at);
#pragma unroll
      for (int j = 0; j < F; ++j)
        o.x[j] = *(const __attribute__((address_space(3))) u32x4*)(
            from + (arow + j * 32) * 128 + at);
    };
    auto read_scales = [&](Scales& o, int s) {
      const lds_u8* const st =
          scales + ((s >> 1) % L::kSpans) * L::kScales + mx_scales_at(s) + late(s);
#pragma unroll
      for (int j = 0; j < F; ++j) o.a[j] = mine(st + (arow + j * 32) * 16);
#pragma unroll
      for (int i = 0; i < FN; ++i) o.w[i] = mine(st + (BM + brow + i * 32) * 16);
    };
    auto multiply = [&](auto which, const Operands& o, const Scales& c) {
      constexpr int S = decltype(which)::value;
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int i = 0; i < FN; ++i)
          acc[i][j] = mx_mfma32<S>(o.w[i], c.w[i], o.x[j], c.a[j], acc[i][j]);
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    using S2 = std::integral_constant<int, 2>;
    using S3 = std::integral_constant<int, 3>;
    using std::false_type;
    using std::true_type;

    // The next stage is in LDS for everyone (all loads but those of the D - 2 stages
    // after it are done; of two stages running one brings scales), and everyone has
    // read all of this one, whose buffer is filled next.
    constexpr int kAllowed = (D - 2) * (kA + kB) + (D - 2) / 2 * kS;
    static_assert((D == 2 || D == 4) && kAllowed < 64, "vmcnt range");
    auto arrive = [&]() {
      wait_vmcnt<kAllowed>();
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    issue(0, true_type{});
#pragma unroll
    for (int s = 1; s < D - 1; ++s) {
      if (s & 1)
        issue(s, false_type{});
      else
        issue(s, true_type{});
    }
    arrive();
    issue(D - 1, false_type{});
    Operands even, odd;
    Scales now, next;
    read(even, 0, 0);
    read_scales(now, 0);
    // (no branch in the loop: the compiler would move the MFMAs past it, behind the
    // barrier)
    auto stage = [&](int s, auto with_scales) {
      read(odd, s, 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(S0{}, even, now);
      __builtin_amdgcn_sched_barrier(0);
      read(even, s, 2);
      __builtin_amdgcn_sched_barrier(0);
      multiply(S1{}, odd, now);
      __builtin_amdgcn_sched_barrier(0);
      read(odd, s, 3);
      __builtin_amdgcn_sched_barrier(0);
      multiply(S2{}, even, now);
      __builtin_amdgcn_sched_barrier(0);
      arrive();
      // (loads first: behind the MFMAs they made 8192^3 2% faster, but 4096 tokens x 2 of 8
      // experts and 1024 x 4096 x 4096 4% slower)
      issue(s + D, with_scales);
      read(even, s + 1, 0);
      read_scales(next, s + 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(S3{}, odd, now);
      __builtin_amdgcn_sched_barrier(0);
      now = next;
    };
    const int pairs = full / 2;
    if (tile.r0 + wm * 32 * F < tile.r1) {
      for (int t = 0; t < pairs; ++t) {
        stage(2 * t, true_type{});
        stage(2 * t + 1, false_type{});
      }
    } else {
      // (a wave without rows only loads, and leaves its SIMD to the others)
      for (int t = 0; t < pairs; ++t) {
        arrive();
        issue(2 * t + D, true_type{});
        arrive();
        issue(2 * t + 1 + D, false_type{});
      }
    }
    wait_vmcnt<0>();
    __syncthreads();
    // a last odd stage, and the one that K cuts: zero codes and scales past the last
    // block (all their loads are done: at most two stages are left, and D were under
    // way)
#pragma unroll 1
    for (int s = 2 * pairs; s < stages; ++s) {
      const int left = G - s * 8;
      if (left < 8) {
        lds_u8* const to = ring + (s % D) * L::kStage;
        lds_u8* const st =
            scales + ((s >> 1) % L::kSpans) * L::kScales + mx_scales_at(s) + late(s);
        for (int i = threadIdx.x; i < (BM + BN) * 8; i += NW * 64) {
          if (((i & 7) ^ mx_turn(i >> 3)) >= left)
            *(__attribute__((address_space(3))) u32x4*)(to + i * 16) = u32x4{0, 0, 0, 0};
          if ((i & 7) >= left) st[(i >> 3) * 16 + (i & 7)] = 0;
        }
        __syncthreads();
      }
      read_scales(now, s);
      read(even, s, 0);
      multiply(S0{}, even, now);
      read(even, s, 1);
      multiply(S1{}, even, now);
      read(even, s, 2);
      multiply(S2{}, even, now);
      read(even, s, 3);
      multiply(S3{}, even, now);
    }
    __syncthreads();

    mx_store_tile<F, FN>(acc, a, tile, wm * F * 32, n0 + wn * FN * 32,
                          reinterpret_cast<float*>(mx_lds) + wave * 32 * L::kOutLd);
  };
  // (half the rows, half the operands: half a tile takes 0.53 of a whole one's time,
  // with one wave of two at work on all of a wave's operands instead about 0.6)
  constexpr int kHalf = FM > 1 ? FM / 2 : FM;
  if (kHalf < FM && tile.r1 - tile.r0 <= BM / 2)
    run(std::integral_constant<int, kHalf>{});
  else
    run(std::integral_constant<int, FM>{});
}

template <int BM, int BN, int WM, int WN, int D, bool kWide, bool kFar>
qp_status launch_tile_of(const MxArgs& a, hipStream_t stream) {
  using L = A4Tile<BM, BN, WM, WN, D>;
  const int64_t slots = w4_tile_slots(a.rows, BM), groups = ceil_div(a.w.rows, BN);
  const int64_t grid = mx_tile_grid(slots, groups, BM >= 256);
  QP_REQUIRE(grid * L::NW * 64 < (INT64_C(1) << 32), QP_EUNSUPPORTED,
             "qgemm_a4w4_mx: rows and channels for more than 2^32 threads");
  auto kern = mx_a4w4_tile_kernel<BM, BN, WM, WN, D, kWide, kFar>;
  static std::atomic<uint64_t> reserved{0};
  if (qp_status st =
          mx_reserve_lds("qgemm_a4w4_mx", reinterpret_cast<const void*>(kern), L::kLds, reserved))
    return st;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(L::NW * 64), L::kLds, stream, a,
                     (uint32_t)slots, (uint32_t)groups);
  return check_launch("qgemm_a4w4_mx (many rows)");
}

template <int BM, int BN, int WM, int WN, int D, bool kFar = false>
qp_status launch_tile(const MxArgs& a, hipStream_t stream) {
  return a.w.G > 12 ? launch_tile_of<BM, BN, WM, WN, D, true, kFar>(a, stream)
                    : launch_tile_of<BM, BN, WM, WN, D, false, kFar>(a, stream);
}

// Which kernel (MxCost, mx_choose).  Measured, cold weights: e.g. 16 x 4096 rows of 16 / 32
// channels 4.9, 5.5 us, 64 x 64 tiles 7.9; 64 x 4096 9.2, 7.3, 8.6; 64 x 11008 23, 18, 11.6; 64
// tokens x 2 of 16 experts of 11008 rows of 32 channels 90, tiles of 64 / 128 / 256 91, 91, 106,
// 256 x 2 of 16 of 4096 59, 47, 56, 66; 512 x 11008 tiles of 64 / 128 / 256 31.9, 25.2, 36.9;
// 4096 x 4096 82, 53, 45.
constexpr MxCost kA4Shapes[] = {
    {kMxRows16x16, 16, 16, 4.9, 2.4, 1.6, "rows16x16"},
    {kMxRows16x32, 16, 32, 5.6, 4.1, 1.9, "rows16x32"},
    {kMxTile64x64, 64, 64, 8.1, 10.0, 4.4, "tile64x64"},
    {kMxTile128x128, 128, 128, 18.0, 25.0, 11.0, "tile128x128"},
    {kMxTile256x256, 256, 256, 44.0, 40.0, 40.0, "tile256x256"},
};

}  // namespace

const MxCost& mx_a4w4_shape(int64_t M, int64_t parts, int64_t N) {
  return mx_choose(kA4Shapes, sizeof(kA4Shapes) / sizeof(MxCost), M, parts, N);
}

qp_status run_mx_a4w4(const MxArgs& a, hipStream_t stream) {
  const int64_t apart = a.a.ldc > a.a.lds ? a.a.ldc : a.a.lds;
  const MxShape shape =
      mx_a4w4_shape(a.rows.M, a.rows.offsets ? a.rows.experts : 1, a.w.rows).shape;
  const bool weights = a.w.ldc < kMxMaxLd && a.w.lds < kMxMaxLd;
  // Rows past the offsets' reach, by tiles of 128 rows and by 16: 64 x 11008 x 4096 13 and 34
  // us, 128 x 4096 x 4096 16 and 27, 1024 rows 26 and 131, 4096 tokens x 2 of 8 experts of
  // 11008 x 4096 346 and 2917 (268 within reach).
  if (!mx_tile_reaches(a.rows, apart) || !weights) {
    if (shape >= kMxTile64x64 && weights) return launch_tile<128, 128, 2, 2, 2, true>(a, stream);
    return mx_launch_rows<mx4_t, 1, 8>(a, stream);
  }
  switch (shape) {
    case kMxTile256x256: return launch_tile<256, 256, 2, 4, 2>(a, stream);
    case kMxTile128x128: return launch_tile<128, 128, 2, 2, 2>(a, stream);
    case kMxTile64x64: return launch_tile<64, 64, 2, 2, 4>(a, stream);
    case kMxRows16x32: return mx_launch_stream<mx4_t, 2, 4>(a, stream);
    default: break;
  }
  return mx_launch_stream<mx4_t, 1, 4>(a, stream);
}

}  // namespace qp
