// mx4_w4_tile.hpp -- many float rows times MXFP4 weights (the mathematics: mx4.hpp).
//
// A workgroup owns BM rows x BN channels, its WM x WN waves 32 FM x 32 FN each, in
// registers.  K goes by in stages of 64: the rows' stage (of f32 rows a plane for
// each of the three bf16 pieces of their values) is in one of D LDS buffers, 128
// bytes of a row side by side; the weights' codes in one of kChunks buffers of 256 K
// (128 bytes of a channel), a quarter of whose channels comes in with every stage.  A
// wave reads its channels' 16 bytes (32 K, lane l: channel l%32, the stage's 32-block
// l/32) and converts a word for each of the stage's four steps; the rows' operand of
// step t is piece 4 (l/32) + t of the row.  Weights are the MFMA's first operand.
//
// 4096^3 bf16, 256 x 256 tiles: 105 us, 1.31 PFLOP/s, the MFMAs busy for 62% of its
// cycles; with K it grows at 1.47 PFLOP/s (the library's product of bf16 matrices of 8192^3
// reaches 1.49), the rest are launch, first loads and the sums' way out.  1024 x 4096 x
// 4096 by 128 x 128 tiles 38 us, 32 x 176128 x 4096 by 32 x 128 99, 3.9 TB/s of weights;
// 4096^3 f32 454 (128 x 128, three MFMAs a term: 0.91 PFLOP/s of them).
//
// f16 rows: the weights go in as f16 and the rows as they are; where one of a
// workgroup's scales turned out to be out of f16's reach and not to be of a block of
// zeros (mx_no_f16_among) it begins again, with the weights as bf16 and the rows as two
// bf16 pieces, twice the MFMAs and the cuts.  (Deciding stage by stage instead doubled
// the registers; a look over all scales first took 64 tokens x 2 of 16 experts of 11008
// x 4096 from 110 to 122 us.)
#pragma once

#include <type_traits>

#include "mx4_rows.hpp"
#include "mx4_stream.hpp"
#include "mx4_tile.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

template <typename T, int BM, int BN, int WM, int WN, int D>
struct W4MxTile {
  static constexpr int NW = WM * WN, FM = BM / (32 * WM), FN = BN / (32 * WN);
  static constexpr int NP = sizeof(T) == 4 ? 3 : 1;  // planes
  static constexpr int kX = BM * 128 * NP, kW = BN * 128, kScales = BN * 8;
  static constexpr int kAhead = D == 2 ? 1 : 2;       // chunks of 256 K under way
  static constexpr int kChunks = kAhead + 1;
  static constexpr int kA = (BM / 8 + NW - 1) / NW;   // direct loads of a stage's rows a wave
  // where a wave without a share loads to
  static constexpr int kIdle = kA * 8 * NW > BM ? 1024 : 0;
  static constexpr int kRing = D * kX + kChunks * (kW + kScales) + kIdle;
  static constexpr int kOut = NW * 32 * mx_out_ld(FN) * 4;
  static constexpr int kLds = kRing > kOut ? kRing : kOut;
};

// kDirect (16-bit rows at multiples of 4 bytes): the rows come by direct loads, and
// the first operands of a stage are read behind the barrier before the last MFMAs of
// the stage before.  Else (D = 2) through registers, where f32 is cut into pieces.
template <typename T, bool kDirect, int BM, int BN, int WM, int WN, int D, bool kOnce>
__global__ __launch_bounds__(WM * WN * 64) void mx_w4_tile_kernel(MxArgs a, uint32_t row_slots,
                                                                 uint32_t col_groups) {
  using L = W4MxTile<T, BM, BN, WM, WN, D>;
  constexpr int NW = L::NW, FM = L::FM, FN = L::FN, NP = L::NP;
  constexpr int kA = L::kA;
  constexpr int kSlots = kDirect ? 1 : kA;  // pieces of eight elements a thread and stage
  constexpr bool kF16 = __is_same(T, f16_t);
  static_assert(BN == 32 * NW && (kDirect || kA * 8 * NW == BM), "shares");
  static_assert(D == 2 || (D == 4 && kDirect), "buffers of the rows");
  extern __shared__ __attribute__((aligned(16))) uint8_t mx_lds[];
  lds_u8* const xbuf = (lds_u8*)mx_lds;
  lds_u8* const wbuf = xbuf + D * L::kX;
  lds_u8* const sbuf = wbuf + L::kChunks * L::kW;
  lds_u8* const idle = sbuf + L::kChunks * L::kScales;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  W4Tile tile;
  uint32_t group;
  if (!mx_take_tile<BM, (BM >= 256)>(a.rows, row_slots, col_groups, tile, group)) return;
  const int64_t n0 = (int64_t)group * BN;
  const int64_t N = a.w.rows, K = a.w.K;
  if (a.rows.offsets && tile.expert == a.rows.experts) {  // rows of no expert
    for (int64_t r = tile.r0 + wave; r < tile.r1; r += NW)
      for (int64_t n = n0 + lane; n < n0 + BN && n < N; n += 64)
        w4_store(a.Y, a.y_dtype, r * a.ldy + n, 0.0f);
    return;
  }

  // what a lane loads: a piece of row lane / 8 of eight; rows past the tile's end
  // repeat its last row
  const int lrow = lane >> 3;
  auto piece = [&](int j) { return (lane & 7) ^ mx_turn((wave * kA + j) * 8 + lrow); };
  const T* xbase = static_cast<const T*>(a.X);
  int64_t first = 0;
  if (!a.rows.map) {
    first = tile.r0;
    xbase += first * a.ldx;
  }
  int64_t source[kA];
  mx_sources(a.rows, tile, first, [&](int j) { return (wave * kA + j) * 8 + lrow; }, source);
  uint32_t vx[kDirect ? kA : 1];
  const T* px[kDirect ? 1 : kSlots];
  if constexpr (kDirect) {
#pragma unroll
    for (int j = 0; j < kA; ++j)
      vx[j] = (uint32_t)(source[j] * a.ldx * (int64_t)sizeof(T)) + piece(j) * 16;
  } else {
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      px[j] = xbase + source[j] * a.ldx;
  }
  const uint8_t* const wbase = a.w.codes + tile.expert * a.w.cstride + n0 * a.w.ldc;
  const uint8_t* const swbase = a.w.scales + tile.expert * a.w.sstride + n0 * a.w.lds;
  const int64_t last_n = N - 1 - n0;
  // quarter q of the channels: rows q BN/4 + wave 8 + lane/8
  uint32_t vw[4], vs;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t n = q * (BN / 4) + wave * 8 + lrow;
    vw[q] = (uint32_t)((n < last_n ? n : last_n) * a.w.ldc) +
            ((lane & 7) ^ mx_turn(wave * 8 + lrow)) * 16;
  }
  static_assert(BN / 4 % 16 == 0, "turn of a quarter's rows");
  {
    const int64_t n = wave * 32 + (lane >> 1);
    vs = (uint32_t)((n < last_n ? n : last_n) * a.w.lds) + (lane & 1) * 4;
  }

  const int G = (int)a.w.G, full = (int)(K / 64), words = (G + 3) / 4;
  auto issue_x = [&](int s) {
    lds_u8* const to = xbuf + (s % D) * L::kX;
#pragma unroll
    for (int j = 0; j < kA; ++j) {
      const int i = wave * kA + j;
      const bool mine = L::kIdle == 0 || i < BM / 8;
      dma_to_lds<16>(xbase, s < full && mine ? 0x7fffffff : 0, mine ? to + i * 1024 : idle, vx[j],
                     s * 128);
    }
  };
  // codes past the row's last block and words past its last scale are read from the
  // 256 K's first; past the last 256 K nothing is asked for
  auto issue_w = [&](int c, int q) {
    const int p = (lane & 7) ^ mx_turn(wave * 8 + lrow);
    const uint32_t back = c * 8 + p < G ? 0u : p * 16u;
    dma_to_lds<16, kOnce>(wbase, c * 8 < G ? 0x7fffffff : 0,
                          wbuf + (c % L::kChunks) * L::kW + (q * (BN / 4) + wave * 8) * 128,
                          vw[q] - back, c * 128);
  };
  auto issue_s = [&](int c) {
    const uint32_t back = c * 2 + (lane & 1) < words ? 0u : (lane & 1) * 4u;
    dma_to_lds<4>(swbase, c * 8 < G ? 0x7fffffff : 0,
                  sbuf + (c % L::kChunks) * L::kScales + wave * 256, vs - back, c * 8);
  };
  // what comes in behind stage s (of place `place` in its 256 K): the rows of stage
  // s + D and the next quarter of the weights of the 256 K that are kAhead on
  auto issue = [&](int s, auto place) {
    constexpr int kNext = (decltype(place)::value + 1) % 4;
    if constexpr (kDirect) issue_x(s + D);
    issue_w((s + 1) / 4 + L::kAhead, kNext);
    if constexpr (kNext == 0) issue_s((s + 1) / 4 + L::kAhead);
  };

  // F x FN operands a wave
  auto run = [&](auto operands) {
    constexpr int F = decltype(operands)::value;
    f32x16 acc[FN][F];

    const int l32 = lane & 31, half = lane >> 5;
    const uint32_t sel = half ? 0x07050301u : 0x06040200u;  // the half's scale of each 64 K
    const int arow = wm * 32 * F + l32, brow = wn * 32 * FN + l32;
    struct Rows {
      u32x4 x[F][NP];
    };
    struct Weights {
      u32x4 q[FN];
      float s[FN];
    };
    auto read_x = [&](Rows& o, int s, int step) {
      const lds_u8* const from = xbuf + (s % D) * L::kX;
      const int at = ((4 * half + step) ^ mx_turn(l32)) * 16;
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int i = 0; i < NP; ++i)
          o.x[j][i] = *(const __attribute__((address_space(3))) u32x4*)(
              from + (i * BM + arow + j * 32) * 128 + at);
    };
    auto read_w = [&](Weights& o, int s) {
      const int c = s >> 2, p = s & 3;
      const lds_u8* const from = wbuf + (c % L::kChunks) * L::kW;
      const lds_u8* const st = sbuf + (c % L::kChunks) * L::kScales;
      const int at = ((2 * p + half) ^ mx_turn(l32)) * 16;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        o.q[i] =
            *(const __attribute__((address_space(3))) u32x4*)(from + (brow + i * 32) * 128 + at);
        o.s[i] = mx_scale(st[(brow + i * 32) * 8 + 2 * p + half]);
      }
    };
    // a step's weights as operands, and the step
    auto unpack = [&](u32x4 (&v)[FN], const Weights& w, int step, auto kind) {
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        if constexpr (decltype(kind)::value)
          v[i] = __builtin_bit_cast(u32x4, mx_unpack_f16(w.q[i][step], w.s[i]));
        else
          v[i] = __builtin_bit_cast(u32x4, mx_unpack(w.q[i][step], w.s[i]));
      }
    };
    auto multiply = [&](const Rows& x, const u32x4 (&v)[FN], auto kind) {
      constexpr bool kAsF16 = decltype(kind)::value;
      constexpr int kPieces = kAsF16 ? 1 : kF16 ? 2 : NP;
#pragma unroll
      for (int j = 0; j < F; ++j) {
        if constexpr (kAsF16) {
#pragma unroll
          for (int i = 0; i < FN; ++i)
            acc[i][j] = mx_mfma_f16(__builtin_bit_cast(f16x8, v[i]),
                                    __builtin_bit_cast(f16x8, x.x[j][0]), acc[i][j]);
        } else {
          bf16x8 xv[kPieces];
          if constexpr (kF16)
            MxFrag<f16_t>{x.x[j][0]}.split(xv);
          else
#pragma unroll
            for (int n = 0; n < NP; ++n) xv[n] = __builtin_bit_cast(bf16x8, x.x[j][n]);
#pragma unroll
          for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int n = 0; n < kPieces; ++n)
              acc[i][j] = mx_mfma_bf16(__builtin_bit_cast(bf16x8, v[i]), xv[n], acc[i][j]);
        }
      }
    };
    // the rows through registers: their pieces of stage s, the part before K
    auto fetch = [&](MxFrag<T> (&f)[kSlots], int s) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        const int64_t k = (int64_t)s * 64 + piece(j) * 8, left = K - k;
        f[j].load_n(px[kDirect ? 0 : j] + (left > 0 ? k : 0),
                    left > 8 ? 8 : left < 0 ? 0 : (int)left);
      }
    };
    auto fetch_full = [&](MxFrag<T> (&f)[kSlots], int s) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        f[j].load(px[kDirect ? 0 : j] + (int64_t)s * 64 + piece(j) * 8);
    };
    auto put_one = [&](const MxFrag<T>& f, int s, int j) {
      lds_u8* const at = xbuf + (s % D) * L::kX + ((wave * kSlots + j) * 8 + lrow) * 128 +
                         (lane & 7) * 16;
      if constexpr (NP == 1) {
        *(__attribute__((address_space(3))) u32x4*)at = f.v;
      } else {
        bf16x8 v[NP];
        f.split(v);
#pragma unroll
        for (int i = 0; i < NP; ++i)
          *(__attribute__((address_space(3))) bf16x8*)(at + i * BM * 128) = v[i];
      }
    };
    auto put = [&](const MxFrag<T> (&f)[kSlots], int s) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j) put_one(f[j], s, j);
    };

    using P0 = std::integral_constant<int, 0>;
    using P1 = std::integral_constant<int, 1>;
    using P2 = std::integral_constant<int, 2>;
    using P3 = std::integral_constant<int, 3>;
    using std::false_type;
    using std::true_type;
    // The next stage is there for everyone (D = 4: all but the loads of the two stages
    // before this one are done, the weights' are four stages ahead of their use), and
    // everyone has read all of this one.
    auto arrive = [&](auto place) {
      constexpr int P = decltype(place)::value;
      // (rows through registers: their loads are left under way, and the weights' are only
      // awaited where their 256 K begin)
      if constexpr (kDirect || P == 3)
        wait_vmcnt<D == 2 ? 0 : 2 * (kA + 1) + (P < 2 ? 1 : 0)>();
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    MxFrag<T> f[kSlots];
    Rows even, odd;
    Weights now, next;
    auto each = [&](auto stage) {
      int s = 0;
      for (; s + 4 <= full; s += 4) {
        stage(s, P0{});
        stage(s + 1, P1{});
        stage(s + 2, P2{});
        stage(s + 3, P3{});
      }
      if (s < full) stage(s, P0{});
      if (s + 1 < full) stage(s + 1, P1{});
      if (s + 2 < full) stage(s + 2, P2{});
    };
    // All whole stages; with f16 weights, whether one of the wave's was no f16 value.
    auto pass = [&](auto kind) {
      bool out = false;
#pragma unroll
      for (int c = 0; c < L::kAhead; ++c) {
#pragma unroll
        for (int q = 0; q < 4; ++q) issue_w(c, q);
        issue_s(c);
      }
      if constexpr (kDirect) {
#pragma unroll
        for (int s = 0; s < D - 1; ++s) issue_x(s);
      } else if (full > 0) {
        fetch_full(f, 0);
        put(f, 0);
      }
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
      wait_vmcnt<0>();
      __syncthreads();
      if constexpr (kDirect) issue_x(D - 1);
      issue_w(L::kAhead, 0);
      issue_s(L::kAhead);
      // a step's unpacking in between the MFMAs of the one before (4096 tokens x 2 of 8 experts
      // of 11008 x 4096 bf16 688 us without, 671 with)
      auto mix = [&] {
#pragma unroll
        for (int i = 0; i < F * FN; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // an MFMA
          __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);  // VALU instructions
        }
      };
      auto look = [&] {
        if constexpr (decltype(kind)::value)
#pragma unroll
          for (int i = 0; i < FN; ++i) out |= !mx_f16_scale(now.s[i]);
      };
      if constexpr (kDirect) {
        u32x4 va[FN], vb[FN];
        read_x(even, 0, 0);
        read_w(now, 0);
        unpack(va, now, 0, kind);
        // (no branch between MFMAs: the compiler would move them past it, behind the
        // barrier)
        auto steps = [&](int s, auto place) {
          read_x(odd, s, 1);
          __builtin_amdgcn_sched_barrier(0);
          unpack(vb, now, 1, kind);
          multiply(even, va, kind);
          mix();
          __builtin_amdgcn_sched_barrier(0);
          read_x(even, s, 2);
          __builtin_amdgcn_sched_barrier(0);
          unpack(va, now, 2, kind);
          multiply(odd, vb, kind);
          look();
          mix();
          __builtin_amdgcn_sched_barrier(0);
          read_x(odd, s, 3);
          __builtin_amdgcn_sched_barrier(0);
          unpack(vb, now, 3, kind);
          multiply(even, va, kind);
          mix();
          __builtin_amdgcn_sched_barrier(0);
          arrive(place);
          // (which first: 4096^3 by 256 x 256 tiles 106 us loads first, 103 last; 1024 x 4096 x
          // 4096 by 128 x 128 40 and 47)
          if constexpr (BM < 256) issue(s, place);
          read_x(even, s + 1, 0);
          read_w(next, s + 1);
          __builtin_amdgcn_sched_barrier(0);
          multiply(odd, vb, kind);
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (BM >= 256) issue(s, place);
          now = next;
          unpack(va, now, 0, kind);
        };
        if (tile.r0 + wm * 32 * F >= tile.r1) {
          // (a wave without rows only loads, and leaves its SIMD to the others)
          each([&](int s, auto place) {
            arrive(place);
            issue(s, place);
          });
        } else {
          each(steps);
        }
      } else {
        // a piece of the next stage's rows is cut and put down and one of the stage after it
        // loaded with every step (4096^3 f32: all at the stage's ends 543 us, so 454)
        static_assert(kDirect || kSlots == 4, "pieces of a step");
        if (full > 0) fetch_full(f, full > 1 ? 1 : 0);
        each([&](int s, auto place) {
          const int after = s + 2 < full ? s + 2 : full - 1;
          read_w(now, s);
          read_x(even, s, 0);
          look();
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            Rows& here = t % 2 ? odd : even;
            if (t < 3) read_x(t % 2 ? even : odd, s, t + 1);
            __builtin_amdgcn_sched_barrier(0);
            u32x4 v[FN];
            unpack(v, now, t, kind);
            multiply(here, v, kind);
            put_one(f[t % kSlots], s + 1, t % kSlots);
            f[t % kSlots].load(px[kDirect ? 0 : t] + (int64_t)after * 64 + piece(t) * 8);
            __builtin_amdgcn_sched_barrier(0);
          }
          arrive(place);
          issue(s, place);
        });
      }
      wait_vmcnt<0>();
      return out;
    };
    if constexpr (kF16) {
      bool out = __syncthreads_or(pass(true_type{}));
      if (out) {
        const int64_t rows = last_n + 1 < BN ? last_n + 1 : BN;
        out = __syncthreads_or(mx_no_f16_among(wbase, a.w.ldc, swbase, a.w.lds, rows, 2 * full,
                                               NW * 64));
      }
      if (out) pass(false_type{});
    } else {
      pass(false_type{});
    }
    __syncthreads();
    if ((int64_t)full * 64 < K) {
      // the stage that K cuts: its rows through registers, zeros from K on; zero scales
      // past the last block (what is found there could be a NaN)
      if constexpr (kDirect) {
        // (the pieces of a direct load's lanes, by plain loads)
        lds_u8* const to = xbuf + (full % D) * L::kX;
#pragma unroll 1
        for (int j = 0; j < kA; ++j) {
          const int row = (wave * kA + j) * 8 + lrow;
          if (row >= BM) break;
          const int64_t k = (int64_t)full * 64 + piece(j) * 8, left = K - k;
          int64_t x[1];
          mx_sources(a.rows, tile, first, [&](int) { return row; }, x);
          const T* p = xbase + x[0] * a.ldx;
          const Piece<T> one =
              load_piece(p + (left > 0 ? k : 0), left > 8 ? 8 : left < 0 ? 0 : (int)left);
          *(__attribute__((address_space(3))) u32x4*)(to + row * 128 + (lane & 7) * 16) = one.v;
        }
      } else {
        fetch(f, full);
        put(f, full);
      }
      __syncthreads();
      read_w(now, full);
      if (2 * full + half >= G) {
#pragma unroll
        for (int i = 0; i < FN; ++i) now.s[i] = mx_scale(0);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        u32x4 v[FN];
        read_x(even, full, t);
        unpack(v, now, t, false_type{});
        multiply(even, v, false_type{});
      }
      __syncthreads();
    }

    mx_store_tile<F, FN>(acc, a, tile, wm * F * 32, n0 + wn * FN * 32,
                          reinterpret_cast<float*>(mx_lds) + wave * 32 * mx_out_ld(FN));
  };
  constexpr int kHalf = kDirect && FM > 1 ? FM / 2 : FM;
  if (kHalf < FM && tile.r1 - tile.r0 <= BM / 2)
    run(std::integral_constant<int, kHalf>{});
  else
    run(std::integral_constant<int, FM>{});
}

template <typename T, bool kDirect, int BM, int BN, int WM, int WN, int D, bool kOnce = false>
qp_status mx_launch_w4_tile(const MxArgs& a, hipStream_t stream) {
  using L = W4MxTile<T, BM, BN, WM, WN, D>;
  const int64_t slots = w4_tile_slots(a.rows, BM), groups = ceil_div(a.w.rows, BN);
  const int64_t grid = mx_tile_grid(slots, groups, BM >= 256);
  QP_REQUIRE(grid * L::NW * 64 < (INT64_C(1) << 32), QP_EUNSUPPORTED,
             "qgemm_w4_mx: rows and channels for more than 2^32 threads");
  auto kern = mx_w4_tile_kernel<T, kDirect, BM, BN, WM, WN, D, kOnce>;
  static std::atomic<uint64_t> reserved{0};
  if (qp_status st =
          mx_reserve_lds("qgemm_w4_mx", reinterpret_cast<const void*>(kern), L::kLds, reserved))
    return st;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(L::NW * 64), L::kLds, stream, a,
                     (uint32_t)slots, (uint32_t)groups);
  return check_launch("qgemm_w4_mx (many rows)");
}

template <typename T>
qp_status mx_run_16bit(const MxArgs& a, hipStream_t stream) {
  const MxShape shape = mx_w4_shape(__is_same(T, f16_t) ? QP_F16 : QP_BF16, a.rows.M,
                                    a.rows.offsets ? a.rows.experts : 1, a.w.rows)
                            .shape;
  // What direct loads cannot take goes through registers: rows at odd addresses or odd
  // strides (bf16 16 x 4096 x 4096 15.9 us and 6.4 by direct loads, 64 rows 28.8 and 9.8, 256
  // 104 and 20, 1024 54 and 39, 4096 167 and 105; 64 tokens x 2 of 16 experts of 11008 x 4096
  // 223 and 93) and rows too far apart.
  const bool weights = a.w.ldc < kMxMaxLd && a.w.lds < kMxMaxLd;
  if ((uintptr_t)a.X % 4 || a.ldx % 2 || !mx_tile_reaches(a.rows, a.ldx * 2) || !weights) {
    if (shape >= kMxTile128x128 && weights)
      return mx_launch_w4_tile<T, false, 128, 128, 2, 2, 2>(a, stream);
    return mx_launch_rows<T, 2, 8>(a, stream);
  }
  switch (shape) {
    case kMxRows16x16: return mx_launch_stream<T, 1, 4>(a, stream);
    case kMxRows16x32: return mx_launch_stream<T, 2, 4>(a, stream);
    case kMxRows16x48: return mx_launch_stream<T, 3, 4>(a, stream);
    // Several rounds of workgroups: two waves each, two to a CU, so that one finds its tile
    // and rows while the other's loads are under way (16 tokens x 2 of 16 experts of 11008 x
    // 4096 bf16 86 and 103 us, 8 experts of 4096 x 4096 with 4 tokens 17.9 and 13.0).
    case kMxRows16x64:
      return mx_row_tiles(a) * ceil_div(a.w.rows, 64) > 512
                 ? mx_launch_stream<T, 4, 2>(a, stream)
                 : mx_launch_stream<T, 4, 4>(a, stream);
    // (loads for once: 32 x 11008 x 4096 bf16 16.1 -> 15.6 us, 256 tokens x 4 of 32 experts of
    // 4096 x 2048 70.4 -> 67.6; 128 x 4096 x 11008 31.2 -> 33.3)
    case kMxTile32x64:
      return mx_read_once(a, 32) ? mx_launch_w4_tile<T, true, 32, 64, 1, 2, 4, true>(a, stream)
                                 : mx_launch_w4_tile<T, true, 32, 64, 1, 2, 4>(a, stream);
    case kMxTile32x128:
      return mx_read_once(a, 32) ? mx_launch_w4_tile<T, true, 32, 128, 1, 4, 4, true>(a, stream)
                                 : mx_launch_w4_tile<T, true, 32, 128, 1, 4, 4>(a, stream);
    // Up to one to a CU, with loads of rows and weights further ahead; else two to a CU
    // (256 x 11008 x 4096 bf16 38 and 49 us, 1024 x 4096 x 4096 39.4 and 40.4; two rounds of
    // the first, 1536 x 4096 x 4096, 70 and 54).
    case kMxTile128x128:
      return w4_tile_slots(a.rows, 128) * ceil_div(a.w.rows, 128) <= 256
                 ? mx_launch_w4_tile<T, true, 128, 128, 2, 2, 4>(a, stream)
                 : mx_launch_w4_tile<T, true, 128, 128, 2, 2, 2>(a, stream);
    default: break;
  }
  return mx_launch_w4_tile<T, true, 256, 256, 2, 4, 2>(a, stream);
}

}  // namespace
}  // namespace qp
