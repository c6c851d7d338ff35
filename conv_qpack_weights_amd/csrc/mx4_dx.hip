// mx4_dx.hip -- the gradient of the products with MXFP4 weights to their rows:
//   dx[r,k] = sum_n dy[r,n] w[n,k]
// The sum runs along the channels, a row of the codes along k: the MFMA operand
// of a column wants eight channels' values of it side by side.  A lane takes a
// word (eight k) of each of eight channels, converts them to bf16 with their
// channels' scales, exactly, and pairs the channels' halves up (32 conversions
// and 32 v_perm for eight operands, no LDS): operand j then holds column 8 i + j
// in lane i of 16, and a lane ends with eight neighbouring columns of a row.
#include <cstdio>
#include <type_traits>

#include "mx4.hpp"
#include "mx4_tile.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

struct MxDxArgs {
  MxMat w;
  W4Rows rows;
  const void* dY;
  int64_t lddy;
  void* dX;
  int32_t dtype;
  int64_t lddx;
  float* part;         // [splits][M][K] when the channels are split over workgroups
};

// low halves of two words: (lo(a), lo(b)) as two bf16, a first
__device__ __forceinline__ uint32_t lo_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

// Words of eight channels -> the operands of eight columns.
__device__ __forceinline__ void mx_columns(const uint32_t (&w)[8], const float (&s)[8],
                                           bf16x8 (&o)[8]) {
  u32x4 c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __builtin_bit_cast(u32x4, mx_unpack(w[i], s[i]));
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    u32x4 lo, hi;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      lo[r] = lo_halves(c[2 * r][m], c[2 * r + 1][m]);
      hi[r] = hi_halves(c[2 * r][m], c[2 * r + 1][m]);
    }
    o[2 * m] = __builtin_bit_cast(bf16x8, lo);
    o[2 * m + 1] = __builtin_bit_cast(bf16x8, hi);
  }
}

// ---- few rows ------------------------------------------------------------------
// A workgroup owns 16 rows and 128 columns of one split of the channels; its
// waves take every kWaves-th step of 32 channels and meet in LDS in a fixed
// order.  More than one split: the sums go to `part`, added up by the kernel
// below.
template <typename T, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void mx_dx_rows_kernel(MxDxArgs a, uint32_t row_slots,
                                                                 uint32_t splits) {
  constexpr int NP = MxFrag<T>::kPieces;
  __shared__ f32x4 red[kWaves][8][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // neighbouring column blocks, which share the channels' lines, on one XCD
  const uint32_t cols = (uint32_t)((a.w.K + 127) / 128);
  const uint32_t id = xcd_run(blockIdx.x, gridDim.x);
  const uint32_t slot = id % row_slots, rest = id / row_slots;
  const uint32_t cb = rest % cols, split = rest / cols;
  const W4Tile tile = w4_find_tile<16>(a.rows, slot);
  if (tile.expert < 0) return;
  const int64_t k0 = (int64_t)cb * 128, N = a.w.rows, K = a.w.K;
  const bool none = a.rows.offsets && tile.expert == a.rows.experts;
  const int ch = lane & 15, quad = lane >> 4;

  f32x4 acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  if (!none) {
    int64_t r = tile.r0 + ch;
    r = r < tile.r1 ? r : tile.r1 - 1;
    const T* const dy = static_cast<const T*>(a.dY) + r * a.lddy;
    // columns past K's last block read the row's first word: not stored
    const bool col_in = k0 / 32 + ch / 4 < a.w.G;
    const uint8_t* codes = a.w.codes + tile.expert * a.w.cstride + (col_in ? k0 / 2 + 4 * ch : 0);
    const uint8_t* scales = a.w.scales + tile.expert * a.w.sstride + k0 / 32;
    const uint32_t shift = 8 * (ch / 4);

    const int64_t steps = (N + 31) / 32;
    for (int64_t s = (int64_t)split * kWaves + wave; s < steps; s += (int64_t)splits * kWaves) {
      const int64_t n0 = s * 32 + quad * 8;
      uint32_t w[8], sc[8];
      MxFrag<T> x;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t n = n0 + i < N ? n0 + i : N - 1;
        w[i] = *reinterpret_cast<const uint32_t*>(codes + n * a.w.ldc);
        sc[i] = *reinterpret_cast<const uint32_t*>(scales + n * a.w.lds);
      }
      const int64_t left = N - n0;
      const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
      x.load_n(dy + (n > 0 ? n0 : 0), n);
      float by[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)  // (a channel past the last: its scale could be a NaN)
        by[i] = mx_scale(i < n ? (sc[i] >> shift) & 0xffu : 0u);
      bf16x8 o[8];
      mx_columns(w, by, o);
      bf16x8 xv[NP];
      x.split(xv);
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int p = 0; p < NP; ++p) acc[j] = mfma32(xv[p], o[j], acc[j]);
    }
  }

  // thread: 8 columns of a row
#pragma unroll
  for (int j = 0; j < 8; ++j) red[wave][j][lane] = acc[j];
  __syncthreads();
  for (int i = threadIdx.x; i < 256; i += kWaves * 64) {
    const int m = i >> 4, c = i & 15;
    const int64_t r = tile.r0 + m, col = k0 + 8 * c;
    if (r >= tile.r1 || col >= K) continue;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = 0.0f;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) y[j] += red[v][j][(m >> 2) * 16 + c][m & 3];
    }
    const int n = K - col < 8 ? (int)(K - col) : 8;
    if (splits > 1)
      w4_store8(a.part + (int64_t)split * a.rows.M * K, QP_F32, r * K + col, y, n);
    else
      w4_store8(a.dX, a.dtype, r * a.lddx + col, y, n);
  }
}

// dx[r] = the splits' sums added up, in order.
__global__ __launch_bounds__(256) void mx_dx_sum_kernel(const float* __restrict__ part, int64_t M,
                                                        int64_t K, uint32_t splits,
                                                        uint32_t pieces, void* dX, int32_t dtype,
                                                        int64_t lddx) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = at / pieces, k = (at - r * pieces) * 8;
  if (r >= M) return;
  const int n = K - k < 8 ? (int)(K - k) : 8;
  float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const float* p = part + r * K + k;
  for (uint32_t s = 0; s < splits; ++s, p += M * K) {
    const Piece<float> lo = load_piece(p, n), hi = load_piece(p + (n > 4 ? 4 : 0), n - 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] += lo.get(i);
      y[4 + i] += hi.get(i);
    }
  }
  w4_store8(dX, dtype, r * lddx + k, y, n);
}

// ---- many rows -----------------------------------------------------------------
// A workgroup owns BM rows x BC columns, its WM x WN waves 32 FM x 64 each, in
// registers.  The channels go by in stages of 64: dY's stage (of f32 rows a plane for
// each of the three bf16 pieces) comes into one of two LDS buffers by direct loads or
// through registers, as the rows of mx4_w4_tile.hpp; the weights' codes and scales into
// one of two small buffers, two stages ahead (loaded by their users instead, two
// bytes at a time, they held a 256 x 256 tile up for a quarter of its time).  A stage
// ahead a thread takes four columns (two bytes) of eight channels from there, converts
// and pairs them up, and writes for each of its columns the eight channels' values, 16
// bytes, to the other of two buffers, so that every weight is converted once in a
// workgroup.  In that buffer column 4u + j of a wave's 64 is row 16 j + u: 16 threads
// then write 16 rows, whose places meet every bank alike (mx_turn).
// f16 rows: as there, again from the start where a weight turned out to be no f16 value.
// 4096^3, 256 x 256 tiles: bf16 117 us (1.17 PFLOP/s), f16 122; 1024 x 4096 x 4096 by 128 x 128
// 49 (rows loaded further ahead: no faster, one wave a SIMD has the conversion, 16 small LDS
// reads and 4 writes, between its MFMAs).
template <typename T, int BM, int BC, int WM, int WN>
struct MxDxTile {
  static constexpr int NW = WM * WN, FM = BM / (32 * WM);
  static constexpr int NP = sizeof(T) == 4 ? 3 : 1;
  static constexpr int kX = BM * 128 * NP, kW = BC * 128;
  static constexpr int kRaw = 32 * BC, kScales = 2 * BC;   // 64 channels' codes and scales
  static constexpr int kIdle = 256;  // where a wave without a share of the scales loads to
  static constexpr int kRing = 2 * (kX + kW + kRaw + kScales) + kIdle;
  static constexpr int kOutLd = 64 + 4;
  static constexpr int kOut = NW * 32 * kOutLd * 4;
  static constexpr int kLds = kRing > kOut ? kRing : kOut;
};

template <typename T, bool kDirect, int BM, int BC, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void mx_dx_tile_kernel(MxDxArgs a, uint32_t row_slots,
                                                                 uint32_t col_groups) {
  using L = MxDxTile<T, BM, BC, WM, WN>;
  constexpr int NW = L::NW, FM = L::FM, FN = 2, NP = L::NP;
  constexpr bool kF16 = __is_same(T, f16_t);
  constexpr int kA = BM / 8 / NW;  // pieces of eight elements of dY a thread and stage
  static_assert(kA * 8 * NW == BM && kA % 2 == 0 && BC == 64 * WN && BC == 32 * NW, "shares");
  extern __shared__ __attribute__((aligned(16))) uint8_t mx_lds[];
  lds_u8* const xbuf = (lds_u8*)mx_lds;
  lds_u8* const wbuf = xbuf + 2 * L::kX;
  lds_u8* const raws = wbuf + 2 * L::kW;
  lds_u8* const scs = raws + 2 * L::kRaw;
  lds_u8* const idle = scs + 2 * L::kScales;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  W4Tile tile;
  uint32_t group;
  if (!mx_take_tile<BM, (BM >= 256)>(a.rows, row_slots, col_groups, tile, group)) return;
  const int64_t k0 = (int64_t)group * BC;
  const int64_t N = a.w.rows, K = a.w.K;
  if (a.rows.offsets && tile.expert == a.rows.experts) {  // rows of no expert
    for (int64_t r = tile.r0 + wave; r < tile.r1; r += NW)
      for (int64_t k = k0 + lane; k < k0 + BC && k < K; k += 64)
        w4_store(a.dX, a.dtype, r * a.lddx + k, 0.0f);
    return;
  }

  // dY: a lane loads a piece of row lane / 8 of eight; rows past the tile's end repeat
  // its last row
  const int lrow = lane >> 3;
  auto piece = [&](int j) { return (lane & 7) ^ mx_turn(j * 8 + lrow); };
  const T* const xbase = static_cast<const T*>(a.dY) + tile.r0 * a.lddy;
  auto row_of = [&](int j) {
    const int64_t r = (wave * kA + j) * 8 + lrow, last = tile.r1 - 1 - tile.r0;
    return (r < last ? r : last) * a.lddy;
  };
  uint32_t vx[kDirect ? kA : 1];
  const T* px[kDirect ? 1 : kA];
#pragma unroll
  for (int j = 0; j < kA; ++j) {
    if constexpr (kDirect)
      vx[j] = (uint32_t)(row_of(j) * (int64_t)sizeof(T)) + piece(j) * 16;
    else
      px[j] = xbase + row_of(j);
  }
  const int full = (int)(N / 64);
  auto issue_x = [&](int s) {
    const int range = s < full ? 0x7fffffff : 0;
    lds_u8* const to = xbuf + (s & 1) * L::kX;
#pragma unroll
    for (int j = 0; j < kA; ++j)
      dma_to_lds<16>(xbase, range, to + (wave * kA + j) * 1024, vx[j], s * 128);
  };
  // through registers: stage s, the part before N
  auto put = [&](const MxFrag<T>& f, int s, int j) {
    lds_u8* const at =
        xbuf + (s & 1) * L::kX + ((wave * kA + j) * 8 + lrow) * 128 + (lane & 7) * 16;
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
  auto fetch_full = [&](MxFrag<T> (&f)[kA], int s) {
#pragma unroll
    for (int j = 0; j < kA; ++j)
      f[j].load(px[kDirect ? 0 : j] + (int64_t)s * 64 + piece(j) * 8);
  };

  // the weights: a lane loads a piece of 32 columns of a channel, and a word of its
  // scales; columns past the last block repeat the group's first (they are not stored)
  const uint8_t* const codes = a.w.codes + tile.expert * a.w.cstride + k0 / 2;
  const uint8_t* const scales = a.w.scales + tile.expert * a.w.sstride + k0 / 32;
  constexpr int kPieces = BC / 32, kWords = BC / 128;  // of a channel
  const int blocks = a.w.G - k0 / 32 < kPieces ? (int)(a.w.G - k0 / 32) : kPieces;
  static_assert(64 * kPieces == 64 * NW, "one load of codes a wave");
  uint32_t vq, vs;
  {
    const int row = threadIdx.x / kPieces, c = threadIdx.x % kPieces;
    vq = (uint32_t)(row * a.w.ldc) + (c < blocks ? c : 0) * 16;
    const int srow = threadIdx.x / kWords & 63, w = threadIdx.x % kWords;
    vs = (uint32_t)(srow * a.w.lds) + (w * 4 < blocks ? w : 0) * 4;
  }
  auto issue_w = [&](int s) {
    const int range = s < full ? 0x7fffffff : 0;
    const int64_t row = s < full ? (int64_t)s * 64 : 0;
    dma_to_lds<16>(codes + row * a.w.ldc, range, raws + (s & 1) * L::kRaw + wave * 1024, vq, 0);
    const bool mine = wave < kWords;
    dma_to_lds<4>(scales + row * a.w.lds, mine ? range : 0,
                  mine ? scs + (s & 1) * L::kScales + wave * 256 : idle, vs, 0);
  };
  // a thread's share: columns 4u .. 4u + 3 of channels 8g .. 8g + 7 of a stage
  const int u = threadIdx.x % (BC / 4), g = threadIdx.x / (BC / 4);
  struct Raw {
    uint32_t q[8], s[8];
  };
  auto read_w = [&](Raw& w, int s) {
    const lds_u8* const q = raws + (s & 1) * L::kRaw + g * 8 * (BC / 2) + 2 * u;
    const lds_u8* const sc = scs + (s & 1) * L::kScales + g * 8 * kPieces + u / 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w.q[i] = *(const __attribute__((address_space(3))) uint16_t*)(q + i * (BC / 2));
      w.s[i] = sc[i * kPieces];
    }
  };
  // the stage that N cuts: channels past the last are zeros of scale 1 (what is found
  // there could be a NaN)
  auto load_w_cut = [&](Raw& w) {
    const bool in = u / 8 < blocks;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t n = (int64_t)full * 64 + g * 8 + i, at = n < N ? n : N - 1;
      const uint32_t q =
          *reinterpret_cast<const uint16_t*>(codes + at * a.w.ldc + (in ? 2 * u : 0));
      const uint32_t v = scales[at * a.w.lds + (in ? u / 8 : 0)];
      w.q[i] = n < N ? q : 0u;
      w.s[i] = n < N ? v : 127u;
    }
  };
  // (there: whether this is a stage at all; f16 weights: `out` is set where one is no
  // f16 value)
  bool out = false;
  // channels 2 r and 2 r + 1 of a share: word r of its four columns' operands
  auto pair_up = [&](u32x4 (&v)[4], const Raw& w, int r, auto kind, bool there) {
    uint32_t c[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t q = w.q[2 * r + i];
      const float by = mx_scale(w.s[2 * r + i]);
      if constexpr (decltype(kind)::value) {
        out |= there && !mx_f16_scale(by);
        c[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, by, 0));
        c[i][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, by, 1));
      } else {
        c[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, by, 0));
        c[i][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, by, 1));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j][r] = j & 1 ? hi_halves(c[0][j / 2], c[1][j / 2]) : lo_halves(c[0][j / 2], c[1][j / 2]);
  };
  auto put_w = [&](const u32x4 (&v)[4], int s) {
    lds_u8* const to = wbuf + (s & 1) * L::kW;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = u / 16 * 64 + j * 16 + u % 16;
      *(__attribute__((address_space(3))) u32x4*)(to + row * 128 + (g ^ mx_turn(row)) * 16) = v[j];
    }
  };
  auto convert = [&](const Raw& w, int s, auto kind, bool there) {
    u32x4 v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) pair_up(v, w, r, kind, there);
    put_w(v, s);
  };

  // F x FN operands a wave
  auto run = [&](auto operands) {
    constexpr int F = decltype(operands)::value;
    f32x16 acc[FN][F];

    const int l32 = lane & 31, half = lane >> 5;
    const int arow = wm * 32 * F + l32, brow = wn * 64 + l32;
    struct Operands {
      u32x4 x[F][NP], w[FN];
    };
    // 16 channels a step: lane l holds eight of row l%32 from 8 (l/32) on
    auto read = [&](Operands& o, int s, int step) {
      const lds_u8* const fx = xbuf + (s & 1) * L::kX;
      const lds_u8* const fw = wbuf + (s & 1) * L::kW;
      const int at = ((2 * step + half) ^ mx_turn(l32)) * 16;
#pragma unroll
      for (int i = 0; i < FN; ++i)
        o.w[i] = *(const __attribute__((address_space(3))) u32x4*)(fw + (brow + i * 32) * 128 + at);
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int n = 0; n < NP; ++n)
          o.x[j][n] = *(const __attribute__((address_space(3))) u32x4*)(
              fx + (n * BM + arow + j * 32) * 128 + at);
    };
    auto multiply = [&](const Operands& o, auto kind) {
      constexpr bool kAsF16 = decltype(kind)::value;
      constexpr int kPieces = kF16 && !kAsF16 ? 2 : NP;
#pragma unroll
      for (int j = 0; j < F; ++j) {
        if constexpr (kAsF16) {
#pragma unroll
          for (int i = 0; i < FN; ++i)
            acc[i][j] = mx_mfma_f16(__builtin_bit_cast(f16x8, o.w[i]),
                                    __builtin_bit_cast(f16x8, o.x[j][0]), acc[i][j]);
        } else {
          bf16x8 xv[kPieces];
          if constexpr (kF16)
            MxFrag<f16_t>{o.x[j][0]}.split(xv);
          else
#pragma unroll
            for (int n = 0; n < NP; ++n) xv[n] = __builtin_bit_cast(bf16x8, o.x[j][n]);
#pragma unroll
          for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int n = 0; n < kPieces; ++n)
              acc[i][j] = mx_mfma_bf16(__builtin_bit_cast(bf16x8, o.w[i]), xv[n], acc[i][j]);
        }
      }
    };

    using std::false_type;
    using std::true_type;
    // everyone's share of the next stage is there, and everyone has read all of this one
    auto arrive = [&]() {
      wait_vmcnt<0>();
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    auto all = [&](auto kind) {
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
      Raw raw;
      MxFrag<T> f[kA];
      Operands even, odd;
      if (full > 0) {
        issue_w(0);
        issue_w(1);
        if constexpr (kDirect) {
          issue_x(0);
        } else {
          fetch_full(f, 0);
#pragma unroll
          for (int j = 0; j < kA; ++j) put(f[j], 0, j);
        }
        arrive();
        read_w(raw, 0);
        convert(raw, 0, kind, true);
        arrive();
        issue_w(2);
        if constexpr (kDirect) {
          issue_x(1);
          read(even, 0, 0);
          read_w(raw, 1);
          // (no branch between MFMAs, as in the products)
          if (tile.r0 + wm * 32 * F < tile.r1) {
            // (the next stage's conversion spread over this one's MFMAs: 4096^3 f16 128 us in
            // one piece, 122 so)
            auto mix = [&] {
#pragma unroll
              for (int i = 0; i < F * FN; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // an MFMA
                __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);  // VALU instructions
              }
            };
            for (int s = 0; s < full; ++s) {
              const bool there = s + 1 < full;
              u32x4 v[4];
              read(odd, s, 1);
              __builtin_amdgcn_sched_barrier(0);
              pair_up(v, raw, 0, kind, there);
              multiply(even, kind);
              mix();
              __builtin_amdgcn_sched_barrier(0);
              read(even, s, 2);
              __builtin_amdgcn_sched_barrier(0);
              pair_up(v, raw, 1, kind, there);
              pair_up(v, raw, 2, kind, there);
              multiply(odd, kind);
              mix();
              __builtin_amdgcn_sched_barrier(0);
              read(odd, s, 3);
              __builtin_amdgcn_sched_barrier(0);
              pair_up(v, raw, 3, kind, there);
              put_w(v, s + 1);
              multiply(even, kind);
              mix();
              __builtin_amdgcn_sched_barrier(0);
              arrive();
              issue_w(s + 3);
              issue_x(s + 2);
              read(even, s + 1, 0);
              read_w(raw, s + 2);
              __builtin_amdgcn_sched_barrier(0);
              multiply(odd, kind);
              __builtin_amdgcn_sched_barrier(0);
            }
          } else {
            // (a wave without rows only brings its share of the weights)
            for (int s = 0; s < full; ++s) {
              read_w(raw, s + 1);
              convert(raw, s + 1, kind, s + 1 < full);
              arrive();
              issue_w(s + 3);
              issue_x(s + 2);
            }
          }
        } else {
          // two pieces of the next stage's rows are cut and put down and two of the stage after
          // it loaded with each of the first two steps (4096^3 f32: all at the stage's ends
          // 600 us, so 556)
          static_assert(kDirect || kA == 4, "pieces of a step");
          fetch_full(f, full > 1 ? 1 : 0);
          for (int s = 0; s < full; ++s) {
            const int after = s + 2 < full ? s + 2 : full - 1;
            read_w(raw, s + 1);
            read(even, s, 0);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              if (t < 3) read(t % 2 ? even : odd, s, t + 1);
              __builtin_amdgcn_sched_barrier(0);
              multiply(t % 2 ? odd : even, kind);
              if (t < 2) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                  const int j = (2 * t + p) % kA;
                  put(f[j], s + 1, j);
                  f[j].load(px[kDirect ? 0 : j] + (int64_t)after * 64 + piece(j) * 8);
                }
              } else if (t == 2) {
                convert(raw, s + 1, kind, s + 1 < full);
              }
              __builtin_amdgcn_sched_barrier(0);
            }
            arrive();
            issue_w(s + 3);
          }
        }
      }
      wait_vmcnt<0>();
      __syncthreads();
      if ((int64_t)full * 64 < N) {
        // the stage that N cuts: its rows through registers, zeros from N on
        load_w_cut(raw);
        convert(raw, full, kind, true);
#pragma unroll 1
        for (int j = 0; j < kA; ++j) {
          const int64_t n = (int64_t)full * 64 + piece(j) * 8, left = N - n;
          const T* p = xbase + row_of(j);
          MxFrag<T> one;
          one.load_n(p + (left > 0 ? n : 0), left > 8 ? 8 : left < 0 ? 0 : (int)left);
          put(one, full, j);
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          read(even, full, t);
          multiply(even, kind);
        }
        __syncthreads();
      }
    };
    if constexpr (kF16) {
      all(true_type{});
      out = __syncthreads_or(out);
      if (out) out = __syncthreads_or(mx_no_f16_among(codes, a.w.ldc, scales, a.w.lds, N, blocks,
                                                      NW * 64));
      if (out) all(false_type{});
    } else {
      all(false_type{});
    }

    // where all the wave's columns are there a lane has 16 neighbouring ones of a row, twice
    if (k0 + wn * 64 + 64 <= K) {
      auto store = [&](auto* X) {
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const int64_t r = tile.r0 + (wm * F + f) * 32 + l32;
          if (r < tile.r1) {
            auto* const at = X + r * a.lddx + k0 + wn * 64 + 16 * half;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float y[8];
#pragma unroll
                for (int t = 0; t < 8; ++t)
                  y[t] = acc[t % 4 / 2][f][t % 2 * 8 + 4 * s + 2 * h + t / 4];
                mx_store8(at + 32 * s + 8 * h, y);
              }
          }
        }
      };
      if (a.dtype == QP_F32)
        store(static_cast<float*>(a.dX));
      else if (a.dtype == QP_BF16)
        store(static_cast<bf16_t*>(a.dX));
      else
        store(static_cast<f16_t*>(a.dX));
      return;
    }
    // else 32 rows at a time through the wave's own LDS
    float* const out = reinterpret_cast<float*>(mx_lds) + wave * 32 * L::kOutLd;
    const int p8 = lane & 7, row_in = lane >> 3;
    const int64_t col = k0 + wn * 64 + p8 * 8;
#pragma unroll 1
    for (int f = 0; f < F; ++f) {
#pragma unroll
      for (int j = 0; j < F; ++j)
        if (j == f) {
#pragma unroll
          for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int at = i * 32 + 8 * (r / 4) + r % 4;  // + 4 half: the weights' row
              out[l32 * L::kOutLd + 4 * (at % 16 + 4 * half) + at / 16] = acc[i][j][r];
            }
        }
      wave_sync();
#pragma unroll 1
      for (int h = 0; h < 32; h += 8) {
        const int64_t r = tile.r0 + (wm * F + f) * 32 + h + row_in;
        if (r < tile.r1 && col < K) {
          const float* src = out + (h + row_in) * L::kOutLd + p8 * 8;
          const f32x4 lo = *reinterpret_cast<const f32x4*>(src);
          const f32x4 hi = *reinterpret_cast<const f32x4*>(src + 4);
          const float y[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          w4_store8(a.dX, a.dtype, r * a.lddx + col, y, K - col < 8 ? (int)(K - col) : 8);
        }
      }
      wave_sync();
    }
  };
  constexpr int kHalf = kDirect && FM > 1 ? FM / 2 : FM;
  if (kHalf < FM && tile.r1 - tile.r0 <= BM / 2)
    run(std::integral_constant<int, kHalf>{});
  else
    run(std::integral_constant<int, FM>{});
}

template <typename T, bool kDirect, int BM, int BC, int WM, int WN>
qp_status launch_dx_tile(const char* what, const MxDxArgs& a, hipStream_t stream) {
  using L = MxDxTile<T, BM, BC, WM, WN>;
  const int64_t slots = w4_tile_slots(a.rows, BM), groups = ceil_div(a.w.K, BC);
  const int64_t grid = mx_tile_grid(slots, groups, BM >= 256);
  QP_REQUIRE(grid * L::NW * 64 < (INT64_C(1) << 32), QP_EUNSUPPORTED,
             "%s: rows and columns for more than 2^32 threads", what);
  auto kern = mx_dx_tile_kernel<T, kDirect, BM, BC, WM, WN>;
  static std::atomic<uint64_t> reserved{0};
  if (qp_status st = mx_reserve_lds(what, reinterpret_cast<const void*>(kern), L::kLds, reserved))
    return st;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(L::NW * 64), L::kLds, stream, a,
                     (uint32_t)slots, (uint32_t)groups);
  return check_launch(what);
}

// Which kernel, and for few rows in how many splits the channels go: enough workgroups
// for the card, no split without a step of 32 channels for each of its waves.
//
// Measured, bf16, 4096 x 4096 weights, cold: 16 rows 11.6 us by the few-row kernel (128 x
// 128 tiles 46), 256 37 (47), 512 71 (49; 256 x 256 tiles 96), 1024 132 (52), 2048 248 (81, 97),
// 4096 456 (156, 119); of 11008 columns 1024 rows 332 (118, 100).  f32 rows: 256 53,
// 512 94, 768 147; tiles 1024 137, 4096 556 to 580.  By expert, 2048 tokens x 2 of 8 of 4096 x
// 4096: bf16 194 (rows at odd addresses, through registers, 292), f32 730.
constexpr int kDxWaves = 8;
struct DxPlan {
  int tile;         // rows of a tile, 0: few rows
  uint32_t splits;
};
constexpr int64_t kDxSplitGroups = 512;  // workgroups that splits may make
int64_t dx_most_splits(const qp_mx4* w) {
  const int64_t most = ceil_div(ceil_div(w->rows, 32), kDxWaves);
  return most > 16 ? 16 : most < 1 ? 1 : most;
}
DxPlan dx_plan(int32_t dtype, int64_t M, const qp_mx4* w) {
  const int64_t parts = w->matrices < M ? w->matrices : M;
  // row tiles of an expert: its last one is half empty on average
  auto groups = [&](int rows, int cols) {
    const double each = (double)M / (double)parts / rows;
    const double tiles = parts > 1 ? (each > 0.5 ? each + 0.5 : 1.0) * (double)parts
                                   : (double)ceil_div(M, rows);
    return tiles * (double)ceil_div(w->K, cols) / 256.0;
  };
  const double few = groups(16, 128), t128 = groups(128, 128);
  // (one to a CU: whole rounds; experts of unlike sizes have more tiles than that)
  double t256 = groups(256, 256) * (parts > 1 ? 1.1 : 1.0);
  t256 = mx_halved_rounds(t256);
  // microseconds at 4096 channels (all grow with them): up to one workgroup a CU, and
  // for the further ones
  auto cost = [](double g, double one, double filled, double more) {
    return one + filled * (g < 1.0 ? g : 1.0) + more * (g > 1.0 ? g - 1.0 : 0.0);
  };
  const bool f32 = dtype == QP_F32;
  const double c0 = f32 ? 9.0 + 21.5 * few : 9.0 + 15.0 * few;
  const double c128 = f32 ? cost(t128, 127.0, 10.0, 138.0) : cost(t128, 46.0, 6.0, 36.0);
  const double c256 = f32 ? 1e300 : cost(t256, 94.0, 25.0, 115.0);
  DxPlan p{0, 1};
  if (c128 < c0 || c256 < c0) {
    p.tile = c256 < c128 ? 256 : 128;
    return p;
  }
  const int64_t wgs = (M / 16 + parts) * ceil_div(w->K, 128);
  const int64_t s = kDxSplitGroups / wgs, most = dx_most_splits(w);
  p.splits = s > most ? (uint32_t)most : s < 1 ? 1u : (uint32_t)s;
  return p;
}

// What the splits of any call of up to M rows of any type can need: for every number of
// splits the most rows that dx_plan gives it (its row tiles are M / 16 + the experts).
size_t dx_ws(int64_t M, const qp_mx4* w) {
  const int64_t E = w->matrices, cols = ceil_div(w->K, 128), splits = dx_most_splits(w);
  int64_t most = 0;
  for (int64_t s = 2; s <= splits; ++s) {
    const int64_t tiles = kDxSplitGroups / s / cols;
    int64_t m = tiles >= E + E / 16 ? 16 * (tiles - E) + 15
                                    : 16 * (tiles / 17) + (tiles % 17 < 15 ? tiles % 17 : 15);
    m = m < M ? m : M;
    most = most > s * m ? most : s * m;
  }
  return (size_t)(4 * most * w->K);
}

template <typename T>
void launch_dx(const MxDxArgs& a, uint32_t slots, uint32_t splits, hipStream_t stream) {
  const int64_t cols = ceil_div(a.w.K, 128);
  hipLaunchKernelGGL((mx_dx_rows_kernel<T, kDxWaves>), dim3((unsigned)(slots * cols * splits)),
                     dim3(kDxWaves * 64), 0, stream, a, slots, splits);
}

template <typename T>
qp_status run_dx_tile(const char* what, const MxDxArgs& a, int tile, hipStream_t stream) {
  if constexpr (sizeof(T) == 4) {
    return launch_dx_tile<T, false, 128, 128, 2, 2>(what, a, stream);
  } else {
    // rows that direct loads cannot take go through registers
    if ((uintptr_t)a.dY % 4 || a.lddy % 2 || !mx_tile_reaches(a.rows, a.lddy * 2))
      return launch_dx_tile<T, false, 128, 128, 2, 2>(what, a, stream);
    if (tile == 256) return launch_dx_tile<T, true, 256, 256, 2, 4>(what, a, stream);
    return launch_dx_tile<T, true, 128, 128, 2, 2>(what, a, stream);
  }
}

qp_status run_dx(const char* what, const void* dY, int32_t dtype, int64_t M, int64_t lddy,
                 const qp_mx4* w, const int32_t* offsets, void* dX, int64_t lddx, void* ws,
                 size_t ws_bytes, hipStream_t stream) {
  QP_REQUIRE(M >= 0, QP_EINVAL, "%s: M is negative", what);
  QP_REQUIRE(M <= kW4MaxRows, QP_EUNSUPPORTED, "%s: more than 2^30 rows", what);
  qp_status st = mx_check(what, "w", w);
  if (st) return st;
  QP_REQUIRE(w->rows > 0, QP_EINVAL, "%s: w has no rows", what);
  QP_REQUIRE(offsets || w->matrices == 1, QP_EINVAL, "%s: one matrix of weights, or offsets", what);
  if (M == 0) return QP_OK;
  if ((st = w4_check_float(what, "dY", dY, dtype, lddy, w->rows))) return st;
  if ((st = w4_check_float(what, "dX", dX, dtype, lddx, w->K))) return st;
  const DxPlan plan = dx_plan(dtype, M, w);
  const uint32_t splits = plan.splits;
  const size_t need = splits > 1 ? dx_ws(M, w) : 0;
  QP_REQUIRE(ws_bytes >= need, QP_ESIZE, "%s: needs a workspace of %zu bytes, has %zu", what, need,
             ws_bytes);
  QP_REQUIRE(!need || (ws && (uintptr_t)ws % 256 == 0), QP_EALIGN,
             "%s: the workspace must be 256-byte aligned", what);
  MxDxArgs a{mx_view(w), W4Rows{offsets, (int32_t)w->matrices, M, nullptr, 1, M}, dY, lddy, dX,
             dtype, lddx, static_cast<float*>(ws)};
  if (plan.tile) {
    if (dtype == QP_F32) return run_dx_tile<float>(what, a, plan.tile, stream);
    if (dtype == QP_BF16) return run_dx_tile<bf16_t>(what, a, plan.tile, stream);
    return run_dx_tile<f16_t>(what, a, plan.tile, stream);
  }
  const int64_t slots = w4_tile_slots(a.rows, 16), cols = ceil_div(w->K, 128);
  QP_REQUIRE(slots * cols * splits * kDxWaves * 64 < (INT64_C(1) << 32), QP_EUNSUPPORTED,
             "%s: rows and columns for more than 2^32 threads", what);
  if (dtype == QP_F32)
    launch_dx<float>(a, (uint32_t)slots, splits, stream);
  else if (dtype == QP_BF16)
    launch_dx<bf16_t>(a, (uint32_t)slots, splits, stream);
  else
    launch_dx<f16_t>(a, (uint32_t)slots, splits, stream);
  if ((st = check_launch(what))) return st;
  if (splits > 1) {
    const int64_t pieces = ceil_div(w->K, 8);
    hipLaunchKernelGGL(mx_dx_sum_kernel, dim3((unsigned)ceil_div(M * pieces, 256)), dim3(256), 0,
                       stream, a.part, M, w->K, splits, (uint32_t)pieces, dX, dtype, lddx);
    return check_launch(what);
  }
  return QP_OK;
}

}  // namespace

void mx_dx_kernel_name(const qp_mx4* w, int32_t dtype, int64_t M, char* name, size_t bytes) {
  const DxPlan p = dx_plan(dtype, M, w);
  if (p.tile)
    std::snprintf(name, bytes, "tile%dx%d", p.tile, p.tile);
  else
    std::snprintf(name, bytes, "rows16x128/%u", p.splits);
}

}  // namespace qp

extern "C" qp_status qgemm_w4_mx_dx_ws_size(int64_t M, const qp_mx4* w, size_t* bytes) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_w4_mx_dx_ws_size";
  QP_REQUIRE(bytes, QP_EINVAL, "%s: bytes is null", what);
  QP_REQUIRE(M >= 0, QP_EINVAL, "%s: M is negative", what);
  QP_REQUIRE(M <= kW4MaxRows, QP_EUNSUPPORTED, "%s: more than 2^30 rows", what);
  qp_status st = mx_check(what, "w", w);
  if (st) return st;
  *bytes = dx_ws(M, w);
  return QP_OK;
}

extern "C" qp_status qgemm_w4_mx_dx(const void* dY, int32_t dtype, int64_t M, int64_t lddy,
                                    const qp_mx4* w, void* dX, int64_t lddx, void* ws,
                                    size_t ws_bytes, hipStream_t stream) {
  qp::clear_error();
  return qp::run_dx("qgemm_w4_mx_dx", dY, dtype, M, lddy, w, nullptr, dX, lddx, ws, ws_bytes,
                    stream);
}

extern "C" qp_status qgemm_w4_mx_experts_dx(const void* dY, int32_t dtype, int64_t M, int64_t lddy,
                                            const qp_mx4* w, const int32_t* offsets, void* dX,
                                            int64_t lddx, void* ws, size_t ws_bytes,
                                            hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_w4_mx_experts_dx";
  QP_REQUIRE(offsets, QP_EINVAL, "%s: offsets is null", what);
  return run_dx(what, dY, dtype, M, lddy, w, offsets, dX, lddx, ws, ws_bytes, stream);
}
