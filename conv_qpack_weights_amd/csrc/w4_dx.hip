// w4_dx.hip -- the gradient of the weight-only int4 product to its rows, dense
// or grouped by expert:
//   dx[r,k] = sum_n dy[r,n] * (s[n,g(k)] * q[n,k] (+ o[n,g(k)]))
// The blob runs along K, and the sum here runs along the channels n, whose
// scales differ.  A lane therefore takes one word (eight K) of eight channels
// and transposes them in registers: nibble j of its eight words, each times
// its channel's scale, is the MFMA operand (eight reduction indexes) of
// column k = 8*(l%16) + j.  Eight MFMAs (j = 0..7) cover a 128-K block, and a
// lane ends with eight consecutive K of a row.
//
// Roundings: s*q (+ o) is formed in f32 and enters as two bf16 pieces (three
// for f32 rows), which miss at most 2^-16 (2^-24) of it; dy enters exactly
// (f16 as two pieces, f32 as three).  Of the pieces' products those are formed
// whose order adds up to less than the number of weight pieces: what is left
// out is below 2^-16 of a term (2^-23 for f32 rows).  Sums are f32.  Two pieces are
// fewer bits than an f32 weight has; a third would be half as many MFMAs again.  Over
// sums of 4096 terms they miss 2.5e-6 (bf16 rows) and 3.8e-6 (f16) of the result in
// the norm, and the rounding of the outputs 1.7e-3 and 2.1e-4.
//
// Groups of 128 on without offsets: a block has one scale a channel, so the rows
// can carry it: dy*s, rounded to f32, goes in as two bf16 pieces (three for f32
// rows), missing at most 2^-16 (2^-23), and q/16 exactly as one.  The weights then
// cost an unpacking only, and f16 rows take two MFMAs instead of three, f32 rows
// three instead of six.
#include <atomic>
#include <cstdio>
#include <type_traits>

#include "w4.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

struct W4DxArgs {
  W4View w;
  W4Rows rows;
  const void* dY;
  int64_t lddy;
  void* dX;
  int32_t dtype;
  int64_t lddx;
};

// Two values rounded to bf16 (nearest, ties to even), the first in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float low_f32(uint32_t p) { return __builtin_bit_cast(float, p << 16); }
__device__ __forceinline__ float high_f32(uint32_t p) {
  return __builtin_bit_cast(float, p & 0xffff0000u);
}

// Eight values as kPieces bf16 each, largest first: every piece is what the
// ones before it leave, rounded to nearest, so n pieces miss at most 2^-8n of
// the value.  What may be among them: kFinite only values that round to finite
// ones (of others the later pieces are NaN); kSpecial infinities and NaNs too,
// whose later pieces are zero; kAnySize also finite values above the largest bf16,
// whose first piece is that largest one and not the infinity they round to.
enum SplitRange { kFinite, kSpecial, kAnySize };
template <int kPieces, SplitRange kRange>
__device__ __forceinline__ void split_bf16(const float (&f)[8], bf16x8 (&o)[kPieces]) {
  u32x4 p[kPieces];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = f[2 * i], b = f[2 * i + 1];
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
      bool fa = true, fb = true;
      float ca = a, cb = b;
      if (kRange != kFinite && n == 0) {
        fa = __builtin_fabsf(a) < __builtin_inff();  // (not a NaN either)
        fb = __builtin_fabsf(b) < __builtin_inff();
      }
      if (kRange == kAnySize && n == 0) {
        constexpr float kLargest = 0x1.fep127f;
        ca = fa ? __builtin_amdgcn_fmed3f(a, -kLargest, kLargest) : a;
        cb = fb ? __builtin_amdgcn_fmed3f(b, -kLargest, kLargest) : b;
      }
      uint32_t h = bf16_pair(ca, cb);
      // (opaque: the compiler would round `a` once more to find the low half)
      asm("" : "+v"(h));
      p[n][i] = h;
      if (n + 1 < kPieces) {
        a = a - low_f32(h);
        b = b - high_f32(h);
        if (kRange != kFinite && n == 0) {
          a = fa ? a : 0.0f;
          b = fb ? b : 0.0f;
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < kPieces; ++n) o[n] = __builtin_bit_cast(bf16x8, p[n]);
}

// dy in bf16 pieces, largest first
template <typename T>
struct YFrag;
template <>
struct YFrag<bf16_t> {
  static constexpr int kPieces = 1, kWPieces = 2, kScaledPieces = 2;
  XFrag<bf16_t> x;
  __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = x.v[i];
      f[2 * i] = low_f32(u);
      f[2 * i + 1] = high_f32(u);
    }
  }
  __device__ __forceinline__ void split(bf16x8 (&o)[1]) const {
    o[0] = __builtin_bit_cast(bf16x8, x.v);
  }
};
template <>
struct YFrag<f16_t> {
  static constexpr int kPieces = 2, kWPieces = 2, kScaledPieces = 2;  // 11 bits: two pieces hold them
  XFrag<f16_t> x;
  __device__ __forceinline__ void values(float (&f)[8]) const {
    const f16x8 h = __builtin_bit_cast(f16x8, x.v);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)h[i];
  }
  __device__ __forceinline__ void split(bf16x8 (&o)[2]) const {
    float f[8];
    values(f);
    split_bf16<2, kSpecial>(f, o);
  }
};
template <>
struct YFrag<float> {
  static constexpr int kPieces = 3, kWPieces = 3, kScaledPieces = 3;
  XFrag<float> x;
  __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = x.v[i / 4][i & 3];
      f[i] = __builtin_bit_cast(float, u);
    }
  }
  __device__ __forceinline__ void split(bf16x8 (&o)[3]) const {
    float f[8];
    values(f);
    split_bf16<3, kAnySize>(f, o);
  }
};

// The words and scales of a lane's eight channels in a 32-channel step; the
// scales stay as they come from memory (a conversion would wait for the load).
template <int kKind>
struct DxWeights {
  uint32_t d[8];
  uint32_t s[8];
  float o[kKind == 2 ? 8 : 1];
  __device__ __forceinline__ float scale(int r) const {
    return __builtin_bit_cast(float, kKind == 1 ? s[r] << 16 : s[r]);
  }
  // times the 16 that q/16 lacks
  __device__ __forceinline__ float s16(int r) const { return scale(r) * 16.0f; }
};

// Where a lane finds them: lane (c, h) takes word c of the block -- 32-K number
// t = c/4, chunk c%4, so K 8c .. 8c+7 -- of channels 8h .. 8h+7 of the step.
template <int kKind>
struct DxSource {
  const uint8_t* q;      // block's words of channel tile 0
  const uint8_t* s;
  const uint8_t* o;
  int64_t q_step, s_step;  // to the next channel tile, in bytes
  uint32_t q_lane, s_lane;

  __device__ __forceinline__ DxSource(const W4View& w, const uint8_t* blob, int64_t blk, int lane) {
    constexpr uint32_t ES = kKind == 1 ? 2 : 4;
    const int c = lane & 15, h = lane >> 4;
    q_step = w.nblk * 1024;
    s_step = w.G4 * 64 * ES;
    q = blob + w.data_off + blk * 1024;
    s = blob + w.scale_off;
    o = blob + w.offs_off;
    const uint32_t g = (uint32_t)(blk * 128 + 32 * (c >> 2)) / (uint32_t)w.group;
    q_lane = (uint32_t)((h >> 1) * q_step) + (h & 1) * 512 + (c & 3) * 16 + (c >> 2) * 4;
    s_lane = (uint32_t)((h >> 1) * s_step) + ((h & 1) * 32 + (g / 4) * 64 + (g & 3)) * ES;
  }
  __device__ __forceinline__ void load(DxWeights<kKind>& w, int64_t step) const {
    const uint8_t* qp = q + 2 * step * q_step + q_lane;
    const uint8_t* sp = s + 2 * step * s_step + s_lane;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      w.d[r] = *reinterpret_cast<const uint32_t*>(qp + r * 64);
      if constexpr (kKind == 1) {
        w.s[r] = *reinterpret_cast<const uint16_t*>(sp + r * 8);
      } else {
        w.s[r] = *reinterpret_cast<const uint32_t*>(sp + r * 16);
      }
      if constexpr (kKind == 2)
        w.o[r] = *reinterpret_cast<const float*>(o + 2 * step * s_step + s_lane + r * 16);
    }
  }
};

// Column j of a lane's eight (0..3: the low nibbles of w.d, 4..7: those of hi,
// the same words shifted down): its eight channels' weights as bf16 pieces.
template <int kKind, int NW>
__device__ __forceinline__ void dx_column(const DxWeights<kKind>& w, const uint32_t (&hi)[8],
                                          const float (&s16)[8], int j, bf16x8 (&o)[NW]) {
  float f[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const uint32_t x = j < 4 ? w.d[r] : hi[r];
    f[r] = nib_f32((x >> (8 * (j & 3))) & 0xffu) * s16[r];
    if constexpr (kKind == 2) f[r] = f[r] + w.o[r];
  }
  split_bf16<NW, kFinite>(f, o);
}

template <int kKind>
__device__ __forceinline__ void dx_prepare(const DxWeights<kKind>& w, uint32_t (&hi)[8],
                                           float (&s16)[8]) {
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    hi[r] = w.d[r] >> 4;
    asm("" : "+v"(hi[r]));  // (one shift; the conversions then select bytes)
    s16[r] = w.s16(r);
  }
}

// Column j as it is, q/16 in bf16: for rows that carry the scales.
template <int kKind>
__device__ __forceinline__ bf16x8 dx_plain_column(const DxWeights<kKind>& w,
                                                  const uint32_t (&hi)[8], int j) {
  uint32_t f[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const uint32_t x = j < 4 ? w.d[r] : hi[r];
    f[r] = __builtin_bit_cast(uint32_t, nib_f32((x >> (8 * (j & 3))) & 0xffu));
  }
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = hi_halves(f[2 * i], f[2 * i + 1]);
  return __builtin_bit_cast(bf16x8, o);
}

// The products of the pieces that count, small ones first.
template <int NY, int NW>
__device__ __forceinline__ f32x4 dx_mfma(const bf16x8 (&y)[NY], const bf16x8 (&w)[NW], f32x4 acc) {
#pragma unroll
  for (int sum = NW - 1; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i < NY; ++i)
      if (sum - i >= 0 && sum - i < NW) acc = mfma32(y[i], w[sum - i], acc);
  return acc;
}

// ---- few rows: the waves (and up to gridDim.z workgroups) share out the channels
// A workgroup owns one 128-K block and 16*kMT rows; each wave takes every
// kWaves-th step of its workgroup's run of 32-channel steps, rows and weights
// straight from memory, the next step's on their way; the sums meet in LDS in a
// fixed order.  With several workgroups per tile (few blocks and rows, many
// channels) each leaves f32 partial sums in the workspace, which
// w4_dx_join_kernel adds up in order.  Bound by the vector instructions that make
// the weights' pieces (some 330 a step and wave, for 16 MFMAs a row fragment):
// 16 x 4096 x 4096 13 us (29 without splits), 16 x 11008 x 4096 18 us,
// 37 x 1037 x 1100 f16 10 us, 512 x 4096 x 4096 51 us (338 TFLOP/s).  kOne: the
// rows carry the scales (groups of 128 on); 1024 x 4096 x 4096 bf16 86 us (94
// without), f16 88 (121), f32 122 (201); 1 x 4096 x 4096 9.3, 8.9, 9.3 us (10.7,
// 10.6, 12.2).
template <typename T, int kKind, bool kOne, int kMT, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void w4_dx_rows_kernel(W4DxArgs a, uint32_t splits,
                                                                 float* part) {
  constexpr int NY = YFrag<T>::kPieces, NW = YFrag<T>::kWPieces;
  constexpr int kRound = 8 / kMT < kWaves ? 8 / kMT : kWaves;  // waves in LDS at a time: 64 KiB
  __shared__ f32x4 red[kRound][kMT * 8][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t nblk = (uint32_t)((a.w.K + 127) / 128);
  const uint32_t blk = blockIdx.x % nblk, rest = blockIdx.x / nblk;
  const uint32_t split = rest % splits, slot = rest / splits;
  const W4Tile tile = w4_find_tile<16 * kMT>(a.rows, slot);
  if (tile.expert < 0) return;
  const int c = lane & 15, h = lane >> 4;

  f32x4 acc[kMT][8];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[m][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  if (!(a.rows.offsets && tile.expert == a.rows.experts)) {
    const DxSource<kKind> src(a.w, a.w.blob + tile.expert * a.w.expert_stride, blk, lane);
    const T* yr[kMT];
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      int64_t r = tile.r0 + m * 16 + c;
      r = r < tile.r1 ? r : tile.r1 - 1;  // repeated rows are not stored
      yr[m] = static_cast<const T*>(a.dY) + r * a.lddy + 8 * h;
    }
    auto step = [&](const DxWeights<kKind>& w, const YFrag<T> (&yf)[kMT]) {
      uint32_t hi[8];
      float s16[8];
      dx_prepare<kKind>(w, hi, s16);
      if constexpr (kOne) {  // the lane's eight channels are those of its rows' elements
        constexpr int NS = YFrag<T>::kScaledPieces;
        bf16x8 y[kMT][NS];
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
          float f[8];
          yf[m].values(f);
#pragma unroll
          for (int r = 0; r < 8; ++r) f[r] = f[r] * w.scale(r);
          split_bf16<NS, kAnySize>(f, y[m]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bf16x8 wv = dx_plain_column<kKind>(w, hi, j);
#pragma unroll
          for (int n = NS - 1; n >= 0; --n)
#pragma unroll
            for (int m = 0; m < kMT; ++m) acc[m][j] = mfma32(y[m][n], wv, acc[m][j]);
        }
        return;
      }
      bf16x8 y[kMT][NY];
#pragma unroll
      for (int m = 0; m < kMT; ++m) yf[m].split(y[m]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        bf16x8 wv[NW];
        dx_column<kKind, NW>(w, hi, s16, j, wv);
#pragma unroll
        for (int m = 0; m < kMT; ++m) acc[m][j] = dx_mfma<NY, NW>(y[m], wv, acc[m][j]);
      }
    };
    const int64_t full = a.w.N / 32, per = (full + splits - 1) / splits;
    const int64_t s0 = split * per < full ? split * per : full;
    const int64_t s1 = s0 + per < full ? s0 + per : full;
    if (s0 + wave < s1) {
      DxWeights<kKind> w[2];
      YFrag<T> y[2][kMT];
      auto load = [&](int p, int64_t i) {
        i = i < s1 ? i : s1 - 1;
        src.load(w[p], i);
#pragma unroll
        for (int m = 0; m < kMT; ++m) y[p][m].x.load(yr[m] + i * 32);
      };
      load(0, s0 + wave);
      for (int64_t i = s0 + wave; i < s1; i += 2 * kWaves) {
        load(1, i + kWaves);
        step(w[0], y[0]);
        load(0, i + 2 * kWaves);
        if (i + kWaves < s1) step(w[1], y[1]);
      }
    }
    // the channels past the last whole step, with the last split's wave 0
    if (full * 32 < a.w.N && wave == 0 && split + 1 == splits) {
      DxWeights<kKind> w;
      YFrag<T> y[kMT];
      src.load(w, full);
      const int64_t left = a.w.N - (full * 32 + 8 * h);
      const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
#pragma unroll
      for (int m = 0; m < kMT; ++m) y[m].x.load_n(yr[m] + (n > 0 ? full * 32 : -8 * h), n);
      step(w, y);
    }
  }

  // Sums over the waves: every thread takes four columns of one row of each 16
  // (2048 sums a fragment over kWaves*64 threads).
  constexpr int kEach = 2048 / (kWaves * 64 * 4);
  static_assert(kEach >= 1, "at most eight waves");
  f32x4 sum[kMT][kEach];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int e = 0; e < kEach; ++e) sum[m][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int r0 = 0; r0 < kWaves; r0 += kRound) {
    if (r0 > 0) __syncthreads();
    if (wave >= r0 && wave < r0 + kRound) {
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) red[wave - r0][m * 8 + j][lane] = acc[m][j];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int id = threadIdx.x + e * kWaves * 64;        // (row, 4-column piece)
        const int row = id >> 5, piece = id & 31;            // 32 pieces of 4 columns
        const int from = (row >> 2) * 16 + (piece >> 1), j0 = (piece & 1) * 4;
#pragma unroll
        for (int w = 0; w < kRound; ++w)
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[m][e][j] += red[w][m * 8 + j0 + j][from][row & 3];
      }
  }
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if constexpr (kOne) sum[m][e] *= 16.0f;
      const int id = threadIdx.x + e * kWaves * 64;
      const int64_t r = tile.r0 + m * 16 + (id >> 5);
      const int64_t k = (int64_t)blk * 128 + (id & 31) * 4;
      if (r >= tile.r1 || k >= a.w.K) continue;
      const int n = a.w.K - k < 4 ? (int)(a.w.K - k) : 4;
      if (splits > 1) {
        // (rows of the partial sums are whole blocks long)
        *reinterpret_cast<f32x4*>(part + ((int64_t)split * a.rows.M + r) * (nblk * 128) + k) =
            sum[m][e];
      } else {
        T* dst = static_cast<T*>(a.dX) + r * a.lddx + k;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < n) dst[j] = from_f32<T>(sum[m][e][j]);
      }
    }
}

// Rows past offsets[experts] are among the tiles, so every row of every split
// has been written.
template <typename T>
__global__ __launch_bounds__(256) void w4_dx_join_kernel(const float* part, uint32_t splits,
                                                         int64_t M, int64_t K, int64_t ldp,
                                                         T* dX, int64_t lddx, uint32_t row_pieces) {
  const uint32_t id = blockIdx.x * 256 + threadIdx.x;
  const uint32_t r = id / row_pieces;
  if (r >= M) return;
  const int64_t k = (int64_t)(id - r * row_pieces) * 4;
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t s = 0; s < splits; ++s)
    sum += *reinterpret_cast<const f32x4*>(part + (s * M + r) * ldp + k);
  T* dst = dX + r * lddx + k;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (k + j < K) dst[j] = from_f32<T>(sum[j]);
}

// ---- many rows (bf16) --------------------------------------------------
// A workgroup of four waves owns 32*kMT rows and two 128-K blocks: wave (rg, kg)
// the rows 16*kMT*rg .. and block kg.  What a 32-channel step costs beside its
// MFMAs is making the weights' pieces, about 40 vector instructions a column of
// eight; the two waves of a block share that out, one the columns of the low
// nibbles, the other those of the high ones, and pass each other their four
// columns through LDS.  A step's rows of dY pass through LDS too (with the
// pieces of quad h of row r at place r ^ 2h of 16: no bank conflicts either way).
// Both are double buffered, one barrier a step: while a wave multiplies its
// partner's columns it makes its own of the next step.  4096 x 4096 x 4096 255 us
// (539 TFLOP/s; the rows kernel 359): matrix unit busy 47% of the cycles, vector
// instructions 47%, one after the other.  Weights made by every wave for itself:
// 279 us; four waves sharing one block with 32 rows each: 331 us; loads two steps
// ahead: 266 us.
template <typename T, int kKind, int kMT>
struct DxLds {
  static constexpr int NY = YFrag<T>::kPieces, NW = YFrag<T>::kWPieces;
  u32x4 y[2][NY][2 * kMT][64];
  u32x4 w[2][2][8][NW][64];  // [buffer][block][column][piece]
};

template <typename T, int kKind, int kMT>
__global__ __launch_bounds__(256, 2) void w4_dx_tile_kernel(W4DxArgs a,
                                                            uint32_t blk_pairs) {
  constexpr int NY = YFrag<T>::kPieces, NW = YFrag<T>::kWPieces;
  constexpr int kFrags = 2 * kMT;  // 16-row fragments of the workgroup
  extern __shared__ __attribute__((aligned(16))) uint8_t dx_lds[];
  DxLds<T, kKind, kMT>& lds = *reinterpret_cast<DxLds<T, kKind, kMT>*>(dx_lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rg = wave & 1, kg = wave >> 1;
  const int c = lane & 15, h = lane >> 4;
  // (each XCD a run of tiles, the blocks of a row tile next to each other)
  uint32_t id = blockIdx.x;
  {
    const uint32_t n = gridDim.x, per = n / 8, rest = n % 8, x = id % 8;
    id = x * per + (x < rest ? x : rest) + id / 8;
  }
  const uint32_t slot = id / blk_pairs;
  const uint32_t nblk = (uint32_t)((a.w.K + 127) / 128);
  const uint32_t blk = (id - slot * blk_pairs) * 2 + kg;
  const W4Tile tile = w4_find_tile<16 * kFrags>(a.rows, slot);
  if (tile.expert < 0) return;
  const int64_t k0 = (int64_t)blk * 128 + 8 * c;
  const int k_left = k0 >= a.w.K ? 0 : a.w.K - k0 < 8 ? (int)(a.w.K - k0) : 8;

  // acc[.][j] holds the wave's own columns in j < 4, its partner's in j >= 4
  f32x4 acc[kMT][8];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[m][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  if (!(a.rows.offsets && tile.expert == a.rows.experts)) {
    const DxSource<kKind> src(a.w, a.w.blob + tile.expert * a.w.expert_stride,
                              blk < nblk ? blk : nblk - 1, lane);
    // staging: four lanes a row's 32 channels, a wave 16 rows at a time
    constexpr int kMine = kFrags / 4;
    static_assert(kMine >= 1, "a fragment a wave and pass");
    const uint8_t* ybase = static_cast<const uint8_t*>(a.dY) + tile.r0 * a.lddy * sizeof(T);
    const int quad = lane & 3, row = lane >> 2;
    const int place = quad * 16 + (row ^ (2 * quad));
    uint32_t yoff[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      int64_t r = (i * 4 + wave) * 16 + row;
      r = tile.r0 + r < tile.r1 ? r : tile.r1 - 1 - tile.r0;
      yoff[i] = (uint32_t)((r * a.lddy + quad * 8) * sizeof(T));
    }
    DxWeights<kKind> w;
    YFrag<T> y[kMine];
    auto fetch = [&](int64_t s) {
      src.load(w, s);
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        y[i].x.load(reinterpret_cast<const T*>(ybase + s * (32 * sizeof(T)) + yoff[i]));
    };
    auto fetch_cut = [&](int64_t s) {
      src.load(w, s);
      const int64_t left = a.w.N - (s * 32 + quad * 8);
      const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        // (a lane with nothing left points at its row's first element)
        y[i].x.load_n(
            reinterpret_cast<const T*>(ybase + yoff[i] + (n > 0 ? s * (int64_t)(32 * sizeof(T))
                                                                : -quad * (int64_t)(8 * sizeof(T)))),
            n);
    };
    float s16[8];
    uint32_t d[8];
    bf16x8 own[4][NW];
    // what was fetched: the rows to LDS, the wave's nibbles to the low places
    auto take = [&](int buf) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        bf16x8 v[NY];
        y[i].split(v);
#pragma unroll
        for (int n = 0; n < NY; ++n)
          lds.y[buf][n][i * 4 + wave][place] = __builtin_bit_cast(u32x4, v[n]);
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        s16[r] = w.s16(r);
        d[r] = w.d[r] >> (rg * 4);
        asm("" : "+v"(d[r]));
      }
    };
    auto make = [&](int buf, int j) {
      dx_column<kKind, NW>(w, d, s16, 4 + j, own[j]);
#pragma unroll
      for (int n = 0; n < NW; ++n)
        lds.w[buf][kg][rg * 4 + j][n][lane] = __builtin_bit_cast(u32x4, own[j][n]);
    };
    auto multiply = [&](const bf16x8 (&yv)[kMT][NY], const bf16x8 (&wv)[NW], int j) {
#pragma unroll
      for (int o = NW - 1; o >= 0; --o)
#pragma unroll
        for (int i = 0; i < NY; ++i)
          if (o - i >= 0 && o - i < NW) {
#pragma unroll
            for (int m = 0; m < kMT; ++m) acc[m][j] = mfma32(yv[m][i], wv[o - i], acc[m][j]);
          }
    };
    // the step in `buf`; kMore: the fetched step goes into the other buffer and
    // step `next` is fetched
    auto step = [&](auto more, int buf, int64_t next) {
      constexpr bool kMore = decltype(more)::value;
      bf16x8 yv[kMT][NY], other[4][NW];
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int n = 0; n < NY; ++n)
          yv[m][n] =
              __builtin_bit_cast(bf16x8, lds.y[buf][n][rg * kMT + m][h * 16 + (c ^ (2 * h))]);
      auto read = [&](int j) {
#pragma unroll
        for (int n = 0; n < NW; ++n)
          other[j][n] = __builtin_bit_cast(bf16x8, lds.w[buf][kg][(rg ^ 1) * 4 + j][n][lane]);
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        if (j == 2) read(0);
        multiply(yv, own[j], j);
      }
      if constexpr (kMore) take(buf ^ 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        if (j < 3) read(j + 1);
        if constexpr (kMore) make(buf ^ 1, j);
        multiply(yv, other[j], 4 + j);
      }
      if constexpr (kMore) fetch(next);
    };
    using std::false_type;
    using std::true_type;
    const int64_t full = a.w.N / 32;
    if (full > 0) {
      fetch(0);
      take(0);
#pragma unroll
      for (int j = 0; j < 4; ++j) make(0, j);
      if (full > 1) {
        fetch(1);
        for (int64_t s = 0; s + 1 < full; ++s) {
          __syncthreads();  // step s is in LDS, everyone is done with s - 1
          step(true_type{}, (int)(s & 1), s + 2 < full ? s + 2 : s + 1);
        }
      }
      __syncthreads();
      step(false_type{}, (int)((full - 1) & 1), 0);
      __syncthreads();
    }
    if (full * 32 < a.w.N) {
      fetch_cut(full);
      take(0);
#pragma unroll
      for (int j = 0; j < 4; ++j) make(0, j);
      __syncthreads();
      step(false_type{}, 0, 0);
    }
  }

#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = tile.r0 + (rg * kMT + m) * 16 + 4 * h + i;
      if (r >= tile.r1) continue;
      T* dst = static_cast<T*>(a.dX) + r * a.lddx + k0;
      // columns 0..3 are those of the low nibbles: wave rg = 0's own
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j] = rg ? acc[m][4 + j][i] : acc[m][j][i];
        f[4 + j] = rg ? acc[m][j][i] : acc[m][4 + j][i];
      }
      if (k_left > 0) store_piece(dst, f, k_left);
    }
}

template <typename T, int kKind, int kMT>
qp_status launch_dx_tile(const W4DxArgs& a, hipStream_t stream) {
  const int64_t slots = w4_tile_slots(a.rows, 32 * kMT);
  const int64_t pairs = ceil_div(a.w.K, 256);
  QP_REQUIRE(slots * pairs * 256 < (INT64_C(1) << 32), QP_EUNSUPPORTED,
             "qgemm_w4 gradient: rows and K for more than 2^32 threads");
  constexpr size_t kLds = sizeof(DxLds<T, kKind, kMT>);
  const auto kern = w4_dx_tile_kernel<T, kKind, kMT>;
  // raise the kernel's LDS limit once per device (threads may race to set it;
  // repeating it is harmless)
  static std::atomic<uint64_t> lds_attr_devices{0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) QP_FAIL(QP_EHIP, "qgemm_w4 gradient: hipGetDevice failed");
  const uint64_t bit = dev >= 0 && dev < 64 ? (UINT64_C(1) << dev) : 0;
  if (bit == 0 || (lds_attr_devices.load(std::memory_order_acquire) & bit) == 0) {
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLds) != hipSuccess)
      QP_FAIL(QP_EHIP, "qgemm_w4 gradient: cannot reserve %zu bytes of LDS", kLds);
    lds_attr_devices.fetch_or(bit, std::memory_order_release);
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)(slots * pairs)), dim3(256), kLds, stream, a,
                     (uint32_t)pairs);
  return check_launch("qgemm_w4 gradient (many rows)");
}

template <typename T, int kKind, bool kOne, int kMT>
qp_status launch_dx_rows(const W4DxArgs& a, int64_t splits, float* part, hipStream_t stream) {
  constexpr int kWaves = 8;
  const int64_t slots = w4_tile_slots(a.rows, 16 * kMT);
  const int64_t blocks = slots * splits * ceil_div(a.w.K, 128);
  QP_REQUIRE(blocks * kWaves * 64 < (INT64_C(1) << 32), QP_EUNSUPPORTED,
             "qgemm_w4 gradient: rows and K for more than 2^32 threads");
  hipLaunchKernelGGL((w4_dx_rows_kernel<T, kKind, kOne, kMT, kWaves>), dim3((unsigned)blocks),
                     dim3(kWaves * 64), 0, stream, a, (uint32_t)splits, part);
  qp_status st = check_launch("qgemm_w4 gradient (few rows)");
  if (st || splits == 1) return st;
  const int64_t pieces = ceil_div(a.w.K, 4);
  hipLaunchKernelGGL((w4_dx_join_kernel<T>), dim3((unsigned)ceil_div(a.rows.M * pieces, 256)),
                     dim3(256), 0, stream, (const float*)part, (uint32_t)splits, a.rows.M, a.w.K,
                     round_up(a.w.K, 128), static_cast<T*>(a.dX), a.lddx, (uint32_t)pieces);
  return check_launch("qgemm_w4 gradient (joining the splits)");
}

// Which kernel, how many rows a workgroup and how many splits of the channels: the
// least of the following estimates, in microseconds.  Measured with bf16 rows,
// N = K = 4096, groups of 32, 1 to 4096 rows: a wave of the few-rows kernel takes
// `step` a 32-channel step while there is up to a workgroup a CU (256), and every
// further round of them takes `more` a step (1, 2 and 4 row fragments: 29, 36 and
// 45 us up to a round, 23, 33 and 44 us every further one); splitting costs a
// second launch and the partial sums' way through memory.  The tile kernel takes
// 155 us for up to a workgroup a CU and 255 us for two, 4096 channels (4096 rows:
// 255 us against 359; 4096 rows of 8 experts 400 against 404; 1024 rows 162
// against 96).  Groups of 128 on, whose rows carry the scales in the few-rows
// kernel, change little there (4096 rows 241 against 349, 2048 rows 161 and 177,
// 3000 of 8 experts 240 and 284).  Where 8 experts' tiles make just a workgroup a
// CU (1536 rows), the empty workgroups of the grid spread them unevenly and the
// tile kernel, taken there, is the slower one (220 against 143).  The few-rows plan must not depend on the rows' type: the workspace
// is asked for without it.
struct DxPlan {
  int frags;       // 16-row fragments of the few-rows kernel
  int64_t splits;
  double cost;
};

double dx_row_tiles(int64_t M, int64_t experts, int64_t rows) {
  if (experts <= 1) return (double)ceil_div(M, rows);
  const double used = (double)(experts < M ? experts : M);
  const double tiles = (double)M / used / (double)rows + 0.5;  // the last one half empty
  return used * (tiles > 1.0 ? tiles : 1.0);
}

DxPlan dx_plan(int64_t M, int64_t experts, int64_t N, int64_t K) {
  constexpr struct {
    int frags;
    double step, more;
  } kCost[] = {{1, 1.6, 1.4}, {2, 2.1, 2.1}, {4, 2.6, 2.75}};
  DxPlan best{1, 1, 1e300};
  const int64_t steps = ceil_div(N, 32), nblk = ceil_div(K, 128);
  for (const auto& c : kCost)
    for (int64_t splits = 1; splits <= 8 && (splits == 1 || splits * 8 <= steps); splits *= 2) {
      const double groups = dx_row_tiles(M, experts, 16 * c.frags) * (double)(nblk * splits);
      const double rounds = (double)(int64_t)((groups + 255.0) / 256.0);
      const double each = (double)ceil_div(ceil_div(steps, splits), 8);
      double cost = 3.0 + each * (c.step + (rounds > 1.0 ? rounds - 1.0 : 0.0) * c.more);
      if (splits > 1) cost += 4.0 + (double)(splits * M * nblk * 128) * 8.0 / 4.0e6;
      if (cost < best.cost) best = DxPlan{c.frags, splits, cost};
    }
  return best;
}

double dx_tile_cost(int64_t M, int64_t experts, int64_t N, int64_t K) {
  const double groups = dx_row_tiles(M, experts, 128) * (double)ceil_div(K, 256);
  const double pairs = (double)(int64_t)(groups / 512.0), rest = groups - pairs * 512.0;
  return 3.0 +
         (pairs * 255.0 + (rest <= 0.0 ? 0.0 : rest <= 256.0 ? 155.0 : 255.0)) * (double)N / 4096.0;
}

int64_t dx_ws_bytes(int64_t M, int64_t experts, int64_t N, int64_t K) {
  const DxPlan p = dx_plan(M, experts, N, K);
  return p.splits == 1 ? 0 : round_up(p.splits * M * round_up(K, 128) * 4, 256);
}

// The tile kernel is for bf16: the pieces of f16 and f32 rows leave it no more
// rows a workgroup than the other has (f16: 242 us against 231 at 2048 rows).
// It addresses its rows by 32-bit offsets from the tile's first.
bool dx_takes_tile(int64_t M, int64_t experts, int64_t N, int64_t K, int32_t dtype, int64_t lddy,
                   const DxPlan& p) {
  return dtype == QP_BF16 && 128 * lddy * 2 < (INT64_C(1) << 32) &&
         dx_tile_cost(M, experts, N, K) < p.cost;
}

template <typename T, int kKind, bool kOne>
qp_status launch_dx_frags(const W4DxArgs& a, const DxPlan& p, float* part, hipStream_t stream) {
  if (p.frags == 1) return launch_dx_rows<T, kKind, kOne, 1>(a, p.splits, part, stream);
  if (p.frags == 2) return launch_dx_rows<T, kKind, kOne, 2>(a, p.splits, part, stream);
  return launch_dx_rows<T, kKind, kOne, 4>(a, p.splits, part, stream);
}

template <typename T, int kKind>
qp_status launch_dx(const W4DxArgs& a, void* ws, hipStream_t stream) {
  const int64_t M = a.rows.M, experts = a.rows.offsets ? a.rows.experts : 1;
  const DxPlan p = dx_plan(M, experts, a.w.N, a.w.K);
  if constexpr (__is_same(T, bf16_t)) {
    if (dx_takes_tile(M, experts, a.w.N, a.w.K, a.dtype, a.lddy, p))
      return launch_dx_tile<T, kKind, 4>(a, stream);
  }
  float* part = static_cast<float*>(ws);
  if constexpr (kKind != 2)
    if (a.w.group >= 128)
      return launch_dx_frags<T, kKind, true>(a, p, part, stream);
  return launch_dx_frags<T, kKind, false>(a, p, part, stream);
}

template <typename T>
qp_status launch_dx_kind(const W4DxArgs& a, int32_t format, void* ws, hipStream_t stream) {
  if (format == 2) return launch_dx<T, 0>(a, ws, stream);
  if (format == 3) return launch_dx<T, 1>(a, ws, stream);
  return launch_dx<T, 2>(a, ws, stream);
}

qp_status dx_entry(const char* what, const void* dY, int32_t dtype, int64_t M, int64_t lddy,
                   const qp_packed_info* w, const void* packed, int64_t expert_stride,
                   int64_t experts, const int32_t* offsets, void* dX, int64_t lddx, void* ws,
                   size_t ws_bytes, hipStream_t stream) {
  QP_REQUIRE(M >= 0, QP_EINVAL, "%s: M is negative", what);
  QP_REQUIRE(M <= kW4MaxRows, QP_EUNSUPPORTED, "%s: more than 2^30 rows", what);
  qp_status st = w4_check_weights(what, w, packed, experts, expert_stride);
  if (st || M == 0) return st;
  if ((st = w4_check_float(what, "dY", dY, dtype, lddy, w->N))) return st;
  if ((st = w4_check_float(what, "dX", dX, dtype, lddx, w->K))) return st;
  const size_t need = (size_t)dx_ws_bytes(M, offsets ? experts : 1, w->N, w->K);
  QP_REQUIRE(ws_bytes >= need, QP_ESIZE, "%s: workspace holds %zu bytes, needs %zu", what, ws_bytes,
             need);
  QP_REQUIRE(need == 0 || (ws && (uintptr_t)ws % 256 == 0), QP_EALIGN,
             "%s: workspace must be non-null and 256-byte aligned", what);
  W4DxArgs a{w4_view(w, packed, expert_stride),
             W4Rows{offsets, (int32_t)experts, M, nullptr, 1, M}, dY, lddy, dX, dtype, lddx};
  if (dtype == QP_F32) return launch_dx_kind<float>(a, w->format, ws, stream);
  if (dtype == QP_BF16) return launch_dx_kind<bf16_t>(a, w->format, ws, stream);
  return launch_dx_kind<f16_t>(a, w->format, ws, stream);
}

}  // namespace

void w4_dx_kernel_name(int64_t M, const qp_packed_info* w, int32_t dtype, int64_t experts,
                       char* name, size_t bytes) {
  const DxPlan p = dx_plan(M, experts, w->N, w->K);
  if (dx_takes_tile(M, experts, w->N, w->K, dtype, w->N, p))
    std::snprintf(name, bytes, "tile");
  else
    std::snprintf(name, bytes, "rows%d/%d", p.frags, (int)p.splits);
}

}  // namespace qp

extern "C" qp_status qgemm_w4_dx_ws_size(int64_t M, const qp_packed_info* w, int64_t experts,
                                         size_t* bytes) {
  using namespace qp;
  clear_error();
  QP_REQUIRE(w && bytes && M >= 0 && M <= kW4MaxRows && experts >= 1 && w->N > 0 && w->K > 0,
             QP_EINVAL, "qgemm_w4_dx_ws_size: bad argument");
  *bytes = M == 0 ? 0 : (size_t)dx_ws_bytes(M, experts, w->N, w->K);
  return QP_OK;
}

extern "C" qp_status qgemm_w4_blockwise_dx(const void* dY, int32_t dtype, int64_t M, int64_t lddy,
                                           const qp_packed_info* w, const void* packedW_dev,
                                           void* dX, int64_t lddx, void* ws, size_t ws_bytes,
                                           hipStream_t stream) {
  using namespace qp;
  clear_error();
  return dx_entry("qgemm_w4_blockwise_dx", dY, dtype, M, lddy, w, packedW_dev, 0, 1, nullptr, dX,
                  lddx, ws, ws_bytes, stream);
}

extern "C" qp_status qgemm_w4_experts_dx(const void* dY, int32_t dtype, int64_t M, int64_t lddy,
                                         const qp_packed_info* w, const void* packedW_dev,
                                         int64_t expert_stride, int64_t experts,
                                         const int32_t* offsets, void* dX, int64_t lddx, void* ws,
                                         size_t ws_bytes, hipStream_t stream) {
  using namespace qp;
  clear_error();
  QP_REQUIRE(offsets, QP_EINVAL, "qgemm_w4_experts_dx: offsets is null");
  return dx_entry("qgemm_w4_experts_dx", dY, dtype, M, lddy, w, packedW_dev, expert_stride, experts,
                  offsets, dX, lddx, ws, ws_bytes, stream);
}
