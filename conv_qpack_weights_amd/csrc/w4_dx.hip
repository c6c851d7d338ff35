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
// out is below 2^-16 of a term (2^-23 for f32 rows).  Sums are f32.
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
// the value.  Where the first piece is an infinity or a NaN (the value is one,
// or rounds up to one) the others are zero.
template <int kPieces>
__device__ __forceinline__ void split_bf16(const float (&f)[8], bf16x8 (&o)[kPieces]) {
  u32x4 p[kPieces];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = f[2 * i], b = f[2 * i + 1];
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
      const uint32_t h = bf16_pair(a, b);
      p[n][i] = h;
      if (n + 1 < kPieces) {
        a = a - low_f32(h);
        b = b - high_f32(h);
        if (n == 0) {
          a = a == a && __builtin_fabsf(a) != __builtin_inff() ? a : 0.0f;
          b = b == b && __builtin_fabsf(b) != __builtin_inff() ? b : 0.0f;
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
  static constexpr int kPieces = 1, kWPieces = 2;
  XFrag<bf16_t> x;
  __device__ __forceinline__ void split(bf16x8 (&o)[1]) const {
    o[0] = __builtin_bit_cast(bf16x8, x.v);
  }
};
template <>
struct YFrag<f16_t> {
  static constexpr int kPieces = 2, kWPieces = 2;  // 11 bits: two pieces hold them
  XFrag<f16_t> x;
  __device__ __forceinline__ void split(bf16x8 (&o)[2]) const {
    const f16x8 h = __builtin_bit_cast(f16x8, x.v);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)h[i];
    split_bf16<2>(f, o);
  }
};
template <>
struct YFrag<float> {
  static constexpr int kPieces = 3, kWPieces = 3;
  XFrag<float> x;
  __device__ __forceinline__ void split(bf16x8 (&o)[3]) const {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = x.v[i / 4][i & 3];
      f[i] = __builtin_bit_cast(float, u);
    }
    split_bf16<3>(f, o);
  }
};

template <typename T, int kKind, int kMT>
struct DxStage {
  uint32_t d[8];
  float s[8];
  float o[kKind == 2 ? 8 : 1];
  YFrag<T> y[kMT];
};

// A workgroup owns one 128-K block and 16*kMT rows; its waves share out the
// channels, 32 a step, and their sums meet in LDS in a fixed order.
template <typename T, int kKind, int kMT, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void w4_dx_kernel(W4DxArgs a) {
  __shared__ f32x4 red[kMT * 8][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const W4Tile tile = w4_find_tile<16 * kMT>(a.rows, blockIdx.y);
  if (tile.expert < 0) return;
  const int64_t blk = blockIdx.x;
  const int c = lane & 15, h = lane >> 4;
  const int64_t k0 = blk * 128 + 8 * c;
  constexpr int kPer = 16 / sizeof(T);

  f32x4 acc[kMT][8];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[m][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const bool real = !(a.rows.offsets && tile.expert == a.rows.experts);
  if (real) {
    const uint8_t* blob = a.w.blob + tile.expert * a.w.expert_stride;
    const T* yr[kMT];
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      int64_t r = tile.r0 + m * 16 + c;
      r = r < tile.r1 ? r : tile.r1 - 1;  // repeated rows are not stored
      yr[m] = static_cast<const T*>(a.dY) + r * a.lddy + 8 * h;
    }
    // lane c's word of a block: group t = c/4, chunk c%4; its scale's group
    const int64_t word = (c & 3) * 16 + (c >> 2) * 4;
    const int64_t g = (blk * 128 + 32 * (c >> 2)) / a.w.group;
    const int64_t se = (g / 4) * 64 + (g & 3);
    auto load_weights = [&](DxStage<T, kKind, kMT>& st, int64_t n0) {
      const int64_t tc = n0 / 16 + (h >> 1);
      const uint8_t* q = blob + a.w.data_off + (tc * a.w.nblk + blk) * 1024 + (h & 1) * 512 + word;
      const int64_t e = tc * a.w.G4 * 64 + (h & 1) * 32 + se;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        st.d[r] = *reinterpret_cast<const uint32_t*>(q + r * 64);
        if constexpr (kKind == 1) {
          const uint32_t u = reinterpret_cast<const uint16_t*>(blob + a.w.scale_off)[e + r * 4];
          st.s[r] = __builtin_bit_cast(float, u << 16);
        } else {
          st.s[r] = reinterpret_cast<const float*>(blob + a.w.scale_off)[e + r * 4];
        }
        if constexpr (kKind == 2)
          st.o[r] = reinterpret_cast<const float*>(blob + a.w.offs_off)[e + r * 4];
      }
    };
    auto step = [&](const DxStage<T, kKind, kMT>& st) {
      constexpr int NY = YFrag<T>::kPieces, NW = YFrag<T>::kWPieces;
      float s16[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) s16[r] = st.s[r] * 16.0f;
      bf16x8 y[kMT][NY];
#pragma unroll
      for (int m = 0; m < kMT; ++m) st.y[m].split(y[m]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int sh = j < 4 ? 8 * j : 8 * (j - 4) + 4;
        float f[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          f[r] = nib_f32(st.d[r] >> sh) * s16[r];
          if constexpr (kKind == 2) f[r] = f[r] + st.o[r];
        }
        bf16x8 w[NW];
        split_bf16<NW>(f, w);
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
          for (int sum = NW - 1; sum >= 0; --sum)  // small products first
#pragma unroll
            for (int i = 0; i < NY; ++i)
              if (sum - i >= 0 && sum - i < NW) acc[m][j] = mfma32(y[m][i], w[sum - i], acc[m][j]);
      }
    };
    const int64_t full = a.w.N / 32;
    for (int64_t i = wave; i < full; i += kWaves) {
      DxStage<T, kKind, kMT> st;
      load_weights(st, i * 32);
#pragma unroll
      for (int m = 0; m < kMT; ++m) st.y[m].x.load(yr[m] + i * 32);
      step(st);
    }
    if (full * 32 < a.w.N && wave == full % kWaves) {
      DxStage<T, kKind, kMT> st;
      load_weights(st, full * 32);
      const int64_t left = a.w.N - (full * 32 + 8 * h);
      const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
#pragma unroll
      for (int m = 0; m < kMT; ++m)
        st.y[m].x.load_n(yr[m] + (n > 0 ? full * 32 : -8 * h), n);
      step(st);
    }
  }

  for (int w = 1; w < kWaves; ++w) {
    if (wave == w) {
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) red[m * 8 + j][lane] = acc[m][j];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[m][j] += red[m * 8 + j][lane];
    }
    __syncthreads();
  }
  if (wave != 0 || k0 >= a.w.K) return;
  const int n = a.w.K - k0 < 8 ? (int)(a.w.K - k0) : 8;
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = tile.r0 + m * 16 + 4 * h + i;
      if (r >= tile.r1) continue;
      T* dst = static_cast<T*>(a.dX) + r * a.lddx + k0;
#pragma unroll
      for (int p = 0; p < 8 / kPer; ++p) {
        float f[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) f[j] = acc[m][p * kPer + j][i];
        if (n > p * kPer) store_piece(dst + p * kPer, f, n - p * kPer);
      }
    }
}

template <typename T, int kKind>
qp_status launch_dx(const W4DxArgs& a, hipStream_t stream) {
  constexpr int kMT = 4, kWaves = 4;
  const int64_t gx = a.w.nblk, gy = w4_tile_slots(a.rows, 16 * kMT);
  QP_REQUIRE(gy <= 65535, QP_EUNSUPPORTED, "qgemm_w4 gradient: too many rows for one launch");
  hipLaunchKernelGGL((w4_dx_kernel<T, kKind, kMT, kWaves>), dim3((unsigned)gx, (unsigned)gy),
                     dim3(kWaves * 64), 0, stream, a);
  return check_launch("qgemm_w4 gradient");
}

template <typename T>
qp_status launch_dx_kind(const W4DxArgs& a, int32_t format, hipStream_t stream) {
  if (format == 2) return launch_dx<T, 0>(a, stream);
  if (format == 3) return launch_dx<T, 1>(a, stream);
  return launch_dx<T, 2>(a, stream);
}

qp_status dx_entry(const char* what, const void* dY, int32_t dtype, int64_t M, int64_t lddy,
                   const qp_packed_info* w, const void* packed, int64_t expert_stride,
                   int64_t experts, const int32_t* offsets, void* dX, int64_t lddx, void* ws,
                   size_t ws_bytes, hipStream_t stream) {
  QP_REQUIRE(M >= 0, QP_EINVAL, "%s: M is negative", what);
  QP_REQUIRE(M <= INT32_MAX, QP_EUNSUPPORTED, "%s: more than 2^31-1 rows", what);
  qp_status st = w4_check_weights(what, w, packed, experts, expert_stride);
  if (st || M == 0) return st;
  if ((st = w4_check_float(what, "dY", dY, dtype, lddy, w->N))) return st;
  if ((st = w4_check_float(what, "dX", dX, dtype, lddx, w->K))) return st;
  W4DxArgs a{w4_view(w, packed, expert_stride),
             W4Rows{offsets, (int32_t)experts, M, nullptr, 1, M}, dY, lddy, dX, dtype, lddx};
  if (dtype == QP_F32) return launch_dx_kind<float>(a, w->format, stream);
  if (dtype == QP_BF16) return launch_dx_kind<bf16_t>(a, w->format, stream);
  return launch_dx_kind<f16_t>(a, w->format, stream);
}

}  // namespace
}  // namespace qp

extern "C" qp_status qgemm_w4_dx_ws_size(int64_t M, const qp_packed_info* w, int64_t experts,
                                         size_t* bytes) {
  using namespace qp;
  clear_error();
  QP_REQUIRE(w && bytes && M >= 0 && experts >= 1, QP_EINVAL, "qgemm_w4_dx_ws_size: bad argument");
  *bytes = 0;
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
