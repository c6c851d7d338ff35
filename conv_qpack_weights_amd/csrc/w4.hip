// w4.hip -- float rows times packed int4 weights with group scales, dense or
// grouped by expert:
//   y[r,n] = clamp(sum_g s[n,g] * P[r,n,g] (+ o[n,g] * S[r,g]) + bias[n], lo, hi)
//   P[r,n,g] = sum_{k in g} x[r,k] q[n,k],   S[r,g] = sum_{k in g} x[r,k]
// The rows stay in their own type (bf16, f16; f32 as three bf16 pieces) and q
// goes into the MFMA exactly, so the only roundings are those of the f32
// sums; the scales multiply the f32 group sums.  q enters as q/16 (what the
// 4-bit conversion gives); the factor 16 leaves exactly at the end.
#include "w4.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

struct W4Args {
  W4View w;
  W4Rows rows;
  const void* X;
  int64_t ldx;
  const float* bias;   // [experts][N] or null
  float lo, hi;
  void* Y;
  int32_t y_dtype;
  int64_t ldy;
};

// The four 32-K scales (or offsets) of a channel's 128-K block: groups of 32
// have one each; a group of 64 serves two; larger groups have one in all
// (kOne), returned in the first place.
template <bool kBf16, bool kOne>
__device__ __forceinline__ f32x4 w4_scales(const uint8_t* p, int64_t tile, int64_t G4, int64_t b,
                                           int32_t group, int ch) {
  const int64_t base = tile * G4 * 64 + ch * 4;
  auto one = [&](int64_t g) -> float {
    const int64_t e = base + (g / 4) * 64 + (g & 3);
    if constexpr (kBf16) {
      const uint32_t u = reinterpret_cast<const uint16_t*>(p)[e];
      return __builtin_bit_cast(float, u << 16);
    } else {
      return reinterpret_cast<const float*>(p)[e];
    }
  };
  f32x4 s;
  if constexpr (kOne) {
    s[0] = one((b * 128) / group);
    s[1] = s[2] = s[3] = s[0];
  } else if (group == 32) {
    const int64_t e = base + b * 64;
    if constexpr (kBf16) {
      const u32x2 u = *reinterpret_cast<const u32x2*>(p + e * 2);
      const uint32_t lo = u.x, hi = u.y;
      s[0] = __builtin_bit_cast(float, lo << 16);
      s[1] = __builtin_bit_cast(float, lo & 0xffff0000u);
      s[2] = __builtin_bit_cast(float, hi << 16);
      s[3] = __builtin_bit_cast(float, hi & 0xffff0000u);
    } else {
      s = *reinterpret_cast<const f32x4*>(p + e * 4);
    }
  } else {  // 64
    s[0] = s[1] = one(2 * b);
    s[2] = s[3] = one(2 * b + 1);
  }
  return s;
}

// One block's operands of a wave: kTiles channel tiles, kFM row fragments.
template <typename T, int kKind, int kFM, int kTiles>
struct W4Stage {
  u32x4 q[kTiles];
  f32x4 s[kTiles];
  f32x4 o[kKind == 2 ? kTiles : 1];
  XFrag<T> x[kFM][4];
};

template <typename T, int kKind, bool kOne, int kFM, int kTiles>
__device__ __forceinline__ void w4_step(const W4Stage<T, kKind, kFM, kTiles>& st,
                                        f32x4 (&acc)[kFM][kTiles]) {
  using V = typename XFrag<T>::vec;
  constexpr int NP = XFrag<T>::kPieces;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 p[kFM][kTiles], sum[kFM];
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
            a = __builtin_fmaf(st.s[c][t], p[f][c][i], a);
            if constexpr (kKind == 2) a = __builtin_fmaf(st.o[c][t], sum[f][i], a);
            acc[f][c][i] = a;
          }
      }
    }
  }
}

// ---- few rows: the waves of a workgroup share out K --------------------------
// A workgroup owns kTiles 16-channel tiles and 16*kFM rows; each wave takes a
// run of 128-K blocks, keeps kAhead of them in flight in registers (weights,
// scales and the rows' pieces, all straight from memory: a wave's rows are
// nobody else's, so LDS would only add a hop), and the waves' sums meet in LDS
// in a fixed order.
template <typename T, int kKind, bool kOne, int kFM, int kTiles, int kWaves, int kAhead>
__global__ __launch_bounds__(kWaves * 64) void w4_rows_kernel(W4Args a) {
  __shared__ f32x4 red[kWaves][kFM * kTiles][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const W4Tile tile = w4_find_tile<16 * kFM>(a.rows, blockIdx.y);
  if (tile.expert < 0) return;
  const int64_t n0 = (int64_t)blockIdx.x * kTiles * 16;
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
  using Stage = W4Stage<T, kKind, kFM, kTiles>;
  auto load_weights = [&](Stage& st, int64_t b) {
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      const int64_t tc = t0 + c < last_tile ? t0 + c : last_tile;
      st.q[c] = *reinterpret_cast<const u32x4*>(blob + a.w.data_off +
                                                (tc * a.w.nblk + b) * 1024 + ch * 64 + quad * 16);
      st.s[c] = w4_scales<kKind == 1, kOne>(blob + a.w.scale_off, tc, a.w.G4, b, a.w.group, ch);
      if constexpr (kKind == 2)
        st.o[c] = w4_scales<false, kOne>(blob + a.w.offs_off, tc, a.w.G4, b, a.w.group, ch);
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
    for (int64_t b = b0; b < b1; b += kAhead) {
#pragma unroll
      for (int p = 0; p < kAhead; ++p) {
        if (b + p < b1) w4_step<T, kKind, kOne, kFM, kTiles>(st[p], acc);
        const int64_t nb = b + p + kAhead;
        load(st[p], nb < b1 ? nb : b1 - 1);
      }
    }
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
    w4_step<T, kKind, kOne, kFM, kTiles>(st, acc);
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
  const int64_t gx = ceil_div(a.w.Npad / 16, kTiles), gy = w4_tile_slots(a.rows, 16 * kFM);
  QP_REQUIRE(gy <= 65535, QP_EUNSUPPORTED, "qgemm_w4: too many rows for one launch");
  hipLaunchKernelGGL((w4_rows_kernel<T, kKind, kOne, kFM, kTiles, kWaves, kAhead>),
                     dim3((unsigned)gx, (unsigned)gy), dim3(kWaves * 64), 0, stream, a);
  return check_launch("qgemm_w4 (few rows)");
}

template <typename T, int kKind, bool kOne>
qp_status launch_w4(const W4Args& a, hipStream_t stream) {
  return launch_rows<T, kKind, kOne, 1, 2, 8, 2>(a, stream);
}

template <typename T>
qp_status launch_w4_kind(const W4Args& a, int32_t format, hipStream_t stream) {
  const bool one = a.w.group >= 128;
  if (format == 2) return one ? launch_w4<T, 0, true>(a, stream) : launch_w4<T, 0, false>(a, stream);
  if (format == 3) return one ? launch_w4<T, 1, true>(a, stream) : launch_w4<T, 1, false>(a, stream);
  return one ? launch_w4<T, 2, true>(a, stream) : launch_w4<T, 2, false>(a, stream);
}

qp_status run_w4(const W4Args& a, int32_t dtype, int32_t format, hipStream_t stream) {
  if (dtype == QP_F32) return launch_w4_kind<float>(a, format, stream);
  if (dtype == QP_BF16) return launch_w4_kind<bf16_t>(a, format, stream);
  return launch_w4_kind<f16_t>(a, format, stream);
}

qp_status check_y(const char* what, const void* Y, int32_t dtype, int32_t y_dtype, int64_t ldy,
                  int64_t N) {
  qp_status st = w4_check_float(what, "Y", Y, y_dtype, ldy, N);
  if (st) return st;
  QP_REQUIRE(y_dtype == dtype || y_dtype == QP_F32, QP_EUNSUPPORTED,
             "%s: outputs are stored in the rows' type or in f32", what);
  return QP_OK;
}

}  // namespace

W4View w4_view(const qp_packed_info* w, const void* packed, int64_t expert_stride) {
  W4View v;
  v.blob = static_cast<const uint8_t*>(packed);
  v.expert_stride = expert_stride;
  v.data_off = w->data_off;
  v.scale_off = w->scale_off;
  v.offs_off = w->format == 4 ? w->zp_off : 0;
  v.N = w->N;
  v.Npad = w->Npad;
  v.K = w->K;
  v.nblk = w->Kpad / 128;
  v.G4 = ceil_div(w->Kpad / w->group, 4);
  v.group = (int32_t)w->group;
  return v;
}

qp_status w4_check_weights(const char* what, const qp_packed_info* w, const void* packed,
                           int64_t experts, int64_t expert_stride) {
  QP_REQUIRE(w && w->format >= 2 && w->format <= 4, QP_EINVAL,
             "%s: weights must be an int4 blob", what);
  // the kernels index the blob by these: hold a description made by hand to them too
  qp_packed_info g;
  qp_status st = blob_geometry(w->format, w->scheme, w->N, w->K, w->group, &g);
  if (st) return st;
  QP_REQUIRE(g.Npad == w->Npad && g.Kpad == w->Kpad && g.data_off == w->data_off &&
                 g.scale_off == w->scale_off && g.zp_off == w->zp_off &&
                 g.total_bytes == w->total_bytes,
             QP_EINVAL, "%s: the weights' description does not match their shape", what);
  QP_REQUIRE(packed, QP_EINVAL, "%s: the weights are null", what);
  QP_REQUIRE((uintptr_t)packed % 256 == 0, QP_EALIGN, "%s: the weights must be 256-byte aligned",
             what);
  QP_REQUIRE(experts >= 1, QP_EINVAL, "%s: needs at least one expert", what);
  QP_REQUIRE(experts <= 65536, QP_EUNSUPPORTED, "%s: more than 65536 experts", what);
  QP_REQUIRE(experts == 1 || (expert_stride >= w->total_bytes && expert_stride % 256 == 0),
             QP_EINVAL, "%s: the experts' blobs must be total_bytes or more apart, a multiple of 256",
             what);
  return QP_OK;
}

qp_status w4_check_float(const char* what, const char* name, const void* p, int32_t dtype,
                         int64_t ld, int64_t cols) {
  QP_REQUIRE(dtype == QP_F32 || dtype == QP_BF16 || dtype == QP_F16, QP_EINVAL,
             "%s: %s must be QP_F32, QP_BF16 or QP_F16 (got %d)", what, name, dtype);
  QP_REQUIRE(ld >= cols, QP_EINVAL, "%s: the stride of %s is below its %lld columns", what, name,
             (long long)cols);
  QP_REQUIRE(p, QP_EINVAL, "%s: %s is null", what, name);
  QP_REQUIRE((uintptr_t)p % elem_bytes(dtype) == 0, QP_EALIGN,
             "%s: %s is not aligned to its elements", what, name);
  return QP_OK;
}

}  // namespace qp

extern "C" qp_status qgemm_w4_blockwise(const void* X, int32_t dtype, int64_t M, int64_t K,
                                        int64_t ldx, const qp_packed_info* w,
                                        const void* packedW_dev, const float* bias, float clamp_lo,
                                        float clamp_hi, void* Y, int32_t y_dtype, int64_t ldy,
                                        hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_w4_blockwise";
  QP_REQUIRE(M >= 0, QP_EINVAL, "%s: M is negative", what);
  QP_REQUIRE(M <= INT32_MAX, QP_EUNSUPPORTED, "%s: more than 2^31-1 rows", what);
  qp_status st = w4_check_weights(what, w, packedW_dev, 1, 0);
  if (st) return st;
  QP_REQUIRE(K == w->K, QP_EINVAL, "%s: the rows have K=%lld but the weights K=%lld", what,
             (long long)K, (long long)w->K);
  QP_REQUIRE(!(clamp_lo > clamp_hi) && clamp_lo == clamp_lo && clamp_hi == clamp_hi, QP_EINVAL,
             "%s: clamp bounds are NaN or reversed", what);
  if (M == 0) return QP_OK;
  if ((st = w4_check_float(what, "X", X, dtype, ldx, K))) return st;
  if ((st = check_y(what, Y, dtype, y_dtype, ldy, w->N))) return st;
  W4Args a{w4_view(w, packedW_dev, 0), W4Rows{nullptr, 1, M, nullptr, 1, M}, X, ldx, bias,
           clamp_lo, clamp_hi, Y, y_dtype, ldy};
  return run_w4(a, dtype, w->format, stream);
}

extern "C" qp_status qgemm_w4_experts(const void* X, int32_t dtype, int64_t x_rows, int64_t K,
                                      int64_t ldx, const int32_t* rows, int64_t row_div, int64_t M,
                                      const qp_packed_info* w, const void* packedW_dev,
                                      int64_t expert_stride, int64_t experts,
                                      const int32_t* offsets, const float* bias, float clamp_lo,
                                      float clamp_hi, void* Y, int32_t y_dtype, int64_t ldy,
                                      hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qgemm_w4_experts";
  QP_REQUIRE(M >= 0 && x_rows >= 0, QP_EINVAL, "%s: a row count is negative", what);
  QP_REQUIRE(M <= INT32_MAX, QP_EUNSUPPORTED, "%s: more than 2^31-1 rows", what);
  qp_status st = w4_check_weights(what, w, packedW_dev, experts, expert_stride);
  if (st) return st;
  QP_REQUIRE(K == w->K, QP_EINVAL, "%s: the rows have K=%lld but the weights K=%lld", what,
             (long long)K, (long long)w->K);
  QP_REQUIRE(!(clamp_lo > clamp_hi) && clamp_lo == clamp_lo && clamp_hi == clamp_hi, QP_EINVAL,
             "%s: clamp bounds are NaN or reversed", what);
  QP_REQUIRE(offsets, QP_EINVAL, "%s: offsets is null", what);
  QP_REQUIRE(rows || x_rows >= M, QP_EINVAL, "%s: X has %lld rows, fewer than M=%lld", what,
             (long long)x_rows, (long long)M);
  QP_REQUIRE(!rows || (row_div >= 1 && row_div <= INT32_MAX), QP_EINVAL, "%s: row_div must be >= 1",
             what);
  if (M == 0) return QP_OK;
  QP_REQUIRE(x_rows > 0, QP_EINVAL, "%s: X has no rows", what);
  if ((st = w4_check_float(what, "X", X, dtype, ldx, K))) return st;
  if ((st = check_y(what, Y, dtype, y_dtype, ldy, w->N))) return st;
  W4Args a{w4_view(w, packedW_dev, expert_stride),
           W4Rows{offsets, (int32_t)experts, M, rows, rows ? row_div : 1, x_rows},
           X, ldx, bias, clamp_lo, clamp_hi, Y, y_dtype, ldy};
  return run_w4(a, dtype, w->format, stream);
}
