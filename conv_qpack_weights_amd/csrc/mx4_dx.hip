// mx4_dx.hip -- the gradient of the products with MXFP4 weights to their rows:
//   dx[r,k] = sum_n dy[r,n] w[n,k]
// The sum runs along the channels, a row of the codes along k: the MFMA operand
// of a column wants eight channels' values of it side by side.  A lane takes a
// word (eight k) of each of eight channels, converts them to bf16 with their
// channels' scales, exactly, and pairs the channels' halves up (32 conversions
// and 32 v_perm for eight operands, no LDS): operand j then holds column 8 i + j
// in lane i of 16, and a lane ends with eight neighbouring columns of a row.
#include "mx4.hpp"

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
// A workgroup owns 16 kFM rows and 128 columns of one split of the channels; its
// waves take every kWaves-th step of 32 channels and meet in LDS in a fixed
// order.  More than one split: the sums go to `part`, added up by the kernel
// below.
template <typename T, int kFM, int kWaves>
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
  const W4Tile tile = w4_find_tile<16 * kFM>(a.rows, slot);
  if (tile.expert < 0) return;
  const int64_t k0 = (int64_t)cb * 128, N = a.w.rows, K = a.w.K;
  const bool none = a.rows.offsets && tile.expert == a.rows.experts;
  const int ch = lane & 15, quad = lane >> 4;

  f32x4 acc[kFM][8];
#pragma unroll
  for (int f = 0; f < kFM; ++f)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[f][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  if (!none) {
    const T* dy[kFM];
#pragma unroll
    for (int f = 0; f < kFM; ++f) {
      int64_t r = tile.r0 + f * 16 + ch;
      r = r < tile.r1 ? r : tile.r1 - 1;
      dy[f] = static_cast<const T*>(a.dY) + r * a.lddy;
    }
    // columns past K's last block read the row's first word: not stored
    const bool col_in = k0 / 32 + ch / 4 < a.w.G;
    const uint8_t* codes = a.w.codes + tile.expert * a.w.cstride + (col_in ? k0 / 2 + 4 * ch : 0);
    const uint8_t* scales = a.w.scales + tile.expert * a.w.sstride + k0 / 32;
    const uint32_t shift = 8 * (ch / 4);

    const int64_t steps = (N + 31) / 32;
    for (int64_t s = (int64_t)split * kWaves + wave; s < steps; s += (int64_t)splits * kWaves) {
      const int64_t n0 = s * 32 + quad * 8;
      uint32_t w[8], sc[8];
      MxFrag<T> x[kFM];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t n = n0 + i < N ? n0 + i : N - 1;
        w[i] = *reinterpret_cast<const uint32_t*>(codes + n * a.w.ldc);
        sc[i] = *reinterpret_cast<const uint32_t*>(scales + n * a.w.lds);
      }
      const int64_t left = N - n0;
      const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
#pragma unroll
      for (int f = 0; f < kFM; ++f) x[f].load_n(dy[f] + (n > 0 ? n0 : 0), n);
      float by[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)  // (a channel past the last: its scale could be a NaN)
        by[i] = mx_scale(i < n ? (sc[i] >> shift) & 0xffu : 0u);
      bf16x8 o[8];
      mx_columns(w, by, o);
#pragma unroll
      for (int f = 0; f < kFM; ++f) {
        bf16x8 xv[NP];
        x[f].split(xv);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int p = 0; p < NP; ++p) acc[f][j] = mfma32(xv[p], o[j], acc[f][j]);
      }
    }
  }

  // thread: 8 columns of a row
#pragma unroll
  for (int f = 0; f < kFM; ++f) {
    if (f) __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) red[wave][j][lane] = acc[f][j];
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += kWaves * 64) {
      const int m = i >> 4, c = i & 15;
      const int64_t r = tile.r0 + f * 16 + m, col = k0 + 8 * c;
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

// In how many splits the channels go: enough workgroups for the card, no split
// without a step of 32 channels for each of its waves.
constexpr int kDxWaves = 8;
uint32_t dx_splits(int64_t M, const qp_mx4* w, int64_t experts) {
  const int64_t parts = experts < M ? experts : M;
  const int64_t groups = (M / 16 + parts) * ceil_div(w->K, 128);
  const int64_t most = ceil_div(ceil_div(w->rows, 32), kDxWaves);
  int64_t s = 512 / groups;
  s = s > most ? most : s;
  s = s > 16 ? 16 : s;
  return s < 1 ? 1u : (uint32_t)s;
}

template <typename T>
void launch_dx(const MxDxArgs& a, uint32_t slots, uint32_t splits, hipStream_t stream) {
  const int64_t cols = ceil_div(a.w.K, 128);
  hipLaunchKernelGGL((mx_dx_rows_kernel<T, 1, kDxWaves>), dim3((unsigned)(slots * cols * splits)),
                     dim3(kDxWaves * 64), 0, stream, a, slots, splits);
}

qp_status dx_ws(int64_t M, const qp_mx4* w, int64_t experts, uint32_t* splits, size_t* bytes) {
  *splits = M > 0 ? dx_splits(M, w, experts) : 1;
  *bytes = *splits > 1 ? (size_t)(4 * (int64_t)*splits * M * w->K) : 0;
  return QP_OK;
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
  uint32_t splits;
  size_t need;
  dx_ws(M, w, w->matrices, &splits, &need);
  QP_REQUIRE(ws_bytes >= need, QP_ESIZE, "%s: needs a workspace of %zu bytes, has %zu", what, need,
             ws_bytes);
  QP_REQUIRE(!need || (ws && (uintptr_t)ws % 256 == 0), QP_EALIGN,
             "%s: the workspace must be 256-byte aligned", what);
  MxDxArgs a{mx_view(w), W4Rows{offsets, (int32_t)w->matrices, M, nullptr, 1, M}, dY, lddy, dX,
             dtype, lddx, static_cast<float*>(ws)};
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
  uint32_t splits;
  return dx_ws(M, w, w->matrices, &splits, bytes);
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
