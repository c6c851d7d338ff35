// moe.hip -- rows of tokens sorted by expert and back, with weights applied,
// and the gradients of both.
//
// T tokens choose top_k experts each; slot s = t*top_k + j is one choice.  A
// slot whose expert id is negative or >= experts is dropped.  The kept slots
// sorted by (expert, slot) are the rows 0 .. offsets[experts]-1; dropped slots
// leave as many rows without a slot at the end.
//   dispatch       Xs[r] = X[slot_of_row[r] / top_k]          (0 without a slot)
//   dispatch grad  dX[t] = sum_j dXs[row(t,j)]                (kept j)
//   combine        Y[t]  = sum_j w[t,j] * Z[row(t,j)]         (kept j, ascending)
//   combine grad   dZ[row(t,j)] = w[t,j] * dY[t],  dw[t,j] = <dY[t], Z[row(t,j)]>
// Products and sums are f32, rounded once when a row is stored.
//
// What bounds them: the row copies move T*H + S*H elements (S = T*top_k) and
// are bound by HBM; every one of them walks the tokens, so that a token's own
// row crosses the memory once and its top_k rows once each.  8192 tokens x 8,
// rows of 4096 16-bit elements (604 MB): the copy 117 us, the weighted sum 120 us,
// 5.0-5.2 TB/s, what a plain 1 GiB device copy reaches on the same card (5.1).
// The sort reads S ids and writes 2*S integers: a launch and a few dependent
// loads (65536 slots, 128 experts: 4.8 + 9.3 us).
#include <type_traits>

#include "dev_util.hpp"
#include "float_types.hpp"
#include "qp_internal.hpp"

#pragma clang fp contract(off)

namespace qp {
namespace {

constexpr int kMaxExperts = 512;   // the ranking kernel keeps 16 x (experts+1) counters in LDS
constexpr int64_t kMaxSlots = INT64_C(1) << 30;
// Workgroups of 256 threads a launch: a launch has fewer than 2^32 threads along
// x.  Calls that need more (tens of millions of tokens) take several launches.
constexpr int64_t kMaxBlocks = INT64_C(1) << 23;

struct Ids {
  const void* p;
  int64_t ld;      // between tokens, in elements
  int32_t top_k, experts;
  bool wide;       // 64-bit ids
};

// The sort key of slot s: its expert, or `experts` if dropped.
__device__ __forceinline__ int32_t slot_key(const Ids& ids, uint32_t s) {
  const uint32_t t = s / (uint32_t)ids.top_k, j = s - t * (uint32_t)ids.top_k;
  const int64_t at = (int64_t)t * ids.ld + j;
  const int64_t id = ids.wide ? static_cast<const int64_t*>(ids.p)[at]
                              : (int64_t)static_cast<const int32_t*>(ids.p)[at];
  return id >= 0 && id < ids.experts ? (int32_t)id : ids.experts;
}

// Rows are moved 16 bytes a lane at any alignment of the elements (2 or 4
// bytes).  A row's last piece starts early enough to end with the row, over
// elements that the piece before it also brings (the same values twice); only
// rows shorter than a piece go element by element.
template <int ES>
struct RowPiece {
  static constexpr int kPer = 16 / ES;
  using vec = u32x4_any;
  using elem = std::conditional_t<ES == 2, uint16_t, uint32_t>;

  // the piece that begins at element e, or where the row's last one does
  __device__ static __forceinline__ int64_t start(int64_t e, int64_t row_elems) {
    return e + kPer > row_elems && e < row_elems ? row_elems - kPer : e;
  }
  // a row shorter than a piece, by one lane
  __device__ static __forceinline__ void short_row(const uint8_t* src, uint8_t* dst, bool kept,
                                                   int64_t row_elems) {
    elem v[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      v[q] = reinterpret_cast<const elem*>(src)[q < row_elems ? q : 0];
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (q < row_elems) reinterpret_cast<elem*>(dst)[q] = kept ? v[q] : 0;
  }
};

// ---- the sort and the copy in one launch, few slots ------------------------
// A wave per slot finds the slot's row by counting: ids below its own, and
// equal ids before it, 64 ids a step and a ballot each; up to kSmallSlots
// slots that is at most 8 steps on ids that sit in LDS.  The token's row is
// on its way to registers meanwhile.  Blocks past the slots' own
// write the offsets, a thread per expert walking over all the slots: that is what
// ends the range of this kernel.  16 tokens x 2 of 8 experts, rows of 4096 bf16:
// 3.3 us, of which an empty launch is about 2 (three launches took 12).
// Replayed in a graph, against the kernels for many slots: the sort alone, 128
// slots of 64 experts 3.4 us (3.8), 256 slots 5.0 (3.7), 1024 15.4 (4.4), 4096
// 59 (5.8); with rows of 4096 bf16, 256 slots 5.2 (8.7), 512 8.9 (9.2; of 8
// experts 9.1 and 7.5, of 512 experts 10.5 both), 1024 16.1 (10.3).
constexpr int kSmallSort = 128;
constexpr int kSmallSlots = 512;
constexpr int kSmallVecs = 4;  // 16-byte pieces of a row a lane holds

template <int ES, bool kCopy, int kSmallThreads>
__global__ __launch_bounds__(kSmallThreads) void moe_small_kernel(
    Ids ids, uint32_t S, uint32_t slot_blocks, const uint8_t* __restrict__ X, int64_t ldx_bytes,
    int64_t row_elems, uint8_t* __restrict__ Xs, int64_t ldxs_bytes, int32_t* __restrict__ offsets,
    int32_t* __restrict__ row_of_slot, int32_t* __restrict__ slot_of_row) {
  using RP = RowPiece<ES>;
  constexpr int kPer = RP::kPer;
  __shared__ int32_t keys[kSmallSlots];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x >= slot_blocks) {  // offsets: a thread per expert (one block column only)
    for (uint32_t s = threadIdx.x; s < S; s += kSmallThreads) keys[s] = slot_key(ids, s);
    __syncthreads();
    const int e = (int)(blockIdx.x - slot_blocks) * kSmallThreads + threadIdx.x;
    if (blockIdx.y == 0 && e <= ids.experts) {
      int32_t n = 0;
      for (uint32_t s = 0; s < S; ++s) n += keys[s] < e;
      offsets[e] = n;
    }
    return;
  }
  const uint32_t s = blockIdx.x * (kSmallThreads / 64) + wave;
  const bool live = s < S;
  // this wave's piece of the token's row
  const int64_t e0 = ((int64_t)blockIdx.y * kSmallVecs * 64 + lane) * kPer;
  typename RP::vec v[kSmallVecs];
  const uint8_t* src = nullptr;
  if (kCopy && live) {
    src = X + (int64_t)(s / (uint32_t)ids.top_k) * ldx_bytes;
#pragma unroll
    for (int i = 0; i < kSmallVecs; ++i) {
      const int64_t e = RP::start(e0 + (int64_t)i * 64 * kPer, row_elems);
      if (e >= 0 && e < row_elems) v[i] = *reinterpret_cast<const typename RP::vec*>(src + e * ES);
    }
  }
  int32_t mine = 0;
  uint32_t row = 0;
  if (S <= 64) {  // every wave reads the ids itself
    const int32_t key = (uint32_t)lane < S ? slot_key(ids, lane) : ids.experts + 1;
    mine = __builtin_amdgcn_readlane(key, (int)(live ? s : 0));
    row = __popcll(__ballot(key < mine)) +
          __popcll(__ballot(key == mine && (uint32_t)lane < s));
  } else {
    for (uint32_t i = threadIdx.x; i < S; i += kSmallThreads) keys[i] = slot_key(ids, i);
    __syncthreads();
    mine = keys[live ? s : 0];
    for (uint32_t i = 0; i < S; i += 64) {
      const int32_t key = i + lane < S ? keys[i + lane] : ids.experts + 1;
      row += __popcll(__ballot(key < mine)) +
             __popcll(__ballot(key == mine && i + lane < s));
    }
  }
  if (!live) return;
  const bool kept = mine < ids.experts;
  if (blockIdx.y == 0 && lane == 0) {
    row_of_slot[s] = kept ? (int32_t)row : -1;
    slot_of_row[row] = kept ? (int32_t)s : -1;
  }
  if constexpr (kCopy) {
    uint8_t* dst = Xs + (int64_t)row * ldxs_bytes;
    if (row_elems < kPer) {
      if (lane == 0) RP::short_row(src, dst, kept, row_elems);
      return;
    }
#pragma unroll
    for (int i = 0; i < kSmallVecs; ++i) {
      const int64_t e = RP::start(e0 + (int64_t)i * 64 * kPer, row_elems);
      if (e >= 0 && e < row_elems) {
        typename RP::vec zero = {0, 0, 0, 0};
        *reinterpret_cast<typename RP::vec*>(dst + e * ES) = kept ? v[i] : zero;
      }
    }
  }
}

// ---- the sort of many slots ------------------------------------------------
// (The two launches with 64 to 256 slots a chunk, and the rows copied by the
// block that ranked them, measured slower from 12000 slots on: 65536 slots with
// rows of 8 KB 205 us against 131.)
// Two launches over chunks of the slots: every block counts its chunk's keys;
// then every block adds up the counts of the chunks before its own (and of
// all chunks, for the experts' first rows), and ranks its slots in order.
// In the ranking a wave takes 64 slots a step: the lanes that hold the same
// key find each other with one ballot per key bit, a lane's rank among them
// is the number of such lanes below it, and a counter per wave and key in LDS
// carries over to the next step.  Integer counts only: the same result
// whatever order the blocks run in.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

inline int64_t sort_chunk(int64_t S) {
  const int64_t rounds = ceil_div(S, (int64_t)kSortThreads * 256);
  return kSortThreads * (rounds < 32 ? rounds : 32);
}

__global__ __launch_bounds__(kSortThreads) void moe_count_kernel(Ids ids, uint32_t S, uint32_t chunk,
                                                                 int32_t* __restrict__ counts) {
  __shared__ int32_t n[kMaxExperts + 1];
  const int E1 = ids.experts + 1;
  for (int e = threadIdx.x; e < E1; e += kSortThreads) n[e] = 0;
  __syncthreads();
  const uint32_t s0 = blockIdx.x * chunk;
  for (uint32_t i = threadIdx.x; i < chunk && s0 + i < S; i += kSortThreads)
    atomicAdd(&n[slot_key(ids, s0 + i)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E1; e += kSortThreads) counts[(int64_t)blockIdx.x * E1 + e] = n[e];
}

// The lanes whose key is this lane's, among the live ones: a ballot a key bit.
__device__ __forceinline__ uint64_t same_key(bool live, int32_t key, int bits) {
  uint64_t same = __ballot(live);
  for (int b = 0; b < bits; ++b) {
    const uint64_t ones = __ballot((key >> b) & 1);
    same &= (key >> b) & 1 ? ones : ~ones;
  }
  return same;
}

// kSelf: every block counts all the slots itself (a
// launch less, but the count grows with the slots).  Alone, called in a row /
// replayed in a graph: 5000 slots of 256 experts 10.1 / 6.9 us, with the
// counting launch 13.5 / 7.9; 12000 of 64 experts 10.8 / 9.3 against 13.0 / 7.0.
constexpr int kSelfSlots = 8192;

template <bool kSelf>
__global__ __launch_bounds__(kSortThreads) void moe_place_kernel(
    Ids ids, uint32_t S, uint32_t chunk, const int32_t* __restrict__ counts,
    int32_t* __restrict__ offsets, int32_t* __restrict__ row_of_slot,
    int32_t* __restrict__ slot_of_row) {
  __shared__ int32_t at[kSortWaves][kMaxExperts + 1];
  __shared__ int32_t before[2 * kSortThreads];  // partial sums, then the scan
  __shared__ int32_t wave_sum[kSortWaves];
  const int E1 = ids.experts + 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t s0 = blockIdx.x * chunk;

  // What comes from memory first, all at once: the wave's first 64 keys, and the
  // counts of the chunks before this one and of all chunks -- E2 threads side by
  // side on the keys (a power of two >= E1), the rest of the threads on further
  // chunks.
  const uint32_t per_wave = chunk / kSortWaves;
  const uint32_t w0 = s0 + wave * per_wave;
  const int32_t key0 = w0 + lane < S ? slot_key(ids, w0 + lane) : 0;
  int E2 = 1;
  while (E2 < E1) E2 *= 2;
  const int parts = kSortThreads / E2;
  const int e = threadIdx.x & (E2 - 1), part = threadIdx.x / E2;
  const int bits = 32 - __builtin_clz((unsigned)ids.experts);  // keys 0 .. experts
  int32_t prev = 0, all = 0;
  if (!kSelf && e < E1) {
#pragma unroll 16
    for (uint32_t b = part; b < gridDim.x; b += parts) {
      const int32_t c = counts[(int64_t)b * E1 + e];
      all += c;
      prev += b < blockIdx.x ? c : 0;
    }
  }

  // own chunk: counts per wave and key
  for (int i = threadIdx.x; i < kSortWaves * E1; i += kSortThreads) at[i / E1][i % E1] = 0;
  __syncthreads();
  if (w0 + lane < S) atomicAdd(&at[wave][key0], 1);
  for (uint32_t i = 64 + lane; i < per_wave; i += 64)
    if (w0 + i < S) atomicAdd(&at[wave][slot_key(ids, w0 + i)], 1);
  if constexpr (kSelf) {
    // (chunks start at multiples of 64: a wave's slots are all before it or none)
    constexpr int kEach = kSelfSlots / kSortThreads;
    int32_t keys[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const uint32_t s = j * kSortThreads + threadIdx.x;
      keys[j] = s < S ? slot_key(ids, s) : -1;
    }
    before[threadIdx.x] = before[kSortThreads + threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const uint32_t i = j * kSortThreads + wave * 64;
      if (i >= S) break;
      const int32_t key = keys[j];
      const bool live = key >= 0;
      // few keys: one addition a key and wave, since lanes of one key queue up
      // (8000 slots of 2 experts 7.8 us, a lane each 12.6; of 14 experts 9.0 and
      // 7.8, unless most slots go to one; 5000 of 256 experts 9.8 and 6.9)
      if (bits <= 4) {
        const uint64_t same = same_key(live, key, bits);
        if (live && __builtin_ctzll(same) == lane) {
          atomicAdd(&before[kSortThreads + key], __popcll(same));
          if (i < s0) atomicAdd(&before[key], __popcll(same));
        }
      } else if (live) {
        atomicAdd(&before[kSortThreads + key], 1);
        if (i < s0) atomicAdd(&before[key], 1);
      }
    }
  } else {
    before[threadIdx.x] = prev;
    before[kSortThreads + threadIdx.x] = all;
  }
  __syncthreads();
  prev = all = 0;
  if (threadIdx.x < (unsigned)E1) {
    for (int p = 0; p < (kSelf ? 1 : parts); ++p) {
      prev += before[p * E2 + threadIdx.x];
      all += before[kSortThreads + p * E2 + threadIdx.x];
    }
  }
  // exclusive scan of `all` over the keys
  int32_t incl = all;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int32_t up = __shfl_up(incl, d);
    if (lane >= d) incl += up;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  int32_t first = incl - all;
  for (int w = 0; w < wave; ++w) first += wave_sum[w];
  if (threadIdx.x < (unsigned)E1) {
    if (blockIdx.x == 0) offsets[threadIdx.x] = first;
    int32_t run = first + prev;
    for (int w = 0; w < kSortWaves; ++w) {
      const int32_t c = at[w][threadIdx.x];
      at[w][threadIdx.x] = run;
      run += c;
    }
  }
  __syncthreads();

  // rank the slots in order
  volatile int32_t* mine = at[wave];
  for (uint32_t i = 0; i < per_wave; i += 64) {
    const uint32_t s = w0 + i + lane;
    const bool live = s < S;
    const int32_t key = i == 0 ? key0 : live ? slot_key(ids, s) : 0;
    const uint64_t same = same_key(live, key, bits);
    const int rank = __popcll(same & ((UINT64_C(1) << lane) - 1));
    int32_t row = 0;
    if (live) row = mine[key] + rank;
    // the first lane of each key moves the key's counter on; a wave's LDS
    // accesses complete in order, so every lane has read it before
    __builtin_amdgcn_wave_barrier();
    if (live && rank == 0) mine[key] = row + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (live) {
      const bool kept = key < ids.experts;
      row_of_slot[s] = kept ? row : -1;
      slot_of_row[row] = kept ? (int32_t)s : -1;
    }
  }
}

// Row copies of many slots: a wave per token and piece of the row; the piece
// is read once and stored to the token's top_k rows (604 MB in 117 us).  Rows
// without a slot are zeroed by the token whose slots have their numbers.
constexpr int kCopyVecs = 4;
template <int ES>
__global__ __launch_bounds__(256) void moe_copy_kernel(
    const uint8_t* __restrict__ X, int64_t ldx_bytes, int64_t row_elems, int64_t T, int32_t top_k,
    const int32_t* __restrict__ row_of_slot, const int32_t* __restrict__ slot_of_row,
    uint8_t* __restrict__ Xs, int64_t ldxs_bytes, int64_t first) {
  using RP = RowPiece<ES>;
  constexpr int kPer = RP::kPer;
  const int lane = threadIdx.x & 63;
  const int64_t t = first + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const int64_t e0 = ((int64_t)blockIdx.y * kCopyVecs * 64 + lane) * kPer;
  const uint8_t* src = X + t * ldx_bytes;
  typename RP::vec v[kCopyVecs];
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i) {
    const int64_t e = RP::start(e0 + (int64_t)i * 64 * kPer, row_elems);
    if (e >= 0 && e < row_elems) v[i] = *reinterpret_cast<const typename RP::vec*>(src + e * ES);
  }
  auto store = [&](int64_t row, bool kept) {
    uint8_t* dst = Xs + row * ldxs_bytes;
    if (row_elems < kPer) {
      if (lane == 0) RP::short_row(src, dst, kept, row_elems);
      return;
    }
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i) {
      const int64_t e = RP::start(e0 + (int64_t)i * 64 * kPer, row_elems);
      if (e >= 0 && e < row_elems) {
        typename RP::vec zero = {0, 0, 0, 0};
        *reinterpret_cast<typename RP::vec*>(dst + e * ES) = kept ? v[i] : zero;
      }
    }
  };
  for (int j = 0; j < top_k; ++j) {
    const int64_t s = t * top_k + j;
    const int32_t row = row_of_slot[s];
    if (row >= 0) store(row, true);
    if (slot_of_row[s] < 0) store(s, false);
  }
}

// ---- the way back ----------------------------------------------------------
// Y[t] = sum_j w[t,j] * Z[row(t,j)] (kWeighted) or without the weights: a
// thread per 16 bytes of a token's row, up to kRowsAhead rows in flight
// (604 MB in 120 us; the sum of a token's gradients, 4099 x 4 rows of 1101 f32,
// 90 MB in 15.7 us, part of it from the cache).
constexpr int kRowsAhead = 8;

template <typename T_, bool kWeighted>
__global__ __launch_bounds__(256) void moe_combine_kernel(
    const T_* __restrict__ Z, int64_t ldz, int64_t T, int32_t top_k, int64_t H,
    const int32_t* __restrict__ row_of_slot, const float* __restrict__ weights, int64_t ldw,
    T_* __restrict__ Y, int64_t ldy, uint32_t pieces, int64_t first) {
  constexpr int kPer = 16 / sizeof(T_);
  const int64_t i = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = i / pieces;
  if (t >= T) return;
  // a row's last piece ends with the row, over elements of the one before it
  int64_t h = (i - t * pieces) * kPer;
  if (h + kPer > H) h = H < kPer ? 0 : H - kPer;
  const int64_t S = T * top_k;
  const int n = H < kPer ? (int)H : kPer;
  float acc[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) acc[q] = 0.0f;
  for (int j0 = 0; j0 < top_k; j0 += kRowsAhead) {
    Piece<T_> v[kRowsAhead];
    float w[kRowsAhead];
    bool kept[kRowsAhead];
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      kept[j] = false;
      w[j] = 1.0f;
      if (j0 + j < top_k) {
        const int64_t row = row_of_slot[t * top_k + j0 + j];
        kept[j] = row >= 0 && row < S;
        if (kWeighted) w[j] = weights[t * ldw + j0 + j];
        if (kept[j]) v[j] = load_piece(Z + row * ldz + h, n);
      }
    }
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      if (!kept[j]) continue;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const float z = v[j].get(q);
        acc[q] = kWeighted ? __builtin_fmaf(w[j], z, acc[q]) : acc[q] + z;
      }
    }
  }
  store_piece(Y + t * ldy + h, acc, n);
}

// Both gradients of the combination: a workgroup per token.  Its dY row is
// read once per kRowsAhead slots; every Z row once; the dot products are
// summed in a fixed order (a thread's pieces, the wave's lanes, the waves).
// Rows of dZ that no slot has are zeroed by the token whose slots have the
// same numbers.  4096 tokens x 8, rows of 4096 bf16 (571 MB): 112 us, 5.1 TB/s.
template <typename T_>
__global__ __launch_bounds__(256) void moe_combine_grad_kernel(
    const T_* __restrict__ dY, int64_t lddy, const T_* __restrict__ Z, int64_t ldz, int64_t T,
    int32_t top_k, int64_t H, const int32_t* __restrict__ row_of_slot,
    const int32_t* __restrict__ slot_of_row, const float* __restrict__ weights, int64_t ldw,
    T_* __restrict__ dZ, int64_t lddz, float* __restrict__ dW, int64_t lddw, int64_t first) {
  constexpr int kPer = 16 / sizeof(T_);
  __shared__ float part[4][kRowsAhead];
  const int64_t t = first + blockIdx.x;
  const int64_t S = T * top_k;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T_* dy = dY + t * lddy;
  for (int j0 = 0; j0 < top_k; j0 += kRowsAhead) {
    int64_t row[kRowsAhead];
    float w[kRowsAhead], dot[kRowsAhead];
    bool bare[kRowsAhead];
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      row[j] = -1;
      dot[j] = 0.0f;
      w[j] = 0.0f;
      bare[j] = false;
      if (j0 + j < top_k) {
        const int64_t s = t * top_k + j0 + j;
        const int64_t r = row_of_slot[s];
        row[j] = r < S ? r : -1;
        w[j] = weights[t * ldw + j0 + j];
        const int64_t slot = slot_of_row[s];
        bare[j] = slot < 0 || slot >= S;
      }
    }
    for (int64_t h0 = (int64_t)threadIdx.x * kPer; h0 < H; h0 += 256 * kPer) {
      // a row's last piece ends with the row: its first `again` elements are the
      // piece before's too, and count once in the dot products
      const int64_t h = h0 + kPer <= H ? h0 : H < kPer ? 0 : H - kPer;
      const int again = (int)(h0 - h);
      const int n = H < kPer ? (int)H : kPer;
      Piece<T_> z[kRowsAhead];
      const Piece<T_> g = load_piece(dy + h, n);
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j)
        if (row[j] >= 0) z[j] = load_piece(Z + row[j] * ldz + h, n);
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j) {
        if (row[j] >= 0) {
          float out[kPer];
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            const float gq = g.get(q);
            out[q] = w[j] * gq;
            const float d = __builtin_fmaf(gq, z[j].get(q), dot[j]);
            dot[j] = q < again ? dot[j] : d;
          }
          store_piece(dZ + row[j] * lddz + h, out, n);
        }
        if (bare[j]) {
          float out[kPer];
#pragma unroll
          for (int q = 0; q < kPer; ++q) out[q] = 0.0f;
          store_piece(dZ + (t * top_k + j0 + j) * lddz + h, out, n);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
#pragma unroll
      for (int d = 32; d > 0; d /= 2) dot[j] += __shfl_xor(dot[j], d);
      if (lane == 0) part[wave][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < kRowsAhead && j0 + (int)threadIdx.x < top_k) {
      const int j = threadIdx.x;
      const int64_t r = row_of_slot[t * top_k + j0 + j];
      const float sum = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
      dW[t * lddw + j0 + j] = r >= 0 && r < S ? sum : 0.0f;
    }
    __syncthreads();
  }
}

// ---- host side -------------------------------------------------------------
qp_status check_route(const char* what, int64_t T, int64_t top_k) {
  QP_REQUIRE(T >= 0 && top_k >= 1, QP_EINVAL, "%s: needs T >= 0 and top_k >= 1 (got %lld, %lld)",
             what, (long long)T, (long long)top_k);
  QP_REQUIRE(top_k <= 1024 && T <= kMaxSlots / top_k, QP_EUNSUPPORTED,
             "%s: top_k above 1024 or more than 2^30 slots (T=%lld, top_k=%lld)", what,
             (long long)T, (long long)top_k);
  return QP_OK;
}

qp_status check_ids(const char* what, int32_t ids_dtype, int64_t T, int64_t top_k, int64_t ldids,
                    int64_t experts) {
  qp_status st = check_route(what, T, top_k);
  if (st) return st;
  QP_REQUIRE(ids_dtype == QP_S32 || ids_dtype == QP_S64, QP_EINVAL,
             "%s: ids must be QP_S32 or QP_S64 (got %d)", what, ids_dtype);
  QP_REQUIRE(ldids >= top_k, QP_EINVAL, "%s: ldids %lld < top_k", what, (long long)ldids);
  QP_REQUIRE(experts >= 1, QP_EINVAL, "%s: needs at least one expert", what);
  QP_REQUIRE(experts <= kMaxExperts, QP_EUNSUPPORTED, "%s: at most %d experts (got %lld)", what,
             kMaxExperts, (long long)experts);
  return QP_OK;
}

qp_status check_float(const char* what, int32_t dtype) {
  QP_REQUIRE(dtype == QP_F32 || dtype == QP_BF16 || dtype == QP_F16, QP_EINVAL,
             "%s: rows must be QP_F32, QP_BF16 or QP_F16 (got %d)", what, dtype);
  return QP_OK;
}

qp_status check_rows(const char* what, const char* name, const void* p, int64_t ld, int64_t H,
                     int32_t dtype) {
  QP_REQUIRE(H >= 1 && ld >= H, QP_EINVAL, "%s: %s needs a row length >= 1 and a stride >= it", what,
             name);
  QP_REQUIRE(H <= (INT64_C(1) << 24), QP_EUNSUPPORTED, "%s: rows above 2^24 elements", what);
  QP_REQUIRE(p != nullptr, QP_EINVAL, "%s: %s is null", what, name);
  QP_REQUIRE((uintptr_t)p % elem_bytes(dtype) == 0, QP_EALIGN,
             "%s: %s is not aligned to its elements", what, name);
  return QP_OK;
}

size_t sort_ws_bytes(int64_t S, int64_t experts) {
  if (S <= kSelfSlots) return 0;
  const int64_t nb = ceil_div(S, sort_chunk(S));
  return (size_t)round_up(nb * (experts + 1) * 4, 256);
}

template <int ES, bool kCopy, int kSmallThreads>
qp_status launch_small_of(const Ids& ids, int64_t S, const void* X, int64_t ldx, int64_t H, void* Xs,
                       int64_t ldxs, int32_t* offsets, int32_t* row_of_slot, int32_t* slot_of_row,
                       hipStream_t stream) {
  const int64_t slot_blocks = ceil_div(S, kSmallThreads / 64);
  const int64_t ofs_blocks = ceil_div(ids.experts + 1, kSmallThreads);
  const int64_t parts = kCopy ? ceil_div(H * ES, kSmallVecs * 64 * 16) : 1;
  hipLaunchKernelGGL((moe_small_kernel<ES, kCopy, kSmallThreads>),
                     dim3((unsigned)(slot_blocks + ofs_blocks), (unsigned)parts),
                     dim3(kSmallThreads), 0, stream, ids, (uint32_t)S, (uint32_t)slot_blocks,
                     static_cast<const uint8_t*>(X), ldx * ES, H, static_cast<uint8_t*>(Xs),
                     ldxs * ES, offsets, row_of_slot, slot_of_row);
  return check_launch("qmoe sort (few slots)");
}

// Up to 64 slots every wave reads the ids itself; above, the waves of a large
// workgroup share them in LDS.
template <int ES, bool kCopy>
qp_status launch_small(const Ids& ids, int64_t S, const void* X, int64_t ldx, int64_t H, void* Xs,
                       int64_t ldxs, int32_t* offsets, int32_t* row_of_slot, int32_t* slot_of_row,
                       hipStream_t stream) {
  return S <= 64 ? launch_small_of<ES, kCopy, 256>(ids, S, X, ldx, H, Xs, ldxs, offsets,
                                                   row_of_slot, slot_of_row, stream)
                 : launch_small_of<ES, kCopy, 1024>(ids, S, X, ldx, H, Xs, ldxs, offsets,
                                                    row_of_slot, slot_of_row, stream);
}

// X null: the sort alone.
qp_status run_sort(const Ids& ids, int64_t T, const void* X, int32_t dtype, int64_t H, int64_t ldx,
                   void* Xs, int64_t ldxs, int32_t* offsets, int32_t* row_of_slot,
                   int32_t* slot_of_row, void* ws, hipStream_t stream) {
  const int64_t S = T * ids.top_k;
  const int es = X ? elem_bytes(dtype) : 4;
  if (S <= (X ? kSmallSlots : kSmallSort)) {
    if (!X)
      return launch_small<4, false>(ids, S, X, 0, 0, Xs, 0, offsets, row_of_slot, slot_of_row,
                                    stream);
    return es == 2 ? launch_small<2, true>(ids, S, X, ldx, H, Xs, ldxs, offsets, row_of_slot,
                                           slot_of_row, stream)
                   : launch_small<4, true>(ids, S, X, ldx, H, Xs, ldxs, offsets, row_of_slot,
                                           slot_of_row, stream);
  }
  const int64_t chunk = sort_chunk(S), nb = ceil_div(S, chunk);
  int32_t* counts = static_cast<int32_t*>(ws);
  qp_status st;
  if (S <= kSelfSlots) {
    hipLaunchKernelGGL((moe_place_kernel<true>), dim3((unsigned)nb), dim3(kSortThreads), 0, stream,
                       ids, (uint32_t)S, (uint32_t)chunk, (const int32_t*)nullptr, offsets,
                       row_of_slot, slot_of_row);
  } else {
    hipLaunchKernelGGL(moe_count_kernel, dim3((unsigned)nb), dim3(kSortThreads), 0, stream, ids,
                       (uint32_t)S, (uint32_t)chunk, counts);
    if ((st = check_launch("qmoe sort (counts)"))) return st;
    hipLaunchKernelGGL((moe_place_kernel<false>), dim3((unsigned)nb), dim3(kSortThreads), 0, stream,
                       ids, (uint32_t)S, (uint32_t)chunk, (const int32_t*)counts, offsets,
                       row_of_slot, slot_of_row);
  }
  st = check_launch("qmoe sort (rows)");
  if (st || !X) return st;
  const int64_t parts = ceil_div(H * es, kCopyVecs * 64 * 16);
  for (int64_t t = 0; t < T; t += 4 * kMaxBlocks) {
    const dim3 grid((unsigned)ceil_div(T - t < 4 * kMaxBlocks ? T - t : 4 * kMaxBlocks, 4),
                    (unsigned)parts);
    if (es == 2)
      hipLaunchKernelGGL((moe_copy_kernel<2>), grid, dim3(256), 0, stream,
                         static_cast<const uint8_t*>(X), ldx * 2, H, T, ids.top_k,
                         (const int32_t*)row_of_slot, (const int32_t*)slot_of_row,
                         static_cast<uint8_t*>(Xs), ldxs * 2, t);
    else
      hipLaunchKernelGGL((moe_copy_kernel<4>), grid, dim3(256), 0, stream,
                         static_cast<const uint8_t*>(X), ldx * 4, H, T, ids.top_k,
                         (const int32_t*)row_of_slot, (const int32_t*)slot_of_row,
                         static_cast<uint8_t*>(Xs), ldxs * 4, t);
  }
  return check_launch("qmoe dispatch (copy)");
}

qp_status sort_entry(const char* what, const void* X, int32_t dtype, int64_t H, int64_t ldx,
                     const void* ids, int32_t ids_dtype, int64_t T, int64_t top_k, int64_t ldids,
                     int64_t experts, void* Xs, int64_t ldxs, int32_t* offsets,
                     int32_t* row_of_slot, int32_t* slot_of_row, void* ws, size_t ws_bytes,
                     hipStream_t stream) {
  qp_status st = check_ids(what, ids_dtype, T, top_k, ldids, experts);
  if (st) return st;
  const int64_t S = T * top_k;
  QP_REQUIRE(offsets && (S == 0 || (ids && row_of_slot && slot_of_row)), QP_EINVAL,
             "%s: null pointer", what);
  QP_REQUIRE((uintptr_t)ids % (ids_dtype == QP_S64 ? 8 : 4) == 0, QP_EALIGN,
             "%s: ids are not aligned to their elements", what);
  const size_t need = sort_ws_bytes(S, experts);
  QP_REQUIRE(ws_bytes >= need, QP_ESIZE, "%s: workspace holds %zu bytes, needs %zu", what, ws_bytes,
             need);
  QP_REQUIRE(need == 0 || (ws && (uintptr_t)ws % 256 == 0), QP_EALIGN,
             "%s: workspace must be non-null and 256-byte aligned", what);
  Ids d{ids, ldids, (int32_t)top_k, (int32_t)experts, ids_dtype == QP_S64};
  return run_sort(d, T, X, dtype, H, ldx, Xs, ldxs, offsets, row_of_slot, slot_of_row, ws, stream);
}

template <typename T_, bool kWeighted>
qp_status launch_combine(const void* Z, int64_t ldz, int64_t T, int64_t top_k, int64_t H,
                         const int32_t* row_of_slot, const float* weights, int64_t ldw, void* Y,
                         int64_t ldy, hipStream_t stream) {
  const int64_t pieces = ceil_div(H * (int64_t)sizeof(T_), 16);
  const int64_t blocks = ceil_div(T * pieces, 256);
  for (int64_t b = 0; b < blocks; b += kMaxBlocks) {
    const int64_t n = blocks - b < kMaxBlocks ? blocks - b : kMaxBlocks;
    hipLaunchKernelGGL((moe_combine_kernel<T_, kWeighted>), dim3((unsigned)n), dim3(256), 0, stream,
                       static_cast<const T_*>(Z), ldz, T, (int32_t)top_k, H, row_of_slot, weights,
                       ldw, static_cast<T_*>(Y), ldy, (uint32_t)pieces, b * 256);
  }
  return check_launch("qmoe combine");
}

template <bool kWeighted>
qp_status combine_any(int32_t dtype, const void* Z, int64_t ldz, int64_t T, int64_t top_k,
                      int64_t H, const int32_t* row_of_slot, const float* weights, int64_t ldw,
                      void* Y, int64_t ldy, hipStream_t stream) {
  if (dtype == QP_F32)
    return launch_combine<float, kWeighted>(Z, ldz, T, top_k, H, row_of_slot, weights, ldw, Y, ldy,
                                            stream);
  if (dtype == QP_BF16)
    return launch_combine<bf16_t, kWeighted>(Z, ldz, T, top_k, H, row_of_slot, weights, ldw, Y, ldy,
                                             stream);
  return launch_combine<f16_t, kWeighted>(Z, ldz, T, top_k, H, row_of_slot, weights, ldw, Y, ldy,
                                          stream);
}

template <typename T_>
qp_status launch_combine_grad(const void* dY, int64_t lddy, const void* Z, int64_t ldz, int64_t T,
                              int64_t top_k, int64_t H, const int32_t* row_of_slot,
                              const int32_t* slot_of_row, const float* weights, int64_t ldw,
                              void* dZ, int64_t lddz, float* dW, int64_t lddw, hipStream_t stream) {
  for (int64_t t = 0; t < T; t += kMaxBlocks) {
    const int64_t n = T - t < kMaxBlocks ? T - t : kMaxBlocks;
    hipLaunchKernelGGL((moe_combine_grad_kernel<T_>), dim3((unsigned)n), dim3(256), 0, stream,
                       static_cast<const T_*>(dY), lddy, static_cast<const T_*>(Z), ldz, T,
                       (int32_t)top_k, H, row_of_slot, slot_of_row, weights, ldw,
                       static_cast<T_*>(dZ), lddz, dW, lddw, t);
  }
  return check_launch("qmoe combine gradient");
}

}  // namespace
}  // namespace qp

extern "C" qp_status qmoe_sort_ws_size(int64_t T, int64_t top_k, int64_t experts, size_t* bytes) {
  using namespace qp;
  clear_error();
  QP_REQUIRE(bytes, QP_EINVAL, "qmoe_sort_ws_size: null argument");
  qp_status st = check_ids("qmoe_sort_ws_size", QP_S32, T, top_k, top_k, experts);
  if (st) return st;
  *bytes = sort_ws_bytes(T * top_k, experts);
  return QP_OK;
}

extern "C" qp_status qmoe_sort(const void* ids, int32_t ids_dtype, int64_t T, int64_t top_k,
                               int64_t ldids, int64_t experts, int32_t* offsets,
                               int32_t* row_of_slot, int32_t* slot_of_row, void* ws,
                               size_t ws_bytes, hipStream_t stream) {
  using namespace qp;
  clear_error();
  return sort_entry("qmoe_sort", nullptr, QP_F32, 0, 0, ids, ids_dtype, T, top_k, ldids, experts,
                    nullptr, 0, offsets, row_of_slot, slot_of_row, ws, ws_bytes, stream);
}

extern "C" qp_status qmoe_dispatch(const void* X, int32_t dtype, int64_t H, int64_t ldx,
                                   const void* ids, int32_t ids_dtype, int64_t T, int64_t top_k,
                                   int64_t ldids, int64_t experts, void* Xs, int64_t ldxs,
                                   int32_t* offsets, int32_t* row_of_slot, int32_t* slot_of_row,
                                   void* ws, size_t ws_bytes, hipStream_t stream) {
  using namespace qp;
  clear_error();
  qp_status st = check_float("qmoe_dispatch", dtype);
  if (!st && T != 0) {
    st = check_rows("qmoe_dispatch", "X", X, ldx, H, dtype);
    if (!st) st = check_rows("qmoe_dispatch", "Xs", Xs, ldxs, H, dtype);
  }
  if (st) return st;
  return sort_entry("qmoe_dispatch", T == 0 ? nullptr : X, dtype, H, ldx, ids, ids_dtype, T, top_k,
                    ldids, experts, Xs, ldxs, offsets, row_of_slot, slot_of_row, ws, ws_bytes,
                    stream);
}

extern "C" qp_status qmoe_dispatch_grad(const void* dXs, int32_t dtype, int64_t T, int64_t top_k,
                                        int64_t H, int64_t lddxs, const int32_t* row_of_slot,
                                        void* dX, int64_t lddx, hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qmoe_dispatch_grad";
  qp_status st = check_float(what, dtype);
  if (!st) st = check_route(what, T, top_k);
  if (st || T == 0) return st;
  if ((st = check_rows(what, "dXs", dXs, lddxs, H, dtype))) return st;
  if ((st = check_rows(what, "dX", dX, lddx, H, dtype))) return st;
  QP_REQUIRE(row_of_slot, QP_EINVAL, "%s: null pointer", what);
  return combine_any<false>(dtype, dXs, lddxs, T, top_k, H, row_of_slot, nullptr, 0, dX, lddx,
                            stream);
}

extern "C" qp_status qmoe_combine(const void* Z, int32_t dtype, int64_t T, int64_t top_k,
                                  int64_t H, int64_t ldz, const int32_t* row_of_slot,
                                  const float* weights, int64_t ldw, void* Y, int64_t ldy,
                                  hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qmoe_combine";
  qp_status st = check_float(what, dtype);
  if (!st) st = check_route(what, T, top_k);
  if (st || T == 0) return st;
  if ((st = check_rows(what, "Z", Z, ldz, H, dtype))) return st;
  if ((st = check_rows(what, "Y", Y, ldy, H, dtype))) return st;
  QP_REQUIRE(row_of_slot && weights, QP_EINVAL, "%s: null pointer", what);
  QP_REQUIRE(ldw >= top_k, QP_EINVAL, "%s: the weights' stride is below top_k", what);
  return combine_any<true>(dtype, Z, ldz, T, top_k, H, row_of_slot, weights, ldw, Y, ldy, stream);
}

extern "C" qp_status qmoe_combine_grad(const void* dY, int64_t lddy, const void* Z, int64_t ldz,
                                       int32_t dtype, int64_t T, int64_t top_k, int64_t H,
                                       const int32_t* row_of_slot, const int32_t* slot_of_row,
                                       const float* weights, int64_t ldw, void* dZ, int64_t lddz,
                                       float* dweights, int64_t lddw, hipStream_t stream) {
  using namespace qp;
  clear_error();
  const char* what = "qmoe_combine_grad";
  qp_status st = check_float(what, dtype);
  if (!st) st = check_route(what, T, top_k);
  if (st || T == 0) return st;
  if ((st = check_rows(what, "dY", dY, lddy, H, dtype))) return st;
  if ((st = check_rows(what, "Z", Z, ldz, H, dtype))) return st;
  if ((st = check_rows(what, "dZ", dZ, lddz, H, dtype))) return st;
  QP_REQUIRE(row_of_slot && slot_of_row && weights && dweights, QP_EINVAL, "%s: null pointer", what);
  QP_REQUIRE(ldw >= top_k && lddw >= top_k, QP_EINVAL,
             "%s: the weights' or their gradient's stride is below top_k", what);
  if (dtype == QP_F32)
    return launch_combine_grad<float>(dY, lddy, Z, ldz, T, top_k, H, row_of_slot, slot_of_row,
                                      weights, ldw, dZ, lddz, dweights, lddw, stream);
  if (dtype == QP_BF16)
    return launch_combine_grad<bf16_t>(dY, lddy, Z, ldz, T, top_k, H, row_of_slot, slot_of_row,
                                       weights, ldw, dZ, lddz, dweights, lddw, stream);
  return launch_combine_grad<f16_t>(dY, lddy, Z, ldz, T, top_k, H, row_of_slot, slot_of_row,
                                    weights, ldw, dZ, lddz, dweights, lddw, stream);
}
