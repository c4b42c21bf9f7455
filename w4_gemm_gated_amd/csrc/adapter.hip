// Low-rank adapters of many requests at once, added beside a shared projection:
//
//   Y[m] += s_a (X[m] . A_a^T) . B_a^T      a = the adapter of row m's sequence
//
// Three kernels.  The plan, made once for a step and used by all of its
// projections, sorts the batch's rows by adapter and cuts each adapter's into tiles
// of at most 64.  The first product (adapter_shrink_kernel) takes tiles x slices
// of K, the last slice of a tile to arrive adds them in order; the second
// (adapter_expand_kernel) takes tiles x columns and updates Y in place.  With one
// token a request both are a chain of round trips over the adapters in use (each
// read once, whatever the order of the requests); with a prompt's chunk the
// second is bound by Y, read and written.
//
// Matrix operands need no staging: A [rank][K] and B [N][rank] are contiguous along
// the summed index, so a lane's eight values are one 16-byte load from memory, as
// X's are.  The products are formed transposed (tokens are the columns of the result): a
// lane then holds four neighbouring ranks, or sixteen neighbouring columns of Y, of
// one token.
//
// H = X . A^T is held in fp32 and enters the second product as two fp16 numbers whose
// sum is H to 2^-22 of the row's largest (scaled by a power of two before): rounding
// it once to fp16 would cost 2^-12 of the adapter's term, and the second product's
// matrix work is small beside its memory traffic.
#include <algorithm>

#include "serve_internal.h"
#include "device_common.h"

namespace spear {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kShrinkThreads = 512, kShrinkWaves = kShrinkThreads / kWave;
constexpr int kPlanThreads = 1024;
constexpr int kPlanHead = 8;      // words: tiles
constexpr int kUnit = kAdapterColumns / kWaves;   // columns of Y that a wave computes
typedef float f4_t __attribute__((ext_vector_type(4)));

// The plan: head, tiles {adapter, first entry of the list, rows, 0}, list of rows.
__device__ __forceinline__ const int4* plan_tiles(const int32_t* plan) { return (const int4*)(plan + kPlanHead); }

// ------------------------------------------------------------------ the plan

__device__ __forceinline__ int64_t sum_before(int64_t v, int64_t* waves, int64_t* total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  int64_t run = v;
#pragma unroll
  for (int o = 1; o < kWave; o *= 2) {
    const int64_t x = __shfl_up(run, o);
    if (lane >= o) run += x;
  }
  __syncthreads();
  if (lane == kWave - 1) waves[wave] = run;
  __syncthreads();
  int64_t before = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / kWave; ++i) {
    if (i < wave) before += waves[i];
    sum += waves[i];
  }
  *total = sum;
  return before + run - v;
}

// One workgroup: rows per adapter, their running sums, then every sequence takes
// its place among its adapter's rows.  (Which place it gets is a matter of order
// of arrival; a row's result does not depend on it.)  Offsets that do not rise
// within the rows give a plan of no tiles.
__global__ void __launch_bounds__(kPlanThreads) adapter_plan_kernel(AdapterPlanArgs a) {
  __shared__ int32_t count[kMaxAdapters];      // rows, then the next free entry of the list
  __shared__ int32_t tile_to[kMaxAdapters];    // running sum of tiles
  __shared__ int32_t list_at[kMaxAdapters];
  __shared__ int64_t waves[kPlanThreads / kWave];
  __shared__ int32_t first_of[kPlanThreads], rows_of[kPlanThreads], place_of[kPlanThreads];
  __shared__ int32_t bad, longs;
  const int tid = threadIdx.x;
  for (int i = tid; i < a.adapters; i += kPlanThreads) count[i] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  for (int b = tid; b < a.batch; b += kPlanThreads) {
    const int32_t from = a.cu[b], to = a.cu[b + 1], of = a.adapter[b];
    if (from < 0 || to < from || to > a.rows) bad = 1;
    else if (of >= 0 && of < a.adapters && to > from) atomicAdd(&count[of], to - from);
  }
  __syncthreads();
  int32_t* list = a.plan + kPlanHead + 4 * (int64_t)a.most_tiles;
  if (bad) {
    if (tid == 0) a.plan[0] = 0;
    return;
  }
  int64_t rows_before = 0, tiles_before = 0, sum;
  for (int i0 = 0; i0 < a.adapters; i0 += kPlanThreads) {
    const int i = i0 + tid;
    const int32_t n = i < a.adapters ? count[i] : 0, tiles = (n + kAdapterTile - 1) / kAdapterTile;
    const int64_t at = rows_before + sum_before(n, waves, &sum);
    rows_before += sum;
    const int64_t t = tiles_before + sum_before(tiles, waves, &sum);
    tiles_before += sum;
    if (i < a.adapters) {
      tile_to[i] = (int32_t)(t + tiles);
      list_at[i] = (int32_t)at;
    }
  }
  __syncthreads();
  const int tiles = (int)min(tiles_before, (int64_t)a.most_tiles);
  if (tid == 0) a.plan[0] = tiles;
  for (int t = tid; t < tiles; t += kPlanThreads) {
    int lo = 0, hi = a.adapters - 1;           // the first adapter whose tiles reach past t
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (tile_to[mid] > t) hi = mid;
      else lo = mid + 1;
    }
    const int in = (t - (lo > 0 ? tile_to[lo - 1] : 0)) * kAdapterTile;
    ((int4*)(a.plan + kPlanHead))[t] = make_int4(lo, list_at[lo] + in, min(count[lo] - in, kAdapterTile), 0);
  }
  __syncthreads();
  for (int i = tid; i < a.adapters; i += kPlanThreads) count[i] = list_at[i];
  __syncthreads();
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int32_t from = 0, n = 0, at = 0;
    if (b < a.batch) {
      const int32_t of = a.adapter[b];
      from = a.cu[b];
      n = of >= 0 && of < a.adapters ? a.cu[b + 1] - from : 0;
      if (n > 0) at = atomicAdd(&count[of], n);
    }
    // Short sequences are written by their thread, long ones by all.
    constexpr int kShort = 16;
    if (n <= kShort)
      for (int i = 0; i < n; ++i) list[at + i] = from + i;
    if (tid == 0) longs = 0;
    __syncthreads();
    if (n > kShort) {
      const int s = atomicAdd(&longs, 1);
      first_of[s] = from;
      rows_of[s] = n;
      place_of[s] = at;
    }
    __syncthreads();
    const int many = longs;
    for (int s = tid / kWave; s < many; s += kPlanThreads / kWave)       // a wave to each
      for (int i = tid % kWave; i < rows_of[s]; i += kWave) list[place_of[s] + i] = first_of[s] + i;
    __syncthreads();
  }
}

// ------------------------------------------------------------- first product

__device__ __forceinline__ void store_f4_dev(__amdgpu_buffer_rsrc_t r, uint32_t byte_offset, const f4_t& v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), r, byte_offset, 0, kCachePolicySc1);
}

struct Tile {
  int adapter, first, rows;
};

// Ranks [rank0, rank0 + 16 RB) of one slice of K for a tile of up to 16 SUB rows: the
// waves take 64 k in turn (whole lines of X and A), and add their sums through LDS.
template <int RB, int SUB>
__device__ __forceinline__ void shrink(const AdapterArgs& a, const Tile& t, const int32_t* list, int rank0, int k_lo,
                                       int k_hi, f4_t* red, __amdgpu_buffer_rsrc_t part) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, c = lane % 16, oct = lane / 16;
  const half_t* x[SUB];
  const half_t* w[RB];
#pragma unroll
  for (int j = 0; j < SUB; ++j) {
    const int32_t row = list[t.first + min(16 * j + c, t.rows - 1)];
    x[j] = (const half_t*)a.X + (int64_t)min(max(row, 0), a.rows - 1) * a.x_stride + 8 * oct;
  }
#pragma unroll
  for (int i = 0; i < RB; ++i)      // (a rank past the last computes the last again, and is not kept)
    w[i] = (const half_t*)a.A + ((int64_t)t.adapter * a.rank + min(rank0 + 16 * i + c, a.rank - 1)) * a.K + 8 * oct;
  f4_t acc[SUB][RB];
#pragma unroll
  for (int j = 0; j < SUB; ++j)
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[j][i] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int kTurn = 64 * kShrinkWaves;
  constexpr int kAhead = SUB * RB >= 8 ? 1 : 2;    // turns whose loads are in flight together
  int k = k_lo + 64 * wave;
  for (; k + (kAhead - 1) * kTurn + 64 <= k_hi; k += kAhead * kTurn) {
    half8_t xv[2 * kAhead][SUB], wv[2 * kAhead][RB];
#pragma unroll
    for (int n = 0; n < 2 * kAhead; ++n) {
      const int at = k + n / 2 * kTurn + n % 2 * 32;
#pragma unroll
      for (int i = 0; i < RB; ++i) wv[n][i] = load_half8(w[i] + at);
#pragma unroll
      for (int j = 0; j < SUB; ++j) xv[n][j] = load_half8(x[j] + at);
    }
#pragma unroll
    for (int n = 0; n < 2 * kAhead; ++n)
#pragma unroll
      for (int j = 0; j < SUB; ++j)
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[j][i] = mfma16x16x32(wv[n][i], xv[n][j], acc[j][i]);
  }
#pragma unroll 1
  for (; k < k_hi; k += kTurn)
#pragma unroll 1
    for (int at = k; at < min(k + 64, k_hi); at += 32) {
      const bool in = at + 8 * oct < k_hi;            // (K and the slices are multiples of 8)
      const int from = in ? at : k_hi - 8 - 8 * oct;
      half8_t xv[SUB], wv[RB];
#pragma unroll
      for (int i = 0; i < RB; ++i) wv[i] = load_half8(w[i] + from);
#pragma unroll
      for (int j = 0; j < SUB; ++j) xv[j] = load_half8(x[j] + from);
#pragma unroll
      for (int i = 0; i < RB; ++i) wv[i] = in ? wv[i] : zero_half8();
#pragma unroll
      for (int j = 0; j < SUB; ++j) xv[j] = in ? xv[j] : zero_half8();
#pragma unroll
      for (int j = 0; j < SUB; ++j)
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[j][i] = mfma16x16x32(wv[i], xv[j], acc[j][i]);
    }
  // The upper four waves' sums to the lower four, theirs to all.
  constexpr int kHalf = kShrinkWaves / 2, kUnits = SUB * RB;
#pragma unroll
  for (int turn = 0; turn < 2; ++turn) {
    __syncthreads();
    if (turn == 0 ? wave >= kHalf : wave < kHalf)
#pragma unroll
      for (int u = 0; u < kUnits; ++u) red[((wave % kHalf) * kUnits + u) * kWave + lane] = acc[u / RB][u % RB];
    __syncthreads();
    if (turn == 0 && wave < kHalf)
#pragma unroll
      for (int u = 0; u < kUnits; ++u) acc[u / RB][u % RB] += red[(wave * kUnits + u) * kWave + lane];
  }
  for (int u = wave; u < kUnits; u += kShrinkWaves) {
    f4_t sum = red[u * kWave + lane];
#pragma unroll
    for (int v = 1; v < kHalf; ++v) sum += red[(v * kUnits + u) * kWave + lane];
    const int row = 16 * (u / RB) + c, rank = rank0 + 16 * (u % RB) + 4 * oct;
    if (row < t.rows && rank < a.rank) store_f4_dev(part, 4u * (uint32_t)(row * a.rank + rank), sum);
  }
}

template <int RB>
__global__ void __launch_bounds__(kShrinkThreads) adapter_shrink_kernel(AdapterArgs a) {
  extern __shared__ f4_t lds[];
  __shared__ float factor[kAdapterTile];
  __shared__ uint32_t arrived;
  const int tile = blockIdx.x / a.slices, slice = blockIdx.x % a.slices, tid = threadIdx.x;
  if (tile >= min(a.plan[0], a.most_tiles)) return;
  const int4 q = plan_tiles(a.plan)[tile];
  const Tile t = {min(max(q.x, 0), a.adapters - 1), min(max(q.y, 0), a.rows - 1), min(max(q.z, 1), kAdapterTile)};
  const int32_t* list = a.plan + kPlanHead + 4 * (int64_t)a.most_tiles;
  const size_t tile_bytes = (size_t)kAdapterTile * a.rank * 4;
  char* parts = a.part + (size_t)tile * a.slices * tile_bytes;
  const __amdgpu_buffer_rsrc_t part = make_rsrc(parts + slice * tile_bytes, (uint32_t)tile_bytes);
  const int k_lo = slice * a.slice_k, k_hi = min(k_lo + a.slice_k, a.K);
  for (int rank0 = 0; rank0 < a.rank; rank0 += 16 * RB) {
    if (t.rows <= 16) shrink<RB, 1>(a, t, list, rank0, k_lo, k_hi, lds, part);
    else shrink<RB, 4>(a, t, list, rank0, k_lo, k_hi, lds, part);
  }
  drain_vm();
  __syncthreads();
  if (a.slices > 1) {
    if (tid == 0) arrived = add_dev_u32(&a.counters[tile], 1u);
    __syncthreads();
    if (arrived != (uint32_t)a.slices - 1) return;
    if (tid == 0) st_dev_u32(&a.counters[tile], 0u);
  }
  // The slices in order; then every row as two fp16 numbers per value.
  float* h = (float*)lds;
  const __amdgpu_buffer_rsrc_t all = make_rsrc(parts, (uint32_t)(tile_bytes * a.slices));
  const int quads = a.rank / 4;
  // (two values of a thread and eight slices in flight together; loads past either end are
  // out of the buffer and give zeros)
  for (int u0 = tid; u0 < t.rows * quads; u0 += 2 * kShrinkThreads) {
    f4_t sum[2] = {};
    for (int s0 = 0; s0 < a.slices; s0 += 8) {
      f4_t v[8][2];
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int u = u0 + i * kShrinkThreads;
          v[n][i] = buffer_load_f4_dev(all, s0 + n < a.slices && u < t.rows * quads
                                                ? (uint32_t)((s0 + n) * tile_bytes) + 16u * u : kOutOfRange);
        }
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) sum[i] += v[n][i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (u0 + i * kShrinkThreads < t.rows * quads) *(f4_t*)(h + 4 * (u0 + i * kShrinkThreads)) = sum[i];
  }
  __syncthreads();
  {
    constexpr int kLanes = kShrinkThreads / kAdapterTile;     // lanes to a row
    const int row = tid / kLanes;
    float most = 0.0f;
    if (row < t.rows)
      for (int i = tid % kLanes; i < a.rank; i += kLanes) {
        const float v = fabsf(h[row * a.rank + i]);
        most = v > most || v != v ? v : most;
      }
#pragma unroll
    for (int o = 1; o < kLanes; o *= 2) {
      const float v = __shfl_xor(most, o);
      most = v > most || v != v ? v : most;
    }
    // The power of two at or below the row's largest (1 where that is zero, infinite or NaN).
    const uint32_t e = float_bits(most) >> 23;
    const float p = e == 0 ? (most > 0.0f ? 0x1p-126f : 1.0f) : e == 255 ? 1.0f : bits_float(e << 23);
    if (tid % kLanes == 0 && row < t.rows) {
      factor[row] = p;
      a.factor[(int64_t)tile * kAdapterTile + row] = p * (a.scale ? a.scale[t.adapter] : 1.0f);
    }
  }
  __syncthreads();
  const int octets = a.rank_pad / 8;
  half_t* out = (half_t*)a.H + (int64_t)tile * kAdapterTile * 2 * a.rank_pad;
  for (int u = tid; u < t.rows * octets; u += kShrinkThreads) {
    const int row = u / octets, o = u % octets;
    half8_t hi = zero_half8(), lo = zero_half8();
    if (8 * o < a.rank) {
      const float inv = 1.0f / factor[row];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        float v = h[row * a.rank + 8 * o + n] * inv;
        if (fabsf(v) > 65504.0f && fabsf(v) < INFINITY) v = copysignf(65504.0f, v);   // (beside an infinity or NaN)
        hi[n] = (half_t)v;
        lo[n] = fabsf(v) < INFINITY ? (half_t)(v - (float)hi[n]) : (half_t)0.0f;
      }
    }
    *(half8_t*)(out + (int64_t)row * 2 * a.rank_pad + 8 * o) = hi;
    *(half8_t*)(out + (int64_t)row * 2 * a.rank_pad + a.rank_pad + 8 * o) = lo;
  }
}

// ------------------------------------------------------------ second product

// A wave's unit of 64 columns: block j of four holds, in operand row i, column
// 32 (j / 2) + 8 (i / 4) + 4 (j % 2) + i % 4, so that a lane's results of two blocks are
// eight neighbouring columns of one token, and a load of all lanes takes whole
// 64-byte pieces of sixteen rows.  SB: 32-rank blocks of B; PACK (rank 8 or 16): both halves of H
// share one block.
//
// With more than 16 rows the four waves share the tile's H through LDS (read by each of
// them from memory it cost 8 us of 32 at 2048 rows and rank 64: the vector caches, not
// memory, were the bound), up to rank 128; Y, B and H are all requested at once.
template <int SB, bool PACK, int SUB, bool LDS>
__device__ __forceinline__ void expand(const AdapterArgs& a, const Tile& t, int tile, int n0, half_t* lds) {
  constexpr int kH = PACK ? 1 : 2 * SB;
  const int tid = threadIdx.x, lane = tid % kWave, c = lane % 16, oct = lane / 16;
  const int32_t* list = a.plan + kPlanHead + 4 * (int64_t)a.most_tiles;
  const half_t* H = (const half_t*)a.H + (int64_t)tile * kAdapterTile * 2 * a.rank_pad;
  const bool some = n0 < a.N, whole = a.y_vectors && n0 + kUnit <= a.N;     // (else column by column)
  half8_t b[4][SB];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = min(n0 + 32 * (j / 2) + 8 * (c / 4) + 4 * (j % 2) + c % 4, a.N - 1);    // (a column past the last is not stored)
    const half_t* row = (const half_t*)a.B + ((int64_t)t.adapter * a.N + n) * a.rank;
#pragma unroll
    for (int s = 0; s < SB; ++s) {
      const int o = PACK ? oct % (a.rank / 8) : 4 * s + oct;
      b[j][s] = load_half8(row + 8 * min(o, a.rank / 8 - 1));
    }
  }
  // H's rows: 2 rank_pad halves, a place of eight more between them in LDS.
  const int octets = a.rank_pad / 4, stride = 8 * octets + 8;
  constexpr int kStage = LDS ? kAdapterTile * 8 * SB / kThreads : 1;      // 16-byte pieces of a thread
  half8_t staged[kStage];
  if constexpr (LDS)
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      const int u = tid + i * kThreads;
      staged[i] = load_half8(H + 8 * (int64_t)min(u, t.rows * octets - 1));
    }
  half_t* y[SUB];
  half8_t old[SUB][2];
  float factor[SUB];
#pragma unroll
  for (int g = 0; g < SUB; ++g) {
    const int at = min(16 * g + c, t.rows - 1);
    const int32_t token = min(max(list[t.first + at], 0), a.rows - 1);
    y[g] = (half_t*)a.Y + (int64_t)token * a.y_stride + n0 + 8 * oct;
    factor[g] = a.factor[(int64_t)tile * kAdapterTile + at];
  }
#pragma unroll
  for (int g = 0; g < SUB; ++g)
    if (whole) {
      old[g][0] = load_half8(y[g]);
      old[g][1] = load_half8(y[g] + 32);
    }
  if constexpr (LDS) {
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      const int u = tid + i * kThreads;
      if (u < t.rows * octets) *(half8_t*)(lds + u / octets * stride + 8 * (u % octets)) = staged[i];
    }
    __syncthreads();
  }
  if (!some) return;
  // (ranks past the last count nothing, whatever lies there)
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int s = 0; s < SB; ++s)
      if (PACK ? oct >= a.rank / 4 : 4 * s + oct >= a.rank / 8) b[j][s] = zero_half8();
#pragma unroll
  for (int g = 0; g < SUB; ++g) {
    if (16 * g >= t.rows) break;
    const int at = min(16 * g + c, t.rows - 1);
    const half_t* hr = LDS ? lds + at * stride : H + (int64_t)at * 8 * octets;
    half8_t h[kH];
    if constexpr (PACK) {
      h[0] = load_half8(hr + 8 * min(oct, a.rank / 4 - 1));
      if (oct >= a.rank / 4) h[0] = zero_half8();
    } else {
#pragma unroll
      for (int s = 0; s < kH; ++s) h[s] = load_half8(hr + 32 * s + 8 * oct);
    }
    f4_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[j] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (PACK) {
        acc[j] = mfma16x16x32(b[j][0], h[0], acc[j]);
      } else {
#pragma unroll
        for (int s = 0; s < SB; ++s) acc[j] = mfma16x16x32(b[j][s], h[SB + s], acc[j]);
#pragma unroll
        for (int s = 0; s < SB; ++s) acc[j] = mfma16x16x32(b[j][s], h[s], acc[j]);
      }
    }
    if (16 * g + c >= t.rows) continue;
    if (whole) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        half8_t o;
#pragma unroll
        for (int n = 0; n < 8; ++n) o[n] = (half_t)__builtin_fmaf(factor[g], acc[2 * v + n / 4][n % 4], (float)old[g][v][n]);
        *(half8_t*)(y[g] + 32 * v) = o;
      }
    } else {
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const int col = 32 * (n / 8) + n % 8;
        if (n0 + 8 * oct + col < a.N)
          y[g][col] = (half_t)__builtin_fmaf(factor[g], acc[n / 4][n % 4], (float)y[g][col]);
      }
    }
  }
}

template <int SB, bool PACK>
__global__ void __launch_bounds__(kThreads) adapter_expand_kernel(AdapterArgs a) {
  constexpr bool kLds = SB <= 4;
  __shared__ __attribute__((aligned(16))) half_t lds[kLds ? kAdapterTile * (64 * SB + 8) : 8];
  const int tile = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks, wave = threadIdx.x / kWave;
  if (tile >= min(a.plan[0], a.most_tiles)) return;
  const int n0 = (chunk * kWaves + wave) * kUnit;
  const int4 q = plan_tiles(a.plan)[tile];
  const Tile t = {min(max(q.x, 0), a.adapters - 1), min(max(q.y, 0), a.rows - 1), min(max(q.z, 1), kAdapterTile)};
  if (t.rows <= 16) expand<SB, PACK, 1, false>(a, t, tile, n0, lds);
  else expand<SB, PACK, 4, kLds>(a, t, tile, n0, lds);
}

template <int RB>
hipError_t shrink_launch(const AdapterArgs& a, hipStream_t s) {
  const size_t red = (size_t)kShrinkWaves / 2 * 4 * RB * kWave * sizeof(f4_t), h = (size_t)kAdapterTile * a.rank * 4;
  const size_t bytes = red > h ? red : h;
  adapter_shrink_kernel<RB><<<dim3((unsigned)(a.most_tiles * a.slices)), dim3(kShrinkThreads), bytes, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_plan(const AdapterPlanArgs& a, void* stream) {
  adapter_plan_kernel<<<dim3(1), dim3(kPlanThreads), 0, (hipStream_t)stream>>>(a);
  return hipGetLastError();
}

int64_t adapter_most_tiles(int64_t rows, int64_t batch, int64_t adapters) {
  const int64_t groups = std::min(std::min(batch, adapters), rows);
  return (rows + (kAdapterTile - 1) * groups) / kAdapterTile;
}

size_t adapter_plan_size(int64_t rows, int64_t batch, int64_t adapters) {
  return 4 * (size_t)(kPlanHead + 4 * adapter_most_tiles(rows, batch, adapters) + rows);
}

// Slices of K by what a call is expected to take: a workgroup reads its rows of X and
// its ranks of A at about 50 bytes a ns, workgroups past the CUs' number wait for a place,
// and slices are joined in 2 us and the time in which one workgroup reads them.
AdapterShape adapter_shape(const spear_adapter_desc_t& d, int cus) {
  AdapterShape s;
  s.tiles = (int)adapter_most_tiles(d.rows, d.batch, d.adapters);
  s.rank_pad = d.rank <= 16 ? d.rank : d.rank <= 32 ? 32 : d.rank <= 64 ? 64 : d.rank <= 128 ? 128 : 256;
  const double rows = s.tiles > 0 ? (double)d.rows / s.tiles : 1.0;
  double least = 0.0;
  s.slices = 1;
  s.slice_k = (int)round_up(d.K, 512);
  for (int64_t n = 1; n <= ceil_div(d.K, 512) && s.tiles <= (int)kMaxEcTiles; n *= 2) {
    const int64_t k = round_up(ceil_div(d.K, n), 512), slices = ceil_div(d.K, k);
    const double read = (double)k * 2.0 * (rows + d.rank) / 50e3, waits = (double)ceil_div(s.tiles * slices, cus);
    const double us = read * waits + (slices > 1 ? 2.0 + (double)slices * rows * d.rank * 4.0 / 40e3 : 0.0);
    if (n == 1 || us < least) {
      least = us;
      s.slice_k = (int)k;
      s.slices = (int)slices;
    }
  }
  size_t at = kSyncHeaderBytes;
  s.H = at;
  at += (size_t)s.tiles * kAdapterTile * 2 * s.rank_pad * 2;
  s.factor = at;
  at += (size_t)s.tiles * kAdapterTile * 4;
  s.part = at;
  at += (size_t)s.tiles * s.slices * kAdapterTile * d.rank * 4;
  s.bytes = at;
  return s;
}

hipError_t launch_adapter(const AdapterArgs& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = a.rank <= 16 ? shrink_launch<1>(a, s) : a.rank <= 32 ? shrink_launch<2>(a, s) : shrink_launch<4>(a, s);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)(a.most_tiles * (int64_t)a.chunks)), block(kThreads);
  if (a.rank <= 16) adapter_expand_kernel<1, true><<<grid, block, 0, s>>>(a);
  else if (a.rank_pad == 32) adapter_expand_kernel<1, false><<<grid, block, 0, s>>>(a);
  else if (a.rank_pad == 64) adapter_expand_kernel<2, false><<<grid, block, 0, s>>>(a);
  else if (a.rank_pad == 128) adapter_expand_kernel<4, false><<<grid, block, 0, s>>>(a);
  else adapter_expand_kernel<8, false><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace spear
