// Low-rank adapters of many requests at once, added beside a shared projection:
//
//   Y[m] += s_a (X[m] . A_a^T) . B_a^T      a = the adapter of row m's sequence
//
// The plan, made once for a step and used by all of its projections, sorts the batch's
// rows by adapter and cuts each adapter's into tiles of at most 64.  The first product
// (adapter_shrink_kernel) takes tiles x slices of K, the last slice of a tile to arrive
// adds them in order; the second (adapter_expand_kernel) takes tiles x columns and
// updates Y in place.  With few rows and a short K one launch does both
// (adapter_fused_kernel).
//
// With one token a request these are chains of round trips over the adapters in use
// (each read once, whatever the order of the requests): 64 rows, 24 adapters of rank 16,
// K = N = 2048 take 8 us a projection in one launch, 11.5 in two.  With a prompt's chunk
// the second product is bound by Y, read and written: 2048 rows of rank 64 from 4096 to
// 14336 columns take 28.5 us for it (117 MB of Y: 4.1 TB/s) and 16.5 for the first (140
// workgroups at 30 bytes a ns, the rate of a CU, and 6 us for the exchange).
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
#include "wave_ops.h"

namespace spear {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kShrinkThreads = 512, kShrinkWaves = kShrinkThreads / kWave;
constexpr int kPlanHead = 8;      // words: tiles
constexpr int kUnit = kAdapterColumns / kWaves;   // columns of Y that a wave computes
typedef float f4_t __attribute__((ext_vector_type(4)));

// The plan: head, tiles {adapter, first entry of the list, rows, 0}, list of rows.
__device__ __forceinline__ const int4* plan_tiles(const int32_t* plan) { return (const int4*)(plan + kPlanHead); }

// ------------------------------------------------------------------ the plan

template <int THREADS>
__device__ __forceinline__ int64_t sum_before(int64_t v, int64_t* waves, int64_t* total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int64_t run = wave_run(v);
  __syncthreads();
  if (lane == kWave - 1) waves[wave] = run;
  __syncthreads();
  int64_t before = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < THREADS / kWave; ++i) {
    if (i < wave) before += waves[i];
    sum += waves[i];
  }
  *total = sum;
  return before + run - v;
}

// One workgroup: rows per adapter, their running sums, and every sequence's place among
// its adapter's rows.  (Which place it gets is a matter of order of arrival; a row's
// result does not depend on it.)  Offsets that do not rise within the rows give a plan
// of no tiles.  A chain of round trips: 3 us at 64 sequences, 4.6 with 2048 rows; for
// up to 256 sequences and adapters by 256 threads (1024, and the places given out in a
// second round of atomics: 5.2 and 5.7).
template <int THREADS>
__global__ void __launch_bounds__(THREADS) adapter_plan_kernel(AdapterPlanArgs a) {
  __shared__ int32_t count[kMaxAdapters];      // rows
  __shared__ int32_t tile_to[kMaxAdapters];    // running sum of tiles
  __shared__ int32_t list_at[kMaxAdapters];
  __shared__ int64_t waves[THREADS / kWave];
  __shared__ int32_t first_of[THREADS], rows_of[THREADS], place_of[THREADS];
  __shared__ int32_t bad, longs;
  const int tid = threadIdx.x;
  for (int i = tid; i < a.adapters; i += THREADS) count[i] = 0;
  if (tid == 0) bad = longs = 0;
  // Sequence b: its rows, its adapter, its place among that one's rows.
  int32_t from = 0, n = 0, of = 0, at = 0;
  auto look = [&](int b) {       // false: its offsets are no plan's
    n = 0;
    if (b >= a.batch) return true;
    from = a.cu[b];
    const int32_t to = a.cu[b + 1];
    of = a.adapter[b];
    if (from < 0 || to < from || to > a.rows) return false;
    if (of >= 0 && of < a.adapters) n = to - from;
    return true;
  };
  bool rises = look(tid);        // (its loads come back while the counts are cleared)
  __syncthreads();
  for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
    if (b0 > 0) rises = look(b0 + tid);
    if (!rises) bad = 1;
    if (n > 0) at = atomicAdd(&count[of], n);
  }
  __syncthreads();
  int32_t* list = a.plan + kPlanHead + 4 * (int64_t)a.most_tiles;
  if (bad) {
    if (tid == 0) a.plan[0] = 0;
    return;
  }
  int64_t before = 0, sum;       // rows and tiles, both under 2^25
  for (int i0 = 0; i0 < a.adapters; i0 += THREADS) {
    const int i = i0 + tid;
    const int32_t rows = i < a.adapters ? count[i] : 0, tiles = (rows + kAdapterTile - 1) / kAdapterTile;
    const int64_t to = before + sum_before<THREADS>((int64_t)rows << 32 | tiles, waves, &sum);
    before += sum;
    if (i < a.adapters) {
      tile_to[i] = (int32_t)to + tiles;
      list_at[i] = (int32_t)(to >> 32);
    }
  }
  __syncthreads();
  const int tiles = min((int32_t)before, a.most_tiles);
  if (tid == 0) a.plan[0] = tiles;
  for (int t = tid; t < tiles; t += THREADS) {
    int lo = 0, hi = a.adapters - 1;           // the first adapter whose tiles reach past t
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (tile_to[mid] > t) hi = mid;
      else lo = mid + 1;
    }
    const int in = (t - (lo > 0 ? tile_to[lo - 1] : 0)) * kAdapterTile;
    ((int4*)(a.plan + kPlanHead))[t] = make_int4(lo, list_at[lo] + in, min(count[lo] - in, kAdapterTile), 0);
  }
  if (a.batch > THREADS) {       // the places were not kept: they are given out again
    __syncthreads();
    for (int i = tid; i < a.adapters; i += THREADS) count[i] = 0;
    __syncthreads();
  }
  for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
    if (a.batch > THREADS) {
      look(b0 + tid);
      if (n > 0) at = atomicAdd(&count[of], n);
    }
    const int place = n > 0 ? list_at[of] + at : 0;
    // Short sequences are written by their thread, long ones by a wave each.
    constexpr int kShort = 16;
    if (n <= kShort)
      for (int i = 0; i < n; ++i) list[place + i] = from + i;
    if (n > kShort) {
      const int s = atomicAdd(&longs, 1);
      first_of[s] = from;
      rows_of[s] = n;
      place_of[s] = place;
    }
    __syncthreads();
    const int many = longs;
    for (int s = tid / kWave; s < many; s += THREADS / kWave)
      for (int i = tid % kWave; i < rows_of[s]; i += kWave) list[place_of[s] + i] = first_of[s] + i;
    __syncthreads();
    if (tid == 0) longs = 0;
    __syncthreads();
  }
}

// ------------------------------------------------------------- first product

__device__ __forceinline__ void store_f4_dev(__amdgpu_buffer_rsrc_t r, uint32_t byte_offset, const f4_t& v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), r, byte_offset, 0, kCachePolicySc1);
}

using Tile = AdapterTile;
__device__ __forceinline__ Tile tile_of(const AdapterArgs& a, int tile) {
  const int4 q = plan_tiles(a.plan)[tile];
  return adapter_tile(q.x, q.y, q.z, a.adapters, a.rows);
}

// Ranks [rank0, rank0 + 16 RB) of one slice of K for a tile of up to 16 SUB rows: the
// waves take 64 k in turn (whole lines of X and A), and add their sums through LDS.
// keep(row, rank, four sums)
template <int RB, int SUB, typename F>
__device__ __forceinline__ void shrink(const AdapterArgs& a, const Tile& t, const int32_t* list, int rank0, int k_lo,
                                       int k_hi, f4_t* red, F keep) {
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
  // The waves' sums, those of w and w + 4 first.  (Where there are many the upper four
  // waves' go to the lower four before: LDS holds them in half the place.)
  constexpr int kHalf = kShrinkWaves / 2, kUnits = SUB * RB;
  __syncthreads();
  if constexpr (SUB > 1) {
    if (wave >= kHalf)
#pragma unroll
      for (int u = 0; u < kUnits; ++u) red[((wave - kHalf) * kUnits + u) * kWave + lane] = acc[u / RB][u % RB];
    __syncthreads();
    if (wave < kHalf)
#pragma unroll
      for (int u = 0; u < kUnits; ++u) acc[u / RB][u % RB] += red[(wave * kUnits + u) * kWave + lane];
    __syncthreads();
  }
  if (SUB == 1 || wave < kHalf)
#pragma unroll
    for (int u = 0; u < kUnits; ++u) red[(wave * kUnits + u) * kWave + lane] = acc[u / RB][u % RB];
  __syncthreads();
  for (int u = wave; u < kUnits; u += kShrinkWaves) {
    f4_t sum = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < kHalf; ++v) {
      f4_t two = red[(v * kUnits + u) * kWave + lane];
      if constexpr (SUB == 1) two += red[((v + kHalf) * kUnits + u) * kWave + lane];
      sum = v == 0 ? two : sum + two;
    }
    const int row = 16 * (u / RB) + c, rank = rank0 + 16 * (u % RB) + 4 * oct;
    if (row < t.rows && rank < a.rank) keep(row, rank, sum);
  }
}

// H's rows (fp32, in LDS) as two fp16 numbers per value, and the factor of each row: the
// power of two that they are relative to times the adapter's scale.
template <int ROWS>
__device__ __forceinline__ void to_halves(const AdapterArgs& a, const Tile& t, const float* h, float* factor, half_t* out,
                                          int stride) {
  constexpr int kLanes = kShrinkThreads / ROWS;     // to a row
  static_assert(kLanes <= kWave, "a row's lanes are of one wave");
  const int tid = threadIdx.x, row = tid / kLanes;
  float most = 0.0f;
  if (row < t.rows)
    for (int i = tid % kLanes; i < a.rank; i += kLanes) {
      const float v = fabsf(h[row * a.rank + i]);
      most = v > most || v != v ? v : most;
    }
  most = lanes_all<kLanes>(most, [](float x, float v) { return v > x || v != v ? v : x; });
  // The power of two at or below the row's largest (1 where that is zero, infinite or NaN).
  const uint32_t e = float_bits(most) >> 23;
  const float p = e == 0 ? (most > 0.0f ? 0x1p-126f : 1.0f) : e == 255 ? 1.0f : bits_float(e << 23);
  if (row < t.rows) {
    const float inv = 1.0f / p;
    for (int o = tid % kLanes; o < a.rank_pad / 8; o += kLanes) {
      half8_t hi = zero_half8(), lo = zero_half8();
      if (8 * o < a.rank) {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          float v = h[row * a.rank + 8 * o + n] * inv;
          if (fabsf(v) > 65504.0f && fabsf(v) < INFINITY) v = copysignf(65504.0f, v);   // (beside an infinity or NaN)
          hi[n] = (half_t)v;
          lo[n] = fabsf(v) < INFINITY ? (half_t)(v - (float)hi[n]) : (half_t)0.0f;
        }
      }
      *(half8_t*)(out + row * stride + 8 * o) = hi;
      *(half8_t*)(out + row * stride + a.rank_pad + 8 * o) = lo;
    }
    if (tid % kLanes == 0) factor[row] = p * (a.scale ? a.scale[t.adapter] : 1.0f);
  }
  __syncthreads();
}

template <int RB>
__global__ void __launch_bounds__(kShrinkThreads) adapter_shrink_kernel(AdapterArgs a) {
  extern __shared__ f4_t lds[];
  __shared__ float factor[kAdapterTile];
  __shared__ uint32_t arrived;
  const int shares = a.slices * a.groups;
  const int tile = blockIdx.x / shares, slice = blockIdx.x % shares / a.groups, tid = threadIdx.x;
  if (tile >= min(a.plan[0], a.most_tiles)) return;
  const Tile t = tile_of(a, tile);
  const int32_t* list = a.plan + kPlanHead + 4 * (int64_t)a.most_tiles;
  const size_t tile_bytes = (size_t)kAdapterTile * a.rank * 4;
  char* parts = a.part + (size_t)tile * a.slices * tile_bytes;
  const __amdgpu_buffer_rsrc_t part = make_rsrc(parts + slice * tile_bytes, (uint32_t)tile_bytes);
  const int k_lo = slice * a.slice_k, k_hi = min(k_lo + a.slice_k, a.K);
  auto keep = [&](int row, int rank, const f4_t& v) { store_f4_dev(part, 4u * (uint32_t)(row * a.rank + rank), v); };
  for (int rank0 = blockIdx.x % a.groups * 16 * RB; rank0 < a.rank; rank0 += a.groups * 16 * RB) {
    if (t.rows <= 16) shrink<RB, 1>(a, t, list, rank0, k_lo, k_hi, lds, keep);
    else shrink<RB, 4>(a, t, list, rank0, k_lo, k_hi, lds, keep);
  }
  drain_vm();
  __syncthreads();
  if (shares > 1) {
    if (tid == 0) arrived = add_dev_u32(&a.counters[tile], 1u);
    __syncthreads();
    if (arrived != (uint32_t)shares - 1) return;
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
  to_halves<kAdapterTile>(a, t, h, factor, (half_t*)a.H + (int64_t)tile * kAdapterTile * 2 * a.rank_pad, 2 * a.rank_pad);
  if (tid < t.rows) a.factor[(int64_t)tile * kAdapterTile + tid] = factor[tid];
}

// ------------------------------------------------------------ second product

// A wave's unit of 64 columns: block j of four holds, in operand row i, column
// 32 (j / 2) + 8 (i / 4) + 4 (j % 2) + i % 4, so that a lane's results of two blocks are
// eight neighbouring columns of one token, and a load of all lanes takes whole
// 64-byte pieces of sixteen rows.  SB: 32-rank blocks of B; PACK (rank 8 or 16): both halves of H
// share one block.
//
template <int SB, int SUB>
struct Operands {
  half8_t b[4][SB], old[SUB][2];
  half_t* y[SUB];
};

template <int SB, bool PACK, int SUB>
__device__ __forceinline__ void request(const AdapterArgs& a, const Tile& t, int n0, Operands<SB, SUB>& r) {
  const int lane = threadIdx.x % kWave, c = lane % 16, oct = lane / 16;
  const int32_t* list = a.plan + kPlanHead + 4 * (int64_t)a.most_tiles;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = min(n0 + 32 * (j / 2) + 8 * (c / 4) + 4 * (j % 2) + c % 4, a.N - 1);    // (a column past the last is not stored)
    const half_t* row = (const half_t*)a.B + ((int64_t)t.adapter * a.N + n) * a.rank;
#pragma unroll
    for (int s = 0; s < SB; ++s) {
      const int o = PACK ? oct % (a.rank / 8) : 4 * s + oct;
      r.b[j][s] = load_half8(row + 8 * min(o, a.rank / 8 - 1));
    }
  }
#pragma unroll
  for (int g = 0; g < SUB; ++g) {
    const int32_t token = min(max(list[t.first + min(16 * g + c, t.rows - 1)], 0), a.rows - 1);
    r.y[g] = (half_t*)a.Y + (int64_t)token * a.y_stride + n0 + 8 * oct;
  }
  if (a.y_vectors && n0 + kUnit <= a.N)      // (else column by column)
#pragma unroll
    for (int g = 0; g < SUB; ++g) {
      r.old[g][0] = load_half8(r.y[g]);
      r.old[g][1] = load_half8(r.y[g] + 32);
    }
}

// The product of a unit, and Y with it.  H's rows are `stride` halves apart.
template <int SB, bool PACK, int SUB>
__device__ __forceinline__ void apply(const AdapterArgs& a, const Tile& t, int n0, Operands<SB, SUB>& r, const half_t* H,
                                      int stride, const float* factor) {
  constexpr int kH = PACK ? 1 : 2 * SB;
  const int lane = threadIdx.x % kWave, c = lane % 16, oct = lane / 16;
  const bool whole = a.y_vectors && n0 + kUnit <= a.N;
  // (ranks past the last count nothing, whatever lies there)
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int s = 0; s < SB; ++s)
      if (PACK ? oct >= a.rank / 4 : 4 * s + oct >= a.rank / 8) r.b[j][s] = zero_half8();
#pragma unroll
  for (int g = 0; g < SUB; ++g) {
    if (16 * g >= t.rows) break;
    const int at = min(16 * g + c, t.rows - 1);
    const half_t* hr = H + at * stride;
    const float f = factor[at];
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
        acc[j] = mfma16x16x32(r.b[j][0], h[0], acc[j]);
      } else {
#pragma unroll
        for (int s = 0; s < SB; ++s) acc[j] = mfma16x16x32(r.b[j][s], h[SB + s], acc[j]);
#pragma unroll
        for (int s = 0; s < SB; ++s) acc[j] = mfma16x16x32(r.b[j][s], h[s], acc[j]);
      }
    }
    if (16 * g + c >= t.rows) continue;
    if (whole) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        half8_t o;
#pragma unroll
        for (int n = 0; n < 8; ++n) o[n] = (half_t)__builtin_fmaf(f, acc[2 * v + n / 4][n % 4], (float)r.old[g][v][n]);
        *(half8_t*)(r.y[g] + 32 * v) = o;
      }
    } else {
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const int col = 32 * (n / 8) + n % 8;
        if (n0 + 8 * oct + col < a.N)
          r.y[g][col] = (half_t)__builtin_fmaf(f, acc[n / 4][n % 4], (float)r.y[g][col]);
      }
    }
  }
}

// With more than 16 rows the four waves share the tile's H through LDS (read by each of
// them from memory it cost 8 us of 32 at 2048 rows and rank 64: the vector caches, not
// memory, were the bound), up to rank 128; Y, B and H are all requested at once.
template <int SB, bool PACK>
__global__ void __launch_bounds__(kThreads) adapter_expand_kernel(AdapterArgs a) {
  constexpr bool kLds = SB <= 4;
  constexpr int kStage = kAdapterTile * 8 * SB / kThreads;      // 16-byte pieces of a thread
  __shared__ __attribute__((aligned(16))) half_t lds[kLds ? kAdapterTile * (64 * SB + 8) : 8];
  const int tile = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks, tid = threadIdx.x, wave = tid / kWave;
  if (tile >= min(a.plan[0], a.most_tiles)) return;
  const int n0 = (chunk * kWaves + wave) * kUnit;
  const Tile t = tile_of(a, tile);
  // (a row: 2 rank_pad halves, and a place of eight more in LDS)
  const int octets = a.rank_pad / 4, stride = 8 * octets + 8;
  const half_t* H = (const half_t*)a.H + (int64_t)tile * kAdapterTile * 8 * octets;
  const float* factor = a.factor + (int64_t)tile * kAdapterTile;
  if (t.rows <= 16) {
    if (n0 >= a.N) return;
    Operands<SB, 1> r;
    request<SB, PACK, 1>(a, t, n0, r);
    apply<SB, PACK, 1>(a, t, n0, r, H, 8 * octets, factor);
    return;
  }
  half8_t staged[kStage];
  if constexpr (kLds)
#pragma unroll
    for (int i = 0; i < kStage; ++i) staged[i] = load_half8(H + 8 * (int64_t)min(tid + i * kThreads, t.rows * octets - 1));
  Operands<SB, 4> r;
  if (n0 < a.N) request<SB, PACK, 4>(a, t, n0, r);
  if constexpr (kLds) {
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      const int u = tid + i * kThreads;
      if (u < t.rows * octets) *(half8_t*)(lds + u / octets * stride + 8 * (u % octets)) = staged[i];
    }
    __syncthreads();
  }
  if (n0 < a.N) apply<SB, PACK, 4>(a, t, n0, r, kLds ? lds : H, kLds ? stride : 8 * octets, factor);
}

// Both products in one launch, for few rows and a short K: every workgroup of a tile forms
// its H by itself (from the XCD's L2, after the first) and applies it to its columns,
// whose B and Y come in meanwhile.  Up to rank 32 a tile of more than 16 rows goes in one
// pass (64 rows of one adapter of rank 16: 16 us, sixteen at a time 26).
template <int RB, int ROWS, int STRIDE>
struct FusedScratch {
  f4_t red[(ROWS > 16 ? kShrinkWaves / 2 * 4 : kShrinkWaves) * RB * kWave];
  float h[ROWS * 16 * RB];
  __attribute__((aligned(16))) half_t halves[ROWS * STRIDE];
  float factor[ROWS];
};
template <int RB, int SB, bool PACK, int SUB, int STRIDE, typename S>
__device__ __forceinline__ void fused(const AdapterArgs& a, const Tile& t, int n0, int n_end, S& s) {
  const int32_t* list = a.plan + kPlanHead + 4 * (int64_t)a.most_tiles;
  Operands<SB, SUB> r;
  if (n0 < n_end) request<SB, PACK, SUB>(a, t, n0, r);
  shrink<RB, SUB>(a, t, list, 0, 0, a.K, s.red, [&](int row, int rank, const f4_t& v) { *(f4_t*)(s.h + row * a.rank + rank) = v; });
  __syncthreads();
  to_halves<16 * SUB>(a, t, s.h, s.factor, s.halves, STRIDE);
  for (int n = n0; n < n_end; n += kShrinkWaves * kUnit) {
    if (n > n0) request<SB, PACK, SUB>(a, t, n, r);
    apply<SB, PACK, SUB>(a, t, n, r, s.halves, STRIDE, s.factor);
  }
}
template <int RB, int SB, bool PACK>
__global__ void __launch_bounds__(kShrinkThreads) adapter_fused_kernel(AdapterArgs a) {
  constexpr int kStride = (PACK ? 32 : 64 * SB) + 8;
  constexpr bool kWhole = RB <= 2;       // (LDS holds the sums of a whole tile's rows)
  __shared__ FusedScratch<RB, kWhole ? kAdapterTile : 16, kStride> s;
  const int tile = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks, wave = threadIdx.x / kWave;
  if (tile >= min(a.plan[0], a.most_tiles)) return;
  const Tile t = tile_of(a, tile);
  const int n_end = min((chunk + 1) * a.chunk_columns, a.N), n0 = chunk * a.chunk_columns + wave * kUnit;
  if (kWhole && t.rows > 16) {
    fused<RB, SB, PACK, 4, kStride>(a, t, n0, n_end, s);
  } else {
    for (int row0 = 0; row0 < t.rows; row0 += 16)
      fused<RB, SB, PACK, 1, kStride>(a, Tile{t.adapter, t.first + row0, min(t.rows - row0, 16)}, n0, n_end, s);
  }
}

template <int RB>
hipError_t shrink_launch(const AdapterArgs& a, hipStream_t s) {
  const size_t red = (size_t)kShrinkWaves / 2 * 4 * RB * kWave * sizeof(f4_t), h = (size_t)kAdapterTile * a.rank * 4;
  const size_t bytes = red > h ? red : h;
  adapter_shrink_kernel<RB><<<dim3((unsigned)(a.most_tiles * (int64_t)a.slices * a.groups)), dim3(kShrinkThreads), bytes, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_plan(const AdapterPlanArgs& a, void* stream) {
  if (a.batch <= 256 && a.adapters <= 256) adapter_plan_kernel<256><<<dim3(1), dim3(256), 0, (hipStream_t)stream>>>(a);
  else adapter_plan_kernel<1024><<<dim3(1), dim3(1024), 0, (hipStream_t)stream>>>(a);
  return hipGetLastError();
}

int64_t adapter_most_tiles(int64_t rows, int64_t batch, int64_t adapters) {
  const int64_t groups = std::min(std::min(batch, adapters), rows);
  return (rows + (kAdapterTile - 1) * groups) / kAdapterTile;
}

size_t adapter_plan_size(int64_t rows, int64_t batch, int64_t adapters) {
  return 4 * (size_t)(kPlanHead + 4 * adapter_most_tiles(rows, batch, adapters) + rows);
}

// The launch shape by what a call is expected to take.  A workgroup reads its rows of X
// and its ranks of A at about 25 bytes a ns, and workgroups past the CUs' number wait for
// a place.  Two launches: slices of K (at least 512, joined in 2 us and the time in which
// one workgroup reads them), and 4 us more than one; ranks past 64 go to workgroups of
// their own (2048 rows of rank 128, 4096 to 4096 columns: 40 us, one after the other 44; 16
// rows of rank 256: 25 and 32).  One launch: all of K in every
// workgroup, for as many columns as leave no more workgroups than CUs.
AdapterShape adapter_shape(const spear_adapter_desc_t& d, int cus) {
  AdapterShape s;
  s.tiles = (int)adapter_most_tiles(d.rows, d.batch, d.adapters);
  s.rank_pad = d.rank <= 16 ? d.rank : d.rank <= 32 ? 32 : d.rank <= 64 ? 64 : d.rank <= 128 ? 128 : 256;
  const double rows = s.tiles > 0 ? (double)d.rows / s.tiles : 1.0;
  // (up to 64 ranks a workgroup, where there are counters to join them)
  const bool joins = s.tiles <= (int)kMaxEcTiles;
  s.groups = joins ? (int)ceil_div(d.rank, kAdapterRanks) : 1;
  const double ranks = s.groups > 1 ? kAdapterRanks : d.rank;
  auto reads = [&](double k, int64_t workgroups) { return k * 2.0 * (rows + ranks) / 25e3 * (double)ceil_div(workgroups, cus); };
  double least = 0.0;
  s.slices = 1;
  s.slice_k = (int)round_up(d.K, 512);
  for (int64_t n = 1; n <= std::min<int64_t>(ceil_div(d.K, 512), 64) && (joins || n == 1); ++n) {
    const int64_t k = round_up(ceil_div(d.K, n), 512), slices = ceil_div(d.K, k);
    const double us = reads((double)k, s.tiles * slices * s.groups) + (slices > 1 ? 2.0 + (double)slices * rows * d.rank * 4.0 / 25e3 : 0.0);
    if (n == 1 || us < least) {
      least = us;
      s.slice_k = (int)k;
      s.slices = (int)slices;
    }
  }
  const int64_t units = ceil_div(d.N, 2 * kAdapterColumns), fit = s.tiles > 0 ? std::max<int64_t>(1, cus / s.tiles) : 1;
  const int64_t chunks = std::min(units, fit);
  s.fused = d.rank <= kAdapterRanks && rows <= 16.0 && reads((double)d.K, s.tiles * chunks) <= least + 4.0;
  s.chunk_columns = s.fused ? (int)(2 * kAdapterColumns * ceil_div(units, chunks)) : kAdapterColumns;
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
  if (a.fused) {
    const dim3 grid((unsigned)(a.most_tiles * (int64_t)a.chunks)), block(kShrinkThreads);
    if (a.rank <= 16) adapter_fused_kernel<1, 1, true><<<grid, block, 0, s>>>(a);
    else if (a.rank_pad == 32) adapter_fused_kernel<2, 1, false><<<grid, block, 0, s>>>(a);
    else adapter_fused_kernel<4, 2, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
  }
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
