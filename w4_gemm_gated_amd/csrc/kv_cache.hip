// The paged key/value cache: new tokens written (fp16 as they are, or
// quantised to 8 bits with one scale per token and head), and sequences read
// back in fp16.
//
// Both kernels are bound by memory: a thread owns eight values of one head
// (16 bytes of fp16, 8 of codes) of the keys and of the values, so every
// fp16 access is 16 bytes wide and a head's row is one contiguous run of
// head_dim / 8 lanes; the keys' and the values' loads are in flight together.  A
// workgroup takes 16 (head_dim 128) or 32 tokens of one head, or twice as many:
// neighbours in a page, so that it touches whole lines of codes and scales (with
// all heads of two tokens instead, a line of scales went to all eight XCDs: 205
// MB fetched for 169, and 10,000 tokens of 8 heads of 64 took 45 us instead of 37).
// Measured with 8 heads of 128: 24 sequences, 80,000 tokens, read back from 8 bits
// in 102 us (498 MB read and written, 4.9 TB/s; a plain copy of 2 GiB reaches
// 4.9) and from fp16 in 117 (656 MB, 5.6 TB/s); 34,000 from fp16 in 45 us; 6,800 tokens quantised, written and read back in 21 us (85 MB); a decode
// step's 48 tokens in 2.7 us of the 7.5 that a launch takes.
#include "serve_internal.h"
#include "device_common.h"

namespace spear {
namespace {

constexpr int kThreads = 256;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

struct AppendK {
  const half_t *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;
  const int64_t* slots;
  void *kc, *vc;
  float *ks, *vs;
  int64_t num_slots;
  int32_t tokens, heads, page_log2;
};

// max over the LANES neighbouring lanes that share a head's row; a NaN stays.
template <int LANES>
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = 1; o < LANES; o *= 2) {
    const float y = __shfl_xor(x, o);
    x = (y > x || y != y) ? y : x;
  }
  return x;
}

// Eight fp16 values -> codes, and the row's scale.  The codes are those of the
// definition's float32 division: the product with the reciprocal is off by less
// than 2^-15 (127 x three roundings of 2^-24), so it gives the same integer
// unless it lies that near the middle of two, and only then (one wave in eight)
// does the wave divide.
template <int LANES>
__device__ __forceinline__ u32x2_t quantise(const half8_t& h, float* scale) {
  float x[8], m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = (float)h[i];
    const float a = fabsf(x[i]);
    m = (a > m || a != a) ? a : m;
  }
  m = row_max<LANES>(m);
  const float s = m / 127.0f;
  *scale = s;
  const float r = 1.0f / s;
  float c[8];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = x[i] * r;
    c[i] = rintf(q);
    near |= !(fabsf(q - c[i]) < 0.5f - 0x1p-14f);   // (also s = 0, infinite or NaN)
  }
  if (near)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = s > 0.0f ? rintf(x[i] / s) : 0.0f;
      c[i] = c[i] == c[i] ? fminf(fmaxf(c[i], -127.0f), 127.0f) : 0.0f;   // 0 * s is then 0 or NaN
    }
  u32x2_t w = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i / 4] |= ((uint32_t)(int32_t)c[i] & 0xFFu) << (8 * (i % 4));
  return w;
}

// LANES = head_dim / 8 threads per (token, head).  One pass over the rows: a
// scale needs only its own row, which lies in the LANES threads' registers.
template <int LANES, bool I8>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendK a) {
  const int head = (int)(blockIdx.x % (uint32_t)a.heads), c = (int)threadIdx.x % LANES;
  const int64_t tok = (int64_t)(blockIdx.x / (uint32_t)a.heads) * (kThreads / LANES) + (int)threadIdx.x / LANES;
  if (tok >= a.tokens) return;   // whole rows leave together
  const int64_t slot = a.slots[tok];
  const half8_t kx = load_half8(a.k + tok * a.k_ts + head * a.k_hs + 8 * c);
  const half8_t vx = load_half8(a.v + tok * a.v_ts + head * a.v_hs + 8 * c);
  if (slot < 0 || slot >= a.num_slots) return;
  const int64_t page = slot >> a.page_log2, place = slot & ((1 << a.page_log2) - 1);
  const int64_t at = ((page * a.heads + head) << a.page_log2) + place;   // row of the cache
  if constexpr (I8) {
    float ks, vs;
    const u32x2_t kw = quantise<LANES>(kx, &ks), vw = quantise<LANES>(vx, &vs);
    ((u32x2_t*)a.kc)[at * LANES + c] = kw;
    ((u32x2_t*)a.vc)[at * LANES + c] = vw;
    if (c == 0) {
      a.ks[at] = ks;
      a.vs[at] = vs;
    }
  } else {
    ((half8_t*)a.kc)[at * LANES + c] = kx;
    ((half8_t*)a.vc)[at * LANES + c] = vx;
  }
}

struct GatherK {
  const int32_t *table, *cu;
  int64_t table_stride;
  const void *kc, *vc;
  const float *ks, *vs;
  half8_t *ko, *vo;
  int32_t batch, rows, heads, page_log2, num_pages;
};

template <bool I8> struct KvVec { typedef half8_t type; };
template <> struct KvVec<true> { typedef u32x2_t type; };

__device__ __forceinline__ half8_t dequantise(const u32x2_t& w, float s) {
  half8_t h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = (half_t)((float)(int8_t)(w[i / 4] >> (8 * (i % 4))) * s);
  return h;
}

// A workgroup's rows belong to few sequences: its first row's is counted by the
// whole wave (the rising entries of cu not above it), and a thread steps on
// from there.  A thread takes ROWS rows, whose loads are in flight together.
template <int LANES, bool I8, int ROWS>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(GatherK a) {
  typedef typename KvVec<I8>::type code_t;
  constexpr int STEP = kThreads / LANES;
  const int head = (int)(blockIdx.x % (uint32_t)a.heads), c = (int)threadIdx.x % LANES;
  const int64_t first = (int64_t)(blockIdx.x / (uint32_t)a.heads) * (STEP * ROWS);
  const int64_t row0 = first + (int)threadIdx.x / LANES;
  int b = -1;
  for (int i = 0; i <= a.batch; i += kWave) {
    const int j = i + (int)threadIdx.x % kWave;
    b += __popcll(__ballot(j <= a.batch && a.cu[j] <= first));
  }
  int64_t at[ROWS];   // place in the cache; -1: a row of no sequence
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t row = row0 + r * STEP;
    while (b < a.batch && a.cu[b + 1] <= row) ++b;
    at[r] = -1;
    if (b >= 0 && b < a.batch && row < a.rows) {
      const int64_t i = row - a.cu[b], entry = table_entry(row, a.cu[b], a.page_log2, a.table_stride);
      if (entry >= 0) {
        const uint32_t page = min((uint32_t)a.table[b * a.table_stride + entry], (uint32_t)a.num_pages - 1);
        at[r] = (((int64_t)page * a.heads + head) << a.page_log2) + (i & ((1 << a.page_log2) - 1));
      }
    }
  }
  code_t kw[ROWS], vw[ROWS];
  float ks[ROWS], vs[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    kw[r] = vw[r] = code_t{};
    ks[r] = vs[r] = 0.0f;
    if (at[r] >= 0) {
      kw[r] = ((const code_t*)a.kc)[at[r] * LANES + c];
      vw[r] = ((const code_t*)a.vc)[at[r] * LANES + c];
      if constexpr (I8) {
        ks[r] = a.ks[at[r]];
        vs[r] = a.vs[at[r]];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t row = row0 + r * STEP;
    if (row >= a.rows) break;
    const int64_t u = (row * a.heads + head) * LANES + c;
    // (written once, not read here)
    if constexpr (I8) {
      __builtin_nontemporal_store(dequantise(kw[r], ks[r]), &a.ko[u]);
      __builtin_nontemporal_store(dequantise(vw[r], vs[r]), &a.vo[u]);
    } else {
      __builtin_nontemporal_store(kw[r], &a.ko[u]);
      __builtin_nontemporal_store(vw[r], &a.vo[u]);
    }
  }
}

template <int LANES, bool I8>
hipError_t launch_gather(const GatherK& k, bool two, hipStream_t st) {
  const int64_t rows = kThreads / LANES * (two ? 2 : 1);   // of a workgroup
  const dim3 grid((unsigned)(ceil_div((int64_t)k.rows, rows) * k.heads)), block(kThreads);
  if (two) kv_gather_kernel<LANES, I8, 2><<<grid, block, 0, st>>>(k);
  else kv_gather_kernel<LANES, I8, 1><<<grid, block, 0, st>>>(k);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, void* stream) {
  AppendK k;
  k.k = (const half_t*)a.k; k.v = (const half_t*)a.v;
  k.k_ts = a.k_ts; k.k_hs = a.k_hs; k.v_ts = a.v_ts; k.v_hs = a.v_hs;
  k.slots = a.slots;
  k.kc = a.k_cache; k.vc = a.v_cache; k.ks = a.k_scale; k.vs = a.v_scale;
  k.num_slots = (int64_t)a.kv.num_pages << a.kv.page_log2;
  k.tokens = a.tokens; k.heads = a.kv.heads; k.page_log2 = a.kv.page_log2;
  const dim3 grid((unsigned)(ceil_div((int64_t)a.tokens, kThreads / (a.kv.dim / 8)) * a.kv.heads)), block(kThreads);
  const hipStream_t st = (hipStream_t)stream;
  const bool i8 = a.kv.dtype == SPEAR_KV_INT8;
  if (a.kv.dim == 64) {
    if (i8) kv_append_kernel<8, true><<<grid, block, 0, st>>>(k);
    else kv_append_kernel<8, false><<<grid, block, 0, st>>>(k);
  } else {
    if (i8) kv_append_kernel<16, true><<<grid, block, 0, st>>>(k);
    else kv_append_kernel<16, false><<<grid, block, 0, st>>>(k);
  }
  return hipGetLastError();
}

hipError_t launch_kv_gather(const KvGatherArgs& a, void* stream) {
  GatherK k;
  k.table = a.table; k.cu = a.cu; k.table_stride = a.table_stride;
  k.kc = a.k_cache; k.vc = a.v_cache; k.ks = a.k_scale; k.vs = a.v_scale;
  k.ko = (half8_t*)a.k_out; k.vo = (half8_t*)a.v_out;
  k.batch = a.batch; k.rows = a.rows; k.heads = a.kv.heads;
  k.page_log2 = a.kv.page_log2; k.num_pages = a.kv.num_pages;
  // Two rows a thread where the outputs pass the 256 MiB that the card caches
  // (from 8 bits 328 MB: 102 us, 110 with one; 61 MB: 38.4, 36.8 with one).
  const bool two = (int64_t)a.rows * a.kv.heads * a.kv.dim * 4 > (int64_t)256 << 20;
  const hipStream_t st = (hipStream_t)stream;
  const bool i8 = a.kv.dtype == SPEAR_KV_INT8;
  if (a.kv.dim == 64) return i8 ? launch_gather<8, true>(k, two, st) : launch_gather<8, false>(k, two, st);
  return i8 ? launch_gather<16, true>(k, two, st) : launch_gather<16, false>(k, two, st);
}

}  // namespace spear
