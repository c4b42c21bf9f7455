// Shared by the two attention kernels (paged_attn.hip for few rows,
// paged_attn_tile.hip for many): arguments, the numbers of their running
// softmax, lane exchanges and the 8-bit codes' way into the matrix cores.
#pragma once

#include "serve_internal.h"
#include "device_common.h"

namespace spear {

struct AttnK {
  const half_t* q;
  int64_t q_ts, q_hs;
  const int32_t *cu, *lens, *table;
  int64_t table_stride;
  const void *kc, *vc;
  const float *ks, *vs;
  half_t* out;
  float* part;          // partial results of row tiles that workgroups share
  uint32_t* counters;   // zero before and after
  int32_t batch, total_q, q_heads, kv_heads, group, max_kv, page_log2, num_pages;
  int32_t part_bytes;
  int32_t cus;          // compute units planned for
  int32_t rows_from, rows_to;   // sequences with more rows than the one and no more than the other are this launch's
  float scale;                  // |scale| * log2(e)
  int32_t negate;               // the scale is negative: queries enter with the other sign
  int32_t check_order;          // do nothing unless the offsets rise
};

hipError_t launch_attention_tiles(const AttnK& k, int dim, bool i8, int grid, hipStream_t st);

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kNone = -0x1.fffffep127f;   // reference of a row that has seen no key: below every finite score
constexpr float kHead = 14.0f;       // a maximum more than this above the reference moves it (by their
                                     // difference: a sum would be rounded up at large scores)
constexpr float kStart = 6.0f;       // .. to this far below the maximum
constexpr float kMaxScale = 1e30f;   // scales above this do not enter the reference

// A value that all lanes hold alike, moved to a scalar register: addresses and
// bounds made of it then are scalar too (a division leaves it in a vector one).
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }

// A buffer resource in scalar registers.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* base, uint32_t bytes) {
  const uint64_t p = (uint64_t)base;
  return make_rsrc((const void*)((uint64_t)uniform((uint32_t)(p >> 32)) << 32 | uniform((uint32_t)p)), uniform(bytes));
}

// ------------------------------------------------------------- the sequences
//
// The lengths are on the device, so every workgroup finds its work by itself, with
// a scan over the sequences (64 a step).

// Sum over the lanes up to and with this one, in the vector unit.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t add_from(uint32_t x) {
  return x + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x = add_from<0x111, 0xF>(x);   // 1, 2, 4, 8 lanes below within 16
  x = add_from<0x112, 0xF>(x);
  x = add_from<0x114, 0xF>(x);
  x = add_from<0x118, 0xF>(x);
  x = add_from<0x142, 0xA>(x);   // lane 15 of the 16 below, then lane 31
  return add_from<0x143, 0xC>(x);
}
__device__ __forceinline__ uint32_t wave_sum(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_readlane((int)wave_scan(x), kWave - 1);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t max_from(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max_from<0x111, 0xF>(x);
  x = max_from<0x112, 0xF>(x);
  x = max_from<0x114, 0xF>(x);
  x = max_from<0x118, 0xF>(x);
  x = max_from<0x142, 0xA>(x);
  return (uint32_t)__builtin_amdgcn_readlane((int)max_from<0x143, 0xC>(x), kWave - 1);
}

struct __attribute__((aligned(16))) Seq {
  int q0, n, kv, tiles;   // first row of q, new tokens, cached tokens, row tiles
};
template <int R>
__device__ __forceinline__ Seq sequence(const AttnK& a, int b) {
  Seq s = {0, 0, 0, 0};
  if (b < a.batch) {
    const int c0 = a.cu[b], c1 = a.cu[b + 1], len = a.lens[b];
    s.q0 = min(max(c0, 0), a.total_q);
    s.n = min(max(c1, s.q0), a.total_q) - s.q0;
    s.kv = min(max(len, 0), a.max_kv);
    const int rows = s.n * a.group;
    s.tiles = rows > a.rows_from && rows <= a.rows_to ? (rows + R - 1) / R : 0;
  }
  return s;
}

// Whether the offsets rise (the same in all workgroups).
__device__ __forceinline__ bool offsets_rise(const AttnK& a, int lane) {
  bool falls = false;
  for (int b = lane; b < a.batch; b += kWave) falls |= a.cu[b + 1] < a.cu[b];
  return !__ballot(falls);
}

// -------------------------------------------------------------- small pieces

// Over the four lanes (c, 0..3) that hold row c: swaps of 16- and 32-lane halves
// (each returns the two halves' values in both).
typedef uint32_t pair_t __attribute__((ext_vector_type(2)));
template <typename F>
__device__ __forceinline__ float over_row(float x, F f) {
  const uint32_t v = float_bits(x);
  const pair_t a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  const uint32_t w = float_bits(f(bits_float(a.x), bits_float(a.y)));
  const pair_t b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return f(bits_float(b.x), bits_float(b.y));
}
__device__ __forceinline__ float row_max4(float x) {
  return over_row(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float row_sum4(float x) {
  return over_row(x, [](float a, float b) { return a + b; });
}

// Codes become fp16 values exactly: a code's byte with its sign bit flipped, under
// the byte 0x64, is the fp16 number 1024 + 128 + code.
constexpr uint32_t kCodeSigns = 0x80808080u, kCodeHigh = 0x64646464u;
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t biased) {   // 0x64b1'64b0, signs flipped
  const half2_t bias = {(half_t)1152.0f, (half_t)1152.0f};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, biased) - bias);
}
// Eight codes of two words, in order.
__device__ __forceinline__ half8_t codes_to_half8(uint32_t lo, uint32_t hi) {
  u32x4_t r;
  lo ^= kCodeSigns;
  hi ^= kCodeSigns;
  r[0] = codes_to_half2(__builtin_amdgcn_perm(kCodeHigh, lo, 0x04010400u));
  r[1] = codes_to_half2(__builtin_amdgcn_perm(kCodeHigh, lo, 0x04030402u));
  r[2] = codes_to_half2(__builtin_amdgcn_perm(kCodeHigh, hi, 0x04010400u));
  r[3] = codes_to_half2(__builtin_amdgcn_perm(kCodeHigh, hi, 0x04030402u));
  return __builtin_bit_cast(half8_t, r);
}

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(4))) int32_t scalar_i32_t;
template <int BYTES> struct Vec;
template <> struct Vec<4> { typedef uint32_t type __attribute__((ext_vector_type(1))); };
template <> struct Vec<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <> struct Vec<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };

__device__ __forceinline__ bool half2_not_finite(uint32_t w) {
  return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
}

// An fp16 number's kind as an fp16 number: 0 finite, 1 infinity, 64 -infinity,
// 4096 NaN.
__device__ __forceinline__ uint32_t kind_of(uint32_t h) {
  if ((h & 0x7C00u) != 0x7C00u) return 0u;
  return (h & 0x03FFu) ? 0x6C00u : (h & 0x8000u) ? 0x5400u : 0x3C00u;
}

// Lanes' 4, 8 or 16 bytes of a buffer.
template <int BYTES>
__device__ __forceinline__ typename Vec<BYTES>::type buffer_vec(__amdgpu_buffer_rsrc_t r, uint32_t offset) {
  typedef typename Vec<BYTES>::type vec_t;
  if constexpr (BYTES == 4) return vec_t{(uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, offset, 0, 0)};
  else if constexpr (BYTES == 8) return __builtin_bit_cast(vec_t, __builtin_amdgcn_raw_buffer_load_b64(r, offset, 0, 0));
  else return __builtin_bit_cast(vec_t, __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0));
}

// A value the compiler knows nothing about: keeps the comparisons of a tile's
// edge inside the (uniform) branches that need them.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Of an 8-bit cache's values: a power of two above their scales, as its exponent.
// It enters the reference, so that weights times scales keep to fp16's range.
// Bounded below, for two reasons.  A score past 2^27 rounds its sum with the exponent
// to a multiple of 16, 32, ..: an exponent above -16 is then off by what the range
// still holds.  And it loses nothing: the largest weight times a scale of 2^-35 is a
// normal fp16 number, while the values of scales from 2^-32 down vanish in fp16.
__device__ __forceinline__ float scale_exponent(float largest) {
  return fmaxf((float)((int)(float_bits(largest) >> 23) - 126), -15.0f);
}

// Queries of a row as a B operand; a negative scale's sign goes here.
__device__ __forceinline__ half8_t query(const half_t* p, bool negate) {
  const half8_t h = load_half8(p);
  return negate ? -h : h;
}

}  // namespace
}  // namespace spear
