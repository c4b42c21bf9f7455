// The draw of next tokens with temperature, top-k, top-p and min-p, and the
// distribution that it draws from.
//
// The rules keep a prefix of the tokens in falling order of their logits, so what
// has to be found is where that order is cut: no sort of the vocabulary is needed,
// only the counts and sums of weights above a value.  A row's vocabulary is shared by
// workgroups of kShare tokens each, in two launches (three for probabilities):
//
//   1. Every share finds its maximum and, for top-k and top-p, a histogram of its
//      weights: bins of 1/16 in log2 of the weight, on one grid for the whole row
//      (t = 16 logit / (T ln 2); bin floor(t)), so that shares need no common
//      maximum first and the row is read once.  A bin holds its count and the sum of
//      its weights' distances from the bin's upper edge in fixed point, both in one
//      64-bit integer (one LDS atomic a token; integer sums have no order).  The
//      row's last share to arrive adds the histograms, sums counts and weights from the
//      top, and finds the bin in which each rule's cut lies.
//   2. Tokens above that bin are drawn from at once (an exponential race: the largest
//      weight / noise, ties to the lowest index), those in it (some hundreds) go
//      to a list; noise is read for tokens that are kept, and for no others.  The last
//      share to arrive cuts the list by a radix selection on (logit, index), ends the
//      race, and sums what is kept.
//   3. Probabilities are written.
//
// The sums decide which token is the last one, and in a flat distribution that token
// has a millionth of the total: weights enter the sums to 2^-34 of themselves, and
// sums are held in 64 bits.
//
// A bin that holds more tokens than the list (equal logits, a very high temperature)
// is cut by the same selection over the row itself, by one workgroup: slow, and right.
#include <algorithm>

#include "serve_internal.h"
#include "device_common.h"

namespace spear {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / kWave;
constexpr int kEach = kSampleShare / kThreads;    // tokens of a thread
constexpr int kBins = 2048;                       // 128 in log2 of the weight
constexpr int kBinsEach = kBins / kThreads;
constexpr double kCut = -126.0 * 16.0;            // weights below 2^-126 of the largest are zero
constexpr int kDefBits = 38;                      // fixed point of a bin's sum of distances
constexpr int kFixBits = 40;                      // fixed point of weights in a selection
constexpr int kSubs = 2048;                       // sub-bins of a selection's step
typedef float f4u_t __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 h8u_t __attribute__((ext_vector_type(8), aligned(2)));
typedef unsigned long long u64;

enum Kind : int32_t { kEmpty, kOne, kRace };      // no token, the first one, a race of several

// What a row's first launch leaves for the others.  t: 16 log2 of a weight, on the
// row's grid; bins are counted from the one of the row's largest; masses are in units
// of that bin's upper edge.
struct RowInfo {
  double c16, tm;            // t of a logit of 1, and of the row's largest
  double first, last;        // tokens of bins before `first` are kept, those of bins past `last` are not ..
  double bin_k;              // .. and top-k's cut lies in this bin (one of them, or past them; -1: no such cut)
  double lim;                // min-p: t - tm at least
  double before, before_k;   // mass before `first`, and before bin_k
  double target;             // top-p's mass if that is known; else (with top-k) p
  u64 end;                   // second launch: key of the last token kept (0: all)
  double inv;                // 1 / mass of what is kept, in units of the largest weight
  int32_t kind, token;       // token: the largest logit's
  int32_t left_k;            // tokens that top-k keeps of its bin
  int32_t by_k, by_p;        // which rules cut
  int32_t heavy;             // the list does not hold the tokens of these bins
  uint32_t listed;           // tokens in the list
};

__device__ __forceinline__ uint32_t rising(float l) {     // rises with l; -0 as +0
  const uint32_t b = float_bits(l + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ u64 key_of(float l, int j) { return ((u64)rising(l) << 32) | (uint32_t)~j; }
__device__ __forceinline__ float logit_of(u64 key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return bits_float(b & 0x80000000u ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ bool valid(float l) { return l > -INFINITY; }
// (an infinite logit lies above all others, and equal ones share a place)
__device__ __forceinline__ double t_of(float l, double c16) { return fmin((double)l * c16, 1e300); }

// The bin of a t, from the one of the row's largest: whole numbers, exact wherever two
// bins are near each other.
__device__ __forceinline__ double bin_of(const RowInfo& o, double t) { return floor(o.tm) - floor(t); }
// log2 of a weight in units of the upper edge of bin `bin`.
__device__ __forceinline__ double below_edge(const RowInfo& o, double t, double bin) {
  return ((t - floor(o.tm)) + (bin - 1.0)) * 0.0625;
}

// The workgroup's maximum, bitwise and / or, and sum, in every thread.
template <typename T, typename F>
__device__ __forceinline__ T block_all(T v, T* lds, F f) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o /= 2) v = f(v, (T)__shfl_xor(v, o));
  __syncthreads();
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) v = f(v, lds[i]);
  return v;
}
__device__ __forceinline__ u64 block_max(u64 v, u64* lds) {
  return block_all(v, lds, [](u64 a, u64 b) { return a > b ? a : b; });
}
__device__ __forceinline__ u64 block_add(u64 v, u64* lds) {
  return block_all(v, lds, [](u64 a, u64 b) { return a + b; });
}

// Running sum (inclusive) over the workgroup.
template <typename T>
__device__ __forceinline__ T block_run(T v, T* lds) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
#pragma unroll
  for (int o = 1; o < kWave; o *= 2) {
    const T x = __shfl_up(v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();
  if (lane == kWave - 1) lds[wave] = v;
  __syncthreads();
  T before = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i)
    if (i < wave) before += lds[i];
  return v + before;
}

// A thread's tokens of a share: vectors of eight in turn.
__device__ __forceinline__ int place(int beg, int i) { return beg + 8 * ((i / 8) * kThreads + (int)threadIdx.x) + i % 8; }

template <bool F16>
__device__ __forceinline__ void load_share(const void* row, int beg, int end, float* l) {
  if (end - beg == kSampleShare) {
    const int at = beg + 8 * (int)threadIdx.x;
    if constexpr (F16) {
      h8u_t v[kEach / 8];
#pragma unroll
      for (int i = 0; i < kEach / 8; ++i) v[i] = *(const h8u_t*)((const half_t*)row + at + i * 8 * kThreads);
#pragma unroll
      for (int i = 0; i < kEach; ++i) l[i] = (float)v[i / 8][i % 8];
    } else {
      f4u_t v[kEach / 4];
#pragma unroll
      for (int i = 0; i < kEach / 4; ++i) v[i] = *(const f4u_t*)((const float*)row + at + (i / 2) * 8 * kThreads + i % 2 * 4);
#pragma unroll
      for (int i = 0; i < kEach; ++i) l[i] = v[i / 4][i % 4];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = min(place(beg, i), end - 1);
      l[i] = F16 ? (float)((const half_t*)row)[j] : ((const float*)row)[j];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (place(beg, i) >= end) l[i] = -INFINITY;
  }
}

struct Rules {
  float t, p, m;
  int32_t k;
  bool one;     // only the first token is kept
};
__device__ __forceinline__ Rules rules_of(const SampleArgs& a, int b) {
  Rules r;
  r.t = a.temperature ? a.temperature[b] : a.one_temperature;
  r.k = a.top_k ? a.top_k[b] : a.one_top_k;
  r.p = a.top_p ? a.top_p[b] : a.one_top_p;
  r.m = a.min_p ? a.min_p[b] : a.one_min_p;
  r.one = !(r.t > 0.0f) || r.k == 1 || r.p <= 0.0f;
  if (r.k <= 0 || r.k >= a.vocab) r.k = 0;
  if (!(r.p < 1.0f)) r.p = 1.0f;
  r.m = r.m > 0.0f ? fminf(r.m, 1.0f) : 0.0f;
  return r;
}

__device__ __forceinline__ const void* row_of(const SampleArgs& a, int b) {
  const int64_t r = a.rows ? a.rows[b] : a.first + b;
  if (r < 0 || r >= a.num_rows) return nullptr;
  return (const char*)a.logits + r * a.stride * (a.f16 ? 2 : 4);
}

__device__ __forceinline__ u64 ld64(const u64* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void st64(u64* p, u64 v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Whether this workgroup is the last of its row's; the counter is then zero again.
__device__ __forceinline__ bool last_of_row(const SampleArgs& a, int b, uint32_t* arrived) {
  if (a.shares == 1) {
    drain_vm();
    __syncthreads();
    return true;
  }
  drain_vm();
  __syncthreads();
  if (threadIdx.x == 0) *arrived = add_dev_u32(&a.counters[b], 1u);
  __syncthreads();
  if (*arrived != (uint32_t)a.shares - 1) return false;
  if (threadIdx.x == 0) st_dev_u32(&a.counters[b], 0u);
  return true;
}

// -------------------------------------------------------------- first launch

template <bool F16>
__global__ void __launch_bounds__(kThreads) sample_bins_kernel(SampleArgs a) {
  __shared__ u64 hist[kBins];
  __shared__ uint32_t counts[kBins];
  __shared__ u64 red[kWaves];
  __shared__ double redd[kWaves];
  __shared__ uint32_t redc[kWaves];
  __shared__ uint32_t arrived;
  __shared__ double found_mass;     // of a search over the bins
  __shared__ int found, found_count, found_in;
  __shared__ double total_mass;
  __shared__ uint32_t total_count;
  const int b = blockIdx.x / a.shares, share = blockIdx.x % a.shares, tid = threadIdx.x;
  const Rules r = rules_of(a, b);
  const void* row = row_of(a, b);
  const bool bins = !r.one && (r.k > 0 || r.p < 1.0f);
  const int beg = share * kSampleShare, end = min(beg + kSampleShare, a.vocab);
  float l[kEach];
  u64 best = 0;
  uint32_t least = ~0u;
  if (row) {
    load_share<F16>(row, beg, end, l);
    float top = -INFINITY, low = INFINITY;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (l[i] > top) {
        top = l[i];
        at = place(beg, i);
      }
      if (valid(l[i])) low = fminf(low, l[i]);
    }
    if (valid(top)) {
      best = key_of(top, at);
      least = rising(low);
    }
  }
  best = block_max(best, red);
  const double c16 = fmax(16.0 / ((double)r.t * 0.693147180559945309417), 1e-300);
  ShareInfo* mine = a.share + (int64_t)b * a.shares + share;
  u64* bins_out = a.hist + ((int64_t)b * a.shares + share) * kBins;
  if (bins && best != 0) {
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    least = block_all(least, redc, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
    const double q = floor(t_of(logit_of(best), c16));
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const double t = t_of(l[i], c16), f = floor(t), rel = q - f;
      if (valid(l[i]) && rel < kBins) {
        // 1 - 2^((t - f - 1) / 16): the first term in 64 bits, the rest is below 2^-10
        const double u = (1.0 - (t - f)) * (0.693147180559945309417 / 16.0);
        const float s = (float)u;
        const float h = s * s * (0.5f - s * (1.0f / 6.0f - s * (1.0f / 24.0f - s * (1.0f / 120.0f))));
        const double d = u - (double)h;
        const u64 fixed = (u64)__double_as_longlong(__builtin_fma(d, (double)(1ull << kDefBits), 0x1p52));
        atomicAdd(&hist[(int)rel], fixed - 0x4330000000000000ull + (1ull << 48));
      }
    }
    const double span = q - floor(t_of(logit_of((u64)least << 32), c16)) + 1.0;
    const int used = span < kBins ? (int)span : kBins;
    __syncthreads();
    for (int i = tid; i < used; i += kThreads) st64(&bins_out[i], hist[i]);
    if (tid == 0) {
      st64(&mine->number, (u64)__double_as_longlong(q));
      st64(&mine->used, (u64)used);
    }
  }
  if (tid == 0) st64(&mine->best, best);
  if (!last_of_row(a, b, &arrived)) return;

  // The row: its largest, ..
  ShareInfo* all = a.share + (int64_t)b * a.shares;
  best = 0;
  for (int s = tid; s < a.shares; s += kThreads) {
    const u64 v = ld64(&all[s].best);
    best = best > v ? best : v;
  }
  best = block_max(best, red);
  RowInfo* info = (RowInfo*)((char*)a.info + (int64_t)b * kSampleInfoBytes);
  static_assert(sizeof(RowInfo) <= kSampleInfoBytes, "room for it");
  RowInfo o;
  o.c16 = c16;
  o.tm = best ? t_of(logit_of(best), c16) : 0.0;
  o.first = INFINITY;
  o.last = o.bin_k = -1.0;
  o.lim = fmax(r.m > 0.0f ? 16.0 * log2((double)r.m) : kCut, kCut);
  o.before = o.before_k = o.target = 0.0;
  o.end = 0;
  o.inv = 1.0;
  o.kind = best == 0 ? kEmpty : r.one ? kOne : kRace;
  o.token = best ? (int)~(uint32_t)best : -1;
  o.left_k = o.by_k = o.by_p = o.heavy = 0;
  o.listed = 0;
  if (o.kind != kRace && a.tokens && tid == 0) a.tokens[b] = o.token;
  if (o.kind == kRace && bins) {
    // .. its bins (a thread's are neighbours), ..
    const double q = floor(o.tm);
    uint32_t n[kBinsEach];
    u64 def[kBinsEach];
#pragma unroll
    for (int i = 0; i < kBinsEach; ++i) n[i] = 0, def[i] = 0;
    for (int s = 0; s < a.shares; ++s) {
      if (ld64(&all[s].best) == 0) continue;
      const double behind = q - __longlong_as_double((long long)ld64(&all[s].number));
      if (!(behind < kBins)) continue;
      const int off = (int)behind, used = (int)ld64(&all[s].used);
      const u64* from = a.hist + ((int64_t)b * a.shares + s) * kBins;
#pragma unroll
      for (int i = 0; i < kBinsEach; ++i) {
        const int at = tid * kBinsEach + i - off;
        if (at >= 0 && at < used) {
          const u64 v = ld64(&from[at]);
          n[i] += (uint32_t)(v >> 48);
          def[i] += v & ((1ull << 48) - 1);
        }
      }
    }
    // .. and their running sums.
    double mass[kBinsEach], mass_to = 0.0;
    uint32_t count_to = 0;
#pragma unroll
    for (int i = 0; i < kBinsEach; ++i) {
      const int at = tid * kBinsEach + i;
      const double edge = ldexp(exp2(-(double)(at % 16) / 16.0), -(at / 16));
      mass[i] = edge * ((double)n[i] - (double)def[i] * (1.0 / (double)(1ull << kDefBits)));
      mass_to += mass[i];
      count_to += n[i];
    }
    const double own_mass = mass_to;
    const uint32_t own_count = count_to;
    mass_to = block_run(mass_to, redd);
    count_to = block_run(count_to, redc);
    __syncthreads();
    if (tid == kThreads - 1) {
      total_mass = mass_to;
      total_count = count_to;
    }
#pragma unroll
    for (int i = 0; i < kBinsEach; ++i) counts[tid * kBinsEach + i] = n[i];
    __syncthreads();
    const double total = total_mass;
    const bool by_k = r.k > 0 && (uint32_t)r.k < total_count;
    // The first bin in which the count reaches k, or the mass a target (the last of any
    // tokens if it never does): its place, what lies before it and in it.
    auto search = [&](bool by_count, double target) {
      __syncthreads();
      if (tid == 0) found = kBins;
      __syncthreads();
      int reaches = kBins, lowest = -1;
      double before = mass_to - own_mass;
      uint32_t count = count_to - own_count;
#pragma unroll
      for (int i = 0; i < kBinsEach; ++i) {
        before += mass[i];
        count += n[i];
        if (n[i] > 0) lowest = tid * kBinsEach + i;
        if (n[i] > 0 && reaches == kBins && (by_count ? count >= (uint32_t)r.k : before >= target))
          reaches = tid * kBinsEach + i;
      }
      if (reaches < kBins) atomicMin(&found, reaches);
      const int bin_end = (int)block_max((u64)(lowest + 1), red) - 1;
      const int bin = found < kBins ? found : bin_end;
      before = mass_to - own_mass;
      count = count_to - own_count;
#pragma unroll
      for (int i = 0; i < kBinsEach; ++i) {
        if (tid * kBinsEach + i == bin) {
          found_count = (int)count;
          found_mass = before;
          found_in = (int)n[i];
        }
        before += mass[i];
        count += n[i];
      }
      __syncthreads();
      return bin;
    };
    int bin_k = kBins, first = kBins, last = kBins;
    double low_sum = total, high_sum = total;
    if (by_k) {
      bin_k = search(true, 0.0);
      o.left_k = r.k - found_count;
      o.before_k = found_mass;
      o.before = found_mass;
      low_sum = found_mass;
      // (the bin's own mass is at most its count at the upper edge)
      high_sum = found_mass + found_in * ldexp(exp2(-(double)(bin_k % 16) / 16.0), -(bin_k / 16));
      first = last = bin_k;
    }
    if (r.p < 1.0f) {
      // Bins in which top-p's cut can lie: rounding, and what top-k keeps of its own bin, leave a range.
      constexpr double kNear = 0x1p-30;
      const int hi = search(false, (double)r.p * low_sum * (1.0 - kNear));
      const double before = found_mass;
      const int lo = search(false, (double)r.p * high_sum * (1.0 + kNear));
      if (hi <= first) {
        first = hi;
        o.before = before;
      }
      last = min(last, lo);
      o.target = by_k ? (double)r.p : (double)r.p * total;
    }
    o.by_k = by_k;
    o.by_p = r.p < 1.0f;
    if (first < kBins) {
      o.first = first;
      o.last = last;
      if (by_k) o.bin_k = bin_k;
      // How many they are.
      u64 listed = 0;
      for (int i = tid; i < kBins; i += kThreads)
        if ((i >= first && i <= last) || (by_k && i == bin_k)) listed += counts[i];
      listed = block_add(listed, red);
      o.heavy = listed > kSampleList;
    }
  }
  if (tid == 0) *info = o;
}

// ------------------------------------------------------------- second launch

// 2^(x / 16) for x <= 0, as fp32: the exponent's whole part apart, so that the rest is
// exact to a few 2^-24.
__device__ __forceinline__ float weight_of(double x16) {
  const double x = x16 * 0.0625, n = rint(x);
  return ldexpf(__builtin_amdgcn_exp2f((float)(x - n)), (int)n);
}

// The race's key of a weight and its noise: the score's bits rise with it; 0 if it
// takes no part.
__device__ __forceinline__ u64 race_key(float w, float noise, int j) {
  const float s = w / noise;
  return w > 0.0f && s >= 0.0f ? ((u64)float_bits(s) << 32) | (uint32_t)~j : 0ull;
}

// A weight in units of the upper edge of a bin, in fixed point.
__device__ __forceinline__ u64 fixed_below(const RowInfo& o, double t, double bin) {
  return (u64)(exp2(below_edge(o, t, bin)) * (double)(1ull << kFixBits));
}

struct Scratch {
  u64 list[kSampleList];
  uint32_t counts[kSubs];
  u64 sums[kSubs];
  u64 red[kWaves];
  uint32_t redc[kWaves];
  double redd[kWaves];
  u64 found_sum;
  uint32_t found_count, listed;
  int found;
  uint32_t arrived;
};

// Every token of a row's list, or of the row itself.
template <bool F16, typename F>
__device__ __forceinline__ void each(const SampleArgs& a, const RowInfo& o, const void* row, const Scratch& s, F f) {
  if (!o.heavy) {
    for (uint32_t i = threadIdx.x; i < s.listed; i += kThreads) f(s.list[i]);
  } else {
    for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
      const float l = F16 ? (float)((const half_t*)row)[j] : ((const float*)row)[j];
      if (valid(l)) f(key_of(l, j));
    }
  }
}

// Of the tokens of bins `first` to `last`, in falling order: the key of the one at which
// the count reaches `count`, or the mass (in units of the upper edge, fixed point)
// `mass`; the last one if it never does.  Each step splits the tokens that are
// left by the eleven bits below those that they all share.
template <bool F16>
__device__ u64 select(const SampleArgs& a, const RowInfo& o, const void* row, Scratch& s, double first, double last,
                      bool by_count, uint32_t count, u64 mass) {
  const int tid = threadIdx.x;
  u64 mask = 0, value = 0;      // tokens left: key & mask == value
  auto here = [&](u64 k) {
    const double bin = bin_of(o, t_of(logit_of(k), o.c16));
    return bin >= first && bin <= last && (k & mask) == value;
  };
  for (;;) {
    u64 all = ~0ull, any = 0;
    each<F16>(a, o, row, s, [&](u64 k) {
      if (here(k)) {
        all &= k;
        any |= k;
      }
    });
    all = block_all(all, s.red, [](u64 x, u64 y) { return x & y; });
    any = block_all(any, s.red, [](u64 x, u64 y) { return x | y; });
    if (all == ~0ull && any == 0) return ~0ull;      // none at all
    if (all == any) return all;                       // one
    const int top = 63 - __builtin_clzll(all ^ any), shift = max(top - 10, 0);
    for (int i = tid; i < kSubs; i += kThreads) {
      s.counts[i] = 0;
      s.sums[i] = 0;
    }
    if (tid == 0) s.found = -1;
    __syncthreads();
    each<F16>(a, o, row, s, [&](u64 k) {
      if (here(k)) {
        const int sub = kSubs - 1 - (int)((k >> shift) & (kSubs - 1));     // the largest first
        atomicAdd(&s.counts[sub], 1u);
        if (!by_count)
          atomicAdd(&s.sums[sub], fixed_below(o, t_of(logit_of(k), o.c16), first));
      }
    });
    __syncthreads();
    constexpr int kOwn = kSubs / kThreads;
    uint32_t n[kOwn], n_own = 0;
    u64 m[kOwn], m_own = 0;
    int lowest = -1;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      n[i] = s.counts[tid * kOwn + i];
      m[i] = s.sums[tid * kOwn + i];
      n_own += n[i];
      m_own += m[i];
      if (n[i] > 0) lowest = tid * kOwn + i;
    }
    uint32_t n_to = block_run(n_own, s.redc) - n_own;
    u64 m_to = block_run(m_own, s.red) - m_own;
    const int end = (int)block_max((u64)(lowest + 1), s.red) - 1;     // the last that holds any
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const bool reaches = by_count ? n_to < count && n_to + n[i] >= count : m_to < mass && m_to + m[i] >= mass;
      if (reaches) {
        s.found = tid * kOwn + i;
        s.found_count = n_to;
        s.found_sum = m_to;
      }
      n_to += n[i];
      m_to += m[i];
    }
    __syncthreads();
    int sub = s.found;
    if (sub < 0) {
      sub = end;          // (the sums fall short by rounding: the last one)
      count = ~0u;
      mass = ~0ull;
    } else {
      count -= s.found_count;
      mass -= s.found_sum;
    }
    mask = ~((1ull << shift) - 1);
    value = (all & ~((2ull << top) - 1)) | ((u64)(kSubs - 1 - sub) << shift);
    if (top < 10) value = (all & ~(u64)(kSubs - 1)) | (u64)(kSubs - 1 - sub);
    __syncthreads();
  }
}

template <bool F16>
__global__ void __launch_bounds__(kThreads) sample_race_kernel(SampleArgs a) {
  __shared__ Scratch s;
  const int b = blockIdx.x / a.shares, share = blockIdx.x % a.shares, tid = threadIdx.x;
  RowInfo* info = (RowInfo*)((char*)a.info + (int64_t)b * kSampleInfoBytes);
  const RowInfo o = *info;
  if (o.kind != kRace) return;
  const void* row = row_of(a, b);
  const int beg = share * kSampleShare, end = min(beg + kSampleShare, a.vocab);
  float l[kEach];
  load_share<F16>(row, beg, end, l);
  if (tid == 0) s.listed = 0;
  __syncthreads();
  // Noise is read where a token is kept: elsewhere the load is out of its buffer.
  const __amdgpu_buffer_rsrc_t noise =
      make_rsrc(a.noise ? a.noise + (int64_t)b * a.vocab : nullptr, a.noise ? (uint32_t)a.vocab * 4u : 0u);
  float e[kEach];
  uint32_t kept = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const double t = t_of(l[i], o.c16);
    const double bin = bin_of(o, t);
    const bool sure = valid(l[i]) && bin < o.first && t - o.tm >= o.lim;
    kept |= (uint32_t)sure << i;
    const bool listed = !o.heavy && valid(l[i]) && ((bin >= o.first && bin <= o.last) || bin == o.bin_k);
    if (listed) {
      const uint32_t at = atomicAdd(&s.listed, 1u);
      if (at < kSampleList) s.list[at] = key_of(l[i], place(beg, i));
    }
    const uint32_t off = sure && a.noise ? 4u * (uint32_t)place(beg, i) : kOutOfRange;
    e[i] = bits_float(__builtin_amdgcn_raw_buffer_load_b32(noise, off, 0, 0));
  }
  u64 best = 0;
  double sum = 0.0;
  if (__any(kept != 0)) {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (kept >> i & 1) {
        const float w = weight_of(t_of(l[i], o.c16) - o.tm);
        sum += (double)w;
        if (a.noise) {
          const u64 k = race_key(w, e[i], place(beg, i));
          best = best > k ? best : k;
        }
      }
  }
  best = block_max(best, s.red);
  sum = block_all(sum, s.redd, [](double x, double y) { return x + y; });
  const uint32_t listed = min(s.listed, (uint32_t)kSampleList);
  ShareInfo* mine = a.share + (int64_t)b * a.shares + share;
  u64* list = a.list + (int64_t)b * kSampleList;
  if (a.shares > 1 && listed > 0) {
    __syncthreads();
    if (tid == 0) s.found_count = add_dev_u32(&info->listed, listed);
    __syncthreads();
    for (uint32_t i = tid; i < listed; i += kThreads)
      if (s.found_count + i < kSampleList) st64(&list[s.found_count + i], s.list[i]);
  }
  if (tid == 0) {
    st64(&mine->best, best);
    st64(&mine->number, (u64)__double_as_longlong(sum));
  }
  if (!last_of_row(a, b, &s.arrived)) return;

  ShareInfo* all = a.share + (int64_t)b * a.shares;
  best = 0;
  sum = 0.0;
  for (int i = tid; i < a.shares; i += kThreads) {
    const u64 v = ld64(&all[i].best);
    best = best > v ? best : v;
  }
  for (int i = 0; i < a.shares; ++i) sum += __longlong_as_double((long long)ld64(&all[i].number));   // (in order)
  u64 last = 0;
  if (o.by_k || o.by_p) {
    if (a.shares > 1) {
      const uint32_t n = min(ld_dev_u32(&info->listed), (uint32_t)kSampleList);
      for (uint32_t i = tid; i < n; i += kThreads) s.list[i] = ld64(&list[i]);
      if (tid == 0) s.listed = n;
    }
    __syncthreads();
    double target = o.target;
    if (o.by_k) {
      last = select<F16>(a, o, row, s, o.bin_k, o.bin_k, true, (uint32_t)o.left_k, 0);
      if (o.by_p) {
        // What top-k left of its bin, and with it top-p's mass.
        u64 part = 0;
        each<F16>(a, o, row, s, [&](u64 k) {
          const double t = t_of(logit_of(k), o.c16);
          if (bin_of(o, t) == o.bin_k && k >= last) part += fixed_below(o, t, o.bin_k);
        });
        part = block_add(part, s.red);
        target *= o.before_k + ldexp((double)part, -kFixBits) * exp2(-o.bin_k * 0.0625);
      }
    }
    if (o.by_p) {
      const double left = (target - o.before) * exp2(o.first * 0.0625);     // in units of the bins' upper edge
      const u64 mass = left > 0.0 ? (u64)fmin(ceil(left * (double)(1ull << kFixBits)), 0x1p62) : 1;
      const u64 by_p = select<F16>(a, o, row, s, o.first, o.last, false, 0, mass);
      last = last > by_p ? last : by_p;
    }
    // The tokens of these bins that are kept.
    u64 more = 0, more_sum = 0;
    each<F16>(a, o, row, s, [&](u64 k) {
      const double t = t_of(logit_of(k), o.c16);
      if (k >= last && bin_of(o, t) >= o.first && t - o.tm >= o.lim) {
        const float w = weight_of(t - o.tm);
        const int j = (int)~(uint32_t)k;
        more_sum += (u64)((double)w * 0x1p40);     // (a sum in fixed point has no order, as the list has none)
        if (a.noise) {
          const u64 v = race_key(w, a.noise[(int64_t)b * a.vocab + j], j);
          more = more > v ? more : v;
        }
      }
    });
    best = best > more ? best : more;
    sum += ldexp((double)block_add(more_sum, s.red), -40);
  }
  best = block_max(best, s.red);
  if (tid == 0) {
    if (a.tokens) a.tokens[b] = best ? (int)~(uint32_t)best : -1;
    info->end = last;
    info->inv = 1.0 / sum;
  }
}

// -------------------------------------------------------------- third launch

template <bool F16>
__global__ void __launch_bounds__(kThreads) sample_probs_kernel(SampleArgs a) {
  const int b = blockIdx.x / a.shares, share = blockIdx.x % a.shares;
  const RowInfo o = *(const RowInfo*)((const char*)a.info + (int64_t)b * kSampleInfoBytes);
  const int beg = share * kSampleShare, end = min(beg + kSampleShare, a.vocab);
  float l[kEach];
  if (o.kind == kRace) load_share<F16>(row_of(a, b), beg, end, l);
  const float inv = (float)o.inv;
  float p[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int j = place(beg, i);
    if (o.kind == kRace) {
      const double x = t_of(l[i], o.c16) - o.tm;
      p[i] = valid(l[i]) && x >= o.lim && key_of(l[i], j) >= o.end ? weight_of(x) * inv : 0.0f;
    } else {
      p[i] = j == o.token ? 1.0f : 0.0f;
    }
  }
  float* out = a.probs + (int64_t)b * a.vocab;
  if (end - beg == kSampleShare) {
#pragma unroll
    for (int i = 0; i < kEach; i += 4) *(f4u_t*)(out + place(beg, i)) = f4u_t{p[i], p[i + 1], p[i + 2], p[i + 3]};
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (place(beg, i) < end) out[place(beg, i)] = p[i];
  }
}

template <bool F16>
hipError_t launch(const SampleArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.shares)), block(kThreads);
  sample_bins_kernel<F16><<<grid, block, 0, s>>>(a);
  if (!a.only_first) sample_race_kernel<F16><<<grid, block, 0, s>>>(a);
  if (a.probs) sample_probs_kernel<F16><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

// Rows of one group: as many as the header has counters for, and shares whose
// histograms take no more than 64 MiB.
SampleShape sample_shape(const spear_sample_desc_t& d) {
  SampleShape s;
  s.shares = (int)ceil_div(d.vocab, kSampleShare);
  s.group = (int)std::max<int64_t>(1, std::min<int64_t>(d.batch, std::min<int64_t>(kMaxEcTiles, 4096 / s.shares)));
  size_t at = kSyncHeaderBytes;
  const size_t shares = (size_t)s.group * s.shares;
  s.info = at;
  at += (size_t)s.group * kSampleInfoBytes;
  s.share = at;
  at += shares * sizeof(ShareInfo);
  s.list = at;
  at += (size_t)s.group * kSampleList * 8;
  s.hist = at;
  at += shares * kBins * 8;
  s.bytes = at;
  return s;
}

hipError_t launch_sample(const SampleArgs& a, void* stream) {
  return a.f16 ? launch<true>(a, (hipStream_t)stream) : launch<false>(a, (hipStream_t)stream);
}

}  // namespace spear
