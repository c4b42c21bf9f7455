// The draw of next tokens with temperature, top-k, top-p and min-p, and the
// distribution that it draws from.
//
// The rules keep a prefix of the tokens in falling order of their logits, so what
// has to be found is where that order is cut: no sort of the vocabulary is needed,
// only the counts and sums of weights above a value.  A row's vocabulary is shared by
// workgroups, in two launches (three for probabilities):
//
//   1. Every share finds its maximum and, for top-k and top-p, a histogram of its
//      weights: 32 bins to a power of two, on one grid for the whole row
//      (t = 32 logit / (T ln 2); bin floor(t)), so that shares need no common
//      maximum first and the row is read once.  A bin holds its count and the sum of
//      its weights' distances from the bin's upper edge in fixed point, both in one
//      64-bit integer (one LDS atomic a token; integer sums have no order).  The
//      row's last share to arrive adds the histograms, sums counts and weights from the
//      top, and finds the bin in which each rule's cut lies.
//   2. Tokens above that bin are drawn from at once (an exponential race: the largest
//      weight / noise, ties to the lowest index), those in it (up to some hundreds) go
//      to a list; noise is read for tokens that are kept, and for no others.  The last
//      share to arrive sorts the list by (logit, index), cuts it by a running sum, ends the
//      race, and sums what is kept.
//   3. Probabilities are written.
//
// The sums decide which token is the last one, and in a flat distribution that token
// has a millionth of the total: weights enter the sums to 2^-34 of themselves, and
// sums are held in 64 bits.
//
// Longer lists are cut by a radix selection, and a bin that holds more tokens than the
// list (equal logits, a very high temperature) by the same selection over the row
// itself, by one workgroup: slow, and right.
#include <algorithm>

#include "serve_internal.h"
#include "device_common.h"

namespace spear {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / kWave;
constexpr int kPer = 32;                          // bins in a power of two
constexpr int kBins = 128 * kPer;
constexpr int kBinsEach = kBins / kThreads;
constexpr double kCut = -126.0 * kPer;            // weights below 2^-126 of the largest are zero
constexpr int kDefBits = 37;                      // fixed point of a bin's sum of distances
constexpr int kFixBits = 40;                      // fixed point of weights in a selection
constexpr int kRanked = kThreads;                 // tokens that are sorted by counting
constexpr int kStaged = 2 * kRanked;              // tokens of the list that a share gathers in LDS
constexpr int kSubs = 1024, kSubBits = 10;        // sub-bins of a selection's step
constexpr double kLn2 = 0.693147180559945309417;
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef float f4u_t __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 h4u_t __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned long long u64;

enum Kind : int32_t { kEmpty, kOne, kRace };      // no token, the first one, a race of several

// What a row's first launch leaves for the others.  t: kPer log2 of a weight, on the
// row's grid; bins are counted from the one of the row's largest; masses are in units
// of that bin's upper edge.  Every limit on t is a limit on the logit too: the least
// fp32 number whose t reaches it (NaN: there is none).
struct RowInfo {
  double scale, q;           // t of a logit of 1, and floor(t) of the row's largest
  double largest;            // the row's largest logit (the largest finite number for infinity)
  double before, before_k;   // mass before bin `first`, and before bin_k
  double target;             // top-p's mass if that is known; else (with top-k) p
  double edge;               // weight at the upper edge of bin `first`
  u64 end;                   // second launch: key of the last token kept (0: all)
  double inv;                // 1 / mass of what is kept, in units of the largest weight
  int32_t first, last;       // tokens of bins before `first` are kept, those of bins past `last` are not ..
  int32_t bin_k;             // .. and top-k's cut lies in this bin (one of them, or past them; -1: no such cut)
  float sure;                // logits from here on are kept (in bins before `first`, within min-p)
  float from, to;            // logits of the bins that are cut: [from, to) ..
  float from_k, to_k;        // .. and those of bin_k, if that lies past them
  float least;               // min-p: no logit below it is kept
  int32_t kind, token;       // token: the largest logit's
  int32_t left_k;            // tokens that top-k keeps of its bin
  int32_t by_k, by_p;        // which rules cut
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
__device__ __forceinline__ double t_of(float l, double scale) { return fmin((double)l * scale, 1e300); }
// The bin of a logit, from the one of the row's largest: whole numbers, exact wherever
// two bins are near each other.
__device__ __forceinline__ double bin_of(const RowInfo& o, float l) { return o.q - floor(t_of(l, o.scale)); }
// A weight in units of the upper edge of bin `bin`, in fixed point.
__device__ __forceinline__ u64 fixed_below(const RowInfo& o, float l, int bin) {
  const double x = ((t_of(l, o.scale) - o.q) + (bin - 1.0)) * (1.0 / kPer);
  return (u64)(exp2(x) * (double)(1ull << kFixBits));
}
// The weight relative to the row's largest, as fp32: the exponent's whole part apart, so
// that the rest is exact to a few 2^-24.  (The difference of the logits first: that of
// their products would be rounded as the products are.)
__device__ __forceinline__ double finite(float l) { return (double)fminf(l, 3.40282347e38f); }
__device__ __forceinline__ float weight_of(const RowInfo& o, float l) {
  const double x = (finite(l) - o.largest) * (o.scale * (1.0 / kPer)), n = rint(x);
  return ldexpf(__builtin_amdgcn_exp2f((float)(x - n)), (int)n);
}
// The least fp32 number with t_of(l, scale) >= t, NaN if there is none; not below the
// lowest finite one.  (The quotient, rounded to fp32, is at most two steps away.)
__device__ __forceinline__ float logit_from(double t, double scale) {
  const float near = (float)fmin(fmax(t / scale, -3.40282347e38), 1e300);
  uint32_t step = rising(near);
  step = step > rising(-3.40282347e38f) + 2 ? step - 2 : rising(-3.40282347e38f);
  for (int i = 0; i < 6; ++i, ++step) {
    const float l = logit_of((u64)step << 32);
    if (t_of(l, scale) >= t) return l;
    if (l == INFINITY) break;
  }
  return __builtin_nanf("");
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

// .. of two values at once.
__device__ __forceinline__ void block_run(double& x, uint32_t& y, double* ldsx, uint32_t* ldsy) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
#pragma unroll
  for (int o = 1; o < kWave; o *= 2) {
    const double p = __shfl_up(x, o);
    const uint32_t q = __shfl_up(y, o);
    if (lane >= o) {
      x += p;
      y += q;
    }
  }
  __syncthreads();
  if (lane == kWave - 1) {
    ldsx[wave] = x;
    ldsy[wave] = y;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWaves; ++i)
    if (i < wave) {
      x += ldsx[i];
      y += ldsy[i];
    }
}

// A thread's tokens of a share: vectors of four in turn, so that the lanes of a wave
// read and write runs of memory whatever the type.
__device__ __forceinline__ int place(int beg, int i) { return beg + 4 * ((i / 4) * kThreads + (int)threadIdx.x) + i % 4; }

// Vectors past the end are read within the row and count as -infinity; the one that
// crosses the end is read again, token by token.
template <bool F16, int EACH>
__device__ __forceinline__ void load_share(const void* row, int beg, int end, int vocab, float* l) {
  if (vocab >= 4) {
    if constexpr (F16) {
      h4u_t v[EACH / 4];
#pragma unroll
      for (int i = 0; i < EACH / 4; ++i) v[i] = *(const h4u_t*)((const half_t*)row + min(place(beg, 4 * i), vocab - 4));
#pragma unroll
      for (int i = 0; i < EACH; ++i) l[i] = (float)v[i / 4][i % 4];
    } else {
      f4u_t v[EACH / 4];
#pragma unroll
      for (int i = 0; i < EACH / 4; ++i) v[i] = *(const f4u_t*)((const float*)row + min(place(beg, 4 * i), vocab - 4));
#pragma unroll
      for (int i = 0; i < EACH; ++i) l[i] = v[i / 4][i % 4];
    }
  }
  if (end - beg < EACH * kThreads) {
#pragma unroll
    for (int i = 0; i < EACH; i += 4) {
      const int at = place(beg, i);
      if (at + 4 > end) {
#pragma unroll
        for (int j = 0; j < 4; ++j) l[i + j] = -INFINITY;
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (at + j < end) l[i + j] = F16 ? (float)((const half_t*)row)[at + j] : ((const float*)row)[at + j];
      }
    }
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
  drain_vm();
  __syncthreads();
  if (a.shares == 1) return true;
  if (threadIdx.x == 0) *arrived = add_dev_u32(&a.counters[b], 1u);
  __syncthreads();
  if (*arrived != (uint32_t)a.shares - 1) return false;
  if (threadIdx.x == 0) st_dev_u32(&a.counters[b], 0u);
  return true;
}

// -------------------------------------------------------------- first launch

// 2^(-i / kPer)
__device__ const double kSteps[kPer] = {
    1.0, 0.9785720620877001, 0.9576032806985737, 0.93708381705515,
    0.9170040432046712, 0.8973545375015536, 0.8781260801866497, 0.859309649061239,
    0.8408964152537145, 0.8228777390769825, 0.8052451659746271, 0.7879904225539432,
    0.7711054127039704, 0.7545822137967114, 0.7384130729697497, 0.7225904034885233,
    0.7071067811865476, 0.691954940981916, 0.6771277734684463, 0.6626183215798707,
    0.6484197773255048, 0.6345254785958666, 0.620928906036742, 0.6076236799902345,
    0.5946035575013605, 0.5818624293887887, 0.5693943173783458, 0.5571933712979462,
    0.5452538663326288, 0.5335702003384118, 0.5221368912137069, 0.5109485743270583};

// The weight at the upper edge of a bin, and a bin's mass.
__device__ __forceinline__ double edge_of(int bin) {
  return kSteps[bin % kPer] * __longlong_as_double((long long)(1023 - bin / kPer) << 52);
}
__device__ __forceinline__ double mass_of(int bin, uint32_t n, u64 def) {
  return edge_of(bin) * ((double)n - (double)def * (1.0 / (double)(1ull << kDefBits)));
}
constexpr double kNear = 0x1p-30;     // a mass this near to a target may lie on either side of it

template <bool F16, int EACH>
__global__ void __launch_bounds__(kThreads) sample_bins_kernel(SampleArgs a) {
  // One share's bins; then the row's: the mass up to and with each bin.
  __shared__ __attribute__((aligned(16))) u64 hist[kBins];
  __shared__ u64 red[kWaves];
  __shared__ double redd[kWaves];
  __shared__ uint32_t redc[kWaves];
  __shared__ short share_off[kThreads], share_used[kThreads];
  __shared__ uint32_t arrived, tokens_all, found_before;
  __shared__ int found;
  __shared__ float limits[6];
  const int b = blockIdx.x / a.shares, share = blockIdx.x % a.shares, tid = threadIdx.x;
  const Rules r = rules_of(a, b);
  const void* row = row_of(a, b);
  const bool bins = !r.one && (r.k > 0 || r.p < 1.0f);
  const int beg = share * EACH * kThreads, end = min(beg + EACH * kThreads, a.vocab);
  float l[EACH];
  u64 best = 0;
  uint32_t least = ~0u;
  if (row) load_share<F16, EACH>(row, beg, end, a.vocab, l);
  if (bins)
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
  if (row) {
    float top = -INFINITY, low = INFINITY;
    int at = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
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
  const double scale = fmax((double)kPer / ((double)r.t * kLn2), 1e-300);
  ShareInfo* mine = a.share + (int64_t)b * a.shares + share;
  if (bins && best != 0) {
    least = block_all(least, redc, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
    const double q = floor(t_of(logit_of(best), scale));
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const double t = t_of(l[i], scale), f = floor(t), rel = q - f;
      if (valid(l[i]) && rel < kBins) {
        // The weight's distance from the bin's upper edge, 1 - e^-u: u in 64 bits, the rest is below 2^-12.
        const double u = (1.0 - (t - f)) * (kLn2 / kPer);
        const float s = (float)u, h = s * s * (0.5f - s * (1.0f / 6.0f - s * (1.0f / 24.0f - s * (1.0f / 120.0f))));
        const double d = __builtin_fma(u, (double)(1ull << kDefBits), -(double)(h * (float)(1ull << kDefBits)));
        atomicAdd(&hist[(int)rel], ((u64)(1u << 16) << 32) | (uint32_t)d);
      }
    }
    const double span = q - floor(t_of(logit_of((u64)least << 32), scale)) + 1.0;
    const int used = span < kBins ? (int)span : kBins;
    u64* bins_out = a.hist + ((int64_t)b * a.shares + share) * kBins;
    __syncthreads();
    // The bins, and their sums: those of the row come from the shares' own.
    double mass = 0.0;
    uint32_t n = 0;
    for (int i = tid; i < used; i += kThreads) {
      const u64 v = hist[i];
      st64(&bins_out[i], v);
      mass += mass_of(i, (uint32_t)(v >> 48), v & ((1ull << 48) - 1));
      n += (uint32_t)(v >> 48);
    }
    mass = block_all(mass, redd, [](double x, double y) { return x + y; });
    n = block_all(n, redc, [](uint32_t x, uint32_t y) { return x + y; });
    if (tid == 0) {
      st64(&mine->number, (u64)__double_as_longlong(q));
      st64(&mine->mass, (u64)__double_as_longlong(mass));
      st64(&mine->used, (u64)n << 32 | (u64)used);
    }
  }
  if (tid == 0) st64(&mine->best, best);
  if (!last_of_row(a, b, &arrived)) return;

  // The row: its largest, ..
  static_assert((1 << 22) / (2 * kSampleLeast) <= kThreads, "a thread for every share");
  u64 number = 0, used = 0, mass_bits = 0;
  best = 0;
  if (tid < a.shares) {
    const ShareInfo* from = a.share + (int64_t)b * a.shares + tid;
    best = ld64(&from->best);
    number = ld64(&from->number);
    used = ld64(&from->used);
    mass_bits = ld64(&from->mass);
  }
  const bool any = best != 0;
  best = block_max(best, red);
  RowInfo* info = (RowInfo*)((char*)a.info + (int64_t)b * kSampleInfoBytes);
  static_assert(sizeof(RowInfo) <= kSampleInfoBytes, "room for it");
  const float largest = logit_of(best);
  RowInfo o;
  o.scale = scale;
  o.q = best ? floor(t_of(largest, scale)) : 0.0;
  o.largest = best ? finite(largest) : 0.0;
  o.before = o.before_k = o.target = 0.0;
  o.edge = o.inv = 1.0;
  o.end = 0;
  o.first = kBins;
  o.last = o.bin_k = -1;
  o.kind = best == 0 ? kEmpty : r.one ? kOne : kRace;
  o.token = best ? (int)~(uint32_t)best : -1;
  o.left_k = o.by_k = o.by_p = 0;
  o.listed = 0;
  if (o.kind != kRace) {
    if (tid == 0) {
      if (a.tokens) a.tokens[b] = o.token;
      *info = o;
    }
    return;
  }
  if (bins) {
    // .. the shares' places and sums, ..
    const double behind = o.q - __longlong_as_double((long long)number);
    const bool near = any && behind < kBins;
    const int off = near ? (int)behind : 0, have = near ? (int)(uint32_t)used : 0;
    if (tid < a.shares) {
      share_off[tid] = (short)off;
      share_used[tid] = (short)have;
    }
    const double part = near ? __longlong_as_double((long long)mass_bits) * edge_of(off) : 0.0;
    const double total = block_all(part, redd, [](double x, double y) { return x + y; });
    const uint32_t tokens = block_all(near ? (uint32_t)(used >> 32) : 0u, redc, [](uint32_t x, uint32_t y) { return x + y; });
    const int rows = (int)block_max((u64)min(off + have, kBins), red);   // bins of the row
    const bool by_k = r.k > 0 && (uint32_t)r.k < tokens;
    // .. and its bins from the top, a thread each, until they hold all that the rules ask for.
    const double ask = r.p < 1.0f ? (double)r.p * total * (1.0 + kNear) : 0.0;
    const u64* from = a.hist + (int64_t)b * a.shares * kBins;
    constexpr int kTogether = 8;      // shares whose loads are in flight together
    double mass_before = 0.0;
    uint32_t tokens_before = 0;
    int turns = 0;
    do {
      const int bin = turns * kThreads + tid;
      uint32_t n = 0;
      u64 def = 0;
      for (int s0 = 0; s0 < a.shares; s0 += kTogether) {
        u64 v[kTogether];
#pragma unroll
        for (int s = 0; s < kTogether; ++s) {
          const int of = min(s0 + s, a.shares - 1), at = bin - share_off[of];
          v[s] = s0 + s < a.shares && at >= 0 && at < share_used[of] ? ld64(&from[(int64_t)of * kBins + at]) : 0;
        }
#pragma unroll
        for (int s = 0; s < kTogether; ++s) {
          n += (uint32_t)(v[s] >> 48);
          def += v[s] & ((1ull << 48) - 1);
        }
      }
      double mass_to = mass_of(bin, n, def);
      uint32_t tokens_to = n;
      block_run(mass_to, tokens_to, redd, redc);
      mass_to += mass_before;
      tokens_to += tokens_before;
      hist[bin] = (u64)__double_as_longlong(mass_to);
      if (by_k && tokens_to >= (uint32_t)r.k && tokens_to - n < (uint32_t)r.k) {
        found = bin;
        found_before = tokens_to - n;
      }
      if (tid == kThreads - 1) tokens_all = tokens_to;
      __syncthreads();
      ++turns;
      mass_before = __longlong_as_double((long long)hist[turns * kThreads - 1]);
      tokens_before = tokens_all;
      __syncthreads();
      // (uniform: all threads have the same sums)
    } while (turns < kBinsEach && turns * kThreads < rows && (by_k ? tokens_before < (uint32_t)r.k : mass_before < ask));
    auto mass_up_to = [&](int bin) { return bin < 0 ? 0.0 : __longlong_as_double((long long)hist[bin]); };
    int bin_k = kBins, first = kBins, last = kBins;
    double low_sum = total, high_sum = total;
    if (by_k) {
      bin_k = found;
      o.left_k = r.k - (int)found_before;
      o.before_k = o.before = low_sum = mass_up_to(bin_k - 1);
      high_sum = mass_up_to(bin_k);
      first = last = bin_k;
    }
    if (r.p < 1.0f) {
      // Bins in which top-p's cut can lie: rounding, and what top-k keeps of its own bin, leave a range.
      // (As many bins as hold less than a mass up to and with them, and the next one.)
      const double low = (double)r.p * low_sum * (1.0 - kNear), high = (double)r.p * high_sum * (1.0 + kNear);
      int hi = 0, lo = 0;
      for (int i = 0; i < turns; ++i) {
        const double m = mass_up_to(i * kThreads + tid);
        hi += __syncthreads_count(m < low);
        lo += __syncthreads_count(m < high);
      }
      hi = min(hi, turns * kThreads - 1);
      if (hi <= first) {
        first = hi;
        o.before = mass_up_to(hi - 1);
      }
      last = min(last, min(lo, turns * kThreads - 1));
      o.target = by_k ? (double)r.p : (double)r.p * total;
    }
    o.by_k = by_k;
    o.by_p = r.p < 1.0f;
    if (first < kBins) {
      o.first = first;
      o.last = last;
      o.edge = edge_of(first);
      if (by_k) o.bin_k = bin_k;
    }
  }
  // The limits as logits, a thread each.
  if (tid < 6) {
    const double tm = t_of(largest, scale), lim = fmax(r.m > 0.0f ? (double)kPer * log2((double)r.m) : kCut, kCut);
    const double above = o.q - o.first + 1.0;        // of bins before `first`
    double t = 0.0;
    bool none = false;
    if (tid == 0) t = tm + lim;
    if (tid == 1) {
      t = o.first < kBins ? fmax(above, tm + lim) : tm + lim;
      none = o.first == 0;
    }
    if (tid == 2) {
      t = o.q - o.last;
      none = o.first >= kBins;
    }
    if (tid == 3) {
      t = above;
      none = o.first == 0;         // (nothing lies above the first bin)
    }
    if (tid == 4) {
      t = o.q - o.bin_k;
      none = o.bin_k <= o.last;
    }
    if (tid == 5) t = o.q - o.bin_k + 1.0;
    limits[tid] = none ? __builtin_nanf("") : logit_from(t, scale);
  }
  __syncthreads();
  if (tid == 0) {
    o.least = limits[0];
    o.sure = limits[1];
    o.from = limits[2];
    o.to = limits[3];
    o.from_k = limits[4];
    o.to_k = limits[5];
    *info = o;
  }
}

// ------------------------------------------------------------- second launch

// The race's key of a weight and its noise: the score's bits rise with it; 0 if it
// takes no part.
__device__ __forceinline__ u64 race_key(float w, float noise, int j) {
  const float s = w / noise;
  return w > 0.0f && s >= 0.0f ? ((u64)float_bits(s) << 32) | (uint32_t)~j : 0ull;
}

struct Scratch {
  __attribute__((aligned(16))) u64 list[kStaged];     // a share's tokens; then the row's, if they are kRanked at most
  u64 sums[kSubs];
  uint32_t counts[kSubs];
  u64 sorted_key[kRanked];
  u64 red[kWaves];
  uint32_t redc[kWaves];
  double redd[kWaves];
  u64 found_sum;
  uint32_t found_count, listed;
  int found;
  uint32_t arrived;
};

// Every token of a row's list, or of the row itself if the list does not hold its n.
template <bool F16, typename F>
__device__ __forceinline__ void each(const SampleArgs& a, const void* row, const u64* list, uint32_t n, F f) {
  if (n <= kSampleList) {
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) f(ld64(&list[i]));
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
// left by the ten bits below those that they all share.
template <bool F16>
__device__ u64 select(const SampleArgs& a, const RowInfo& o, const void* row, const u64* list, uint32_t listed,
                      Scratch& s, int first, int last, bool by_count, uint32_t count, u64 mass) {
  const int tid = threadIdx.x;
  u64 mask = 0, value = 0;      // tokens left: key & mask == value
  auto here = [&](u64 k) {
    const double bin = bin_of(o, logit_of(k));
    return bin >= first && bin <= last && (k & mask) == value;
  };
  for (;;) {
    u64 all = ~0ull, any = 0;
    each<F16>(a, row, list, listed, [&](u64 k) {
      if (here(k)) {
        all &= k;
        any |= k;
      }
    });
    all = block_all(all, s.red, [](u64 x, u64 y) { return x & y; });
    any = block_all(any, s.red, [](u64 x, u64 y) { return x | y; });
    if (all == ~0ull && any == 0) return ~0ull;      // none at all
    if (all == any) return all;                       // one
    const int top = 63 - __builtin_clzll(all ^ any), shift = max(top - (kSubBits - 1), 0);
    for (int i = tid; i < kSubs; i += kThreads) {
      s.counts[i] = 0;
      s.sums[i] = 0;
    }
    if (tid == 0) s.found = -1;
    __syncthreads();
    each<F16>(a, row, list, listed, [&](u64 k) {
      if (here(k)) {
        const int sub = kSubs - 1 - (int)((k >> shift) & (kSubs - 1));     // the largest first
        atomicAdd(&s.counts[sub], 1u);
        if (!by_count)
          atomicAdd(&s.sums[sub], fixed_below(o, logit_of(k), first));
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
    if (top < kSubBits - 1) value = (all & ~(u64)(kSubs - 1)) | (u64)(kSubs - 1 - sub);
    __syncthreads();
  }
}

// The cuts among the n <= kRanked tokens of the list, all of them at once: every token's
// place in the order by counting those before it (two threads to a token where they
// are few), the masses before it by a running sum in that order.
struct Cut {
  u64 end;          // key of the last token kept (~0: none of these)
  u64 best, sum;    // the race among those kept, and their mass in fixed point
};
__device__ __forceinline__ Cut cut_ranked(const SampleArgs& a, const RowInfo& o, int b, Scratch& s, int n) {
  const int tid = threadIdx.x;
  u64* sorted = s.sums;
  float* sorted_noise = (float*)(sorted + kRanked);
  static_assert(kSubs >= kRanked + kRanked / 2, "room for both");
  const int parts = n <= kThreads / 2 ? 2 : 1, own = tid % (kThreads / parts), part = tid / (kThreads / parts);
  const u64 key = own < n ? s.list[own] : 0;
  const float* noise = a.noise ? a.noise + (int64_t)b * a.vocab : nullptr;
  float e = 0.0f;
  if (noise && own < n && part == 0) e = noise[(int)~(uint32_t)key];
  const float own_l = logit_of(key);
  const u64 own_mass = own < n && part == 0 ? fixed_below(o, own_l, o.first) : 0;
  if (tid < n) s.counts[tid] = 0;
  if (tid == 0 && n % 2) s.list[n] = 0;      // (read in pairs)
  __syncthreads();
  if (own < n) {
    const int pairs = (n + 1) / 2, half = (pairs + parts - 1) / parts, to = min((part + 1) * half, pairs);
    uint32_t before = 0;
#pragma unroll 4
    for (int j = part * half; j < to; ++j) {
      const u64 x = s.list[2 * j], y = s.list[2 * j + 1];
      before += (x > key ? 1u : 0u) + (y > key ? 1u : 0u);
    }
    atomicAdd(&s.counts[own], before);
  }
  __syncthreads();
  if (own < n && part == 0) {
    const uint32_t at = s.counts[own];
    sorted[at] = own_mass;
    sorted_noise[at] = e;
    s.sorted_key[at] = key;
  }
  __syncthreads();
  const bool here = tid < n;
  const u64 k = here ? s.sorted_key[tid] : 0, mass = here ? sorted[tid] : 0;
  const float l = logit_of(k);
  const int bin = here ? (int)bin_of(o, l) : kBins;
  bool kept = here && bin <= o.last;
  double target = o.target;
  const double unit = o.edge * (1.0 / (double)(1ull << kFixBits));
  if (o.by_k) {
    const int ahead = __syncthreads_count(here && bin < o.bin_k);
    const bool of_k = here && (bin < o.bin_k || tid - ahead < o.left_k);
    kept &= of_k;
    if (o.by_p) target *= o.before_k + (double)block_add(of_k && bin == o.bin_k ? mass : 0, s.red) * unit;
  }
  if (o.by_p) {
    const u64 to = block_run(mass, s.red);
    kept &= o.before + (double)(to - mass) * unit < target;
  }
  const int many = __syncthreads_count(kept);
  Cut c;
  c.end = many > 0 ? s.sorted_key[many - 1] : ~0ull;
  c.best = c.sum = 0;
  if (kept && l >= o.least) {
    const float w = weight_of(o, l);
    c.sum = (u64)((double)w * 0x1p40);
    if (noise) c.best = race_key(w, sorted_noise[tid], (int)~(uint32_t)k);
  }
  return c;
}

// The same for any number of tokens, by selections.
template <bool F16>
__device__ Cut cut_selected(const SampleArgs& a, const RowInfo& o, const void* row, int b, const u64* list,
                            uint32_t listed, Scratch& s) {
  Cut c = {0, 0, 0};
  double target = o.target;
  if (o.by_k) {
    c.end = select<F16>(a, o, row, list, listed, s, o.bin_k, o.bin_k, true, (uint32_t)o.left_k, 0);
    if (o.by_p) {
      // What top-k left of its bin, and with it top-p's mass.
      u64 part = 0;
      each<F16>(a, row, list, listed, [&](u64 k) {
        if (bin_of(o, logit_of(k)) == o.bin_k && k >= c.end) part += fixed_below(o, logit_of(k), o.bin_k);
      });
      part = block_add(part, s.red);
      target *= o.before_k + ldexp((double)part, -kFixBits) * edge_of(o.bin_k);
    }
  }
  if (o.by_p) {
    const double left = (target - o.before) / o.edge;     // in units of the bins' upper edge
    const u64 mass = left > 0.0 ? (u64)fmin(ceil(left * (double)(1ull << kFixBits)), 0x1p62) : 1;
    const u64 by_p = select<F16>(a, o, row, list, listed, s, o.first, o.last, false, 0, mass);
    c.end = c.end > by_p ? c.end : by_p;
  }
  each<F16>(a, row, list, listed, [&](u64 k) {
    const float l = logit_of(k);
    if (k >= c.end && bin_of(o, l) >= o.first && l >= o.least) {
      const float w = weight_of(o, l);
      const int j = (int)~(uint32_t)k;
      c.sum += (u64)((double)w * 0x1p40);     // (a sum in fixed point has no order, as the list has none)
      if (a.noise) {
        const u64 v = race_key(w, a.noise[(int64_t)b * a.vocab + j], j);
        c.best = c.best > v ? c.best : v;
      }
    }
  });
  return c;
}

template <bool F16, int EACH>
__global__ void __launch_bounds__(kThreads) sample_race_kernel(SampleArgs a) {
  __shared__ Scratch s;
  const int b = blockIdx.x / a.shares, share = blockIdx.x % a.shares, tid = threadIdx.x;
  const void* row = row_of(a, b);
  const int beg = share * EACH * kThreads, end = min(beg + EACH * kThreads, a.vocab);
  float l[EACH];
  if (row) load_share<F16, EACH>(row, beg, end, a.vocab, l);     // (requested before the row's kind is known)
  RowInfo* info = (RowInfo*)((char*)a.info + (int64_t)b * kSampleInfoBytes);
  const RowInfo o = *info;
  if (o.kind != kRace) return;
  if (tid == 0) s.listed = 0;
  __syncthreads();
  u64* list = a.list + (int64_t)b * kSampleList;
  // Noise is read where a token is kept: elsewhere the load is out of its buffer.
  const __amdgpu_buffer_rsrc_t noise =
      make_rsrc(a.noise ? a.noise + (int64_t)b * a.vocab : nullptr, a.noise ? (uint32_t)a.vocab * 4u : 0u);
  u64 best = 0;
  double sum = 0.0;
  uint32_t kept = 0, cut = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    kept |= (uint32_t)(l[i] >= o.sure) << i;
    cut |= (uint32_t)((l[i] >= o.from && !(l[i] >= o.to)) || (l[i] >= o.from_k && !(l[i] >= o.to_k))) << i;
  }
  if (__any(kept != 0)) {
    float e[EACH];
#pragma unroll
    for (int i = 0; i < EACH; i += 4) {
      const int at = place(beg, i);
      const bool some = (kept >> i & 15) && a.noise;
      const f4_t v = __builtin_bit_cast(f4_t, __builtin_amdgcn_raw_buffer_load_b128(
          noise, some && at + 4 <= end ? 4u * (uint32_t)at : kOutOfRange, 0, 0));
#pragma unroll
      for (int j = 0; j < 4; ++j) e[i + j] = v[j];
      if (end - beg < EACH * kThreads && some && at + 4 > end) {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (at + j < end) e[i + j] = a.noise[(int64_t)b * a.vocab + at + j];
      }
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const float w = kept >> i & 1 ? weight_of(o, l[i]) : 0.0f;
      sum += (double)w;
      const u64 k = a.noise ? race_key(w, e[i], place(beg, i)) : 0;
      best = best > k ? best : k;
    }
  }
  if (cut != 0) {
#pragma unroll
    for (int i = 0; i < EACH; ++i)
      if (cut >> i & 1) {
        const u64 k = key_of(l[i], place(beg, i));
        const uint32_t at = atomicAdd(&s.listed, 1u);
        if (at < kStaged) {
          s.list[at] = k;
        } else {
          const uint32_t to = add_dev_u32(&info->listed, 1u);
          if (to < kSampleList) st64(&list[to], k);
        }
      }
  }
  best = block_max(best, s.red);
  sum = block_all(sum, s.redd, [](double x, double y) { return x + y; });
  const uint32_t staged = min(s.listed, (uint32_t)kStaged);
  ShareInfo* mine = a.share + (int64_t)b * a.shares + share;
  if (staged > 0) {
    if (tid == 0) s.found_count = add_dev_u32(&info->listed, staged);
    __syncthreads();
    for (uint32_t i = tid; i < staged; i += kThreads)
      if (s.found_count + i < kSampleList) st64(&list[s.found_count + i], s.list[i]);
  }
  if (tid == 0) {
    st64(&mine->best, best);
    st64(&mine->number, (u64)__double_as_longlong(sum));
  }
  if (!last_of_row(a, b, &s.arrived)) return;

  best = 0;
  sum = 0.0;
  const bool cuts = o.by_k || o.by_p;
  uint32_t n = 0;
  u64 key = 0;
  if (cuts) {
    n = ld_dev_u32(&info->listed);
    key = ld64(&list[tid]);           // (with the count: which of them are tokens is known then)
  }
  if (tid < a.shares) {
    const ShareInfo* from = a.share + (int64_t)b * a.shares + tid;
    best = ld64(&from->best);
    sum = __longlong_as_double((long long)ld64(&from->number));
  }
  sum = block_all(sum, s.redd, [](double x, double y) { return x + y; });     // (always in the same order)
  u64 last = 0;
  if (cuts) {
    Cut c;
    if (n <= kRanked) {
      if (tid < (int)n) s.list[tid] = key;
      __syncthreads();
      c = cut_ranked(a, o, b, s, (int)n);
    } else {
      c = cut_selected<F16>(a, o, row, b, list, n, s);
    }
    last = c.end;
    best = best > c.best ? best : c.best;
    sum += ldexp((double)block_add(c.sum, s.red), -40);
  }
  best = block_max(best, s.red);
  if (tid == 0) {
    if (a.tokens) a.tokens[b] = best ? (int)~(uint32_t)best : -1;
    info->end = last;
    info->inv = 1.0 / sum;
  }
}

// -------------------------------------------------------------- third launch

template <bool F16, int EACH>
__global__ void __launch_bounds__(kThreads) sample_probs_kernel(SampleArgs a) {
  const int b = blockIdx.x / a.shares, share = blockIdx.x % a.shares;
  const void* row = row_of(a, b);
  const int beg = share * EACH * kThreads, end = min(beg + EACH * kThreads, a.vocab);
  float l[EACH], p[EACH];
  if (row) load_share<F16, EACH>(row, beg, end, a.vocab, l);
  const RowInfo o = *(const RowInfo*)((const char*)a.info + (int64_t)b * kSampleInfoBytes);
  bool some = false;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    if (o.kind == kRace) some |= l[i] >= o.least;
    p[i] = o.kind == kOne && place(beg, i) == o.token ? 1.0f : 0.0f;
  }
  if (__any(some)) {
    const float inv = (float)o.inv;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const bool kept = l[i] >= o.sure || (l[i] >= o.least && key_of(l[i], place(beg, i)) >= o.end);
      p[i] = kept ? weight_of(o, l[i]) * inv : 0.0f;
    }
  }
  float* out = a.probs + (int64_t)b * a.vocab;
#pragma unroll
  for (int i = 0; i < EACH; i += 4) {
    const int at = place(beg, i);
    if (at + 4 <= end) {
      *(f4u_t*)(out + at) = f4u_t{p[i], p[i + 1], p[i + 2], p[i + 3]};
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (at + j < end) out[at + j] = p[i + j];
    }
  }
}

template <bool F16, int EACH>
hipError_t launch(const SampleArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.shares)), block(kThreads);
  sample_bins_kernel<F16, EACH><<<grid, block, 0, s>>>(a);
  if (!a.only_first) sample_race_kernel<F16, EACH><<<grid, block, 0, s>>>(a);
  if (a.probs) sample_probs_kernel<F16, EACH><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_share(const SampleArgs& a, hipStream_t s) {
  return a.share_tokens == 8 * kThreads ? launch<F16, 8>(a, s) : launch<F16, 16>(a, s);
}

}  // namespace

// Shares of 8192 tokens (4096 where the batch has few), as many of a row as a
// workgroup has threads; rows of one group: as many as the header has counters for, and
// shares whose bins take no more than 128 MiB.
SampleShape sample_shape(const spear_sample_desc_t& d) {
  SampleShape s;
  const int64_t large = kSampleLeast * 2;
  s.share_tokens = (int)(d.batch * ceil_div(d.vocab, kSampleLeast) <= 512 ? kSampleLeast : large);
  s.shares = (int)ceil_div(d.vocab, s.share_tokens);
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
  return a.f16 ? launch_share<true>(a, (hipStream_t)stream) : launch_share<false>(a, (hipStream_t)stream);
}

}  // namespace spear
