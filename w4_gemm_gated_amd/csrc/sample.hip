// The draw of next tokens with temperature, top-k, top-p and min-p, and the
// distribution that it draws from.
//
// The rules keep a prefix of the tokens in falling order of their logits, so what
// has to be found is where that order is cut: no sort of the vocabulary is needed,
// only the counts and sums of weights above a value.  Launches:
//
//   bins   A workgroup a share of a row: its maximum and, for top-k and top-p, a
//          histogram of its weights: 32 bins to a power of two, on one grid for the
//          whole row (t = 32 logit / (T ln 2); bin floor(t)), so that shares need no
//          common maximum first and the row is read once.  A bin holds its count and
//          the sum of its weights' distances from the bin's upper edge in fixed point,
//          both in one 64-bit integer (one LDS atomic a token; integer sums have no
//          order).
//   cuts   A workgroup a row: adds the shares' bins from the top until they hold what
//          the rules ask for, finds the bin in which each rule's cut lies, and turns the
//          limits on t into limits on the logit, which cost the next launches one
//          comparison a token.
//   race   A workgroup a part of a row: tokens above that bin are drawn from at once (an
//          exponential race: the largest weight / noise, ties to the lowest index),
//          those in it (up to some hundreds) go to a list; noise is read where tokens are
//          kept or listed, and nowhere else.
//   end    A workgroup a row: sorts the list by (logit, index), cuts it by a running
//          sum, ends the race, and sums what is kept.
//   probs  Probabilities, if they are asked for.
//
// A row that is a single share (up to 16384 tokens) has its cuts found in the launch of its
// bins, one that is a single part (up to 4096) ends in the launch of its race: 16 x 1000
// tokens take 12.4 us in two launches, 17.3 in four.
//
// The sums decide which token is the last one, and in a flat distribution that token
// has a millionth of the total: weights enter the sums to 2^-33 of themselves (five fp32
// roundings of a term below 2^-12; past |l| / T = 2^20 the product t, rounded to 64 bits, is
// off by more), and sums are held in 64 bits.
//
// What a call takes (replayed from a graph): 2 x 32000 tokens 18 us, a chain of four
// launches of 3 to 5 us, whatever they do; 64 x 128001 fp16 logits under mixed rules 43:
// 13 for the bins (23 vector instructions a token for the histogram, 14 of them in 64 bits,
// some ten for the row's largest and least, and 4.5 us of launch, loads and exchanges), 8 for the cuts (a row's bins are read by one CU), 13 for the race (logits
// and the noise's lines at 3 TB/s), 9 for the ends; distributions of 144 x 32000 tokens
// 40.  The launches' shapes follow from how fast one CU goes, which is
// some 25 bytes a ns whatever the pattern.
//
// Longer lists are cut by a radix selection, and a bin that holds more tokens than the
// list (equal logits, a very high temperature) by the same selection over the row
// itself, by one workgroup: 64 x 128001 tokens within 0.05 of each other take 290 us.
#include <algorithm>
#include <type_traits>

#include "serve_internal.h"
#include "wave_ops.h"

namespace spear {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / kWave;
constexpr int kPer = 32;                          // bins in a power of two
constexpr int kBins = 128 * kPer;
constexpr double kCut = -126.0 * kPer;            // weights below 2^-126 of the largest are zero
constexpr int kDefBits = 37;                      // fixed point of a bin's sum of distances
constexpr int kFixBits = 40;                      // fixed point of weights in a selection
constexpr int kRanked = kThreads / 2;             // tokens that are sorted by counting
constexpr int kStaged = 1024;                 // tokens of the list that a share gathers in LDS
constexpr int kSubs = 1024, kSubBits = 10;        // sub-bins of a selection's step
constexpr double kLn2 = 0.693147180559945309417;
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef float f4u_t __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 h4u_t __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned long long u64;

enum Kind : int32_t { kEmpty, kOne, kRace };      // no token, the first one, a race of several

// What the cuts leave of a row for the launches after them.  t: kPer log2 of a weight, on the
// row's grid; bins are counted from the one of the row's largest; masses are in units
// of that bin's upper edge.  Every limit on t is a limit on the logit too: the least
// fp32 number whose t reaches it (NaN: there is none).
struct RowInfo {
  double scale, q;           // t of a logit of 1, and floor(t) of the row's largest
  double largest;            // the row's largest logit (the largest finite number for infinity)
  double before, before_k;   // mass before bin `first`, and before bin_k
  double target;             // top-p's mass if that is known; else (with top-k) p
  double edge;               // weight at the upper edge of bin `first`
  u64 end;                   // from the row's end: key of the last token kept (0: all)
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
  int32_t finer;             // a selection by mass counts in units of 2^-(kFixBits + finer) of `edge`
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
// 2^(-i / kPer)  (correctly rounded)
__device__ const double kSteps[kPer] = {
    0x1.0000000000000p+0, 0x1.f50765b6e4540p-1, 0x1.ea4afa2a490dap-1, 0x1.dfc97337b9b5fp-1,
    0x1.d5818dcfba487p-1, 0x1.cb720dcef9069p-1, 0x1.c199bdd85529cp-1, 0x1.b7f76f2fb5e47p-1,
    0x1.ae89f995ad3adp-1, 0x1.a5503b23e255dp-1, 0x1.9c49182a3f090p-1, 0x1.93737b0cdc5e5p-1,
    0x1.8ace5422aa0dbp-1, 0x1.82589994cce13p-1, 0x1.7a11473eb0187p-1, 0x1.71f75e8ec5f74p-1,
    0x1.6a09e667f3bcdp-1, 0x1.6247eb03a5585p-1, 0x1.5ab07dd485429p-1, 0x1.5342b569d4f82p-1,
    0x1.4bfdad5362a27p-1, 0x1.44e086061892dp-1, 0x1.3dea64c123422p-1, 0x1.371a7373aa9cbp-1,
    0x1.306fe0a31b715p-1, 0x1.29e9df51fdee1p-1, 0x1.2387a6e756238p-1, 0x1.1d4873168b9aap-1,
    0x1.172b83c7d517bp-1, 0x1.11301d0125b51p-1, 0x1.0b5586cf9890fp-1, 0x1.059b0d3158574p-1};

// The weight at the upper edge of a bin.  (`steps`: kSteps in LDS, a round trip to memory less.)
__device__ __forceinline__ double edge_of(const double* steps, int bin) {
  return steps[bin % kPer] * __longlong_as_double((long long)(1023 - bin / kPer) << 52);
}
// The distance of a weight from its bin's upper edge, 1 - e^-u with u = ln 2 / kPer below
// `in` = t - floor(t), times 2^kDefBits: u in 64 bits, the rest is below 2^-12.
__device__ __forceinline__ double distance(double in) {
  const double u = (1.0 - in) * (kLn2 / kPer);
  const float s = (float)u, h = s * s * (0.5f - s * (1.0f / 6.0f - s * (1.0f / 24.0f)));
  return __builtin_fma(u, (double)(1ull << kDefBits), -(double)(h * (float)(1ull << kDefBits)));
}
// A weight in units of the upper edge of bin `bin`, its own or one above it, in fixed point.
__device__ __forceinline__ u64 fixed_below(const RowInfo& o, const double* steps, float l, int bin, double fine = 1.0) {
  const double t = t_of(l, o.scale), f = floor(t);
  const double w = (double)(1ull << kFixBits) - distance(t - f) * (double)(1 << (kFixBits - kDefBits));
  return (u64)(w * edge_of(steps, min((int)(o.q - f) - bin, kBins - 1)) * fine);
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

// The workgroup's maximum, bitwise and / or, and sum, in every thread.  (`none`: what leaves
// any value as it is.)
template <typename T, typename F>
__device__ __forceinline__ T block_all(T v, T none, T* lds, F f) {
  v = wave_all(v, none, f);
  __syncthreads();
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) v = f(v, lds[i]);
  return v;
}
__device__ __forceinline__ u64 block_max(u64 v, u64* lds) {
  return block_all(v, (u64)0, lds, [](u64 a, u64 b) { return a > b ? a : b; });
}
__device__ __forceinline__ u64 block_add(u64 v, u64* lds) {
  return block_all(v, (u64)0, lds, [](u64 a, u64 b) { return a + b; });
}

// Running sum (inclusive) over the workgroup.
template <typename T>
__device__ __forceinline__ T block_run(T v, T* lds) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  v = wave_run(v);
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
  x = wave_run(x);
  y = wave_run(y);
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

__device__ __forceinline__ double scale_of(const Rules& r) { return fmax((double)kPer / ((double)r.t * kLn2), 1e-300); }

__device__ __forceinline__ const void* row_of(const SampleArgs& a, int b) {
  const int64_t r = a.rows ? a.rows[b] : a.first + b;
  if (r < 0 || r >= a.num_rows) return nullptr;
  return (const char*)a.logits + r * a.stride * (a.f16 ? 2 : 4);
}

// ------------------------------------------------------------- bins and cuts

// (`step`: kSteps of the bin, the same for all of a thread's)
static_assert(kThreads % kPer == 0, "a thread's bins have one place in their powers of two");
__device__ __forceinline__ double mass_of(int bin, double step, uint32_t n, u64 def) {
  return step * __longlong_as_double((long long)(1023 - bin / kPer) << 52) * ((double)n - (double)def * (1.0 / (double)(1ull << kDefBits)));
}
constexpr double kNear = 0x1p-30;     // a mass this near to a target may lie on either side of it

struct BinsScratch {
  u64 hist[kBins];
  u64 red[kWaves];
  double redd[kWaves];
  uint32_t redc[kWaves], tokens[kWaves];
};
struct CutScratch {
  double steps[kPer];
  double redd[kWaves];
  uint32_t redc[kWaves];
  short share_off[kSampleShares], share_used[kSampleShares];
  uint32_t tokens_all, found_before;
  int found, hi, lo;
  float limits[6];
};

// From a row's shares: its largest, and the bins in which the cuts lie.  `mine`: the share of
// this lane's number; bin_of_row(bin, n, def) adds what the shares have in a bin of the
// row's; mass_to: the row's mass (the bits of a double) up to and with each bin.
template <typename F>
__device__ __forceinline__ void find_cuts(const SampleArgs& a, int b, const Rules& r, ShareInfo mine, double scale,
                                          double step, CutScratch& s, u64* mass_to, F bin_of_row) {
  const int tid = threadIdx.x;
  const bool bins = !r.one && (r.k > 0 || r.p < 1.0f);
  // The row: its largest, ..
  // (every wave for itself: a share a lane, or several)
  const ShareInfo* shares = a.share + (int64_t)b * a.shares;
  const int lane = tid % kWave;
  u64 best = mine.best;
  for (int i = lane + kWave; i < a.shares; i += kWave) best = best > shares[i].best ? best : shares[i].best;
  best = wave_max(best, (u64)0);
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
  o.finer = 0;
  if (o.kind != kRace) {
    if (tid == 0) {
      if (a.tokens) a.tokens[b] = o.token;
      *info = o;
    }
    return;
  }
  if (bins) {
    // .. the shares' places and sums, ..
    double total = 0.0;
    uint32_t tokens = 0;
    int rows = 0;        // bins of the row
    for (int i = lane; i < a.shares; i += kWave) {
      if (i >= kWave) mine = shares[i];
      const double behind = o.q - __longlong_as_double((long long)mine.number);
      const bool near = mine.best != 0 && behind < kBins;
      const int off = near ? (int)behind : 0, have = near ? (int)(uint32_t)mine.used : 0;
      s.share_off[i] = (short)off;
      s.share_used[i] = (short)have;
      total += near ? __longlong_as_double((long long)mine.mass) * edge_of(s.steps, off) : 0.0;
      tokens += near ? (uint32_t)(mine.used >> 32) : 0u;
      rows = max(rows, min(off + have, kBins));
    }
    total = wave_sum(total);
    tokens = wave_sum(tokens);
    rows = wave_max(rows, 0);
    __syncthreads();
    bool by_k = r.k > 0 && (uint32_t)r.k < tokens;
    // .. and its bins from the top, one to a thread, until they hold all that the rules ask
    // for (one CU reads them: bins that need not be read are time saved).
    const double ask = r.p < 1.0f ? (double)r.p * total * (1.0 + kNear) : 0.0;
    auto mass_up_to = [&](int bin) { return bin < 0 ? 0.0 : __longlong_as_double((long long)mass_to[bin]); };
    double mass_before = 0.0;
    uint32_t tokens_before = 0;
    int bins_read = 0;
    do {
      const int bin = bins_read + tid;
      uint32_t n = 0;
      u64 def = 0;
      bin_of_row(bin, n, def);
      double to = mass_of(bin, step, n, def);
      uint32_t tokens_to = n;
      block_run(to, tokens_to, s.redd, s.redc);
      tokens_to += tokens_before;
      mass_to[bin] = (u64)__double_as_longlong(to + mass_before);
      if (by_k && tokens_to >= (uint32_t)r.k && tokens_to - n < (uint32_t)r.k) {
        s.found = bin;
        s.found_before = tokens_to - n;
      }
      if (tid == kThreads - 1) s.tokens_all = tokens_to;
      __syncthreads();
      bins_read += kThreads;
      mass_before = mass_up_to(bins_read - 1);
      tokens_before = s.tokens_all;
      __syncthreads();
      // (uniform: all threads have the same sums)
    } while (bins_read < rows && (by_k ? tokens_before < (uint32_t)r.k : mass_before < ask));
    // (a share whose own largest is far below the row's counts tokens that weigh nothing here)
    by_k = by_k && tokens_before >= (uint32_t)r.k;
    int bin_k = kBins, first = kBins, last = kBins;
    double low_sum = total, high_sum = total;
    if (by_k) {
      bin_k = s.found;
      o.left_k = r.k - (int)s.found_before;
      o.before_k = o.before = low_sum = mass_up_to(bin_k - 1);
      high_sum = mass_up_to(bin_k);
      first = last = bin_k;
    }
    if (r.p < 1.0f) {
      // Bins in which top-p's cut can lie: rounding, and what top-k keeps of its own bin, leave a range.
      // (As many bins as hold less than a mass up to and with them, and the next one.)
      const double low = (double)r.p * low_sum * (1.0 - kNear), high = (double)r.p * high_sum * (1.0 + kNear);
      if (tid == 0) s.hi = s.lo = bins_read - 1;
      __syncthreads();
      for (int i = tid; i < bins_read; i += kThreads) {        // (the masses rise)
        const double m = mass_up_to(i), before = mass_up_to(i - 1);
        if (m >= low && (before < low || i == 0)) s.hi = i;
        if (m >= high && (before < high || i == 0)) s.lo = i;
      }
      __syncthreads();
      const int hi = s.hi, lo = s.lo;
      if (hi <= first) {
        first = hi;
        o.before = mass_up_to(hi - 1);
      }
      last = min(last, lo);
      o.target = by_k ? (double)r.p : (double)r.p * total;
    }
    o.by_k = by_k;
    o.by_p = r.p < 1.0f;
    if (first < kBins) {
      o.first = first;
      o.last = last;
      o.edge = edge_of(s.steps, first);
      // A selection adds the masses of bins `first` to `last`, and where these are several in
      // units no coarser than keep the sum below 2^62.  (With a top-k that cuts far below, light
      // tokens by the thousand may follow a heavy one, each a few 2^-40 of its bin's edge.)
      if (first < last) {
        const double most = fmax(mass_up_to(last) * (1.0 + kNear) - mass_up_to(first - 1), o.edge);
        const int power = (int)((__double_as_longlong(most) >> 52) - (__double_as_longlong(o.edge) >> 52));
        o.finer = max(20 - power, 0);
      }
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
    s.limits[tid] = none ? __builtin_nanf("") : logit_from(t, scale);
  }
  __syncthreads();
  if (tid == 0) {
    o.least = s.limits[0];
    o.sure = s.limits[1];
    o.from = s.limits[2];
    o.to = s.limits[3];
    o.from_k = s.limits[4];
    o.to_k = s.limits[5];
    *info = o;
  }
}

// ONE: a row is a single share, whose cuts are found at once, from the bins in LDS.
template <bool F16, int EACH, bool ONE>
__global__ void __launch_bounds__(kThreads) sample_bins_kernel(SampleArgs a) {
  __shared__ BinsScratch s;
  __shared__ std::conditional_t<ONE, CutScratch, char> cut;
  const int b = blockIdx.x / a.shares, share = blockIdx.x % a.shares, tid = threadIdx.x;
  const Rules r = rules_of(a, b);
  const void* row = row_of(a, b);
  const bool bins = !r.one && (r.k > 0 || r.p < 1.0f);
  const int beg = share * EACH * kThreads, end = min(beg + EACH * kThreads, a.vocab);
  const double step = kSteps[tid % kPer];
  float l[EACH];
  u64 best = 0;
  uint32_t least = ~0u;
  if (row) load_share<F16, EACH>(row, beg, end, a.vocab, l);
  if (bins)
    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
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
  best = wave_max(best, (u64)0);
  least = wave_all(least, ~0u, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
  if (tid % kWave == 0) {
    s.red[tid / kWave] = best;
    s.redc[tid / kWave] = least;
  }
  __syncthreads();      // (and the bins are cleared)
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    best = best > s.red[i] ? best : s.red[i];
    least = least < s.redc[i] ? least : s.redc[i];
  }
  const double scale = scale_of(r);
  ShareInfo mine = {best, 0, 0, 0};
  if (bins && best != 0) {
    const double q = floor(t_of(logit_of(best), scale));
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const double t = t_of(l[i], scale), f = floor(t), rel = q - f;
      if (valid(l[i]) && rel < kBins) {
        atomicAdd(&s.hist[(int)rel], ((u64)(1u << 16) << 32) | (uint32_t)distance(t - f));
      }
    }
    const double span = q - floor(t_of(logit_of((u64)least << 32), scale)) + 1.0;
    const int used = span < kBins ? (int)span : kBins;
    __syncthreads();
    // The bins, and their sums: those of the row come from the shares' own.
    double mass = 0.0;
    uint32_t n = 0;
    for (int i = tid; i < used; i += kThreads) {
      const u64 v = s.hist[i];
      if constexpr (!ONE) a.hist[((int64_t)b * a.shares + share) * kBins + i] = v;
      mass += mass_of(i, step, (uint32_t)(v >> 48), v & ((1ull << 48) - 1));
      n += (uint32_t)(v >> 48);
    }
    mass = wave_sum(mass);
    n = wave_sum(n);
    if (tid % kWave == 0) {
      s.redd[tid / kWave] = mass;
      s.tokens[tid / kWave] = n;
    }
    __syncthreads();
    mass = s.redd[0];
    n = s.tokens[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) {
      mass += s.redd[i];
      n += s.tokens[i];
    }
    mine = {best, (u64)__double_as_longlong(q), (u64)__double_as_longlong(mass), (u64)n << 32 | (u64)used};
  }
  if constexpr (ONE) {
    if (tid < kPer) cut.steps[tid] = step;
    __syncthreads();
    // (a thread's bins give way to the masses up to them)
    find_cuts(a, b, r, mine, scale, step, cut, s.hist, [&](int bin, uint32_t& n, u64& def) {
      n = (uint32_t)(s.hist[bin] >> 48);
      def = s.hist[bin] & ((1ull << 48) - 1);
    });
  } else {
    if (tid == 0) a.share[(int64_t)b * a.shares + share] = mine;
  }
}

__global__ void __launch_bounds__(kThreads) sample_cuts_kernel(SampleArgs a) {
  __shared__ CutScratch s;
  __shared__ u64 mass_to[kBins];
  const int b = blockIdx.x;
  const ShareInfo mine = a.share[(int64_t)b * a.shares + min((int)threadIdx.x % kWave, a.shares - 1)];
  const Rules r = rules_of(a, b);
  const double step = kSteps[threadIdx.x % kPer];
  if (threadIdx.x < kPer) s.steps[threadIdx.x] = step;
  __syncthreads();
  const u64* from = a.hist + (int64_t)b * a.shares * kBins;
  find_cuts(a, b, r, mine, scale_of(r), step, s, mass_to, [&](int bin, uint32_t& n, u64& def) {
    constexpr int kTogether = 8;      // shares whose loads are in flight together
    for (int i0 = 0; i0 < a.shares; i0 += kTogether) {
      u64 v[kTogether];
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        const int of = min(i0 + i, a.shares - 1), at = bin - s.share_off[of];
        v[i] = i0 + i < a.shares && at >= 0 && at < s.share_used[of] ? from[(int64_t)of * kBins + at] : 0;
      }
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        n += (uint32_t)(v[i] >> 48);
        def += v[i] & ((1ull << 48) - 1);
      }
    }
  });
}

// --------------------------------------------------------- race and its end

// The race's key of a weight and its noise: the score's bits rise with it; 0 if it
// takes no part.
__device__ __forceinline__ u64 race_key(float w, float noise, int j) {
  const float s = w / noise;
  return w > 0.0f && s >= 0.0f ? ((u64)float_bits(s) << 32) | (uint32_t)~j : 0ull;
}

// What a share needs in LDS; and what the end of a row needs beside it.
struct Staged {
  __attribute__((aligned(16))) u64 list[kStaged];     // a share's tokens; then the row's, if they are kRanked at most
  float noise[kStaged];           // of these tokens
  u64 red[kWaves];
  double redd[kWaves];
  uint32_t found_count, listed;
};
struct Scratch : Staged {
  u64 sums[kSubs];
  uint32_t counts[kSubs];
  u64 sorted_key[kRanked];
  double steps[kPer];
  uint32_t redc[kWaves];
  u64 found_sum;
  int found;
};

// Every token of a row's list, or of the row itself if the list does not hold its n.
template <bool F16, typename F>
__device__ __forceinline__ void each(const SampleArgs& a, const void* row, const u64* list, uint32_t n, F f) {
  if (n <= kSampleList) {
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) f(list[i]);
  } else {
    constexpr int kOwn = 16;
#pragma unroll 1
    for (int beg = 0; beg < a.vocab; beg += kOwn * kThreads) {
      float l[kOwn];
      load_share<F16, kOwn>(row, beg, min(beg + kOwn * kThreads, a.vocab), a.vocab, l);
#pragma unroll 1
      for (int i = 0; i < kOwn; i += 4) {        // (f is long)
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if (valid(l[n])) f(key_of(l[n], place(beg, i) + n));
#pragma unroll
        for (int n = 0; n + 4 < kOwn; ++n) l[n] = l[n + 4];
      }
    }
  }
}

// A wave's own sorting: the place of each of its first n lanes' keys, largest first
// (other lanes keep theirs), values moved to their places, and running sums.
__device__ __forceinline__ int place_in_wave(u64 key, int n) {
  const int lane = threadIdx.x % kWave;
  int at = 0;
  for (int j = 0; j < n; ++j) at += of_lane(key, j) > key;
  return lane < n ? at : lane;
}
__device__ __forceinline__ uint32_t push(uint32_t v, int to) { return (uint32_t)__builtin_amdgcn_ds_permute(4 * to, (int)v); }
__device__ __forceinline__ u64 push(u64 v, int to) { return (u64)push((uint32_t)(v >> 32), to) << 32 | push((uint32_t)v, to); }
// Of the tokens of bins `first` to `last`, in falling order: the key of the one at which
// the count reaches `count`, or the mass (in the row's units, fixed point) `mass`; the last one if it never does.  Each step splits the tokens that are
// left by the ten bits below those that they all share.
template <bool F16>
__device__ u64 select(const SampleArgs& a, const RowInfo& o, const void* row, const u64* list, uint32_t listed,
                      Scratch& s, int first, int last, bool by_count, uint32_t count, u64 mass, double fine) {
  const int tid = threadIdx.x;
  u64 mask = 0, value = 0;      // tokens left: key & mask == value
  // The bins as logits.  (Top-k's is one of several that top-p's cut may lie in, or past them.)
  float low = o.from, high = o.to;
  if (first > o.last) {
    low = o.from_k;
    high = o.to_k;
  } else if (first != o.first || last != o.last) {
    low = logit_from(o.q - last, o.scale);
    high = first == 0 ? __builtin_nanf("") : logit_from(o.q - first + 1.0, o.scale);
  }
  auto here = [&](u64 k) {
    const float l = logit_of(k);
    return l >= low && !(l >= high) && (k & mask) == value;
  };
  for (;;) {
    u64 all = ~0ull, any = 0;
    each<F16>(a, row, list, listed, [&](u64 k) {
      if (here(k)) {
        all &= k;
        any |= k;
      }
    });
    all = block_all(all, ~0ull, s.red, [](u64 x, u64 y) { return x & y; });
    any = block_all(any, 0ull, s.red, [](u64 x, u64 y) { return x | y; });
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
        if (!by_count) atomicAdd(&s.sums[sub], fixed_below(o, s.steps, logit_of(k), first, fine));
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
    const uint32_t left = s.counts[sub];
    mask = ~((1ull << shift) - 1);
    value = (all & ~((2ull << top) - 1)) | ((u64)(kSubs - 1 - sub) << shift);
    if (top < kSubBits - 1) value = (all & ~(u64)(kSubs - 1)) | (u64)(kSubs - 1 - sub);
    __syncthreads();
    if (left <= kWave) {
      // Few are left: every wave sorts them for itself.
      if (tid == 0) s.found_count = 0;
      __syncthreads();
      each<F16>(a, row, list, listed, [&](u64 k) {
        if (here(k)) s.sorted_key[atomicAdd(&s.found_count, 1u)] = k;
      });
      __syncthreads();
      const int lane = tid % kWave, n = (int)s.found_count;
      u64 key = lane < n ? s.sorted_key[lane] : 0;
      key = push(key, place_in_wave(key, n));
      u64 before = lane < n && !by_count ? fixed_below(o, s.steps, logit_of(key), first, fine) : 0;
      const u64 own = before;
      before = wave_run(before) - own;
      const bool in = lane < n && (by_count ? (uint32_t)lane < count : before < mass);
      return of_lane(key, max(__popcll(__ballot(in)) - 1, 0));
    }
  }
}

struct Cut {
  u64 end;          // key of the last token kept (~0: none of these)
  u64 best, sum;    // the race among those kept, and their mass in fixed point
};

// The cuts among a list of no more tokens than a wave has lanes: every wave for itself,
// without a barrier.
__device__ __forceinline__ Cut cut_in_wave(const SampleArgs& a, const RowInfo& o, const double* steps, int n, u64 key,
                                           float noise) {
  const int lane = threadIdx.x % kWave;
  const bool here = lane < n;
  const int to = place_in_wave(key, n);
  key = push(here ? key : 0, to);
  noise = bits_float(push(float_bits(noise), to));
  const float l = logit_of(key);
  const int bin = here ? (int)bin_of(o, l) : kBins;
  const u64 mass = here ? fixed_below(o, steps, l, o.first) : 0;
  bool kept = here && bin <= o.last;
  double target = o.target;
  const double unit = o.edge * (1.0 / (double)(1ull << kFixBits));
  if (o.by_k) {
    const int ahead = __popcll(__ballot(here && bin < o.bin_k));
    const bool of_k = here && (bin < o.bin_k || lane - ahead < o.left_k);
    kept &= of_k;
    if (o.by_p)
      target *= o.before_k + (double)of_lane(wave_run(of_k && bin == o.bin_k ? mass : 0), kWave - 1) * unit;
  }
  if (o.by_p) kept &= o.before + (double)(wave_run(mass) - mass) * unit < target;
  const int many = __popcll(__ballot(kept));
  Cut c;
  c.end = many > 0 ? of_lane(key, many - 1) : ~0ull;
  c.best = c.sum = 0;
  if (kept && l >= o.least) {
    const float w = weight_of(o, l);
    c.sum = (u64)((double)w * 0x1p40);
    if (a.noise) c.best = race_key(w, noise, (int)~(uint32_t)key);
  }
  return c;
}

// The cuts among the n <= kRanked tokens of the list: every token's place in the order by
// counting those before it, the masses before it by a running sum in that order.
__device__ __forceinline__ Cut cut_ranked(const SampleArgs& a, const RowInfo& o, Scratch& s, int n) {
  const int tid = threadIdx.x;
  u64* sorted = s.sums;
  float* sorted_noise = (float*)(sorted + kRanked);
  static_assert(kSubs >= kRanked + kRanked / 2, "room for both");
  const int own = tid % kRanked, part = tid / kRanked;       // two threads to a token
  const u64 key = own < n ? s.list[own] : 0;
  const float e = own < n ? s.noise[own] : 0.0f;
  const float own_l = logit_of(key);
  const u64 own_mass = own < n && part == 0 ? fixed_below(o, s.steps, own_l, o.first) : 0;
  if (tid < n) s.counts[tid] = 0;
  if (tid == 0 && n % 2) s.list[n] = 0;      // (read in pairs)
  __syncthreads();
  if (own < n) {
    const int pairs = (n + 1) / 2, half = (pairs + 1) / 2, to = min((part + 1) * half, pairs);
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
    if (a.noise) c.best = race_key(w, sorted_noise[tid], (int)~(uint32_t)k);
  }
  return c;
}

// The same for any number of tokens, by selections.
template <bool F16>
__device__ Cut cut_selected(const SampleArgs& a, const RowInfo& o, const void* row, int b, const u64* list,
                            uint32_t listed, Scratch& s) {
  Cut c = {0, 0, 0};
  const double fine = (double)(1 << o.finer);
  double target = o.target;
#pragma unroll 1
  for (int rule = 0; rule < 2; ++rule) {       // top-k, then top-p
    const bool by_count = rule == 0;
    if (!(by_count ? o.by_k : o.by_p)) continue;
    const double left = (target - o.before) / o.edge;     // top-p's mass in units of the bins' upper edge
    const u64 mass = left > 0.0 ? (u64)fmin(ceil(left * ((double)(1ull << kFixBits) * fine)), 0x1p62) : 1;
    const u64 end = select<F16>(a, o, row, list, listed, s, by_count ? o.bin_k : o.first, by_count ? o.bin_k : o.last,
                                by_count, (uint32_t)o.left_k, mass, fine);
    c.end = c.end > end ? c.end : end;
    if (by_count && o.by_p) {
      // What top-k left of its bin, and with it top-p's mass.
      u64 part = 0;
      each<F16>(a, row, list, listed, [&](u64 k) {
        if (bin_of(o, logit_of(k)) == o.bin_k && k >= c.end) part += fixed_below(o, s.steps, logit_of(k), o.bin_k);
      });
      part = block_add(part, s.red);
      target *= o.before_k + ldexp((double)part, -kFixBits) * edge_of(s.steps, o.bin_k);
    }
  }
  // The mass of what is kept.  A list has no order, so its terms are whole numbers, whose sum has
  // none either (4094 of them lose 2^-28 of the row's largest at most).  Of a row every thread
  // adds the same tokens in the same order, and their parts below 2^-40 count: a long row's
  // light tokens, cut off there, are missed by all that they hold together (4 million of
  // 1.99 2^-40 each: 2^-18).
  const bool whole = listed <= kSampleList;
  double sum = 0.0;
  each<F16>(a, row, list, listed, [&](u64 k) {
    const float l = logit_of(k);
    if (k >= c.end && !(l >= o.to) && l >= o.least) {
      const float w = weight_of(o, l);
      const int j = (int)~(uint32_t)k;
      const double term = (double)w * 0x1p40;
      sum += whole ? floor(term) : term;
      if (a.noise) {
        const u64 v = race_key(w, a.noise[(int64_t)b * a.vocab + j], j);
        c.best = c.best > v ? c.best : v;
      }
    }
  });
  c.sum = (u64)sum;
  return c;
}

// The list of n tokens cut, and the race's end.  key, e: the list's first tokens, one to a lane;
// best, sum: the race and the mass of what is kept without it, over a wave's lanes.  With
// n <= kWave one wave, else all.
template <bool F16>
__device__ __forceinline__ void end_row(const SampleArgs& a, int b, const RowInfo& o, RowInfo* info, const u64* list,
                                        const float* list_noise, uint32_t n, u64 key, float e, u64 best, double sum,
                                        Scratch& s) {
  const int tid = threadIdx.x, lane = tid % kWave;
  Cut c = {0, 0, 0};
  bool split = false;       // whether c is each thread's part, or each wave's whole
  if (o.by_k || o.by_p) {
    if (n <= kWave) {
      c = cut_in_wave(a, o, s.steps, (int)n, key, e);
    } else if (n <= kRanked) {
      if (tid < (int)n) {
        s.list[tid] = list[tid];
        s.noise[tid] = list_noise[tid];
      }
      __syncthreads();
      c = cut_ranked(a, o, s, (int)n);
      split = true;
    } else {
      c = cut_selected<F16>(a, o, row_of(a, b), b, list, n, s);
      split = true;
    }
  }
  best = best > c.best ? best : c.best;
  best = wave_max(best, (u64)0);
  sum = wave_sum(sum);
  c.sum = wave_sum(c.sum);
  if (split) {
    __syncthreads();
    if (lane == 0) {
      s.red[tid / kWave] = best;
      s.sums[tid / kWave] = c.sum;
    }
    __syncthreads();
    c.sum = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      best = best > s.red[i] ? best : s.red[i];
      c.sum += s.sums[i];
    }
  }
  sum += ldexp((double)c.sum, -40);
  if (tid == 0) {
    if (a.tokens) a.tokens[b] = best ? (int)~(uint32_t)best : -1;
    info->end = c.end;
    info->inv = 1.0 / sum;
  }
}

// From a row's parts and list: the list cut, and the race's end.
template <bool F16>
__device__ __forceinline__ void end_race(const SampleArgs& a, int b, Scratch& s) {
  const int tid = threadIdx.x;
  RowInfo* info = (RowInfo*)((char*)a.info + (int64_t)b * kSampleInfoBytes);
  const u64* list = a.list + (int64_t)b * kSampleList;
  const float* list_noise = a.list_noise + (int64_t)b * kSampleList;
  const int lane = tid % kWave;
  // The row, and what its list's first tokens and its parts are if it has any: all of it
  // requested at once, every wave for itself.
  const u64 key = list[lane];
  const float e = list_noise[lane];
  const PartInfo* parts = a.part + (int64_t)b * a.parts;
  PartInfo from = parts[min(lane, a.parts - 1)];
  const RowInfo o = *info;
  if (tid < kPer) s.steps[tid] = kSteps[tid];
  if (o.kind != kRace) return;
  const uint32_t n = o.by_k || o.by_p ? o.listed : 0;
  if (n <= kWave && tid >= kWave) return;         // one wave does what there is
  u64 best = 0;
  double sum = 0.0;
  for (int i = lane; i < a.parts; i += kWave) {
    if (i >= kWave) from = parts[i];
    best = best > from.best ? best : from.best;
    sum += from.mass;
  }
  if (n > kWave) __syncthreads();
  else __builtin_amdgcn_wave_barrier();           // (a wave's LDS operations are in order)
  end_row<F16>(a, b, o, info, list, list_noise, n, key, e, best, sum, s);
}

// ONE: a row is a single part, which ends at once.
template <bool F16, bool ONE>
__global__ void __launch_bounds__(kThreads) sample_race_kernel(SampleArgs a) {
  constexpr int EACH = kSampleLeast / kThreads;
  __shared__ std::conditional_t<ONE, Scratch, Staged> s;
  const int b = blockIdx.x / a.parts, part = blockIdx.x % a.parts, tid = threadIdx.x;
  const void* row = row_of(a, b);
  const int beg = part * EACH * kThreads, end = min(beg + EACH * kThreads, a.vocab);
  float l[EACH];
  if (row) load_share<F16, EACH>(row, beg, end, a.vocab, l);     // (requested before the row's kind is known)
  RowInfo* info = (RowInfo*)((char*)a.info + (int64_t)b * kSampleInfoBytes);
  const RowInfo o = *info;
  if (o.kind != kRace) return;
  if (tid == 0) s.listed = 0;
  if constexpr (ONE)
    if (tid < kPer) s.steps[tid] = kSteps[tid];
  __syncthreads();
  u64* list = a.list + (int64_t)b * kSampleList;
  float* list_noise = a.list_noise + (int64_t)b * kSampleList;
  // Noise is read where a token is kept or listed: elsewhere the load is out of its buffer.
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
  if (__any((kept | cut) != 0)) {
    float e[EACH];
#pragma unroll
    for (int i = 0; i < EACH; i += 4) {
      const int at = place(beg, i);
      const bool some = ((kept | cut) >> i & 15) && a.noise;
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
    if (__any(kept != 0)) {
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
            s.noise[at] = e[i];
          } else if constexpr (!ONE) {
            const uint32_t to = add_dev_u32(&info->listed, 1u);
            if (to < kSampleList) list[to] = k;      // (a list this long is cut without its noise)
          }
        }
    }
  }
  best = wave_max(best, (u64)0);
  sum = wave_sum(sum);
  if (tid % kWave == 0) {
    s.red[tid / kWave] = best;
    s.redd[tid / kWave] = sum;
  }
  __syncthreads();
  if constexpr (ONE) {
    // (a list that LDS does not hold: the row itself)
    const uint32_t n = s.listed <= kStaged ? s.listed : kSampleList + 1;
    if (n <= kWave && tid >= kWave) return;
    const int lane = tid % kWave;
    best = lane < kWaves ? s.red[lane] : 0;
    sum = lane < kWaves ? s.redd[lane] : 0.0;
    end_row<F16>(a, b, o, info, s.list, s.noise, n, s.list[lane], s.noise[lane], best, sum, s);
    return;
  }
  const uint32_t staged = min(s.listed, (uint32_t)kStaged);
  if (tid == 0) {
    if (staged > 0) s.found_count = add_dev_u32(&info->listed, staged);
    for (int i = 1; i < kWaves; ++i) {
      best = best > s.red[i] ? best : s.red[i];
      sum += s.redd[i];
    }
    a.part[(int64_t)b * a.parts + part] = {best, sum};
  }
  if (staged > 0) {
    __syncthreads();
    for (uint32_t i = tid; i < staged; i += kThreads)
      if (s.found_count + i < kSampleList) {
        list[s.found_count + i] = s.list[i];
        list_noise[s.found_count + i] = s.noise[i];
      }
  }
}

template <bool F16>
__global__ void __launch_bounds__(kThreads) sample_end_kernel(SampleArgs a) {
  __shared__ Scratch s;
  end_race<F16>(a, blockIdx.x, s);
}

// --------------------------------------------------------- the distributions

template <bool F16>
__global__ void __launch_bounds__(kThreads) sample_probs_kernel(SampleArgs a) {
  constexpr int EACH = kSampleLeast / kThreads;
  const int b = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const void* row = row_of(a, b);
  const int beg = part * EACH * kThreads, end = min(beg + EACH * kThreads, a.vocab);
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
  const dim3 grid((unsigned)(a.batch * a.shares)), parts((unsigned)(a.batch * a.parts)), rows((unsigned)a.batch),
      block(kThreads);
  if (a.shares == 1) {
    sample_bins_kernel<F16, EACH, true><<<grid, block, 0, s>>>(a);
  } else {
    sample_bins_kernel<F16, EACH, false><<<grid, block, 0, s>>>(a);
    sample_cuts_kernel<<<rows, block, 0, s>>>(a);
  }
  if (!a.only_first) {
    if (a.parts == 1) {
      sample_race_kernel<F16, true><<<parts, block, 0, s>>>(a);
    } else {
      sample_race_kernel<F16, false><<<parts, block, 0, s>>>(a);
      sample_end_kernel<F16><<<rows, block, 0, s>>>(a);
    }
  }
  if (a.probs) sample_probs_kernel<F16><<<parts, block, 0, s>>>(a);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_share(const SampleArgs& a, hipStream_t s) {
  return a.share_tokens == 8 * kThreads    ? launch<F16, 8>(a, s)
         : a.share_tokens == 16 * kThreads ? launch<F16, 16>(a, s)
                                           : launch<F16, 32>(a, s);
}

}  // namespace

// Shares of 4096, 8192 or 16384 tokens: the bins take what the fullest CU has to
// do (0.36 us per 1024 tokens and 0.3 per workgroup), and the workgroup that sums a row's
// bins 0.35 us per share (shares of 4096 and 8192: 2 x 32000 tokens 17.6 and 18.3 us,
// 144 x 32000 41.5 and 39.8).  A row of one share saves that launch (16 x 1000 tokens 17.3
// and 14.8 us, 16 x 8000 17.6 and 16.3, 16 x 16000 17.8 in four shares and 18.4 in one).  Rows of one group: up to 4096 shares, whose bins take 128 MiB;
// their lists take 48 KiB a row.  What stays in LDS (the bins of rows of one share, the lists
// of rows of one part) has no place in the workspace.
SampleShape sample_shape(const spear_sample_desc_t& d) {
  SampleShape s;
  constexpr int kCus = 256;
  double least = 0.0;
  for (int tokens = kSampleLeast; tokens <= 4 * kSampleLeast; tokens *= 2) {
    const int64_t shares = ceil_div(d.vocab, tokens);
    const double us = (0.36 * std::min(tokens, d.vocab) / 1024 + 0.3) * (double)ceil_div(d.batch * shares, kCus) +
                      (shares > 1 ? 2.7 + 0.35 * (double)shares : 0.0);
    if (shares <= kSampleShares && (least == 0.0 || us < least)) {
      least = us;
      s.share_tokens = tokens;
      s.shares = (int)shares;
    }
  }
  s.group = (int)std::max<int64_t>(1, std::min<int64_t>(d.batch, std::min<int64_t>(kMaxEcTiles, 4096 / s.shares)));
  size_t at = kSyncHeaderBytes;
  const size_t shares = (size_t)s.group * s.shares;
  s.info = at;
  at += (size_t)s.group * kSampleInfoBytes;
  s.parts = (int)ceil_div(d.vocab, kSampleLeast);
  const size_t listed = s.parts > 1 ? (size_t)s.group : 0, binned = s.shares > 1 ? shares : 0;      // rows, shares
  s.share = at;
  at += binned * sizeof(ShareInfo);
  s.part = at;
  at += listed * s.parts * sizeof(PartInfo);
  s.list = at;
  at += listed * kSampleList * 8;
  s.hist = at;
  at += binned * kBins * 8;
  s.list_noise = at;
  at += listed * kSampleList * 4;
  s.bytes = at;
  return s;
}

hipError_t launch_sample(const SampleArgs& a, void* stream) {
  return a.f16 ? launch_share<true>(a, (hipStream_t)stream) : launch_share<false>(a, (hipStream_t)stream);
}

}  // namespace spear
