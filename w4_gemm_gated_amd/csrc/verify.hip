// Verification of drafted tokens (speculative sampling).
//
// Acceptance needs one probability per drafted token; the draw of the next
// token needs one row of the target's and the draft's probabilities and of
// the noise.  So the rows of the other positions are never read, and the
// kernel is bound by one pass over those three rows (or, for a few sequences,
// by latency).  `splits` workgroups share a sequence: each finds the number of
// accepted tokens by itself (a few scattered loads, no exchange) and scans its
// share of the vocabulary.  The race's winner is the maximum of the 64-bit
// keys (score bits, ~index): scores are not negative, so their bits rise with
// them, and ties go to the lowest index whatever the order of the workgroups.
// The last workgroup of a sequence to arrive takes the maximum over the
// others' and writes the token.  Measured: 64 sequences of 128,001 entries in
// 19.2 us (98 MB, 5.1 TB/s with the start and the exchange; 23 with the noise
// requested after the count and vectors past a share's end read one by one), 2 of
// 32,000 in 6.3 us.
//
// A residual that is zero everywhere (p <= q at every entry although a token
// was refused: only rounding makes it so) is rare; the last workgroup then
// scans the target's row by itself.
#include "serve_internal.h"
#include "device_common.h"

namespace spear {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                       // 16-byte loads per row in flight
constexpr int kStep = kThreads * 4 * kUnroll;    // entries of one round
typedef float f4u_t __attribute__((ext_vector_type(4), aligned(4)));   // rows start at any entry

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// A thread's best entry so far; it sees rising j, so a tie keeps the lower one.
struct Best {
  float score = -1.0f;
  int j = 0;
  __device__ __forceinline__ void see(float w, float noise, int at) {
    const float s = w / noise;
    const bool better = w > 0.0f && s > score;
    score = better ? s : score;
    j = better ? at : j;
  }
  __device__ __forceinline__ uint64_t key() const {
    return score >= 0.0f ? ((uint64_t)float_bits(score) << 32) | (uint32_t)~j : 0ull;
  }
};

// Where a thread's vector i of the round at r0 lies, kept within the share.
__device__ __forceinline__ int place(int r0, int i, int end) {
  return min(r0 + 4 * ((int)threadIdx.x + i * kThreads), end - 4);
}

// The noise of a share's first round (of at least four entries).
struct Ahead {
  f4u_t e[kUnroll];
  __device__ __forceinline__ void load(const float* __restrict__ noise, int beg, int end) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) e[i] = *(const f4u_t*)(noise + place(beg, i, end));
  }
};

// Best key of the entries [beg, end) of one row, `ahead` the first noise if it is
// there already.  MODE 0: w = p; 1: w = p - q; 2: w = p - [j = x].  Vectors past
// the end are read within it and count nothing, so that the last round's loads
// are in flight together as every other's.
template <int MODE>
__device__ __forceinline__ uint64_t scan(const float* __restrict__ p, const float* __restrict__ q,
                                         const float* __restrict__ e, int x, int beg, int end, const Ahead* ahead) {
  Best best;
  auto weight = [x](float p, float q, int j) { return MODE == 0 ? p : MODE == 1 ? p - q : j == x ? p - 1.0f : p; };
  for (int r0 = beg; r0 + 3 < end; r0 += kStep) {
    f4u_t pv[kUnroll], qv[kUnroll], ev[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int j = place(r0, i, end);
      pv[i] = *(const f4u_t*)(p + j);
      if (MODE == 1) qv[i] = *(const f4u_t*)(q + j);
      if (ahead && r0 == beg) ev[i] = ahead->e[i];
      else ev[i] = *(const f4u_t*)(e + j);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int j = r0 + 4 * ((int)threadIdx.x + i * kThreads);
      if (r0 + kStep > end && j + 3 >= end) {
        pv[i] = f4u_t{0.0f, 0.0f, 0.0f, 0.0f};
        if (MODE == 1) qv[i] = pv[i];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) best.see(weight(pv[i][k], MODE == 1 ? qv[i][k] : 0.0f, j + k), ev[i][k], j + k);
    }
  }
  // The last one to three entries.
  const int j = end - (end - beg) % 4 + (int)threadIdx.x;
  if (j < end) best.see(weight(p[j], MODE == 1 ? q[j] : 0.0f, j), e[j], j);
  return best.key();
}

// The workgroup's maximum, in every thread.
__device__ uint64_t block_max(uint64_t v, uint64_t* lds) {
#pragma unroll
  for (int o = 32; o > 0; o /= 2) v = max64(v, __shfl_xor(v, o));
  __syncthreads();
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int i = 1; i < kThreads / kWave; ++i) v = max64(v, lds[i]);
  return v;
}

__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyArgs a) {
  __shared__ uint64_t lds[kThreads / kWave];
  __shared__ uint32_t arrived;
  const int b = blockIdx.x / a.splits, part = blockIdx.x % a.splits;
  const int lane = threadIdx.x % kWave;
  const int K = a.drafts;
  const float* target = a.target + b * a.target_bs;
  const float* draft = a.draft ? a.draft + b * a.draft_bs : nullptr;
  const int32_t* drafted = a.drafted + (int64_t)b * K;

  const int share = (int)((((int64_t)a.vocab + a.splits - 1) / a.splits + 3) / 4 * 4);
  const int beg = (int)min((int64_t)part * share, (int64_t)a.vocab);
  const int end = (int)min((int64_t)beg + share, (int64_t)a.vocab);
  const float* e = a.noise + (int64_t)b * a.vocab;
  // (does not depend on the kept tokens, so it comes in while those are counted)
  Ahead ahead;
  if (beg + 3 < end) ahead.load(e, beg, end);

  // Kept tokens: lanes take one drafted token each, the first refusal counts.
  // (The token, its random number and the sequence's length are requested
  // together, whether the length needs them or not.)
  int n = K, kept = -1;
  for (int i0 = 0; i0 < K; i0 += kWave) {
    const int i = min(i0 + lane, K - 1);
    const int x = drafted[i];
    const float u = a.u[(int64_t)b * K + i];
    if (i0 == 0 && a.num_drafts) n = min(max(a.num_drafts[b], 0), K);
    const bool in = x >= 0 && x < a.vocab;
    const float q = draft && in ? draft[i * a.draft_rs + x] : 1.0f;
    const float p = in ? target[i * a.target_rs + x] : 0.0f;
    const uint64_t stop = __ballot(i0 + lane >= n || !(u * q < p));
    if (stop) {
      kept = min(i0 + __builtin_ctzll(stop), n);
      break;
    }
  }
  if (kept < 0) kept = n;

  // The race over this workgroup's share.
  const float* p = target + kept * a.target_rs;
  uint64_t best;
  if (kept == n) best = scan<0>(p, nullptr, e, -1, beg, end, &ahead);
  else if (draft) best = scan<1>(p, draft + kept * a.draft_rs, e, -1, beg, end, &ahead);
  else best = scan<2>(p, nullptr, e, drafted[kept], beg, end, &ahead);
  best = block_max(best, lds);

  if (a.splits > 1) {
    uint64_t* parts = a.part + (int64_t)b * a.splits;
    if (threadIdx.x == 0) {
      __hip_atomic_store(&parts[part], best, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      drain_vm();
      arrived = add_dev_u32(&a.counters[b], 1u);
    }
    __syncthreads();
    if (arrived != (uint32_t)a.splits - 1) return;
    best = 0;
    for (int i = threadIdx.x; i < a.splits; i += kThreads)
      best = max64(best, __hip_atomic_load(&parts[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    best = block_max(best, lds);
    if (threadIdx.x == 0) st_dev_u32(&a.counters[b], 0u);
  }
  if (best == 0 && kept < n) best = block_max(scan<0>(p, nullptr, e, -1, 0, a.vocab, nullptr), lds);
  const int token = best ? (int)~(uint32_t)best : -1;
  if (threadIdx.x == 0) a.accepted[b] = kept;
  for (int i = threadIdx.x; i <= K; i += kThreads)
    a.tokens[(int64_t)b * (K + 1) + i] = i < kept ? drafted[i] : i == kept ? token : -1;
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& a, void* stream) {
  verify_kernel<<<dim3((unsigned)(a.batch * (int64_t)a.splits)), dim3(kThreads), 0, (hipStream_t)stream>>>(a);
  return hipGetLastError();
}

// Workgroups per sequence: a round (kStep entries) each at least, and the four
// workgroups per CU that the GPU holds at once.  Sequences past the header's counters have
// a workgroup each.
int verify_splits(const spear_verify_desc_t& d, int cus) {
  if (d.batch > (int)kMaxEcTiles) return 1;
  const int64_t rounds = ceil_div(d.vocab, kStep), fill = ceil_div((int64_t)4 * cus, d.batch > 0 ? d.batch : 1);
  return (int)(rounds < fill ? rounds : fill);
}

}  // namespace spear
