// A step's plan: which sequences get their new tokens' pages, and the block
// tables, offsets, slots and positions that follow.
//
// Everything comes from running sums over the sequences: of the pages laid on the
// stack of free ones, of the pages wanted, and of the new tokens.  A sequence is
// served while the last two stay within what there is, so those that are served
// come before all that are not, and the offsets of the latter are the totals.
// The sums take a microsecond or two of latency and no bandwidth, so every
// workgroup forms all of them by itself (no second launch, no exchange) and then
// fills as many rows as it has threads: it marks the rows at which its sequences
// begin, a running maximum finds every row's own, and the row looks up its page, in
// the table or, if it is a new one, on the stack.  A new page's first row is always
// a new one: its thread writes the entry of the block table.
//
// The stack is read below its old top and written above it, and a taken page that was
// laid on it in the same call is read from the block table that it left: no
// workgroup reads what another writes.  Only state that is updated in place
// is written by the last workgroup to arrive.
#include "serve_internal.h"
#include "wave_ops.h"

namespace spear {
namespace {

// What sequence b asks for and gives back.
struct Wish {
  int32_t lens, held;
  int32_t ask, need, freed;   // new tokens, pages missing and pages past what it needs
  bool valid;
};

__device__ __forceinline__ Wish wish_of(const KvPlanArgs& a, int b) {
  Wish w = {0, 0, 0, 0, 0, false};
  if (b >= a.batch) return w;
  w.lens = a.lens[b];
  w.held = a.held[b];
  const int32_t ask = a.ask[b];
  const int64_t page = (int64_t)1 << a.page_log2;
  const int64_t want = ((int64_t)w.lens + ask + page - 1) >> a.page_log2;
  w.valid = w.lens >= 0 && ask >= 0 && w.held >= 0 && w.held <= a.max_pages && want <= a.max_pages &&
            w.held * page >= w.lens;
  if (w.valid) {
    w.ask = ask;
    w.need = max((int)want - w.held, 0);
    w.freed = max(w.held - (int)want, 0);
  }
  return w;
}

// Sums over the sequences up to one: pages given back, new tokens, pages missing.
struct Sums {
  int64_t freed, ask, need;
};
__device__ __forceinline__ void add(Sums& a, const Sums& b) {
  a.freed += b.freed;
  a.ask += b.ask;
  a.need += b.need;
}

// Sums before each thread's values, and those of all threads.
template <int THREADS>
__device__ __forceinline__ Sums running(const Sums& own, Sums* waves, Sums* total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  Sums v = {wave_run(own.freed), wave_run(own.ask), wave_run(own.need)};
  __syncthreads();
  if (lane == kWave - 1) waves[wave] = v;
  __syncthreads();
  v = {v.freed - own.freed, v.ask - own.ask, v.need - own.need};
  Sums sum = {0, 0, 0};
#pragma unroll
  for (int i = 0; i < THREADS / kWave; ++i) {
    if (i == wave) add(v, sum);
    add(sum, waves[i]);
  }
  *total = sum;
  return v;
}

// .. and the running maximum of numbers from -1.
template <int THREADS>
__device__ __forceinline__ int running_max(int v, int* waves) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  v = wave_run(v, -1, [](int a, int b) { return max(a, b); });
  __syncthreads();
  if (lane == kWave - 1) waves[wave] = v;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < THREADS / kWave; ++i)
    if (i < wave) v = max(v, waves[i]);
  return v;
}

// A sequence with rows in this workgroup's range, kept at the place of the first.
struct Begin {
  int32_t seq, pos, held;   // pos: the first such row's position
  int64_t take;             // pages taken before its own
};

// EACH: neighbouring sequences of a thread.
template <int THREADS, int EACH>
__global__ void __launch_bounds__(THREADS) kv_plan_kernel(KvPlanArgs a) {
  constexpr int kChunk = THREADS * EACH;
  __shared__ Sums waves[THREADS / kWave];
  __shared__ int max_waves[THREADS / kWave];
  __shared__ Begin begin[THREADS];
  __shared__ int marked[THREADS];
  __shared__ int64_t freed_to[kChunk];        // running sum of freed pages in one chunk of sequences
  __shared__ int32_t held_of[kChunk];
  __shared__ int32_t freed_page[THREADS];     // pages taken here that were laid on the stack in this call
  __shared__ unsigned long long given_rows, given_pages, lowest, highest;
  __shared__ uint32_t arrived;
  const int tid = threadIdx.x, lane = tid % kWave;
  const int chunks = (a.batch + kChunk - 1) / kChunk;
  const int64_t row0 = (int64_t)blockIdx.x * THREADS;

  marked[tid] = -1;
  if (tid == 0) {
    given_rows = given_pages = 0;
    lowest = ~0ull;
    highest = 0;
  }
  const int64_t old = min(max(*a.free_count, 0), a.free_slots);
  // Pages laid on the stack, all of them before any is taken.
  Wish w[EACH];
  Sums sum = {0, 0, 0}, v = {0, 0, 0};
  auto look = [&](int c) {
#pragma unroll
    for (int e = 0; e < EACH; ++e) w[e] = wish_of(a, c * kChunk + tid * EACH + e);
    Sums own = {0, 0, 0};
#pragma unroll
    for (int e = 0; e < EACH; ++e) add(own, {w[e].freed, w[e].ask, w[e].need});
    v = running<THREADS>(own, waves, &sum);
  };
  int64_t freed = 0;
  for (int c = 0; c < chunks; ++c) {
    look(c);
    freed += sum.freed;
  }
  const int64_t top = old + freed;
  // (the running sums' barriers come after the clearing above)

  // Who is served, and the first row of each sequence in the range.
  const bool writes_state = !a.in_place && blockIdx.x == 0;
  auto serve = [&](bool rows_too, bool state) {
    int64_t rows_before = 0, pages_before = 0;
    for (int c = 0; c < chunks; ++c) {
      if (chunks > 1) look(c);
      int64_t rows_to = rows_before + v.ask, pages_to = pages_before + v.need;
      int64_t rows_given = -1, pages_given = 0;
#pragma unroll
      for (int e = 0; e < EACH; ++e) {
        rows_to += w[e].ask;
        pages_to += w[e].need;
        if (w[e].valid && rows_to <= a.rows && pages_to <= top) {
          rows_given = rows_to;
          pages_given = pages_to;
        }
      }
      // (the sums rise: a wave's last served sequence has the largest)
      const uint64_t some = __ballot(rows_given >= 0);
      if (some != 0 && lane == 63 - __builtin_clzll(some)) {
        atomicMax(&given_rows, (unsigned long long)rows_given);
        atomicMax(&given_pages, (unsigned long long)pages_given);
      }
      __syncthreads();
      rows_to = rows_before + v.ask;
      pages_to = pages_before + v.need;
#pragma unroll
      for (int e = 0; e < EACH; ++e) {
        const int b = c * kChunk + tid * EACH + e;
        const int64_t first = min(rows_to, (int64_t)given_rows);
        rows_to += w[e].ask;
        pages_to += w[e].need;
        const bool given = w[e].valid && rows_to <= a.rows && pages_to <= top;
        const int32_t n = given ? w[e].ask : 0;
        if (rows_too && n > 0 && first < row0 + THREADS && first + n > row0) {
          const int at = (int)max(first - row0, (int64_t)0);
          begin[at] = {b, w[e].lens + (int)(row0 + at - first), w[e].held, pages_to - w[e].need};
          marked[at] = at;
        }
        if (state && b < a.batch) {
          a.cu_q[b] = (int32_t)first;
          a.kv_lens[b] = w[e].lens + n;
          a.held_out[b] = w[e].held - w[e].freed + (given ? w[e].need : 0);
        }
      }
      rows_before += sum.ask;
      pages_before += sum.need;
    }
    if (state && tid == 0) {
      a.cu_q[a.batch] = (int32_t)given_rows;
      *a.free_out = (int32_t)min(top - (int64_t)given_pages, (int64_t)a.free_slots);
    }
  };
  serve(true, writes_state);
  __syncthreads();
  const int64_t total_rows = (int64_t)given_rows, total_pages = (int64_t)given_pages;

  // This thread's row.
  const int64_t row = row0 + tid;
  const int own = running_max<THREADS>(marked[tid], max_waves);
  const bool used = row < total_rows && own >= 0;
  Begin s = {0, 0, 0, 0};
  int pos = -1;
  int32_t page = 0;
  int64_t from = -1;        // place on the stack of a page that is taken
  if (used) {
    s = begin[own];
    pos = s.pos + (tid - own);
    const int entry = pos >> a.page_log2;
    if (entry < s.held) {
      page = a.table[s.seq * a.table_stride + entry];
    } else {
      from = top - 1 - (s.take + (entry - s.held));
      if (from < old) page = a.free_pages[from];
    }
  }
  if (freed > 0) {
    // Pages laid on the stack in this call: their places are found by the running
    // sum of the sequences that gave them.
    const bool mine = from >= old;
    const uint64_t some = __ballot(mine);       // (`from` falls as the rows rise)
    if (mine && lane == 63 - __builtin_clzll(some)) atomicMin(&lowest, (unsigned long long)(from - old));
    if (mine && lane == __builtin_ctzll(some)) atomicMax(&highest, (unsigned long long)(from - old) + 1);
    __syncthreads();
    const int64_t lo = (int64_t)lowest, hi = (int64_t)highest;     // (at most THREADS: every page has a row here)
    const int64_t stay = min(top - total_pages, (int64_t)a.free_slots) - old;   // of those laid on it, these remain
    int64_t before = 0;
    for (int c = 0; c < chunks; ++c) {
      if (chunks > 1) look(c);
      int64_t to = before + v.freed;
#pragma unroll
      for (int e = 0; e < EACH; ++e) {
        to += w[e].freed;
        freed_to[tid * EACH + e] = to;
        held_of[tid * EACH + e] = w[e].held;
      }
      __syncthreads();
      auto find = [&](int64_t i) {       // page i of those laid on the stack, which this chunk gave
        int at = 0;
#pragma unroll
        for (int step = kChunk / 2; step > 0; step /= 2)
          if (freed_to[at + step - 1] <= i) at += step;
        return a.table[(int64_t)(c * kChunk + at) * a.table_stride + (held_of[at] - (int)(freed_to[at] - i))];
      };
      const int64_t end = before + sum.freed;
      if (lo + tid < hi && lo + tid >= before && lo + tid < end) freed_page[tid] = find(lo + tid);
      for (int64_t i = row0 + tid; i < stay; i += (int64_t)gridDim.x * THREADS)
        if (i >= before && i < end) a.free_pages[old + i] = find(i);
      before = end;
      __syncthreads();
    }
    if (mine) page = freed_page[from - old - lo];
  }
  if (row < a.rows) {
    const int in_page = pos & ((1 << a.page_log2) - 1);
    if (from >= 0 && in_page == 0) a.table[s.seq * a.table_stride + (pos >> a.page_log2)] = page;
    a.slots[row] = used ? ((int64_t)page << a.page_log2) + in_page : -1;
    a.positions[row] = pos;
    a.sequence[row] = used ? s.seq : -1;
  }

  if (!a.in_place) return;
  if (gridDim.x > 1) {
    // (every wave's reads of the state have come back: what follows from them has been written)
    __syncthreads();
    if (tid == 0) {
      drain_vm();
      arrived = add_dev_u32(a.counter, 1u);
    }
    __syncthreads();
    if (arrived != gridDim.x - 1) return;
    if (tid == 0) st_dev_u32(a.counter, 0u);
  }
  __syncthreads();
  serve(false, true);
}

}  // namespace

// Few sequences go with small workgroups: more of them share the rows, and their
// sums are shorter.  Up to 2048 sequences stay in registers from one sum to the next
// (1500 of them, 4864 new tokens: 8 us; read again for every sum, by 1024 threads of one
// each, 39).  96 sequences of a token each: 3.6 us, of which 2 are those of any launch
// that reads memory twice in a row; chunks of 41 prompts, 79064 tokens: 4.0.  With the state
// in place, which the last workgroup to arrive writes from sums formed again: 3.8 (96
// sequences), 10.2 (1500) and 8.0 (the prompts, in 309 workgroups).
int kv_plan_threads(int batch) { return batch <= 1024 ? 256 : 512; }

hipError_t launch_kv_plan(const KvPlanArgs& a, void* stream) {
  const dim3 grid((unsigned)(a.rows > 0 ? ceil_div(a.rows, a.threads) : 1)), block((unsigned)a.threads);
  hipStream_t s = (hipStream_t)stream;
  if (a.batch <= 256) kv_plan_kernel<256, 1><<<grid, block, 0, s>>>(a);
  else if (a.batch <= 1024) kv_plan_kernel<256, 4><<<grid, block, 0, s>>>(a);
  else kv_plan_kernel<512, 4><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace spear
