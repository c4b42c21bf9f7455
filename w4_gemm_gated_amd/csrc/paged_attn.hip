// Attention of new tokens over a paged key/value cache.
//
// For one kv head, the query heads that share it and a sequence's new tokens
// give rows r = token * group + head; a workgroup takes R = 16 * RT of them.  Its
// keys are walked in tiles of KT by its four waves in turn (wave w takes tiles
// w, w + 4, ..), each with its own running softmax, joined through LDS at the
// end.  K and V go from memory straight into matrix-core operands:
//
//   S^T = K Q^T   A operand = keys (lane (c, t): key c of a 16-key tile),
//                 B operand = rows; result lane (c, t): row c, keys 4t .. 4t+3.
//   O^T += V^T P^T  the two 16-key tiles of a 32-key group give lane (c, t) the
//                 keys 4t .. 4t+3 and 16+4t .. 16+4t+3: exactly the eight k
//                 slots of its P^T operand, so P never leaves its lane.  The
//                 V^T operand needs the same eight keys at one d per lane: lane
//                 (c, t) loads them at d = DL c .. DL c + DL - 1 (DL = D / 16,
//                 whole rows per 16 lanes) and picks element j of each for the
//                 product of d = DL c + j.  A register transpose within the
//                 lane; no LDS.
//
// The statistics belong to row c and are the same in its four lanes t (two lane
// swaps a tile).  The weights are exp2(s - m) with a reference m that only
// moves (and the sums only rescale) when a tile's maximum passes m by 14: they
// stay below 2^14, and m starts 6 below the first maximum, which keeps the
// fp16 rounding of small weights relative (subnormals start 2^-20 below the
// largest).  An 8-bit cache: codes become fp16 exactly; a key's scale
// multiplies its scores, a value's scale its weight, and the exponent of the
// largest such scale that the row sees in a tile counts with the tile's maximum,
// so that the fp16 weights keep their range (sums and totals share the
// reference, so it cancels in the end).
//
// The work is laid end to end, in steps of one key tile per wave, head after
// head, sequence after sequence, and cut into equal shares, one per workgroup,
// however the lengths differ.  The lengths are on the device, so every
// workgroup finds its share by itself with a scan over the sequences.  Under
// load a dependent load takes microseconds, so a workgroup finds the next row
// tile of its share before it walks the present one, and requests the next one's
// queries and first keys and values before it writes the present one's result.
// A row tile that several workgroups share leaves one partial result (fp32) per
// workgroup in the workspace; the last of them to arrive joins them in order, so
// the result does not depend on scheduling.  Data passes between workgroups as
// everywhere here: device-coherent stores, a drain, a counter.
//
// Memory bounds it.  Measured (8 kv heads of 128; reading pages and computing
// nothing reaches 6.0 TB/s): 64 sequences of 4096 keys over 8 bits 100 us (5.5
// TB/s), of 2048 in fp16 107 us (5.0); 96 of 64 .. 8192 over 8 bits 88 us (4.7),
// in fp16 170; 24 of 500 .. 6000 with drafts 32 us over 8 bits, 68 in fp16;
// two of 54,000 and 60,000 in fp16 95 us (4.9); a few short ones 12 us, of
// which the launch and the chain length - table - keys take 8.  In fp16 at head
// dimension 128 19 (16 rows) and 59 (32 rows) registers are kept in memory; without
// the rare code for infinite and NaN values it would be 9 and none.
#include <algorithm>

#include "attn_common.h"

namespace spear {
namespace {

// ------------------------------------------------------------ the main kernel

// Equal shares of n steps for w workgroups: the first `more` take one step more.
struct Shares {
  uint32_t each, more;
  __device__ uint32_t begin(uint32_t w) const { return w * each + min(w, more); }
  __device__ uint32_t owner(uint32_t s) const {
    const uint32_t head = more * (each + 1);
    return s < head ? s / (each + 1) : more + (s - head) / each;
  }
};

// A row tile counts this many steps more than it has where shares are cut, for
// what its start and its result take (24 drafts of 500 .. 6000 keys 34.0 -> 32.4
// us, 96 sequences of 64 .. 8192 in fp16 176 -> 171, 256 of 512 67 -> 64; with three
// 31.9, 173, 66).  A share that begins among them begins with the next row tile.
constexpr uint32_t kTileCost = 2;
constexpr int kSeqs = 512;   // sequences kept in LDS; more are read again where needed

// Steps of KS keys that a sequence's row tile takes.
template <int KS>
__device__ __forceinline__ int steps_of(const Seq& s) { return max((s.kv + KS - 1) / KS, 1); }

// A share's part of a row tile: steps [step0, step1) of its `steps`.
struct Part {
  int b, q0, head, pos0, rows, r0, rows_here, steps, step0, step1;
  int see_all, k1, k_stop;   // keys below are seen by all rows; from here on by none; .. not this part's
  uint32_t unit0;            // the row tile's first step of all
};

template <int D, bool I8, int RT>
struct Shape {
  static constexpr int R = 16 * RT;
  static constexpr int KT = 32;                  // keys of a wave's tile
  static constexpr int KS = KT * kWaves;         // keys of a step
  static constexpr int SLOT = R * (D + 2);       // floats of a partial result: sums [R][D], references, totals
};

// A barrier for data in LDS alone: loads and stores in flight stay so.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Joins the `pieces` partial results of a row tile (rows `rows_here` of them in
// use) and writes the result.  Threads take four columns of a row each; with few
// columns, several groups of threads take every so many pieces.  Loads of
// eight pieces are in flight together.
template <int D, int R, int SLOT>
__device__ __forceinline__ void join(const AttnK& a, float* lds, int rows_here, int r0, int q0, int head, uint32_t w0,
                                     int pieces) {
  const __amdgpu_buffer_rsrc_t pr = make_rsrc(a.part, (uint32_t)a.part_bytes);
  const int cols = rows_here * (D / 4);
  const int groups = cols < kThreads ? kThreads / cols : 1;
  constexpr int BATCH = 8;
  for (int c0 = 0; c0 < cols; c0 += kThreads) {
    const int col = groups > 1 ? (int)threadIdx.x % cols : c0 + (int)threadIdx.x;
    const int grp = groups > 1 ? (int)threadIdx.x / cols : 0;
    const bool on = col < cols && grp < groups;
    const int row = col / (D / 4), d = col % (D / 4) * 4;
    float M = kNone, sum = 0.0f;
    float4_t o = zero_float4();
    if (on) {
      for (int i0 = grp; i0 < pieces; i0 += BATCH * groups) {
        float4_t po[BATCH];
        float pm[BATCH], pl[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int piece = i0 + i * groups;
          // the first piece is its workgroup's second result, the others first ones
          const uint32_t slot = 2 * (w0 + (uint32_t)piece) + (piece == 0 ? 1u : 0u);
          const uint32_t at = piece < pieces ? slot * (uint32_t)(SLOT * 4) : kOutOfRange;
          po[i] = buffer_load_f4_dev(pr, at + (uint32_t)(row * D + d) * 4);
          pm[i] = bits_float(__builtin_amdgcn_raw_buffer_load_b32(pr, at + (uint32_t)(R * D + row) * 4, 0, kCachePolicySc1));
          pl[i] = bits_float(__builtin_amdgcn_raw_buffer_load_b32(pr, at + (uint32_t)(R * D + R + row) * 4, 0, kCachePolicySc1));
        }
        float to = M;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          if (i0 + i * groups >= pieces) pm[i] = kNone;   // its sums read as zero
          to = fmaxf(to, pm[i]);
        }
        const float f = __builtin_amdgcn_exp2f(M - to);
        M = to;
        sum *= f;
        o *= f;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const float g = __builtin_amdgcn_exp2f(pm[i] - M);
          sum += pl[i] * g;
          o += po[i] * g;
        }
      }
    }
    if (groups > 1) {
      float* mine = lds + threadIdx.x * 8;
      *(float4_t*)mine = o;
      mine[4] = M;
      mine[5] = sum;
      __syncthreads();
      if (on && grp == 0) {
        for (int g = 1; g < groups; ++g) {
          const float* other = lds + (threadIdx.x + g * cols) * 8;
          const float to = fmaxf(M, other[4]);
          const float f = __builtin_amdgcn_exp2f(M - to), e = __builtin_amdgcn_exp2f(other[4] - to);
          sum = sum * f + other[5] * e;
          o = o * f + *(const float4_t*)other * e;
          M = to;
        }
      }
    }
    if (on && grp == 0) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // nothing seen: zeros
      half4_t h;
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = (half_t)(o[k] * inv);
      const int r = r0 + row;
      *(half4_t*)(a.out + ((q0 + (int64_t)(r / a.group)) * a.q_heads + head * a.group + r % a.group) * D + d) = h;
    }
  }
}

template <int D, bool I8, int RT>
__global__ void __launch_bounds__(kThreads, RT == 1 ? 3 : 2) attn_kernel(AttnK a) {
  typedef Shape<D, I8, RT> S;
  constexpr int R = S::R, KT = S::KT, KS = S::KS, SLOT = S::SLOT;
  constexpr int NS = KT / 16;                 // 16-key tiles
  constexpr int NG = KT / 32;                 // 32-key groups
  constexpr int E = I8 ? 1 : 2;               // bytes of a cached value
  constexpr int RB = D * E;                   // bytes of a cached row
  constexpr int NM = D / 32;                  // matrix instructions along d
  constexpr int KL = RB / 64;                 // 16-byte K loads of a lane and 16-key tile
  constexpr int DL = D / 16;                  // d values of a lane's V load
  typedef typename Vec<DL * E>::type vvec_t;
  constexpr int OS = D + 4;                   // row stride of the sums in LDS
  __shared__ __attribute__((aligned(16))) float s_o[kWaves][R][OS];
  __shared__ float s_m[kWaves][R], s_l[kWaves][R];
  __shared__ Seq s_seq[kSeqs];
  __shared__ uint32_t s_arrived;
  static_assert(sizeof(s_o) >= kThreads * 32, "the join's exchange fits");

  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane % 16, t = lane / 16;

  if (a.check_order && !offsets_rise(a, lane)) return;

  // This workgroup's share.  Whole row tiles where those come out even on the
  // workgroups: sequences of like length (64 of 2k, 512 row tiles: 112 us, 123 cut
  // into 768 shares), or all so short that a join would cost more than it saves.
  // Otherwise steps: as many shares as workgroups fit on the GPU (96 sequences of
  // 64 .. 8192: 89 us, 97 in pieces of one length), or, with fewer row tiles than
  // CUs, one for each CU, two where lengths differ much (two contexts of 54k and
  // 60k at 200, 256, 488, 720: 90, 93, 99, 104 us; 24 drafts of 500 .. 6000 at 256,
  // 340, 512, 800: 38, 36, 36, 38); but none of under four steps.
  // (The sequences are kept in LDS: a load from memory for the next row tile would
  // wait for all keys and values on their way.)
  for (int b = threadIdx.x; b < kSeqs && b < (a.batch + kWave - 1) / kWave * kWave; b += kThreads)
    s_seq[b] = sequence<R>(a, b);
  __syncthreads();
  auto seq_of = [&](int b) { return b < kSeqs ? s_seq[b] : sequence<R>(a, b); };
  uint32_t steps = 0, tiles = 0, longest = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kWave) {
    const Seq s = seq_of(b0 + lane);
    const uint32_t n = (uint32_t)steps_of<KS>(s);
    steps += (uint32_t)s.tiles * n;
    tiles += (uint32_t)s.tiles;
    longest = max(longest, s.tiles > 0 ? n : 0u);
  }
  steps = wave_sum(steps);
  tiles = wave_sum(tiles);
  longest = wave_max(longest);
  if (tiles == 0) return;
  const uint32_t cus = (uint32_t)a.cus, units = tiles * (uint32_t)a.kv_heads;
  const bool even = (uint64_t)longest * tiles * 2 <= (uint64_t)steps * 3;
  const uint32_t rounds = (units + gridDim.x - 1) / gridDim.x;
  const bool whole_tiles = longest <= 8 ? units <= gridDim.x
                                        : even && units >= cus && (rounds == 1 || rounds * gridDim.x * 7 <= units * 8);
  // (few row tiles of like length share evenly by themselves: 8 of 4096 keys 31 us, 33
  // with the cost)
  const uint32_t cost = even && units < cus ? 0 : kTileCost;
  const uint32_t per_head = whole_tiles ? tiles : steps + cost * tiles, total = per_head * (uint32_t)a.kv_heads;
  uint32_t groups = whole_tiles ? min(units, gridDim.x)
                    : min(min(gridDim.x, units >= cus ? gridDim.x : even ? cus : 2 * cus),
                          max(units, steps * (uint32_t)a.kv_heads / 4));
  if (blockIdx.x >= groups) return;
  const uint32_t each = uniform(total / groups);
  const Shares shares = {each, total - each * groups};
  const uint32_t end = shares.begin(blockIdx.x + 1);

  // The row tile that holds step (or is row tile) `at` of all.
  auto find = [&](uint32_t at) {
    Part u;
    u.head = (int)uniform(at / per_head);
    const uint32_t p = at - (uint32_t)u.head * per_head;
    u.b = u.q0 = u.rows = u.r0 = u.pos0 = u.k1 = u.step0 = 0;
    u.steps = 1;
    u.unit0 = at;
    int n = 0, kv = 0;
    uint32_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kWave) {
      const Seq s = seq_of(b0 + lane);
      const uint32_t mine = (uint32_t)s.tiles * (whole_tiles ? 1u : (uint32_t)steps_of<KS>(s) + cost);
      const uint32_t upto = before + wave_scan(mine);
      const uint64_t past = __ballot(upto > p);
      if (past) {
        const int l = __builtin_ctzll(past);
        n = __builtin_amdgcn_readlane(s.n, l);
        kv = __builtin_amdgcn_readlane(s.kv, l);
        u.b = b0 + l;
        u.q0 = __builtin_amdgcn_readlane(s.q0, l);
        u.steps = max((kv + KS - 1) / KS, 1);
        const uint32_t off = p - (uint32_t)__builtin_amdgcn_readlane((int)(upto - mine), l);
        const uint32_t rt = whole_tiles ? off
                            : __builtin_amdgcn_readlane(s.tiles, l) == 1 ? 0u : uniform(off / ((uint32_t)u.steps + cost));
        u.step0 = whole_tiles ? 0 : (int)(off - rt * ((uint32_t)u.steps + cost));
        u.unit0 = at - (uint32_t)u.step0;
        u.r0 = (int)rt * R;
        break;
      }
      before = (uint32_t)__builtin_amdgcn_readlane((int)upto, kWave - 1);
    }
    u.rows = n * a.group;                                          // of the sequence
    u.rows_here = min(R, u.rows - u.r0);
    u.pos0 = kv - n;                                               // position of token 0
    u.step1 = whole_tiles ? u.steps : (int)min((uint32_t)u.steps, end - u.unit0);
    u.see_all = uniform(min(u.pos0 + u.r0 / a.group + 1, kv));
    u.k1 = uniform(min(max(u.pos0 + (u.r0 + u.rows_here - 1) / a.group + 1, 0), kv));
    u.k_stop = min(u.k1, u.step1 * KS);
    return u;
  };

  const int place_mask = (1 << a.page_log2) - 1;
  const uint32_t koff = (uint32_t)(c * RB + 16 * t), voff = (uint32_t)(4 * t * RB + c * (DL * E));

  // What is on its way: the queries as B operands (the k order follows the K
  // loads'), and the next tile's keys and values.  A 16-key tile lies within one
  // page, so its place is the same for all lanes; rows from k1 on lie outside the
  // buffer and read as zeros, and a tile past the share reads nothing.
  const uint32_t page_rows = (uint32_t)a.kv_heads << a.page_log2;
  half8_t qf[RT][NM];
  int lim[RT];                           // keys below this are seen by the lane's row
  u32x4_t kr[NS][KL];
  vvec_t vr[NG][8];
  float4_t ksc[NS], vsc[NS];
  uint32_t page[NS], later_page[NS];     // of the tile requested next, and of the one after it
  const scalar_i32_t* table;             // (constant address space and a scalar index: scalar loads, which the
                                         // waits for keys and values do not count)
  const unsigned char *kc, *vc;
  const float *ks, *vs;
  int base, k1, k_stop, last_key;
  auto page_of = [&](int key) { return (uint32_t)table[uniform(min(key, last_key) >> a.page_log2)]; };
  auto load_k = [&](int base, const uint32_t* pages) {
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const int key = base + 16 * n;
        const uint64_t row = (uint64_t)min(pages[n], (uint32_t)a.num_pages - 1) * page_rows + (uint32_t)(key & place_mask);
        const uint32_t rows = base < k_stop ? (uint32_t)min(max(k1 - key, 0), 16) : 0u;
        const __amdgpu_buffer_rsrc_t r = uniform_rsrc(kc + row * RB, rows * RB);
#pragma unroll
        for (int i = 0; i < KL; ++i) kr[n][i] = buffer_vec<16>(r, koff + 64 * i);
        if constexpr (I8) ksc[n] = __builtin_bit_cast(float4_t, buffer_vec<16>(uniform_rsrc(ks + row, rows ? 64u : 0u), 16 * t));
      }
    };
    auto load_v = [&](int base, const uint32_t* pages) {
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const int key = base + 16 * n;
        const uint64_t row = (uint64_t)min(pages[n], (uint32_t)a.num_pages - 1) * page_rows + (uint32_t)(key & place_mask);
        const uint32_t rows = base < k_stop ? (uint32_t)min(max(k1 - key, 0), 16) : 0u;
        const __amdgpu_buffer_rsrc_t r = uniform_rsrc(vc + row * RB, rows * RB);
#pragma unroll
        for (int s = 0; s < 4; ++s) vr[n / 2][4 * (n % 2) + s] = buffer_vec<DL * E>(r, voff + s * RB);
        if constexpr (I8) vsc[n] = __builtin_bit_cast(float4_t, buffer_vec<16>(uniform_rsrc(vs + row, rows ? 64u : 0u), 16 * t));
      }
    };

  auto begin = [&](const Part& u) {
    k1 = u.k1;
    k_stop = u.k_stop;
    last_key = max(k1 - 1, 0);
    base = (u.step0 * kWaves + wave) * KT;
    table = (const scalar_i32_t*)(uintptr_t)(a.table + (int64_t)uniform(u.b) * a.table_stride);
    const int64_t head_row = (int64_t)u.head << a.page_log2;
    kc = (const unsigned char*)a.kc + head_row * RB;
    vc = (const unsigned char*)a.vc + head_row * RB;
    ks = I8 ? a.ks + head_row : nullptr;
    vs = I8 ? a.vs + head_row : nullptr;
#pragma unroll
    for (int n = 0; n < NS; ++n) page[n] = page_of(base + 16 * n);
#pragma unroll
    for (int n = 0; n < NS; ++n) later_page[n] = page_of(base + KS + 16 * n);
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      const int r = u.r0 + 16 * x + c;
      const bool ok = r < u.rows;
      const int tok = ok ? r / a.group : 0, h = ok ? u.head * a.group + r % a.group : 0;
      lim[x] = ok ? min(u.pos0 + tok + 1, k1) : k1;
      const half_t* qp = a.q + (u.q0 + (int64_t)tok) * a.q_ts + h * a.q_hs;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const int d = I8 ? 64 * (m / 2) + 16 * t + 8 * (m % 2) : 32 * m + 8 * t;
        qf[x][m] = ok ? load_half8(qp + d) : zero_half8();
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // (the order is that of the loop: with another one the compiler's wait for
    // the keys at its top would also wait for the values)
    load_k(base, page);
    __builtin_amdgcn_sched_barrier(0);
    load_v(base, page);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < NS; ++n) page[n] = later_page[n];
  };

  // The row tile after u, or `end`.
  auto after = [&](const Part& u) { return whole_tiles ? u.unit0 + 1u : u.unit0 + (uint32_t)u.steps + cost; };
  Part u = find(shares.begin(blockIdx.x));
  if (u.step0 >= u.steps) {
    if (after(u) >= end) return;
    u = find(after(u));
  }
  begin(u);
  for (;;) {
    const uint32_t next = after(u);
    const bool more = next < end;
    const Part then = find(more ? next : u.unit0);
    const int see_all = u.see_all;
    if (a.negate) {
#pragma unroll
      for (int x = 0; x < RT; ++x)
#pragma unroll
        for (int m = 0; m < NM; ++m) qf[x][m] = -qf[x][m];
    }
    float4_t acc[RT][DL];
    float mref[RT], l[RT];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      mref[x] = kNone;
      l[x] = 0.0f;
#pragma unroll
      for (int j = 0; j < DL; ++j) acc[x][j] = zero_float4();
    }
    bool noted = false;
    for (; base < k_stop; base += KS) {
      // Scores; the next tile's keys are requested as soon as these are used.
      float4_t st[RT][NS];
      float4_t kscale[NS];
#pragma unroll
      for (int n = 0; n < NS; ++n) {
#pragma unroll
        for (int x = 0; x < RT; ++x) st[x][n] = zero_float4();
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          half8_t kf;
          if constexpr (I8) kf = codes_to_half8(kr[n][m / 2][2 * (m % 2)], kr[n][m / 2][2 * (m % 2) + 1]);
          else kf = __builtin_bit_cast(half8_t, kr[n][m]);
#pragma unroll
          for (int x = 0; x < RT; ++x) st[x][n] = mfma16x16x32(kf, qf[x][m], st[x][n]);
        }
        if constexpr (I8) kscale[n] = ksc[n] * a.scale;
      }
      __builtin_amdgcn_sched_barrier(0);
      load_k(base + KS, page);
#pragma unroll
      for (int n = 0; n < NS; ++n) later_page[n] = page_of(base + 2 * KS + 16 * n);
      __builtin_amdgcn_sched_barrier(0);

      const bool edge = base + KT > see_all;
      float top[RT], tall = 0.0f;
      bool move = false;
      if constexpr (I8) {   // the largest finite scale of the tile's values
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) tall = fmaxf(tall, vsc[n][i] > kMaxScale ? 0.0f : vsc[n][i]);
        tall = scale_exponent(row_max4(tall));
      }
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        top[x] = -INFINITY;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (I8) st[x][n][i] *= kscale[n][i];
            else st[x][n][i] *= a.scale;
          }
        if (edge) {
          const int left = opaque(lim[x] - base - 4 * t);
#pragma unroll
          for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (16 * n + i >= left) st[x][n][i] = -INFINITY;
        }
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) top[x] = fmaxf(top[x], st[x][n][i]);
        top[x] = row_max4(top[x]);
        if constexpr (I8) {
          float e = tall;
          if (edge) {         // of those that the row sees
            e = 0.0f;
            const int left = opaque(lim[x] - base - 4 * t);
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) e = fmaxf(e, vsc[n][i] > kMaxScale || 16 * n + i >= left ? 0.0f : vsc[n][i]);
            e = scale_exponent(row_max4(e));
          }
          top[x] += e;
        }
        move |= top[x] - mref[x] > kHead;
      }
      if (__ballot(move)) {
#pragma unroll
        for (int x = 0; x < RT; ++x) {
          const float to = top[x] - mref[x] > kHead ? top[x] - kStart : mref[x];
          const float f = __builtin_amdgcn_exp2f(mref[x] - to);
          mref[x] = to;
          l[x] *= f;
#pragma unroll
          for (int j = 0; j < DL; ++j) acc[x][j] *= f;
        }
      }
      // Weights (B operands).
      half8_t pf[RT][NG];
#pragma unroll
      for (int x = 0; x < RT; ++x) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float p = __builtin_amdgcn_exp2f(st[x][n][i] - mref[x]);
            l[x] += p;
            if constexpr (I8) p *= vsc[n][i];
            pf[x][n / 2][4 * (n % 2) + i] = (half_t)p;
          }
        if constexpr (I8) {
          if (edge) {   // a scale that a row must not see may be infinite or NaN
            const int left = opaque(lim[x] - base - 4 * t);
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (16 * n + i >= left) pf[x][n / 2][4 * (n % 2) + i] = (half_t)0.0f;
          }
        }
      }
      // Values that some row must not see may be infinite or NaN, which a weight
      // of zero would not remove (codes are always finite).
      if constexpr (!I8) {
        if (edge) {
          bool odd = false;
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
              for (int w = 0; w < DL / 2; ++w) odd |= half2_not_finite(vr[g][s][w]);
          if (__ballot(odd)) {
            // Rare.  A product of their kinds (1: inf, 64: -inf, 4096: NaN; exact
            // for 32 keys) with what each row sees says which sums they reach:
            // bits, kept in this wave's part of s_o, that become values when the
            // sums are complete.  Then they leave the tile.
            uint32_t* note = (uint32_t*)s_o[wave] + lane;
            uint32_t bits[3 * RT];
#pragma unroll
            for (int i = 0; i < 3 * RT; ++i) bits[i] = noted ? note[i * kWave] : 0u;
            noted = true;
#pragma unroll
            for (int x = 0; x < RT; ++x)
#pragma unroll
              for (int g = 0; g < NG; ++g) {
                half8_t seen;
#pragma unroll
                for (int s = 0; s < 8; ++s)
                  seen[s] = (half_t)(base + 32 * g + 16 * (s / 4) + 4 * t + s % 4 < lim[x] ? 1.0f : 0.0f);
#pragma unroll
                for (int j = 0; j < DL; ++j) {
                  u32x4_t w;
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    w[k] = kind_of((vr[g][2 * k][j / 2] >> (16 * (j % 2))) & 0xFFFFu) |
                           kind_of((vr[g][2 * k + 1][j / 2] >> (16 * (j % 2))) & 0xFFFFu) << 16;
                  const float4_t kinds = mfma16x16x32(__builtin_bit_cast(half8_t, w), seen, zero_float4());
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const int n = (int)kinds[k];
                    const uint32_t bit = 1u << (4 * j + k);
                    bits[3 * x] |= n & 63 ? bit : 0u;
                    bits[3 * x + 1] |= n & 4032 ? bit : 0u;
                    bits[3 * x + 2] |= n >> 12 ? bit : 0u;
                  }
                }
              }
#pragma unroll
            for (int i = 0; i < 3 * RT; ++i) note[i * kWave] = bits[i];
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
              for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int w = 0; w < DL / 2; ++w) {
                  const uint32_t v = vr[g][s][w];
                  vr[g][s][w] = ((v & 0x7C00u) == 0x7C00u ? 0u : v & 0xFFFFu) |
                                ((v & 0x7C000000u) == 0x7C000000u ? 0u : v & 0xFFFF0000u);
                }
          }
        }
      }
      // O^T += V^T P^T: element j of the eight keys, for d = DL c + j.
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int j = 0; j < DL; ++j) {
          u32x4_t w;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t lo = vr[g][2 * k][j * E / 4], hi = vr[g][2 * k + 1][j * E / 4];
            if constexpr (I8) {
              // bytes j % 4 of both words, under 0x64, sign bits flipped
              const uint32_t sel = 0x0c000c04u + (uint32_t)(j % 4) * 0x00010001u;
              w[k] = codes_to_half2(__builtin_amdgcn_perm(lo, hi, sel) ^ 0x64806480u);
            } else {
              w[k] = __builtin_amdgcn_perm(hi, lo, j % 2 ? 0x07060302u : 0x05040100u);
            }
          }
          const half8_t vf = __builtin_bit_cast(half8_t, w);
#pragma unroll
          for (int x = 0; x < RT; ++x) acc[x][j] = mfma16x16x32(vf, pf[x][g], acc[x][j]);
        }
      __builtin_amdgcn_sched_barrier(0);
      load_v(base + KS, page);
#pragma unroll
      for (int n = 0; n < NS; ++n) page[n] = later_page[n];
      __builtin_amdgcn_sched_barrier(0);
    }

    if (more) begin(then);

    if (!I8 && noted) {
      const uint32_t* note = (const uint32_t*)s_o[wave] + lane;
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        const uint32_t inf = note[3 * x * kWave], minus = note[(3 * x + 1) * kWave], nan = note[(3 * x + 2) * kWave];
#pragma unroll
        for (int j = 0; j < DL; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t bit = 1u << (4 * j + k);
            if (inf & bit) acc[x][j][k] += INFINITY;
            if (minus & bit) acc[x][j][k] -= INFINITY;
            if (nan & bit) acc[x][j][k] = NAN;
          }
      }
      asm volatile("" ::: "memory");   // all notes are read before the sums take their place
    }
    // Join the waves.  Lane (c, t) holds row c at d = DL (4 t + k) + j.
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      l[x] = row_sum4(l[x]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < DL; j += 4) {
          float4_t o = {acc[x][j][k], acc[x][j + 1][k], acc[x][j + 2][k], acc[x][j + 3][k]};
          *(float4_t*)&s_o[wave][16 * x + c][DL * (4 * t + k) + j] = o;
        }
      if (t == 0) {
        s_m[wave][16 * x + c] = mref[x];
        s_l[wave][16 * x + c] = l[x];
      }
    }
    lds_barrier();
    const bool whole = u.step0 == 0 && u.step1 == u.steps;
    const uint32_t slot = 2 * blockIdx.x + (u.step0 == 0 ? 1u : 0u);
    for (int v = threadIdx.x; v < u.rows_here * (D / 4); v += kThreads) {
      const int row = v / (D / 4), d = v % (D / 4) * 4;
      float M = s_m[0][row];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) M = fmaxf(M, s_m[w][row]);
      float sum = 0.0f;
      float4_t o = zero_float4();
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(s_m[w][row] - M);
        sum += s_l[w][row] * f;
        o += *(const float4_t*)&s_o[w][row][d] * f;
      }
      if (whole) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // nothing seen: zeros
        half4_t h;
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = (half_t)(o[k] * inv);
        const int r = u.r0 + row;
        *(half4_t*)(a.out + ((u.q0 + (int64_t)(r / a.group)) * a.q_heads + u.head * a.group + r % a.group) * D + d) = h;
      } else {
        const __amdgpu_buffer_rsrc_t pr = make_rsrc(a.part, (uint32_t)a.part_bytes);
        const uint32_t p = slot * (uint32_t)(SLOT * 4);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, o), pr, p + (uint32_t)(row * D + d) * 4, 0,
                                               kCachePolicySc1);
        if (d == 0) {
          __builtin_amdgcn_raw_buffer_store_b32(float_bits(M), pr, p + (uint32_t)(R * D + row) * 4, 0, kCachePolicySc1);
          __builtin_amdgcn_raw_buffer_store_b32(float_bits(sum), pr, p + (uint32_t)(R * D + R + row) * 4, 0,
                                                kCachePolicySc1);
        }
      }
    }
    if (!whole) {
      drain_vm();
      lds_barrier();
      const uint32_t w0 = shares.owner(u.unit0);
      const int pieces = (int)(shares.owner(u.unit0 + (uint32_t)u.steps - 1) - w0) + 1;
      if (threadIdx.x == 0) s_arrived = add_dev_u32(&a.counters[w0], 1u);
      lds_barrier();
      if (s_arrived == (uint32_t)pieces - 1) {
        if (threadIdx.x == 0) st_dev_u32(&a.counters[w0], 0u);
        join<D, R, SLOT>(a, &s_o[0][0][0], u.rows_here, u.r0, u.q0, u.head, w0, pieces);
      }
    }
    if (!more) break;
    lds_barrier();
    u = then;
  }
}

template <int D, bool I8, int RT>
hipError_t launch(const AttnK& k, const AttnPlan& p, hipStream_t st) {
  attn_kernel<D, I8, RT><<<dim3(p.grid), dim3(kThreads), 0, st>>>(k);
  return hipGetLastError();
}

}  // namespace

AttnPlan attn_plan(const spear_attention_desc_t& d, int cus) {
  AttnPlan p;
  const int64_t H = d.kv.kv_heads, group = d.q_heads / H, dim = d.kv.head_dim;
  const int64_t most_rows = (int64_t)d.max_q * group;
  // Few rows: this kernel, 16 or 32 at a time.  More: tiles of 128, unless other
  // sequences of the batch have few (a decode step beside a prompt's chunk);
  // then each kernel takes its own.
  p.tiles = most_rows > 32;
  p.both = p.tiles && (int64_t)d.total_q < d.batch * (int64_t)d.max_q;
  p.row_tiles = (p.tiles ? group : most_rows) > 16 ? 2 : 1;
  p.few_rows = 16 * p.row_tiles;
  const int64_t R = p.few_rows;
  p.cus = std::min(cus, 512);
  const int64_t max_kv = (int64_t)d.max_pages * d.kv.page_size;
  const int64_t rows = (int64_t)d.total_q * group;
  // The kernels count work in 32 bits: steps of 128 keys of all row tiles here,
  // row tiles of a head times 64 keys in the other.
  const int64_t few = p.tiles ? (p.both ? d.batch : 0) : d.batch + rows / R;
  p.fits = few * (ceil_div(max_kv, 32 * kWaves) + kTileCost) * H <= INT32_MAX &&
           (p.tiles ? d.batch + rows / 128 : 0) * ceil_div(max_kv, 64) <= INT32_MAX / 2;
  // (in a batch of both kinds a sequence of few rows is one row tile)
  p.check_few = !p.both && !counts_hold(d.batch, rows, R, max_kv, 32 * kWaves, kTileCost, H, INT32_MAX);
  p.check_tiles = !counts_hold(d.batch, rows, 128, max_kv, 64, 0, 1, INT32_MAX / 2);
  // One share for each workgroup that the GPU holds at once; no more of them than
  // there can be steps.
  const int64_t held = (int64_t)(p.row_tiles == 1 ? 3 : 2) * p.cus;
  p.grid = (int)std::min(held, few * ceil_div(max_kv, 32 * kWaves) * H);
  // Items of the tile kernel: row tiles, and the pieces of split ones, fewer than
  // twice the items aimed at.  That many partial results have to fit, and half as
  // many counters.
  const int64_t tile_pieces = (int64_t)2 * p.cus;
  p.tile_grid = !p.tiles ? 0 : (int)round_up(std::min((d.batch + rows / 128) * H + tile_pieces, (int64_t)1 << 20), H);
  p.part = kSyncHeaderBytes;
  p.part_bytes = (size_t)2 * p.grid * R * (dim + 2) * 4;
  p.tile_part = p.part + p.part_bytes;
  p.tile_part_bytes = p.tiles ? (size_t)2 * tile_pieces * 128 * (dim + 2) * 4 : 0;
  p.bytes = p.tile_part + p.tile_part_bytes;
  return p;
}

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, void* stream) {
  AttnK k;
  k.q = (const half_t*)a.q; k.q_ts = a.q_ts; k.q_hs = a.q_hs;
  k.cu = a.cu_q; k.lens = a.kv_lens; k.table = a.table; k.table_stride = a.table_stride;
  k.kc = a.k_cache; k.vc = a.v_cache; k.ks = a.k_scale; k.vs = a.v_scale;
  k.out = (half_t*)a.out; k.counters = (uint32_t*)a.workspace;
  k.batch = a.batch; k.total_q = a.total_q; k.q_heads = a.q_heads; k.kv_heads = a.kv.heads;
  k.group = a.group; k.max_kv = a.max_kv; k.page_log2 = a.kv.page_log2; k.num_pages = a.kv.num_pages;
  // (a scale of zero: so small that every score counts as zero, yet a masked
  // one, minus infinity, stays one)
  k.cus = p.cus;
  k.scale = a.scale == 0.0f ? 1e-37f : (a.scale < 0.0f ? -a.scale : a.scale) * kLog2e;
  k.negate = a.scale < 0.0f ? 1 : 0;
  const hipStream_t st = (hipStream_t)stream;
  const bool i8 = a.kv.dtype == SPEAR_KV_INT8, two = p.row_tiles == 2;
  if (p.tiles) {
    k.rows_from = p.both ? p.few_rows : 0;
    k.rows_to = INT32_MAX;
    k.part = (float*)((char*)a.workspace + p.tile_part);
    k.part_bytes = (int32_t)p.tile_part_bytes;
    k.check_order = p.check_tiles;
    const hipError_t e = launch_attention_tiles(k, a.kv.dim, i8, p.tile_grid, st);
    if (e != hipSuccess || !p.both) return e;
  }
  k.rows_from = 0;
  k.rows_to = p.both ? p.few_rows : INT32_MAX;
  k.part = (float*)((char*)a.workspace + p.part);
  k.part_bytes = (int32_t)p.part_bytes;
  k.check_order = p.check_few;
  if (a.kv.dim == 64) {
    if (i8) return two ? launch<64, true, 2>(k, p, st) : launch<64, true, 1>(k, p, st);
    return two ? launch<64, false, 2>(k, p, st) : launch<64, false, 1>(k, p, st);
  }
  if (i8) return two ? launch<128, true, 2>(k, p, st) : launch<128, true, 1>(k, p, st);
  return two ? launch<128, false, 2>(k, p, st) : launch<128, false, 1>(k, p, st);
}

}  // namespace spear
