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
// Long sequences are cut into pieces (attn_common.h).  Pieces leave their sums in the workspace in
// fp32, and the last of a row tile's to arrive joins them in order, so the result
// does not depend on scheduling.  Data passes between workgroups as everywhere
// here: device-coherent stores, a drain, a counter.
#include <algorithm>

#include "attn_common.h"

namespace spear {
namespace {

// ------------------------------------------------------------ the main kernel

constexpr uint32_t kMostItems = 4;   // items per CU aimed at, at most

template <int D, bool I8, int RT>
struct Shape {
  static constexpr int R = 16 * RT;
  static constexpr int KT = 32;                  // keys of a wave's tile
  static constexpr int KS = KT * kWaves;         // keys of a step
  static constexpr int SLOT = R * (D + 2);       // floats of a partial result: sums [R][D], references, totals
};

// Joins the `pieces` partial results of a row tile (rows `rows_here` of them in
// use) and writes the result.  Threads take four columns of a row each; with few
// columns, several groups of threads take every so many pieces.  Loads of
// eight pieces are in flight together.
template <int D, int R, int SLOT>
__device__ __forceinline__ void join(const AttnK& a, float* lds, int rows_here, int r0, int q0, int head,
                                     uint32_t slot0, int pieces) {
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
          const uint32_t slot = slot0 + (uint32_t)(piece * a.kv_heads);
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
  __shared__ uint32_t s_arrived;
  static_assert(sizeof(s_o) >= kThreads * 32, "the join's exchange fits");

  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane % 16, t = lane / 16;

  const Seq seq0 = sequence<R>(a, lane);
  // Sequences of like length: no more than one item for each CU (two would share
  // one), so the pieces are counted as if every row tile wasted one; and no
  // pieces if the row tiles come out even on the CUs by themselves (64 sequences
  // of 2k, two row tiles a CU: 111 us, 125 cut in two).  Otherwise four items for
  // each CU, which end at different times, the next ones taking their places (96
  // sequences of 64 .. 8192 at 1, 2, 3, 4, 7 items a CU: 120, 98, 99, 97, 95 us,
  // and fp16 213, 200, 196, 191, 187; two of 54k and 60k at 200, 256, 264, 488,
  // 720 items: 90, 93, 121, 99, 104).
  const Load load = load_of<R>(a, seq0, lane);
  const bool even = (uint64_t)load.longest * load.tiles * 2 <= (uint64_t)load.work * 3;
  const uint32_t cus = (uint32_t)a.cus, units = load.tiles * (uint32_t)a.kv_heads;
  uint32_t target = (RT == 1 ? kMostItems : 2) * cus;   // (two workgroups of 32 rows fill a CU)
  if (even) {
    if (units < cus) target = max(cus - units, cus / 4);
    else if (((units + cus - 1) / cus) * cus * 7 <= units * 8) target = 0;
  }
  const int piece = target ? piece_keys<KS>(a, load.work, target) : kWhole;
  const int head = (int)uniform(blockIdx.x % (uint32_t)a.kv_heads);

  const int place_mask = (1 << a.page_log2) - 1;
  const uint32_t koff = (uint32_t)(c * RB + 16 * t), voff = (uint32_t)(4 * t * RB + c * (DL * E));

  for (uint32_t index = blockIdx.x / (uint32_t)a.kv_heads;; index += gridDim.x / (uint32_t)a.kv_heads) {
    Item u;
    if (!find<R>(a, seq0, piece, uniform(index), lane, &u)) break;
    const int rows = u.n * a.group;                                // of the sequence
    const int r0 = u.rt * R;
    const int rows_here = min(R, rows - r0);
    const int pos0 = u.kv - u.n;                                   // position of token 0
    const int see_all = uniform(min(pos0 + r0 / a.group + 1, u.kv));   // keys below this are seen by every row
    const int k1 = uniform(min(max(pos0 + (r0 + rows_here - 1) / a.group + 1, 0), u.kv));   // .. from this on by none
    const int pieces = pieces_of(k1, piece);                       // of this row tile: those that hold keys
    if (u.piece >= pieces) continue;
    const int step0 = u.piece * (piece / KS);
    const int k_stop = pieces == 1 ? k1 : min(k1, step0 * KS + piece);   // this workgroup's keys end here

    // Queries as B operands; the k order follows the K loads'.
    half8_t qf[RT][NM];
    int lim[RT];                                                   // keys below this are seen by the lane's row
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      const int r = r0 + 16 * x + c;
      const bool ok = r < rows;
      const int tok = ok ? r / a.group : 0, h = ok ? head * a.group + r % a.group : 0;
      lim[x] = ok ? min(pos0 + tok + 1, k1) : k1;
      const half_t* qp = a.q + (u.q0 + (int64_t)tok) * a.q_ts + h * a.q_hs;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const int d = I8 ? 64 * (m / 2) + 16 * t + 8 * (m % 2) : 32 * m + 8 * t;
        qf[x][m] = ok ? query(qp + d, a.negate) : zero_half8();
      }
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

    // Memory: a 16-key tile lies within one page, so its place is the same for
    // all lanes.  Rows from k1 on lie outside the buffer and read as zeros; a
    // tile past the share reads nothing.
    // (constant address space and a scalar index: scalar loads, which the waits
    // for keys and values do not count)
    const scalar_i32_t* table = (const scalar_i32_t*)(uintptr_t)(a.table + (int64_t)uniform(u.b) * a.table_stride);
    const int last_key = max(k1 - 1, 0);
    auto page_of = [&](int key) {
      return (uint32_t)table[uniform(min(key, last_key) >> a.page_log2)];
    };
    const int64_t head_row = (int64_t)head << a.page_log2;
    const unsigned char* kc = (const unsigned char*)a.kc + head_row * RB;
    const unsigned char* vc = (const unsigned char*)a.vc + head_row * RB;
    const float* ks = I8 ? a.ks + head_row : nullptr;
    const float* vs = I8 ? a.vs + head_row : nullptr;
    const uint32_t page_rows = (uint32_t)a.kv_heads << a.page_log2;
    u32x4_t kr[NS][KL];
    vvec_t vr[NG][8];
    float4_t ksc[NS], vsc[NS];
    uint32_t page[NS], later_page[NS];   // of the tile requested next, and of the one after it
    // Bytes of a 16-key tile's rows that hold keys of this workgroup's share.
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

    bool noted = false;
    int base = (step0 * kWaves + wave) * KT;
#pragma unroll
    for (int n = 0; n < NS; ++n) page[n] = page_of(base + 16 * n);
#pragma unroll
    for (int n = 0; n < NS; ++n) later_page[n] = page_of(base + KS + 16 * n);
    // (the order is that of the loop: with another one the compiler's wait for
    // the keys at its top would also wait for the values)
    load_k(base, page);
    __builtin_amdgcn_sched_barrier(0);
    load_v(base, page);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < NS; ++n) page[n] = later_page[n];
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
        move |= top[x] > mref[x] + kHead;
      }
      if (__ballot(move)) {
#pragma unroll
        for (int x = 0; x < RT; ++x) {
          const float to = top[x] > mref[x] + kHead ? top[x] - kStart : mref[x];
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
              // bytes j % 4 of both words, zero extended to halves
              const uint32_t sel = 0x0c000c04u + (uint32_t)(j % 4) * 0x00010001u;
              w[k] = codes_to_half2(__builtin_amdgcn_perm(lo, hi, sel));
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
    __syncthreads();
    const bool whole = pieces == 1;
    const uint32_t slot0 = (uint32_t)u.slot * (uint32_t)a.kv_heads + (uint32_t)head;   // pieces: kv_heads apart
    const uint32_t slot = slot0 + (uint32_t)(u.piece * a.kv_heads);
    for (int v = threadIdx.x; v < rows_here * (D / 4); v += kThreads) {
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
        const int r = r0 + row;
        *(half4_t*)(a.out + ((u.q0 + (int64_t)(r / a.group)) * a.q_heads + head * a.group + r % a.group) * D + d) = h;
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
      __syncthreads();
      // (a split row tile has two slots at least)
      uint32_t* counter = a.counters + (uint32_t)(u.slot / 2) * (uint32_t)a.kv_heads + (uint32_t)head;
      if (threadIdx.x == 0) s_arrived = add_dev_u32(counter, 1u);
      __syncthreads();
      if (s_arrived == (uint32_t)pieces - 1) {
        if (threadIdx.x == 0) st_dev_u32(counter, 0u);
        join<D, R, SLOT>(a, &s_o[0][0][0], rows_here, r0, u.q0, head, slot0, pieces);
      }
    }
    __syncthreads();
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
  // The kernels count work (tiles times 64 keys) and items in 32 bits.
  p.fits = (d.batch + rows / (p.tiles && !p.both ? 128 : R)) * ceil_div(max_kv, 64) <= INT32_MAX / 2;
  const int64_t most = (int64_t)1 << 20;
  // Items: row tiles, and the pieces of split ones: fewer than twice the items
  // aimed at.  That many partial results have to fit, and half as many counters.
  const int64_t pieces = (int64_t)kMostItems * p.cus, tile_pieces = (int64_t)2 * p.cus;
  const int64_t tiles = p.tiles ? d.batch : d.batch + rows / R;
  // (with few row tiles, items beyond two a CU are second ones of a workgroup:
  // workgroups without any would only be in the others' way)
  const int64_t items = tiles * H + pieces;
  p.grid = p.tiles && !p.both ? 0
           : (int)round_up(tiles * H < p.cus ? std::min(items, (int64_t)2 * p.cus) : std::min(items, most), H);
  p.tile_grid = !p.tiles ? 0 : (int)round_up(std::min((d.batch + rows / 128) * H + tile_pieces, most), H);
  p.part = kSyncHeaderBytes;
  p.part_bytes = p.grid ? (size_t)2 * pieces * R * (dim + 2) * 4 : 0;
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
    k.min_piece = 256;   // shorter ones cost more in their partial sums than they save
    const hipError_t e = launch_attention_tiles(k, a.kv.dim, i8, p.tile_grid, st);
    if (e != hipSuccess || !p.both) return e;
  }
  k.rows_from = 0;
  k.rows_to = p.both ? p.few_rows : INT32_MAX;
  k.part = (float*)((char*)a.workspace + p.part);
  k.part_bytes = (int32_t)p.part_bytes;
  k.min_piece = 512;   // four steps; 256 took 20 us instead of 15 for one sequence of 8k
  if (a.kv.dim == 64) {
    if (i8) return two ? launch<64, true, 2>(k, p, st) : launch<64, true, 1>(k, p, st);
    return two ? launch<64, false, 2>(k, p, st) : launch<64, false, 1>(k, p, st);
  }
  if (i8) return two ? launch<128, true, 2>(k, p, st) : launch<128, true, 1>(k, p, st);
  return two ? launch<128, false, 2>(k, p, st) : launch<128, false, 1>(k, p, st);
}

}  // namespace spear
