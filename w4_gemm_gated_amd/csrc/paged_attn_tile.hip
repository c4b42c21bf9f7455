// Attention of many new tokens (a prompt's chunk) over a paged key/value cache.
//
// As in paged_attn.hip, rows are r = token * group + head of the query heads
// that share a kv head, S^T = K Q^T and O^T = V^T P^T, so that P goes from one
// product's result registers into the other's operand without leaving its lane.
// Here the matrix cores bound the work: a workgroup takes 128 rows, 32 for each of
// its four waves, and all waves share a tile of 64 keys in LDS (two stages: the
// next tile is requested before this one is used).
//
//   - fp16 tiles go straight from memory to LDS; 16-byte units are permuted
//     within their row by the row's number on the way (the lane's source
//     address), so the fragment reads hit all banks.  8-bit tiles pass through
//     registers, where codes become fp16 once for all four waves.
//   - K fragments are 16-byte reads of a row; V^T fragments are transposing
//     reads (within 16 lanes, lane 4e + q gives the address of row e's four
//     values at 4q, and lane i receives column i of the four rows).
//   - in fp16 the request runs ahead by less than a tile: the compiler takes a read
//     of one stage to alias the copies into the other, and waits for these before
//     the tile's first keys (64) or first values (128) are read.  The other
//     workgroup of the CU covers that wait.
//   - the softmax reference moves rarely, the 8-bit scales enter the scores and
//     the weights, and infinities in values that some row must not see are kept
//     out, all as described in paged_attn.hip.
//
// The matrix work of a key and row is 4 D flops, the vector work about seven
// instructions, nearly the same time: two workgroups per CU let one's softmax
// run under the other's products.
//
// Row tiles are cut into pieces of their keys where there are too few for the GPU.
// Items are numbered with the kv head fastest and a sequence's last row tile, which
// sees the most keys, first: workgroups are dealt to the eight XCDs in turn, so
// those that run at a time on one XCD walk the same head's keys together and its
// L2 serves all but the first of them.  (Equal shares of the keys for all
// workgroups were measured on 2048 tokens over 8192 keys: the workgroups of a head
// stood at different keys, 4 MB of them, and 2.7 GB instead of 0.08 came from
// beyond the L2: 633 us instead of 419 then.)  Pieces leave their sums in the
// workspace; the last of a row tile's to arrive joins them in order.
//
// Measured (32 query heads on 8 kv heads): 8 x 2048 tokens over 4096 keys in
// 942 us at head dimension 128 and 599 us at 64 (876 and 689 TFLOP/s; a large
// library product reaches 1104), 1125 and 758 us over an 8-bit cache; one chunk
// of 700 tokens over 2571 keys in 49, 31, 57 and 40 us.  Counted at the first of
// these sizes in fp16, vector and matrix instructions together fill 90 % (128) and
// all (64) of the cycles.  At 128 the code for infinite and NaN values, inlined but
// rarely run, costs registers: 187 are kept in memory around the loop in fp16, none
// within it (without that code none at all; four over 8 bits).
#include "attn_common.h"

namespace spear {
namespace {

constexpr int kRows = 128;                  // of a workgroup
constexpr int kWaveRows = kRows / kWaves;   // 32: two 16-row operands
constexpr int kKeys = 64;                   // of a tile
constexpr int kNS = kKeys / 16;             // 16-key tiles
constexpr int kNG = kKeys / 32;             // 32-key groups
constexpr int kRT = kWaveRows / 16;
constexpr float kLarge = 0x1p20f;           // references past this are large
constexpr int kSchedMatrix = 0x8, kSchedLdsRead = 0x100;   // instruction classes of the issue order

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __fp16 fp16x4_t __attribute__((__vector_size__(4 * sizeof(__fp16))));
typedef __attribute__((address_space(3))) fp16x4_t lds_fp16x4_t;

// An item of work is a row tile of a kv head and its keys, or a piece of them:
// pieces of one call have the same length in keys, a multiple of a tile's, that of
// the work (in row tiles times 64 keys) over `target` items, but no shorter than
// kMinPiece: those cost more in their partial sums than they save.
constexpr int kWhole = 1 << 30, kMinPiece = 256;
__device__ __forceinline__ int piece_keys(const AttnK& a, uint32_t work, uint32_t target) {
  // (a float's quotient, rounded up past its error: no 64-bit division)
  const float q = (float)work * (float)a.kv_heads / (float)target;
  const uint32_t per = uniform((uint32_t)fminf(q * (1.0f + 0x1p-20f) + 1.0f, 0x1p25f));
  return (int)max(min(per, (uint32_t)(kWhole / kKeys)) * kKeys, (uint32_t)kMinPiece);
}
// What the sequences add up to: work and row tiles.
struct Load {
  uint32_t work, tiles;
};
__device__ __forceinline__ Load load_of(const AttnK& a, const Seq& s0, int lane) {
  Load l = {0, 0};
  for (int b0 = 0; b0 < a.batch; b0 += kWave) {
    const Seq s = b0 == 0 ? s0 : sequence<kRows>(a, b0 + lane);
    l.work += (uint32_t)s.tiles * (uint32_t)((s.kv + kKeys - 1) / kKeys);
    l.tiles += (uint32_t)s.tiles;
  }
  l.work = wave_sum(l.work);
  l.tiles = wave_sum(l.tiles);
  return l;
}

__device__ __forceinline__ int pieces_of(int kv, int piece) { return kv > piece ? (kv + piece - 1) / piece : 1; }

// Item `index` of a kv head: sequence, row tile (the last, which sees the most
// keys, first) and piece.  `slot` numbers the pieces of split row tiles: this
// row tile's first.
struct Item {
  int b, q0, n, kv, rt, piece, slot;
};
__device__ __forceinline__ bool find(const AttnK& a, const Seq& s0, int piece, uint32_t index, int lane, Item* it) {
  uint32_t before = 0, slots = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kWave) {
    const Seq s = b0 == 0 ? s0 : sequence<kRows>(a, b0 + lane);
    const int np = pieces_of(s.kv, piece);
    const uint32_t mine = (uint32_t)s.tiles * (uint32_t)np, split = np > 1 ? mine : 0;
    const uint32_t upto = before + wave_scan(mine), slot_upto = slots + wave_scan(split);
    const uint64_t past = __ballot(upto > index);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int tiles = __builtin_amdgcn_readlane(s.tiles, l), n = __builtin_amdgcn_readlane(np, l);
      const int at = (int)(index - (uint32_t)__builtin_amdgcn_readlane((int)(upto - mine), l));
      it->b = b0 + l;
      it->q0 = __builtin_amdgcn_readlane(s.q0, l);
      it->n = __builtin_amdgcn_readlane(s.n, l);
      it->kv = __builtin_amdgcn_readlane(s.kv, l);
      it->piece = tiles == 1 ? at : uniform(at / tiles);
      it->rt = tiles - 1 - (at - it->piece * tiles);
      it->slot = __builtin_amdgcn_readlane((int)(slot_upto - split), l) + it->rt * n;
      return true;
    }
    before = (uint32_t)__builtin_amdgcn_readlane((int)upto, kWave - 1);
    slots = (uint32_t)__builtin_amdgcn_readlane((int)slot_upto, kWave - 1);
  }
  return false;
}

// The largest of 16 lanes' values, none of them negative or NaN (whose bits are
// ordered as the numbers are), by rotations in the vector unit.
__device__ __forceinline__ float max16(float x) {
  uint32_t v = float_bits(x);
  v = max_from<0x128, 0xF>(v);   // 8, 4, 2 and 1 lanes on
  v = max_from<0x124, 0xF>(v);
  v = max_from<0x122, 0xF>(v);
  return bits_float(max_from<0x121, 0xF>(v));
}

template <int D, bool I8>
__global__ void __launch_bounds__(kThreads, 2) attn_tile_kernel(AttnK a) {
  constexpr int RB = D * (I8 ? 1 : 2);        // bytes of a cached row
  constexpr int NM = D / 32, NJ = D / 16;     // matrix instructions along d: of S and of O
  constexpr int UPR = D / 8;                  // 16-byte units of a row in LDS
  constexpr int SLOT = kRows * (D + 2);
  constexpr int CR = I8 ? RB / 64 : 1;        // 16-byte code loads of a lane and 16-key share
  __shared__ __attribute__((aligned(16))) half_t s_k[2][kKeys * D], s_v[2][kKeys * D];
  __shared__ __attribute__((aligned(16))) float s_ks[2][I8 ? kKeys : 4], s_vs[2][I8 ? kKeys : 4];
  __shared__ __attribute__((aligned(16))) float s_tall[2][kWaves];   // largest finite scale of each wave's 16 values
  __shared__ uint32_t s_odd[I8 ? 1 : 6][kThreads];   // see note_odd
  __shared__ uint32_t s_arrived;

  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane % 16, t = lane / 16;
  // Rows 0 .. 7 put a pair of units in different bank groups (the transposing
  // reads), rows 0 .. 15 one unit (the plain ones).
  auto swizzle = [](int row) { return (UPR == 16 ? (row & 7) << 1 : (row & 6)) | ((row >> 3) & 1); };

  if (a.check_order && !offsets_rise(a, lane)) return;
  const Seq seq0 = sequence<kRows>(a, lane);
  // Two workgroups run on a CU; no pieces if the row tiles alone are near to that.
  const Load load = load_of(a, seq0, lane);
  const uint32_t held = 2 * (uint32_t)a.cus;
  const int piece = (uint64_t)load.tiles * (uint32_t)a.kv_heads * 4 >= (uint64_t)held * 3
                        ? kWhole : piece_keys(a, load.work, held);

  const int place_mask = (1 << a.page_log2) - 1;
  const uint32_t page_rows = (uint32_t)a.kv_heads << a.page_log2;
  const int head = (int)uniform(blockIdx.x % (uint32_t)a.kv_heads);

  for (uint32_t index = blockIdx.x / (uint32_t)a.kv_heads;; index += gridDim.x / (uint32_t)a.kv_heads) {
    Item u;
    if (!find(a, seq0, piece, uniform(index), lane, &u)) break;
    const int rows = u.n * a.group, r0 = u.rt * kRows;
    const int rows_here = min(kRows, rows - r0);
    const int pos0 = u.kv - u.n;
    const int k1 = uniform(min(max(pos0 + (r0 + rows_here - 1) / a.group + 1, 0), u.kv));
    const int pieces = uniform(pieces_of(k1, piece));          // of this row tile: those that hold keys
    if (u.piece >= pieces) continue;
    const int step0 = u.piece * (piece / kKeys);
    const int steps = (k1 + kKeys - 1) / kKeys;
    const int step1 = pieces == 1 ? steps : min(steps, step0 + piece / kKeys);

    const int tile_see_all = uniform(min(pos0 + r0 / a.group + 1, u.kv));   // keys below this are seen by all rows

    // This wave's rows.
    const int w0 = r0 + wave * kWaveRows;
    const bool busy = w0 < rows;
    const int see_all = uniform(busy ? min(pos0 + w0 / a.group + 1, u.kv) : 0);
    const int see_any = uniform(busy ? min(max(pos0 + (min(w0 + kWaveRows, rows) - 1) / a.group + 1, 0), u.kv) : 0);
    half8_t qf[kRT][NM];
    int lim[kRT];
#pragma unroll
    for (int x = 0; x < kRT; ++x) {
      const int r = w0 + 16 * x + c;
      const bool ok = r < rows;
      const int tok = ok ? r / a.group : 0, h = ok ? head * a.group + r % a.group : 0;
      lim[x] = ok ? min(pos0 + tok + 1, k1) : see_any;
      const half_t* qp = a.q + (u.q0 + (int64_t)tok) * a.q_ts + h * a.q_hs;
#pragma unroll
      for (int m = 0; m < NM; ++m) qf[x][m] = ok ? query(qp + 32 * m + 8 * t, a.negate) : zero_half8();
    }

    float4_t acc[kRT][NJ];
    float mref[kRT], l[kRT];
    uint64_t large = 0;   // lanes with a large reference
#pragma unroll
    for (int x = 0; x < kRT; ++x) {
      mref[x] = kNone;
      l[x] = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[x][j] = zero_float4();
    }

    // A wave brings 16 keys of a tile, which lie within one page.  Rows from k1
    // on lie outside the buffer and become zeros.
    const scalar_i32_t* table = (const scalar_i32_t*)(uintptr_t)(a.table + (int64_t)uniform(u.b) * a.table_stride);
    const int last_key = max(k1 - 1, 0);
    auto page_of = [&](int step) {
      return (uint32_t)table[uniform(min(step * kKeys + 16 * wave, last_key) >> a.page_log2)];
    };
    const int64_t head_row = (int64_t)head << a.page_log2;
    const unsigned char* kc = (const unsigned char*)a.kc + head_row * RB;
    const unsigned char* vc = (const unsigned char*)a.vc + head_row * RB;
    // An 8-bit tile on its way, requested as soon as the one before is in LDS.
    // (Two, in two sets of registers, gained nothing at D = 64 and spilled at 128:
    // 8 x 2048 tokens over 4096 keys 1230 us, 1143 with one.)
    struct Codes {
      u32x4_t k[CR], v[CR];
      float ks, vs;
    };
    Codes codes;
    auto fetch = [&](int step, uint32_t page, int buf, Codes& r8) {
      const int key = step * kKeys + 16 * wave;
      const uint64_t row = (uint64_t)min(page, (uint32_t)a.num_pages - 1) * page_rows + (uint32_t)(key & place_mask);
      const uint32_t in = (uint32_t)min(max(k1 - key, 0), 16);
      const __amdgpu_buffer_rsrc_t kr = uniform_rsrc(kc + row * RB, in * RB), vr = uniform_rsrc(vc + row * RB, in * RB);
      if constexpr (I8) {
#pragma unroll
        for (int i = 0; i < CR; ++i) {
          r8.k[i] = buffer_vec<16>(kr, 1024 * i + 16 * lane);
          r8.v[i] = buffer_vec<16>(vr, 1024 * i + 16 * lane);
        }
        const uint32_t so = lane < 16 ? 4 * lane : kOutOfRange;
        const __amdgpu_buffer_rsrc_t ksr = uniform_rsrc(a.ks + head_row + row, in * 4);
        const __amdgpu_buffer_rsrc_t vsr = uniform_rsrc(a.vs + head_row + row, in * 4);
        r8.ks = bits_float(__builtin_amdgcn_raw_buffer_load_b32(ksr, so, 0, 0));
        r8.vs = bits_float(__builtin_amdgcn_raw_buffer_load_b32(vsr, so, 0, 0));
      } else {
#pragma unroll
        for (int i = 0; i < 16 * RB / 1024; ++i) {
          const int r = i * (1024 / RB) + lane / UPR;
          const uint32_t off = (uint32_t)(r * RB + ((lane % UPR) ^ swizzle(r)) * 16);
          const int to = (16 * wave + i * (1024 / RB)) * D;
          __builtin_amdgcn_raw_ptr_buffer_load_lds(kr, (lds_void_t*)(s_k[buf] + to), 16, off, 0, 0, 0);
          __builtin_amdgcn_raw_ptr_buffer_load_lds(vr, (lds_void_t*)(s_v[buf] + to), 16, off, 0, 0, 0);
        }
      }
    };
    // 8-bit tiles: codes to fp16, into LDS.
    auto put = [&](int buf, const Codes& r8) {
      if constexpr (I8) {
#pragma unroll
        for (int i = 0; i < CR; ++i) {
          const int r = 16 * wave + i * (1024 / RB) + lane / (RB / 16), unit = 2 * (lane % (RB / 16));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int to = r * D + ((unit + h) ^ swizzle(r)) * 8;
            *(half8_t*)(s_k[buf] + to) = codes_to_half8(r8.k[i][2 * h], r8.k[i][2 * h + 1]);
            *(half8_t*)(s_v[buf] + to) = codes_to_half8(r8.v[i][2 * h], r8.v[i][2 * h + 1]);
          }
        }
        if (lane < 16) {
          s_ks[buf][16 * wave + lane] = r8.ks * a.scale;
          s_vs[buf][16 * wave + lane] = r8.vs;
        }
        const float tall = max16(r8.vs > 0.0f && r8.vs <= kMaxScale ? r8.vs : 0.0f);
        if (lane == 0) s_tall[buf][wave] = tall;
      }
    };

    auto v_fragment = [&](int buf, int g, int j) {
      const int e = c / 4, q = c % 4;
      half8_t vf;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 32 * g + 16 * h + 4 * t + e;
        const half_t* p = s_v[buf] + row * D + ((2 * j + q / 2) ^ swizzle(row)) * 8 + (q % 2) * 4;
        const half4_t v = __builtin_bit_cast(half4_t, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4_t*)p));
#pragma unroll
        for (int k = 0; k < 4; ++k) vf[4 * h + k] = v[k];
      }
      return vf;
    };

    auto compute = [&](int step, int buf) {
      const int base = step * kKeys + 4 * t;            // the lane's first key
      const bool edge = step * kKeys + kKeys > see_all;
      // Scores.
      float4_t st[kRT][kNS];
#pragma unroll
      for (int n = 0; n < kNS; ++n) {
        const int row = 16 * n + c;
#pragma unroll
        for (int x = 0; x < kRT; ++x) st[x][n] = zero_float4();
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          const half8_t kf = *(const half8_t*)(s_k[buf] + row * D + ((4 * m + t) ^ swizzle(row)) * 8);
#pragma unroll
          for (int x = 0; x < kRT; ++x) st[x][n] = mfma16x16x32(kf, qf[x][m], st[x][n]);
        }
      }
      // Issue order: four fragment reads ahead of the products that use them.
      __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 4, 0);
#pragma unroll
      for (int i = 0; i < kNS * NM - 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedMatrix, kRT, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(kSchedMatrix, 4 * kRT, 0);
      __builtin_amdgcn_sched_barrier(0);
      // The first values are requested under the softmax.
      constexpr int AHEAD = 4;
      half8_t first[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) first[j] = v_fragment(buf, 0, j);
      float4_t vs[kNS];
      if constexpr (I8) {
#pragma unroll
        for (int n = 0; n < kNS; ++n) {
          const float4_t ks = *(const float4_t*)(s_ks[buf] + 16 * n + 4 * t);
          vs[n] = *(const float4_t*)(s_vs[buf] + 16 * n + 4 * t);
#pragma unroll
          for (int x = 0; x < kRT; ++x) st[x][n] *= ks;
        }
      }
      if (edge) {
#pragma unroll
        for (int x = 0; x < kRT; ++x) {
          const int left = opaque(lim[x] - base);
#pragma unroll
          for (int n = 0; n < kNS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (16 * n + i >= left) st[x][n][i] = -INFINITY;
        }
      }
      float top[kRT];
      bool move = false;
#pragma unroll
      for (int x = 0; x < kRT; ++x) {
        top[x] = -INFINITY;
#pragma unroll
        for (int n = 0; n < kNS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) top[x] = fmaxf(top[x], st[x][n][i]);
        top[x] = row_max4(top[x]);
      }
      if constexpr (I8) {
        const float4_t w = *(const float4_t*)s_tall[buf];
        const float tall = scale_exponent(fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])));
#pragma unroll
        for (int x = 0; x < kRT; ++x) {
          float e = tall;
          if (edge) {         // of the values that the row sees
            e = 0.0f;
            const int left = opaque(lim[x] - base);
#pragma unroll
            for (int n = 0; n < kNS; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) e = fmaxf(e, vs[n][i] > kMaxScale || 16 * n + i >= left ? 0.0f : vs[n][i]);
            e = scale_exponent(row_max4(e));
          }
          top[x] += e;
        }
      } else {
#pragma unroll
        for (int x = 0; x < kRT; ++x) top[x] *= a.scale;
      }
#pragma unroll
      for (int x = 0; x < kRT; ++x) move |= top[x] - mref[x] > kHead;
      // A reference is a rounded product, the weights' argument an exact one less it:
      // at scores past 2^24 they differ by whole numbers, past 2^27 by more than
      // fp16's range leaves room for.  So where a reference is large (rarely) the
      // scores are rounded as their maximum was.
      float by = a.scale;
      if (__ballot(move) | large) {
#pragma unroll
        for (int x = 0; x < kRT; ++x) {
          const float to = top[x] - mref[x] > kHead ? top[x] - kStart : mref[x];
          const float f = __builtin_amdgcn_exp2f(mref[x] - to);
          mref[x] = to;
          l[x] *= f;
#pragma unroll
          for (int j = 0; j < NJ; ++j) acc[x][j] *= f;
          if constexpr (!I8) large |= __ballot(fabsf(to) > kLarge && to != kNone);
        }
        if (!I8 && large) {
          by = 1.0f;
#pragma unroll
          for (int x = 0; x < kRT; ++x)
#pragma unroll
            for (int n = 0; n < kNS; ++n) st[x][n] *= a.scale;
        }
      }
      half8_t pf[kRT][kNG];
#pragma unroll
      for (int x = 0; x < kRT; ++x) {
#pragma unroll
        for (int n = 0; n < kNS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float s = st[x][n][i];
            float p = __builtin_amdgcn_exp2f(I8 ? s - mref[x] : __builtin_fmaf(s, by, -mref[x]));
            l[x] += p;
            if constexpr (I8) p *= vs[n][i];
            pf[x][n / 2][4 * (n % 2) + i] = (half_t)p;
          }
      }
      if constexpr (I8) {
        if (edge) {   // a scale that a row must not see may be infinite or NaN
#pragma unroll
          for (int x = 0; x < kRT; ++x) {
            const int left = opaque(lim[x] - base);
#pragma unroll
            for (int n = 0; n < kNS; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (16 * n + i >= left) pf[x][n / 2][4 * (n % 2) + i] = (half_t)0.0f;
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      // O^T += V^T P^T, ahead of the other workgroup's softmax: a product takes one
      // issue of its sixteen cycles.
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int g = 0; g < kNG; ++g)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const half8_t vf = g == 0 && j < AHEAD ? first[j] : v_fragment(buf, g, j);
#pragma unroll
          for (int x = 0; x < kRT; ++x) acc[x][j] = mfma16x16x32(vf, pf[x][g], acc[x][j]);
        }
#pragma unroll
      for (int i = 0; i < kNG * NJ - AHEAD; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedLdsRead, 2, 1);
        __builtin_amdgcn_sched_group_barrier(kSchedMatrix, kRT, 1);
      }
      __builtin_amdgcn_sched_group_barrier(kSchedMatrix, AHEAD * kRT, 1);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(0);
    };

    // Infinities and NaN among values that some row must not see (a weight of
    // zero would not remove them): all waves look through the tile, alike; if
    // there are any (rarely), each notes which of its sums they reach (the
    // product of their kinds with what each row sees), bits that `spread` turns
    // into the values when the sums are complete, and they leave the tile.
    bool noted = false;
    auto note_odd = [&](int step, int buf) {
      bool odd = false;
#pragma unroll
      for (int i = 0; i < kKeys * D / 8 / kWave; ++i) {
        const u32x4_t w = *(const u32x4_t*)(s_v[buf] + (i * kWave + lane) * 8);
#pragma unroll
        for (int k = 0; k < 4; ++k) odd |= half2_not_finite(w[k]);
      }
      if (!__ballot(odd)) return;
      uint32_t bits[6];
#pragma unroll
      for (int i = 0; i < 6; ++i) bits[i] = noted ? s_odd[i][threadIdx.x] : 0u;
      noted = true;
      if (busy) {
        const int base = step * kKeys + 4 * t;
#pragma unroll
        for (int g = 0; g < kNG; ++g)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const u32x4_t w = __builtin_bit_cast(u32x4_t, v_fragment(buf, g, j));
            u32x4_t kind;
#pragma unroll
            for (int k = 0; k < 4; ++k) kind[k] = kind_of(w[k] & 0xFFFFu) | kind_of(w[k] >> 16) << 16;
#pragma unroll
            for (int x = 0; x < kRT; ++x) {
              half8_t seen;
#pragma unroll
              for (int k = 0; k < 8; ++k)
                seen[k] = (half_t)(base + 32 * g + 16 * (k / 4) + k % 4 < lim[x] ? 1.0f : 0.0f);
              const float4_t kinds = mfma16x16x32(__builtin_bit_cast(half8_t, kind), seen, zero_float4());
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int n = (int)kinds[k];
                const uint32_t bit = 1u << (4 * j + k);
                bits[x] |= n & 63 ? bit : 0u;
                bits[2 + x] |= n & 4032 ? bit : 0u;
                bits[4 + x] |= n >> 12 ? bit : 0u;
              }
            }
          }
      }
#pragma unroll
      for (int i = 0; i < 6; ++i) s_odd[i][threadIdx.x] = bits[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kKeys * D / 8 / kThreads; ++i) {
        u32x4_t* p = (u32x4_t*)(s_v[buf] + (i * kThreads + threadIdx.x) * 8);
        u32x4_t w = *p;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = ((w[k] & 0x7C00u) == 0x7C00u ? 0u : w[k] & 0xFFFFu) |
                 ((w[k] & 0x7C000000u) == 0x7C000000u ? 0u : w[k] & 0xFFFF0000u);
        *p = w;
      }
      __syncthreads();
    };
    auto spread = [&]() {
#pragma unroll
      for (int x = 0; x < kRT; ++x) {
        const uint32_t inf = s_odd[x][threadIdx.x], minus = s_odd[2 + x][threadIdx.x], nan = s_odd[4 + x][threadIdx.x];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t bit = 1u << (4 * j + k);
            if (inf & bit) acc[x][j][k] += INFINITY;
            if (minus & bit) acc[x][j][k] -= INFINITY;
            if (nan & bit) acc[x][j][k] = NAN;
          }
      }
    };

    uint32_t page = page_of(step0);             // of the tile requested next
    if constexpr (I8) {
      auto one = [&](int step, int buf) {
        put(buf, codes);
        __syncthreads();                        // the tile is in LDS; the other stage is free
        if (step + 1 < step1) fetch(step + 1, page, 0, codes);
        page = page_of(step + 2);
        if (step * kKeys < see_any) compute(step, buf);
      };
      if (step0 < step1) fetch(step0, page, 0, codes);
      page = page_of(step0 + 1);
      for (int step = step0; step < step1; step += 2) {
        one(step, 0);
        if (step + 1 < step1) one(step + 1, 1);
      }
    } else {
      if (step0 < step1) fetch(step0, page, step0 & 1, codes);
      page = page_of(step0 + 1);
      for (int step = step0; step < step1; ++step) {
        const int buf = step & 1;
        // Every wave waits for its own copies of this tile, also one that computed
        // nothing since it asked for them (a barrier waits for no copies); then
        // the tile is in LDS, and the other stage is free.  (Written so that the
        // compiler does not see the wait: told of it, it waits for the next tile's
        // copies before this tile's scores, 1020 instead of 960 us for 8 x 2048
        // tokens over 4096 keys at head dimension 128.)
        drain_vm();
        __syncthreads();
        if (step + 1 < step1) {
          fetch(step + 1, page, buf ^ 1, codes);
          page = page_of(step + 2);
        }
        if (step * kKeys + kKeys > tile_see_all) note_odd(step, buf);
        if (step * kKeys < see_any) compute(step, buf);
      }
    }

    // Lane (c, t) holds row c at d = 16 j + 4 t + i.
    if constexpr (!I8)
      if (noted) spread();
#pragma unroll
    for (int x = 0; x < kRT; ++x) l[x] = row_sum4(l[x]);
    auto write = [&]() {
#pragma unroll
      for (int x = 0; x < kRT; ++x) {
        const int r = w0 + 16 * x + c;
        if (r >= rows) continue;
        const float inv = l[x] == 0.0f ? 0.0f : 1.0f / l[x];   // nothing seen: zeros
        half_t* o = a.out + ((u.q0 + (int64_t)(r / a.group)) * a.q_heads + head * a.group + r % a.group) * D + 4 * t;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          half4_t h;
#pragma unroll
          for (int k = 0; k < 4; ++k) h[k] = (half_t)(acc[x][j][k] * inv);
          *(half4_t*)(o + 16 * j) = h;
        }
      }
    };
    if (pieces == 1) {
      write();
    } else {
      // A partial result, in the lanes' own order.
      const __amdgpu_buffer_rsrc_t pr = make_rsrc(a.part, (uint32_t)a.part_bytes);
      const uint32_t slot0 = (uint32_t)u.slot * (uint32_t)a.kv_heads + (uint32_t)head;   // pieces: kv_heads apart
      // (a split row tile has two slots at least)
      uint32_t* counter = a.counters + (uint32_t)(u.slot / 2) * (uint32_t)a.kv_heads + (uint32_t)head;
      const uint32_t own = (slot0 + (uint32_t)(u.piece * a.kv_heads)) * (uint32_t)(SLOT * 4);
      const uint32_t sums = (uint32_t)wave * (kRT * NJ * 1024) + (uint32_t)lane * 16;
      const uint32_t stats = (uint32_t)(kRows * D + wave * kWaveRows + c) * 4;
      if (busy) {
#pragma unroll
        for (int x = 0; x < kRT; ++x) {
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[x][j]), pr,
                                                   own + sums + (x * NJ + j) * 1024, 0, kCachePolicySc1);
          if (t == 0) {
            __builtin_amdgcn_raw_buffer_store_b32(float_bits(mref[x]), pr, own + stats + 64 * x, 0, kCachePolicySc1);
            __builtin_amdgcn_raw_buffer_store_b32(float_bits(l[x]), pr, own + stats + 64 * x + kRows * 4, 0,
                                                  kCachePolicySc1);
          }
        }
      }
      drain_vm();
      __syncthreads();
      if (threadIdx.x == 0) s_arrived = add_dev_u32(counter, 1u);
      __syncthreads();
      if (s_arrived == (uint32_t)pieces - 1) {
        if (threadIdx.x == 0) st_dev_u32(counter, 0u);
        if (busy) {
          // All pieces in order, this workgroup's own among them.
#pragma unroll
          for (int x = 0; x < kRT; ++x) {
            mref[x] = kNone;
            l[x] = 0.0f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[x][j] = zero_float4();
          }
          for (int i = 0; i < pieces; ++i) {
            const uint32_t p = (slot0 + (uint32_t)(i * a.kv_heads)) * (uint32_t)(SLOT * 4);
#pragma unroll
            for (int x = 0; x < kRT; ++x) {
              float4_t o[NJ];
#pragma unroll
              for (int j = 0; j < NJ; ++j) o[j] = buffer_load_f4_dev(pr, p + sums + (x * NJ + j) * 1024);
              const float m = bits_float(__builtin_amdgcn_raw_buffer_load_b32(pr, p + stats + 64 * x, 0, kCachePolicySc1));
              const float n = bits_float(
                  __builtin_amdgcn_raw_buffer_load_b32(pr, p + stats + 64 * x + kRows * 4, 0, kCachePolicySc1));
              const float to = fmaxf(mref[x], m);
              const float f = __builtin_amdgcn_exp2f(mref[x] - to), g = __builtin_amdgcn_exp2f(m - to);
              mref[x] = to;
              l[x] = l[x] * f + n * g;
#pragma unroll
              for (int j = 0; j < NJ; ++j) acc[x][j] = acc[x][j] * f + o[j] * g;
            }
          }
          write();
        }
      }
    }
    __syncthreads();                            // the stages are free for the next unit
  }
}

}  // namespace

hipError_t launch_attention_tiles(const AttnK& k, int dim, bool i8, int grid, hipStream_t st) {
  const dim3 g(grid), b(kThreads);
  if (dim == 64) {
    if (i8) attn_tile_kernel<64, true><<<g, b, 0, st>>>(k);
    else attn_tile_kernel<64, false><<<g, b, 0, st>>>(k);
  } else {
    if (i8) attn_tile_kernel<128, true><<<g, b, 0, st>>>(k);
    else attn_tile_kernel<128, false><<<g, b, 0, st>>>(k);
  }
  return hipGetLastError();
}

}  // namespace spear
