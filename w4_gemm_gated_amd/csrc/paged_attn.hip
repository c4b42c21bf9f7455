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
// multiplies its scores, a value's scale its weight, divided by a power of two
// above the scales that the row has seen so far (moved the same way), so that
// the fp16 weights keep their range.
//
// Long sequences with few rows are split over workgroups.  The lengths are on
// the device, so every workgroup finds its item by itself: the chunk length
// follows from the total work and the GPU's size, and a scan over the
// sequences locates the item (64 sequences a step).  Split items leave their
// sums in the workspace in fp32; a second launch joins them in order.
#include "serve_internal.h"
#include "device_common.h"

namespace spear {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kNone = -1e30f;      // reference of a row that has seen no key
constexpr float kHead = 14.0f;       // a maximum this far above the reference moves it
constexpr float kStart = 6.0f;       // .. to this far below the maximum
constexpr float kMaxScale = 1e30f;   // scales above this do not move the common one

struct AttnK {
  const half_t* q;
  int64_t q_ts, q_hs;
  const int32_t *cu, *lens, *table;
  int64_t table_stride;
  const void *kc, *vc;
  const float *ks, *vs;
  half_t* out;
  float* part;
  int32_t batch, total_q, q_heads, kv_heads, group, max_kv, page_log2, num_pages;
  int32_t target, min_chunk;   // per kv head
  float scale;                 // scale * log2(e)
};

// ------------------------------------------------------------- the schedule

struct Seq {
  int q0, n, kv, tiles;   // first row of q, new tokens, cached tokens, row tiles
};

template <int R>
__device__ __forceinline__ Seq sequence(const AttnK& a, int b) {
  Seq s = {0, 0, 0, 0};
  if (b < a.batch) {
    s.q0 = min(max(a.cu[b], 0), a.total_q);
    s.n = min(max(a.cu[b + 1], s.q0), a.total_q) - s.q0;
    s.kv = min(max(a.lens[b], 0), a.max_kv);
    s.tiles = (int)(((int64_t)s.n * a.group + R - 1) / R);
  }
  return s;
}

__device__ __forceinline__ int64_t wave_sum(int64_t x) {
#pragma unroll
  for (int o = 1; o < kWave; o *= 2) x += __shfl_xor(x, o);
  return x;
}
__device__ __forceinline__ int wave_scan(int x, int lane) {
#pragma unroll
  for (int o = 1; o < kWave; o *= 2) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Keys of a split item: the whole work over the items aimed at, whole rounds
// of the four waves.
template <int R, int KT>
__device__ __forceinline__ int chunk_keys(const AttnK& a, int lane) {
  int64_t work = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kWave) {
    const Seq s = sequence<R>(a, b0 + lane);
    work += (int64_t)s.tiles * s.kv;
  }
  work = wave_sum(work);
  const int64_t c = (work + a.target - 1) / a.target;
  const int64_t most = c > a.min_chunk ? c : a.min_chunk;
  return (int)min((most + KT * kWaves - 1) / (KT * kWaves) * (KT * kWaves), (int64_t)1 << 30);
}

__device__ __forceinline__ int pieces(int kv, int chunk) { return kv > chunk ? (kv + chunk - 1) / chunk : 1; }

// What one item covers.  COUNT 0: items of the main launch (index = row tile x
// piece); 1: rows of split sequences (the joining launch).  The first partial
// slot of the sequence and of its pieces counts split sequences only.
struct Item {
  int b, q0, n, kv, at, pieces, slot;   // at: index within the sequence
  bool found;
};
template <int R, int COUNT>
__device__ __forceinline__ Item find(const AttnK& a, int chunk, int index, int lane) {
  Item it;
  it.found = false;
  int before = 0, slots = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kWave) {
    const Seq s = sequence<R>(a, b0 + lane);
    const int np = pieces(s.kv, chunk);
    const int split = np > 1 ? s.tiles * np : 0;
    const int mine = COUNT == 0 ? s.tiles * np : np > 1 ? s.n * a.group : 0;
    const int upto = before + wave_scan(mine, lane);
    const uint64_t past = __ballot(upto > index);
    const int slot_upto = slots + wave_scan(split, lane);
    if (past) {
      const int l = __builtin_ctzll(past);
      it.found = true;
      it.b = b0 + l;
      it.q0 = __shfl(s.q0, l);
      it.n = __shfl(s.n, l);
      it.kv = __shfl(s.kv, l);
      it.pieces = __shfl(np, l);
      it.at = index - __shfl(upto - mine, l);
      it.slot = __shfl(slot_upto - split, l);
      break;
    }
    before = __shfl(upto, kWave - 1);
    slots = __shfl(slot_upto, kWave - 1);
  }
  return it;
}

// -------------------------------------------------------------- small pieces

// Over the four lanes (c, 0..3) that hold row c.
__device__ __forceinline__ float row_max4(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float row_sum4(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// Codes b0 and b1 (bytes i of two words, sign included) -> two fp16 values.
// Byte | 0x6400 with the sign bit flipped is the fp16 number 1024 + 128 + code.
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t bytes) {   // bytes 0x00b1'00b0
  const half2_t bias = {(half_t)1152.0f, (half_t)1152.0f};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, bytes ^ 0x64806480u) - bias);
}
// Eight codes of two words, in order.
__device__ __forceinline__ half8_t codes_to_half8(uint32_t lo, uint32_t hi) {
  u32x4_t r;
  r[0] = codes_to_half2(__builtin_amdgcn_perm(lo, lo, 0x0c010c00u));
  r[1] = codes_to_half2(__builtin_amdgcn_perm(lo, lo, 0x0c030c02u));
  r[2] = codes_to_half2(__builtin_amdgcn_perm(hi, hi, 0x0c010c00u));
  r[3] = codes_to_half2(__builtin_amdgcn_perm(hi, hi, 0x0c030c02u));
  return __builtin_bit_cast(half8_t, r);
}

template <int BYTES> struct Vec;
template <> struct Vec<4> { typedef uint32_t type __attribute__((ext_vector_type(1))); };
template <> struct Vec<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <> struct Vec<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };

__device__ __forceinline__ bool half2_not_finite(uint32_t w) {
  return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
}

// ------------------------------------------------------------ the main kernel

template <int D, bool I8, int RT>
__global__ void __launch_bounds__(kThreads) attn_kernel(AttnK a) {
  constexpr int R = 16 * RT;
  constexpr int KT = I8 ? 64 : 32;            // keys of a wave's tile: the same bytes in flight
  constexpr int NS = KT / 16;                 // 16-key tiles
  constexpr int NG = KT / 32;                 // 32-key groups
  constexpr int E = I8 ? 1 : 2;               // bytes of a cached value
  constexpr int NM = D / 32;                  // matrix instructions along d
  constexpr int KL = D * E / 64;              // 16-byte K loads of a lane and 16-key tile
  constexpr int DL = D / 16;                  // d values of a lane's V load
  typedef typename Vec<DL * E>::type vvec_t;
  constexpr int OS = D + 4;                   // row stride of the sums in LDS
  __shared__ float s_o[kWaves][R][OS];
  __shared__ float s_m[kWaves][R], s_l[kWaves][R];

  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int c = lane % 16, t = lane / 16;
  const int head = blockIdx.x % a.kv_heads;
  const int chunk = chunk_keys<R, KT>(a, lane);

  for (int index = blockIdx.x / a.kv_heads;; index += gridDim.x / a.kv_heads) {
    const Item it = find<R, 0>(a, chunk, index, lane);
    if (!it.found) break;
    const int rt = it.at / it.pieces, piece = it.at % it.pieces;
    const int rows = it.n * a.group;                     // of the sequence
    const int r0 = rt * R;
    const int first_tok = r0 / a.group;
    const int last_tok = min(r0 + R, rows) - 1 >= 0 ? (min(r0 + R, rows) - 1) / a.group : 0;
    const int pos0 = it.kv - it.n;                       // position of token 0
    const int see_all = min(pos0 + first_tok + 1, it.kv);          // keys below this are seen by every row
    const int k_end = min(max(pos0 + last_tok + 1, 0), it.kv);     // .. from this on by none
    const int k0 = piece * chunk;
    const int k1 = it.pieces == 1 ? k_end : min(k0 + chunk, k_end);

    // Queries as B operands; the k order follows the K loads' below.
    half8_t qf[RT][NM];
    int lim[RT];                                         // keys below this are seen by the lane's row
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      const int r = r0 + 16 * x + c;
      const int tok = r / a.group, h = head * a.group + r % a.group;
      const bool ok = r < rows;
      lim[x] = ok ? pos0 + tok + 1 : k_end;
      const half_t* qp = a.q + (it.q0 + (int64_t)(ok ? tok : 0)) * a.q_ts + (ok ? h : 0) * a.q_hs;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const int d = I8 ? 64 * (m / 2) + 16 * t + 8 * (m % 2) : 32 * m + 8 * t;
        qf[x][m] = ok ? load_half8(qp + d) : zero_half8();
      }
    }

    float4_t acc[RT][DL];
    float mref[RT], l[RT], vref[RT];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      mref[x] = kNone;
      l[x] = 0.0f;
      vref[x] = 0.0f;
#pragma unroll
      for (int j = 0; j < DL; ++j) acc[x][j] = zero_float4();
    }

    const int32_t* table = a.table + (int64_t)it.b * a.table_stride;
    const int place_mask = (1 << a.page_log2) - 1;
    for (int base = k0 + wave * KT; base < k1; base += kWaves * KT) {
      // Loads.  A 16-key tile lies within one page; tiles past the end read
      // the last page that holds keys.
      u32x4_t kr[NS][KL];
      vvec_t vr[NG][8];
      float4_t ksc[NS], vsc[NS];
      const unsigned char* vbase[NS];
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const int key = min(base + 16 * n, (k1 - 1) & ~15);
        const uint32_t page = min((uint32_t)table[key >> a.page_log2], (uint32_t)a.num_pages - 1);
        const int64_t row = (((int64_t)page * a.kv_heads + head) << a.page_log2) + (key & place_mask);
        const unsigned char* kb = (const unsigned char*)a.kc + row * (D * E);
        vbase[n] = (const unsigned char*)a.vc + row * (D * E);
#pragma unroll
        for (int i = 0; i < KL; ++i) kr[n][i] = *(const u32x4_t*)(kb + c * (D * E) + 64 * i + 16 * t);
        if constexpr (I8) {
          ksc[n] = *(const float4_t*)(a.ks + row + 4 * t);
          vsc[n] = *(const float4_t*)(a.vs + row + 4 * t);
        }
      }
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int s = 0; s < 8; ++s)
          vr[g][s] = *(const vvec_t*)(vbase[2 * g + s / 4] + (4 * t + s % 4) * (D * E) + c * (DL * E));

      // Scores.
      float4_t st[RT][NS];
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
      }
      const bool edge = base + KT > min(see_all, k1);
      float top[RT], vmax[RT];
      bool move = false;
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        if constexpr (I8) {
          // The largest finite scale among the values the row sees: others must
          // not take the range from its weights.
          vmax[x] = 0.0f;
#pragma unroll
          for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool out = vsc[n][i] > kMaxScale || (edge && base + 16 * n + 4 * t + i >= min(lim[x], k1));
              vmax[x] = fmaxf(vmax[x], out ? 0.0f : vsc[n][i]);
            }
          vmax[x] = row_max4(vmax[x]);
          move |= vmax[x] > vref[x];
        }
        top[x] = -INFINITY;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float s = st[x][n][i] * a.scale;
            if constexpr (I8) s *= ksc[n][i];
            if (edge && base + 16 * n + 4 * t + i >= min(lim[x], k1)) s = -INFINITY;
            st[x][n][i] = s;
            top[x] = fmaxf(top[x], s);
          }
        top[x] = row_max4(top[x]);
        move |= top[x] > mref[x] + kHead;
      }
      if (__ballot(move)) {
#pragma unroll
        for (int x = 0; x < RT; ++x) {
          float vscale = 1.0f;
          if constexpr (I8) {
            if (vmax[x] > vref[x]) {   // the next power of two
              const float to = bits_float((float_bits(vmax[x]) & 0x7F800000u) + 0x00800000u);
              vscale = vref[x] > 0.0f ? vref[x] / to : 0.0f;
              vref[x] = to;
            }
          }
          const float to = top[x] > mref[x] + kHead ? top[x] - kStart : mref[x];
          const float f = __builtin_amdgcn_exp2f(mref[x] - to);
          mref[x] = to;
          l[x] *= f;
#pragma unroll
          for (int j = 0; j < DL; ++j) acc[x][j] *= f * vscale;
        }
      }
      // Weights (B operands) and, for V's edge, which lanes see which keys.
      half8_t pf[RT][NG];
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        // the reciprocal of a power of two, exactly
        const float vinv = I8 && vref[x] > 0.0f ? bits_float(0x7F000000u - float_bits(vref[x])) : 0.0f;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float p = __builtin_amdgcn_exp2f(st[x][n][i] - mref[x]);
            l[x] += p;
            if constexpr (I8) {
              const float w = p * (vsc[n][i] * vinv);
              p = edge && base + 16 * n + 4 * t + i >= min(lim[x], k1) ? 0.0f : w;
            }
            pf[x][n / 2][4 * (n % 2) + i] = (half_t)p;
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
            for (int s = 0; s < 8; ++s) {
              const int key = base + 32 * g + 16 * (s / 4) + 4 * t + s % 4;
#pragma unroll
              for (int w = 0; w < DL / 2; ++w) {
                if (key >= k1) vr[g][s][w] = 0u;
                else if (key >= see_all) odd |= half2_not_finite(vr[g][s][w]);
              }
            }
          if (__ballot(odd)) {
            // Rare: such keys leave the matrix product, and each row that sees
            // them adds them by itself.
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
              for (int s = 0; s < 8; ++s) {
                const int n = 2 * g + s / 4, i = s % 4;
                if (base + 16 * n + 4 * t + i >= see_all)
#pragma unroll
                  for (int w = 0; w < DL / 2; ++w) vr[g][s][w] = 0u;
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) {
                  const int key = base + 16 * n + 4 * tt + i;
                  if (key < see_all || key >= k1) continue;
                  const half_t* row = (const half_t*)(vbase[n] + (4 * tt + i) * (D * E));
#pragma unroll
                  for (int x = 0; x < RT; ++x) {
                    const float p = __shfl((float)pf[x][g][s], c + 16 * tt);
                    if (key < lim[x])
#pragma unroll
                      for (int j = 0; j < DL; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[x][j][k] += p * (float)row[DL * (4 * t + k) + j];
                  }
                }
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
    }

    // Join the waves.  Lane (c, t) holds row c at d = DL (4 t + k) + j.
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      l[x] = row_sum4(l[x]);
      const float f = I8 ? vref[x] : 1.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < DL; j += 4) {
          float4_t o = {acc[x][j][k] * f, acc[x][j + 1][k] * f, acc[x][j + 2][k] * f, acc[x][j + 3][k] * f};
          *(float4_t*)&s_o[wave][16 * x + c][DL * (4 * t + k) + j] = o;
        }
      if (t == 0) {
        s_m[wave][16 * x + c] = mref[x];
        s_l[wave][16 * x + c] = l[x];
      }
    }
    __syncthreads();
    constexpr int UNITS = R * D / 8;
    for (int u = threadIdx.x; u < UNITS; u += kThreads) {
      const int row = u / (D / 8), d = u % (D / 8) * 8;
      const int r = r0 + row;
      if (r >= rows) break;
      float M = s_m[0][row];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) M = fmaxf(M, s_m[w][row]);
      float sum = 0.0f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(s_m[w][row] - M);
        sum += s_l[w][row] * f;
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] += s_o[w][row][d + k] * f;
      }
      if (it.pieces == 1) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // nothing seen: zeros
        half8_t h;
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = (half_t)(o[k] * inv);
        const int tok = r / a.group, qh = head * a.group + r % a.group;
        *(half8_t*)(a.out + ((it.q0 + (int64_t)tok) * a.q_heads + qh) * D + d) = h;
      } else {
        const int64_t slot = (int64_t)(it.slot + it.at) * a.kv_heads + head;
        float* p = a.part + slot * (R * (D + 2));
        *(float4_t*)(p + row * D + d) = *(float4_t*)&o[0];
        *(float4_t*)(p + row * D + d + 4) = *(float4_t*)&o[4];
        if (d == 0) {
          p[R * D + row] = M;
          p[R * D + R + row] = sum;
        }
      }
    }
    __syncthreads();
  }
}

// Joins the pieces of split rows: a workgroup takes one row of one kv head, its
// waves a quarter of the pieces each, all in a fixed order.
template <int D, int KT, int R>
__global__ void __launch_bounds__(kThreads) attn_combine_kernel(AttnK a) {
  constexpr int DL = D / kWave;
  __shared__ float s_o[kWaves][D], s_m[kWaves], s_l[kWaves];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int head = blockIdx.x % a.kv_heads;
  const int chunk = chunk_keys<R, KT>(a, lane);
  for (int index = blockIdx.x / a.kv_heads;; index += gridDim.x / a.kv_heads) {
    const Item it = find<R, 1>(a, chunk, index, lane);
    if (!it.found) break;
    const int rt = it.at / R, row = it.at % R;
    const float* base = a.part + ((int64_t)(it.slot + rt * it.pieces) * a.kv_heads + head) * (R * (D + 2));
    const int64_t step = (int64_t)a.kv_heads * (R * (D + 2));
    float M = kNone, sum = 0.0f, o[DL];
#pragma unroll
    for (int k = 0; k < DL; ++k) o[k] = 0.0f;
    for (int i0 = wave; i0 < it.pieces; i0 += 8 * kWaves) {
      float pm[8], pl[8], po[8][DL];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int piece = i0 + i * kWaves;
        const float* p = base + min(piece, it.pieces - 1) * step;
        pm[i] = p[R * D + row];
        pl[i] = p[R * D + R + row];
#pragma unroll
        for (int k = 0; k < DL; ++k) po[i][k] = p[row * D + lane * DL + k];
        if (piece >= it.pieces) {
          pm[i] = kNone;
          pl[i] = 0.0f;
#pragma unroll
          for (int k = 0; k < DL; ++k) po[i][k] = 0.0f;
        }
      }
      float to = M;
#pragma unroll
      for (int i = 0; i < 8; ++i) to = fmaxf(to, pm[i]);
      const float f = __builtin_amdgcn_exp2f(M - to);
      M = to;
      sum *= f;
#pragma unroll
      for (int k = 0; k < DL; ++k) o[k] *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = __builtin_amdgcn_exp2f(pm[i] - M);
        sum += pl[i] * g;
#pragma unroll
        for (int k = 0; k < DL; ++k) o[k] += po[i][k] * g;
      }
    }
#pragma unroll
    for (int k = 0; k < DL; ++k) s_o[wave][lane * DL + k] = o[k];
    if (lane == 0) {
      s_m[wave] = M;
      s_l[wave] = sum;
    }
    __syncthreads();
    if (threadIdx.x < D) {
      const int d = threadIdx.x;
      float to = s_m[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) to = fmaxf(to, s_m[w]);
      float total = 0.0f, v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float g = __builtin_amdgcn_exp2f(s_m[w] - to);
        total += s_l[w] * g;
        v += s_o[w][d] * g;
      }
      const int tok = it.at / a.group, qh = head * a.group + it.at % a.group;
      a.out[((it.q0 + (int64_t)tok) * a.q_heads + qh) * D + d] = (half_t)(total == 0.0f ? 0.0f : v / total);
    }
    __syncthreads();
  }
}

template <int D, bool I8, int RT>
hipError_t launch(const AttnK& k, const AttnPlan& p, hipStream_t st) {
  attn_kernel<D, I8, RT><<<dim3(p.grid), dim3(kThreads), 0, st>>>(k);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.combine_grid == 0) return e;
  attn_combine_kernel<D, I8 ? 64 : 32, 16 * RT><<<dim3(p.combine_grid), dim3(kThreads), 0, st>>>(k);
  return hipGetLastError();
}

}  // namespace

AttnPlan attn_plan(const spear_attention_desc_t& d, int cus) {
  AttnPlan p;
  const int64_t H = d.kv.kv_heads, group = d.q_heads / H;
  p.row_tiles = (int64_t)d.max_q * group > 16 ? 2 : 1;
  const int64_t R = 16 * p.row_tiles;
  const int64_t per_head = ceil_div((int64_t)4 * cus, H);   // split items aimed at
  p.target = (int)per_head;
  p.min_chunk = d.kv.dtype == SPEAR_KV_INT8 ? 256 : 128;     // one tile for each wave
  // Row tiles: no sequence has more than its rows need, nor more than one not full.
  int64_t tiles = d.batch + (int64_t)d.total_q * group / R;
  const int64_t most = d.batch * ceil_div((int64_t)d.max_q * group, R);
  if (most < tiles) tiles = most;
  const int64_t max_kv = (int64_t)d.max_pages * d.kv.page_size;
  const bool split = max_kv > p.min_chunk;
  const int64_t cap = (int64_t)16 * cus * 4;                 // workgroups; the rest in turns
  int64_t items = tiles + (split ? per_head : 0);
  if (items * H > cap) items = ceil_div(cap, H);
  p.grid = (int)(items * H);
  // A sequence is split when it is longer than the chunk, so its pieces are
  // fewer than twice its share of the target.
  const int64_t slots = split ? 2 * per_head : 0;
  int64_t rows = (int64_t)d.total_q * group;
  if (rows * H > 4 * cus) rows = ceil_div((int64_t)4 * cus, H);
  p.combine_grid = split ? (int)(rows * H) : 0;
  p.part = kSyncHeaderBytes;
  p.bytes = split ? p.part + (size_t)(slots * H * R * (d.kv.head_dim + 2) * 4) : 0;
  return p;
}

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, void* stream) {
  AttnK k;
  k.q = (const half_t*)a.q; k.q_ts = a.q_ts; k.q_hs = a.q_hs;
  k.cu = a.cu_q; k.lens = a.kv_lens; k.table = a.table; k.table_stride = a.table_stride;
  k.kc = a.k_cache; k.vc = a.v_cache; k.ks = a.k_scale; k.vs = a.v_scale;
  k.out = (half_t*)a.out; k.part = a.part;
  k.batch = a.batch; k.total_q = a.total_q; k.q_heads = a.q_heads; k.kv_heads = a.kv.heads;
  k.group = a.group; k.max_kv = a.max_kv; k.page_log2 = a.kv.page_log2; k.num_pages = a.kv.num_pages;
  k.target = p.target; k.min_chunk = p.min_chunk;
  k.scale = a.scale * kLog2e;
  const hipStream_t st = (hipStream_t)stream;
  const bool i8 = a.kv.dtype == SPEAR_KV_INT8, two = p.row_tiles == 2;
  if (a.kv.dim == 64) {
    if (i8) return two ? launch<64, true, 2>(k, p, st) : launch<64, true, 1>(k, p, st);
    return two ? launch<64, false, 2>(k, p, st) : launch<64, false, 1>(k, p, st);
  }
  if (i8) return two ? launch<128, true, 2>(k, p, st) : launch<128, true, 1>(k, p, st);
  return two ? launch<128, false, 2>(k, p, st) : launch<128, false, 1>(k, p, st);
}

}  // namespace spear
