// kq_kv_attention: attention over key/value rows held in 4 bits.
//
//   out = sum_j softmax_j(scale q . k_j) v_j,   k_j, v_j = D (c - 8)
//
// One pass over the keys with a running maximum and sum.  A workgroup takes a
// run of 64-key steps of one 16-row tile of a (request, kv head); its four
// waves take steps in turn, each with sums of its own, merged through LDS at
// the end.  Both products run on v_mfma_f32_16x16x32_f16, transposed so that
// nothing moves between lanes in between:
//   S^T [16 keys x 16 rows] = K [16 x d] Q^T; lane l holds row l % 16, keys
//     4 (l / 16) .. + 3 of each of a step's four 16-key groups.
//   O^T [16 d x 16 rows] += V^T [16 d x 32 keys] P^T; its operand wants for
//     lane l eight keys of row l % 16, and which key stands in which place is
//     free as long as V^T agrees, so the places are given to the very keys
//     whose probabilities the lane holds.
// K operands: lane l reads quarter l / 16 of key l % 16's codes, contiguous in
// memory; the matrix steps then run over values in that order, and so do the
// queries.  V operands need eight keys of one value per lane: codes go through
// LDS and come back through the 4-bit transposing read (ds_read_b64_tr_b4: 16
// rows of 16 nibbles per 16 lanes, the row addresses free), which hands lane l
// value l % 16 of 16 keys.  Codes become float16 by or-ing them into 1024's
// mantissa, times the block's scale.
//
// Measured (8 kv heads, groups of 4, d = 128): 64 requests of 200 to 8192 keys
// 67 us, 4.0 TB/s of cache; 4 of 131072 keys 121 us, 4.9 TB/s (a plain read of
// as many bytes 43 and 91 us).  Every byte is fetched once; the vector units
// are busy 52 and 59% of the time (416 of a step's 500 operations unpack),
// waves wait 32 and 24% of theirs: two waves a SIMD do not hide all of a step's
// loads and LDS trips behind the other's unpacking.  Short ones are bound by
// latency: 330 keys of one request 9 us with its launch.
#include "kq_kv_attn.h"

namespace kq {
namespace {

// Waves of a workgroup: four, or eight where short requests leave the GPU
// mostly idle (a step of one wave takes 2 us, so a request of 330 keys, six
// steps, is 11 us with four waves and 9 us with eight).
constexpr int WAVES = 4, MORE_WAVES = 8;

// LDS of one wave: a step's rows of codes and their scales, keys and values.
// Row strides are odd multiples of 16 bytes, which puts 16 neighbouring rows
// on distinct banks.  Wide heads use one place for both, one after the other.
template <int NB>
struct Stage {
  static constexpr bool SHARED = NB > 5;
  static constexpr int ROW = 16 * (NB | 1);
  static constexpr int ONE = STEP * ROW + STEP * NB * 2;  // rows, then scales [block][64]
  static constexpr int BYTES = SHARED ? ONE : 2 * ONE;
};
// A wave's part of LDS takes its steps, then its sums for the merge: 16 rows
// of D floats, four apart more so that the rows of a lane group lie on
// distinct banks.
template <int NB>
constexpr int region_bytes() {
  constexpr int m = 16 * (32 * NB + 4) * 4;
  return Stage<NB>::BYTES > m ? Stage<NB>::BYTES : m;
}

template <int NB, int WAVES>
__global__ __launch_bounds__(64 * WAVES, NB <= 2 ? 4 : 2) void attn_split_kernel(AttnArgs a) {
  constexpr int D = 32 * NB;
  constexpr int DT = D / 16;  // 16-value tiles of O^T
  // 16-key groups are whole numbers of 16-byte pieces to a load of the wave:
  // which group a load belongs to is then the same for all lanes
  constexpr bool WHOLE = NB % 4 == 0;
  // K scales of a lane: one where its quarter row lies inside a block, one per
  // block where it covers whole ones, else one per dword
  constexpr int KS = NB == 1 || NB == 2 || NB == 4 ? 1 : NB == 8 ? 2 : NB;
  constexpr int REGION = region_bytes<NB>();
  __shared__ __attribute__((aligned(16))) uint8_t lds[WAVES * REGION];
  __shared__ float merge_m[WAVES][16], merge_l[WAVES][16];
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x, wg = blockIdx.y + gridDim.y * blockIdx.z;

  // the workgroup's part of all steps, or (few_wgs = 0) all of tile wg
  int s = wg, sub = 0;
  Share share;
  if (a.few_wgs == 0) {
    if (a.one_tile ? s >= a.n_seqs : !find_tile(a, wg, 16, 0, a.few_rows, s, sub)) return;
  } else if (!find_share<16>(a, wg, a.few_wgs, WAVES, 0, a.few_rows, s, sub, share)) {
    return;
  }

  for (;; ++sub) {
    const Seq sq = load_seq(a, s);
    const int rows = sq.n * a.group;
    if (sub * 16 >= rows || rows > a.few_rows) {  // (a request with one tile may have none, or more)
      if (a.few_wgs == 0 || ++s >= a.n_seqs) return;
      sub = -1;
      continue;
    }
    const int r0 = sub * 16, r1 = r0 + 15 < rows ? r0 + 15 : rows - 1;
    const Keys keys = key_range(a, sq, r0, r1);
    const int steps = keys.end > keys.lo ? (keys.end - keys.lo + STEP - 1) / STEP : 0;
    int st0 = 0, st1 = steps, pieces = 1, first = 0;
    if (a.few_wgs > 0) {
      if (share.x >= share.x1) return;
      if (!take_steps<16>(share, steps, st0, st1, first, pieces)) continue;
    }
    {
      const int row = r0 + col;
      const bool live = row < rows;
      const int qt = token_of(a, row), tok = sq.row0 + qt, head = h * a.group + row - qt * a.group;
      // positions of this lane's row, of the tile's first and last
      const int p = live ? sq.len - sq.n + qt : -1;
      const int p0 = sq.len - sq.n + token_of(a, r0), p1 = sq.len - sq.n + token_of(a, r1);
      if (a.where && st0 == 0 && threadIdx.x < 16 && live) {
        int32_t* w = a.where + 2 * ((int64_t)tok * a.hq + head);
        w[0] = pieces > 1 ? -pieces : 0;
        w[1] = first * 16 + col;
      }

      uint8_t* kcodes = lds + wave * REGION;
      uint8_t* vcodes = kcodes + (Stage<NB>::SHARED ? 0 : Stage<NB>::ONE);
      uint16_t* kscales = (uint16_t*)(kcodes + STEP * Stage<NB>::ROW);
      uint16_t* vscales = (uint16_t*)(vcodes + STEP * Stage<NB>::ROW);
      const ConstInts pages = (ConstInts)(a.table + (int64_t)s * a.width);

      // registers of a step in flight
      struct {
        u32x4 kw[NB], vw[NB];
        uint32_t ks[(NB + 1) / 2], vs[(NB + 1) / 2], ok;
      } f;
      const auto page_ids = [&](int st, int (&ids)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = keys.lo + st * STEP + 16 * i;
          // (below 64 keys a page a step's groups may lie in different ones)
          ids[i] = st < st1 && k < keys.end && (i == 0 || a.page_shift < 6) ? pages[k >> a.page_shift] : -1;
        }
      };
      // codes in 16-byte pieces, lanes on consecutive ones; scales a lane to a key
      const auto load_rows = [&](const uint8_t* cache, const Groups& gr, u32x4 (&w)[NB], uint32_t (&sc)[(NB + 1) / 2]) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int piece = i * 64 + lane, key = piece / NB, b = piece % NB;
          const int64_t at = WHOLE ? gr.codes[4 * i / NB] : pick4(gr.codes, key >> 4);
          // (read once: nontemporal, 8 to 13% faster on caches larger than the last-level cache)
          w[i] = __builtin_nontemporal_load((const u32x4*)(cache + at + (uint32_t)((key & 15) * (D / 2) + 16 * b)));
        }
        const uint8_t* sp = cache + pick4(gr.scales, g) + (uint32_t)(col * (D / 16));
        if constexpr (NB % 2 == 0) {
          load_dwords<NB / 2>(sp, sc);
        } else {
#pragma unroll
          for (int b = 0; b < NB; b += 2) sc[b / 2] = ld_u16(sp + 2 * b) | (b + 1 < NB ? ld_u16(sp + 2 * b + 2) << 16 : 0u);
        }
      };
      // K: row of key k at k, scales [block][key % 16][key / 16], a lane's four
      // tiles side by side
      const auto stage_k = [&]() {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int piece = i * 64 + lane;
          *(u32x4*)(kcodes + (piece / NB) * Stage<NB>::ROW + 16 * (piece % NB)) = f.kw[i];
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) kscales[b * 64 + col * 4 + g] = (uint16_t)(f.ks[b / 2] >> (16 * (b & 1)));
      };
      // V: row of key 16 i + 4 c + j at 16 c + 4 i + j, so that lane group c's
      // keys lie together; scales in the order of the operands
      const auto stage_v = [&](int base, uint32_t ok) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int piece = i * 64 + lane, key = piece / NB, b = piece % NB;
          const int lr = ((key >> 2) & 3) * 16 + (key >> 4) * 4 + (key & 3);
          *(u32x4*)(vcodes + lr * Stage<NB>::ROW + 16 * b) = f.vw[i];
        }
        // bytes behind the last key are anything, NaN included: their values enter as 0 * code
        const bool good = ((ok >> g) & 1u) && base + lane < keys.end;
        const int pos = ((lane >> 2) & 3) * 16 + (g >> 1) * 8 + (lane & 3) * 2 + (g & 1);
#pragma unroll
        for (int b = 0; b < NB; ++b) vscales[b * 64 + pos] = (uint16_t)((good ? f.vs[b / 2] : 0u) >> (16 * (b & 1)));
      };

      int ids[4], ids_next[4];
      page_ids(st0 + wave, ids);
      page_ids(st0 + wave + WAVES, ids_next);
      u32x4 q_raw[NB];
      load_query<NB, 8 * NB, 8>(a, tok, head, live, g, q_raw);
      {
        const Groups gr = groups_of<D>(a, ids, keys.lo + (st0 + wave) * STEP, keys.end, h);
        if (st0 + wave < st1) {
          load_rows(a.kc, gr, f.kw, f.ks);
          load_rows(a.vc, gr, f.vw, f.vs);
        }
        f.ok = gr.ok;
      }
      half8_t q[NB];
      float factor;
      query_operands<NB>(a, q_raw, q, factor);

      float4_t o[DT];
#pragma unroll
      for (int t = 0; t < DT; ++t) o[t] = float4_t{0, 0, 0, 0};
      float4_t l4 = {0, 0, 0, 0};
      float m = NEG_INF, limit = NEG_INF, bias = 0.f;

      for (int st = st0 + wave; st < st1; st += WAVES) {
        const int base = keys.lo + st * STEP, after = st + WAVES;
        const uint32_t ok = f.ok;
        // into LDS; the registers take the next step at once (two steps ahead
        // were slower: 82 us against 73 for 64 requests of up to 8192 keys)
        stage_k();
        if constexpr (!Stage<NB>::SHARED) stage_v(base, ok);
        const Groups gr = groups_of<D>(a, ids_next, keys.lo + after * STEP, keys.end, h);
        f.ok = gr.ok;
        if (after < st1) {
          load_rows(a.kc, gr, f.kw, f.ks);
          if constexpr (!Stage<NB>::SHARED) load_rows(a.vc, gr, f.vw, f.vs);
        }
        page_ids(after + WAVES, ids_next);
        // S^T; dword j of quarter g lies in block (g NB + j) / 4
        float4_t sc[4];
        {
          uint32_t sc4[KS][2];
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            const int b = KS == NB ? (g * NB + j) >> 2 : KS == 2 ? 2 * g + j : (g * NB) >> 2;
            const u32x2 v = *(const u32x2*)(kscales + b * 64 + col * 4);
            sc4[j][0] = v.x; sc4[j][1] = v.y;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[NB];
            load_dwords<NB>(kcodes + (16 * i + col) * Stage<NB>::ROW + g * (D / 8), w);
            sc[i] = float4_t{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              const half2_t pair = as_h2(sc4[KS == NB ? j : KS == 2 ? j / 4 : 0][i >> 1]);
              const half_t v = i & 1 ? pair.y : pair.x;
              const half2_t kv = half2_t{v, v};
              const H2x4 u = unpack8(w[j]);
              sc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                  operand(u.v[0] * kv, u.v[1] * kv, u.v[2] * kv, u.v[3] * kv), q[j], sc[i], 0, 0, 0);
            }
          }
        }
        if constexpr (Stage<NB>::SHARED) {
          stage_v(base, ok);
          if (after < st1) load_rows(a.vc, gr, f.vw, f.vs);
        }
        if (base + STEP - 1 > p0 || (a.window > 0 && base <= p1 - a.window) || ok != 15u) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int k = base + 16 * i + 4 * g + j;
              const bool see = ((ok >> i) & 1u) && k <= p && (a.window <= 0 || k > p - a.window);
              sc[i][j] = see ? sc[i][j] : NEG_INF;
            }
        }
        // running maximum; the sums move to a new one only when it is well above the old
        float mx = sc[0][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[i >> 2][i & 3]);
        mx = groups_max(mx);
        if (__any(!(mx <= limit))) {
          const float corr = move_maximum(mx, factor, sc, m, limit, bias);
          l4 *= corr;
#pragma unroll
          for (int t = 0; t < DT; ++t) o[t] *= corr;
        }
        // P^T operands: places (2 s, 2 s + 1) hold keys s of groups 2 m and 2 m + 1
        half8_t pt[2];
#pragma unroll
        for (int mm = 0; mm < 2; ++mm)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            pt[mm][2 * j] = (half_t)__builtin_amdgcn_exp2f(fmaf(sc[2 * mm][j], factor, bias));
            pt[mm][2 * j + 1] = (half_t)__builtin_amdgcn_exp2f(fmaf(sc[2 * mm + 1][j], factor, bias));
          }
        // sums of the (rounded) probabilities: one more row tile of V^T, all ones
        const half_t one = (half_t)1.f;
        const half8_t ones = half8_t{one, one, one, one, one, one, one, one};
        l4 = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pt[0], l4, 0, 0, 0);
        l4 = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pt[1], l4, 0, 0, 0);
        // O^T += V^T P^T
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const u32x4 s0 = *(const u32x4*)(vscales + b * 64 + g * 16), s1 = *(const u32x4*)(vscales + b * 64 + g * 16 + 8);
          const uint32_t vsc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            typedef int v2i __attribute__((ext_vector_type(2)));
            typedef v2i __attribute__((address_space(3))) lds_v2i;
            const v2i w = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                (lds_v2i*)(vcodes + (g * 16 + col) * Stage<NB>::ROW + 16 * b + 8 * t));
#pragma unroll
            for (int mm = 0; mm < 2; ++mm) {
              const H2x4 u = unpack8((uint32_t)w[mm]);
              o[2 * b + t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                  operand(u.v[0] * as_h2(vsc[4 * mm]), u.v[1] * as_h2(vsc[4 * mm + 1]),
                          u.v[2] * as_h2(vsc[4 * mm + 2]), u.v[3] * as_h2(vsc[4 * mm + 3])),
                  pt[mm], o[2 * b + t], 0, 0, 0);
            }
          }
        }
      }

      // merge: every wave's sums into its part of LDS, then each thread joins
      // the four of its values
      // (indices from an opaque copy: nothing of this is computed ahead of the
      // steps, where it would push their registers to memory)
      int tid = threadIdx.x;
      asm volatile("" : "+v"(tid));
      const int mcol = tid & 15, mg = (tid & 63) >> 4;
      float* mine = (float*)(lds + wave * REGION);
#pragma unroll
      for (int t = 0; t < DT; ++t) *(float4_t*)(mine + mcol * (D + 4) + 16 * t + 4 * mg) = o[t];
      if (mg == 0) {
        merge_m[wave][mcol] = sums_at(m, factor);
        merge_l[wave][mcol] = l4[0];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < (16 * D / 4 + 64 * WAVES - 1) / (64 * WAVES); ++k) {
        const int i = k * 64 * WAVES + tid, r = i / (D / 4), c = i % (D / 4) * 4;
        if (r >= 16 || r0 + r >= rows) break;
        float mx = merge_m[0][r];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) mx = fmaxf(mx, merge_m[w][r]);
        const float ref = mx == NEG_INF ? 0.f : mx;
        float l = 0.f;
        float4_t v = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
          const float f = __builtin_amdgcn_exp2f(merge_m[w][r] - ref);
          l += f * merge_l[w][r];
          v += f * *(const float4_t*)((const float*)(lds + w * REGION) + r * (D + 4) + c);
        }
        if (pieces == 1) {
          const int t = token_of(a, r0 + r);
          const int64_t orow = (int64_t)(sq.row0 + t) * a.hq + h * a.group + r0 + r - t * a.group;
          store4(a.out, a.out_type, orow * D + c, v * (l == 0.f ? 0.f : 1.f / l));  // no key seen: zeros
        } else {
          const int64_t pr = (((int64_t)wg * a.hkv + h) * 2 + (st0 == 0 ? 1 : 0)) * 16 + r;
          store4<0>(a.few, pr * D + c, v);
          if (c == 0) {
            float* ml = a.few + (int64_t)a.few_wgs * a.hkv * 32 * D + 2 * pr;
            ml[0] = mx;
            ml[1] = l;
          }
        }
      }
      __syncthreads();  // the next tile reuses the LDS
    }
    if (a.few_wgs == 0 && !a.one_tile) return;
  }
}

// Joins the sums of rows whose keys several workgroups shared: d / 4 threads
// to a piece; a workgroup takes one row with as many of its pieces side by
// side as fit (SIDE: few rows, many pieces), or as many rows as fit.
template <bool SIDE>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  __shared__ float4_t part[SIDE ? 256 : 1];
  const int64_t n_rows = (int64_t)a.tokens * a.hq;
  const int per = a.d / 4, fit = 256 / per, k = threadIdx.x / per, c = (threadIdx.x % per) * 4;
  const int64_t row = SIDE ? blockIdx.x : (int64_t)blockIdx.x * fit + k;
  if (!SIDE && (k >= fit || row >= n_rows)) return;
  const int tok = (int)(row / a.hq), h = token_of(a, (int)(row - (int64_t)tok * a.hq));  // (a head's kv head likewise)
  const int b = ((ConstInts)a.cu)[0], e = ((ConstInts)a.cu)[a.n_seqs];
  if (tok < b || tok >= e) return;  // no request's row: nothing was written for it
  int n = a.where[2 * row];
  if (n == 0) return;  // written by the workgroup itself
  // shared by n workgroups, the first of them and the row of its tile in `at`
  const bool few = n < 0;
  n = few ? -n : n;
  const int at = a.where[2 * row + 1], shift = few ? 4 : a.many_shift, wgs = few ? a.few_wgs : a.many_wgs;
  // (bounds for offsets that are not a batch's: rows no request owns hold anything)
  if (at < 0 || (at >> shift) >= wgs || n > wgs - (at >> shift)) return;
  const float* sums = few ? a.few : a.many;
  const float* ml = sums + (((int64_t)wgs * a.hkv * 2) << shift) * a.d;
  const auto piece = [&](int i) -> int64_t {
    return (((((int64_t)(at >> shift) + i) * a.hkv + h) * 2 + (i == 0 ? 1 : 0)) << shift) + (at & ((1 << shift) - 1));
  };
  float m = NEG_INF, l = 0.f;
  float4_t o = {0, 0, 0, 0};
  if constexpr (SIDE) {
    // every wave finds the maximum and the sum for itself, 64 pieces at a time
    const int lane = threadIdx.x & 63;
    for (int i = lane; i < n; i += 64) m = fmaxf(m, ml[2 * piece(i)]);
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor(m, x, 64));
    const float ref = m == NEG_INF ? 0.f : m;
    for (int i = lane; i < n; i += 64) l += __builtin_amdgcn_exp2f(ml[2 * piece(i)] - ref) * ml[2 * piece(i) + 1];
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) l += __shfl_xor(l, x, 64);
    if (k < fit) {
#pragma unroll 4
      for (int i = k; i < n; i += fit) {
        const int64_t r = piece(i);
        o += __builtin_amdgcn_exp2f(ml[2 * r] - ref) * *(const float4_t*)(sums + r * a.d + c);
      }
    }
  } else {
    for (int i = 0; i < n; ++i) m = fmaxf(m, ml[2 * piece(i)]);
    const float ref = m == NEG_INF ? 0.f : m;
    for (int i = 0; i < n; ++i) {
      const int64_t r = piece(i);
      const float w = __builtin_amdgcn_exp2f(ml[2 * r] - ref);
      l += w * ml[2 * r + 1];
      o += w * *(const float4_t*)(sums + r * a.d + c);
    }
  }
  if constexpr (SIDE) {
    part[threadIdx.x] = o;
    __syncthreads();
    if (k > 0) return;
    for (int i = 1; i < fit && i < n; ++i) o += part[i * per + threadIdx.x];
  }
  store4(a.out, a.out_type, row * a.d + c, o * (l == 0.f ? 0.f : 1.f / l));
}

}  // namespace

// rows of a request up to which its own 16-row tiles beat a share of a prompt
// tile, when a batch holds both
constexpr int FEW_ROWS = 32;

AttnPlan attn_plan(int64_t tokens, int64_t n_seqs, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t max_new,
                   int64_t max_kv, int64_t window) {
  AttnPlan p;
  // keys that a request's rows see; a narrower bound never asks for more workspace
  if (window > 0 && window + max_new < max_kv) max_kv = window + max_new;
  const int64_t group = q_heads / kv_heads, most = (max_new < tokens ? max_new : tokens) * group;
  p.one_tile = most <= 16;
  const int64_t all = tokens * group;
  // Which kernels run.  Few rows a request, or short requests whose 16-row
  // tiles have CUs to themselves (100 tokens, 8 kv heads: 10 us against 15):
  // 16-row tiles.  One request of many rows: prompt tiles.  Else each request
  // goes where its rows fit.
  const bool brief = max_kv <= 512 && (all / 16 + n_seqs) * kv_heads <= 512;
  p.few_rows = most <= 64 || brief ? 0x7FFFFFFF : n_seqs == 1 ? 0 : FEW_ROWS;
  p.few_tiles = p.one_tile ? n_seqs : p.few_rows == 0 ? 0 : all / 16 + n_seqs;
  if (p.few_rows == FEW_ROWS && p.few_tiles > n_seqs * (FEW_ROWS / 16)) p.few_tiles = n_seqs * (FEW_ROWS / 16);
  const int tile = attn_prompt_rows(d);
  p.many_tiles = p.few_rows == 0x7FFFFFFF ? 0 : all / tile + n_seqs;
  // 16-row tiles: one workgroup to each where none has much work, or where
  // they are so many that even unequal ones fill the GPU; else as many
  // workgroups as run at once (two on each of 256 CUs, four with narrow heads),
  // each with the same number of steps
  const int64_t at_once = d <= 64 ? 1024 : 512;
  p.few_wgs = 0;
  if (p.few_tiles > 0 && max_kv > 1024 && n_seqs <= 1024 && p.few_tiles * kv_heads < 8 * at_once)
    p.few_wgs = (int)((at_once + kv_heads - 1) / kv_heads);
  // eight waves to a workgroup where each has a CU or so to itself
  p.more_waves = p.few_wgs == 0 && p.few_tiles * kv_heads <= 512 && max_kv > STEP * WAVES;
  // Prompt tiles: one workgroup to a CU, 2 us a step.  A workgroup to a tile, a
  // request's longest first, needs no sums joined; even shares leave no CU
  // idle, at some 25 us, or 50 where each has several tiles.  What they save,
  // in steps, with `full` steps in the longest tile and `fresh` fewer in the
  // shortest: all CUs' work but the tiles', where the tiles are fewer; else the last
  // round of equal tiles, and more where requests are unequal.  (1024 tokens
  // after 16000, 8 kv heads: 336 us against 536; 128 after 4000 47 against
  // 136; but prompts of 1024 and 4096 tokens 53 and 238 against 46 and 193.)
  // It grows with max_kv, so that the workspace does.
  p.many_wgs = 0;
  if (p.many_tiles > 0 && kv_heads <= 64) {
    const int64_t wgs = 256 / kv_heads * kv_heads, all_tiles = p.many_tiles * kv_heads;
    const int64_t seen = window + tile / group + 1;  // keys of a tile's rows under a window
    const double full = (double)(((window > 0 && seen < max_kv ? seen : max_kv) + STEP - 1) / STEP);
    const double news = (double)(max_new < tokens ? max_new : tokens) / STEP, fresh = news < full ? news : full;
    const double each = (double)all_tiles / wgs, rounds = (double)((all_tiles + wgs - 1) / wgs);
    const double saved = each < 1 ? full - each * (full - fresh / 2)
                                  : (rounds - each) * (full - fresh) + (n_seqs > 1 ? 0.3 * full : 0.);
    if (saved > (each < 1 ? 12 : 24)) p.many_wgs = (int)(256 / kv_heads);
  }
  const int64_t many = (int64_t)p.many_wgs * kv_heads * 2 * tile, few = (int64_t)p.few_wgs * kv_heads * 32;
  p.few_at = many * (d + 2) * 4;
  p.where_at = p.few_at + few * (d + 2) * 4;
  p.bytes = many + few > 0 ? p.where_at + tokens * q_heads * 8 : 0;
  return p;
}

hipError_t launch_kv_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.many_tiles > 0) {
    e = launch_attn_prompt(a, p, s);
    if (e != hipSuccess) return e;
  }
  if (p.few_tiles > 0) {
    const int64_t n = a.few_wgs > 0 ? a.few_wgs : p.few_tiles, gy = n < 32768 ? n : 32768;
    const dim3 grid((unsigned)a.hkv, (unsigned)gy, (unsigned)((n + gy - 1) / gy));
    const auto go = [&](auto four, auto eight) {
      if (p.more_waves) hipLaunchKernelGGL(eight, grid, dim3(64 * MORE_WAVES), 0, s, a);
      else hipLaunchKernelGGL(four, grid, dim3(64 * WAVES), 0, s, a);
    };
    switch (a.d / 32) {
      case 1: go(attn_split_kernel<1, WAVES>, attn_split_kernel<1, MORE_WAVES>); break;
      case 2: go(attn_split_kernel<2, WAVES>, attn_split_kernel<2, MORE_WAVES>); break;
      case 3: go(attn_split_kernel<3, WAVES>, attn_split_kernel<3, MORE_WAVES>); break;
      case 4: go(attn_split_kernel<4, WAVES>, attn_split_kernel<4, MORE_WAVES>); break;
      case 5: go(attn_split_kernel<5, WAVES>, attn_split_kernel<5, MORE_WAVES>); break;
      case 6: go(attn_split_kernel<6, WAVES>, attn_split_kernel<6, MORE_WAVES>); break;
      case 7: go(attn_split_kernel<7, WAVES>, attn_split_kernel<7, MORE_WAVES>); break;
      default: go(attn_split_kernel<8, WAVES>, attn_split_kernel<8, MORE_WAVES>); break;
    }
    e = hipGetLastError();
  }
  if (e != hipSuccess || p.bytes == 0) return e;
  const int64_t n_rows = (int64_t)a.tokens * a.hq, fit = 256 / (a.d / 4);
  // (2048 rows of one or two pieces: 7.6 us side by side, 4.7 us packed; 128 rows of 24: packed 22 us)
  if (n_rows <= 1024) hipLaunchKernelGGL(attn_join_kernel<true>, dim3((unsigned)n_rows), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(attn_join_kernel<false>, dim3((unsigned)((n_rows + fit - 1) / fit)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace kq
