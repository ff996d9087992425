// kq_kv_attention: attention over key/value rows held in 4 bits.
//
//   out = sum_j softmax_j(scale q . k_j) v_j,   k_j, v_j = D (c - 8)
//
// One pass over the keys with a running maximum and sum.  A workgroup takes
// one 16-row tile of a (request, kv head); its four waves take 64-key steps in
// turn, each with sums of its own, merged through LDS at the end.  Both
// products run on v_mfma_f32_16x16x32_f16, transposed so that nothing moves
// between lanes in between:
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
#include "kq_kv_attn.h"

namespace kq {
namespace {

constexpr int WAVES = 4;
constexpr int STEP = 64;  // keys of one step

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
// LDS to hand one wave's sums to another: O^T [d][16], then maximum and sum
template <int NB>
constexpr int merge_bytes() { return 16 * 32 * NB * 4 + 2 * 16 * 4; }
template <int NB>
constexpr int lds_bytes() {
  constexpr int s = WAVES * Stage<NB>::BYTES, m = 2 * merge_bytes<NB>();
  return s > m ? s : m;
}

template <int NB>
__global__ __launch_bounds__(64 * WAVES, NB <= 4 ? 3 : 2) void attn_split_kernel(AttnArgs a) {
  constexpr int D = 32 * NB;
  constexpr int DT = D / 16;  // 16-value tiles of O^T
  // 16-key groups are whole numbers of 16-byte pieces to a load of the wave:
  // which group a load belongs to is then the same for all lanes
  constexpr bool WHOLE = NB % 4 == 0;
  // K scales of a lane: one where its quarter row lies inside a block, one per
  // block where it covers whole ones, else one per dword
  constexpr int KS = NB == 1 || NB == 2 || NB == 4 ? 1 : NB == 8 ? 2 : NB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[lds_bytes<NB>()];
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x % a.hkv, tile = blockIdx.x / a.hkv, split = blockIdx.y;

  int s = tile, sub = 0;
  if (!a.one_tile) {
    if (!find_tile(a, tile, 16, 0, a.few_rows, s, sub)) return;
  }
  const Seq sq = load_seq(a, s);
  const int rows = sq.n * a.group;
  // with one tile to a request, a request that has more walks its own
  for (; sub * 16 < rows; ++sub) {
    const int r0 = sub * 16, r1 = r0 + 15 < rows ? r0 + 15 : rows - 1;
    const Keys keys = key_range(a, sq, r0, r1);
    const int n_split = split_count(a, keys);
    const int row = r0 + col;
    const bool live = row < rows;
    const int tok = sq.row0 + row / a.group, head = h * a.group + row % a.group;
    const int64_t orow = (int64_t)tok * a.hq + head;
    // positions of this lane's row, of the tile's first and last
    const int p = live ? sq.len - sq.n + row / a.group : -1;
    const int p0 = sq.len - sq.n + r0 / a.group, p1 = sq.len - sq.n + r1 / a.group;

    int32_t* counts = (int32_t*)(a.part + part_rows(a.tokens, a.hq, a.splits) * (D + 2));
    if (a.splits > 1 && split == 0 && threadIdx.x < 16 && live) counts[orow] = n_split > 1 ? n_split : 0;
    if (n_split == 0 && split == 0) {
      for (int t = wave; t < DT; t += WAVES)
        if (live) store4(a.out, a.out_type, orow * D + 16 * t + 4 * g, float4_t{0, 0, 0, 0});
    }
    if (split < n_split) {
      const int steps = (keys.end - keys.lo + STEP - 1) / STEP;
      const int st0 = (int)((int64_t)steps * split / n_split), st1 = (int)((int64_t)steps * (split + 1) / n_split);

      uint8_t* kcodes = lds + wave * Stage<NB>::BYTES;
      uint8_t* vcodes = kcodes + (Stage<NB>::SHARED ? 0 : Stage<NB>::ONE);
      uint16_t* kscales = (uint16_t*)(kcodes + STEP * Stage<NB>::ROW);
      uint16_t* vscales = (uint16_t*)(vcodes + STEP * Stage<NB>::ROW);
      // read only here, so scalar loads may fetch it
      const auto* pages = (const __attribute__((address_space(4))) int32_t*)(a.table + (int64_t)s * a.width);

      // registers of the step in flight
      u32x4 kw[NB], vw[NB];
      uint32_t ks[(NB + 1) / 2], vs[(NB + 1) / 2];
      const auto page_ids = [&](int st, int (&ids)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = keys.lo + st * STEP + 16 * i;
          ids[i] = st < st1 && k < keys.end ? pages[k >> a.page_shift] : -1;
        }
      };
      // codes in 16-byte pieces, lanes on consecutive ones; scales a lane to a key
      const auto load_rows = [&](const uint8_t* cache, const Groups& gr, u32x4 (&w)[NB], uint32_t (&sc)[(NB + 1) / 2]) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int piece = i * 64 + lane, key = piece / NB, b = piece % NB;
          const int64_t at = WHOLE ? gr.codes[4 * i / NB] : pick4(gr.codes, key >> 4);
          w[i] = ld_16B(cache + at + (uint32_t)((key & 15) * (D / 2) + 16 * b));
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
          *(u32x4*)(kcodes + (piece / NB) * Stage<NB>::ROW + 16 * (piece % NB)) = kw[i];
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) kscales[b * 64 + col * 4 + g] = (uint16_t)(ks[b / 2] >> (16 * (b & 1)));
      };
      // V: row of key 16 i + 4 c + j at 16 c + 4 i + j, so that lane group c's
      // keys lie together; scales in the order of the operands
      const auto stage_v = [&](int base, uint32_t ok) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int piece = i * 64 + lane, key = piece / NB, b = piece % NB;
          const int lr = ((key >> 2) & 3) * 16 + (key >> 4) * 4 + (key & 3);
          *(u32x4*)(vcodes + lr * Stage<NB>::ROW + 16 * b) = vw[i];
        }
        // bytes behind the last key are anything, NaN included: their values enter as 0 * code
        const bool good = ((ok >> g) & 1u) && base + lane < keys.end;
        const int pos = ((lane >> 2) & 3) * 16 + (g >> 1) * 8 + (lane & 3) * 2 + (g & 1);
#pragma unroll
        for (int b = 0; b < NB; ++b) vscales[b * 64 + pos] = (uint16_t)((good ? vs[b / 2] : 0u) >> (16 * (b & 1)));
      };

      int ids[4], ids_next[4];
      page_ids(st0 + wave, ids);
      page_ids(st0 + wave + WAVES, ids_next);
      half8_t q[NB];
      float factor;
      load_query<NB, 8 * NB, 8>(a, (const uint16_t*)a.q + (int64_t)tok * a.q_stride + (int64_t)head * D, live, g, q, factor);
      // probabilities may reach 2^8 before the sums are brought to a new maximum
      const float slack = 8.f / factor;

      float4_t o[DT];
#pragma unroll
      for (int t = 0; t < DT; ++t) o[t] = float4_t{0, 0, 0, 0};
      float4_t l4 = {0, 0, 0, 0};
      float m = NEG_INF;

      Groups gr = groups_of<D>(a, ids, keys.lo + (st0 + wave) * STEP, keys.end, h);
      if (st0 + wave < st1) {
        load_rows(a.kc, gr, kw, ks);
        load_rows(a.vc, gr, vw, vs);
      }
      for (int st = st0 + wave; st < st1; st += WAVES) {
        const int base = keys.lo + st * STEP;
        const uint32_t ok = gr.ok;
        const bool more = st + WAVES < st1;
        // into LDS; the registers take the next step at once
        stage_k();
        if constexpr (!Stage<NB>::SHARED) stage_v(base, ok);
        gr = groups_of<D>(a, ids_next, base + WAVES * STEP, keys.end, h);
        if (more) {
          load_rows(a.kc, gr, kw, ks);
          if constexpr (!Stage<NB>::SHARED) load_rows(a.vc, gr, vw, vs);
        }
        page_ids(st + 2 * WAVES, ids_next);
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
          if (more) load_rows(a.vc, gr, vw, vs);
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
        if (__any(!(mx <= m + slack))) {
          mx = fmaxf(mx, m);
          const float corr = mx == NEG_INF ? 1.f : __builtin_amdgcn_exp2f((m - mx) * factor);
          m = mx;
          l4 *= corr;
#pragma unroll
          for (int t = 0; t < DT; ++t) o[t] *= corr;
        }
        const float bias = m == NEG_INF ? 0.f : -m * factor;
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
      float l = l4[0];

      // merge: waves 2, 3 into 0, 1, then 1 into 0
#pragma unroll
      for (int half = WAVES / 2; half > 0; half >>= 1) {
        __syncthreads();
        float* buf = (float*)(lds + (wave & (half - 1)) * merge_bytes<NB>());
        if (wave >= half && wave < 2 * half) {
#pragma unroll
          for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) buf[(16 * t + 4 * g + j) * 16 + col] = o[t][j];
          if (g == 0) { buf[D * 16 + col] = m; buf[D * 16 + 16 + col] = l; }
        }
        __syncthreads();
        if (wave < half) {
          const float m2 = buf[D * 16 + col], l2 = buf[D * 16 + 16 + col];
          const float mx = fmaxf(m, m2), ref = mx == NEG_INF ? 0.f : mx;
          const float c1 = __builtin_amdgcn_exp2f((m - ref) * factor), c2 = __builtin_amdgcn_exp2f((m2 - ref) * factor);
          m = mx;
          l = l * c1 + l2 * c2;
#pragma unroll
          for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[t][j] = o[t][j] * c1 + buf[(16 * t + 4 * g + j) * 16 + col] * c2;
        }
      }
      if (wave == 0 && live) {
        if (n_split == 1) {
          const float inv = l == 0.f ? 0.f : 1.f / l;  // no key seen: zeros
#pragma unroll
          for (int t = 0; t < DT; ++t) store4(a.out, a.out_type, orow * D + 16 * t + 4 * g, o[t] * inv);
        } else {
          const int64_t pr = (int64_t)split * a.tokens * a.hq + orow;
#pragma unroll
          for (int t = 0; t < DT; ++t) store4<0>(a.part, pr * D + 16 * t + 4 * g, o[t]);
          if (g == 0) {
            float* ml = a.part + part_rows(a.tokens, a.hq, a.splits) * D + 2 * pr;
            ml[0] = m == NEG_INF ? NEG_INF : m * factor;  // in powers of two, for the merge
            ml[1] = l;
          }
        }
      }
      __syncthreads();  // the next tile reuses the LDS
    }
    if (!a.one_tile) break;
  }
}

// Joins the partial sums of split rows: a thread per 4 values of a row.
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  const int per = a.d / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / per;
  const int c = (int)(i - row * per) * 4;
  const int64_t n_rows = (int64_t)a.tokens * a.hq;
  if (row >= n_rows) return;
  int b = a.cu[0], e = a.cu[a.n_seqs];
  b = b < 0 ? 0 : b;
  const int tok = (int)(row / a.hq);
  if (tok < b || tok >= e) return;  // no request's row: its count was not written
  const int64_t pr = part_rows(a.tokens, a.hq, a.splits);
  const int32_t* counts = (const int32_t*)(a.part + pr * (a.d + 2));
  int n = counts[row];
  n = n > a.splits ? a.splits : n;
  if (n <= 1) return;  // written by the workgroup itself
  const float* ml = a.part + pr * a.d;
  float m = NEG_INF;
  for (int s = 0; s < n; ++s) m = fmaxf(m, ml[2 * (s * n_rows + row)]);
  const float ref = m == NEG_INF ? 0.f : m;
  float4_t o = {0, 0, 0, 0};
  float l = 0.f;
  for (int s = 0; s < n; ++s) {
    const int64_t r = s * n_rows + row;
    const float w = __builtin_amdgcn_exp2f(ml[2 * r] - ref);
    l += w * ml[2 * r + 1];
    o += w * *(const float4_t*)(a.part + r * a.d + c);
  }
  store4(a.out, a.out_type, row * a.d + c, o * (l == 0.f ? 0.f : 1.f / l));
}

}  // namespace

// rows of a request up to which its own 16-row tiles beat a share of a prompt
// tile, when a batch holds both
constexpr int FEW_ROWS = 32;

AttnPlan attn_plan(int64_t tokens, int64_t n_seqs, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t max_new,
                   int64_t max_kv) {
  AttnPlan p;
  const int64_t group = q_heads / kv_heads, most = (max_new < tokens ? max_new : tokens) * group;
  p.one_tile = most <= 16;
  // Which kernels run.  Requests of few rows only: 16-row tiles.  One request
  // of many rows: prompt tiles.  Else each request goes where its rows fit.
  p.few_rows = most <= 64 ? 0x7FFFFFFF : n_seqs == 1 ? 0 : FEW_ROWS;
  const int64_t all = tokens * group;
  p.few_tiles = p.one_tile ? n_seqs : p.few_rows == 0 ? 0 : all / 16 + n_seqs;
  if (p.few_rows == FEW_ROWS && p.few_tiles > n_seqs * (FEW_ROWS / 16)) p.few_tiles = n_seqs * (FEW_ROWS / 16);
  const int tile = attn_prompt_rows(d);
  p.many_tiles = p.few_rows == 0x7FFFFFFF ? 0 : all / tile + n_seqs;
  int64_t chunk;
  if (p.many_tiles > 0) {
    // prompt tiles: one workgroup to a CU.  Split rows write and read float32
    // sums, which costs as much as some 500 keys, so only where tiles alone
    // leave a good part of the CUs idle, and 1024 keys at least
    const int64_t wgs = p.many_tiles * kv_heads, want = (256 + wgs - 1) / wgs;
    chunk = wgs >= 192 ? max_kv : (max_kv + want - 1) / want;
    chunk = chunk < 1024 ? 1024 : chunk;
  } else {
    // enough workgroups for three on each of 256 CUs, none with fewer than 256
    // keys; never more than 4096 keys to one, whose length differs from others'
    const int64_t wgs = p.few_tiles * kv_heads, want = (768 + wgs - 1) / wgs;
    chunk = (max_kv + want - 1) / want;
    chunk = chunk < 256 ? 256 : chunk > 4096 ? 4096 : chunk;
  }
  p.chunk = (int)((chunk + 63) / 64 * 64);
  p.splits = (int)((max_kv + p.chunk - 1) / p.chunk);
  p.splits = p.splits < 1 ? 1 : p.splits > 256 ? 256 : p.splits;
  p.bytes = p.splits > 1 ? part_rows(tokens, q_heads, p.splits) * (d + 2) * 4 + tokens * q_heads * 4 : 0;
  return p;
}

hipError_t launch_kv_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.many_tiles > 0) {
    e = launch_attn_prompt(a, p, s);
    if (e != hipSuccess) return e;
  }
  if (p.few_tiles > 0) {
    const dim3 grid((unsigned)(p.few_tiles * a.hkv), (unsigned)a.splits), block(64 * WAVES);
    const auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, block, 0, s, a); };
    switch (a.d / 32) {
      case 1: go(attn_split_kernel<1>); break;
      case 2: go(attn_split_kernel<2>); break;
      case 3: go(attn_split_kernel<3>); break;
      case 4: go(attn_split_kernel<4>); break;
      case 5: go(attn_split_kernel<5>); break;
      case 6: go(attn_split_kernel<6>); break;
      case 7: go(attn_split_kernel<7>); break;
      default: go(attn_split_kernel<8>); break;
    }
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t n = (int64_t)a.tokens * a.hq * (a.d / 4);
  hipLaunchKernelGGL(attn_join_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace kq
