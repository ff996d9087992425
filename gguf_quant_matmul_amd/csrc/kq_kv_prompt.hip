// kq_kv_attention for many rows that share keys (prompts): the same products
// as kq_kv_attn.hip, but a workgroup's eight waves share each 64-key step.  A
// wave takes C 16-row tiles of its own; the step's keys and values are
// unpacked to float16 once, by all waves together, into LDS in the order of
// the matrix operands, and every wave reads them from there.
//
// A step is K Q^T (matrix cores), the softmax (vector unit), V^T P^T (matrix
// cores) and the unpacking of a coming step (vector unit).  Two waves share a
// SIMD, and with one barrier a step at the same place they would want the
// same unit at the same time.  So the second four waves meet the barrier
// after their K Q^T instead of at the end of the step: in the round between
// two barriers they run softmax, V^T P^T and unpacking of one step, then
// K Q^T of the next, beside the first four's K Q^T, softmax, V^T P^T.  The
// round of step r unpacks step r + 1 (two places for keys, three for values,
// of which V(r - 1) and V(r) are being read) and fetches the one after.
//
// Measured: a prompt of 4096 tokens (8 kv heads, groups of 4, d = 128) 162 us
// among others, 850 TFLOP/s of its causal products (a large library product
// reaches 1190), 200 us by itself; 2048 tokens after 30000 1.04 ms, 1000
// TFLOP/s.  A step of a workgroup takes 2 us.  Bound by the vector units, busy
// 52% of the time with softmax and unpacking, and the matrix cores, busy 38%,
// which run beside each other only in part.
#include "kq_kv_attn.h"

namespace kq {
namespace {

constexpr int PW = 8;     // waves

template <int NB>
struct Prompt {
  static constexpr int C = NB <= 4 ? 2 : 1;             // 16-row tiles of a wave (its sums fill the registers)
  static constexpr int ROWS = PW * C * 16;              // rows of a workgroup
  static constexpr int UNITS = (2 * NB + PW - 1) / PW;  // unpacking units of a wave: 64 pieces of 32 values
  static constexpr int HALF = STEP * 32 * NB * 2;       // float16 keys (or values) of a step
  static constexpr int RAW = STEP * 16 + STEP * 2;      // one block's codes and scales, on the way to the transposing read
  // three places for values where 160 KB hold them; else two, and all waves
  // meet at the end of the step
  static constexpr bool OFFSET = 5 * HALF + NB * RAW <= 160 * 1024;
  static constexpr int VB = OFFSET ? 3 : 2;
  static constexpr int LDS = (2 + VB) * HALF + NB * RAW;
};

// SHARE: the workgroup takes an even share of all requests' steps, tile by
// tile, else one tile (without the loop over tiles its registers suffice).
template <int NB, bool SHARE>
__global__ __launch_bounds__(64 * PW, 2) void attn_prompt_kernel(AttnArgs a) {
  typedef Prompt<NB> T;
  constexpr int D = 32 * NB, DT = D / 16, C = T::C;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x % a.hkv, wg = blockIdx.x / a.hkv;

  int s = 0, sub = 0;
  Share share;
  if constexpr (SHARE) {
    if (!find_share<T::ROWS>(a, wg, a.many_wgs, 4, a.few_rows, 0x7FFFFFFF, s, sub, share)) return;
  } else {
    if (!find_tile(a, wg, T::ROWS, a.few_rows, 0x7FFFFFFF, s, sub)) return;
  }
  for (;; ++sub) {
    int lane = threadIdx.x & 63;
    // nothing made of it is kept from tile to tile (12 registers went to memory)
    if constexpr (SHARE) asm volatile("" : "+v"(lane));
    const int col = lane & 15, g = lane >> 4;
    const Seq sq = load_seq(a, s);
    const int rows = sq.n * a.group;
    if (sub * T::ROWS >= rows || rows <= a.few_rows) {
      if (!SHARE || ++s >= a.n_seqs) return;
      sub = -1;
      continue;
    }
    // (a workgroup to a tile: the tiles with the most keys first)
    const int tile = SHARE ? sub : (rows + T::ROWS - 1) / T::ROWS - 1 - sub;
    const int r0 = tile * T::ROWS, r1 = r0 + T::ROWS < rows ? r0 + T::ROWS - 1 : rows - 1;
    const Keys keys = key_range(a, sq, r0, r1);
    const int steps = keys.end > keys.lo ? (keys.end - keys.lo + STEP - 1) / STEP : 0;
    int st0 = 0, st1 = steps, pieces = 1, first = 0;
    if constexpr (SHARE) {
      if (share.x >= share.x1) return;
      if (!take_steps<T::ROWS>(share, steps, st0, st1, first, pieces)) continue;
    }

    // the wave's rows: positions of its first and last, none if w0 > w1
    const int w0 = r0 + wave * C * 16, w1 = w0 + C * 16 - 1 < rows ? w0 + C * 16 - 1 : rows - 1;
    const int p0 = sq.len - sq.n + token_of(a, w0), p1 = w0 <= w1 ? sq.len - sq.n + token_of(a, w1) : -1;
    int p[C];
    bool live[C];
    u32x4 q_raw[C][NB];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int row = w0 + 16 * c + col;
      live[c] = row < rows;
      const int qt = token_of(a, row), tok = sq.row0 + qt, head = h * a.group + row - qt * a.group;
      if (a.where && st0 == 0 && g == 0 && live[c]) {
        int32_t* w = a.where + 2 * ((int64_t)tok * a.hq + head);
        w[0] = pieces > 1 ? pieces : 0;
        w[1] = first * T::ROWS + row - r0;
      }
      p[c] = live[c] ? sq.len - sq.n + qt : -1;
      load_query<NB, 8, 32>(a, tok, head, live[c], g, q_raw[c]);
    }
    const int32_t* pages = a.table + (int64_t)s * a.width;

    // Unpacking is shared out in units: unit u < NB is 64 pieces (32 values) of
    // keys, lanes on consecutive pieces; unit NB + b block b of 64 value rows, a
    // lane to a row.  Everything is asked for a step or more before it is
    // needed: page ids, then codes and scales at the addresses they give, then
    // (values) the write to LDS that the transposing read wants.
    const int page_mask = (1 << a.page_shift) - 1;
    const uint64_t page_bytes = (uint64_t)a.hkv * (uint64_t)a.page_head_bytes;
    // the page id of key `lane` of a step (any id for keys behind the last)
    const auto page_id = [&](int st) {
      const int k = keys.lo + st * STEP + lane;
      return pages[(k < keys.end ? k : keys.end - 1) >> a.page_shift];
    };
    // ... -1 where there is no such key or no such page
    const auto checked = [&](int st, int id) {
      return keys.lo + st * STEP + lane < keys.end && (uint32_t)id < (uint32_t)a.pages ? id : -1;
    };
    // offsets of the codes and scales of a row in the cache; page 0 for id -1
    const auto row_at = [&](int key, int id, uint64_t& codes, uint64_t& scales) {
      const uint64_t at =
          (uint64_t)(uint32_t)(id < 0 ? 0 : id) * page_bytes + (uint64_t)h * (uint64_t)a.page_head_bytes;
      const uint32_t row = (uint32_t)(key & page_mask);
      codes = at + row * (uint32_t)(D / 2);
      scales = at + ((uint32_t)(D / 2) << a.page_shift) + row * (uint32_t)(D / 16);
    };
    struct Pieces {
      u32x4 raw[T::UNITS];
      uint16_t scale[T::UNITS];
    };
    const auto fetch_k = [&](int st, int id, Pieces& x) {
#pragma unroll
      for (int k = 0; k < T::UNITS; ++k) {
        const int u = wave + PW * k;
        if (u >= NB) continue;
        const int piece = u * 64 + lane, key = piece / NB, b = piece % NB;
        uint64_t codes, scales;
        row_at(keys.lo + st * STEP + key, __shfl(id, key, 64), codes, scales);
        x.raw[k] = ld_16B(a.kc + codes + 16 * b);
        x.scale[k] = (uint16_t)ld_u16(a.kc + scales + 2 * b);
      }
    };
    const auto fetch_v = [&](int st, int id, Pieces& x) {
#pragma unroll
      for (int k = 0; k < T::UNITS; ++k) {
        const int u = wave + PW * k;
        if (u < NB || u >= 2 * NB) continue;
        uint64_t codes, scales;
        row_at(keys.lo + st * STEP + lane, id, codes, scales);
        x.raw[k] = ld_16B(a.vc + codes + 16 * (u - NB));
        x.scale[k] = (uint16_t)ld_u16(a.vc + scales + 2 * (u - NB));
      }
    };
    const auto stage_v = [&](const Pieces& x, int id) {
#pragma unroll
      for (int k = 0; k < T::UNITS; ++k) {
        const int u = wave + PW * k;
        if (u < NB || u >= 2 * NB) continue;
        uint8_t* rows16 = lds + (2 + T::VB) * T::HALF + (u - NB) * T::RAW;  // this unit's own
        uint16_t* scales = (uint16_t*)(rows16 + STEP * 16);
        *(u32x4*)(rows16 + (((lane >> 2) & 3) * 16 + g * 4 + (lane & 3)) * 16) = x.raw[k];
        // bytes behind the last key are anything, NaN included: their values enter as 0 * code
        scales[((lane >> 2) & 3) * 16 + (g >> 1) * 8 + (lane & 3) * 2 + (g & 1)] = (uint16_t)(id >= 0 ? x.scale[k] : 0);
      }
    };
    const auto unpack = [&](int kb, int vb, const Pieces& y) {
      uint8_t* kbuf = lds + kb * T::HALF;
      uint8_t* vbuf = lds + (2 + vb) * T::HALF;
#pragma unroll
      for (int k = 0; k < T::UNITS; ++k) {
        const int u = wave + PW * k;
        if (u < NB) {
          const uint32_t w[4] = {y.raw[k].x, y.raw[k].y, y.raw[k].z, y.raw[k].w};
          const int piece = u * 64 + lane, key = piece / NB, b = piece % NB;
          const half_t sc = __builtin_bit_cast(half_t, y.scale[k]);
          const half2_t s2 = half2_t{sc, sc};
          // operand (key group, block): lane group j holds values 8 j .. of the
          // block; keys are swizzled by the block so that neighbouring lanes'
          // writes, and a lane group's reads, meet distinct banks
          uint8_t* dst = kbuf + (((key >> 4) * NB + b) * 64 + ((key & 15) ^ ((b & 3) * 4))) * 16;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const H2x4 x = unpack8(w[j]);
            *(half8_t*)(dst + j * 256) = operand(x.v[0] * s2, x.v[1] * s2, x.v[2] * s2, x.v[3] * s2);
          }
        } else if (u < 2 * NB) {
          const int b = u - NB;
          const uint8_t* rows16 = lds + (2 + T::VB) * T::HALF + b * T::RAW;
          const uint16_t* scales = (const uint16_t*)(rows16 + STEP * 16);
          const u32x4 s0 = *(const u32x4*)(scales + g * 16), s1 = *(const u32x4*)(scales + g * 16 + 8);
          const uint32_t vsc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
          typedef int v2i __attribute__((ext_vector_type(2)));
          typedef v2i __attribute__((address_space(3))) lds_v2i;
          v2i v[2];
#pragma unroll
          for (int t = 0; t < 2; ++t)
            v[t] = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_v2i*)(rows16 + (g * 16 + col) * 16 + 8 * t));
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int mm = 0; mm < 2; ++mm) {
              const H2x4 x = unpack8((uint32_t)v[t][mm]);
              *(half8_t*)(vbuf + (((b * 2 + t) * 2 + mm) * 64 + lane) * 16) =
                  operand(x.v[0] * as_h2(vsc[4 * mm]), x.v[1] * as_h2(vsc[4 * mm + 1]), x.v[2] * as_h2(vsc[4 * mm + 2]),
                          x.v[3] * as_h2(vsc[4 * mm + 3]));
            }
        }
      }
    };

    half8_t q[C][NB];
    float factor[C];
#pragma unroll
    for (int c = 0; c < C; ++c) query_operands<NB>(a, q_raw[c], q[c], factor[c]);
    float4_t o[DT][C], l4[C];
    float m[C], limit[C], bias[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int t = 0; t < DT; ++t) o[t][c] = float4_t{0, 0, 0, 0};
      l4[c] = float4_t{0, 0, 0, 0};
      m[c] = limit[c] = NEG_INF;
      bias[c] = 0.f;
    }

    // operands of key group i, of block b of the values
    const auto read_k = [&](const uint8_t* kbuf, int i, half8_t (&f)[NB]) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
        f[j] = *(const half8_t*)(kbuf + ((i * NB + j) * 64 + g * 16 + (col ^ ((j & 3) * 4))) * 16);
    };
    const auto read_v = [&](const uint8_t* vbuf, int b, half8_t (&f)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = *(const half8_t*)(vbuf + ((b * 4 + j) * 64 + lane) * 16);
    };

    const int late = T::OFFSET && wave >= PW / 2 ? 1 : 0;
    const int steps_here = st1 - st0;
    // on equal terms the older waves of a SIMD win the vector unit, reach the
    // barrier early and wait there for the others
    if (late) __builtin_amdgcn_s_setprio(1);
    uint64_t oks = 0;  // which key groups have a page: four bits a step, the current one lowest
    const auto group_bits = [&](int id) -> uint64_t {
      const uint64_t m = __ballot(id >= 0);  // a group's first key tells for all of it
      return (m & 1) | (m >> 15 & 2) | (m >> 30 & 4) | (m >> 45 & 8);
    };
    // The pieces on their way are keys of step round + 2 and values of step
    // round + 3; the ids of those steps and the one after.
    Pieces x;
    int id_k = 0, id_v = 0, id_next = 0;
    if (steps_here > 0) {
      // (steps behind the last are fetched from page 0 and unpacked to places that nothing reads)
      int id[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) id[i] = page_id(st0 + i);
#pragma unroll
      for (int i = 0; i < 4; ++i) id[i] = checked(st0 + i, id[i]);
      oks = group_bits(id[0]) | group_bits(id[1]) << 4 | group_bits(id[2]) << 8;
      Pieces x0, x1;
      fetch_k(st0, id[0], x0);
      fetch_v(st0, id[0], x0);
      fetch_k(st0 + 1, id[1], x1);
      fetch_v(st0 + 1, id[1], x1);
      fetch_v(st0 + 2, id[2], x);
      stage_v(x0, id[0]);
      unpack(0, 0, x0);
      stage_v(x1, id[1]);
      if (late) {
        unpack(1, 1, x1);
        stage_v(x, id[2]);
        fetch_k(st0 + 2, id[2], x);
        fetch_v(st0 + 3, id[3], x);
        oks |= group_bits(id[3]) << 12;
        id_k = id[2];
        id_v = id[3];
        id_next = id[4];
      } else {
        id_k = id[1];
        id_v = id[2];
        id_next = page_id(st0 + 3);
#pragma unroll
        for (int k = 0; k < T::UNITS; ++k)
          if (wave + PW * k < NB) { x.raw[k] = x1.raw[k]; x.scale[k] = x1.scale[k]; }
      }
    }
    __syncthreads();
    int vb = 0;  // step n's place among the values
    for (int n = 0; n < steps_here; ++n) {
      const int base = keys.lo + (st0 + n) * STEP;
      const uint32_t ok = (uint32_t)oks & 15u;
      const bool active = base <= p1 && (a.window <= 0 || base + STEP - 1 > p0 - a.window);
      // S^T; each group's operands are read while the group before is multiplied
      // (the scheduling barriers keep that order)
      float4_t sc[C][4];
      if (active) {
        const uint8_t* kbuf = lds + (n & 1) * T::HALF;
        half8_t kf[2][NB];
        read_k(kbuf, 0, kf[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i < 3) read_k(kbuf, i + 1, kf[(i + 1) & 1]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int c = 0; c < C; ++c) sc[c][i] = float4_t{0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int c = 0; c < C; ++c)
              sc[c][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[i & 1][j], q[c][j], sc[c][i], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (late) __syncthreads();
      if (active) {
        const uint8_t* vbuf = lds + (2 + vb) * T::HALF;
        half8_t vf[2][4];
        read_v(vbuf, 0, vf[0]);
        if (base + STEP - 1 > p0 || (a.window > 0 && base <= p1 - a.window) || ok != 15u) {
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int k = base + 16 * i + 4 * g + j;
                const bool see = ((ok >> i) & 1u) && k <= p[c] && (a.window <= 0 || k > p[c] - a.window);
                sc[c][i][j] = see ? sc[c][i][j] : NEG_INF;
              }
        }
        // running maximum; the sums move to a new one only when it is well above the old
        half8_t pt[C][2];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float mx = sc[c][0][0];
#pragma unroll
          for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[c][i >> 2][i & 3]);
          mx = groups_max(mx);
          if (__any(!(mx <= limit[c]))) {
            const float corr = move_maximum(mx, factor[c], sc[c], m[c], limit[c], bias[c]);
            l4[c] *= corr;
#pragma unroll
            for (int t = 0; t < DT; ++t) o[t][c] *= corr;
          }
          // P^T operands: places (2 s, 2 s + 1) hold keys s of groups 2 m and 2 m + 1
#pragma unroll
          for (int mm = 0; mm < 2; ++mm)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              pt[c][mm][2 * j] = (half_t)__builtin_amdgcn_exp2f(fmaf(sc[c][2 * mm][j], factor[c], bias[c]));
              pt[c][mm][2 * j + 1] = (half_t)__builtin_amdgcn_exp2f(fmaf(sc[c][2 * mm + 1][j], factor[c], bias[c]));
            }
          // sums of the (rounded) probabilities: one more row tile of V^T, all ones
          const half_t one = (half_t)1.f;
          const half8_t ones = half8_t{one, one, one, one, one, one, one, one};
          l4[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pt[c][0], l4[c], 0, 0, 0);
          l4[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pt[c][1], l4[c], 0, 0, 0);
        }
        // O^T += V^T P^T, read ahead likewise
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (b + 1 < NB) read_v(vbuf, b + 1, vf[(b + 1) & 1]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < C; ++c)
              o[2 * b + (j >> 1)][c] =
                  __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[b & 1][j], pt[c][j & 1], o[2 * b + (j >> 1)][c], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      // the round's step + 1 is unpacked; its values were staged the round before
      const int round = n + late;
      int vn = vb + 1 + late;
      vn = vn >= T::VB ? vn - T::VB : vn;
      unpack((round + 1) & 1, vn, x);
      stage_v(x, id_v);
      id_k = id_v;
      id_v = checked(st0 + round + 3, id_next);
      id_next = page_id(st0 + round + 4);
      oks = oks >> 4 | group_bits(id_v) << (4 * (2 + late));
      fetch_k(st0 + round + 2, id_k, x);
      fetch_v(st0 + round + 3, id_v, x);
      vb = vb + 1 == T::VB ? 0 : vb + 1;
      if (!late) __syncthreads();
    }

#pragma unroll
    for (int c = 0; c < C; ++c) {
      int ocol = col;
      asm volatile("" : "+v"(ocol));  // (computed here, not kept over the steps)
      const int row = w0 + 16 * c + ocol, qt = token_of(a, row);
      if (row >= rows) continue;
      const int64_t orow = (int64_t)(sq.row0 + qt) * a.hq + h * a.group + row - qt * a.group;
      const float l = l4[c][0];
      if (!SHARE || pieces == 1) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // no key seen: zeros
#pragma unroll
        for (int t = 0; t < DT; ++t) store4(a.out, a.out_type, orow * D + 16 * t + 4 * g, o[t][c] * inv);
      } else {
        const int64_t pr = (((int64_t)wg * a.hkv + h) * 2 + (st0 == 0 ? 1 : 0)) * T::ROWS + row - r0;
#pragma unroll
        for (int t = 0; t < DT; ++t) store4<0>(a.many, pr * D + 16 * t + 4 * g, o[t][c]);
        if (g == 0) {
          float* ml = a.many + (int64_t)a.many_wgs * a.hkv * 2 * T::ROWS * D + 2 * pr;
          ml[0] = sums_at(m[c], factor[c]);  // for the join
          ml[1] = l;
        }
      }
    }
    if (!SHARE) return;
    if (late) __builtin_amdgcn_s_setprio(0);
    __syncthreads();  // the next tile reuses the LDS
  }
}

template <int NB>
hipError_t launch_prompt(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const dim3 grid((unsigned)((a.many_wgs > 0 ? a.many_wgs : p.many_tiles) * a.hkv));
  if (a.many_wgs > 0) hipLaunchKernelGGL((attn_prompt_kernel<NB, true>), grid, dim3(64 * PW), Prompt<NB>::LDS, s, a);
  else hipLaunchKernelGGL((attn_prompt_kernel<NB, false>), grid, dim3(64 * PW), Prompt<NB>::LDS, s, a);
  return hipGetLastError();
}

}  // namespace

int attn_prompt_rows(int64_t d) { return d <= 128 ? Prompt<4>::ROWS : Prompt<8>::ROWS; }

hipError_t launch_attn_prompt(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  switch (a.d / 32) {
    case 1: return launch_prompt<1>(a, p, s);
    case 2: return launch_prompt<2>(a, p, s);
    case 3: return launch_prompt<3>(a, p, s);
    case 4: return launch_prompt<4>(a, p, s);
    case 5: return launch_prompt<5>(a, p, s);
    case 6: return launch_prompt<6>(a, p, s);
    case 7: return launch_prompt<7>(a, p, s);
    default: return launch_prompt<8>(a, p, s);
  }
}

}  // namespace kq
