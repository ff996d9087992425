// kq_kv_attention for many rows that share keys (prompts): the same products
// as kq_kv_attn.hip, but a workgroup's eight waves share each 64-key step.  A
// wave takes C 16-row tiles of its own; the step's keys and values are
// unpacked to float16 once, by all waves together, into LDS in the order of
// the matrix operands, and every wave reads them from there.  Two steps'
// buffers: while one is multiplied the next is unpacked, and the one after
// that is on its way from memory; one barrier a step.
#include "kq_kv_attn.h"

namespace kq {
namespace {

constexpr int PW = 8;     // waves
constexpr int STEP = 64;  // keys of one step

template <int NB>
struct Prompt {
  static constexpr int C = NB <= 4 ? 2 : 1;             // 16-row tiles of a wave (its sums fill the registers)
  static constexpr int ROWS = PW * C * 16;              // rows of a workgroup
  static constexpr int UNITS = (2 * NB + PW - 1) / PW;  // unpacking units of a wave: 64 pieces of 32 values
  static constexpr int HALF = STEP * 32 * NB * 2;       // float16 keys (or values) of a step
  static constexpr int RAW = STEP * 16 + STEP * 2;      // one block's codes and scales, on the way to the transposing read
  static constexpr int LDS = 4 * HALF + NB * RAW;
};

template <int NB>
__global__ __launch_bounds__(64 * PW, 2) void attn_prompt_kernel(AttnArgs a) {
  typedef Prompt<NB> T;
  constexpr int D = 32 * NB, DT = D / 16, C = T::C;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x % a.hkv, split = blockIdx.y;

  int s = 0, sub = 0;
  if (!find_tile(a, blockIdx.x / a.hkv, T::ROWS, a.few_rows, 0x7FFFFFFF, s, sub)) return;
  const Seq sq = load_seq(a, s);
  const int rows = sq.n * a.group;
  sub = (rows + T::ROWS - 1) / T::ROWS - 1 - sub;  // the tiles with the most keys first
  const int r0 = sub * T::ROWS, r1 = r0 + T::ROWS < rows ? r0 + T::ROWS - 1 : rows - 1;
  const Keys keys = key_range(a, sq, r0, r1);
  const int n_split = split_count(a, keys);

  // the wave's rows: positions of its first and last, none if w0 > w1
  const int w0 = r0 + wave * C * 16, w1 = w0 + C * 16 - 1 < rows ? w0 + C * 16 - 1 : rows - 1;
  const int p0 = sq.len - sq.n + w0 / a.group, p1 = w0 <= w1 ? sq.len - sq.n + w1 / a.group : -1;
  int64_t orow[C];
  int p[C];
  bool live[C];
  half8_t q[C][NB];
  float factor[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int row = w0 + 16 * c + col;
    live[c] = row < rows;
    const int tok = sq.row0 + row / a.group, head = h * a.group + row % a.group;
    orow[c] = (int64_t)tok * a.hq + head;
    p[c] = live[c] ? sq.len - sq.n + row / a.group : -1;
    load_query<NB, 8, 32>(a, (const uint16_t*)a.q + (int64_t)tok * a.q_stride + (int64_t)head * D, live[c], g, q[c],
                          factor[c]);
  }
  if (split >= (n_split > 0 ? n_split : 1)) return;
  if (a.splits > 1 && split == 0 && g == 0) {
    int32_t* counts = (int32_t*)(a.part + part_rows(a.tokens, a.hq, a.splits) * (D + 2));
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (live[c]) counts[orow[c]] = n_split > 1 ? n_split : 0;
  }

  const int steps = (keys.end - keys.lo + STEP - 1) / STEP;
  const int st0 = n_split ? (int)((int64_t)steps * split / n_split) : 0;
  const int st1 = n_split ? (int)((int64_t)steps * (split + 1) / n_split) : 0;
  const auto* pages = (const __attribute__((address_space(4))) int32_t*)(a.table + (int64_t)s * a.width);

  // the pieces of a step that this wave unpacks: unit u < NB is 64 pieces of
  // keys (lanes on consecutive pieces), unit NB + b block b of 64 values rows
  u32x4 raw[T::UNITS];
  uint16_t rsc[T::UNITS];
  const auto fetch = [&](int st) {
    int ids[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = keys.lo + st * STEP + 16 * i;
      ids[i] = k < keys.end ? pages[k >> a.page_shift] : -1;
    }
    const int base = keys.lo + st * STEP;
    const Groups gr = groups_of<D>(a, ids, base, keys.end, h);
#pragma unroll
    for (int k = 0; k < T::UNITS; ++k) {
      const int u = wave + PW * k;
      if (u < NB) {
        const int piece = u * 64 + lane, key = piece / NB, b = piece % NB;
        raw[k] = ld_16B(a.kc + pick4(gr.codes, key >> 4) + (uint32_t)((key & 15) * (D / 2) + 16 * b));
        rsc[k] = (uint16_t)ld_u16(a.kc + pick4(gr.scales, key >> 4) + (uint32_t)((key & 15) * (D / 16) + 2 * b));
      } else if (u < 2 * NB) {
        const int b = u - NB;
        raw[k] = ld_16B(a.vc + pick4(gr.codes, g) + (uint32_t)(col * (D / 2) + 16 * b));
        const uint32_t sc = ld_u16(a.vc + pick4(gr.scales, g) + (uint32_t)(col * (D / 16) + 2 * b));
        // bytes behind the last key are anything, NaN included: their values enter as 0 * code
        rsc[k] = ((gr.ok >> g) & 1u) && base + lane < keys.end ? (uint16_t)sc : (uint16_t)0;
      }
    }
    return gr.ok;
  };
  const auto unpack = [&](int buf) {
    uint8_t* kbuf = lds + buf * 2 * T::HALF;
    uint8_t* vbuf = kbuf + T::HALF;
#pragma unroll
    for (int k = 0; k < T::UNITS; ++k) {
      const int u = wave + PW * k;
      const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
      if (u < NB) {
        const int piece = u * 64 + lane, key = piece / NB, b = piece % NB;
        const half_t sc = __builtin_bit_cast(half_t, rsc[k]);
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
        uint8_t* rows16 = lds + 4 * T::HALF + b * T::RAW;  // this unit's own
        uint16_t* scales = (uint16_t*)(rows16 + STEP * 16);
        *(u32x4*)(rows16 + (((lane >> 2) & 3) * 16 + g * 4 + (lane & 3)) * 16) = raw[k];
        scales[((lane >> 2) & 3) * 16 + (g >> 1) * 8 + (lane & 3) * 2 + (g & 1)] = rsc[k];
        const u32x4 s0 = *(const u32x4*)(scales + g * 16), s1 = *(const u32x4*)(scales + g * 16 + 8);
        const uint32_t vsc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          typedef int v2i __attribute__((ext_vector_type(2)));
          typedef v2i __attribute__((address_space(3))) lds_v2i;
          const v2i v = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_v2i*)(rows16 + (g * 16 + col) * 16 + 8 * t));
#pragma unroll
          for (int mm = 0; mm < 2; ++mm) {
            const H2x4 x = unpack8((uint32_t)v[mm]);
            *(half8_t*)(vbuf + (((b * 2 + t) * 2 + mm) * 64 + lane) * 16) =
                operand(x.v[0] * as_h2(vsc[4 * mm]), x.v[1] * as_h2(vsc[4 * mm + 1]), x.v[2] * as_h2(vsc[4 * mm + 2]),
                        x.v[3] * as_h2(vsc[4 * mm + 3]));
          }
        }
      }
    }
  };

  float4_t o[DT][C], l4[C];
  float m[C], slack[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int t = 0; t < DT; ++t) o[t][c] = float4_t{0, 0, 0, 0};
    l4[c] = float4_t{0, 0, 0, 0};
    m[c] = NEG_INF;
    slack[c] = 8.f / factor[c];  // probabilities may reach 2^8 before the sums are brought to a new maximum
  }

  uint32_t ok = 0, ok_next = 0;
  if (st0 < st1) {
    ok = fetch(st0);
    unpack(0);
    if (st0 + 1 < st1) ok_next = fetch(st0 + 1);
  }
  __syncthreads();
  for (int st = st0; st < st1; ++st) {
    const int buf = (st - st0) & 1, base = keys.lo + st * STEP;
    uint32_t ok_after = 0;
    if (st + 1 < st1) {
      unpack(buf ^ 1);
      if (st + 2 < st1) ok_after = fetch(st + 2);
    }
    if (base <= p1 && (a.window <= 0 || base + STEP - 1 > p0 - a.window)) {
      const uint8_t* kbuf = lds + buf * 2 * T::HALF;
      const uint8_t* vbuf = kbuf + T::HALF;
      // S^T
      float4_t sc[C][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int c = 0; c < C; ++c) sc[c][i] = float4_t{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const half8_t kf = *(const half8_t*)(kbuf + ((i * NB + j) * 64 + g * 16 + (col ^ ((j & 3) * 4))) * 16);
#pragma unroll
          for (int c = 0; c < C; ++c) sc[c][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, q[c][j], sc[c][i], 0, 0, 0);
        }
      }
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
        if (__any(!(mx <= m[c] + slack[c]))) {
          mx = fmaxf(mx, m[c]);
          const float corr = mx == NEG_INF ? 1.f : __builtin_amdgcn_exp2f((m[c] - mx) * factor[c]);
          m[c] = mx;
          l4[c] *= corr;
#pragma unroll
          for (int t = 0; t < DT; ++t) o[t][c] *= corr;
        }
        const float bias = m[c] == NEG_INF ? 0.f : -m[c] * factor[c];
        // P^T operands: places (2 s, 2 s + 1) hold keys s of groups 2 m and 2 m + 1
#pragma unroll
        for (int mm = 0; mm < 2; ++mm)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            pt[c][mm][2 * j] = (half_t)__builtin_amdgcn_exp2f(fmaf(sc[c][2 * mm][j], factor[c], bias));
            pt[c][mm][2 * j + 1] = (half_t)__builtin_amdgcn_exp2f(fmaf(sc[c][2 * mm + 1][j], factor[c], bias));
          }
        // sums of the (rounded) probabilities: one more row tile of V^T, all ones
        const half_t one = (half_t)1.f;
        const half8_t ones = half8_t{one, one, one, one, one, one, one, one};
        l4[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pt[c][0], l4[c], 0, 0, 0);
        l4[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pt[c][1], l4[c], 0, 0, 0);
      }
      // O^T += V^T P^T
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int mm = 0; mm < 2; ++mm) {
          const half8_t vf = *(const half8_t*)(vbuf + ((t * 2 + mm) * 64 + lane) * 16);
#pragma unroll
          for (int c = 0; c < C; ++c) o[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pt[c][mm], o[t][c], 0, 0, 0);
        }
    }
    ok = ok_next;
    ok_next = ok_after;
    __syncthreads();
  }

#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (!live[c]) continue;
    const float l = l4[c][0];
    if (n_split <= 1) {
      const float inv = l == 0.f ? 0.f : 1.f / l;  // no key seen: zeros
#pragma unroll
      for (int t = 0; t < DT; ++t) store4(a.out, a.out_type, orow[c] * D + 16 * t + 4 * g, o[t][c] * inv);
    } else {
      const int64_t pr = (int64_t)split * a.tokens * a.hq + orow[c];
#pragma unroll
      for (int t = 0; t < DT; ++t) store4<0>(a.part, pr * D + 16 * t + 4 * g, o[t][c]);
      if (g == 0) {
        float* ml = a.part + part_rows(a.tokens, a.hq, a.splits) * D + 2 * pr;
        ml[0] = m[c] == NEG_INF ? NEG_INF : m[c] * factor[c];  // in powers of two, for the merge
        ml[1] = l;
      }
    }
  }
}

template <int NB>
hipError_t launch_prompt(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.many_tiles * a.hkv), (unsigned)a.splits);
  hipLaunchKernelGGL((attn_prompt_kernel<NB>), grid, dim3(64 * PW), Prompt<NB>::LDS, s, a);
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
