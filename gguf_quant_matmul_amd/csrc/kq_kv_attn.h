// Pieces shared by the attention kernels over the 4-bit cache
// (kq_kv_attention): a request's rows and the keys they see, page lookups,
// and the unpacking of 4-bit keys and values into matrix operands.
//
// The rows of a (request, kv head) are its new tokens times the group of
// query heads that share the kv head: row r is token r / group, query head
// kv_head * group + r % group.
//
// Three things are rounded to float16, half a step (2^-11) each, because the
// matrix cores take them so: keys and values, whose exact D (c - 8) has up to
// 14 bits, and probabilities, which are summed as rounded.  A float16 result is
// then 4e-4 from the exact one, of which its own rounding is 2.1e-4.  Exact
// keys would need the scales applied behind the products, block by block (one
// more vector operation for every product sum of 32 values and row), exact
// values and probabilities these in two terms, twice the matrix work.
#pragma once

#include "kq_internal.h"

namespace kq {

constexpr float NEG_INF = -__builtin_inff();

// A request as the kernels see it: device data clamped to what is in bounds.
struct Seq {
  int row0, n;  // first token row, new tokens
  int len;      // keys
};
typedef const __attribute__((address_space(4))) int32_t* ConstInts;  // read only here: scalar loads may fetch it
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int s) {
  int b = ((ConstInts)a.cu)[s], e = ((ConstInts)a.cu)[s + 1];
  b = b < 0 ? 0 : b > a.tokens ? a.tokens : b;
  e = e < b ? b : e > a.tokens ? a.tokens : e;
  const int64_t cap = a.width << a.page_shift;
  int64_t len = ((ConstInts)a.lens)[s];
  len = len < 0 ? 0 : len > cap ? cap : len;
  return Seq{b, e - b, (int)len};
}

// Token of a request's row (a shift where the group is a power of two: an
// integer division is some 25 instructions).
__device__ __forceinline__ int token_of(const AttnArgs& a, int row) {
  return a.group_shift >= 0 ? row >> a.group_shift : (int)((uint32_t)row / (uint32_t)a.group);
}

// Keys that rows r0 .. r1 of a request see: lo (64-aligned) .. end - 1.
struct Keys {
  int lo, end;
};
__device__ __forceinline__ Keys key_range(const AttnArgs& a, const Seq& q, int r0, int r1) {
  const int p0 = q.len - q.n + token_of(a, r0), p1 = q.len - q.n + token_of(a, r1);  // positions
  Keys k;
  k.end = p1 + 1 > 0 ? p1 + 1 : 0;
  const int64_t lo = a.window > 0 ? (int64_t)p0 - a.window + 1 : 0;
  k.lo = (lo > 0 ? (int)lo : 0) & ~63;
  return k;
}
constexpr int STEP = 64;  // keys of one step
constexpr float HEADROOM = 7.f;  // log2 of the weight of a running maximum

// What a tile costs beside its steps, in steps: its start and its end.  (Shares
// of steps alone gave some workgroups ten short tiles: 9 requests of mixed
// prompts 377 us against 350, a prompt of 4096 tokens 284 against 240.)
template <int ROWS>
constexpr int TILE_EXTRA = ROWS == 16 ? 6 : 5;

// Cost of a tile of ROWS rows of a request; a tile without keys counts as
// one step, so that someone writes its zeros.
template <int ROWS>
__device__ __forceinline__ int tile_cost(const AttnArgs& a, const Seq& q, int sub) {
  const int rows = q.n * a.group, r0 = sub * ROWS, r1 = r0 + ROWS - 1 < rows ? r0 + ROWS - 1 : rows - 1;
  const Keys k = key_range(a, q, r0, r1);
  return (k.end > k.lo ? (k.end - k.lo + STEP - 1) / STEP : 1) + TILE_EXTRA<ROWS>;
}
// ... of all tiles of a request with more than `above` and at most `most` rows
// (64-bit: 2^21 tiles of 2^24 steps are within the bounds on a call's sizes).
template <int ROWS>
__device__ __forceinline__ uint64_t request_cost(const AttnArgs& a, int s, int above, int most) {
  if (s >= a.n_seqs) return 0;
  const Seq q = load_seq(a, s);
  const int rows = q.n * a.group;
  if (rows <= above || rows > most) return 0;
  uint64_t n = 0;
  for (int sub = 0; sub * ROWS < rows; ++sub) n += (uint32_t)tile_cost<ROWS>(a, q, sub);
  return n;
}

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) << 32 |
         (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v);
}
// inclusive prefix sum over the wave's lanes
__device__ __forceinline__ uint64_t wave_prefix(uint64_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t t = __shfl_up(v, o, 64);
    if (lane >= o) v += t;
  }
  return v;
}

// The part of one of `wgs` workgroups (of a kv head) that share out the cost
// of all those requests' tiles evenly, `least` to one at least: x0 .. x1 - 1
// of the whole, `size` to a workgroup.
// A tile's steps come first, then its extra, which nobody works on.  The part
// begins in tile `sub` of request s, whose own begins at x.  False for a
// workgroup without a part.  Every wave finds it for itself, 64 requests
// and then 64 tiles at a time.
struct Share {
  uint64_t x, x0, x1, size;
};
template <int ROWS>
__device__ __forceinline__ bool find_share(const AttnArgs& a, int wg, int wgs, int least, int above, int most, int& s,
                                           int& sub, Share& r) {
  const int lane = threadIdx.x & 63;
  uint64_t total = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 64) {
    uint64_t n = request_cost<ROWS>(a, s0 + lane, above, most);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o, 64);
    total += n;
  }
  total = uniform64(total);
  r.size = (total + wgs - 1) / (uint64_t)wgs;
  r.size = r.size < (uint64_t)least ? least : r.size;
  r.x0 = r.size * (uint64_t)wg;
  r.x1 = r.x0 + r.size < total ? r.x0 + r.size : total;
  if (r.x0 >= total) return false;
  // (both searches find their place, total > x0, unless someone changes the
  // lengths meanwhile; they end even so)
  uint64_t x = 0;
  s = -1;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 64) {
    const uint64_t n = request_cost<ROWS>(a, s0 + lane, above, most), incl = wave_prefix(n);
    const uint64_t hit = __ballot(x + incl > r.x0);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      s = s0 + l;
      x += __shfl(incl - n, l, 64);
      break;
    }
    x += __shfl(incl, 63, 64);
  }
  s = __builtin_amdgcn_readfirstlane(s);
  if (s < 0) return false;
  const Seq q = load_seq(a, s);
  const int tiles = (q.n * a.group + ROWS - 1) / ROWS;
  for (int t0 = 0; t0 < tiles; t0 += 64) {
    const uint64_t n = t0 + lane < tiles ? (uint64_t)tile_cost<ROWS>(a, q, t0 + lane) : 0, incl = wave_prefix(n);
    const uint64_t hit = __ballot(x + incl > r.x0);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      sub = __builtin_amdgcn_readfirstlane(t0 + l);
      r.x = uniform64(x + __shfl(incl - n, l, 64));
      return true;
    }
    x += __shfl(incl, 63, 64);
  }
  return false;
}
// The workgroup's steps st0 .. st1 - 1 of a tile of `steps` steps that begins at
// r.x (r.x moves on to the next tile), the first workgroup that has some of
// the tile's and how many have.  False where the part begins in the tile's extra.
template <int ROWS>
__device__ __forceinline__ bool take_steps(Share& r, int steps, int& st0, int& st1, int& first, int& pieces) {
  const uint64_t x = r.x, end = x + (steps > 0 ? steps : 1);
  r.x = end + TILE_EXTRA<ROWS>;
  if (r.x0 >= end) return false;
  st0 = r.x0 > x ? (int)(r.x0 - x) : 0;
  st1 = r.x1 < end ? (int)(r.x1 - x) : steps;
  first = (int)(x / r.size);
  pieces = (int)((end - 1) / r.size) - first + 1;
  return true;
}

// Request and tile index inside it of tile `tile`, the tiles of the requests
// with more than `above` and at most `most` rows numbered one after the other
// (`rows` rows to a tile); false past the last.  Every wave scans the requests
// 64 at a time.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int tile, int rows, int above, int most, int& seq,
                                          int& sub) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 64) {
    const int s = s0 + lane;
    int64_t t = 0;
    if (s < a.n_seqs) {
      const int r = load_seq(a, s).n * a.group;
      t = r > above && r <= most ? (r + rows - 1) / rows : 0;
    }
    int64_t incl = t;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t u = __shfl_up(incl, o, 64);
      if (lane >= o) incl += u;
    }
    const uint64_t hit = __ballot(before + incl > tile);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      seq = s0 + l;
      sub = (int)(tile - before - (__shfl(incl, l, 64) - __shfl(t, l, 64)));
      seq = __builtin_amdgcn_readfirstlane(seq);
      sub = __builtin_amdgcn_readfirstlane(sub);
      return true;
    }
    before += __shfl(incl, 63, 64);
  }
  return false;
}

// A step's four 16-key groups: byte offsets of their codes and scales in the
// caches, and which of them are there (a group past the last key or without a
// page of the cache reads page 0 and is left out).  Uniform over the wave.
struct Groups {
  int64_t codes[4], scales[4];
  uint32_t ok;  // bit i
};
template <int D>
__device__ __forceinline__ Groups groups_of(const AttnArgs& a, const int (&ids)[4], int base, int end, int h) {
  Groups r;
  r.ok = 0;
  const int mask = (1 << a.page_shift) - 1;
  const int64_t behind = (int64_t)(D / 2) << a.page_shift;  // a page's scales follow its codes
  if (a.page_shift >= 6) {  // a step lies in one page
    const bool ok = ids[0] >= 0 && ids[0] < a.pages;
    const int64_t at = ((int64_t)(ok ? ids[0] : 0) * a.hkv + h) * a.page_head_bytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.codes[i] = at + (int64_t)((base & mask) + 16 * i) * (D / 2);
      r.scales[i] = at + behind + (int64_t)((base & mask) + 16 * i) * (D / 16);
      r.ok |= ok && base + 16 * i < end ? 1u << i : 0u;
    }
    return r;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = base + 16 * i;
    const bool ok = k < end && ids[i] >= 0 && ids[i] < a.pages;
    const int64_t at = ((int64_t)(ok ? ids[i] : 0) * a.hkv + h) * a.page_head_bytes;
    r.codes[i] = at + (int64_t)(k & mask) * (D / 2);
    r.scales[i] = at + behind + (int64_t)(k & mask) * (D / 16);
    r.ok |= ok ? 1u << i : 0u;
  }
  return r;
}

template <typename T>
__device__ __forceinline__ T pick4(const T (&v)[4], int i) {
  const T lo = i & 1 ? v[1] : v[0], hi = i & 1 ? v[3] : v[2];
  return i & 2 ? hi : lo;
}

// N consecutive dwords from a 4-byte aligned address (16- or 8-byte loads
// where N allows them).
template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t* p, uint32_t* r) {
  constexpr int Q = N / 4, H = (N % 4) / 2;
  typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(4)));
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const u32x4 v = ld_16B_a4(p + 16 * i);
    r[4 * i] = v.x; r[4 * i + 1] = v.y; r[4 * i + 2] = v.z; r[4 * i + 3] = v.w;
  }
  if constexpr (H) {
    const u2 v = *(const u2*)(p + 16 * Q);
    r[4 * Q] = v.x; r[4 * Q + 1] = v.y;
  }
  if constexpr (N % 2) r[N - 1] = ld_u32(p + 4 * (N - 1));
}

// Eight codes (nibbles of w) as float16 pairs (n0, n4) (n1, n5) (n2, n6)
// (n3, n7), each c - 8: a nibble or-ed into the low mantissa bits of 1024 is
// 1024 + c, one or-ed four bits higher 1024 + 16 c; both come out exactly.
struct H2x4 {
  half2_t v[4];
};
__device__ __forceinline__ H2x4 unpack8(uint32_t w) {
  // in a vector register, so that and-or is one instruction (it takes one
  // scalar operand, the mask): 13 instead of 17 for eight values
  uint32_t M = 0x64006400u;
  asm("" : "+v"(M));
  const uint32_t u = w >> 8;
  const half2_t k0 = half2_t{(half_t)1032.f, (half_t)1032.f}, k1 = half2_t{(half_t)-72.f, (half_t)-72.f},
                s = half2_t{(half_t)0.0625f, (half_t)0.0625f};
  H2x4 r;
  r.v[0] = as_h2((w & 0x000F000Fu) | M) - k0;
  r.v[1] = __builtin_elementwise_fma(as_h2((w & 0x00F000F0u) | M), s, k1);
  r.v[2] = as_h2((u & 0x000F000Fu) | M) - k0;
  r.v[3] = __builtin_elementwise_fma(as_h2((u & 0x00F000F0u) | M), s, k1);
  return r;
}
__device__ __forceinline__ half8_t operand(half2_t a, half2_t b, half2_t c, half2_t d) {
  return half8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Eight values of a query row in unpack8's order (0 4 1 5 2 6 3 7).
__device__ __forceinline__ half8_t query_order(half8_t v) {
  return __builtin_shufflevector(v, v, 0, 4, 1, 5, 2, 6, 3, 7);
}

// Maximum over the four lane groups that hold one query's keys (lanes l,
// l ^ 16, l ^ 32, l ^ 48): two row swaps, which stay in the vector unit where
// a shuffle would go through LDS.
__device__ __forceinline__ float groups_max(float v) {
  uint32_t x = __builtin_bit_cast(uint32_t, v);
  auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  // copies: __builtin_bit_cast of a vector's element reads element 0
  uint32_t lo = r[0], hi = r[1];
  v = fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
  x = __builtin_bit_cast(uint32_t, v);
  r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  lo = r[0];
  hi = r[1];
  return fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
}

// Query operands of one row for NB = d / 32 matrix steps: lane group g of
// step s holds eight values from g * GS + s * SS on.  bfloat16 values are scaled by
// a power of two that brings the row's largest near 2^14, which float16
// holds exactly down to 2^-28 of the largest; `factor` takes that power of two
// back out of the products, times scale * log2(e).  A negative scale is put
// into the queries' signs, so that factor > 0 and the largest product has the
// largest weight.
// In two parts, so that other loads can go out before the first is waited for.
template <int NB, int GS, int SS>
__device__ __forceinline__ void load_query(const AttnArgs& a, int64_t tok, int head, bool live, int g, u32x4 (&raw)[NB]) {
  const uint16_t* row = (const uint16_t*)a.q + tok * a.q_stride + (int64_t)head * (32 * NB) + g * GS;
#pragma unroll
  for (int s = 0; s < NB; ++s) raw[s] = live ? *(const u32x4*)(row + s * SS) : u32x4{0, 0, 0, 0};
}
template <int NB>
__device__ __forceinline__ void query_operands(const AttnArgs& a, const u32x4 (&raw)[NB], half8_t (&q)[NB],
                                               float& factor) {
  const float log2e = 1.4426950408889634f;
  const bool neg = a.scale < 0.f;
  factor = fabsf(a.scale);
  if (a.q_bf16) {
    float v[NB][8], amax = 0.f;
#pragma unroll
    for (int s = 0; s < NB; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = raw[s][i];
        v[s][2 * i] = __builtin_bit_cast(float, w << 16);
        v[s][2 * i + 1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
        amax = fmaxf(amax, fmaxf(fabsf(v[s][2 * i]), fabsf(v[s][2 * i + 1])));
      }
    amax = groups_max(amax);
    // NaN and infinities keep their places; a row of zeros keeps its size
    int e = amax > 0.f && amax < __builtin_inff() ? (int)((__builtin_bit_cast(uint32_t, amax) >> 23) & 255u) - 127 : 14;
    e = e < -100 ? -100 : e;
    const float up = __builtin_bit_cast(float, (uint32_t)(127 + 14 - e) << 23);
    factor *= __builtin_bit_cast(float, (uint32_t)(127 - 14 + e) << 23);
#pragma unroll
    for (int s = 0; s < NB; ++s) {
      half8_t h;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (half_t)(neg ? -v[s][i] * up : v[s][i] * up);
      q[s] = query_order(h);
    }
  } else {
#pragma unroll
    for (int s = 0; s < NB; ++s) {
      const u32x4 w = raw[s];
      half8_t h = __builtin_bit_cast(half8_t, w);
      if (neg) h = -h;
      q[s] = query_order(h);
    }
  }
  // a zero factor would turn masked -inf into NaN; above 2^80 products, whole
  // multiples of 2^-48 below 2^40, give the weights they give at 2^80 (unequal
  // ones are at least 2^32 apart), and their logits could pass float32
  factor = fminf(fmaxf(factor * log2e, 1.17549435e-38f), 0x1p80f);
}

// A row's softmax over the steps: weights are 2^(product * factor + bias), of
// products up to `limit`, with bias = 7 - m * factor for a running maximum m.
// Moves m, limit and bias for a step whose largest product passes the limit
// (NaN does); returns what the sums so far are to be multiplied by.
//   Weights enter the matrix cores as float16, each off by half a step, 2^-11
// of itself.  The 2^7 at the maximum (with the 2^8 below, half of what float16
// holds) is for the small ones: those of 2^-21 of it and more keep that
// precision and nothing above 2^-32 is lost, where 1 would lose all below
// 2^-25; 131072 keys of 2^-25 each are 0.4% of a row.  It is in the sums too,
// and goes out with the quotient.
//   The limit is above m by 2^8 in weights, so that few steps move m.
//   Where m * factor is so large that a float32 there is 1/2 or more from the
// next, the bias would be off by its rounding, and weights that should be at
// most 1 come out infinite, or all of them zero.  Such a row takes m off the
// products themselves, which is exact near it, and has no limit above it: all
// its steps come here (every row doing so would be one more vector operation a
// weight: prompts 4% slower, as with a branch of its own in the step).
__device__ __forceinline__ float move_maximum(float mx, float factor, float4_t (&sc)[4], float& m, float& limit,
                                              float& bias) {
  mx = fmaxf(mx, m);
  const float corr = mx == NEG_INF ? 1.f : __builtin_amdgcn_exp2f((m - mx) * factor);
  m = mx;
  const bool none = m == NEG_INF, far = !none && fabsf(m * factor) >= 4194304.f;
  limit = none || far ? NEG_INF : m + 8.f * __builtin_amdgcn_rcpf(factor);
  bias = none ? 0.f : far ? HEADROOM : fmaf(-m, factor, HEADROOM);
#pragma unroll
  for (int i = 0; i < 16; ++i) sc[i >> 2][i & 3] -= far ? m : 0.f;
  return corr;
}

// log2 of what a row's sums are to be multiplied by beside others of the row:
// the very bias of its weights, negative.
__device__ __forceinline__ float sums_at(float m, float factor) {
  return m == NEG_INF ? NEG_INF : fmaf(m, factor, -HEADROOM);
}

template <int OUT>
__device__ __forceinline__ void store4(void* out, int64_t i, float4_t v) {
  if constexpr (OUT == 0) {
    *(float4_t*)((float*)out + i) = v;
  } else if constexpr (OUT == 1) {
    typedef half_t h4 __attribute__((ext_vector_type(4)));
    *(h4*)((half_t*)out + i) = h4{(half_t)v.x, (half_t)v.y, (half_t)v.z, (half_t)v.w};
  } else {
    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
    *(b4*)((__bf16*)out + i) = b4{(__bf16)v.x, (__bf16)v.y, (__bf16)v.z, (__bf16)v.w};
  }
}
__device__ __forceinline__ void store4(void* out, int type, int64_t i, float4_t v) {
  if (type == 0) store4<0>(out, i, v);
  else if (type == 1) store4<1>(out, i, v);
  else store4<2>(out, i, v);
}

}  // namespace kq
