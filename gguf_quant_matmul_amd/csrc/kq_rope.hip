// kq_rope: rows of queries and keys rotated to their positions.
//
//   x_i' = m (x_i cos a - x_j sin a),  x_j' = m (x_j cos a + x_i sin a),  a = p f_i
//
// with (i, j) = (i, i + rot / 2) or (2 i, 2 i + 1).  A wave takes a token (few
// tokens: a slice of its heads): it finds the token's request among the
// offsets, 64 of them at a time, computes the rot / 2 angles, a lane to one,
// and shares their cosines and sines through LDS over all heads.  The angle is
// exact in float64 (31 + 24 bits of 53 are lost only beyond 2^29 tokens) and is
// brought to a quarter turn there; sine and cosine are then float32 Taylor
// sums, 2^-23 off at most, so that far positions are as exact as near ones.
// Rows are read and written once, 16 bytes a lane.
//   Measured: 7.7k tokens of 40 heads of 128 in bfloat16, half of each turned,
// 34.7 us, 4.6 TB/s of the 4.8 that a large copy reaches; 64 tokens 4.0 us
// by themselves (3.3 one behind the other in a graph), bound by the launch and three
// dependent loads.
#include "kq_internal.h"

namespace kq {
namespace {

constexpr int ROPE_WAVES = 4;
constexpr int ROPE_AHEAD = 4;  // units of a lane whose loads are out at once

template <int T> struct Elem;
template <> struct Elem<0> { typedef float type; };
template <> struct Elem<1> { typedef half_t type; };
template <> struct Elem<2> { typedef __bf16 type; };

// Position of token `tok`: that of its row in its request; -1 where it has
// none.  The same in all lanes.
__device__ __forceinline__ int64_t position_of(const RopeArgs& a, int tok) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = a.n_seqs;
  for (;;) {
    // the first request that ends behind the token lies in lo .. hi - 1
    const int step = (hi - lo + 63) / 64, last = lo + (lane + 1) * step - 1, i = last < hi ? last : hi - 1;
    const int end = a.cu[i + 1];
    int begin = 0, len = 0;
    if (step == 1) {
      begin = a.cu[i];
      len = a.lens[i];
    }
    const uint64_t hit = __ballot(end > tok);
    if (!hit) return -1;
    const int l = __builtin_ctzll(hit);
    if (step == 1) {
      const int64_t b = __shfl(begin, l, 64), e = __shfl(end, l, 64), n = __shfl(len, l, 64);
      return b <= tok ? (n < 0 ? 0 : n) - (e < a.tokens ? e : a.tokens) + tok : -1;
    }
    lo += l * step;
    hi = lo + step < hi ? lo + step : hi;
  }
}

__device__ __forceinline__ void sin_cos(double angle, float& s, float& c) {
  // quarter turns, and what is left of the angle (pi / 2 in two parts: 107 bits)
  const double turns = __builtin_rint(angle * 0.63661977236758134308);
  double r = __builtin_fma(-turns, 1.57079632679489655800, angle);
  r = __builtin_fma(-turns, 6.12323399573676603587e-17, r);
  const float x = (float)r, y = x * x;
  // |x| <= pi / 4: the first terms left out are 2e-9 and 1e-10
  float u = fmaf(y, 2.7557319e-6f, -1.9841270e-4f);  // 1 / 9!, 1 / 7!
  u = fmaf(y, u, 8.3333333e-3f);
  u = fmaf(y, u, -1.6666667e-1f);
  const float sn = fmaf(x * y, u, x);
  float v = fmaf(y, -2.7557319e-7f, 2.4801587e-5f);  // 1 / 10!, 1 / 8!
  v = fmaf(y, v, -1.3888889e-3f);
  v = fmaf(y, v, 4.1666667e-2f);
  v = fmaf(y, v, -0.5f);
  const float cn = fmaf(y, v, 1.f);
  const int q = (int)((long long)turns & 3);
  s = q & 1 ? cn : sn;
  c = q & 1 ? sn : cn;
  s = q & 2 ? -s : s;
  c = (q + 1) & 2 ? -c : c;
}

// V values a lane and load: 8, or 4 where rot / 2 is no multiple of 8.  A unit
// is V values of one head that make V / 2 pairs of neighbours, V of the lower half with V of the upper one, or
// (rows written apart) V of the values behind rot.  The units that turn come
// first, so that few waves hold both kinds.
template <int T, bool PAIRS, int V>
__global__ __launch_bounds__(64 * ROPE_WAVES) void rope_kernel(RopeArgs a, int slices, uint32_t turn, uint32_t inv_turn,
                                                               uint32_t keep, uint32_t inv_keep) {
  typedef typename Elem<T>::type E;
  typedef E EV __attribute__((ext_vector_type(V)));
  constexpr int F = PAIRS ? V / 2 : V;  // frequencies of a unit
  __shared__ __attribute__((aligned(16))) float cosines[ROPE_WAVES][128], sines[ROPE_WAVES][128];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t item = blockIdx.x * ROPE_WAVES + wave;
  const int tok = (int)(item / (uint32_t)slices), slice = (int)(item - (uint32_t)tok * (uint32_t)slices);
  const bool some = tok < a.tokens;
  const uint32_t heads = a.hq + a.hkv, turning = heads * turn, units = turning + heads * keep;
  const int half = a.rot / 2;

  struct Unit {
    EV lo, hi;
    E* out;
    int c, on;  // (on: 1 turned, 2 carried over)
  };
  const auto load = [&](uint32_t u, Unit& x) {
    const bool turns = u < turning;
    const uint32_t n = turns ? u : u - turning, per = turns ? turn : keep;
    const uint32_t head = per == 1 ? n : __umulhi(n, turns ? inv_turn : inv_keep);
    const bool is_q = head < (uint32_t)a.hq;
    const int64_t h = is_q ? head : head - a.hq;
    x.c = (int)(n - head * per);
    x.on = !some || u >= units ? 0 : turns ? 1 : (is_q ? a.copy_q : a.copy_k) ? 2 : 0;
    const int at = turns ? x.c * V : a.rot + x.c * V;
    const E* in = (const E*)(is_q ? a.q : a.k) + tok * (is_q ? a.q_stride : a.k_stride) + h * a.d + at;
    x.out = (E*)(is_q ? a.q_out : a.k_out) + tok * (is_q ? a.q_out_stride : a.k_out_stride) + h * a.d + at;
    if (x.on) x.lo = *(const EV*)in;
    if (!PAIRS && x.on == 1) x.hi = *(const EV*)(in + half);
  };
  Unit x[ROPE_AHEAD];
  uint32_t u = (uint32_t)slice * 64 + lane;
#pragma unroll
  for (int i = 0; i < ROPE_AHEAD; ++i) load(u + (uint32_t)(i * slices * 64), x[i]);

  float f0 = 0.f, f1 = 0.f;
  if (lane < half) f0 = a.inv_freq[lane];
  if (lane + 64 < half) f1 = a.inv_freq[lane + 64];
  const int64_t p = some ? position_of(a, tok) : -1;
  if (p >= 0) {
    float s, c;
    sin_cos((double)p * (double)f0, s, c);
    cosines[wave][lane] = c * a.mscale;
    sines[wave][lane] = s * a.mscale;
    if (half > 64) {
      sin_cos((double)p * (double)f1, s, c);
      cosines[wave][lane + 64] = c * a.mscale;
      sines[wave][lane + 64] = s * a.mscale;
    }
  }
  __syncthreads();
  if (p < 0) return;

  const auto store = [&](Unit& x) {
    if (x.on == 1) {
      const float* cs = &cosines[wave][x.c * F];
      const float* sn = &sines[wave][x.c * F];
      EV lo, hi;
      if constexpr (PAIRS) {
#pragma unroll
        for (int j = 0; j < F; ++j) {
          const float r = (float)x.lo[2 * j], i = (float)x.lo[2 * j + 1];
          lo[2 * j] = (E)(r * cs[j] - i * sn[j]);
          lo[2 * j + 1] = (E)(i * cs[j] + r * sn[j]);
        }
        *(EV*)x.out = lo;
      } else {
#pragma unroll
        for (int j = 0; j < F; ++j) {
          const float r = (float)x.lo[j], i = (float)x.hi[j];
          lo[j] = (E)(r * cs[j] - i * sn[j]);
          hi[j] = (E)(i * cs[j] + r * sn[j]);
        }
        *(EV*)x.out = lo;
        *(EV*)(x.out + half) = hi;
      }
    } else if (x.on == 2) {
      *(EV*)x.out = x.lo;
    }
  };
  for (;;) {
#pragma unroll
    for (int i = 0; i < ROPE_AHEAD; ++i) store(x[i]);
    u += (uint32_t)(ROPE_AHEAD * slices * 64);
    if (u - lane >= units) return;
#pragma unroll
    for (int i = 0; i < ROPE_AHEAD; ++i) load(u + (uint32_t)(i * slices * 64), x[i]);
  }
}

template <int T, bool PAIRS, int V>
hipError_t launch(const RopeArgs& a, hipStream_t s) {
  const uint32_t turn = (uint32_t)(a.rot / (PAIRS ? V : 2 * V));
  const uint32_t keep = a.copy_q || a.copy_k ? (uint32_t)((a.d - a.rot) / V) : 0u;
  const int64_t rounds = ((int64_t)(a.hq + a.hkv) * (turn + keep) + 63) / 64;  // of a token's wave
  // a token's rounds over up to 2048 / tokens waves: slices start earlier, but
  // each computes the angles (40 heads of 128, in a graph: 64 tokens 3.3 us in five slices,
  // 5.2 in one; 512 4.7 in two, 4.9 in five, 6.0 in one; 4096 15.9 in one,
  // 17.8 in two)
  int64_t slices = 2048 / a.tokens;
  slices = slices > rounds ? rounds : slices < 1 ? 1 : slices;
  const int64_t wgs = (a.tokens * slices + ROPE_WAVES - 1) / ROPE_WAVES;
  // x / n by the high half of x * ceil(2^32 / n): exact for x below 2^19 and n in 2..64
  const auto inv = [](uint32_t n) { return n > 1 ? (uint32_t)((((uint64_t)1 << 32) + n - 1) / n) : 0u; };
  hipLaunchKernelGGL((rope_kernel<T, PAIRS, V>), dim3((unsigned)wgs), dim3(64 * ROPE_WAVES), 0, s, a, (int)slices, turn,
                     inv(turn), keep, inv(keep));
  return hipGetLastError();
}

template <int T>
hipError_t launch(const RopeArgs& a, bool pairs, hipStream_t s) {
  if (a.rot % 16 == 0) return pairs ? launch<T, true, 8>(a, s) : launch<T, false, 8>(a, s);
  return pairs ? launch<T, true, 4>(a, s) : launch<T, false, 4>(a, s);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int type, bool pairs, hipStream_t s) {
  return type == 0 ? launch<0>(a, pairs, s) : type == 1 ? launch<1>(a, pairs, s) : launch<2>(a, pairs, s);
}

}  // namespace kq
