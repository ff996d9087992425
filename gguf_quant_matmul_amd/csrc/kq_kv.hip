// Key/value cache in 4 bits: block tables and slot maps (kq_block_tables),
// rows encoded into slots (kq_kv_store) and decoded from slots (kq_kv_load).
// The cache layout is stated in kq.h.
#include "kq_internal.h"

#pragma clang fp contract(off)

namespace kq {
namespace {

// ---- block tables -----------------------------------------------------------
//
// With p(x) = ceil(x / page), request s needs p(ctx + new) - p(ctx) pages;
// its rows start at the sum of new over the requests before it and its pages
// in the free list at the sum of their needs.  Both sums are prefix sums over
// all requests, and every workgroup computes them for itself (thread i takes a
// strip of consecutive requests, then one scan over the 256 strips), so one
// launch does without communication between workgroups: a handful of
// kilobytes from L2 in place of a second launch.  The call is bound by latency
// (a launch, two dependent loads and the scan): 3.7 us on the GPU for 64
// requests, 4.3 for 500 mixed ones.  The sums are 32-bit and
// saturate: all that is asked of one past its bound (rows, free pages; both
// below 2^31) is that it is past.  A request whose rows pass the buffer takes
// no pages, yet its need may be counted: its rows end behind the bound, so do
// those of all later requests that add any, and only those need pages.  The
// workgroup then fills the table rows and slots of its own requests, a wave to
// a request; blockIdx.y shares out the rows of long requests.
constexpr int BT_THREADS = 256, BT_WAVES = BT_THREADS / 64;
constexpr int BT_REQS = 64;  // most requests of one workgroup

__device__ __forceinline__ uint32_t add_sat(uint32_t x, uint32_t y) { return __builtin_elementwise_add_sat(x, y); }

// inclusive saturating prefix sum over a wave's lanes: within rows of 16 by
// row shifts, then the last lane of a row, and of the first half, broadcast
__device__ __forceinline__ uint32_t wave_scan_sat(uint32_t v) {
  v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));  // row_shr:1
  v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
  v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
  v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
  v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));  // row_bcast:15 into rows 1 and 3
  v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));  // row_bcast:31 into rows 2 and 3
  return v;
}

struct Req {             // one request of the workgroup's range
  uint32_t row, end;     // its rows
  uint32_t take;         // pages taken by the requests before it
  int ctx, held, total, fit;
};

__global__ __launch_bounds__(BT_THREADS) void block_tables_kernel(
    const int32_t* __restrict__ ctx_lens, const int32_t* __restrict__ new_lens, int n_seqs, int page_shift,
    const int32_t* __restrict__ free_pages, int64_t n_free, const int32_t* __restrict__ free_head, int32_t* table,
    int64_t width, int32_t* __restrict__ slots, uint32_t tokens, int32_t* __restrict__ cu, int32_t* __restrict__ lens,
    int32_t* __restrict__ head_out, uint32_t* __restrict__ status, int reqs) {
  __shared__ uint32_t wrows[BT_WAVES], wneed[BT_WAVES];
  __shared__ Req req[BT_REQS];
  __shared__ uint32_t wflag[BT_WAVES], wtaken[BT_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int first = blockIdx.x * reqs;  // the workgroup's requests are first .. first + reqs - 1
  const int64_t page1 = ((int64_t)1 << page_shift) - 1;
  const int strip = (n_seqs + BT_THREADS - 1) / BT_THREADS;
  const int s0 = tid * strip, s1 = s0 + strip < n_seqs ? s0 + strip : n_seqs;

  // rows and pages of a request; reasons (status bits) to refuse it but for
  // the bounds on the sums
  const auto want = [&](int64_t c, int64_t n, int& held, int& total, uint32_t& bad) -> uint32_t {
    bad = 0;
    held = total = 0;
    if (c < 0 || n < 0) { bad = 8u; return 0; }
    const int64_t h = (c + page1) >> page_shift, t = (c + n + page1) >> page_shift;
    if (t > width || c + n > 0x7FFFFFFF) { bad = 2u; return 0; }
    held = (int)h;
    total = (int)t;
    return (uint32_t)(t - h);
  };
  const int64_t head = free_head[0];
  uint32_t rows = 0, need = 0;
  for (int s = s0; s < s1; ++s) {
    const int c = ctx_lens[s], n = new_lens[s];
    int held, total;
    uint32_t bad;
    need = add_sat(need, want(c, n, held, total, bad));
    rows = add_sat(rows, n > 0 ? n : 0);
  }
  const uint32_t rows_incl = wave_scan_sat(rows), need_incl = wave_scan_sat(need);
  if (lane == 63) { wrows[wave] = rows_incl; wneed[wave] = need_incl; }
  __syncthreads();
  // sums before the strip: the waves before, then the lanes before
  uint32_t row = 0, cum = 0, all_rows = 0;
#pragma unroll
  for (int w = 0; w < BT_WAVES; ++w) {
    if (w < wave) { row = add_sat(row, wrows[w]); cum = add_sat(cum, wneed[w]); }
    all_rows = add_sat(all_rows, wrows[w]);
  }
  const uint32_t lane_rows = __shfl_up(rows_incl, 1, 64), lane_need = __shfl_up(need_incl, 1, 64);
  if (lane > 0) { row = add_sat(row, lane_rows); cum = add_sat(cum, lane_need); }

  const uint32_t avail = head >= 0 && head <= n_free ? (uint32_t)(n_free - head) : 0u;
  uint32_t flags = 0, taken = 0;
  for (int s = s0; s < s1; ++s) {
    const int c = ctx_lens[s], n = new_lens[s];
    const uint32_t end = add_sat(row, n > 0 ? n : 0);
    int held, total;
    uint32_t bad;
    const uint32_t m = want(c, n, held, total, bad), sum = add_sat(cum, m);
    if (n > 0 && end > tokens && !(bad & 8u)) bad |= 4u;
    const bool fit = !bad && (m == 0 || sum <= avail);
    if (!bad && !fit) bad = 1u;
    flags |= bad;
    if (fit && m > 0) taken = sum;  // sums only grow: the last one that fits
    if (s >= first && s < first + reqs) req[s - first] = Req{row, end, cum, c, held, total, (int)fit};
    cum = sum;
    row = end;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    // (sums only grow, so the last lane that took pages has the wave's count)
    const uint64_t took = __ballot(taken > 0);
    const uint32_t most = took ? __builtin_amdgcn_readlane(taken, 63 - __builtin_clzll(took)) : 0u;
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) all |= __ballot(flags >> i & 1u) ? 1u << i : 0u;
    if (lane == 0) { wflag[wave] = all; wtaken[wave] = most; }
  }
  __syncthreads();
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) {
    for (int w = 0; w < BT_WAVES; ++w) {
      flags |= wflag[w];
      taken = wtaken[w] > taken ? wtaken[w] : taken;
    }
    head_out[0] = (int32_t)(head + taken);
    if (status) *status = flags;
    cu[0] = 0;
  }
  if (blockIdx.y == 0) {
    for (int i = tid; i < reqs && first + i < n_seqs; i += BT_THREADS) {
      const Req& r = req[i];
      cu[first + i + 1] = (int32_t)(r.end < tokens ? r.end : tokens);
      lens[first + i] = r.fit ? (int32_t)(r.ctx + (r.end - r.row)) : 0;
    }
  }
  for (int i = wave; i < reqs && first + i < n_seqs; i += BT_WAVES) {
    const Req r = req[i];
    int32_t* trow = table + (int64_t)(first + i) * width;
    const int32_t* fresh = free_pages + head + r.take - r.held;  // id of new page j: fresh[j]
    if (r.fit)
      for (int64_t j = r.held + (int64_t)blockIdx.y * 64 + lane; j < r.total; j += (int64_t)gridDim.y * 64)
        trow[j] = fresh[j];
    const int64_t end = r.end < tokens ? r.end : tokens;
    for (int64_t t = r.row + (int64_t)blockIdx.y * 64 + lane; t < end; t += (int64_t)gridDim.y * 64) {
      int64_t slot = -1;
      if (r.fit) {
        const int64_t pos = r.ctx + (t - r.row), j = pos >> page_shift;
        const int64_t id = j < r.held ? trow[j] : fresh[j];
        slot = (id << page_shift) + (pos & page1);
        if (id < 0 || slot > 0x7FFFFFFF) slot = -1;
      }
      slots[t] = (int32_t)slot;
    }
  }
  // rows behind the last request
  const int64_t wgs = (int64_t)gridDim.x * gridDim.y, wg = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  for (int64_t t = all_rows + wg * BT_THREADS + tid; t < tokens; t += wgs * BT_THREADS) slots[t] = -1;
}

// ---- cache rows -------------------------------------------------------------
//
// A thread takes 8 consecutive values (one dword of codes), four neighbouring
// lanes a block; their maximum goes round by two DPP quad exchanges.  Long
// calls are bound by HBM, the store also by the vector units (82% busy while it
// works): each row is read and written once, with 16- or 32-byte loads and
// stores; the kernels' 4-byte code stores of neighbouring
// lanes make up whole 64-byte lines from head size 128 on.  A decode step's
// are bound by the launch and two dependent loads.  Measured, store and load
// together: 8192 bfloat16 rows of 8 heads, d = 128, 20.6 us, 3.7 TB/s; 64 rows
// 8.6 us.  Apart and on rows not in cache: 13.1 and 12.5 us, float32 ones 19.7
// and 23.0 us, 3.9 and 3.3 TB/s.
constexpr int KV_THREADS = 256;
template <int T> struct Elem;
template <> struct Elem<0> { typedef float type; };
template <> struct Elem<1> { typedef half_t type; };
template <> struct Elem<2> { typedef __bf16 type; };

__device__ __forceinline__ float quad_max(float v) {
  const auto mov = [](float x, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v = fmaxf(v, mov(v, std::integral_constant<int, 0xB1>{}));  // quad_perm [1, 0, 3, 2]
  return fmaxf(v, mov(v, std::integral_constant<int, 0x4E>{}));  // quad_perm [2, 3, 0, 1]
}

// x / n by the high half of x * ceil(2^32 / n): exact here, where n <= 32 and
// x (a piece of a row) is below 2^17.
uint32_t inv_of(int64_t n) { return (uint32_t)((((uint64_t)1 << 32) + n - 1) / n); }

// Eight values of a row as codes (nibble i: value i), and their block's scale.
// FULL: float32 rows; else float16 or bfloat16.
template <bool FULL, typename E8>
__device__ __forceinline__ uint32_t encode8(E8 raw, half_t& scale) {
  float x[8], amax = 0.f, odd = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = (float)raw[i];
    amax = fmaxf(amax, fabsf(x[i]));
    odd = __builtin_fmaf(x[i], 0.f, odd);  // NaN for a NaN (or an infinity)
  }
  if (__any(!(amax <= 65504.f) || odd != odd)) {  // rare: values to be brought into range
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -65504.f), 65504.f) : 0.f;
      amax = fmaxf(amax, fabsf(x[i]));
    }
  }
  amax = quad_max(amax);
  scale = (half_t)fminf(amax / 7.f, 8188.f);
  const float D = (float)scale, inv = D > 0.f ? __builtin_amdgcn_rcpf(D) : 0.f;
  float q[8];
  if constexpr (FULL) {
    // of scale 0 every residual is below the half step, and code 8 is stored
    const float h = D > 0.f ? 0.5f * D : __builtin_inff();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // rint(x / D) from the reciprocal is the nearest code or its neighbour;
      // the residual x - D q is exact in float32 (D q has 15 bits and, for q
      // != 0, lies within a factor of two of x), so the comparison with D / 2
      // settles it, a tie going to the lower code
      q[i] = rintf(x[i] * inv);
      const float r = __builtin_fmaf(-D, q[i], x[i]);
      q[i] += r > h ? 1.f : 0.f;
      q[i] -= r <= -h ? 1.f : 0.f;
    }
  } else {
    // x - (k + 1/2) D is a multiple of 2^-12 of D's power of two where x has
    // 11 bits or fewer, so x / D is a tie or 2^-12 and more away from one; the
    // reciprocal's product is off by less than 2^-19.  Ties, and nothing else,
    // lie within 2^-14 of k + 1/2, and the ceiling below takes them down.
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __builtin_ceilf(__builtin_fmaf(x[i], inv, -0.50006103515625f));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = __builtin_amdgcn_fmed3f(q[i], -8.f, 7.f);
  // four codes to 16 bits in float32, exactly
  const auto four = [](float a, float b, float c, float d) {
    return (uint32_t)__builtin_fmaf(d, 4096.f, __builtin_fmaf(c, 256.f, __builtin_fmaf(b, 16.f, a + 34952.f)));
  };
  return four(q[0], q[1], q[2], q[3]) | four(q[4], q[5], q[6], q[7]) << 16;
}

// A thread takes the same piece of the token's key and of its value: both
// loads are out before the slot is known.
template <int T>
__global__ __launch_bounds__(KV_THREADS) void kv_store_kernel(const void* __restrict__ k, const void* __restrict__ v,
                                                              int64_t tokens, int heads, int d, int64_t k_stride,
                                                              int64_t v_stride, const int32_t* __restrict__ slots,
                                                              uint8_t* __restrict__ kc, uint8_t* __restrict__ vc,
                                                              int64_t n_slots, int page_shift, uint32_t inv_per) {
  typedef typename Elem<T>::type E;
  typedef E E8 __attribute__((ext_vector_type(8)));
  const uint32_t per = d / 8, pieces = heads * per;  // of a head, of a row
  const uint32_t g = blockIdx.x * KV_THREADS + threadIdx.x, t = g / pieces;  // (fewer than 2^31 pieces a call)
  if (t >= tokens) return;  // pieces is a multiple of 4: a block's four lanes leave together
  const uint32_t piece = g - t * pieces, head = __umulhi(piece, inv_per), c = piece - head * per;
  const E8 kr = *(const E8*)((const E*)k + t * k_stride + (int64_t)piece * 8);
  const E8 vr = *(const E8*)((const E*)v + t * v_stride + (int64_t)piece * 8);
  const int64_t slot = slots[t];
  if (slot < 0 || slot >= n_slots) return;
  half_t ks, vs;
  const uint32_t kw = encode8<T == 0>(kr, ks), vw = encode8<T == 0>(vr, vs);
  const int64_t page_rows = (int64_t)1 << page_shift, row = slot & (page_rows - 1);
  const int64_t base = ((slot >> page_shift) * heads + head) * (page_rows * (d / 2 + d / 16));
  const int64_t at = base + row * (d / 2) + c * 4, sat = base + page_rows * (d / 2) + row * (d / 16) + (c >> 2) * 2;
  *(uint32_t*)(kc + at) = kw;
  *(uint32_t*)(vc + at) = vw;
  if ((c & 3) == 0) {
    *(half_t*)(kc + sat) = ks;
    *(half_t*)(vc + sat) = vs;
  }
}

template <int T>
__global__ __launch_bounds__(KV_THREADS) void kv_load_kernel(const uint8_t* __restrict__ kc,
                                                             const uint8_t* __restrict__ vc, int64_t n_slots,
                                                             int page_shift, int heads, int d,
                                                             const int32_t* __restrict__ slots, int64_t tokens,
                                                             void* __restrict__ k, void* __restrict__ v,
                                                             uint32_t inv_per) {
  typedef typename Elem<T>::type E;
  typedef E E8 __attribute__((ext_vector_type(8)));
  const uint32_t per = d / 8, pieces = heads * per;  // of a head, of a row
  const uint32_t g = blockIdx.x * KV_THREADS + threadIdx.x, t = g / pieces;  // (fewer than 2^31 pieces a call)
  if (t >= tokens) return;
  const int64_t slot = slots[t];
  if (slot < 0 || slot >= n_slots) return;
  const uint32_t piece = g - t * pieces, head = __umulhi(piece, inv_per), c = piece - head * per;
  const int64_t page_rows = (int64_t)1 << page_shift, row = slot & (page_rows - 1);
  const int64_t base = ((slot >> page_shift) * heads + head) * (page_rows * (d / 2 + d / 16));
  const int64_t at = base + row * (d / 2) + c * 4, sat = base + page_rows * (d / 2) + row * (d / 16) + (c >> 2) * 2;
  const uint32_t kw = ld_u32(kc + at), vw = ld_u32(vc + at), ks = ld_u16(kc + sat), vs = ld_u16(vc + sat);
  const auto decode = [](uint32_t w, uint32_t s) {
    const float D = f16_to_f32(s);
    E8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (E)(D * (float)((int)((w >> (4 * i)) & 15u) - 8));  // exact in float32
    return o;
  };
  *(E8*)((E*)k + (int64_t)g * 8) = decode(kw, ks);  // rows are dense here
  *(E8*)((E*)v + (int64_t)g * 8) = decode(vw, vs);
}

}  // namespace

hipError_t launch_block_tables(const int32_t* ctx, const int32_t* nw, int64_t n_seqs, int page_shift,
                               const int32_t* free_pages, int64_t n_free, const int32_t* free_head, int32_t* table,
                               int64_t width, int32_t* slots, int64_t tokens, int32_t* cu, int32_t* lens,
                               int32_t* head_out, uint32_t* status, hipStream_t s) {
  // four requests to a workgroup (one a wave); above 4096 requests more of
  // them, so that the repeated prefix sums stay small beside the filling
  int64_t reqs = (n_seqs + 1023) / 1024;
  reqs = reqs < 4 ? 4 : reqs > BT_REQS ? BT_REQS : reqs;
  int64_t gx = (n_seqs + reqs - 1) / reqs;
  gx = gx < 1 ? 1 : gx;
  // about 512 rows of the average request to a wave
  const int64_t per = n_seqs > 0 ? tokens / n_seqs : tokens;
  int64_t gy = (per + 511) / 512;
  gy = gy < 1 ? 1 : gy > 64 ? 64 : gy;
  hipLaunchKernelGGL(block_tables_kernel, dim3((unsigned)gx, (unsigned)gy), dim3(BT_THREADS), 0, s, ctx, nw,
                     (int)n_seqs, page_shift, free_pages, n_free, free_head, table, width, slots,
                     (uint32_t)tokens, cu, lens, head_out, status, (int)reqs);
  return hipGetLastError();
}

hipError_t launch_kv_store(const void* k, const void* v, int type, int64_t tokens, int64_t heads, int64_t d,
                           int64_t k_stride, int64_t v_stride, const int32_t* slots, uint8_t* kc, uint8_t* vc,
                           int64_t pages, int page_shift, hipStream_t s) {
  const int64_t n = tokens * heads * (d / 8);
  const dim3 grid((unsigned)((n + KV_THREADS - 1) / KV_THREADS));
  const auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(KV_THREADS), 0, s, k, v, tokens, (int)heads, (int)d, k_stride, v_stride, slots,
                       kc, vc, pages << page_shift, page_shift, inv_of(d / 8));
  };
  if (type == 0) go(kv_store_kernel<0>);
  else if (type == 1) go(kv_store_kernel<1>);
  else go(kv_store_kernel<2>);
  return hipGetLastError();
}

hipError_t launch_kv_load(const uint8_t* kc, const uint8_t* vc, int64_t pages, int page_shift, int64_t heads,
                          int64_t d, const int32_t* slots, int64_t tokens, void* k, void* v, int type, hipStream_t s) {
  const int64_t n = tokens * heads * (d / 8);
  const dim3 grid((unsigned)((n + KV_THREADS - 1) / KV_THREADS));
  const auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(KV_THREADS), 0, s, kc, vc, pages << page_shift, page_shift, (int)heads, (int)d,
                       slots, tokens, k, v, inv_of(d / 8));
  };
  if (type == 0) go(kv_load_kernel<0>);
  else if (type == 1) go(kv_load_kernel<1>);
  else go(kv_load_kernel<2>);
  return hipGetLastError();
}

}  // namespace kq
