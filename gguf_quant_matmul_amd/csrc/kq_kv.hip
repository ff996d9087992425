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
// strip of consecutive requests; two sums over the 256 strips), so one launch
// does without communication between workgroups: a handful of kilobytes from
// L2 in place of a second launch.  The call is bound by latency (a launch,
// two dependent loads and two scans).  The workgroup then fills the table rows and
// slots of its own requests, a wave to a request; blockIdx.y shares out the
// rows of long requests.
constexpr int BT_THREADS = 256, BT_WAVES = BT_THREADS / 64;
constexpr int BT_REQS = 64;  // most requests of one workgroup

// exclusive prefix sum over the workgroup's threads; total to all threads
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* wsum, int64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t t = __shfl_up(incl, o, 64);
    if (lane >= o) incl += t;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < BT_WAVES; ++w) {
    if (w < wave) before += wsum[w];
    total += wsum[w];
  }
  __syncthreads();
  return before + incl - v;
}

struct Req {       // one request of the workgroup's range
  int64_t row, end;  // its rows
  int64_t take;      // pages taken by the requests before it
  int ctx, held, total, fit;
};

__global__ __launch_bounds__(BT_THREADS) void block_tables_kernel(
    const int32_t* __restrict__ ctx_lens, const int32_t* __restrict__ new_lens, int n_seqs, int page_shift,
    const int32_t* __restrict__ free_pages, int64_t n_free, const int32_t* __restrict__ free_head, int32_t* table,
    int64_t width, int32_t* __restrict__ slots, int64_t tokens, int32_t* __restrict__ cu, int32_t* __restrict__ lens,
    int32_t* __restrict__ head_out, uint32_t* __restrict__ status, int reqs) {
  __shared__ int64_t wsum[BT_WAVES];
  __shared__ Req req[BT_REQS];
  __shared__ uint32_t wflag[BT_WAVES];
  __shared__ int64_t wtaken[BT_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int first = blockIdx.x * reqs;  // the workgroup's requests are first .. first + reqs - 1
  const int64_t page1 = ((int64_t)1 << page_shift) - 1;
  const int64_t head = free_head[0];
  const int64_t avail = head >= 0 && head <= n_free ? n_free - head : 0;
  const int strip = (n_seqs + BT_THREADS - 1) / BT_THREADS;
  const int64_t s0 = (int64_t)tid * strip, s1 = s0 + strip < n_seqs ? s0 + strip : n_seqs;

  int64_t rows = 0, all_rows, all_need;
  for (int64_t s = s0; s < s1; ++s) rows += new_lens[s] > 0 ? new_lens[s] : 0;
  const int64_t row0 = block_scan(rows, wsum, all_rows);

  // a request's page need, with the reasons (status bits) it is refused for
  const auto need = [&](int64_t s, int64_t end, int& held, int& total, uint32_t& bad) -> int64_t {
    const int64_t c = ctx_lens[s], n = new_lens[s];
    bad = 0;
    held = total = 0;
    if (c < 0 || n < 0) { bad = 8u; return 0; }
    const int64_t h = (c + page1) >> page_shift, t = (c + n + page1) >> page_shift;
    if (t > width) bad |= 2u;
    if (n > 0 && end > tokens) bad |= 4u;
    if (c + n > 0x7FFFFFFF) bad |= 2u;
    if (bad) return 0;
    held = (int)h;
    total = (int)t;
    return t - h;
  };
  int64_t want = 0;
  for (int64_t s = s0, row = row0; s < s1; ++s) {
    const int64_t end = row + (new_lens[s] > 0 ? new_lens[s] : 0);
    int h, t;
    uint32_t bad;
    want += need(s, end, h, t, bad);
    row = end;
  }
  int64_t cum = block_scan(want, wsum, all_need);

  uint32_t flags = 0;
  int64_t taken = 0;
  for (int64_t s = s0, row = row0; s < s1; ++s) {
    const int64_t end = row + (new_lens[s] > 0 ? new_lens[s] : 0);
    int held, total;
    uint32_t bad;
    const int64_t m = need(s, end, held, total, bad);
    const bool fit = !bad && (m == 0 || cum + m <= avail);
    if (!bad && !fit) bad = 1u;
    flags |= bad;
    if (fit && m > 0) taken = cum + m;  // sums only grow: the last one that fits
    if (s >= first && s < first + reqs)
      req[s - first] = Req{row, end, cum, ctx_lens[s], held, total, (int)fit};
    cum += m;
    row = end;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      flags |= __shfl_xor(flags, o, 64);
      const int64_t t = __shfl_xor(taken, o, 64);
      taken = t > taken ? t : taken;
    }
    if (lane == 0) { wflag[wave] = flags; wtaken[wave] = taken; }
  }
  __syncthreads();
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) {
    for (int w = 1; w < BT_WAVES; ++w) {
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
// lanes a block; their maximum goes round by two DPP quad exchanges.  Bound by
// HBM: each row is read and written once, with 16- or 32-byte loads and
// stores; the kernels' 4-byte code stores of neighbouring lanes make up whole
// 64-byte lines from head size 128 on.
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

// Grid: x over (token, 8-value piece of the row), y = 0 keys, 1 values.
template <int T>
__global__ __launch_bounds__(KV_THREADS) void kv_store_kernel(const void* __restrict__ k, const void* __restrict__ v,
                                                              int64_t tokens, int heads, int d, int64_t k_stride,
                                                              int64_t v_stride, const int32_t* __restrict__ slots,
                                                              uint8_t* __restrict__ kc, uint8_t* __restrict__ vc,
                                                              int64_t n_slots, int page_shift) {
  typedef typename Elem<T>::type E;
  typedef E E8 __attribute__((ext_vector_type(8)));
  const int pieces = heads * (d / 8);
  const int64_t g = (int64_t)blockIdx.x * KV_THREADS + threadIdx.x;
  const int64_t t = g / pieces;
  if (t >= tokens) return;  // pieces is a multiple of 4: a block's four lanes leave together
  const int64_t slot = slots[t];
  if (slot < 0 || slot >= n_slots) return;
  const int piece = (int)(g - t * pieces), head = piece / (d / 8), c = piece - head * (d / 8);
  const bool val = blockIdx.y;
  const E8 raw = *(const E8*)((const E*)(val ? v : k) + t * (val ? v_stride : k_stride) + (int64_t)head * d + c * 8);
  float x[8], amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = (float)raw[i];
    x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -65504.f), 65504.f) : 0.f;
    amax = fmaxf(amax, fabsf(x[i]));
  }
  amax = quad_max(amax);
  const half_t dh = (half_t)fminf(amax / 7.f, 8188.f);
  const float D = (float)dh, inv = D > 0.f ? __builtin_amdgcn_rcpf(D) : 0.f, h = 0.5f * D;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // rint(x / D) from the reciprocal is the nearest code or its neighbour;
    // the residual x - D q is exact in float32 (D q has 15 bits and, for q
    // != 0, lies within a factor of two of x), so the comparison with D / 2
    // settles it, a tie going to the lower code; all codes of scale 0 stand
    // for 0 and code 8 is the one stored
    float q = rintf(x[i] * inv);
    const float r = __builtin_fmaf(-D, q, x[i]);
    q += r > h && D > 0.f ? 1.f : 0.f;
    q -= r <= -h && D > 0.f ? 1.f : 0.f;
    q = fminf(fmaxf(q, -8.f), 7.f);
    w |= (uint32_t)((int)q + 8) << (4 * i);
  }
  const int64_t page_rows = (int64_t)1 << page_shift, row = slot & (page_rows - 1);
  uint8_t* base = (val ? vc : kc) + ((slot >> page_shift) * heads + head) * (page_rows * (d / 2 + d / 16));
  *(uint32_t*)(base + row * (d / 2) + c * 4) = w;
  if ((c & 3) == 0) *(half_t*)(base + page_rows * (d / 2) + row * (d / 16) + (c >> 2) * 2) = dh;
}

template <int T>
__global__ __launch_bounds__(KV_THREADS) void kv_load_kernel(const uint8_t* __restrict__ kc,
                                                             const uint8_t* __restrict__ vc, int64_t n_slots,
                                                             int page_shift, int heads, int d,
                                                             const int32_t* __restrict__ slots, int64_t tokens,
                                                             void* __restrict__ k, void* __restrict__ v) {
  typedef typename Elem<T>::type E;
  typedef E E8 __attribute__((ext_vector_type(8)));
  const int pieces = heads * (d / 8);
  const int64_t g = (int64_t)blockIdx.x * KV_THREADS + threadIdx.x;
  const int64_t t = g / pieces;
  if (t >= tokens) return;
  const int64_t slot = slots[t];
  if (slot < 0 || slot >= n_slots) return;
  const int piece = (int)(g - t * pieces), head = piece / (d / 8), c = piece - head * (d / 8);
  const bool val = blockIdx.y;
  const int64_t page_rows = (int64_t)1 << page_shift, row = slot & (page_rows - 1);
  const uint8_t* base = (val ? vc : kc) + ((slot >> page_shift) * heads + head) * (page_rows * (d / 2 + d / 16));
  const uint32_t w = ld_u32(base + row * (d / 2) + c * 4);
  const float D = f16_to_f32(ld_u16(base + page_rows * (d / 2) + row * (d / 16) + (c >> 2) * 2));
  E8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (E)(D * (float)((int)((w >> (4 * i)) & 15u) - 8));  // exact in float32
  *(E8*)((E*)(val ? v : k) + t * ((int64_t)heads * d) + (int64_t)head * d + c * 8) = o;
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
                     (int)n_seqs, page_shift, free_pages, n_free, free_head, table, width, slots, tokens, cu, lens,
                     head_out, status, (int)reqs);
  return hipGetLastError();
}

hipError_t launch_kv_store(const void* k, const void* v, int type, int64_t tokens, int64_t heads, int64_t d,
                           int64_t k_stride, int64_t v_stride, const int32_t* slots, uint8_t* kc, uint8_t* vc,
                           int64_t pages, int page_shift, hipStream_t s) {
  const int64_t n = tokens * heads * (d / 8);
  const dim3 grid((unsigned)((n + KV_THREADS - 1) / KV_THREADS), 2);
  const auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(KV_THREADS), 0, s, k, v, tokens, (int)heads, (int)d, k_stride, v_stride, slots,
                       kc, vc, pages << page_shift, page_shift);
  };
  if (type == 0) go(kv_store_kernel<0>);
  else if (type == 1) go(kv_store_kernel<1>);
  else go(kv_store_kernel<2>);
  return hipGetLastError();
}

hipError_t launch_kv_load(const uint8_t* kc, const uint8_t* vc, int64_t pages, int page_shift, int64_t heads,
                          int64_t d, const int32_t* slots, int64_t tokens, void* k, void* v, int type, hipStream_t s) {
  const int64_t n = tokens * heads * (d / 8);
  const dim3 grid((unsigned)((n + KV_THREADS - 1) / KV_THREADS), 2);
  const auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, dim3(KV_THREADS), 0, s, kc, vc, pages << page_shift, page_shift, (int)heads, (int)d,
                       slots, tokens, k, v);
  };
  if (type == 0) go(kv_load_kernel<0>);
  else if (type == 1) go(kv_load_kernel<1>);
  else go(kv_load_kernel<2>);
  return hipGetLastError();
}

}  // namespace kq
