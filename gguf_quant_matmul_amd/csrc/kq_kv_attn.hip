// kq_kv_attention: the plan of a call, the join of sums that workgroups shared,
// and the launches.  The kernels are in kq_kv_split.h and kq_kv_prompt.h.
#include "kq_kv_split.h"

namespace kq {
namespace {

// Joins the sums of rows whose keys several workgroups shared: d / 4 threads
// to a piece; a workgroup takes one row with as many of its pieces side by
// side as fit (SIDE: few rows, many pieces), or as many rows as fit.
// PREFIX: rows that also have sums over a shared prefix take them in here.
template <bool SIDE, bool PREFIX>
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
  int at = a.where[2 * row + 1];
  const bool more = PREFIX && (at & PREFIX_TOO);
  if constexpr (PREFIX) at &= ~PREFIX_TOO;
  const int64_t prow = (int64_t)tok * a.group + (row - (int64_t)tok * a.hq - (int64_t)h * a.group);
  const int shift = few ? 4 : a.many_shift, wgs = few ? a.few_wgs : a.many_wgs;
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
    if (more) m = prefix_max(a, h, prow, m);
    const float ref = m == NEG_INF ? 0.f : m;
    for (int i = lane; i < n; i += 64) l += __builtin_amdgcn_exp2f(ml[2 * piece(i)] - ref) * ml[2 * piece(i) + 1];
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) l += __shfl_xor(l, x, 64);
    if (k == 0 && more) add_prefix(a, h, prow, c, ref, l, o);
    if (k < fit) {
#pragma unroll 4
      for (int i = k; i < n; i += fit) {
        const int64_t r = piece(i);
        o += __builtin_amdgcn_exp2f(ml[2 * r] - ref) * *(const float4_t*)(sums + r * a.d + c);
      }
    }
  } else {
    for (int i = 0; i < n; ++i) m = fmaxf(m, ml[2 * piece(i)]);
    if (more) m = prefix_max(a, h, prow, m);
    const float ref = m == NEG_INF ? 0.f : m;
    if (more) add_prefix(a, h, prow, c, ref, l, o);
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

static void plan_workspace(AttnPlan& p, int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d) {
  const int64_t many = (int64_t)p.many_wgs * kv_heads * 2 * attn_prompt_rows(d), few = (int64_t)p.few_wgs * kv_heads * 32;
  p.few_at = many * (d + 2) * 4;
  p.where_at = p.few_at + few * (d + 2) * 4;
  p.bytes = many + few > 0 ? p.where_at + tokens * q_heads * 8 : 0;
}

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
  plan_workspace(p, tokens, q_heads, kv_heads, d);
  return p;
}

// A plan's 16-row tiles where their rows see at most `seen` keys, far fewer
// than the requests may hold (a window, the keys behind a prefix): the tiles are
// then of about one size, and a workgroup to each beats even shares, whose
// workgroups hold pieces of two tiles and whose sums are joined, but where few
// tiles of many steps leave CUs idle: up to half as many steps as tiles,
// 16 at least, 128 at most.  (8 kv heads of 128, groups of 4, a window of 2000:
// 32 requests 22 us against 32, 64 39 against 51; 8 requests, 1000: 13.4
// against 16.2; 4000: 31 against 21.5.)  Eight waves to each where every one
// has a CU, four where they share (64 requests, a window of 2000 and 4 sinks: 37
// us against 40).
void plan_tiles(AttnPlan& p, int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t seen) {
  const int64_t steps = (seen + STEP - 1) / STEP, tiles = p.few_tiles * kv_heads;
  const int64_t most = tiles / 2 < 16 ? 16 : tiles / 2 > 128 ? 128 : tiles / 2;
  if (p.few_wgs > 0 && steps <= most) {
    p.few_wgs = 0;
    plan_workspace(p, tokens, q_heads, kv_heads, d);
  }
  if (p.few_wgs == 0) p.more_waves = tiles <= (d > 128 ? 128 : 256) && seen > STEP * WAVES;
}

// What no plan passes whose tokens, requests, new tokens and lengths are at most
// these: fewer 16-row tiles may be shared where more are not, and a prompt's
// tiles likewise, so that a plan's own bytes go up and down.  (attn_plan and
// plan_tiles: 16-row tiles are shared above 1024 keys, prompt tiles where that
// saves 12 steps, which tiles of as few do not hold.)
int64_t plan_most(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t max_new, int64_t max_kv) {
  const int64_t most = (max_new < tokens ? max_new : tokens) * (q_heads / kv_heads), at_once = d <= 64 ? 1024 : 512;
  AttnPlan p;
  p.few_wgs = max_kv > 1024 ? (int)((at_once + kv_heads - 1) / kv_heads) : 0;
  p.many_wgs = most > 64 && kv_heads <= 64 && max_kv > 12 * STEP ? (int)(256 / kv_heads) : 0;
  plan_workspace(p, tokens, q_heads, kv_heads, d);
  return p.bytes;
}

template <bool PREFIX>
static hipError_t launch_join(const AttnArgs& a, hipStream_t s) {
  const int64_t n_rows = (int64_t)a.tokens * a.hq, fit = 256 / (a.d / 4);
  // (2048 rows of one or two pieces: 7.6 us side by side, 4.7 us packed; 128 rows of 24: packed 22 us)
  if (n_rows <= 1024) hipLaunchKernelGGL((attn_join_kernel<true, PREFIX>), dim3((unsigned)n_rows), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((attn_join_kernel<false, PREFIX>), dim3((unsigned)((n_rows + fit - 1) / fit)), dim3(256), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_attn_join(const AttnArgs& a, bool prefix, hipStream_t s) {
  return prefix ? launch_join<true>(a, s) : launch_join<false>(a, s);
}

hipError_t launch_kv_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.many_tiles > 0 && (e = launch_attn_prompt(a, p, s)) != hipSuccess) return e;
  if (p.few_tiles > 0) e = launch_split<PLAIN>(a, p, s);
  return e != hipSuccess || p.bytes == 0 ? e : launch_attn_join(a, false, s);
}

}  // namespace kq
