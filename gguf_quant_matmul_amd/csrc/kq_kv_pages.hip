// Pages of the 4-bit cache shared and moved: kq_kv_fork, kq_kv_free,
// kq_kv_compact, kq_kv_copy_pages.
//
// refs[p] counts the holders of page p beyond its first.  Counts change by
// integer atomics, whose sums no order changes; what goes by order (which
// fresh page a fork takes, where a freed page goes) goes by prefix sums.
#include "kq_internal.h"

namespace kq {
namespace {

// inclusive prefix sum over a wave's lanes
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// ---- fork -------------------------------------------------------------------
//
// Fork i takes a fresh page if its length ends inside one: the one behind
// those of the forks before it.  Every workgroup sums over all forks itself
// (a thread a strip, then one scan over the strips), so that one launch does;
// then a wave copies a fork's row of page ids and counts their new holder.
// Bound by latency (a launch, two dependent loads, the scan): 8 forks of 330
// tokens 3.0 us, 256 of up to 8000 4.8.
constexpr int FORK_THREADS = 256, FORK_WAVES = FORK_THREADS / 64;
constexpr int FORK_MOST = 64;  // forks of a workgroup

struct Fork {
  int parent, child, whole, part, fit;
  uint32_t before;  // fresh pages that earlier forks ask for
};

__global__ __launch_bounds__(FORK_THREADS) void kv_fork_kernel(
    const int32_t* __restrict__ parents, const int32_t* __restrict__ children, const int32_t* __restrict__ lens, int n,
    int page_shift, int32_t* table, int n_seqs, int64_t width, int32_t* __restrict__ refs, int64_t pages,
    const int32_t* __restrict__ free_pages, int64_t n_free, const int32_t* __restrict__ free_head,
    int32_t* __restrict__ copy_src, int32_t* __restrict__ copy_dst, int32_t* __restrict__ head_out,
    uint32_t* __restrict__ status, int each) {
  __shared__ uint32_t wave_need[FORK_WAVES], wave_flags[FORK_WAVES], wave_taken[FORK_WAVES];
  __shared__ Fork fork[FORK_MOST];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int first = blockIdx.x * each;
  const int strip = (n + FORK_THREADS - 1) / FORK_THREADS;
  const int i0 = tid * strip, i1 = i0 + strip < n ? i0 + strip : n;
  const auto ask = [&](int i, Fork& f, uint32_t& bad) -> uint32_t {
    f.parent = parents[i];
    f.child = children[i];
    const int len = lens[i];
    f.whole = len >> page_shift;
    f.part = (len & ((1 << page_shift) - 1)) != 0;
    bad = len < 0 ? 8u
          : (uint32_t)f.parent >= (uint32_t)n_seqs || (uint32_t)f.child >= (uint32_t)n_seqs || f.parent == f.child ? 4u
          : (int64_t)f.whole + f.part > width ? 2u : 0u;
    return bad ? 0u : (uint32_t)f.part;
  };
  const int64_t head = free_head[0];
  uint32_t need = 0;
  for (int i = i0; i < i1; ++i) {
    Fork f;
    uint32_t bad;
    need += ask(i, f, bad);
  }
  const uint32_t incl = wave_scan(need);
  if (lane == 63) wave_need[wave] = incl;
  __syncthreads();
  uint32_t cum = incl - need;
#pragma unroll
  for (int w = 0; w < FORK_WAVES; ++w) cum += w < wave ? wave_need[w] : 0u;

  const uint32_t avail = head >= 0 && head <= n_free ? (uint32_t)(n_free - head) : 0u;
  uint32_t flags = 0, taken = 0;
  for (int i = i0; i < i1; ++i) {
    Fork f;
    uint32_t bad;
    const uint32_t m = ask(i, f, bad);
    f.before = cum;
    cum += m;
    f.fit = !bad && (m == 0 || cum <= avail);
    if (!bad && !f.fit) bad = 1u;
    flags |= bad;
    if (f.fit && m > 0) taken = cum;  // sums only grow: the last one that fits
    if (i >= first && i < first + each) fork[i - first] = f;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    const uint64_t took = __ballot(taken > 0);
    const uint32_t most = took ? __builtin_amdgcn_readlane(taken, 63 - __builtin_clzll(took)) : 0u;
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) all |= __ballot(flags >> i & 1u) ? 1u << i : 0u;
    if (lane == 0) {
      wave_flags[wave] = all;
      wave_taken[wave] = most;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) {
    flags = taken = 0;
    for (int w = 0; w < FORK_WAVES; ++w) {
      flags |= wave_flags[w];
      taken = wave_taken[w] > taken ? wave_taken[w] : taken;
    }
    head_out[0] = (int32_t)(head + taken);
    if (status) *status = flags;
  }
  for (int i = wave; i < each && first + i < n; i += FORK_WAVES) {
    const Fork f = fork[i];
    const int32_t* from = table + (int64_t)f.parent * width;
    int32_t* to = table + (int64_t)f.child * width;
    if (blockIdx.y == 0 && lane == 0) {
      int32_t src = -1, dst = -1;
      if (f.fit && f.part) {
        src = from[f.whole];
        dst = free_pages[head + f.before];
        to[f.whole] = dst;
      }
      copy_src[first + i] = src;
      copy_dst[first + i] = dst;
    }
    if (!f.fit) continue;
    for (int64_t j = (int64_t)blockIdx.y * 64 + lane; j < f.whole; j += (int64_t)gridDim.y * 64) {
      const int32_t id = from[j];
      to[j] = id;
      if (id >= 0 && id < pages) atomicAdd(refs + id, 1);
    }
  }
}

// ---- free -------------------------------------------------------------------
//
// One launch takes every given entry off its page's count; the second collects
// the pages whose count fell below 0 in the order of their ids, by one
// workgroup: where the first of them goes wants all of them counted.  Its
// threads read 32 counts each at once, and again for the second pass only
// where there are more.  Both are bound by latency.  (One launch for both,
// its one workgroup taking the entries off first: 14.2 us against 10.6 for 5
// of 64 requests.)  500 of 500 with 34000 pages take 13.9 us.
//
// A page of the free list has count 0, like one of one holder.  So that it is not
// listed twice when it is given back once more, the first launch also adds 2^28
// to the counts of the list's pages (sums know no order), and the second takes
// that off again: 0.8 to 1.0 us of a call, 5 of 64 requests 8.9 -> 9.9, 500 of
// 500 13.1 -> 13.9.
constexpr int COLLECT_THREADS = 1024, COLLECT_WAVES = COLLECT_THREADS / 64;
constexpr int LISTED_SHIFT = 28;  // (counts are below half of 2^28)

__global__ __launch_bounds__(256) void kv_release_kernel(const int32_t* __restrict__ first, const int32_t* __restrict__ last,
                                                         int n_seqs, const int32_t* __restrict__ table, int64_t width,
                                                         int32_t* __restrict__ refs, int64_t pages,
                                                         const int32_t* __restrict__ free_pages, int64_t n_free,
                                                         const int32_t* __restrict__ free_head, int row_wgs) {
  if ((int)blockIdx.x >= row_wgs) {
    const int64_t head = free_head[0], step = (int64_t)(gridDim.x - row_wgs) * gridDim.y * 256;
    const int64_t i0 = ((int64_t)(blockIdx.x - row_wgs) * gridDim.y + blockIdx.y) * 256 + threadIdx.x;
#pragma unroll 4
    for (int64_t i = head >= 0 && head <= n_free ? head + i0 : n_free; i < n_free; i += step) {
      const int32_t id = free_pages[i];
      if (id >= 0 && id < pages) atomicAdd(refs + id, 1 << LISTED_SHIFT);
    }
    return;
  }
  const int lane = threadIdx.x & 63, s = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (s >= n_seqs) return;
  int64_t j0 = first[s], j1 = last[s];
  j0 = j0 < 0 ? 0 : j0;
  j1 = j1 > width ? width : j1;
  const int32_t* row = table + (int64_t)s * width;
#pragma unroll 4
  for (int64_t j = j0 + (int64_t)blockIdx.y * 64 + lane; j < j1; j += (int64_t)gridDim.y * 64) {
    const int32_t id = row[j];
    if (id >= 0 && id < pages) atomicSub(refs + id, 1);
  }
}

__global__ __launch_bounds__(COLLECT_THREADS) void kv_collect_kernel(int32_t* __restrict__ refs, int64_t pages,
                                                                     int32_t* __restrict__ free_pages, int64_t n_free,
                                                                     const int32_t* __restrict__ free_head,
                                                                     int32_t* __restrict__ head_out,
                                                                     uint32_t* __restrict__ status) {
  constexpr int AHEAD = 32;
  __shared__ uint32_t counts[COLLECT_WAVES], overs[COLLECT_WAVES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t head = free_head[0];
  // a wave takes a run of pages
  const int64_t run = ((pages + COLLECT_WAVES - 1) / COLLECT_WAVES + 63) & ~(int64_t)63;
  const int64_t p0 = wave * run, p1 = p0 + run < pages ? p0 + run : pages;
  int32_t v[AHEAD];
  const auto load = [&](int64_t p) {
    const int left = p1 - p < 64 * AHEAD ? (int)(p1 - p) : 64 * AHEAD;  // pages from p on
    const int32_t* at = refs + p;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) v[i] = i * 64 + lane < left ? at[i * 64 + lane] : 0;
  };
  uint32_t mine = 0;  // (the same in all lanes)
  int32_t least = 0, listed_least = 0;
  for (int64_t p = p0; p < p1; p += 64 * AHEAD) {
    load(p);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      // how often the page is listed, modulo 16
      const int32_t times = (int32_t)((uint32_t)v[i] + (1u << (LISTED_SHIFT - 1))) >> LISTED_SHIFT;
      if (times != 0) {
        const int32_t count = (int32_t)((uint32_t)v[i] - ((uint32_t)times << LISTED_SHIFT));
        listed_least = count < listed_least ? count : listed_least;
        v[i] = count < 0 ? 0 : count;
        refs[p + i * 64 + lane] = v[i];
      }
      mine += __popcll(__ballot(v[i] < 0));
      least = v[i] < least ? v[i] : least;
    }
  }
  const uint32_t over = __ballot(least < -1 || listed_least < 0) ? 1u : 0u;
  if (lane == 0) {
    counts[wave] = mine;
    overs[wave] = over;
  }
  __syncthreads();
  uint32_t before = 0, total = 0, any = 0;
#pragma unroll
  for (int w = 0; w < COLLECT_WAVES; ++w) {
    before += w < wave ? counts[w] : 0u;
    total += counts[w];
    any |= overs[w];
  }
  if (threadIdx.x == 0) {
    const int64_t left = head - total;
    head_out[0] = (int32_t)(left < 0 ? 0 : left);
    if (status) *status = any | (left < 0 ? 2u : 0u);
  }
  if (mine == 0) return;
  int64_t at = head - total + before;  // place of the wave's next page
  for (int64_t p = p0; p < p1; p += 64 * AHEAD) {
    if (run > 64 * AHEAD) load(p);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const uint64_t dead = __ballot(v[i] < 0);
      if (!dead) continue;
      if (v[i] < 0) {
        const int64_t page = p + i * 64 + lane, place = at + __popcll(dead & (((uint64_t)1 << lane) - 1));
        refs[page] = 0;
        if (place >= 0 && place < n_free) free_pages[place] = (int32_t)page;
      }
      at += __popcll(dead);
    }
  }
}

// ---- compact ----------------------------------------------------------------
//
// A bit a page in LDS says which are free.  With c held pages in all, the free
// pages below c (the first free ones) are the holes, the held ones from c on
// the movers; as many of each.  A page's place among either is its rank among
// the free pages: a wave takes a run of pages, 64 at a time, and counts on from
// the free pages of the waves before.  Tables, counts and the free list are
// renumbered by the same workgroup up to 8 elements a thread, which saves a
// launch (500 pages and as many entries 3.9 us a call against 6.1, 5000 8.7
// against 7.1), else by a second launch.
constexpr int COMPACT_THREADS = 1024, COMPACT_WAVES = COMPACT_THREADS / 64;

// What table entries, counts and the free list are read from and written to.
struct Renumber {
  const int32_t *table, *refs, *free_pages;
  int32_t *table_out, *refs_out, *free_out;
  int64_t n_entries, n_free;
  int pages;
};
// Elements t0, t0 + step, .. by the new ids; the first `head` of the free list
// stay.
__device__ __forceinline__ void renumber(const Renumber& r, const int32_t* remap, int64_t head, int64_t t0, int64_t step) {
  const int64_t held = r.pages - (r.n_free - head);
  for (int64_t i = t0; i < r.n_entries; i += step) {
    const int32_t id = r.table[i];
    r.table_out[i] = id >= 0 && id < r.pages ? remap[id] : -1;
  }
  for (int64_t p = t0; p < r.pages; p += step) {
    // (a hole's count is written with that of the page that moves into it)
    const int32_t to = remap[p], count = r.refs[p];
    if (to >= 0) r.refs_out[to] = count;
    if (p >= held) r.refs_out[p] = 0;
  }
  for (int64_t i = t0; i < r.n_free; i += step) r.free_out[i] = i < head ? r.free_pages[i] : (int32_t)(held + i - head);
}

template <bool ALL>
__global__ __launch_bounds__(COMPACT_THREADS) void kv_compact_kernel(Renumber r, const int32_t* free_head, int32_t* remap,
                                                                     int32_t* copy_src, int32_t* copy_dst, int64_t n_copy,
                                                                     int32_t* head_out, uint32_t* status) {
  const int32_t* free_pages = r.free_pages;
  const int64_t n_free = r.n_free;
  const int pages = r.pages;
  extern __shared__ uint64_t bits[];  // 64 pages each
  __shared__ uint32_t frees[COMPACT_WAVES], holes[COMPACT_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int words = (pages + 63) / 64, run = (words + COMPACT_WAVES - 1) / COMPACT_WAVES;
  for (int i = tid; i < words; i += COMPACT_THREADS) bits[i] = 0;
  const int64_t head = free_head[0];
  __syncthreads();
#pragma unroll 4
  for (int64_t i = head >= 0 && head <= n_free ? head + tid : n_free; i < n_free; i += COMPACT_THREADS) {
    const int32_t id = free_pages[i];
    if (id >= 0 && id < pages) atomicOr((uint32_t*)bits + (id >> 5), 1u << (id & 31));
  }
  __syncthreads();
  const int w0 = wave * run, w1 = w0 + run < words ? w0 + run : words;  // the wave's words
  uint32_t mine = 0;
  for (int w = w0 + lane; w < w1; w += 64) mine += __popcll(bits[w]);
  mine = __builtin_amdgcn_readlane(wave_scan(mine), 63);
  if (lane == 0) frees[wave] = mine;
  __syncthreads();
  uint32_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < COMPACT_WAVES; ++w) {
    before += w < wave ? frees[w] : 0u;
    total += frees[w];
  }
  const int held = pages - (int)total;
  mine = 0;
  for (int w = w0 + lane; w < w1 && w * 64 < held; w += 64)
    mine += __popcll(held - w * 64 < 64 ? bits[w] & (((uint64_t)1 << (held - w * 64)) - 1) : bits[w]);
  mine = __builtin_amdgcn_readlane(wave_scan(mine), 63);
  if (lane == 0) holes[wave] = mine;
  __syncthreads();
  uint32_t moves = 0;
#pragma unroll
  for (int w = 0; w < COMPACT_WAVES; ++w) moves += holes[w];
  for (int w = w0; w < w1; ++w) {
    const uint64_t word = bits[w];
    const int id = w * 64 + lane, n = (int)before + __popcll(word & (((uint64_t)1 << lane) - 1));  // free pages before
    before += __popcll(word);
    if (id >= pages) continue;
    const bool is_free = word >> lane & 1u;
    if (is_free || id < held) remap[id] = is_free ? -1 : id;
    if (is_free != (id < held)) continue;
    // a hole, or a mover behind held - moves pages that stay
    const int at = is_free ? n : id - n - (held - (int)moves);
    if (at < n_copy) (is_free ? copy_dst : copy_src)[at] = id;
  }
  __threadfence_block();
  __syncthreads();
  for (int64_t i = tid; i < n_copy; i += COMPACT_THREADS) {
    if (i < (int64_t)moves) remap[copy_src[i]] = copy_dst[i];
    else copy_src[i] = copy_dst[i] = -1;
  }
  if (tid == 0) {
    if (status) *status = head != n_free - total ? 1u : 0u;
    head_out[0] = (int32_t)(n_free - total);
  }
  if constexpr (ALL) {
    __threadfence_block();
    __syncthreads();
    renumber(r, remap, n_free - total, tid, COMPACT_THREADS);
  }
}

__global__ __launch_bounds__(256) void kv_renumber_kernel(Renumber r, const int32_t* __restrict__ remap,
                                                          const int32_t* __restrict__ free_head) {
  renumber(r, remap, free_head[0], (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// ---- copy -------------------------------------------------------------------
//
// A workgroup copies pieces of 16 KB of one cache, all of a thread's loads
// before its stores.  Bound by HBM: 2660 pages of 36 KB a cache, 393 MB, 81 us,
// 4.8 TB/s, what a large copy reaches.
constexpr int COPY_THREADS = 256, COPY_AHEAD = 4;
constexpr int COPY_PIECE = COPY_THREADS * COPY_AHEAD * 16;

__global__ __launch_bounds__(COPY_THREADS) void kv_copy_pages_kernel(const int32_t* __restrict__ src,
                                                                     const int32_t* __restrict__ dst, int64_t n,
                                                                     uint8_t* kc, uint8_t* vc, int64_t pages,
                                                                     int64_t bytes, int pieces) {
  const int64_t work = n * 2 * pieces;
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
    const int64_t pair = w / (2 * pieces);
    const int rest = (int)(w - pair * (2 * pieces)), piece = rest >> 1;
    const int64_t from = src[pair], to = dst[pair];
    if (from < 0 || from >= pages || to < 0 || to >= pages || from == to) continue;
    uint8_t* cache = rest & 1 ? vc : kc;
    const uint8_t* s = cache + from * bytes;
    uint8_t* d = cache + to * bytes;
    const int64_t at = (int64_t)piece * COPY_PIECE + threadIdx.x * 16;
    u32x4 v[COPY_AHEAD];
#pragma unroll
    for (int i = 0; i < COPY_AHEAD; ++i)
      if (at + i * COPY_THREADS * 16 < bytes) v[i] = *(const u32x4*)(s + at + i * COPY_THREADS * 16);
#pragma unroll
    for (int i = 0; i < COPY_AHEAD; ++i)
      if (at + i * COPY_THREADS * 16 < bytes) *(u32x4*)(d + at + i * COPY_THREADS * 16) = v[i];
  }
}

}  // namespace

hipError_t launch_kv_fork(const int32_t* parents, const int32_t* children, const int32_t* lens, int64_t n, int page_shift,
                          int32_t* table, int64_t n_seqs, int64_t width, int32_t* refs, int64_t pages,
                          const int32_t* free_pages, int64_t n_free, const int32_t* free_head, int32_t* copy_src,
                          int32_t* copy_dst, int32_t* head_out, uint32_t* status, hipStream_t s) {
  // four forks to a workgroup (one a wave); above 1024 more of them, so that
  // the repeated sums stay small beside the rows (256 forks 3.4 us with 4 to a
  // workgroup, 5.8 with 16; 4096 46 with 4, 19 with 16, 28 with 64; 16384 340
  // with 16, 107 with 64)
  int64_t each = n / 256;
  each = each < 4 ? 4 : each > FORK_MOST ? FORK_MOST : each;
  const int64_t gx = n > 0 ? (n + each - 1) / each : 1;
  // long rows are shared out: 512 entries to a wave (8 forks of 6250 entries
  // 7.5 us in eight parts, 8.8 in seven, 39 in one)
  int64_t gy = (width + 511) / 512;
  gy = gy < 1 ? 1 : gy > 64 ? 64 : gy;
  hipLaunchKernelGGL(kv_fork_kernel, dim3((unsigned)gx, (unsigned)gy), dim3(FORK_THREADS), 0, s, parents, children, lens,
                     (int)n, page_shift, table, (int)n_seqs, width, refs, pages, free_pages, n_free, free_head, copy_src,
                     copy_dst, head_out, status, (int)each);
  return hipGetLastError();
}

hipError_t launch_kv_free(const int32_t* first, const int32_t* last, int64_t n_seqs, const int32_t* table, int64_t width,
                          int32_t* refs, int64_t pages, int32_t* free_pages, int64_t n_free, const int32_t* free_head,
                          int32_t* head_out, uint32_t* status, hipStream_t s) {
  if (n_seqs > 0 && width > 0) {
    // 256 entries of a row to a wave (8 requests of 6250 entries 11.2 us in
    // thirteen parts, 12.7 in eight, 44 in one)
    int64_t gy = (width + 255) / 256;
    gy = gy > 64 ? 64 : gy;
    const int64_t rows = (n_seqs + 3) / 4;
    // the list's pages a thread to each, by up to 1024 workgroups
    const int64_t wgs = (n_free + 255) / 256, lists = ((wgs < 1024 ? wgs : 1024) + gy - 1) / gy;
    hipLaunchKernelGGL(kv_release_kernel, dim3((unsigned)(rows + lists), (unsigned)gy), dim3(256), 0, s, first, last,
                       (int)n_seqs, table, width, refs, pages, free_pages, n_free, free_head, (int)rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kv_collect_kernel, dim3(1), dim3(COLLECT_THREADS), 0, s, refs, pages, free_pages, n_free, free_head,
                     head_out, status);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const int32_t* free_pages, int64_t n_free, const int32_t* free_head, const int32_t* table,
                             int64_t n_entries, const int32_t* refs, int64_t pages, int32_t* table_out, int32_t* refs_out,
                             int32_t* free_out, int32_t* remap, int32_t* copy_src, int32_t* copy_dst, int64_t n_copy,
                             int32_t* head_out, uint32_t* status, hipStream_t s) {
  const Renumber r = {table, refs, free_pages, table_out, refs_out, free_out, n_entries, n_free, (int)pages};
  const bool all = n_entries + pages + n_free <= 8 * COMPACT_THREADS;
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(1), dim3(COMPACT_THREADS), (size_t)((pages + 63) / 64 * 8), s, r, free_head, remap,
                       copy_src, copy_dst, n_copy, head_out, status);
  };
  if (all) go(kv_compact_kernel<true>);
  else go(kv_compact_kernel<false>);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || all) return e;
  int64_t most = n_entries > pages ? n_entries : pages;
  most = n_free > most ? n_free : most;
  const int64_t wgs = (most + 255) / 256;
  hipLaunchKernelGGL(kv_renumber_kernel, dim3((unsigned)(wgs < 2048 ? wgs : 2048)), dim3(256), 0, s, r, remap, head_out);
  return hipGetLastError();
}

hipError_t launch_kv_copy_pages(const int32_t* src, const int32_t* dst, int64_t n, uint8_t* kc, uint8_t* vc, int64_t pages,
                                int64_t bytes, hipStream_t s) {
  const int64_t pieces = (bytes + COPY_PIECE - 1) / COPY_PIECE, work = n * 2 * pieces;
  hipLaunchKernelGGL(kv_copy_pages_kernel, dim3((unsigned)(work < 65536 ? work : 65536)), dim3(COPY_THREADS), 0, s, src, dst,
                     n, kc, vc, pages, bytes, (int)pieces);
  return hipGetLastError();
}

}  // namespace kq
