// kq_kv_attention_prefix: the plan of the prefix's part, and 16-row tiles.
#include "kq_kv_split.h"

namespace kq {

// Prompt tiles unpack a step once for 256 rows, 16-row tiles start and end
// sooner and split finer: 16-row tiles up to as much work as they do in some
// 35 us.  (8 kv heads of 128, groups of 4, one own key: 16 requests behind
// 16384 keys 27.6 us against 32.0 with prompt tiles, 24 36.2 against 34.1; 32
// behind 4096 21.3 against 24.0; 16 heads of 64, no groups: 128 requests behind
// 16384 52.7 against 48.7, 96 43.7 against 44.2.)  As many parts as there are
// CUs (prompt tiles) or workgroups at once, of 2 or 4 steps at least (128 rows
// behind 1024 keys: prompt tiles 19.6 us with 2, 22.4 with 4).
constexpr int64_t PROMPT_WGS = 256, LEAST_STEPS = 2;
PrefixPlan prefix_plan(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t prefix_len) {
  PrefixPlan f;
  const int64_t rows = tokens * (q_heads / kv_heads), steps = (prefix_len + STEP - 1) / STEP;
  f.prompt = (double)((rows + 15) / 16 * kv_heads) * (double)(steps * (d / 32)) > 45000.;
  const int tile = f.prompt ? attn_prompt_rows(d) : 16;
  f.tiles = (rows + tile - 1) / tile;
  const int64_t at_once = f.prompt ? PROMPT_WGS : d <= 64 ? 1024 : 512, least = f.prompt ? LEAST_STEPS : 4;
  int64_t n = at_once / (f.tiles * kv_heads);
  n = n > steps / least ? steps / least : n;
  n = n > MAX_SPLITS ? MAX_SPLITS : n;
  f.splits = n < 1 ? 1 : (int)n;
  f.bytes = (f.splits * tokens * q_heads * (d + 2) * 4 + 15) & ~(int64_t)15;
  return f;
}

// Fewer rows are cut into more parts, so that a batch that shrinks may have more
// sums (32 heads of 128 behind 16384 keys: 34.1 MB for 64 rows' tokens, 17.3 for
// 65).  What holds for all: parts of more than one times their tiles fill
// PROMPT_WGS prompt tiles at most (as many 16-row tiles as run at once have fewer
// rows), and there are no more of them than the steps and MAX_SPLITS give.
int64_t prefix_need(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t prefix_len, int64_t max_new,
                    int64_t max_kv) {
  const int64_t one = tokens * q_heads, steps = (prefix_len + STEP - 1) / STEP, cuts = steps / LEAST_STEPS;
  const int64_t parts = cuts < 1 ? 1 : cuts < MAX_SPLITS ? cuts : MAX_SPLITS, full = PROMPT_WGS * attn_prompt_rows(d);
  int64_t rows = one * parts < full ? one * parts : full;
  rows = rows < one ? one : rows;
  return ((rows * (d + 2) * 4 + 15) & ~(int64_t)15) + plan_most(tokens, q_heads, kv_heads, d, max_new, max_kv);
}

hipError_t launch_kv_attention_prefix(const AttnArgs& a, const AttnPlan& p, const PrefixPlan& f, hipStream_t s) {
  hipError_t e;
  if (f.prompt) {
    e = launch_flat_prompt(a, f, s);
  } else {
    AttnPlan few = p;
    few.few_tiles = f.tiles;
    few.more_waves = 0;
    e = launch_split<FLAT>(a, few, s);
  }
  if (e != hipSuccess) return e;
  if (p.many_tiles > 0 && (e = launch_tail_prompt(a, p, s)) != hipSuccess) return e;
  if (p.few_tiles > 0) e = launch_split<TAIL>(a, p, s);
  return e != hipSuccess || p.bytes == 0 ? e : launch_attn_join(a, true, s);
}

}  // namespace kq
