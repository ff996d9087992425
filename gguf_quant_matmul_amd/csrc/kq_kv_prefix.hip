// kq_kv_attention_prefix: the plan of the prefix's part, and 16-row tiles.
#include "kq_kv_split.h"

namespace kq {

PrefixPlan prefix_plan(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t prefix_len) {
  PrefixPlan f;
  const int64_t rows = tokens * (q_heads / kv_heads), steps = (prefix_len + STEP - 1) / STEP;
  f.prompt = rows > 32;
  const int tile = f.prompt ? attn_prompt_rows(d) : 16;
  f.tiles = (rows + tile - 1) / tile;
  const int64_t at_once = f.prompt ? 256 : d <= 64 ? 1024 : 512, least = 4;
  int64_t n = at_once / (f.tiles * kv_heads);
  n = n > steps / least ? steps / least : n;
  n = n > MAX_SPLITS ? MAX_SPLITS : n;
  f.splits = n < 1 ? 1 : (int)n;
  f.bytes = (f.splits * tokens * q_heads * (d + 2) * 4 + 15) & ~(int64_t)15;
  return f;
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
