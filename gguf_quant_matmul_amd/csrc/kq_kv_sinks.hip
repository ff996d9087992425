// kq_kv_attention_sinks: 16-row tiles.
#include "kq_kv_split.h"

namespace kq {

AttnPlan sinks_plan(int64_t tokens, int64_t n_seqs, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t max_new,
                    int64_t max_kv, int64_t window, int64_t sinks) {
  AttnPlan p = attn_plan(tokens, n_seqs, q_heads, kv_heads, d, max_new, max_kv, window + sinks);
  const int64_t seen = window + sinks + max_new;
  plan_tiles(p, tokens, q_heads, kv_heads, d, seen < max_kv ? seen : max_kv);
  return p;
}

hipError_t launch_kv_attention_sinks(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.many_tiles > 0 && (e = launch_sinks_prompt(a, p, s)) != hipSuccess) return e;
  if (p.few_tiles > 0) e = launch_split<SINKS>(a, p, s);
  return e != hipSuccess || p.bytes == 0 ? e : launch_attn_join(a, false, s);
}

}  // namespace kq
