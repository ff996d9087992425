// kq_kv_attention_sinks: 16-row tiles.
#include "kq_kv_split.h"

namespace kq {

hipError_t launch_kv_attention_sinks(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.many_tiles > 0 && (e = launch_sinks_prompt(a, p, s)) != hipSuccess) return e;
  if (p.few_tiles > 0) e = launch_split<SINKS>(a, p, s);
  return e != hipSuccess || p.bytes == 0 ? e : launch_attn_join(a, false, s);
}

}  // namespace kq
