// kq_kv_attention_prefix: prompt tiles.
#include "kq_kv_prompt.h"

namespace kq {

hipError_t launch_tail_prompt(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  return launch_prompt<TAIL>(a, a.many_wgs > 0 ? a.many_wgs : p.many_tiles, s);
}

hipError_t launch_flat_prompt(const AttnArgs& a, const PrefixPlan& f, hipStream_t s) {
  return launch_prompt<FLAT>(a, f.tiles * a.splits, s);
}

}  // namespace kq
