// kq_kv_attention_sinks: prompt tiles.
#include "kq_kv_prompt.h"

namespace kq {

hipError_t launch_sinks_prompt(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  return launch_prompt<SINKS>(a, a.many_wgs > 0 ? a.many_wgs : p.many_tiles, s);
}

}  // namespace kq
