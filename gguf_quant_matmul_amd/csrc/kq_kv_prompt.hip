// kq_kv_attention: prompt tiles.
#include "kq_kv_prompt.h"

namespace kq {

int attn_prompt_rows(int64_t d) { return d <= 128 ? Prompt<4>::ROWS : Prompt<8>::ROWS; }

hipError_t launch_attn_prompt(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  return launch_prompt<PLAIN>(a, a.many_wgs > 0 ? a.many_wgs : p.many_tiles, s);
}

}  // namespace kq
