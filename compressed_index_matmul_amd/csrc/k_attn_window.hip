// attn_prompt_window: the launches of the kernels in attn_prompt_kernel.h under a
// sliding window with sinks.
//
// A workgroup walks the tiles of the sinks and then those from its first query's
// window on, so the work is that of window + sinks keys a query and of the part
// tiles at both ends of its 128 queries' windows; only tiles that an end or the
// sinks' end cuts are masked.
//
// Heads of 256 spill 6 to 8 registers.
//
// Measured: 14,919 tokens under a window of 1024 with four sinks, 32/8 heads of 128, bf16:
// 294 us, 0.76 PFLOP/s of visible pairs (the part tiles at both ends add 15 %) where the
// whole prompts take 720.  Looking for values that are not finite only after a sum
// shows one cost more than clearing them in every masked tile (301 and 322 us).
#include "attn_prompt_kernel.h"

namespace vqmm {

hipError_t launch_attn_window(const AttnView &a, const PromptPlan &p, uint16_t *out, float *lse, void *ws, hipStream_t s) {
  const PromptOut o = prompt_out(p, out, lse, ws);
  if (a.d == 64) return a.f16 ? prompt_d<64, 64, true, true, true>(a, p, o, s) : prompt_d<64, 64, false, true, true>(a, p, o, s);
  if (a.d == 128) return a.f16 ? prompt_d<128, 32, true, true, true>(a, p, o, s) : prompt_d<128, 32, false, true, true>(a, p, o, s);
  return a.f16 ? prompt_d<256, 32, true, true, true>(a, p, o, s) : prompt_d<256, 32, false, true, true>(a, p, o, s);
}

}  // namespace vqmm
