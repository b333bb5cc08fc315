// Attention for a batch whose sequences share long beginnings, on tcgen05 (cache_prompt.cuh): the
// shared part, the plan's units of 256 rows of all the group's sequences over a run of its tokens;
// and the own parts of sequences with many rows, behind the kernel of few rows.
#include <string>

#include "cache_prompt.cuh"
#include "cache_shared.cuh"
#include "csa_internal.h"

namespace csa {

int cache_prefix_launch(const csa_kv_cache& cache, const csa_kv_batch& batch,
                        const AttendCall& call, const SharedPlan& plan, bool own,
                        cudaStream_t stream, const DeviceInfo& dev, std::string& err) {
  PromptArgs a =
      prompt_args(cache, batch, call, own ? &plan.head->own : &plan.head->shared, dev);
  a.plan = plan;
  return own ? launch_prompt<kOwnPart>(a, cache, stream, dev, err)
             : launch_prompt<kSharedPart>(a, cache, stream, dev, err);
}

}  // namespace csa
