// The shared part of attention for a batch whose sequences share long beginnings, on tcgen05
// (cache_prompt.cuh): the plan's units, 256 rows of all the group's sequences over a run of its
// tokens, whose results the kernel of the sequences' own parts joins.
#include <string>

#include "cache_prompt.cuh"
#include "cache_shared.cuh"
#include "csa_internal.h"

namespace csa {

int cache_prefix_launch(const csa_kv_cache& cache, const csa_kv_batch& batch,
                        const AttendCall& call, const SharedPlan& plan, cudaStream_t stream,
                        const DeviceInfo& dev, std::string& err) {
  PromptArgs a = prompt_args(cache, batch, call, &plan.head->list, dev);
  a.plan = plan;
  return launch_prompt<true>(a, cache, stream, dev, err);
}

}  // namespace csa
