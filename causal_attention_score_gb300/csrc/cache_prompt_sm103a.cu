// Attention of many new tokens per sequence over the paged 8-bit cache, on tcgen05
// (cache_prompt.cuh): behind the kernel for few rows, which leaves it the list.
#include <string>

#include "cache_prompt.cuh"
#include "csa_internal.h"

namespace csa {

int cache_prompt_launch(const csa_kv_cache& cache, const csa_kv_batch& batch,
                        const AttendCall& call, PromptList* list, cudaStream_t stream,
                        const DeviceInfo& dev, std::string& err) {
  return launch_prompt<kWhole>(prompt_args(cache, batch, call, list, dev), cache, stream, dev, err);
}

}  // namespace csa
