// Attention of new tokens over the paged 8-bit cache: the call for few rows per sequence and kv
// head (cache_rows.cuh) and, behind it, for prompts (cache_prompt.cuh).
#include <algorithm>
#include <string>

#include "cache_rows.cuh"
#include "csa_internal.h"

namespace csa {

size_t cache_attention_workspace_bytes(int head_size) { return rows_workspace_bytes(head_size); }

int cache_attention_launch(const csa_kv_cache& cache, const csa_kv_batch& batch,
                           const AttendCall& call, cudaStream_t stream, const DeviceInfo& dev,
                           std::string& err) {
  AttendArgs a = rows_args(cache, batch, call, call.workspace, dev);
  const int sms = std::min(dev.sm_count, kMaxSms);
  const long long most_rows = static_cast<long long>(batch.max_new) * a.group;
  const long long batch_rows = static_cast<long long>(batch.rows) * a.group;
  // Whether the batch's rows could be prompts enough, however they are shared out.
  a.prompt_blocks = static_cast<long long>(kBlocksPerSm) * sms;
  const long long sequences = std::min<long long>(batch.sequences, batch_rows / (kRowLimit + 1));
  const bool prompts = most_rows > kRowLimit &&
                       (batch_rows / 16 + sequences) * cache.heads > a.prompt_blocks;
  if (!prompts) a.prompt_blocks = 0;
  // Rows a block. 16 read the codes of 9 to 16 rows once instead of twice, but cost 8 and
  // fewer a second product for nothing and a third group of warps: 64 sequences of 16 rows
  // over 4K tokens take 69 us with 16, 81 us with 8; a batch of 4, 8 and 12 rows takes
  // 81 us with 16, 62 us with 8. So: 16 where a token alone has more than 8, or where
  // the batch's average does (prompts, which are another kernel's, left out of it).
  const bool one = most_rows <= 8 ||
                   (a.group <= 8 && (prompts || batch_rows <= 8LL * batch.sequences));
  int rc = CSA_OK;
  cudaError_t e = launch_rows<false>(a, one, cache.format, sms, dev, stream, rc, err);
  if (rc != CSA_OK) {
    err = "cache_attention_forward: " + err;
    return rc;
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    err = std::string("cache_attention_forward: launch: ") + cudaGetErrorString(e);
    return CSA_ERR_LAUNCH;
  }
  if (prompts) {
    rc = cache_prompt_launch(cache, batch, call, a.list, stream, dev, err);
    if (rc != CSA_OK) {
      err = "cache_attention_forward: " + err;
      return rc;
    }
  }
  return CSA_OK;
}

}  // namespace csa
