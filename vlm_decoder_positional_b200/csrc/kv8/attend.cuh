// The two attention kernels' launches and workspaces.
#pragma once

#include "kv8.cuh"

namespace cmr {
namespace kv8 {

size_t attend_rows_workspace(int32_t num_seqs, int64_t n_tokens, int32_t hq, int32_t hk,
                             int32_t head_dim);
cudaError_t launch_attend_rows(const AttendArgs& a, cudaStream_t stream);

}  // namespace kv8
}  // namespace cmr
