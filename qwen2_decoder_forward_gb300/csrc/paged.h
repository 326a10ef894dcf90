// Launchers of the paged key / value cache operators (checked arguments).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/qwen2.h"

namespace qwen2 {
namespace paged {

struct Pool;
struct Batch;
struct Rows;
struct AttnArgs;

// paged_rows.cu
cudaError_t enqueue_write(const Pool& kv, const Batch& b, const qwen2_paged_write_opts* o, int format, int head_dim,
                          int n_head, int dtype, bool out_bf16, const Rows& q, const Rows& q_out, const Rows& k,
                          const Rows& v, cudaStream_t st);
cudaError_t enqueue_read(const Pool& kv, const Batch& b, int format, int head_dim, const int* out_start, int n_out,
                         int dtype, const Rows& k, const Rows& v, cudaStream_t st);

// paged_attn.cu
struct AttnCall {
    int format, head_dim, n_head, dtype;
    bool causal;
    float scale;
    float* lse;
    void* workspace;
};
// Workspace bytes on a device of n_sm SMs.
long long attn_workspace(const Batch& b, const Pool& kv, int head_dim, int n_head, int n_sm);
cudaError_t enqueue_attention(const Pool& kv, const Batch& b, const AttnCall& c, const Rows& q, const Rows& out,
                              int n_sm, cudaStream_t st);

// paged_attn_tc.cu
struct TcMaps {
    CUtensorMap q, k, v;
    int kv_rank[3];
};
// Packed rows per tile for a group of query heads.
int tc_tile_rows(int group);
// Tensor maps of a call; false where the strides do not allow them.
bool tc_encode(TcMaps& m, const Pool& kv, const AttnCall& c, const Rows& q, int n_rows);
// chained: launched right behind the few-rows kernel, which it may overlap.
cudaError_t enqueue_attention_tc(const TcMaps& m, const AttnArgs& a, int format, int head_dim, bool bf16, int n_sm,
                                 bool chained, cudaStream_t st);

}  // namespace paged
}  // namespace qwen2
