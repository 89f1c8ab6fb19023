// dcp_paged_attention_bf16.cu -- the paged attention kernel instances for bf16 data.
#include "dcp_paged_attention.cuh"

namespace dcp_host {

int32_t paged_attention_bf16(const dcp::AttentionArgs &a, cudaStream_t stream) {
    return paged_attention<dcp::Bf16>(a, stream);
}

int64_t attention_workspace_bf16(int32_t group, int32_t head_dim) {
    return attention_workspace<dcp::Bf16>(group, head_dim);
}

int32_t attention_resident_bf16(int32_t group, int32_t head_dim, int box, bool cluster, int32_t *out) {
    return attention_resident<dcp::Bf16>(group, head_dim, box, cluster, out);
}

cudaError_t attention_timeouts_bf16(unsigned long long &count, int32_t reset) {
    return attention_timeouts(count, reset);
}

}  // namespace dcp_host
