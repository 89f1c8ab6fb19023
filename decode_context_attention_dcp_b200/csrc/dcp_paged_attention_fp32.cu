// dcp_paged_attention_fp32.cu -- the paged attention kernel instances for fp32 data.
#include "dcp_paged_attention.cuh"

namespace dcp_host {

int32_t paged_attention_fp32(const dcp::AttentionArgs &a, cudaStream_t stream) {
    return paged_attention<dcp::Fp32>(a, stream);
}

int64_t attention_workspace_fp32(int32_t group, int32_t head_dim) {
    return attention_workspace<dcp::Fp32>(group, head_dim);
}

int32_t attention_resident_fp32(int32_t group, int32_t head_dim, int box, bool cluster, int32_t *out) {
    return attention_resident<dcp::Fp32>(group, head_dim, box, cluster, out);
}

cudaError_t attention_timeouts_fp32(unsigned long long &count, int32_t reset) {
    return attention_timeouts(count, reset);
}

}  // namespace dcp_host
