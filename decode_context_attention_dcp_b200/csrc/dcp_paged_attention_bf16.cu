// dcp_paged_attention_bf16.cu -- the paged attention kernel instances for bf16 data.
#include "dcp_paged_attention.cuh"

namespace dcp_host {

int32_t paged_attention_bf16(const dcp::AttentionArgs &a, cudaStream_t stream) {
    return paged_attention<dcp::Bf16>(a, stream);
}

}  // namespace dcp_host
