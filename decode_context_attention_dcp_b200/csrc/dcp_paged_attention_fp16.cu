// dcp_paged_attention_fp16.cu -- the paged attention kernel instances for fp16 data.
#include "dcp_paged_attention.cuh"

namespace dcp_host {

int32_t paged_attention_fp16(const dcp::AttentionArgs &a, cudaStream_t stream) {
    return paged_attention<dcp::Fp16>(a, stream);
}

}  // namespace dcp_host
