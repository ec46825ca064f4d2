// Decode attention for heads of 32 and 64 values.
#include "attn.cuh"

namespace rfp2 {

cudaError_t attn_d32(const AttnArgs &a, int sms, cudaStream_t stream) {
    return attn_by_columns<1>(a, sms, stream);
}
cudaError_t attn_d64(const AttnArgs &a, int sms, cudaStream_t stream) {
    return attn_by_columns<2>(a, sms, stream);
}

}  // namespace rfp2
