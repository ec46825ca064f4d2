// Decode attention for heads of 96 and 128 values.
#include "attn.cuh"

namespace rfp2 {

cudaError_t attn_d96(const AttnArgs &a, int sms, cudaStream_t stream) {
    return attn_by_columns<3>(a, sms, stream);
}
cudaError_t attn_d128(const AttnArgs &a, int sms, cudaStream_t stream) {
    return attn_by_columns<4>(a, sms, stream);
}

}  // namespace rfp2
