// Decode attention for heads of 224 and 256 values.
#include "attn.cuh"

namespace rfp2 {

cudaError_t attn_d224(const AttnArgs &a, int sms, cudaStream_t stream) {
    return attn_by_columns<7>(a, sms, stream);
}
cudaError_t attn_d256(const AttnArgs &a, int sms, cudaStream_t stream) {
    return attn_by_columns<8>(a, sms, stream);
}

}  // namespace rfp2
