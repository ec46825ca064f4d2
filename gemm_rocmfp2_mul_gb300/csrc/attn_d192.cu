// Decode attention for heads of 160 and 192 values.
#include "attn.cuh"

namespace rfp2 {

cudaError_t attn_d160(const AttnArgs &a, int sms, cudaStream_t stream) {
    return attn_by_columns<5>(a, sms, stream);
}
cudaError_t attn_d192(const AttnArgs &a, int sms, cudaStream_t stream) {
    return attn_by_columns<6>(a, sms, stream);
}

}  // namespace rfp2
