// The attention backward for bf16 tensors.
#include "attention_bwd.h"

namespace ret {
namespace attn {
template int bwd_rows<uint16_t>(const AttnFwd& a);
template hipError_t launch_bwd_q<uint16_t>(const AttnBwd& a, float* stats, float* lam_part, float* part, int shares, hipStream_t s);
template hipError_t launch_bwd_kv<uint16_t>(const AttnBwd& a, const float* stats, float* part, int shares, hipStream_t s);
}  // namespace attn
}  // namespace ret
