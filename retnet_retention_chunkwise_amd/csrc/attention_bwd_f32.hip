// The attention backward for fp32 tensors.
#include "attention_bwd.h"

namespace ret {
namespace attn {
template int bwd_rows<float>(const AttnFwd& a);
template hipError_t launch_bwd_q<float>(const AttnBwd& a, float* stats, float* lam_part, float* part, int shares, hipStream_t s);
template hipError_t launch_bwd_kv<float>(const AttnBwd& a, const float* stats, float* part, int shares, hipStream_t s);
}  // namespace attn
}  // namespace ret
