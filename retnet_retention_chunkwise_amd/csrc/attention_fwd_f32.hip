// The attention forward for fp32 tensors.
#include "attention_fwd.h"

namespace ret {
namespace attn {
template int fwd_rows<float>(const AttnFwd& a);
template hipError_t launch_fwd<float>(const AttnFwd& a, const Partial& part, hipStream_t s);
}  // namespace attn
}  // namespace ret
