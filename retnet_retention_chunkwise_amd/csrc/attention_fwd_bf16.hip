// The attention forward for bf16 tensors.
#include "attention_fwd.h"

namespace ret {
namespace attn {
template int fwd_rows<uint16_t>(const AttnFwd& a);
template hipError_t launch_fwd<uint16_t>(const AttnFwd& a, const Partial& part, hipStream_t s);
}  // namespace attn
}  // namespace ret
