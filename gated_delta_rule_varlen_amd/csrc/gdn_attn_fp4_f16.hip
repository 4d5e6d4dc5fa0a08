// gdn_attn_fp4_f16.hip -- the kernels of the attention over a 4-bit cache for fp16 I/O.
#include "gdn_attn_fp4.hpp"

namespace gdn {
namespace attn {
GDN_ATTN_FP4_INSTANCES(F16)
}  // namespace attn
}  // namespace gdn
