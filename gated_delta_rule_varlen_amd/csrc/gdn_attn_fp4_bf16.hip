// gdn_attn_fp4_bf16.hip -- the kernels of the attention over a 4-bit cache for bf16 I/O.
#include "gdn_attn_fp4.hpp"

namespace gdn {
namespace attn {
GDN_ATTN_FP4_INSTANCES(BF16)
}  // namespace attn
}  // namespace gdn
