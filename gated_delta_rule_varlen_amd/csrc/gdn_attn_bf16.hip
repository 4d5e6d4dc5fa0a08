// gdn_attn_bf16.hip -- the attention tile kernels for bf16 I/O.
#include "gdn_attn.hpp"

namespace gdn {
namespace attn {
GDN_ATTN_INSTANCES(BF16)
}  // namespace attn
}  // namespace gdn
