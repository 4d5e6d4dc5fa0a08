// gdn_attn_f16.hip -- the attention tile kernels for f16 I/O.
#include "gdn_attn.hpp"

namespace gdn {
namespace attn {
GDN_ATTN_INSTANCES(F16)
}  // namespace attn
}  // namespace gdn
