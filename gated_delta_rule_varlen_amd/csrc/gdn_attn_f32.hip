// gdn_attn_f32.hip -- the attention tile kernels for f32 I/O.
#include "gdn_attn.hpp"

namespace gdn {
namespace attn {
GDN_ATTN_INSTANCES(F32)
}  // namespace attn
}  // namespace gdn
