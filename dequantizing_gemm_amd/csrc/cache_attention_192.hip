// cache_attention_192.hip -- the attention kernel for code rows of 192 channels.
#include "cache_attention_launch.h"

namespace int4dq {
template hipError_t launch_attention_width<6>(const AttentionArgs&, const Schedule&, const Workspace&, hipStream_t);
}
