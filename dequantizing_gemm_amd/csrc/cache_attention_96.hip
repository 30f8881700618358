// cache_attention_96.hip -- the attention kernel for code rows of 96 channels.
#include "cache_attention_launch.h"

namespace int4dq {
template hipError_t launch_attention_width<3>(const AttentionArgs&, const Schedule&, const Workspace&, hipStream_t);
}
