// cache_attention_256.hip -- the attention kernel for code rows of 256 channels.
#include "cache_attention_launch.h"

namespace int4dq {
template hipError_t launch_attention_width<8, false>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<false>&, hipStream_t);
}
