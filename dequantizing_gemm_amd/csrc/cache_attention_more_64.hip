// cache_attention_more_64.hip -- the attention kernel for code rows of 64 channels, with
// first tokens that stay visible and with parts of a batch that shares tokens.
#include "cache_attention_launch.h"

namespace int4dq {
template hipError_t launch_attention_width<2, true>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<true>&, hipStream_t);
}
