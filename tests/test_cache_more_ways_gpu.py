"""The 4-bit cache's attention tests once more by way of the kernels for first tokens and shared
tokens: a window of one token with all others as first tokens sees what a call without a window
sees, and so does a call that is given shared tokens."""
import types

import pytest
import torch

from tests.test_cache_edges_gpu import (test_any_bits_before_the_window, test_hidden_tokens_scales,  # noqa: F401
                                        test_largest_scales, test_negative_scales, test_scores_far_from_zero,
                                        test_smallest_scales, test_value_scales_far_apart)
from tests.test_cache_forms_gpu import (test_a_few_more_tiles_than_fit, test_broadcast_rows_and_heads,  # noqa: F401
                                        test_graphs_that_share_a_workspace, test_long_sequences,
                                        test_many_query_heads_of_one, test_prompts, test_sequences_that_share_pages,
                                        test_the_longest_sequence)
from tests.test_cache_gpu import test_attention_query_strides, test_attention_values_of_very_different_sizes  # noqa: F401
from tests.test_cache_plans_gpu import test_bad_plans, test_bad_plans_of_many_sequences, test_two_streams_that_share_out  # noqa: F401

pytestmark = pytest.mark.gpu


def through(dq, way):
    def attention(q, cache, page_table, lengths, starts=None, **kw):
        if kw.get("causal", True) and not kw.get("window") and way == "first":
            kw.update(window=1, sinks=2 ** 40)
        elif way == "shared":
            one = page_table.shape[0] == 1          # a sequence may share its first tokens with itself
            n = lengths // 8 * 5 if one else torch.zeros(1, dtype=torch.int32, device=q.device)
            kw.update(shared=n.to(torch.int32), share_from=1)
        return dq.int4_cache_attention(q, cache, page_table, lengths, starts, **kw)

    def workspace(name):
        more = dict(shared=True, share_from=1) if way == "shared" else {}
        return lambda *a, **kw: getattr(dq, name)(*a, **kw, **more)

    sizes = ("cache_attention_workspace", "cache_attention_workspace_bytes")
    names = {n: getattr(dq, n) for n in dir(dq) if not n.startswith("__")}
    return types.SimpleNamespace(**{**names, "int4_cache_attention": attention, **{n: workspace(n) for n in sizes}})


@pytest.fixture(scope="module", params=["first", "shared"])
def dq(request):
    import dequantizing_gemm_amd as dq
    return through(dq, request.param)
