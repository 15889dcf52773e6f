"""The partition counts of a cascade over a row-scaled e4m3 cache."""
import pytest
import torch

import paged_varlen_attention_attn_gb300 as pa
from test_row_scaled_attention_gpu import Case, built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("reqs,prefix,bound", [
    ([(1, 1184), (1, 900), (1, 700)], 160, 7),  # the suffixes: 1024 keys at most
    ([(1, 2048)], 1024, 7),                     # one token: both passes decode 1024 keys
    ([(1, 200), (1, 180)], 160, 1)])
def test_a_cascades_decode_passes_take_the_bounded_count(reqs, prefix, bound, D):
    # partitions are merged in an order that shows in the last bits
    c = Case(350 + D, reqs, 8, 2, D, 16)
    c.bt[1:, :prefix // 16] = c.bt[0, :prefix // 16]
    args, kw = c.args(), c.kw()
    out = pa.cascade_forward(*args, common_prefix_len=prefix, **kw)
    forced = pa.cascade_forward(*args, common_prefix_len=prefix, num_splits=bound, **kw)
    torch.cuda.synchronize()
    c.check(out)
    assert torch.equal(out, forced)
