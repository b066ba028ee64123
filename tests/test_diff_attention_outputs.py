"""Outputs that differential attention refuses (no device: no call gets to a launch)."""

import pytest

from equivariant_gnn_message_amd import e3conv as E

from .test_diff_attention_host import FAKE, forward
from .test_graph_ops_host import attention_args


@pytest.mark.parametrize("sizes", [dict(), dict(num_graphs=1, num_q=1, num_k=100000)], ids=str)
def test_refuses_one_array_for_both_results(sizes):
    """Two waves (or the join) would write both to the same place."""
    assert forward(attention_args(**sizes), out=FAKE, second=FAKE) == 1
    assert "one array" in E.e3conv_last_error_detail()
    assert forward(attention_args(num_q=0, q=None), out=FAKE, second=FAKE) == 0       # nothing is written
