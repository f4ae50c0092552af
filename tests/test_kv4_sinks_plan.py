"""How a window over many sequences of unknown lengths is cut, seen from its workspace.  No GPU."""
import pytest

from block_wise_int4_amd import mnb
from tests.test_decoder_abi import desc

H, D = 32, 128


def splits(batch, max_kv, window, sinks, new=1):
    """Pieces of a row set; sinks None: of the call without first tokens."""
    d = desc(q_heads=H, kv_heads=8, head_dim=D, group_size=128)
    if sinks is None:
        n = mnb.mnb_attention_kv4_workspace_bytes(d, batch, batch * new, new, max_kv)
    else:
        n = mnb.mnb_attention_kv4_sinks_workspace_bytes(d, batch, batch * new, new, max_kv, window, sinks)
    assert mnb.mnb_last_error() == "" and n % (batch * new * H * (D + 2) * 4) == 0
    return max(1, n // (batch * new * H * (D + 2) * 4))


@pytest.mark.parametrize("new", [1, 5])
@pytest.mark.parametrize("batch", [40, 64, 128, 300, 2000])
def test_no_workgroup_walks_a_long_window_alone(batch, new):
    """A batch may hold one long sequence among short ones: its keys are cut, up to as many pieces as without first tokens."""
    most = splits(batch, 1 << 20, 0, None, new)
    for window in (4096, 8000, 16384, 60000):
        pieces = -(-(window + 64 + new) // 5120)
        assert splits(batch, 65536, window, 4, new) == min(pieces, most), window


def test_one_workgroup_a_row_set_where_that_is_a_piece():
    for batch in (32, 64, 500):
        assert splits(batch, 65536, 4096, 4) == 1
