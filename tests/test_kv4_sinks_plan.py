"""How a window over many sequences of unknown lengths is cut, seen from its workspace.  No GPU."""
import pytest

from block_wise_int4_amd import mnb
from tests.test_decoder_abi import desc

H, D = 32, 128


def splits(batch, max_kv, window, sinks, new=1):
    d = desc(q_heads=H, kv_heads=8, head_dim=D, group_size=128)
    n = mnb.mnb_attention_kv4_sinks_workspace_bytes(d, batch, batch * new, new, max_kv, window, sinks)
    assert mnb.mnb_last_error() == "" and n % (batch * new * H * (D + 2) * 4) == 0
    return max(1, n // (batch * new * H * (D + 2) * 4))


@pytest.mark.parametrize("new", [1, 5])
@pytest.mark.parametrize("batch", [16, 32, 40, 64, 300, 3000])
def test_no_workgroup_walks_a_long_window_alone(batch, new):
    """A batch may hold one long sequence among short ones: its keys are cut, up to 3072 workgroups' worth."""
    sets = batch * 8                                    # 20 rows of a key head are one set
    for window in (4096, 8000, 16384, 60000):
        n = splits(batch, 65536, window, 4, new)
        pieces = -(-(window + 64 + new) // 5120)
        if 256 % sets == 0 or sets > 256:
            assert n >= min(pieces, max(1, 3072 // sets)), (window, n)
        assert n <= max(-(-3072 // sets), 256 // sets, 1), (window, n)


def test_a_window_of_one_piece_is_not_cut():
    for batch in (32, 64, 500):
        assert splits(batch, 65536, 4096, 4) == 1
