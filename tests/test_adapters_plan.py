"""The sizes of the exact GPU tests of the adapters reach the forms that they are there for.  No GPU."""
import pytest

from tests.adapters_plan import build
from tests.test_gpu_adapters_exact import IDS, SIZES


@pytest.fixture(scope="module")
def plan_of(tmp_path_factory):
    return build(str(tmp_path_factory.mktemp("plan")))


@pytest.mark.parametrize("f16", [1, 0], ids=["f16", "f32"])
@pytest.mark.parametrize("case", SIZES, ids=IDS)
def test_sizes_reach_their_forms(plan_of, case, f16):
    size, want = case
    got = plan_of(*size, f16)._asdict()
    assert {k: got[k] for k in want} == want
    if got["down_tile"] == 64:
        assert got["splits"] > 1                       # joined sums of the 64-row form too


def test_every_form_of_many_rows_is_reached(plan_of):
    plans = [plan_of(*size, f16) for size, _ in SIZES for f16 in (0, 1)]
    forms = {(p.down_tile, p.down_ranks) for p in plans if not p.one}
    assert forms >= {(64, 1), (64, 2), (64, 4)}
    forms = {(p.up_tile, p.pitch, p.up_blocks) for p in plans if not p.one}
    assert forms >= {(64, 16, 1), (64, 32, 1), (64, 64, 2), (64, 128, 2), (32, 64, 1), (32, 128, 1), (32, 128, 2)}
