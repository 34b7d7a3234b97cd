"""What a plan holds for the operators of shared prompts: small plans stay
small, and a call on a plan that is just large enough cuts its tiles all the
same."""
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb
from tests import gpu_util as G
from tests.test_shared_gpu import check, make

pytestmark = pytest.mark.gpu

PART = 128 * 513 * 4                                   # a partial of 128 rows
BLOCK = 128 * 1152                                     # a 128-key block


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def test_a_plan_for_appending_and_forking_holds_no_partials_of_the_attention():
    """One request of 64 rows: a block of keys and the one behind it, the split
    partials of its 64 query rows (one per split of at least 64 keys), and
    tables; nothing of 128 rows per SM pair."""
    with mb.Plan(1, 1, 64, 64, 4096, 64, torch.bfloat16) as plan:
        assert plan.workspace_bytes() < 2 * BLOCK + PART + 65536


def test_a_short_plan_holds_partials_for_the_pairs_it_can_use():
    """Two requests of 280 rows, 64 query rows each: a tile each at most, of
    three steps or less, so a few pairs of 76."""
    with mb.Plan(2, 4, 16, 1, 1024, 280, torch.bfloat16) as plan:
        assert plan.workspace_bytes() < 7 * BLOCK + 16 * PART


@pytest.mark.parametrize("sizes,shared,own,T,H", [
    ([1], [0], [255], 1, 128),                         # one step
    ([1], [500], [11], 1, 128),                        # two steps, whole
    ([1], [1200], [100], 1, 128),                      # cut in two and three
    ([1], [2500], [300], 1, 129),                      # two tiles
    ([2], [1000], [100, 900], 1, 128),
    ([1, 1, 1], [700, 700, 700], [9, 5, 2], 3, 64),
    ([20], [400], list(range(20)), 1, 16),
])
def test_calls_that_fill_their_plan(sizes, shared, own, T, H):
    case = make(sizes, shared, own, T, H, seed=80)
    check(case)
    with G.make_plan(case[0]) as plan:
        assert plan.max_kv_len == max(case[0].kv_lens.tolist())
