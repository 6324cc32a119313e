"""Forms of the shared-prefix attention beside those of test_gpu_prefix_step.py, with its bounds:
batches of many requests, of mixed requests and of long prompts, the caller's own buffers, calls
side by side, pages and lengths that are not there, and sizes that pass 32 bits in the plan."""
import pytest
import torch

from test_gpu_prefix_step import Case, dsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("H,requests", [(8, 300), (20, 131), (1, 400)])
def test_many_requests_with_keys_of_their_own(H, requests):
    # whole own tiles of few rows that straddle the blocks of 128 rows which their results stand in
    reqs = [(1 + i % 3 if i % 7 else 0, 201 + (37 * i) % 400) for i in range(requests)]
    Case(H, 16, 200, reqs, pad=2, seed=H).check()
