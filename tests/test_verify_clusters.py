"""Drafts verified by clusters of every size that csrc/pool_rules.h hands out over long vocabularies:
between eight and sixteen CTAs there is none."""
import pytest

from tests.test_verify import Drafts, _ea, float64_want_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("kind,draft", [("bf16", True), ("fp32", False)])
@pytest.mark.parametrize("B,V", [(1, 32_769), (3, 50_257), (24, 61_441), (30, 61_441), (60, 40_009), (90, 33_001),
                                 (140, 30_011)])
def test_sizes(kind, draft, B, V):
    w = Drafts([3, 1, 2] * (B // 3) + [2] * (B % 3), V, kind, draft, seed=B)
    got = w.run()
    keep = range(0, w.B, max(1, w.B // 8))
    assert [(got[0][b], got[1][b]) for b in keep] == float64_want_of(w, keep)
    assert _ea().device_status() == 0
