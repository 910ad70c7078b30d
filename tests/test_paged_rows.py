"""GPU parity of ragged chunks that take the row kernel (up to 32 packed rows per kv head over
an e4m3 cache), as serving calls it: max_new given and smaller than T, empty and unequal
chunks, one and two warps per key tile. Bounds as in test_paged.py."""
import pytest
import torch

from tests.paged_inputs import Batch
from tests.test_paged import check_attention, oracle, run_prefill
from workloads import MASK_CAUSAL, MASK_NONE, MASK_SLIDING_WINDOW, SCORE_ALIBI, SCORE_SOFTCAP

pytestmark = pytest.mark.gpu

# new tokens, with a longest chunk of 4 and empty ones; cached tokens below and above a tile,
# an empty cache behind new tokens among them
NEW = [4, 0, 1, 3, 0, 4, 2, 4, 1]
LENS = [4, 0, 700, 33, 90, 1300, 2, 129, 0]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def parity(w, what, max_new, split=None, **kw):
    import exact_io_aware_13_gb300 as ea
    o, lse = run_prefill(w, split=split, max_new=max_new, **kw)
    assert ea.device_status() == 0
    check_attention(o[:w.rows], lse[:w.rows], [x[:w.rows] for x in oracle(w, **kw)], what)


@pytest.mark.parametrize("split", [128, 256, 1 << 20])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [2, 4, 6, 8, 5])     # 8, 16, 24, 32 and 20 rows per kv head
def test_ragged_chunks(G, d, split):
    for mask, window in ((MASK_CAUSAL, 0), (MASK_NONE, 0), (MASK_SLIDING_WINDOW, 50)):
        w = Batch(NEW, LENS, Hq=2 * G, Hkv=2, d=d, page=16, kind="e4m3", seed=G + d, spare_rows=3)
        parity(w, f"G {G} mask {mask} split {split}", 4, split, mask=mask, window=window)


@pytest.mark.parametrize("score", [SCORE_ALIBI, SCORE_SOFTCAP, SCORE_ALIBI | SCORE_SOFTCAP])
@pytest.mark.parametrize("G", [4, 7])
def test_ragged_chunks_scores(G, score):
    for d, page in ((64, 8), (128, 64)):
        w = Batch(NEW, LENS, Hq=G, Hkv=1, d=d, page=page, kind="e4m3", seed=60)
        parity(w, f"G {G} score {score}", 4, 256, mask=MASK_CAUSAL, score=score)


@pytest.mark.parametrize("G", [1, 3, 5])
def test_many_sequences(G):
    """More sequences than a warp has lanes; chunks of 0 to 6 tokens."""
    new = [(7 * i) % 7 if i % 3 else (5 * i) % 7 for i in range(75)]
    lens = [n + (11 * i) % 90 for i, n in enumerate(new)]
    w = Batch(new, lens, Hq=2 * G, Hkv=2, page=8, kind="e4m3", seed=61)
    for split, mask in ((None, MASK_CAUSAL), (128, MASK_NONE)):
        parity(w, f"75 sequences G {G}", max(new), split, mask=mask)


def test_same_rows_as_the_tile_kernel():
    """The same chunks with max_new left out are tiles: both kernels within their bounds, and
    rows behind the last sequence untouched in either."""
    import exact_io_aware_13_gb300 as ea
    w = Batch(NEW, LENS, Hq=12, Hkv=2, d=128, page=32, kind="e4m3", seed=62, spare_rows=40)
    c = w.cuda()
    ref = [x[:w.rows] for x in oracle(w)]
    msl = c["table"].shape[1] * w.page
    for max_new in (4, w.T):
        o = torch.full((w.T, w.Hq, w.d), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((w.T, w.Hq), 5.0, device="cuda")
        ws = torch.empty(ea.prefill_workspace_size(w.T, w.Hq, w.d, msl, 128), dtype=torch.uint8,
                         device="cuda")
        ea.prefill_paged_into(c["q"], c["k_cache"], c["v_cache"], c["table"], c["offsets"],
                              c["seq_lens"], o, lse, ws, max_new=max_new, max_seq_len=msl,
                              split_keys=128, scale=w.d ** -0.5, kv_exp=c["kv_exp"],
                              mask_kind=MASK_CAUSAL)
        assert ea.device_status() == 0
        check_attention(o[:w.rows], lse[:w.rows], ref, f"max_new {max_new}")
        assert bool((o[w.rows:] == 3.0).all()) and bool((lse[w.rows:] == 5.0).all())
