"""pa_bm_evict while copy-on-write pairs are queued: a block that the eviction rewrites or frees
may be the source of a copy that has not been made, or its target."""
import pytest


@pytest.fixture(scope="module")
def BM():
    from paged_kv_cache_53_gb300 import build
    build.build()
    from paged_kv_cache_53_gb300 import block_manager
    return block_manager


def _forked(BM):
    bm = BM.BlockManager(12, 4)
    bm.add_sequence(1, range(14))  # 0 .. 3
    bm.fork(1, 2)
    bm.append_tokens(2, [5])       # block 3 is to be copied to 4
    return bm


def _state(bm):
    return ([bm.block_table(s) for s in (1, 2)], [bm.num_tokens(s) for s in (1, 2)],
            [bm.refcount(b) for b in range(12)], bm.free_queue())


@pytest.mark.parametrize("ids,keep", [
    ([1], [13]),         # keeps the pair's source, to be written in place
    ([1], [6]),          # frees it
    ([2], [13]),         # keeps its target in place
    ([1, 2], [6, 6]),
    ([1, 2], [14, 13]),  # only one of the two is cut
])
def test_queued_copies_come_first(BM, ids, keep):
    bm = _forked(BM)
    before = _state(bm)
    with pytest.raises(BM.PaError, match="copy-on-write"):
        bm.evict(ids, keep)
    assert _state(bm) == before
    assert bm.take_copies().tolist() == [[3, 4]]
    bm.evict(ids, keep)
    assert [bm.num_tokens(s) for s in ids] == keep


def test_a_call_that_cuts_nothing_is_not_refused(BM):
    bm = _forked(BM)
    before = _state(bm)
    bm.evict([1, 2], [14, 15])
    bm.evict([], [])
    assert _state(bm) == before
    assert bm.take_copies().tolist() == [[3, 4]]
