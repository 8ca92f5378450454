"""pkv_bm_truncate and the promise of reserve on admit: what a sequence was
admitted for can be appended whatever is truncated on the way."""
import random

import pytest

from paged_kv_cache_06_gb300 import ops
from paged_kv_cache_06_gb300.block_manager import BlockManager

NO_BLOCKS = 6


def test_truncation_into_a_shared_prefix_takes_the_copys_block_or_refuses():
    bm = BlockManager(num_blocks=3, block_size=4, max_blocks_per_row=3)
    pid, _ = bm.register_prefix(8)
    bm.admit(1, prompt_len=9, max_new_tokens=3, prefix_id=pid)
    before = bm.stats()
    with pytest.raises(ops.PagedKVError) as e:
        bm.truncate(1, 6)              # no block is free for the copy of the second one
    assert e.value.status == NO_BLOCKS
    assert bm.stats() == before and bm.table(1)[1] == 9
    bm.truncate(1, 8)                  # above the shared blocks
    for k in range(4):
        assert bm.append_slot(1)[0] == 8 + k

    bm = BlockManager(num_blocks=4, block_size=4, max_blocks_per_row=3)
    pid, ids = bm.register_prefix(8)
    bm.admit(1, prompt_len=9, max_new_tokens=3, prefix_id=pid)
    bm.truncate(1, 6)
    assert bm.stats()["free_blocks"] == 0
    bm.truncate(1, 5)                  # the block is there already
    with pytest.raises(ops.PagedKVError):
        bm.truncate(1, 3)              # the first block's copy is not
    pos, cow = bm.append_slot(1)
    assert pos == 5 and cow is not None and cow[0] == int(ids[1])
    for k in range(6):
        assert bm.append_slot(1) == (6 + k, None)
    bm.free(1)
    bm.release_prefix(pid)
    assert bm.stats()["used_blocks"] == 0


def test_without_a_reservation_nothing_is_promised():
    bm = BlockManager(num_blocks=3, block_size=4, max_blocks_per_row=3)
    pid, _ = bm.register_prefix(8)
    bm.admit(1, prompt_len=9, max_new_tokens=3, prefix_id=pid, reserve=False)
    bm.truncate(1, 6)
    with pytest.raises(ops.PagedKVError) as e:
        bm.append_slot(1)
    assert e.value.status == NO_BLOCKS


@pytest.mark.parametrize("seed", range(40))
def test_a_reserved_sequence_always_reaches_its_length(seed):
    rng = random.Random(seed)
    bs = rng.choice([1, 4, 8])
    bm = BlockManager(num_blocks=rng.randint(8, 40), block_size=bs, max_blocks_per_row=12)
    pid, _ = bm.register_prefix(rng.randint(0, 3 * bs))
    live = {}
    for sid in range(6):
        prompt, new = rng.randint(1, 4 * bs), rng.randint(1, 4 * bs)
        try:
            bm.admit(sid, prompt, new, prefix_id=pid)
            live[sid] = [prompt, prompt + new]
        except ops.PagedKVError as e:
            assert e.status == NO_BLOCKS
    for _ in range(200):
        if not live:
            break
        sid = rng.choice(list(live))
        n, top = live[sid]
        if rng.random() < 0.4:
            new = rng.randint(0, n)
            before = bm.stats()
            try:
                bm.truncate(sid, new)
                live[sid][0] = new
            except ops.PagedKVError as e:
                assert e.status == NO_BLOCKS and bm.stats() == before
        else:
            for _ in range(min(rng.randint(1, 6), top - n)):
                assert bm.append_slot(sid)[0] == live[sid][0]
                live[sid][0] += 1
    for sid, (n, top) in live.items():      # and all of them to the end, one after the other
        for k in range(n, top):
            assert bm.append_slot(sid)[0] == k
    for sid in live:
        bm.free(sid)
    bm.release_prefix(pid)
    assert bm.stats()["used_blocks"] == 0
