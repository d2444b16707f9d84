"""Plans of the runtime on the host: which blocks a chunk or a step takes for
itself after a fork, and which tokens may be committed."""

import random

import pytest

from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from paged_kv_cache_56_gb300.runtime import PagedKVCache


@pytest.fixture(scope="module")
def L():
    return ensure_built()


def make_cache(blocks=16, bs=16, int8=False, layers=1):
    return PagedKVCache(layers, blocks, 4, 2, 64, bs, int8, max_slots=4, max_blocks_per_seq=8, device="cpu")


def grow(c, r, n, blocks=0):
    c.add_sequence(r, blocks)
    c.plan_chunk([r], [n])
    c.commit_chunk([r], [n])


def written(c, r, start, n):
    return c.table(r)[start // c.bs:-(-(start + n) // c.bs)]


def test_a_chunk_writes_no_block_that_another_sequence_holds(L):
    """Blocks that a sequence held before it was forked, the whole of which the chunk writes."""
    c = make_cache()
    grow(c, 1, 20, blocks=4)
    c.fork(1, 2)
    before = c.table(1)
    p = c.plan_chunk([1, 2], [30, 30])
    assert not set(written(c, 1, 20, 30)) & set(written(c, 2, 20, 30))
    assert c.table(1)[0] == c.table(2)[0] == before[0]                      # full and shared still
    assert [list(x[:4]) for x in p.tables] == [c.table(1), c.table(2)]
    # the begun block's rows are copied; those behind it hold none yet
    assert p.cow == [(before[1], c.table(1)[1])] or p.cow == [(before[1], c.table(2)[1])]
    c.close()


def test_a_chunk_that_follows_an_unwritten_plan(L):
    c = make_cache()
    c.add_sequence(1)
    c.plan_chunk([1], [40])  # three blocks, one token of them kept
    c.commit_chunk([1], [1])
    c.fork(1, 2)
    c.plan_chunk([1, 2], [31, 31])
    assert not set(written(c, 1, 1, 31)) & set(written(c, 2, 1, 31))
    c.close()


def test_a_sequence_alone_in_its_batch_leaves_the_other_ones_blocks(L):
    c = make_cache()
    grow(c, 1, 32, blocks=4)  # at a block's end: no begun block
    c.fork(1, 2)
    before = c.table(1)
    p = c.plan_chunk([2], [20])
    assert c.table(1) == before and not set(written(c, 2, 32, 20)) & set(before)
    assert not p.cow  # nothing to copy
    c.commit_chunk([2], [20])
    assert not c.plan_chunk([1], [20]).cow and c.table(1) == before  # held by it alone now
    c.close()


@pytest.mark.parametrize("int8", [False, True])
def test_a_step_writes_no_block_that_another_sequence_holds(L, int8):
    """A step that begins a block which a fork left shared."""
    c = make_cache(int8=int8)
    grow(c, 1, 16, blocks=3)
    c.fork(1, 2)  # (at a block's end: no tail to copy)
    before = c.table(1)
    p = c.plan_step([1, 2])
    assert p.block_ids[0] != p.block_ids[1] and before[1] in p.block_ids
    assert [t[1] for t in p.tables] == list(p.block_ids) and p.tables_changed and not p.cow
    c.commit_step([1, 2])
    assert not c.plan_step([1, 2]).cow
    c.close()


def test_the_last_holder_of_a_block_needs_no_copy(L):
    """Holders of one block in one plan take a copy each but the last, if nobody else holds it."""
    for others, free, ok in ((0, 1, True), (0, 0, False), (1, 1, False), (1, 2, True)):
        c = make_cache(blocks=2 + free)
        grow(c, 1, 20)
        c.fork(1, 2)
        if others:
            c.fork(1, 3)
        before = c.table(1)
        if ok:
            p = c.plan_chunk([1, 2], [3, 3])
            assert len(p.cow) == 1 + others and pkv.pkv_num_free(c.alloc) == 0
            assert c.table(1)[1] != c.table(2)[1] and (not others or c.table(3) == before)
        else:
            with pytest.raises(pkv.PkvError) as e:
                c.plan_chunk([1, 2], [3, 3])
            assert e.value.code == pkv.PKV_ERR_OOM
            assert c.table(1) == c.table(2) == before and pkv.pkv_num_free(c.alloc) == free
        c.close()


@pytest.mark.parametrize("int8", [False, True])
def test_fewer_tokens_than_planned_may_be_kept_where_the_cache_still_holds_them(L, int8):
    """Rejected drafts. An INT8 cache has the partly filled block in the slot's one tail, which a chunk that passes the
    block's end fills with the next block's rows: a context may then end only in that last block, or at a block's end."""
    bs = 16
    for start in (0, 5, 14, 15, 16):
        for n in (1, 2, 5, 18, 33):
            for keep in range(n + 1):
                c = make_cache(int8=int8, bs=bs)
                grow(c, 1, start)
                c.plan_chunk([1], [n])
                end = start + keep
                if not int8 or end % bs == 0 or end // bs == (start + n) // bs:
                    c.commit_chunk([1], [keep])
                    assert c.seqs[1].length == end
                else:
                    with pytest.raises(ValueError):
                        c.commit_chunk([1], [keep])
                    assert c.seqs[1].length == start
                    c.commit_chunk([1], [n])  # the whole chunk still may
                    assert c.seqs[1].length == start + n
                c.close()


def test_a_commit_is_all_or_nothing_and_never_of_more_than_planned(L):
    c = make_cache(int8=True)
    grow(c, 1, 14)
    grow(c, 2, 3)
    c.plan_chunk([1, 2], [5, 5])
    for counts in ([1, 5], [5, 6], [5, -1], [5]):
        with pytest.raises(ValueError):
            c.commit_chunk([1, 2], counts)
        assert c.seqs[1].length == 14 and c.seqs[2].length == 3
    c.commit_chunk([2, 1], [2, 5])
    assert c.seqs[1].length == 19 and c.seqs[2].length == 5
    with pytest.raises(ValueError):  # nothing is planned any more
        c.commit_chunk([2], [1])
    c.commit_chunk([2], [0])
    c.close()


def test_a_chunk_does_not_write_a_shared_prefix(L):
    """Blocks attached in front of a sequence are read-only: its length starts behind them."""
    c = make_cache()
    grow(c, 1, 32)
    c.add_sequence(2, shared_blocks=c.table(1))
    for start, n, ok in ((0, 5, False), (31, 3, False), (32, 3, True), (0, 0, True)):
        c.seqs[2].length = start
        before = c.table(2)
        if ok:
            c.plan_chunk([2], [n])
        else:
            with pytest.raises(ValueError, match="prefix"):
                c.plan_chunk([2], [n])
            assert c.table(2) == before
    c.commit_chunk([2], [0])
    c.seqs[2].length = 32
    c.plan_chunk([2], [3])
    c.commit_chunk([2], [3])
    c.fork(2, 3)  # the child's prefix is the parent's
    c.seqs[3].length = 31
    with pytest.raises(ValueError, match="prefix"):
        c.plan_chunk([3], [1])
    c.close()


@pytest.mark.parametrize("seed", range(40))
def test_random_walks_never_write_a_block_of_two_sequences(L, seed):
    """Chunks, steps, forks, rejected drafts and blocks ahead of their tokens, in a pool that runs out now and then."""
    rng = random.Random(seed)
    int8 = seed % 2 == 1
    c = make_cache(blocks=rng.choice([9, 20]), int8=int8)
    alive, nxt = [], 0

    def writes_alone(reqs, spans):
        """spans: tokens (from, to) that each request writes."""
        for r, (a, b) in zip(reqs, spans):
            mine = c.table(r)[a // c.bs:-(-b // c.bs)] if b > a else []
            assert len(mine) == (-(-b // c.bs) - a // c.bs if b > a else 0)
            for other in alive:
                if other != r:
                    assert not set(mine) & set(c.table(other)), (seed, r, other)

    for _ in range(60):
        kind = rng.random()
        try:
            if kind < 0.2 and len(alive) < 4:
                c.add_sequence(nxt, rng.choice([0, 0, 1, 3]))
                alive.append(nxt)
                nxt += 1
            elif kind < 0.35 and alive and len(alive) < 4:
                p = rng.choice(alive)
                if int8 and c.seqs[p].length % c.bs:
                    continue  # (its tail's copy needs a GPU)
                c.fork(p, nxt)
                alive.append(nxt)
                nxt += 1
            elif kind < 0.45 and alive:
                c.remove_sequence(alive.pop(rng.randrange(len(alive))))
            elif kind < 0.65 and alive:
                reqs = [r for r in rng.sample(alive, rng.randint(1, len(alive))) if c.seqs[r].length < 8 * c.bs]
                p = c.plan_step(reqs)
                writes_alone(reqs, [(n, n + 1) for n in p.positions.tolist()])
                assert len({b for _, b in p.cow}) == len(p.cow)
                c.commit_step(reqs)
            elif alive:
                reqs = rng.sample(alive, rng.randint(1, len(alive)))
                counts = [rng.choice([0, 1, 5, 16, 40]) for _ in reqs]
                before = {r: c.table(r) for r in reqs}
                free = pkv.pkv_num_free(c.alloc)
                try:
                    p = c.plan_chunk(reqs, counts)
                except (pkv.PkvError, ValueError):
                    assert {r: c.table(r) for r in reqs} == before and pkv.pkv_num_free(c.alloc) == free
                    continue
                start = [c.seqs[r].length for r in reqs]
                writes_alone(reqs, [(s, s + n) for s, n in zip(start, counts)])
                for r, s in zip(reqs, start):  # rows written before are kept: the same block, or a copy of it
                    for i in range(-(-s // c.bs)):
                        now = c.table(r)[i]
                        assert now == before[r][i] or ((before[r][i], now) in p.cow and i == s // c.bs and s % c.bs)
                keep = [rng.randint(0, n) for n in counts]
                try:
                    c.commit_chunk(reqs, keep)
                except ValueError:
                    assert int8
                    c.commit_chunk(reqs, counts)
        except pkv.PkvError as e:
            assert e.code == pkv.PKV_ERR_OOM
    c.close()


def test_a_step_without_room_takes_no_copies(L):
    """plan_step that runs out of blocks after a fork: nothing has changed, so no copy is lost."""
    c = make_cache(blocks=4)
    grow(c, 1, 5)
    c.fork(1, 2)
    grow(c, 3, 16)
    c.add_sequence(4, 1)
    before = [c.table(r) for r in (1, 2, 3)]
    with pytest.raises(pkv.PkvError) as e:
        c.plan_step([1, 3])  # a copy and a new block, one is free
    assert e.value.code == pkv.PKV_ERR_OOM
    assert [c.table(r) for r in (1, 2, 3)] == before and pkv.pkv_num_free(c.alloc) == 1
    c.remove_sequence(4)
    p = c.plan_step([1, 3])
    assert len(p.cow) == 1 and p.cow[0][0] == before[0][0]
    c.commit_step([1, 3])
    assert not c.plan_step([2]).cow  # the last holder keeps the block
    c.close()


@pytest.mark.parametrize("bs", [16, 64])
def test_drafts_that_can_always_be_rejected(L, bs):
    """Behind a token that stays, as many drafted ones as commit_chunk says: any number of them may be kept."""
    for start in list(range(2 * bs)):
        p = start + 1
        drafts = bs - 1 - p % bs
        for keep in {1, 1 + drafts // 2, 1 + drafts}:
            c = make_cache(int8=True, bs=bs)
            grow(c, 1, start)
            c.plan_chunk([1], [1 + drafts])
            c.commit_chunk([1], [keep])
            assert c.seqs[1].length == start + keep
            c.close()
