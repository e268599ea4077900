"""pa_bm_evict: the block manager's part of an eviction, against a model of
its contract, alone and among the other calls."""
import random

import pytest

import paged_kv_cache_262_gb300 as pa
from paged_kv_cache_262_gb300 import build as pbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    pbuild.build()


def test_own_blocks_stay_and_the_tail_is_released():
    bm = pa.BlockManager(16, 4)
    bm.add_seq(0, 22)  # 6 blocks
    before = bm.block_table(0)
    assert bm.evict(0, 9) == before[:3]
    assert bm.block_table(0) == before[:3] and bm.seq_len(0) == 9
    assert bm.num_free() == 13 and [bm.ref_count(b) for b in before] == [1, 1, 1, 0, 0, 0]
    slot, cow = bm.append(0)  # token 9 goes behind the kept ones
    assert slot == before[2] * 4 + 1 and cow is None or tuple(cow) == (-1, -1)


@pytest.mark.parametrize("keep", [22, 23, 10**6])
def test_nothing_to_evict(keep):
    bm = pa.BlockManager(16, 4)
    bm.add_seq(0, 22)
    t = bm.block_table(0)
    assert bm.evict(0, keep) == t and bm.block_table(0) == t and bm.seq_len(0) == 22 and bm.num_free() == 10
    bm.add_seq(1, 0)
    assert bm.evict(1, 1) == []


def test_shared_blocks_are_replaced():
    bm = pa.BlockManager(16, 4)
    bm.add_seq(0, 16)
    bm.fork(0, 1)
    bm.append(1)
    bm.append(1)  # a block of its own, 18 tokens
    shared, t1 = bm.block_table(0), bm.block_table(1)
    assert t1[:4] == shared
    dst = bm.evict(1, 7)
    assert len(dst) == 2 and not set(dst) & set(t1) and bm.block_table(1) == dst
    assert bm.block_table(0) == shared and [bm.ref_count(b) for b in shared] == [1] * 4
    assert bm.ref_count(t1[4]) == 0 and all(bm.ref_count(b) == 1 for b in dst)
    assert bm.num_free() == 16 - 4 - 2
    # the other holder is alone with its blocks now: in place
    assert bm.evict(0, 5) == shared[:2]


def test_fresh_blocks_are_none_of_the_released_ones():
    """With no free block left the released tail must not be handed out: it
    is a source of the same eviction."""
    bm = pa.BlockManager(5, 4)
    bm.add_seq(0, 16)
    bm.fork(0, 1)
    bm.append(1)
    assert bm.num_free() == 0
    t = bm.block_table(1)
    with pytest.raises(pa.PaError) as e:
        bm.evict(1, 4)
    assert e.value.status == pa.PA_ERR_OOM
    assert bm.block_table(1) == t and bm.seq_len(1) == 17 and bm.num_free() == 0


def test_refusals_leave_everything():
    import ctypes
    bm = pa.BlockManager(16, 4, 8)
    bm.add_seq(0, 10)
    lib, n, buf = pa.load(), ctypes.c_int(-7), (ctypes.c_int32 * 8)()
    f = lib.pa_bm_evict
    assert f(None, 0, 4, buf, 8, ctypes.byref(n)) == pa.PA_ERR_INVALID
    assert f(bm._h, 0, 0, buf, 8, ctypes.byref(n)) == pa.PA_ERR_INVALID
    assert f(bm._h, 0, -1, buf, 8, ctypes.byref(n)) == pa.PA_ERR_INVALID
    assert f(bm._h, 0, 4, buf, 8, None) == pa.PA_ERR_INVALID
    assert f(bm._h, 0, 8, None, 8, ctypes.byref(n)) == pa.PA_ERR_INVALID
    assert f(bm._h, 9, 4, buf, 8, ctypes.byref(n)) == pa.PA_ERR_STATE
    assert f(bm._h, 0, 8, buf, 1, ctypes.byref(n)) == pa.PA_ERR_INVALID and n.value == 2
    assert bm.seq_len(0) == 10 and bm.num_free() == 13
    bm.swap_out(0)
    assert f(bm._h, 0, 4, buf, 8, ctypes.byref(n)) == pa.PA_ERR_STATE


def test_overwritten_blocks_leave_the_prefix_cache():
    bm = pa.BlockManager(32, 4)
    prompt = list(range(20))
    bm.add_seq_tokens(0, prompt)
    assert bm.num_cached_blocks() == 5
    bm.evict(0, 10)
    assert bm.num_cached_blocks() == 0  # the rewritten ones, and what continued them
    assert bm.add_seq_tokens(1, prompt) == 0
    # the evicted sequence's later blocks are not registered
    for t in range(6):
        bm.append(0, 100 + t)
    assert bm.num_cached_blocks() == 5
    # a shared prompt stays cached for its other user, and for new ones
    bm.fork(1, 2)
    bm.evict(2, 6)
    assert bm.num_cached_blocks() == 5 and bm.add_seq_tokens(3, prompt) == 20


@pytest.mark.parametrize("seed", range(8))
def test_among_the_other_calls(seed):
    """Random calls: reference counts are the tables' multiplicities, free
    blocks the rest, lengths fit the tables, and an evicted sequence's table
    is its own."""
    r = random.Random(seed)
    bm, B, N = pa.BlockManager(48, 4), 4, 48
    lens, nxt = {}, 0
    for _ in range(400):
        op = r.random()
        try:
            if op < 0.2 or not lens:
                if r.random() < 0.5:
                    n = r.randint(0, 30)
                    bm.add_seq(nxt, n)
                else:
                    n = r.randint(0, 30)
                    bm.add_seq_tokens(nxt, [r.randint(0, 1) for _ in range(n)])
                lens[nxt] = n
                nxt += 1
                continue
            s = r.choice(list(lens))
            if op < 0.3:
                bm.fork(s, nxt)
                lens[nxt] = lens[s]
                nxt += 1
            elif op < 0.6:
                bm.append(s, r.choice((None, r.randint(0, 1))))
                lens[s] += 1
            elif op < 0.85:
                keep, t = r.randint(1, 30), bm.block_table(s)
                dst = bm.evict(s, keep)
                n = min(keep, lens[s])
                assert len(dst) == -(-n // B)
                if keep < lens[s]:
                    lens[s] = n
                    assert all(bm.ref_count(b) == 1 for b in dst)
                    assert all(d == t[i] or d not in t for i, d in enumerate(dst))
                else:
                    assert dst == t
            else:
                bm.free_seq(s)
                del lens[s]
        except pa.PaError as e:
            assert e.status == pa.PA_ERR_OOM
        held = {}
        for s in lens:
            assert bm.seq_len(s) == lens[s]
            t = bm.block_table(s)
            assert len(t) == -(-lens[s] // B) and len(set(t)) == len(t)
            for b in t:
                held[b] = held.get(b, 0) + 1
        assert [bm.ref_count(b) for b in range(N)] == [held.get(b, 0) for b in range(N)]
        assert bm.num_free() == N - len(held)


# ---------------------------------------------------------------- several at once
def test_a_batch_replaces_what_any_of_it_reads():
    """Two holders of the same blocks and a third sequence: one by one, the
    last holder would stay in place over the first one's source, and released
    tails would come back as fresh blocks."""
    bm = pa.BlockManager(32, 4)
    bm.add_seq(0, 16)
    bm.fork(0, 1)
    bm.append(1)
    bm.add_seq(2, 30)
    tables, lens = bm.block_tables([0, 1, 2], 10)
    assert lens.tolist() == [16, 17, 30]
    dst, new = bm.evict_batch([0, 1, 2], [6, 9, 13], 10, pad=-7)
    assert new.tolist() == [6, 9, 13] and dst.shape == (3, 10)
    rows = [dst[i, :n].tolist() for i, n in enumerate((2, 3, 4))]
    assert [(dst[i, n:] == -7).all() for i, n in enumerate((2, 3, 4))] == [True] * 3
    assert rows[2] == tables[2, :4].tolist()  # its own, in place
    assert not (set(rows[0]) | set(rows[1])) & set(tables[tables >= 0].tolist())
    assert len(set(sum(rows, []))) == 9
    assert [bm.block_table(s) for s in range(3)] == rows and [bm.seq_len(s) for s in range(3)] == [6, 9, 13]
    assert bm.num_free() == 32 - 9


def test_a_batch_of_one_is_the_single_call():
    for keep in (1, 4, 5, 16, 17, 40):
        a, b = pa.BlockManager(32, 4), pa.BlockManager(32, 4)
        for m in (a, b):
            m.add_seq(0, 16)
            m.fork(0, 1)
            m.append(1)
        dst, new = a.evict_batch([1], [keep], 8)
        one = b.evict(1, keep)
        assert dst[0, :len(one)].tolist() == one and (dst[0, len(one):] == -1).all()
        assert new.tolist() == [b.seq_len(1)] and a.num_free() == b.num_free()
    dst, new = a.evict_batch([], [], 4)
    assert dst.shape == (0, 4) and new.shape == (0,)


def test_a_batch_with_sequences_that_stay():
    bm = pa.BlockManager(16, 4)
    bm.add_seq(0, 12)
    bm.fork(0, 1)
    t = bm.block_table(0)
    dst, new = bm.evict_batch([0, 1], [12, 5], 3)
    assert dst[0].tolist() == t and new.tolist() == [12, 5]
    assert not set(dst[1, :2].tolist()) & set(t) and bm.block_table(0) == t and bm.num_free() == 16 - 5


def test_a_refused_batch_leaves_everything():
    import numpy as np
    bm = pa.BlockManager(8, 4, 8)
    bm.add_seq(0, 16)
    bm.fork(0, 1)
    bm.append(1)
    bm.add_seq(2, 3)
    state = lambda: ([bm.block_table(s) for s in (0, 1, 2)], [bm.seq_len(s) for s in (0, 1, 2)],  # noqa: E731
                     bm.num_free())
    was = state()
    for ids, keep, mb, status in (([0, 9], [4, 4], 8, pa.PA_ERR_STATE), ([0, 0], [4, 4], 8, pa.PA_ERR_INVALID),
                                  ([0, 1], [4, 0], 8, pa.PA_ERR_INVALID), ([0, 1], [4, -3], 8, pa.PA_ERR_INVALID),
                                  ([2, 1], [1, 9], 2, pa.PA_ERR_INVALID), ([0, 1], [6, 6], 8, pa.PA_ERR_OOM)):
        with pytest.raises(pa.PaError) as e:
            bm.evict_batch(ids, keep, mb)
        assert e.value.status == status and state() == was
    with pytest.raises(ValueError):
        bm.evict_batch([0, 1], [4], 8)
    f = pa.load().pa_bm_evict_batch
    i, k, o = (np.array(x, np.int32) for x in ([0], [4], [0, 0]))
    P = lambda x: x.ctypes.data  # noqa: E731
    assert f(None, P(i), P(k), 1, P(o), 2, -1, None) == pa.PA_ERR_INVALID
    assert f(bm._h, None, P(k), 1, P(o), 2, -1, None) == pa.PA_ERR_INVALID
    assert f(bm._h, P(i), None, 1, P(o), 2, -1, None) == pa.PA_ERR_INVALID
    assert f(bm._h, P(i), P(k), 1, None, 2, -1, None) == pa.PA_ERR_INVALID
    assert f(bm._h, P(i), P(k), -1, P(o), 2, -1, None) == pa.PA_ERR_INVALID
    assert f(bm._h, P(i), P(k), 1, P(o), -1, -1, None) == pa.PA_ERR_INVALID
    assert f(bm._h, None, None, 0, None, 0, -1, None) == pa.PA_OK and state() == was
    bm.swap_out(2)
    with pytest.raises(pa.PaError) as e:
        bm.evict_batch([0, 2], [1, 1], 8)
    assert e.value.status == pa.PA_ERR_STATE
    assert f(bm._h, P(i), P(k), 1, P(o), 2, -1, None) == pa.PA_OK and bm.seq_len(0) == 4


@pytest.mark.parametrize("seed", range(8))
def test_batches_among_the_other_calls(seed):
    """Random calls: a batch's destinations are distinct, each its sequence's
    own entry or a block that no table of the batch held; the counts, the free
    blocks and the prefix cache's answers fit the tables afterwards."""
    r = random.Random(100 + seed)
    B, N = 4, 64
    bm, lens, nxt = pa.BlockManager(N, B), {}, 0
    for _ in range(300):
        op = r.random()
        try:
            if op < 0.25 or not lens:
                n = r.randint(0, 30)
                bm.add_seq_tokens(nxt, [r.randint(0, 1) for _ in range(n)])
                lens[nxt], nxt = n, nxt + 1
            elif op < 0.4:
                s = r.choice(list(lens))
                bm.fork(s, nxt)
                lens[nxt], nxt = lens[s], nxt + 1
            elif op < 0.6:
                ids = r.sample(list(lens), r.randint(1, len(lens)))
                bm.append_batch(ids, [r.randint(0, 1) for _ in ids])
                for s in ids:
                    lens[s] += 1
            elif op < 0.9:
                ids = r.sample(list(lens), r.randint(1, len(lens)))
                keep = [r.randint(1, 30) for _ in ids]
                src, _ = bm.block_tables(ids, 40)
                dst, new = bm.evict_batch(ids, keep, 40)
                read = set(src[src >= 0].tolist())
                written = []
                for i, s in enumerate(ids):
                    n = -(-min(keep[i], lens[s]) // B)
                    assert new[i] == min(keep[i], lens[s]) and (dst[i, n:] == -1).all()
                    assert all(d == src[i, j] or d not in read for j, d in enumerate(dst[i, :n].tolist()))
                    if keep[i] < lens[s]:
                        written += dst[i, :n].tolist()
                        assert not set(dst[i, :n].tolist()) & {int(x) for j in range(len(ids)) if j != i
                                                               for x in src[j] if x >= 0}
                        lens[s] = keep[i]
                    assert bm.block_table(s) == dst[i, :n].tolist()
                assert len(set(written)) == len(written)
            else:
                s = r.choice(list(lens))
                bm.free_seq(s)
                del lens[s]
        except pa.PaError as e:
            assert e.status == pa.PA_ERR_OOM
            if r.random() < 0.5:
                s = r.choice(list(lens))
                bm.free_seq(s)
                del lens[s]
        held = {}
        for s in lens:
            t = bm.block_table(s)
            assert bm.seq_len(s) == lens[s] and len(t) == -(-lens[s] // B) and len(set(t)) == len(t)
            for b in t:
                held[b] = held.get(b, 0) + 1
        assert [bm.ref_count(b) for b in range(N)] == [held.get(b, 0) for b in range(N)]
        assert bm.num_free() == N - len(held) and 0 <= bm.num_cached_blocks() <= N
