"""Host bookkeeping of the page pool against a plain model, and what its calls cost (no GPU needed)."""
import random
import time

import pytest

from sub_bit_kv_b200 import lvq


@pytest.fixture(scope="module", autouse=True)
def built():
    from sub_bit_kv_b200 import _build
    _build.build()


@pytest.mark.parametrize("n_pages,seed", [(1, 0), (63, 1), (64, 2), (65, 3), (700, 4)])
def test_pool_against_a_model(n_pages, seed):
    """Pages taken, shared, given back and renumbered at random: ids lowest first, holders, all or nothing."""
    rng = random.Random(seed)
    pool, holders = lvq.PagePool(n_pages), [0] * n_pages
    for _ in range(300):
        held = [i for i in range(n_pages) if holders[i]]
        free = [i for i in range(n_pages) if not holders[i]]
        op = rng.choice(["alloc", "alloc", "share", "free", "free", "bad", "renumber"])
        if op == "alloc":
            k = rng.randint(0, max(1, n_pages // 3))
            if k > len(free):
                with pytest.raises(lvq.LvqError) as e:
                    pool.alloc(k)
                assert e.value.status == lvq.LVQ_ECAPACITY
            else:
                assert pool.alloc(k) == free[:k]
                for i in free[:k]:
                    holders[i] = 1
        elif op == "bad":
            some = rng.sample(held, rng.randint(0, len(held)))
            wrong = rng.choice([[-1], [n_pages], free[:1], some[:1] * 2])
            if wrong:
                ids = some + wrong if wrong[0] not in some else some + wrong[1:]
                rng.shuffle(ids)
                for call in (pool.share, pool.free):
                    with pytest.raises(lvq.LvqError) as e:
                        call(ids)
                    assert e.value.status == lvq.LVQ_EINVAL
        elif op == "renumber":
            to = rng.sample(range(n_pages), len(held))
            new, moved = [-1] * n_pages, [0] * n_pages
            for i, j in zip(held, to):
                new[i], moved[j] = j, holders[i]
            pool.renumber(new)
            holders = moved
        else:
            ids = rng.sample(held, rng.randint(0, len(held)))
            (pool.share if op == "share" else pool.free)(ids)
            for i in ids:
                holders[i] += 1 if op == "share" else -1
        assert [pool.holders(i) for i in range(n_pages)] == holders
        assert pool.available() == sum(h == 0 for h in holders)


def test_giving_pages_back_costs_no_set_of_them():
    """Giving back 16384 pages: less than Python takes to build one set of their ids.  (One
    walk over the ids; node by node in ordered sets it took 30 times as long.)"""
    n = 16384
    pool = lvq.PagePool(n)
    raw = (lvq.ctypes.c_int32 * n)()
    order = list(range(n))
    random.Random(0).shuffle(order)

    def least(f):
        best = float("inf")
        for _ in range(9):
            t = time.perf_counter()
            f()
            best = min(best, time.perf_counter() - t)
        return best

    def turn():
        assert lvq.lib().lvq_pool_alloc(pool._h, n, raw) == lvq.LVQ_OK
        raw[:] = order
        t = time.perf_counter()
        assert lvq.lib().lvq_pool_free(pool._h, raw, n) == lvq.LVQ_OK
        return time.perf_counter() - t

    lib_s = min(turn() for _ in range(9))
    assert lib_s < least(lambda: set(order)), lib_s
