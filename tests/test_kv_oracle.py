"""The paged cache oracle against closed forms, invariants and brute force."""
import math
import random

import numpy as np
import pytest

from oracle import kv


def random_plan(rng, B, page, max_pages, max_new, free_extra, release=0.2):
    cap = page * max_pages
    kv_len, written, acc, rel, new, pages = [], [], [], [], [], []
    for _ in range(B):
        w = rng.randint(0, min(max_new, 6))
        length = rng.randint(0, cap - w - max_new - 1)
        kv_len.append(length)
        written.append(w)
        acc.append(rng.randint(-1, w - 1) if w else rng.choice([-1, 0]))
        rel.append(int(rng.random() < release))
        new.append(rng.randint(0, max_new))
        pages.append(-(-(length + w) // page))
    total = sum(pages) + free_extra
    ids = list(range(total))
    rng.shuffle(ids)
    table, at = [], 0
    for b in range(B):
        table.append(ids[at:at + pages[b]] + [-7] * (max_pages - pages[b]))
        at += pages[b]
    free = ids[at:] + [-9] * at
    return kv_len, written, acc, rel, new, table, pages, free, free_extra


@pytest.mark.parametrize("seed", range(20))
def test_plan_conserves_pages_and_maps_distinct_slots(seed):
    rng = random.Random(seed)
    B, page, mp, mx = rng.randint(1, 12), rng.choice([1, 3, 16]), 20, rng.randint(1, 9)
    if page * mp <= mx + 8:
        mx = 2
    args = random_plan(rng, B, page, mp, mx, rng.randint(0, 30))
    o = kv.plan(*args, page, mx)
    owned = [int(o["block_table"][b][j]) for b in range(B) for j in range(o["pages"][b])]
    left = list(o["free_pages"][:o["free_count"]])
    assert sorted(owned + left) == list(range(len(args[7])))
    slots = o["slot_map"][o["slot_map"] >= 0]
    assert len(set(slots.tolist())) == len(slots) == int(o["q_len"].sum())
    for b in range(B):
        n_after = int(o["kv_len"][b]) + int(o["q_len"][b])
        assert o["pages"][b] * page >= n_after
        if o["q_len"][b] or not o["starved"]:
            assert o["pages"][b] == -(-n_after // page) or o["starved"]


def test_attend_of_one_key_is_its_value_and_uniform_keys_average():
    rng = np.random.default_rng(0)
    k = rng.normal(size=(4, 2, 1, 8))
    v = rng.normal(size=(4, 2, 1, 8))
    q = rng.normal(size=(1, 1, 2, 8))
    out, lse, _, _ = kv.attend(q, k, v, [[2, 0, 1, 3]], [0], [1], None, 0.5)
    assert np.allclose(out[0, 0], v[2, 0, 0])
    assert np.allclose(lse[0, 0], 0.5 * (q[0, 0] @ k[2, 0, 0]))
    k[:] = 1.0
    out, lse, _, _ = kv.attend(q, k, v, [[2, 0, 1, 3]], [6], [1], None, 0.5)
    order = [v[2], v[0], v[1], v[3][:1]]
    assert np.allclose(out[0, 0], np.concatenate(order).mean((0, 1)))
    assert np.allclose(lse[0, 0], 0.5 * q[0, 0].sum(-1) + math.log(7))


def test_attend_chain_is_the_tree_of_a_line_and_siblings_do_not_see_each_other():
    rng = np.random.default_rng(1)
    k, v = rng.normal(size=(2, 4, 2, 4)), rng.normal(size=(2, 4, 2, 4))
    q = rng.normal(size=(1, 3, 2, 4))
    chain = kv.attend(q, k, v, [[1, 0]], [2], [3], None, 1.0)
    line = kv.attend(q, k, v, [[1, 0]], [2], [3], [[-1, 0, 1]], 1.0)
    assert np.array_equal(chain[0], line[0])
    star = kv.attend(q, k, v, [[1, 0]], [2], [3], [[-1, 0, 0]], 1.0)
    assert np.array_equal(star[0][0, 1], chain[0][0, 1])
    v[1, 3] += 100.0  # node 1: an ancestor of node 2 in the line, not in the star
    assert np.array_equal(kv.attend(q, k, v, [[1, 0]], [2], [3], [[-1, 0, 0]], 1.0)[0][0, 2],
                          star[0][0, 2])
    assert not np.array_equal(kv.attend(q, k, v, [[1, 0]], [2], [3], None, 1.0)[0][0, 2],
                              chain[0][0, 2])


def test_commit_moves_the_path_and_nothing_else():
    cache = np.arange(2 * 3 * 4, dtype=np.float64).reshape(2, 3, 4, 1, 1)
    out = kv.commit(cache, [[2, 0, 1]], [3], [[0, 2, 5, -1]], [2])
    # positions 4, 5 take positions 5, 8; page 0 holds positions 4..7, page 1 8..11
    want = cache.copy()
    want[:, 0, 0], want[:, 0, 1] = cache[:, 0, 1], cache[:, 1, 0]
    assert np.array_equal(out, want)
    assert np.array_equal(kv.commit(cache, [[2, 0, 1]], [3], [[0, 2, 5, -1]], [-1]), cache)
