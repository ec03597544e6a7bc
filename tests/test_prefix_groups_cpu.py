"""SequenceTables.prefix_groups over batches of any make-up: groups that pkv_paged_attention_decode_prefix takes."""
import numpy as np
import pytest

from paged_kv_cache_71_gb300.block_manager import MAX_PREFIX_GROUPS, SequenceTables

S = 4


def _valid(tabs, sids, cu, pre):
    """Every row in one group, no more groups than the call takes, every prefix shared by all of its sequences with tokens and
    found in the first row's table."""
    assert cu.dtype == pre.dtype == np.int32 and len(cu) == len(pre) + 1 <= MAX_PREFIX_GROUPS + 1
    assert cu[0] == 0 and cu[-1] == len(sids) and (np.diff(cu) > 0).all()
    for g, p in enumerate(pre):
        assert p % S == 0
        first = tabs.table(sids[cu[g]])[: p // S]
        assert len(first) == p // S
        for sid in sids[cu[g]:cu[g + 1]]:
            assert tabs.length(sid) == 0 or (p <= tabs.length(sid) and tabs.table(sid)[: p // S] == first)


def _saved(tabs, sids, cu, pre):
    alive = [tabs.length(s) > 0 for s in sids]
    return sum((sum(alive[cu[g]:cu[g + 1]]) - 1) * int(p) // S for g, p in enumerate(pre) if p)


@pytest.mark.parametrize("n", [2048, 2049, 3000, 8192])
def test_many_sequences_that_share_nothing(n):
    tabs = SequenceTables(2 * n, S)
    for s in range(n):
        tabs.prefill(s, 1 + s % (2 * S))
    cu, pre = tabs.prefix_groups(range(n))
    _valid(tabs, range(n), cu, pre)
    assert (pre == 0).all()


def test_sharing_groups_among_thousands_that_share_nothing():
    tabs = SequenceTables(40000, S)
    sids = []
    for s in range(3000):
        tabs.prefill(s, 5)
        sids.append(s)
        if s % 100 == 50:
            tabs.prefill(("r", s), 3 * S)
            sids.append(("r", s))
            for c in range(3):
                tabs.fork(("r", s), ("f", s, c))
                sids.append(("f", s, c))
    cu, pre = tabs.prefix_groups(sids)
    _valid(tabs, sids, cu, pre)
    assert (pre > 0).sum() == 30 and len(pre) == 61 and _saved(tabs, sids, cu, pre) == 30 * 3 * 3


@pytest.mark.parametrize("pairs", [2048, 2049, 3000, 4096])
def test_more_sharing_groups_than_the_call_takes(pairs):
    """Pairs over 1 to 7 blocks: the ones over the fewest are given up, and no more of them than needed."""
    tabs = SequenceTables(10 * pairs, S)
    sids = []
    for s in range(pairs):
        tabs.prefill(s, S * (1 + s % 7) + 1)
        tabs.fork(s, (s, 1))
        sids += [s, (s, 1)]
    cu, pre = tabs.prefix_groups(sids)
    _valid(tabs, sids, cu, pre)
    kept = (pre > 0).sum()
    if pairs == 2048:
        assert kept == 2048
    else:  # one more group kept would be too many (up to two joins are lost with it)
        assert MAX_PREFIX_GROUPS - 2 <= len(pre) <= MAX_PREFIX_GROUPS and kept >= MAX_PREFIX_GROUPS // 2
        given_up = set(range(1, 8)) - set((pre[pre > 0] // S).tolist())
        least = int(pre[pre > 0].min()) // S
        assert given_up == set(range(1, least))  # the smallest savings, all of them below what is kept


def test_rows_without_tokens_stay_in_their_group():
    tabs = SequenceTables(64, S)
    tabs.prefill("a", 2 * S + 1)
    for c in ("b", "c"):
        tabs.fork("a", c)
    for z in ("z0", "z1", "z2", "z3"):
        tabs.prefill(z, 0)
    tabs.prefill("d", 7)
    sids = ["z0", "z1", "a", "z2", "b", "c", "z3", "d"]
    cu, pre = tabs.prefix_groups(sids)
    _valid(tabs, sids, cu, pre)
    assert cu.tolist() == [0, 2, 7, 8] and pre.tolist() == [0, 2 * S, 0]
    cu, pre = tabs.prefix_groups(["z0", "z1"])
    assert cu.tolist() == [0, 2] and pre.tolist() == [0]


@pytest.mark.parametrize("seed", range(4))
def test_random_batches(seed):
    rng = np.random.default_rng(seed)
    tabs = SequenceTables(200000, S)
    sids = []
    for i in range(2500):
        tabs.prefill(i, int(rng.integers(0, 6 * S)) * (rng.random() > 0.1))
        sids.append(i)
        for c in range(int(rng.integers(0, 3))):
            tabs.fork(i, (i, c))
            for _ in range(int(rng.integers(0, 5))):
                tabs.next_slot((i, c))
            sids.append((i, c))
    _valid(tabs, sids, *tabs.prefix_groups(sids))
