"""Caches that lie between one another, as the pass that norms, rotates and appends takes them.  What passes is
seen by a later check's refusal, so that nothing is enqueued (no device needed)."""
import itertools

import numpy as np
import pytest

from test_q8kv_refusals import E, M, P, lib, project, seq  # noqa: F401

TOK = 128


def refused(lib, views):  # noqa: F811
    """Whether two caches are said to overlap; else the call's q does, on the projection."""
    assert project(lib, views=views, q=P) == E
    said = lib.luce_last_error()
    assert (b"cache" in said) != (b"projection" in said), said
    return b"cache" in said


def test_slices_of_a_pool_along_its_tokens_pass(lib):  # noqa: F811
    """K and V of four slots as slices of [2][Hkv][4 x 64][128]: the heads of one lie between those of the others."""
    head = 4 * 64 * TOK
    views = [seq(k=P + M + 2 * s * 64 * TOK, v=P + 2 * M + 2 * s * 64 * TOK, row0=4 * s, head=head) for s in range(4)]
    assert not refused(lib, views)
    views[2] = seq(k=views[2].k, v=P + M + 2 * 64 * TOK, row0=8, head=head)        # V of slot 2 is K of slot 1
    assert refused(lib, views)


def test_keys_and_values_of_a_token_side_by_side_pass(lib):  # noqa: F811
    """[Hkv][cap][2][128] and [Hkv][2][cap][128]."""
    assert not refused(lib, [seq(k=P + M, v=P + M + 2 * TOK, tok=2 * TOK, head=64 * 2 * TOK)])
    assert not refused(lib, [seq(k=P + M, v=P + M + 2 * 64 * TOK, head=2 * 64 * TOK)])
    assert refused(lib, [seq(k=P + M, v=P + M + 2 * 64, tok=2 * TOK, head=64 * 2 * TOK)])
    assert refused(lib, [seq(k=P + M, v=P + M + 2 * TOK, head=64 * TOK)])


def test_one_cache_at_other_rows_passes(lib):  # noqa: F811
    assert not refused(lib, [seq(length=10, n=4), seq(length=14, n=4, row0=4)])
    assert not refused(lib, [seq(length=14, n=4), seq(length=10, n=4, row0=4)])
    assert refused(lib, [seq(length=10, n=4), seq(length=13, n=4, row0=4)])
    assert refused(lib, [seq(length=13, n=4), seq(length=10, n=4, row0=4)])


def test_unlike_strides_that_may_meet_are_refused(lib):  # noqa: F811
    assert refused(lib, [seq(head=4 * 64 * TOK), seq(k=P + M + 2 * 64 * TOK, v=P + 2 * M + 2 * 64 * TOK, row0=4, head=2 * 64 * TOK)])


def test_against_every_value(lib):  # noqa: F811
    """Two slots at random places of a small room: refused exactly where they share a value."""
    rng = np.random.default_rng(0)
    met = 0
    for _ in range(3000):
        tok, cap = int(rng.choice([128, 136, 256, 384])), int(rng.integers(1, 6))
        head = tok * cap + 8 * int(rng.integers(0, 80))
        heads, sets, views, row0 = 2, [], [], 0
        n = [int(rng.integers(1, cap + 1)) for _ in range(2)]
        for s in range(2):
            at = [8 * int(rng.integers(0, 500)) for _ in range(2)]
            length = int(rng.integers(n[s], cap + 1))
            for a in at:
                sets.append({a + g * head + i * tok + x for g, i, x in itertools.product(range(heads), range(length - n[s], length), range(0, 128, 8))})
            views.append(seq(k=P + M + 2 * at[0], v=P + M + 2 * at[1], length=length, n=n[s], row0=row0, cap=cap, head=head, tok=tok))
            row0 += n[s]
        want = any(a & b for a, b in itertools.combinations(sets, 2))
        met += want
        assert refused(lib, views) == want
    assert 300 < met < 2700
