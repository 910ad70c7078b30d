"""Pins of the pool oracle: cases small enough to be followed by hand."""
import numpy as np

from oracle import pool_oracle as P


def test_fork_counts_holders():
    table, lens, refs = [[2, 0, 9], [1, 9, 9], [9, 9, 9]], [20, 16, 0], [1, 1, 1, 0]
    t, n, r = P.fork(table, lens, refs, [0, 0, 0], 16)
    assert t == [[2, 0, 9], [2, 0, 9], [2, 0, 9]] and n == [20, 20, 20] and r == [3, 0, 3, 0]
    t, n, r = P.fork(table, lens, refs, [1, -1, 0], 16)
    assert t == [[1, -1, 9], [-1, 9, 9], [2, 0, 9]] and n == [16, 0, 20] and r == [1, 1, 1, 0]


def test_resize_copies_before_a_shared_page_is_written():
    table, refs = [[3, 1], [3, 1]], [0, 2, 0, 2, 0]
    t, n, r, missing, copies = P.resize(table, [12, 12], refs, [13, 14], 8)
    # both write into page 1: row 0 keeps it, row 1 copies its 4 tokens
    assert t == [[3, 1], [3, 0]] and r == [1, 1, 0, 2, 0] and copies == [(1, 0, 4)] and missing == 0
    t, n, r, missing, copies = P.resize(table, [12, 12], [0, 3, 0, 2, 0], [13, 12], 8)
    assert t == [[3, 0], [3, 1]] and r == [1, 2, 0, 2, 0] and copies == [(1, 0, 4)]


def test_resize_gives_back_first():
    table, refs = [[0, 1, 2], [-1, -1, -1]], [1, 1, 1]
    t, n, r, missing, _ = P.resize(table, [24, 0], refs, [3, 16], 8)
    assert missing == 0 and t == [[0, -1, -1], [1, 2, -1]] and r == [1, 1, 1]
    t, n, r, missing, _ = P.resize(table, [24, 0], refs, [9, 16], 8)
    assert missing == 1 and t == table and n == [24, 0] and r == refs


def test_resize_window():
    # 8 tokens stay visible to token 30: those from 23 on; pages 0 and 1 (0-15) have passed
    t, n, r, missing, _ = P.resize([[4, 3, 2, 1]], [30], [0, 1, 1, 1, 1], [31], 8, window=8)
    assert t == [[-1, -1, 2, 1]] and r == [0, 1, 1, 0, 0]
    t, *_ = P.resize([[4, 3, 2, 1]], [31], [0, 1, 1, 1, 1], [32], 8, window=8)
    assert t == [[-1, -1, -1, 1]]                            # 31 - 7 = 24: page 2 ends at 23


def test_compact():
    table, refs, used, page_map, moves = P.compact([[5, 1, 7]], [20], [0, 1, 0, 0, 0, 2, 0, 1], 8)
    assert used == 3 and moves == [(7, 0), (5, 2)]
    assert table == [[2, 1, 0]] and refs == [1, 1, 2, 0, 0, 0, 0, 0]
    assert page_map == [-1, 1, -1, -1, -1, 2, -1, 0]


def test_verify():
    p = np.array([[0.5, 0.25, 0.25], [0.0, 0.5, 0.5], [0.25, 0.25, 0.5]])
    q = np.array([[0.25, 0.5, 0.25], [1.0, 0.0, 0.0], [0.0, 0.0, 0.0]])
    run = lambda tokens, u, s: P.verify(p, q, tokens, [0, 3], u, [s])  # noqa: E731
    assert run([9, 0, 0], [0.99, 0.5, 9], 0.0) == ([1], [1])  # token 0 stays, then p = 0: residual
    assert run([9, 0, 0], [0.99, 0.5, 9], 0.5) == ([1], [2])
    assert run([9, 1, 1], [0.4, 0.9, 9], 0.3) == ([2], [1])   # all stay: the last row of p
    assert run([9, 1, 1], [0.5, 0.9, 9], 0.99) == ([0], [0])  # 0.5 * 0.5 is not below 0.25
    # without draft probabilities: p of the draft against u, the residual leaves the draft out
    assert P.verify(p, None, [9, 0, 1], [0, 3], [0.5, 0, 9], [0.6]) == ([0], [2])
    assert P.verify(p, None, [9, 0, 1], [0, 3], [0.4, 0.4, 9], [0.5]) == ([2], [2])
    assert P.verify(p, q, [9, 0, 1], [0, 0, 1], [0, 0, 0], [0.5, 0.5]) == ([0, 0], [-1, 1])
