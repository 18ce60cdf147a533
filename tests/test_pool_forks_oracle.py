"""The pool's restatement by hand: which pairs of a fork are left out."""
from oracle import decoding_oracle as O


def test_a_pair_that_reads_another_pairs_dst_is_made():
    p = O.Pool([[0, 1], [2, 3], [-1, -1]], [1, 1, 1, 1], 16)
    p.fork([0, 1], [1, 2], [32, 20])                  # 1 is a src: the first pair is left out, the second is not
    assert p.table == [[0, 1], [2, 3], [2, 3]] and p.ref == [1, 1, 2, 2]


def test_a_dst_named_twice_is_left_alone():
    p = O.Pool([[0, 1], [-1, -1], [-1, -1]], [1, 1], 16)
    p.fork([0, 0, 0], [1, 1, 2], [32, 32, 16])
    assert p.table == [[0, 1], [-1, -1], [0, -1]] and p.ref == [2, 1]
