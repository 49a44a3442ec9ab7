"""The serial reference of the cache's release against the plan that follows."""
import numpy as np

from oracle import attention as A


def test_a_released_row_without_a_page_gives_no_page():
    table = np.array([[-1, 1], [7, 7]], np.int32)
    lens, table, free, n = A.release([1, 0], np.array([32, 0], np.int32), table, np.array([9, 9, 9], np.int32), 0, 16)
    assert n == 1 and free.tolist() == [1, 9, 9] and table[0].tolist() == [-1, -1] and lens.tolist() == [0, 0]
    table, lens, slots, left = A.plan([0, 0], [0, 0, 32], table, free, n, 16, 32)
    assert lens.tolist() == [0, 0] and (slots == -1).all() and left == 1
