"""Host-side checks of the paged cache at the ends of what its calls allow."""
import _paged_ref as ref


def test_fork_of_rows_that_end_in_a_missing_page_by_hand():
    p = ref.Pages([[0, 1, -1, -1], [2, 3, 5, -1]], [20, 20], 8, 8)
    assert p.fork() == ([1, 1, 1, 1, 0, 1, 0, 0], 0, [])
    assert p.table == [[0, 1, -1, -1], [2, 3, 5, -1]] and p.d_pos == [16, 20]
    # a window gives back what no token from the rounded row on attends
    p = ref.Pages([[3, -1], [6, 4]], [12, 12], 8, 8)
    p.fork(window=4)
    assert p.table == [[3, -1], [-1, 4]] and p.d_pos == [8, 12]
