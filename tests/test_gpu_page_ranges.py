"""Ranges of tf_kv_pages_free that lie outside the row (B200)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("first,end,bad", [
    (None, [-1, 2], True),          # an end before the row
    ([0, 0], [-5, 1], True),
    ([4, 0], None, True),           # a start past the row's end
    ([4, 0], [3, 1], True),
    ([-1, 0], [2, 1], True),
    ([0, 0], [4, 1], True),
    ([3, 0], None, False),          # the row's very end: nothing of it
    ([2, 0], [1, 1], False),        # an empty range inside the row
    ([0, 0], [0, 1], False)])
def test_a_range_outside_the_row_is_reported_and_frees_nothing(first, end, bad):
    import verify_paged_gqa_b200 as tf
    refs, status = dev([1] * 6), torch.zeros(1, dtype=torch.int32, device="cuda")
    table = dev([[0, 1, 2], [3, 4, 5]])
    tf.tf_kv_pages_free(refs, 16, table, None if first is None else dev(first), None if end is None else dev(end), status=status)
    assert int(status) == (tf.TF_DEV_BAD_LEN if bad else 0)
    lo, hi = 0 if first is None else first[1], 3 if end is None else end[1]
    assert table.tolist() == [[0, 1, 2], [-1 if lo <= j < hi else 3 + j for j in range(3)]]
    assert refs.tolist() == [1] * 3 + [0 if lo <= j < hi else 1 for j in range(3)]
