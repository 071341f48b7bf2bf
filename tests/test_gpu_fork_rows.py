"""Forks into spare rows of the parents' own table (B200)."""
import pytest
import torch

import pages_ref

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("P,stride", [(16, 5), (1, 300), (64, 1)])
def test_children_in_the_rows_behind_their_parents(P, stride):
    import verify_paged_gqa_b200 as tf
    S, N = 3, 6
    lens = [stride * P, max(1, stride * P // 2), 0]
    refs, table, at = [0] * (S * stride + 4), [], 0
    for n in lens:
        pages = -(-n // P)
        table.append(list(range(at, at + pages)) + [-1] * (stride - pages))
        at += pages
    for page in range(at):
        refs[page] = 1
    parents = [0, 1, 0, -1, 2, 0]
    whole = dev(table + [[-9] * stride for _ in range(N)])
    d_refs, new_lens, status = dev(refs), dev([-9] * N), torch.zeros(1, dtype=torch.int32, device="cuda")
    tf.tf_kv_pages_fork(d_refs, P, whole, dev(lens + [0] * N), dev(parents), whole[S:], new_lens, status=status)
    want, want_lens = pages_ref.fork(refs, P, table, lens, parents, stride)
    assert int(status) == 0
    assert whole.tolist() == table + want and new_lens.tolist() == want_lens and d_refs.tolist() == refs
