"""Streams whose positions come near 2^31, over few pages: a sliding-window
layer holds the pages of its window and sinks only (B200)."""
import math

import pytest
import torch

import window_ref
from test_gpu_window import CLUSTER, TENSOR_CORE, big_workspace

pytestmark = pytest.mark.gpu

LAST = 2 ** 31 - 1


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d,G,rows", [(128, 4, 1), (128, 8, 8), (128, 4, 100), (256, 4, 5), (512, 8, 4), (512, 4, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (333, 4), (300, 130)])
@pytest.mark.parametrize("P", [65536, 40000])
def test_a_window_layers_step(d, G, rows, window, sinks, P):
    import verify_paged_gqa_b200 as tf
    Hkv, L = 2, 1400
    g = torch.Generator(device="cuda")
    g.manual_seed(d + rows + window)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    lens = [LAST, LAST - 70, 70001, LAST // 2]
    S, stride = len(lens), -(-LAST // P)
    held = sorted({(s, p // P) for s, n in enumerate(lens) for p in (0, n - rows - window, n - 1)})
    pools = [torch.full((len(held) + 1, Hkv, P, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.full((S, stride), -1, dtype=torch.int32)
    for page, (s, j) in enumerate(held):
        table[s, j] = page
    table = table.cuda()
    q = r(S, rows, Hkv * G, d)
    lin = [(r(L, Hkv, d), r(L, Hkv, d)) for _ in lens]   # (the same set of positions in a short cache)
    for s, n in enumerate(lens):
        at = [(i, i) for i in range(sinks)] + [(L - rows - window + i, n - rows - window + i) for i in range(window)]
        for pool, x in zip(pools, lin[s]):
            for i, pos in at:
                pool[int(table[s, pos // P]), :, pos % P] = x[i]
    # the step's own rows: turned by nothing (a frequency of zero) and written by the library
    rope = tf.Rope(torch.zeros(d // 2, device="cuda"))
    k_rows, v_rows = (torch.stack([x[c][L - rows:] for x in lin]) for c in (0, 1))
    positions = dev([[[n - rows + w] for w in range(rows)] for n in lens])
    turned = tf.tf_kv_put_rows_rope(*pools, table, dev(lens), q, k_rows, v_rows, positions, rope, LAST)
    assert torch.equal(turned, q)
    for kernel in (0, TENSOR_CORE, CLUSTER):
        out = torch.full(q.shape, float("nan"), dtype=torch.float32, device="cuda")
        tf.tf_testing_paged_attn_window(*pools, table, dev(lens), q, window, sinks, 1.0 / math.sqrt(d), out, big_workspace(), LAST,
                                        kernel=kernel)
        assert tf.tf_workspace_status(big_workspace()) == 0
        for s in range(S):
            ref, bound = window_ref.attend(q[s], *lin[s], window, sinks, 1.0 / math.sqrt(d))
            assert ((out[s].double() - ref).abs() <= bound).all(), (kernel, s)


@pytest.mark.parametrize("P", [65536, 40000])
def test_pages_of_the_last_positions(P):
    import verify_paged_gqa_b200 as tf
    stride = -(-LAST // P)
    refs, status = dev([0] * 8), torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.full((1, stride), -1, dtype=torch.int32, device="cuda")
    moves = torch.zeros((9, 4), dtype=torch.int32, device="cuda")
    last = (LAST - 1) // P
    tf.tf_kv_pages_grow(refs, P, table, dev([LAST]), P + 5, moves, status=status)
    new = sorted({(LAST - P - 5) // P, last - 1, last})
    assert [j for j in range(stride - 4, stride) if int(table[0, j]) >= 0] == new and refs.tolist() == [1] * len(new) + [0] * (8 - len(new))
    tf.tf_kv_pages_free_window(refs, P, table, dev([LAST]), 1, 4, status=status)
    assert int((table >= 0).sum()) == (1 if LAST % P else 0) and int(status) == 0
    child, n = torch.full((1, stride), -9, dtype=torch.int32, device="cuda"), dev([0])
    tf.tf_kv_pages_fork(refs, P, table, dev([LAST]), dev([0]), child, n, status=status)
    assert torch.equal(child, table) and int(n) == LAST and int(status) == 0
    tf.tf_kv_pages_free(refs, P, child, status=status)
    tf.tf_kv_pages_compact(refs, P, table, moves, status=status)
    assert int(table[0, last]) == 0 and int(status) == 0 and refs.tolist() == [1] + [0] * 7
