"""The operators together, as a sliding-window layer of a serving loop runs
them (B200): streams grow page by page, rows are turned and written, attended
over the window, pages behind it are freed, streams are forked and dropped and
the pool is compacted; every output against attention over linear caches that
no page operator ever touched, in 64 bits."""
import math
import random

import numpy as np
import pytest
import torch

import window_ref

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d,P,window,sinks,seed", [(128, 16, 40, 4, 0), (128, 64, 100, 0, 1), (256, 37, 90, 40, 2), (512, 16, 33, 1, 3)])
def test_a_window_layer_of_a_serving_loop(d, P, window, sinks, seed):
    import verify_paged_gqa_b200 as tf
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    Hkv, G, S, stride, axes = 2, 4, 5, 1024 // P, 3
    scale = 1.0 / math.sqrt(d)
    n_pages = S * (-(-(window + sinks + 80) // P) + 4)      # far fewer than S * stride
    kp, vp = (torch.full((n_pages, Hkv, P, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    refs, status = torch.zeros(n_pages, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    tables = [torch.full((S, stride), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    moves = torch.zeros((1 + n_pages * 8, 4), dtype=torch.int32, device="cuda")
    inv = torch.from_numpy((10000.0 ** (-np.arange(d // 2) * 2.0 / d)).astype(np.float32)).cuda()
    rope = tf.Rope(inv, [i % axes for i in range(d // 2)], axes)
    lens = [0] * S
    linear = [(torch.zeros(0, Hkv, d, dtype=torch.bfloat16, device="cuda"),) * 2 for _ in range(S)]
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")

    for step in range(24):
        rows = rng.choice([1, 1, 1, 3, 8, 60]) if step else 60
        lens = [n + rows for n in lens]
        if max(lens) > stride * P:
            break
        table, d_lens = tables[0], dev(lens)
        tf.tf_kv_pages_grow(refs, P, table, d_lens, rows, moves, status=status)
        tf.tf_kv_pages_move(kp, vp, moves, status=status)
        qkv = torch.randn(S, rows, Hkv * (G + 2), d, generator=g, device="cuda").to(torch.bfloat16)
        pos = torch.randint(0, 5000, (S, rows, axes), generator=g, device="cuda", dtype=torch.int32)
        k_rows, v_rows = qkv[:, :, Hkv * G:Hkv * (G + 1)], qkv[:, :, Hkv * (G + 1):]
        q = tf.tf_kv_put_rows_rope(kp, vp, table, d_lens, qkv[:, :, :Hkv * G], k_rows, v_rows, pos, rope, max(lens))
        # the linear caches take the turned keys as the pages hold them
        lin_pool = tuple(torch.zeros((S, Hkv, rows, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        tf.tf_kv_put_rows_rope(*lin_pool, torch.arange(S, dtype=torch.int32, device="cuda")[:, None].contiguous(), dev([rows] * S),
                               None, k_rows, v_rows, pos, rope, rows)
        linear = [tuple(torch.cat([old, new[s].transpose(0, 1)]) for old, new in zip(linear[s], lin_pool)) for s in range(S)]
        fn = tf.tf_paged_attn_decode_window if rows == 1 else tf.tf_paged_attn_verify_window if rows <= 8 else tf.tf_paged_attn_prompt_window
        out = fn(kp, vp, table, d_lens, q, window, sinks, scale, torch.empty(q.shape, dtype=torch.float32, device="cuda"), ws, max(lens))
        for s in range(S):
            ref, bound = window_ref.attend(q[s], *linear[s], window, sinks, scale)
            assert ((out[s].double() - ref).abs() <= bound).all(), (step, s)
        tf.tf_kv_pages_free_window(refs, P, table, d_lens, window, sinks, status=status)
        if step % 3 == 1:   # beams are reordered: some go on twice, others end
            parents = [rng.randrange(S) for _ in range(S)]
            new_lens = torch.empty(S, dtype=torch.int32, device="cuda")
            tf.tf_kv_pages_fork(refs, P, table, d_lens, dev(parents), tables[1], new_lens, status=status)
            tf.tf_kv_pages_free(refs, P, table, status=status)
            tables.reverse()
            lens = [lens[p] for p in parents]
            linear = [linear[p] for p in parents]
            assert new_lens.tolist() == lens
        if step % 4 == 2:
            tf.tf_kv_pages_compact(refs, P, tables[0], moves, status=status)
            tf.tf_kv_pages_move(kp, vp, moves, status=status)
            live = int((refs > 0).sum())
            assert int(tables[0].max()) < live and not bool((refs[live:] > 0).any())
        # every page's holders are the table's entries
        held = tables[0][tables[0] >= 0].long()
        assert torch.equal(torch.bincount(held, minlength=n_pages).int(), refs)
        assert int(status) == 0, int(status)
        assert tf.tf_workspace_status(ws) == 0
    assert step > 8
