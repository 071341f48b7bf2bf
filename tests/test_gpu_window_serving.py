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


def test_pages_past_offsets_of_32_bits():
    """Pools of more than 2^32 values each (8.6 GB): rows are written, attended
    to and moved at both ends."""
    import verify_paged_gqa_b200 as tf
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    P, Hkv, G, d, n = 512, 8, 4, 128, 700
    n_pages = 2 ** 32 // (P * Hkv * d) + 8
    kp, vp = (torch.empty((n_pages, Hkv, P, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kp.numel() > 2 ** 32
    ids = [[n_pages - 1, 0], [1, n_pages - 2]]
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    for page in sum(ids, []):
        refs[page] = 1
    table, lens = dev(ids), dev([n, n])
    k, v = (torch.randn(2, n, Hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pos = torch.zeros(2, n, 1, dtype=torch.int32, device="cuda")     # the turn by 0 keeps every bit
    tf.tf_kv_put_rows_rope(kp, vp, table, lens, None, k, v, pos, tf.Rope(torch.ones(d // 2, device="cuda")), n)
    ws, moves = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda"), torch.zeros((1 + n_pages // 2, 4), dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn(2, 8, Hkv * G, d, generator=g, device="cuda").to(torch.bfloat16)

    def attend():
        for kernel in (1, 2):
            out = tf.tf_testing_paged_attn_window(kp, vp, table, lens, q, 300, 4, 0.1, torch.empty(q.shape, dtype=torch.float32, device="cuda"),
                                                  ws, n, kernel=kernel)
            for s in range(2):
                ref, bound = window_ref.attend(q[s], k[s], v[s], 300, 4, 0.1)
                assert ((out[s].double() - ref).abs() <= bound).all()
    attend()
    tf.tf_kv_pages_compact(refs, P, table, moves, status=status)
    tf.tf_kv_pages_move(kp, vp, moves, status=status)
    assert moves[0].tolist() == [2, 4, 0, 0] and table.tolist() == [[3, 0], [1, 2]]
    attend()
    # and out to the far end
    moves[0, 0] = 1
    moves[1] = dev([3, n_pages - 3, P, 0])
    tf.tf_kv_pages_move(kp, vp, moves, status=status)
    table[0, 0] = n_pages - 3
    kp[3] = float("nan")
    attend()
    assert int(status) == 0 and tf.tf_workspace_status(ws) == 0


FIRST_CALL = """
import torch, verify_paged_gqa_b200 as tf
i32 = dict(dtype=torch.int32, device="cuda")
kp, vp = (torch.randn(8, 2, 64, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
table, lens, ws = torch.arange(8, **i32).view(2, 4), torch.full((2,), 200, **i32), torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")
refs, moves, status = torch.ones(8, **i32), torch.zeros((16, 4), **i32), torch.zeros(1, **i32)
rope, pos = tf.Rope(torch.ones(64, device="cuda")), torch.ones((2, {rows}, 1), **i32)
qkv = torch.randn(2, {rows}, 12, 128, device="cuda").to(torch.bfloat16)
q_out = torch.zeros((2, {rows}, 8, 128), dtype=torch.bfloat16, device="cuda")
out = torch.zeros((2, {rows}, 8, 128), device="cuda")
def step():
    tf.tf_kv_pages_grow(refs, 64, table, lens, {rows}, moves, status=status)
    tf.tf_kv_pages_move(kp, vp, moves, status=status)
    tf.tf_kv_put_rows_rope(kp, vp, table, lens, qkv[:, :, :8], qkv[:, :, 8:10], qkv[:, :, 10:], pos, rope, 256, q_out=q_out)
    tf.tf_testing_paged_attn_window(kp, vp, table, lens, q_out, 100, 4, 0.1, out, ws, 256, kernel={kernel})
    tf.tf_kv_pages_compact(refs, 64, table, moves, status=status)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
got = out.clone()
out.zero_()
step()
assert bool(got.any()) and torch.equal(got, out)
assert int(status) == 0 and tf.tf_workspace_status(ws) == 0
"""


@pytest.mark.parametrize("rows,kernel", [(1, 2), (8, 1), (100, 1)])
def test_the_first_calls_of_a_process_may_be_captured(rows, kernel):
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(rows=rows, kernel=kernel)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
