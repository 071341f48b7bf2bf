"""One workspace, sized once from the largest shape a program runs, serves
every smaller call (B200)."""
import ctypes
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

PTR = 1 << 12   # an aligned address; sizing reads no buffer


def window_bytes(d, Hkv, G, S, rows, max_len, window, sinks, P=512):
    import verify_paged_gqa_b200._abi as lib
    pool = lib.tf_kv_pool(PTR, PTR, 64, Hkv, P, d)
    st = lib.tf_streams(PTR, -(-max_len // P), PTR, S, max_len)
    n = lib.raw.tf_paged_attn_window_workspace_bytes(ctypes.byref(pool), ctypes.byref(st), Hkv * G, rows, window, sinks)
    assert n > 0
    return n


@pytest.mark.parametrize("d", [128, 256, 512])
@pytest.mark.parametrize("Hkv,G", [(2, 8), (1, 1), (8, 4), (3, 5)])
@pytest.mark.parametrize("rows", [1, 8, 100])
def test_window_workspace_of_the_largest_shape_holds_every_smaller_one(d, Hkv, G, rows):
    most = window_bytes(d, Hkv, G, 64, rows, 9000, 4096, 4)
    for S, r, n, window, sinks in itertools.product((1, 2, 4, 8, 16, 31, 64), sorted({1, 2, rows // 2 or 1, rows}),
                                                    (rows, 300, 2048, 9000), (1, 500, 4096, 1 << 20), (0, 4, 130)):
        if r <= rows and n >= r:
            assert window_bytes(d, Hkv, G, S, r, n, window, sinks) <= most, (S, r, n, window, sinks)


@pytest.mark.parametrize("d,P,most,calls", [
    (512, 64, (64, 1), [(64, 1), (8, 1), (4, 1), (1, 1)]),
    (256, 512, (32, 8), [(32, 8), (5, 8), (2, 3), (32, 1)]),
    (128, 37, (8, 200), [(8, 200), (1, 200), (3, 60), (8, 12), (1, 1)])])
def test_smaller_window_calls_run_in_it(d, P, most, calls):
    """Every stream reads the same pages: the calls' sizes count here."""
    import verify_paged_gqa_b200 as tf
    Hkv, G, L, window, sinks = 2, 8, 5000, 4096, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    n_pages = -(-L // P)
    kp, vp = r(n_pages, Hkv, P, d), r(n_pages, Hkv, P, d)
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(d)).to(torch.int32).cuda()

    def streams(S):
        return table.expand(S, n_pages).contiguous(), (L - torch.arange(S, device="cuda", dtype=torch.int32))

    ws = torch.zeros(tf.tf_paged_attn_window_workspace_bytes(kp, vp, *streams(most[0]), Hkv * G, most[1], window, sinks, L),
                     dtype=torch.uint8, device="cuda")
    big = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    for S, rows in calls:
        t, n = streams(S)
        q = r(S, rows, Hkv * G, d)
        fn = (tf.tf_paged_attn_decode_window if rows == 1 else
              tf.tf_paged_attn_verify_window if rows <= 8 else tf.tf_paged_attn_prompt_window)
        outs = [fn(kp, vp, t, n, q, window, sinks, d ** -0.5, torch.empty(q.shape, dtype=torch.float32, device="cuda"), w, L)
                for w in (ws, big)]
        assert torch.isfinite(outs[0]).all() and torch.equal(*outs), (S, rows)
    assert tf.tf_workspace_status(ws) == 0


def plain_bytes(d, Hkv, G, S, rows, max_len, P=512):
    import verify_paged_gqa_b200._abi as lib
    pool = lib.tf_kv_pool(PTR, PTR, 64, Hkv, P, d)
    st = lib.tf_streams(PTR, -(-max_len // P), PTR, S, max_len)
    n = lib.raw.tf_paged_attn_workspace_bytes(ctypes.byref(pool), ctypes.byref(st), Hkv * G, rows)
    assert n > 0
    return n


@pytest.mark.parametrize("d", [128, 256, 512])
@pytest.mark.parametrize("Hkv,G", [(2, 8), (8, 4), (3, 5)])
@pytest.mark.parametrize("rows", [1, 8, 448, 1000])
def test_workspace_of_the_largest_shape_holds_every_smaller_one(d, Hkv, G, rows):
    most = plain_bytes(d, Hkv, G, 16, rows, 9000)
    for S, r, n in itertools.product((1, 2, 4, 9, 16), sorted({1, 2, 8, 60, rows // 2 or 1, rows}), (rows, 300, 2048, 9000)):
        if r <= rows and n >= r:
            assert plain_bytes(d, Hkv, G, S, r, n) <= most, (S, r, n)


def test_a_shorter_prompt_chunk_runs_in_the_workspace_of_a_longer_one():
    """112 row blocks of 128 rows are taken whole, one to a CTA; 104 are split
    over all CTAs, whose partials take more room."""
    import verify_paged_gqa_b200 as tf
    Hkv, G, L = 8, 4, 2048
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    kp, vp = r(4, Hkv, 512, 128), r(4, Hkv, 512, 128)
    table, lens = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32, device="cuda"), torch.tensor([L], dtype=torch.int32, device="cuda")
    ws = torch.zeros(tf.tf_paged_attn_workspace_bytes(kp, vp, table, lens, Hkv * G, 14 * 32, L), dtype=torch.uint8, device="cuda")
    for rows in (14 * 32, 13 * 32, 100, 9, 4, 1):
        q = r(1, rows, Hkv * G, 128)
        fn = tf.tf_paged_attn_decode if rows == 1 else tf.tf_paged_attn_verify if rows <= 8 else tf.tf_paged_attn_prompt
        out = fn(kp, vp, table, lens, q, 128 ** -0.5, torch.empty(q.shape, dtype=torch.float32, device="cuda"), ws, L)
        assert torch.isfinite(out).all(), rows
    assert tf.tf_workspace_status(ws) == 0
