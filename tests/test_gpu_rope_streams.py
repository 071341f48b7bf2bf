"""The row write with rotary positions on a stream of its own (B200)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", ["stream", "pointer"])
def test_new_queries_take_no_memory_that_another_stream_still_reads(handle):
    """A freed block is handed out again in the order of the stream it belongs
    to: turned queries that are written on another stream must not be one."""
    import verify_paged_gqa_b200 as tf
    S, Hkv, G, d = 64, 2, 4, 128
    pool = torch.zeros((S, Hkv, 16, d), dtype=torch.bfloat16, device="cuda")
    table = torch.arange(S, dtype=torch.int32, device="cuda")[:, None].contiguous()
    lens = torch.full((S,), 5, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    r = lambda h: torch.randn((S, 1, h, d), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = r(Hkv * G), r(Hkv), r(Hkv)
    pos = torch.full((S, 1, 1), 7, dtype=torch.int32, device="cuda")
    rope = tf.Rope(torch.linspace(1, 0.1, d // 2, device="cuda"))
    side = torch.cuda.Stream()
    want = tf.tf_kv_put_rows_rope(pool, pool.clone(), table, lens, q, k, v, pos, rope, 16)
    saved = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        x = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
        torch.cuda._sleep(100_000_000)      # about 50 ms of this stream
        saved.copy_(x)                      # x is read after that
        del x
        got = tf.tf_kv_put_rows_rope(pool, pool, table, lens, q, k, v, pos, rope, 16,
                                     stream=side if handle == "stream" else side.cuda_stream)
        torch.cuda.synchronize()
        assert bool((saved == 3.0).all())
        assert torch.equal(got, want)


def test_the_legacy_default_stream_by_its_handle():
    import verify_paged_gqa_b200 as tf
    pool = torch.zeros((1, 1, 16, 128), dtype=torch.bfloat16, device="cuda")
    one = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    row = torch.ones((1, 1, 1, 128), dtype=torch.bfloat16, device="cuda")
    rope = tf.Rope(torch.zeros(64, device="cuda"))
    for side in (None, torch.cuda.Stream()):
        with torch.cuda.stream(side):
            torch.cuda.synchronize()
            q = tf.tf_kv_put_rows_rope(pool, pool, one, one[0] + 1, row, row, row, one[:, :, None].contiguous(), rope, 16, stream=0)
            torch.cuda.synchronize()
            assert torch.equal(q, row)
