"""Sliding-window attention with sinks against its definition in 64 bits (B200)."""
import functools
import math

import pytest
import torch

import window_ref

pytestmark = pytest.mark.gpu


TENSOR_CORE, CLUSTER = 1, 2


@functools.cache
def big_workspace():
    return torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")


class WindowCase:
    """Pools in which only the positions that some row sees hold numbers: every
    other slot is NaN, and the table entries of pages that no row sees name no
    page at all."""

    def __init__(self, lens, rows, window, sinks, d=128, Hkv=2, G=4, P=64, seed=0, edge=0.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.rows, self.window, self.sinks, self.scale = rows, window, sinks, 1.0 / math.sqrt(d)
        S = len(lens)
        self.max_len = max(lens)
        stride = -(-self.max_len // P)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q = r(S, rows, Hkv * G, d)
        self.table = torch.full((S, stride), -1, dtype=torch.int32)
        self.k, self.v, held = [], [], []
        for s, n in enumerate(lens):
            k, v = r(n, Hkv, d), r(n, Hkv, d)
            cols = window_ref.visible(n, rows, window, sinks, "cuda").any(0)
            if edge:
                # the first and last position of the window and of the sinks
                # weigh most, so that a row that misses one is far off
                for w in (0, rows - 1):
                    at = n - rows + w
                    for j in (at - window + 1, at, sinks - 1, 0):
                        if 0 <= j < n:
                            k[j] = (edge * self.q[s, w].float().view(Hkv, G, d).mean(1)).to(torch.bfloat16)
            k[~cols] = float("nan")
            v[~cols] = float("nan")
            self.k.append(k)
            self.v.append(v)
            held += [(s, j) for j in sorted({int(p) // P for p in cols.nonzero()[:, 0].tolist()})]
        n_pages = len(held) + 3
        ids = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        shape = (n_pages, Hkv, P, d)
        self.k_pool = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v_pool = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        for (s, j), page in zip(held, ids):
            self.table[s, j] = page
            lo, hi = j * P, min((j + 1) * P, lens[s])
            self.k_pool[page, :, :hi - lo] = self.k[s][lo:hi].transpose(0, 1)
            self.v_pool[page, :, :hi - lo] = self.v[s][lo:hi].transpose(0, 1)
        self.table = self.table.cuda()

    def call(self, window=None, sinks=None, max_len=None, out=None, ws=None, kernel=None):
        import verify_paged_gqa_b200 as tf
        window = self.window if window is None else window
        sinks = self.sinks if sinks is None else sinks
        max_len = self.max_len if max_len is None else max_len
        fn = (tf.tf_paged_attn_decode_window if self.rows == 1 else
              tf.tf_paged_attn_verify_window if self.rows <= 8 else tf.tf_paged_attn_prompt_window)
        if ws is None:
            ws = self.workspace(max_len)
        if kernel is not None:   # one of the two, whichever the library would take
            fn = lambda *a: tf.tf_testing_paged_attn_window(*a, kernel=kernel)  # noqa: E731
            ws = big_workspace()
        if out is None:
            out = torch.full(self.q.shape, float("nan"), dtype=torch.float32, device="cuda")
        fn(self.k_pool, self.v_pool, self.table, self.lens, self.q, window, sinks, self.scale, out, ws, max_len)
        status = tf.tf_workspace_status(ws)
        assert status == 0, hex(status)
        return out

    def workspace(self, max_len=None):
        import verify_paged_gqa_b200 as tf
        n = tf.tf_paged_attn_window_workspace_bytes(self.k_pool, self.v_pool, self.table, self.lens, self.q.shape[2],
                                                    self.rows, self.window, self.sinks, max_len or self.max_len)
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    def check(self, out):
        for s in range(len(self.k)):
            ref, bound = window_ref.attend(self.q[s], self.k[s], self.v[s], self.window, self.sinks, self.scale)
            off = (out[s].double() - ref).abs()
            assert torch.isfinite(out[s]).all(), s
            assert (off <= bound).all(), (s, float((off / bound).max()))


@pytest.mark.parametrize("d,G,P", [(128, 4, 64), (128, 8, 512), (128, 1, 37), (256, 4, 128), (256, 3, 16),
                                   (512, 4, 64), (512, 8, 200)])
@pytest.mark.parametrize("rows", [1, 2, 5, 8])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (100, 0), (130, 4), (333, 130), (257, 64)])
def test_short_windows(d, G, P, rows, window, sinks):
    lens = [rows, rows + window + sinks, 700 + rows, 1024, max(rows, window + sinks + 1), 1537]
    c = WindowCase(lens, rows, window, sinks, d=d, G=G, P=P, seed=d + G + P + rows + window + sinks, edge=0.5)
    c.check(c.call())
    c.check(c.call(kernel=TENSOR_CORE))
    c.check(c.call(kernel=CLUSTER))


@pytest.mark.parametrize("P", [512, 128, 100, 37, 5, 1])
@pytest.mark.parametrize("rows,G", [(9, 8), (40, 4), (100, 3), (300, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 4), (333, 5), (128, 129)])
def test_prompt_chunks(P, rows, G, window, sinks):
    lens = [rows, rows + 1000, max(rows, window + sinks), 641]
    c = WindowCase(lens, rows, window, sinks, G=G, P=P, seed=P + rows + window, edge=0.5)
    c.check(c.call())
    c.check(c.call(kernel=TENSOR_CORE))
    c.check(c.call(kernel=CLUSTER))


@pytest.mark.parametrize("d,rows", [(256, 64), (512, 33)])
def test_prompt_chunks_of_wide_heads(d, rows):
    c = WindowCase([rows, 900], rows, 200, 4, d=d, G=8, P=64, seed=d, edge=0.5)
    c.check(c.call(kernel=TENSOR_CORE))
    c.check(c.call(kernel=CLUSTER))


@pytest.mark.parametrize("rows,G,window,sinks,lens", [
    (64, 8, 6000, 4, [14000, 6100]), (700, 4, 5000, 4, [12000]), (8, 8, 9000, 130, [30000, 9200, 9130]),
    (1, 4, 4096, 4, [40960, 9000, 4100, 17]), (1, 8, 8192, 64, [32768, 8192, 8256, 8257]),
    (8, 8, 2048, 4, [20000, 2055, 131072]), (512, 4, 1024, 4, [9216, 600]), (1, 4, 30000, 1000, [40000, 31001])])
def test_long_contexts_over_many_cta_ranges(rows, G, window, sinks, lens):
    c = WindowCase(lens, rows, window, sinks, G=G, P=512, Hkv=2, seed=rows + window)
    c.check(c.call(kernel=TENSOR_CORE))
    c.check(c.call(kernel=CLUSTER))


def test_many_streams_and_repeated_runs_are_bitwise_equal():
    lens = [1 + (37 * i) % 900 for i in range(150)]
    c = WindowCase(lens, 1, 200, 4, P=64, Hkv=1, seed=5)
    for kernel in (TENSOR_CORE, CLUSTER):
        a = c.call(kernel=kernel)
        c.check(a)
        assert torch.equal(a, c.call(kernel=kernel))


@pytest.mark.parametrize("d", [128, 256, 512])
@pytest.mark.parametrize("rows", [1, 6, 64])
def test_a_window_past_every_length_sees_the_whole_context(d, rows):
    """The same set of positions, however it is said: equal outputs, bit for bit."""
    c = WindowCase([rows, 300 + rows, 1111], rows, 1 << 20, 0, d=d, seed=d + rows)
    for kernel in (TENSOR_CORE, CLUSTER):
        a = c.call(kernel=kernel)
        c.check(a)
        assert torch.equal(a, c.call(window=2 ** 31 - 1, sinks=2 ** 31 - 1, kernel=kernel))
        assert torch.equal(a, c.call(window=1, sinks=c.max_len, kernel=kernel))


@pytest.mark.parametrize("d,G,rows,window,lens", [
    (128, 8, 8, 900, [3000, 1308]), (128, 4, 1, 900, [3000, 1301]), (256, 8, 3, 900, [3000, 1303]), (512, 4, 4, 900, [3000, 1304]),
    (128, 4, 100, 900, [3000, 1400]), (128, 1, 3, 900, [3000]), (128, 4, 4, 2000, [3000, 1304]),
    # many tiles of one block: sums are folded, between and along with changes of reference
    (128, 8, 8, 6000, [9000] * 60), (256, 8, 8, 3000, [5000] * 40), (512, 8, 8, 2500, [4000] * 40), (128, 4, 300, 5000, [8000] * 4)])
def test_growing_scores(d, G, rows, window, lens):
    """K scaled up along the context: running maxima move many times."""
    c = WindowCase(lens, rows, window, 40, d=d, G=G, P=512, seed=rows + d)
    for s in range(len(lens)):
        ramp = (1.0 + 14.0 * torch.arange(c.k[s].shape[0], device="cuda") / c.k[s].shape[0])[:, None, None]
        c.k[s] = (c.k[s].float() * ramp).to(torch.bfloat16)
        for j, page in enumerate(c.table[s].tolist()):
            if page >= 0:
                rows_k = c.k[s][j * 512:(j + 1) * 512]
                c.k_pool[page, :, :rows_k.shape[0]] = rows_k.transpose(0, 1)
    c.check(c.call(kernel=TENSOR_CORE))
    c.check(c.call(kernel=CLUSTER))


@pytest.mark.parametrize("d,G,P,rows", [(128, 8, 512, 8), (512, 8, 64, 4), (128, 4, 37, 200)])
def test_a_withheld_arrival_times_out_and_the_next_call_is_clean(d, G, P, rows):
    """The tensor-core kernels' bounded waits, as in the plain calls' failure test."""
    import verify_paged_gqa_b200 as tf
    c = WindowCase([60000, 3000], rows, 20000, 4, d=d, G=G, P=P, Hkv=1, seed=d + rows)
    ws, out = big_workspace(), torch.zeros(c.q.shape, dtype=torch.float32, device="cuda")
    tf.tf_workspace_status(ws)
    tf.tf_testing_paged_attn_window(c.k_pool, c.v_pool, c.table, c.lens, c.q, 20000, 4, c.scale, out, ws, c.max_len,
                                    kernel=TENSOR_CORE, wait_limit_cycles=20_000_000, withhold=1)
    torch.cuda.synchronize()
    ws[4:8].zero_()
    assert tf.tf_workspace_status(ws) & tf.TF_DEV_TIMEOUT
    c.check(c.call(kernel=TENSOR_CORE))


def test_lengths_out_of_range_and_bad_pages_are_reported():
    import verify_paged_gqa_b200 as tf
    c = WindowCase([900, 1500], 1, 200, 4, P=64, seed=9)
    ws, out = c.workspace(1200), torch.zeros(c.q.shape, dtype=torch.float32, device="cuda")
    call = lambda: tf.tf_paged_attn_decode_window(c.k_pool, c.v_pool, c.table, c.lens, c.q, 200, 4, c.scale, out, ws, 1200)  # noqa: E731
    call()
    assert tf.tf_workspace_status(ws) == tf.TF_DEV_BAD_LEN
    assert torch.isnan(out[1]).all() and torch.isfinite(out[0]).all()
    c.table[0, 0] = c.k_pool.shape[0]   # the sinks' page
    call()
    assert tf.tf_workspace_status(ws) & tf.TF_DEV_BAD_PAGE


@pytest.mark.parametrize("d,G,rows,S,Hkv", [(128, 4, 300, 20, 2), (128, 8, 8, 170, 1), (128, 4, 40, 3, 2), (128, 2, 70, 300, 1),
                                           (256, 4, 8, 160, 1), (512, 4, 8, 5, 3), (512, 8, 4, 300, 1)])
@pytest.mark.parametrize("kernel", [0, TENSOR_CORE, CLUSTER])
def test_units_of_streams_out_of_range_among_others(d, G, rows, S, Hkv, kernel):
    """Fewer units than the GPU has CTAs, more, and many more; some streams too
    long, one too short, one of just the call's rows.  Nothing past the output
    is written."""
    import verify_paged_gqa_b200 as tf
    lens = [rows + (53 * i) % 400 for i in range(S)]
    c = WindowCase(lens, rows, 90, 4, d=d, G=G, P=64, Hkv=Hkv, seed=S + d)
    bad = {0: 2000, S // 2: rows - 1, S - 1: -5}
    for s, n in bad.items():
        c.lens[s] = n
    flat = torch.full((c.q.numel() + 4096,), 7.0, dtype=torch.float32, device="cuda")
    out, ws = flat[:c.q.numel()].view(c.q.shape), big_workspace()
    tf.tf_testing_paged_attn_window(c.k_pool, c.v_pool, c.table, c.lens, c.q, 90, 4, c.scale, out, ws, c.max_len, kernel=kernel)
    assert tf.tf_workspace_status(ws) == tf.TF_DEV_BAD_LEN
    assert bool((flat[c.q.numel():] == 7.0).all())
    for s in bad:
        assert torch.isnan(out[s]).all()
    for s in set(range(S)) - set(bad):
        ref, bound = window_ref.attend(c.q[s], c.k[s], c.v[s], 90, 4, c.scale)
        assert ((out[s].double() - ref).abs() <= bound).all(), s


def test_refusals_that_need_the_device():
    import verify_paged_gqa_b200 as tf
    c = WindowCase([900, 1500], 1, 200, 4, P=64, seed=9)
    out, ws = torch.zeros(c.q.shape, dtype=torch.float32, device="cuda"), c.workspace()
    call = lambda scale, ws: tf.tf_paged_attn_decode_window(c.k_pool, c.v_pool, c.table, c.lens, c.q, 200, 4, scale, out, ws, 1500)  # noqa: E731
    for scale, w, want in ((float("nan"), ws, tf.TF_EINVAL), (float("inf"), ws, tf.TF_EINVAL), (0.1, ws[:-16], tf.TF_ENOSPACE)):
        with pytest.raises(tf.TFError) as e:
            call(scale, w)
        assert e.value.status == want
    assert not out.any()


def test_a_captured_call_follows_the_lengths():
    import verify_paged_gqa_b200 as tf
    c = WindowCase([1500, 1200, 700], 1, 400, 4, P=64, seed=11)
    c.window = 300   # the pool holds 100 positions more than the calls see
    out, ws = torch.empty(c.q.shape, dtype=torch.float32, device="cuda"), c.workspace()
    call = lambda: tf.tf_paged_attn_decode_window(c.k_pool, c.v_pool, c.table, c.lens, c.q, 300, 4, c.scale, out, ws, 1500)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    full = (c.lens.clone(), c.k, c.v)
    for back in (0, 1, 63, 64, 99):
        c.lens.copy_(full[0] - back)
        c.k, c.v = ([t[:len(t) - back] for t in kv] for kv in full[1:])
        out.fill_(float("nan"))
        graph.replay()
        c.check(out)
    assert tf.tf_workspace_status(ws) == 0


@pytest.mark.parametrize("d,G,rows,S,Hkv", [(128, 4, 40, 3, 2), (128, 4, 120, 30, 2), (128, 8, 8, 160, 1), (512, 4, 8, 5, 3)])
def test_captured_tensor_core_calls_follow_the_lengths(d, G, rows, S, Hkv):
    """Units in pieces and whole ones, replayed with shorter streams."""
    import verify_paged_gqa_b200 as tf
    c = WindowCase([500 + rows + (29 * i) % 300 for i in range(S)], rows, 400, 4, d=d, G=G, P=64, Hkv=Hkv, seed=d + S)
    c.window = 300   # the pool holds 100 positions more than the calls see
    out, ws = torch.empty(c.q.shape, dtype=torch.float32, device="cuda"), big_workspace()
    call = lambda: tf.tf_testing_paged_attn_window(c.k_pool, c.v_pool, c.table, c.lens, c.q, 300, 4, c.scale, out, ws, c.max_len, kernel=TENSOR_CORE)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    full = (c.lens.clone(), c.k, c.v)
    for back in (0, 1, 64, 99):
        c.lens.copy_(full[0] - back)
        c.k, c.v = ([t[:len(t) - back] for t in kv] for kv in full[1:])
        out.fill_(float("nan"))
        graph.replay()
        c.check(out)
    assert tf.tf_workspace_status(ws) == 0


def test_another_stream_and_two_workspaces():
    a = WindowCase([2000, 900], 8, 500, 4, G=8, seed=21)
    b = WindowCase([1800, 400], 1, 700, 0, d=256, seed=22)
    outs = [torch.empty(c.q.shape, dtype=torch.float32, device="cuda") for c in (a, b)]
    wss = [a.workspace(), b.workspace()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for c, o, w, st in zip((a, b), outs, wss, streams):
            with torch.cuda.stream(st):
                c.call(out=o, ws=w)
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])
