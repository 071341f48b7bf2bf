"""The row write with rotary positions against its definition in 64 bits (B200).

A turned value is a cos t - b sin t with fp32 cos, sin and products (each to
2^-22 of its size, the angle's own rounding to half turns included) and one
rounding to bf16: it is within |a| 2^-20 + |b| 2^-20 + half a bf16 step of the
exact value, 2^-8 of it (and the smallest bf16 spacing, for results that
underflow)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


class RopeCase:
    def __init__(self, S, W, Hkv, G, d, P, rotary, axes, adjacent, seed, far=4096, fused=True, axis_of=None):
        import verify_paged_gqa_b200 as tf
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.S, self.W, self.P = S, W, P
        Hq = Hkv * G
        lens = rng.integers(W, W + 3 * P + 5, S).astype(np.int32)
        self.max_len = int(lens.max())
        stride = -(-self.max_len // P)
        n_pages = S * stride + 2
        self.table = torch.from_numpy(rng.permutation(n_pages)[:S * stride].reshape(S, stride).astype(np.int32)).cuda()
        self.lens = torch.from_numpy(lens).cuda()
        r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.k_pool, self.v_pool = r(n_pages, Hkv, P, d), r(n_pages, Hkv, P, d)
        if fused:
            qkv = r(S, W, Hq + 2 * Hkv, d)
            self.q, self.k, self.v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        else:
            self.q, self.k, self.v = r(S, W, Hq, d), r(S, W, Hkv, d), r(S, W, Hkv, d)
        half = rotary // 2
        self.axis = [(i * 7 + 3) % axes for i in range(half)] if axis_of is None else axis_of
        self.positions = torch.from_numpy(rng.integers(-far, far + 1, (S, W, axes)).astype(np.int32)).cuda()
        self.inv_freq = torch.from_numpy((10000.0 ** (-np.arange(half) * 2.0 / rotary)).astype(np.float32)).cuda()
        self.rotary, self.adjacent = rotary, adjacent
        self.rope = tf.Rope(self.inv_freq, self.axis, axes, adjacent=adjacent)

    def turned(self, x):
        """Exact values of the turned rows, and how far a result may be off."""
        half = self.rotary // 2
        x = x.double()
        t = self.positions.double()[..., torch.tensor(self.axis, device="cuda")] * self.inv_freq.double()
        c, s = torch.cos(t)[:, :, None], torch.sin(t)[:, :, None]
        y, room = x.clone(), torch.zeros_like(x)
        ia, ib = (slice(0, self.rotary, 2), slice(1, self.rotary, 2)) if self.adjacent else (slice(0, half), slice(half, self.rotary))
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        room[..., ia] = room[..., ib] = (a.abs() + b.abs()) * 2.0 ** -20
        room[..., :self.rotary] += y[..., :self.rotary].abs() * 2.0 ** -8 + 2.0 ** -133
        return y, room

    def check(self, call=None):
        import verify_paged_gqa_b200 as tf
        want_q, room_q = self.turned(self.q)
        want_k, room_k = self.turned(self.k)
        before = self.k_pool.clone(), self.v_pool.clone()
        q = (call or (lambda: tf.tf_kv_put_rows_rope(self.k_pool, self.v_pool, self.table, self.lens, self.q, self.k, self.v,
                                                     self.positions, self.rope, self.max_len)))()
        assert ((q.double() - want_q).abs() <= room_q).all()
        touched = torch.zeros(self.k_pool.shape[0], self.P, dtype=torch.bool, device="cuda")
        for s in range(self.S):
            n = int(self.lens[s])
            for r in range(self.W):
                pos = n - self.W + r
                page, slot = int(self.table[s, pos // self.P]), pos % self.P
                assert ((self.k_pool[page, :, slot].double() - want_k[s, r]).abs() <= room_k[s, r]).all()
                assert torch.equal(self.v_pool[page, :, slot], self.v[s, r])
                touched[page, slot] = True
        keep = ~touched[:, None, :, None].expand_as(self.k_pool)
        assert torch.equal(self.k_pool[keep], before[0][keep]) and torch.equal(self.v_pool[keep], before[1][keep])
        return q


@pytest.mark.parametrize("d,rotary", [(128, 128), (128, 64), (128, 2), (128, 90), (256, 256), (256, 18), (512, 512), (512, 16),
                                      (512, 250)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("axes,W,P", [(1, 1, 512), (3, 1, 37), (3, 7, 16), (4, 40, 5)])
def test_rows_turned_and_written(d, rotary, adjacent, axes, W, P):
    RopeCase(3, W, 2, 3, d, P, rotary, axes, adjacent, seed=d + rotary + W).check()


@pytest.mark.parametrize("d,rotary,adjacent", [(128, 128, False), (128, 64, True), (512, 208, False)])
def test_rows_that_fill_the_gpu(d, rotary, adjacent):
    """From 4,096 rows on a warp takes a row: the same bits as row by row."""
    import verify_paged_gqa_b200 as tf
    c = RopeCase(3, 1500, 2, 3, d, 64, rotary, 3, adjacent, seed=d)
    q = tf.tf_kv_put_rows_rope(c.k_pool, c.v_pool, c.table, c.lens, c.q, c.k, c.v, c.positions, c.rope, c.max_len)
    want, room = c.turned(c.q)
    assert ((q.double() - want).abs() <= room).all()
    pools = torch.zeros_like(c.k_pool), torch.zeros_like(c.v_pool)
    for s in range(3):
        one = tf.tf_kv_put_rows_rope(*pools, c.table[s:s + 1], c.lens[s:s + 1], c.q[s:s + 1], c.k[s:s + 1], c.v[s:s + 1],
                                     c.positions[s:s + 1], c.rope, c.max_len)
        assert torch.equal(one[0], q[s])
        n = int(c.lens[s])
        pos = torch.arange(n - 1500, n, device="cuda")
        page, slot = c.table[s].long()[pos // 64], pos % 64
        for a, b in zip((c.k_pool, c.v_pool), pools):
            assert torch.equal(a[page, :, slot], b[page, :, slot])


@pytest.mark.parametrize("far", [0, 1 << 20, 2 ** 31 - 1])
def test_far_positions(far):
    RopeCase(4, 5, 1, 4, 128, 64, 128, 3, False, seed=far % 1000, far=far).check()


def test_sections_and_separate_rows():
    RopeCase(2, 9, 2, 4, 128, 64, 128, 3, False, seed=3, fused=False, axis_of=[0] * 16 + [1] * 24 + [2] * 24).check()


@pytest.mark.parametrize("rotary,adjacent", [(128, False), (128, True), (90, False), (90, True)])
def test_in_place_queries(rotary, adjacent):
    import verify_paged_gqa_b200 as tf
    c = RopeCase(3, 33, 2, 4, 128, 64, rotary, 3, adjacent, seed=rotary, fused=False)
    c.check(lambda: tf.tf_kv_put_rows_rope(c.k_pool, c.v_pool, c.table, c.lens, c.q, c.k, c.v, c.positions, c.rope, c.max_len,
                                           q_out=c.q))


def test_keys_alone_and_a_captured_call():
    import verify_paged_gqa_b200 as tf
    c = RopeCase(5, 2, 2, 4, 128, 64, 128, 3, False, seed=8)
    other = RopeCase(5, 2, 2, 4, 128, 64, 128, 3, False, seed=8)
    assert tf.tf_kv_put_rows_rope(c.k_pool, c.v_pool, c.table, c.lens, None, c.k, c.v, c.positions, c.rope, c.max_len) is None
    other.check()
    assert torch.equal(c.k_pool, other.k_pool) and torch.equal(c.v_pool, other.v_pool)
    q_out = torch.empty(c.q.shape, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tf.tf_kv_put_rows_rope(c.k_pool, c.v_pool, c.table, c.lens, c.q, c.k, c.v, c.positions, c.rope, c.max_len, q_out=q_out)
    c.positions.add_(17)
    c.check(lambda: (graph.replay(), q_out)[1])


def test_rows_out_of_range_are_skipped_and_kept_dims_keep_their_bits():
    import verify_paged_gqa_b200 as tf
    c = RopeCase(4, 3, 1, 2, 128, 64, 64, 1, False, seed=12)
    c.q[..., 64:] = float("nan")
    c.k[..., 64:] = float("inf")
    c.lens[0] = 2                      # fewer positions than rows
    c.lens[1] = c.max_len + 1
    c.table[2] = -1
    c.table[3] = c.k_pool.shape[0]
    before = c.k_pool.clone(), c.v_pool.clone()
    want, room = c.turned(c.q[..., :64])
    q = tf.tf_kv_put_rows_rope(c.k_pool, c.v_pool, c.table, c.lens, c.q, c.k, c.v, c.positions, c.rope, c.max_len)
    assert torch.equal(before[0], c.k_pool) and torch.equal(before[1], c.v_pool)
    assert ((q[..., :64].double() - want).abs() <= room).all()
    assert torch.equal(q[..., 64:].view(torch.int16), c.q[..., 64:].contiguous().view(torch.int16))


def test_same_angle_turns_a_dot_product_into_a_difference_of_positions():
    """Rows turned by p and q keep a dot product that depends on p - q alone."""
    import verify_paged_gqa_b200 as tf
    c = RopeCase(1, 2, 1, 1, 128, 64, 128, 1, False, seed=4)
    x = torch.randn(128, device="cuda").to(torch.bfloat16)
    dots = []
    for base in (0, 1000, 500000):
        c.q[:] = x
        c.positions[0, :, 0] = torch.tensor([base, base + 9], device="cuda")
        q = tf.tf_kv_put_rows_rope(c.k_pool, c.v_pool, c.table, c.lens, c.q, c.k, c.v, c.positions, c.rope, c.max_len)
        dots.append(float(q[0, 0, 0].double() @ q[0, 1, 0].double()))
    norm = float(x.double() @ x.double())
    # each factor is off by at most 2^-8 of its size: 2 * 2^-8 of the norm, twice
    assert max(dots) - min(dots) <= 4 * 2.0 ** -8 * norm
    assert math.isfinite(norm)
