"""Forking, growing, freeing and compacting the cache's pages (B200): whole
numbers and copied bits, equal to the plain bookkeeping's."""
import random

import pytest
import torch

import pages_ref

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Cache:
    """One pool's pages on the GPU, and the same in plain Python beside it."""

    def __init__(self, n_pages, P, rows, stride, Hkv=2, d=128, seed=0):
        self.P, self.stride = P, stride
        self.refs, self.table = [0] * n_pages, [[-1] * stride for _ in range(rows)]
        self.lens = [0] * rows
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        bits = lambda: torch.randint(-2 ** 15, 2 ** 15, (n_pages, Hkv, P, d), dtype=torch.int16, device="cuda", generator=g)  # noqa: E731
        self.k, self.v = bits(), bits()
        self.push()

    def push(self):
        self.d_refs, self.d_table, self.d_lens = dev(self.refs), dev(self.table), dev(self.lens)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.moves = torch.full((1 + max(len(self.refs), 64), 4), -7, dtype=torch.int32, device="cuda")

    def fill(self, rng, share=0.0):
        """Random lengths; pages drawn in random order, some shared by neighbours."""
        ids = list(range(len(self.refs)))
        rng.shuffle(ids)
        for s in range(len(self.table)):
            n = rng.randint(0, self.stride * self.P)
            self.lens[s] = n
            for j in range(-(-n // self.P)):
                prev = self.table[s - 1][j] if s else -1
                if prev >= 0 and rng.random() < share:
                    self.table[s][j] = prev
                elif ids:
                    self.table[s][j] = ids.pop()
                else:
                    self.lens[s] = j * self.P
                    break
                self.refs[self.table[s][j]] += 1
        self.push()

    def same(self, status=0):
        assert self.d_refs.tolist() == self.refs
        assert self.d_table.tolist() == self.table
        assert int(self.status) == status
        self.status.zero_()

    def pools(self):
        return self.k.view(torch.bfloat16), self.v.view(torch.bfloat16)

    def move(self, moves):
        """The list's moves on the GPU, against the plain ones."""
        import verify_paged_gqa_b200 as tf
        want = self.k.clone(), self.v.clone()
        for p in want:
            pages_ref.move(p, moves)
        tf.tf_kv_pages_move(*self.pools(), self.moves, status=self.status)
        assert torch.equal(self.k, want[0]) and torch.equal(self.v, want[1])

    def list(self):
        n = int(self.moves[0, 0])
        return [tuple(m[:3]) for m in self.moves[1:1 + n].tolist()]


@pytest.mark.parametrize("P", [1, 16, 37, 512])
@pytest.mark.parametrize("seed", range(3))
def test_fork_free_and_grow_against_the_plain_bookkeeping(P, seed):
    import verify_paged_gqa_b200 as tf
    rng = random.Random(100 * P + seed)
    S, N, stride = rng.randint(1, 40), rng.randint(1, 60), rng.randint(2, 9)
    c = Cache(S * stride + 5 * N + 8, P, S, stride, seed=seed)
    c.fill(rng, share=0.5)
    parents = [rng.randint(-1, S - 1) for _ in range(N)]
    d_stride = stride + rng.randint(1, 3)
    new, new_lens = torch.full((N, d_stride), -9, dtype=torch.int32, device="cuda"), torch.full((N,), -9, dtype=torch.int32, device="cuda")
    tf.tf_kv_pages_fork(c.d_refs, P, c.d_table, c.d_lens, dev(parents), new, new_lens, status=c.status)
    table, lens = pages_ref.fork(c.refs, P, c.table, c.lens, parents, d_stride)
    c.same()
    assert new.tolist() == table and new_lens.tolist() == lens
    # the parents go
    tf.tf_kv_pages_free(c.d_refs, P, c.d_table, status=c.status)
    pages_ref.free(c.refs, c.table)
    c.same()
    # the children grow, by one position or several pages
    rows = rng.choice([1, 2, P, min(2 * P + 1, d_stride * P - stride * P + 1)])
    lens = [min(n + rows, d_stride * P) if n else 0 for n in lens]
    lens = [n if n >= rows else 0 for n in lens]
    moves = pages_ref.grow(c.refs, P, table, lens, rows)
    c.moves = torch.full((1 + N * ((rows + P - 2) // P + 1), 4), -7, dtype=torch.int32, device="cuda")
    tf.tf_kv_pages_grow(c.d_refs, P, new, dev(lens), rows, c.moves, status=c.status)
    assert moves is not None
    c.same()
    assert new.tolist() == table and c.list() == moves
    c.move(moves)
    # and drop a part: the first entries, the last ones
    first = [rng.randint(0, d_stride) for _ in lens]
    end = [rng.randint(0, d_stride) for _ in lens]
    tf.tf_kv_pages_free(c.d_refs, P, new, dev(first), dev(end), status=c.status)
    pages_ref.free(c.refs, table, first, end)
    c.same()
    assert new.tolist() == table


@pytest.mark.parametrize("P,window,sinks", [(1, 1, 0), (16, 1, 0), (16, 40, 4), (37, 100, 40), (64, 64, 64), (64, 65, 1), (512, 5000, 4)])
def test_free_behind_a_window(P, window, sinks):
    import verify_paged_gqa_b200 as tf
    rng = random.Random(P + window)
    c = Cache(400, P, 12, 20, seed=1)
    c.fill(rng, share=0.3)
    for lens in (c.lens, [min(n + 3, 20 * P) for n in c.lens]):
        tf.tf_kv_pages_free_window(c.d_refs, P, c.d_table, dev(lens), window, sinks, status=c.status)
        pages_ref.free_window(c.refs, P, c.table, lens, window, sinks)
        c.same()


@pytest.mark.parametrize("n_pages,P", [(1, 16), (7, 16), (1000, 16), (5000, 1), (9001, 1), (300, 100)])
@pytest.mark.parametrize("share", [0.0, 0.6])
def test_compact(n_pages, P, share):
    import verify_paged_gqa_b200 as tf
    rng = random.Random(n_pages + P)
    c = Cache(n_pages, P, 1 + n_pages // 40, 30, Hkv=1, seed=2)
    c.fill(rng, share=share)
    first = [rng.randint(0, 15) for _ in c.lens]
    end = [rng.randint(0, 30) for _ in c.lens]
    pages_ref.free(c.refs, c.table, first, end)
    c.push()
    moves, n_live = pages_ref.compact(c.refs, c.table)
    tf.tf_kv_pages_compact(c.d_refs, P, c.d_table, c.moves, status=c.status)
    c.same()
    assert c.moves[0, :2].tolist() == [len(moves), n_live]
    assert [m[:2] for m in c.list()] == moves and all(m[2] == P for m in c.list())
    c.move([(a, b, P) for a, b in moves])
    # a packed pool has nothing to move
    tf.tf_kv_pages_compact(c.d_refs, P, c.d_table, c.moves, status=c.status)
    c.same()
    assert c.moves[0, :2].tolist() == [0, n_live]


@pytest.mark.parametrize("d,Hkv,P", [(128, 1, 1), (128, 8, 512), (256, 3, 37), (512, 2, 200), (128, 2, 100)])
def test_moves_of_whole_and_partial_pages(d, Hkv, P):
    rng = random.Random(d + P)
    c = Cache(40, P, 1, 1, Hkv=Hkv, d=d, seed=3)
    ids = list(range(40))
    rng.shuffle(ids)
    moves = [(ids[2 * i], ids[2 * i + 1], rng.choice([0, 1, P // 2, P - 1, P, P])) for i in range(17)]
    moves[3] = (-1, moves[3][1], P)
    c.moves[0, 0] = len(moves)
    c.moves[1:1 + len(moves), :3] = dev(moves)
    c.move(moves)
    assert int(c.status) == 0
    # a list longer than its room is cut to it, and ids outside the pool are skipped
    import verify_paged_gqa_b200 as tf
    before = c.k.clone()
    c.moves[0, 0] = 1 << 30
    c.moves[1:, 0] = 40
    c.moves[1:, 1:3] = 1
    tf.tf_kv_pages_move(*c.pools(), c.moves, status=c.status)
    assert int(c.status) == tf.TF_DEV_BAD_PAGE and torch.equal(before, c.k)


def test_grow_without_enough_pages_changes_nothing():
    import verify_paged_gqa_b200 as tf
    c = Cache(6, 16, 4, 3, seed=4)
    c.table, c.lens = [[0, 1, -1], [0, 1, -1], [2, -1, -1], [-1] * 3], [32, 30, 16, 0]
    c.refs = [2, 2, 1, 0, 1, 1]          # one page is free; pages 4 and 5 are held elsewhere
    c.push()
    lens = [33, 31, 17, 0]               # a fresh page, a copy, a fresh page
    assert pages_ref.grow(list(c.refs), 16, [list(r) for r in c.table], lens, 1) is None
    tf.tf_kv_pages_grow(c.d_refs, 16, c.d_table, dev(lens), 1, c.moves, status=c.status)
    c.same(status=tf.TF_DEV_NO_PAGE)
    assert c.list() == []
    before = c.k.clone()
    tf.tf_kv_pages_move(*c.pools(), c.moves, status=c.status)
    assert torch.equal(before, c.k)
    c.refs[4] = c.refs[5] = 0
    c.push()
    moves = pages_ref.grow(c.refs, 16, c.table, lens, 1)
    tf.tf_kv_pages_grow(c.d_refs, 16, c.d_table, dev(lens), 1, c.moves, status=c.status)
    c.same()
    assert c.list() == moves == [(-1, 3, 0), (1, 4, 14), (-1, 5, 0)]


def test_two_streams_grow_into_the_page_they_share():
    import verify_paged_gqa_b200 as tf
    c = Cache(5, 64, 2, 1, seed=5)
    c.table, c.lens, c.refs = [[3], [3]], [10, 10], [0, 0, 1, 2, 0]
    c.push()
    moves = pages_ref.grow(c.refs, 64, c.table, [11, 11], 1)
    tf.tf_kv_pages_grow(c.d_refs, 64, c.d_table, dev([11, 11]), 1, c.moves, status=c.status)
    c.same()
    assert c.refs == [1, 1, 1, 0, 0] and c.list() == moves
    c.move(moves)


def test_bad_entries_are_reported_and_left():
    import verify_paged_gqa_b200 as tf
    c = Cache(8, 16, 3, 2, seed=6)
    c.table, c.lens, c.refs = [[0, 9], [1, -1], [5, -1]], [32, 16, 16], [1, 1, 0, 0, 0, 0, 0, 0]
    c.push()
    tf.tf_kv_pages_free(c.d_refs, 16, c.d_table, status=c.status)   # 9 is no page, 5 has no holder
    assert int(c.status) == tf.TF_DEV_BAD_PAGE
    assert c.d_refs.tolist() == [0] * 8 and c.d_table.tolist() == [[-1, 9], [-1, -1], [-1, -1]]
    c.push()
    tf.tf_kv_pages_free(c.d_refs, 16, c.d_table, dev([-1, 0, 0]), dev([1, 3, 1]), status=c.status)
    assert int(c.status) == tf.TF_DEV_BAD_LEN | tf.TF_DEV_BAD_PAGE
    assert c.d_refs.tolist() == c.refs
    c.push()
    new, lens = torch.full((4, 1), -9, dtype=torch.int32, device="cuda"), torch.full((4,), -9, dtype=torch.int32, device="cuda")
    # a parent of two pages in rows of one, one outside the table, a page without a holder
    tf.tf_kv_pages_fork(c.d_refs, 16, c.d_table, c.d_lens, dev([0, 3, 2, 1]), new, lens, status=c.status)
    assert int(c.status) == tf.TF_DEV_BAD_LEN | tf.TF_DEV_BAD_PAGE
    assert new.tolist() == [[-1], [-1], [-1], [1]] and lens.tolist() == [0, 0, 16, 16]
    assert c.d_refs.tolist() == [1, 2, 0, 0, 0, 0, 0, 0]
    c.push()
    tf.tf_kv_pages_grow(c.d_refs, 16, c.d_table, dev([33, 3, 16]), 5, c.moves, status=c.status)
    assert int(c.status) == tf.TF_DEV_BAD_LEN | tf.TF_DEV_BAD_PAGE and int(c.moves[0, 0]) == 0
    c.push()
    tf.tf_kv_pages_compact(c.d_refs, 16, c.d_table, c.moves, status=c.status)
    assert int(c.status) == tf.TF_DEV_BAD_PAGE and c.d_refs.tolist() == c.refs


def test_no_child_takes_a_page_that_nobody_holds():
    """Many children of one parent look at the same count at once."""
    import verify_paged_gqa_b200 as tf
    stride, N = 300, 512
    refs = dev([j % 2 for j in range(stride)])      # every other page has no holder
    table, lens = dev([list(range(stride))]), dev([stride * 16])
    new, new_lens = torch.full((N, stride), -9, dtype=torch.int32, device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tf.tf_kv_pages_fork(refs, 16, table, lens, dev([0] * N), new, new_lens, status=status)
    assert refs.tolist() == [(N + 1) * (j % 2) for j in range(stride)]
    assert bool((new == dev([j if j % 2 else -1 for j in range(stride)])).all())
    assert int(status) == tf.TF_DEV_BAD_PAGE


def test_streams_of_pages_need_no_pages():
    import verify_paged_gqa_b200 as tf
    c = Cache(8, 16, 0, 2, seed=7)
    t, n = torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0,), dtype=torch.int32, device="cuda")
    tf.tf_kv_pages_fork(c.d_refs, 16, t, n, n, t, n)
    tf.tf_kv_pages_free(c.d_refs, 16, t)
    tf.tf_kv_pages_free_window(c.d_refs, 16, t, n, 4, 0)
    tf.tf_kv_pages_grow(c.d_refs, 16, t, n, 1, c.moves)
    tf.tf_kv_pages_compact(c.d_refs, 16, t, c.moves)
    assert c.moves[0].tolist() == [0, 0, 0, 0]
    tf.tf_kv_pages_move(*c.pools(), c.moves)


def test_a_captured_beam_step_replays():
    import verify_paged_gqa_b200 as tf
    rng = random.Random(9)
    c = Cache(200, 16, 12, 6, seed=8)
    c.fill(rng, share=0.7)
    keep = c.d_refs.clone(), c.d_table.clone()
    parents = dev([rng.randint(0, 11) for _ in range(12)])
    new, lens = torch.full((12, 7), -1, dtype=torch.int32, device="cuda"), torch.zeros(12, dtype=torch.int32, device="cuda")

    def step():
        tf.tf_kv_pages_fork(c.d_refs, 16, c.d_table, c.d_lens, parents, new, lens, status=c.status)
        tf.tf_kv_pages_free(c.d_refs, 16, c.d_table, status=c.status)
        lens.add_(1)
        tf.tf_kv_pages_grow(c.d_refs, 16, new, lens, 1, c.moves, status=c.status)
        tf.tf_kv_pages_move(*c.pools(), c.moves, status=c.status)

    step()
    want = c.d_refs.clone(), c.d_table.clone(), new.clone(), lens.clone(), c.moves.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        c.d_refs.copy_(keep[0])
        c.d_table.copy_(keep[1])
        new.fill_(-1)
        graph.replay()
        for a, b in zip((c.d_refs, c.d_table, new, lens, c.moves), want):
            assert torch.equal(a, b)
    assert int(c.status) == 0
