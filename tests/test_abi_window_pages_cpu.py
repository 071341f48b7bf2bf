"""Refusals of the sliding-window, rotary and page calls, before any of them
touches the device (no GPU)."""
import ctypes

import pytest

PTR = 1 << 12   # a plausible aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    from verify_paged_gqa_b200 import build
    build.build()
    from verify_paged_gqa_b200 import _abi
    return _abi


def ref(x):
    return None if x is None else ctypes.byref(x)


def pool(lib, **kw):
    return lib.tf_kv_pool(**{**dict(k_pool=PTR, v_pool=PTR, n_pages=8, n_kv_heads=2, page_size=512, head_dim=128), **kw})


def streams(lib, **kw):
    return lib.tf_streams(**{**dict(table=PTR, table_stride=4, lens=PTR, n_streams=2, max_len=2048), **kw})


@pytest.mark.parametrize("window,sinks,pool_kw,want", [
    (0, 4, {}, "TF_EINVAL"), (-5, 0, {}, "TF_EINVAL"), (16, -1, {}, "TF_EINVAL"), (16, 4, {"head_dim": 64}, "TF_EUNSUPPORTED"),
    (16, 4, {"n_pages": 1 << 22, "page_size": 512}, "TF_EUNSUPPORTED"),   # more than 2^31 - 1 rows
    (16, 4, {"k_pool": PTR + 2}, "TF_EINVAL")])
def test_window_refusals(lib, window, sinks, pool_kw, want):
    p, st = pool(lib, **pool_kw), streams(lib)
    tail = (window, sinks, 0.1, PTR, PTR, 1 << 30, None)
    assert lib.raw.tf_paged_attn_decode_window(ref(p), ref(st), PTR, 8, *tail) == getattr(lib, want)
    assert lib.raw.tf_paged_attn_verify_window(ref(p), ref(st), PTR, 8, 4, *tail) == getattr(lib, want)
    assert lib.raw.tf_paged_attn_prompt_window(ref(p), ref(st), PTR, 8, 40, *tail) == getattr(lib, want)
    assert lib.raw.tf_paged_attn_window_workspace_bytes(ref(p), ref(st), 8, 1, window, sinks) == 0


def test_window_rows_and_buffers(lib):
    p, st = pool(lib), streams(lib)
    v, pr = lib.raw.tf_paged_attn_verify_window, lib.raw.tf_paged_attn_prompt_window
    assert v(ref(p), ref(st), PTR, 8, 9, 16, 4, 0.1, PTR, PTR, 1 << 30, None) == lib.TF_EINVAL
    assert pr(ref(p), ref(st), PTR, 8, 4097, 16, 4, 0.1, PTR, PTR, 1 << 30, None) == lib.TF_EINVAL
    assert v(ref(p), ref(st), PTR, 7, 4, 16, 4, 0.1, PTR, PTR, 1 << 30, None) == lib.TF_EINVAL
    assert v(None, ref(st), PTR, 8, 4, 16, 4, 0.1, PTR, PTR, 1 << 30, None) == lib.TF_EINVAL


def rope(lib, axes=None, **kw):
    r = lib.tf_rope(**{**dict(inv_freq=PTR, pair_axis=None, rotary_dim=128, n_axes=3, adjacent=0), **kw})
    if axes is not None:
        r.keep = (ctypes.c_uint8 * len(axes))(*axes)
        r.pair_axis = ctypes.addressof(r.keep)
    return r


def put(lib, p, st, r, positions=PTR, q=PTR, qs=1024, qo=2 * PTR, hq=8, k=PTR, ks=256, v=PTR, vs=256, rows=2):
    return lib.raw.tf_kv_put_rows_rope(ref(p), ref(st), ref(r), positions, q, qs, qo, hq, k, ks, v, vs, rows, None)


def test_rope_refusals(lib):
    p, st = pool(lib), streams(lib)
    bad = [rope(lib, rotary_dim=0), rope(lib, rotary_dim=3), rope(lib, rotary_dim=130), rope(lib, n_axes=0), rope(lib, n_axes=5),
           rope(lib, adjacent=2), rope(lib, axes=[0] * 63 + [3]), rope(lib, inv_freq=None), None]
    for r in bad:
        assert put(lib, p, st, r) == lib.TF_EINVAL
    good = rope(lib, axes=[2] * 64)
    for kw in (dict(rows=0), dict(rows=2049), dict(positions=None), dict(q=None), dict(q=PTR + 2), dict(qo=None), dict(qs=1023),
               dict(qs=1028), dict(qs=512), dict(hq=-1), dict(k=None), dict(ks=248), dict(ks=260), dict(v=PTR + 8), dict(vs=0),
               dict(qo=PTR, qs=2048)):   # (turned in place over rows that lie apart)
        assert put(lib, p, st, good, **kw) == lib.TF_EINVAL, kw
    assert put(lib, pool(lib, head_dim=64), st, good) == lib.TF_EUNSUPPORTED
    none = streams(lib, n_streams=0, table=None, lens=None)
    assert put(lib, p, none, good, positions=None, q=None, qo=None, k=None, v=None) == lib.TF_OK


def test_page_call_refusals(lib):
    raw, ok = lib.raw, lib.tf_kv_pages(PTR, 100, 16)
    bad = [lib.tf_kv_pages(None, 100, 16), lib.tf_kv_pages(PTR + 4, 100, 16), lib.tf_kv_pages(PTR, 0, 16),
           lib.tf_kv_pages(PTR, 100, 0), None]
    for pg in bad:
        assert raw.tf_kv_pages_fork(ref(pg), PTR, 4, PTR, 2, PTR, 2, PTR, 4, PTR, None, None) == lib.TF_EINVAL
        assert raw.tf_kv_pages_free(ref(pg), PTR, 4, 2, None, None, None, None) == lib.TF_EINVAL
        assert raw.tf_kv_pages_free_window(ref(pg), PTR, 4, PTR, 2, 16, 0, None, None) == lib.TF_EINVAL
        assert raw.tf_kv_pages_grow(ref(pg), PTR, 4, PTR, 2, 1, PTR, 1 << 20, None, None) == lib.TF_EINVAL
        assert raw.tf_kv_pages_compact(ref(pg), PTR, 4, 2, PTR, 1 << 20, None, None) == lib.TF_EINVAL
    fork = lambda **k: raw.tf_kv_pages_fork(ref(ok), *{**dict(st=PTR, ss=4, sl=PTR, n=2, par=PTR, m=2, dt=PTR, ds=4, dl=PTR, status=None,  # noqa: E731
                                                              stream=None), **k}.values())
    for k in (dict(st=None), dict(ss=0), dict(sl=None), dict(n=-1), dict(par=None), dict(m=-1), dict(dt=None), dict(ds=0), dict(dl=None),
              dict(status=PTR + 2), dict(n=1 << 30), dict(m=1 << 30)):
        assert fork(**k) == lib.TF_EINVAL, k
    assert fork(m=0, par=None, dt=None, dl=None) == lib.TF_OK
    assert raw.tf_kv_pages_free(ref(ok), None, 4, 2, None, None, None, None) == lib.TF_EINVAL
    assert raw.tf_kv_pages_free(ref(ok), None, 4, 0, None, None, None, None) == lib.TF_OK
    for window, sinks, lens in ((0, 0, PTR), (16, -1, PTR), (16, 0, None)):
        assert raw.tf_kv_pages_free_window(ref(ok), PTR, 4, lens, 2, window, sinks, None, None) == lib.TF_EINVAL
    grow = lambda rows, moves, size, lens=PTR: raw.tf_kv_pages_grow(ref(ok), PTR, 4, lens, 2, rows, moves, size, None, None)  # noqa: E731
    assert grow(0, PTR, 1 << 20) == grow(1, None, 1 << 20) == grow(1, PTR + 8, 1 << 20) == grow(1, PTR, 1 << 20, None) == lib.TF_EINVAL
    # rows = 18 over pages of 16 touch three pages at most: six entries and the head
    assert grow(1, PTR, 47) == grow(18, PTR, 6 * 16) == grow(2 ** 31 - 1, PTR, 1 << 20) == lib.TF_ENOSPACE
    compact = lambda moves, size: raw.tf_kv_pages_compact(ref(ok), PTR, 4, 2, moves, size, None, None)  # noqa: E731
    assert compact(None, 1 << 20) == compact(PTR + 8, 1 << 20) == lib.TF_EINVAL
    assert compact(PTR, 50 * 16) == lib.TF_ENOSPACE
    for p, moves, size in ((None, PTR, 64), (pool(lib), None, 64), (pool(lib), PTR + 4, 64), (pool(lib), PTR, 15),
                           (pool(lib, v_pool=None), PTR, 64)):
        assert raw.tf_kv_pages_move(ref(p), moves, size, None, None) == lib.TF_EINVAL
    assert raw.tf_kv_pages_move(ref(pool(lib, head_dim=64)), PTR, 64, None, None) == lib.TF_EUNSUPPORTED


def test_python_checks(lib):
    import torch
    import verify_paged_gqa_b200 as tf
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    kp = bf(4, 2, 16, 128)
    table, lens, inv = i32(2, 3), i32(2), torch.zeros(64)
    with pytest.raises(ValueError):
        tf.Rope(inv, [0] * 63, 1)
    with pytest.raises(ValueError):
        tf.Rope(inv, [0] * 63 + [1], 1)
    r = tf.Rope(inv, None, 3)
    ok = dict(q=bf(2, 5, 4, 128), k=bf(2, 5, 2, 128), v=bf(2, 5, 2, 128), pos=i32(2, 5, 3))
    call = lambda q_out=None, **k: (lambda a: tf.tf_kv_put_rows_rope(kp, kp, table, lens, a["q"], a["k"], a["v"], a["pos"], r, 40,  # noqa: E731
                                                                     q_out=q_out, stream=0))({**ok, **k})
    for kw in (dict(pos=i32(2, 5, 2)), dict(pos=i32(3, 5, 3)), dict(k=bf(2, 5, 1, 128)), dict(v=bf(2, 4, 2, 128)),
               dict(k=bf(2, 5, 128, 2).transpose(2, 3)), dict(q=bf(5, 2, 4, 128).transpose(0, 1)), dict(q_out=bf(2, 5, 4, 64))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=torch.zeros(2, 5, 4, 128)), dict(pos=torch.zeros(2, 5, 3)), dict(k=bf(2, 5, 256))):
        with pytest.raises(TypeError):
            call(**kw)
    refs, moves = i32(4), i32(8, 4)
    with pytest.raises(ValueError):
        tf.tf_kv_pages_grow(refs, 16, table, i32(3), 1, moves, stream=0)
    with pytest.raises(ValueError):
        tf.tf_kv_pages_grow(refs, 16, table, lens, 1, i32(8, 3), stream=0)
    with pytest.raises(TypeError):
        tf.tf_kv_pages_free(refs, 16, table, status=torch.zeros(1), stream=0)
    with pytest.raises(ValueError):
        tf.tf_kv_pages_fork(refs, 16, table, lens, i32(5), i32(4, 3), i32(4), stream=0)


def test_page_counts_that_indexes_cannot_pass(lib):
    """The kernels step past the last page and entry by up to a block's worth
    in 32 bits: counts so near 2^31 are refused."""
    raw, ok = lib.raw, lib.tf_kv_pages(PTR, 100, 16)
    for n in (2 ** 31 - 1, 2 ** 31 - 8191):
        many = lib.tf_kv_pages(PTR, n, 16)
        assert raw.tf_kv_pages_free(ref(many), PTR, 4, 2, None, None, None, None) == lib.TF_EINVAL
        assert raw.tf_kv_pages_grow(ref(many), PTR, 4, PTR, 2, 1, PTR, 1 << 20, None, None) == lib.TF_EINVAL
        assert raw.tf_kv_pages_compact(ref(many), PTR, 4, 2, PTR, 1 << 40, None, None) == lib.TF_EINVAL
        assert raw.tf_kv_pages_free(ref(ok), PTR, n, 1, None, None, None, None) == lib.TF_EINVAL
        assert raw.tf_kv_pages_fork(ref(ok), PTR, 4, PTR, 2, PTR, 1, PTR, n, PTR, None, None) == lib.TF_EINVAL


def test_a_stream_handle_that_is_no_pointer(lib):
    import torch
    import verify_paged_gqa_b200 as tf
    none = torch.zeros((0, 3), dtype=torch.int32)
    with pytest.raises(OverflowError):
        tf.tf_kv_pages_free(torch.zeros(0, dtype=torch.int32), 16, none, stream=1 << 70)
