"""Device arrays of 32-bit values that are not 4-byte aligned are refused: a
kernel that read one would fault (no GPU; nothing is launched)."""
import ctypes

import pytest

PTR, ODD = 1 << 12, (1 << 12) + 2


@pytest.fixture(scope="module")
def lib():
    from verify_paged_gqa_b200 import build
    build.build()
    from verify_paged_gqa_b200 import _abi
    return _abi


ref = ctypes.byref


def pool(lib):
    return lib.tf_kv_pool(PTR, PTR, 8, 2, 512, 128)


def streams(lib, table=PTR, lens=PTR):
    return lib.tf_streams(table, 4, lens, 2, 2048)


@pytest.mark.parametrize("kw", [dict(table=ODD), dict(lens=ODD), dict(table=PTR + 1), dict(lens=PTR + 3)])
def test_streams(lib, kw):
    p, st, r = pool(lib), streams(lib, **kw), lib.raw
    tail = (0.1, PTR, PTR, 1 << 30, None)
    assert r.tf_kv_put_rows(ref(p), ref(st), PTR, PTR, 2, None) == lib.TF_EINVAL
    assert r.tf_paged_attn_decode(ref(p), ref(st), PTR, 8, *tail) == lib.TF_EINVAL
    assert r.tf_paged_attn_verify(ref(p), ref(st), PTR, 8, 2, *tail) == lib.TF_EINVAL
    assert r.tf_paged_attn_prompt(ref(p), ref(st), PTR, 8, 40, *tail) == lib.TF_EINVAL
    assert r.tf_paged_attn_verify_window(ref(p), ref(st), PTR, 8, 2, 16, 4, *tail) == lib.TF_EINVAL
    assert r.tf_kv_copy_state(ref(p), ref(st), ref(p), PTR, 4, None, None) == lib.TF_EINVAL
    rope = lib.tf_rope(PTR, None, 128, 1, 0)
    assert r.tf_kv_put_rows_rope(ref(p), ref(st), ref(rope), PTR, None, 0, None, 0, PTR, 256, PTR, 256, 2, None) == lib.TF_EINVAL


def test_the_state_copys_destination_table(lib):
    p, st = pool(lib), streams(lib)
    assert lib.raw.tf_kv_copy_state(ref(p), ref(st), ref(p), ODD, 4, None, None) == lib.TF_EINVAL


def test_rope(lib):
    p, st = pool(lib), streams(lib)
    for inv, positions in ((ODD, PTR), (PTR, ODD)):
        rope = lib.tf_rope(inv, None, 128, 1, 0)
        assert lib.raw.tf_kv_put_rows_rope(ref(p), ref(st), ref(rope), positions, None, 0, None, 0, PTR, 256, PTR, 256, 2,
                                           None) == lib.TF_EINVAL


def test_page_calls(lib):
    r, pg = lib.raw, lib.tf_kv_pages(PTR, 100, 16)
    for at in (1, 3, 5, 7, 9):   # src_table, src_lens, parents, dst_table, dst_lens
        a = [ref(pg), PTR, 4, PTR, 2, PTR, 2, PTR, 4, PTR, None, None]
        a[at] = ODD
        assert r.tf_kv_pages_fork(*a) == lib.TF_EINVAL, at
    assert r.tf_kv_pages_free(ref(pg), PTR, 4, 2, ODD, None, None, None) == lib.TF_EINVAL
    assert r.tf_kv_pages_free(ref(pg), PTR, 4, 2, None, ODD, None, None) == lib.TF_EINVAL
    assert r.tf_kv_pages_free_window(ref(pg), PTR, 4, ODD, 2, 16, 0, None, None) == lib.TF_EINVAL
    assert r.tf_kv_pages_grow(ref(pg), PTR, 4, ODD, 2, 1, PTR, 1 << 20, None, None) == lib.TF_EINVAL
    assert r.tf_kv_pages_move(ref(pool(lib)), PTR, 64, ODD, None) == lib.TF_EINVAL
