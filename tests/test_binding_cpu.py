"""The compiled binding's life beside the library (no GPU): what needs it and
what does not, when it is rebuilt, and that other threads run during a call."""
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def built():
    from verify_paged_gqa_b200 import build
    build.build()
    return build


def python(code, timeout=120):
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, capture_output=True, text=True, timeout=timeout)
    assert r.returncode == 0, r.stdout + r.stderr


def test_calls_of_the_library_alone_need_no_binding(built):
    """Without it (here: its import fails) the ctypes calls work, and a call that
    it marshals names what is missing."""
    python("""
        import sys
        sys.modules["verify_paged_gqa_b200._binding"] = None   # importing it raises ImportError
        import torch
        import verify_paged_gqa_b200 as tf
        assert tf.tf_status_str(0).startswith("TF_OK")
        none = torch.zeros((0, 3), dtype=torch.int32)
        lens = torch.zeros(0, dtype=torch.int32)
        pool = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16)
        rows = torch.zeros((0, 1, 2, 128), dtype=torch.bfloat16)
        tf.tf_kv_put_rows(pool, pool, none, lens, rows, rows, 40, stream=0)
        try:
            tf.tf_kv_pages_free(torch.zeros(4, dtype=torch.int32), 16, none, stream=0)
        except ImportError as e:
            assert "verify_paged_gqa_b200.build" in str(e), e
        else:
            raise AssertionError("no error")
    """)


def test_another_python_or_torch_rebuilds_the_binding(built, monkeypatch):
    """_binding.so loads under the Python and torch it was compiled against
    only; file times do not tell."""
    made = []
    assert built.up_to_date()
    monkeypatch.setattr(built, "build_binding", lambda: made.append(1))
    built.build()
    assert made == []
    import torch
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert not built.up_to_date()
    built.build()
    assert made == [1]
