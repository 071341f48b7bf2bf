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


FAKE = """
#include <unistd.h>
volatile int entered;
int entered_now(void) { return entered; }
int tf_kv_pages_free(void) {  /* a launch that waits, as one into a full queue does */
    entered = 1;
    for (int i = 0; i < 200 && entered == 1; ++i)
        usleep(10000);
    return entered == 2 ? 0 : 4;
}
void let_go(void) { entered = 2; }
"""


def test_other_threads_run_while_a_call_launches(built, tmp_path):
    """A launch may wait for room in the stream's queue, and what makes room may
    be a host function that another Python thread has to run."""
    import re
    import shutil
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    with open(os.path.join(built.CSRC, "binding.cpp")) as f:
        names = re.findall(r"^ +X\\((tf_\\w+)\\)".replace("\\\\", "\\"), f.read(), re.M)
    assert "tf_kv_pages_free" in names
    src, so = tmp_path / "fake.c", tmp_path / "libfake.so"
    src.write_text(FAKE + "".join(f"int {n}(void) {{ return 0; }}\n" for n in names if n != "tf_kv_pages_free"))
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    python(f"""
        import ctypes, threading, time
        import torch
        from verify_paged_gqa_b200 import _abi
        _abi._binding.attach({str(so)!r})
        fake = ctypes.CDLL({str(so)!r})
        args = (torch.zeros(0, dtype=torch.int32), 16, torch.zeros((0, 3), dtype=torch.int32), None, None, None, 0)
        got = []
        t = threading.Thread(target=lambda: got.append(_abi._binding.tf_kv_pages_free(*args)))
        t.start()
        while not fake.entered_now() and t.is_alive():
            time.sleep(0.001)
        fake.let_go()
        t.join()
        assert got == [0], got
    """)
