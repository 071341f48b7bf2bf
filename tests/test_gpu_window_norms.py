"""Long sliding windows in the norm, kernel by kernel (B200): see window_norms."""
import pytest
import torch

import window_norms
import window_ref
from test_gpu_window import CLUSTER, TENSOR_CORE, WindowCase

pytestmark = pytest.mark.gpu


def off(c, out):
    """The worst stream of a few (each of them is attended on its own)."""
    S = len(c.k)
    return max(window_norms.off(out[s], window_ref.attend(c.q[s], c.k[s], c.v[s], c.window, c.sinks, c.scale)[0])
               for s in (0, S // 2, S - 1))


# (as many streams as leave every unit whole on one CTA: its sums run over the
# whole window, 65 tiles)
@pytest.mark.parametrize("d,G,rows", [(128, 4, 1), (128, 8, 1), (128, 4, 4), (256, 4, 1), (256, 8, 2), (512, 8, 1), (512, 4, 1)])
def test_cluster_kernel(d, G, rows):
    c = WindowCase([9000] * 76, rows, 8200, 4, d=d, G=G, P=512, Hkv=1, seed=d + G + rows)
    assert off(c, c.call(kernel=CLUSTER)) < window_norms.CLUSTER


@pytest.mark.parametrize("d,G,rows", [(128, 8, 4), (128, 8, 8), (128, 4, 3), (256, 8, 4), (512, 8, 4), (256, 4, 20)])
def test_position_major_kernel_folds(d, G, rows):
    c = WindowCase([9000] * 76, rows, 8200, 4, d=d, G=G, P=512, Hkv=1, seed=d + G + rows)
    assert off(c, c.call(kernel=TENSOR_CORE)) < window_norms.FOLDED


@pytest.mark.parametrize("window,most", [(900, window_norms.FOLDED), (2048, window_norms.UNFOLDED), (4604, window_norms.UNFOLDED),
                                         (4700, window_norms.FOLDED), (8200, window_norms.FOLDED)])
def test_prompt_kernel(window, most):
    c = WindowCase([9000] * 20, 100, window, 4, G=4, P=512, Hkv=1, seed=window)
    assert off(c, c.call(kernel=TENSOR_CORE)) < most
