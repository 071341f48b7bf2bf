"""Scales of zero (every visible position weighs the same) and below it: any
finite scale is accepted, and the softmax is that of scale * q . k (B200)."""
import pytest
import torch

import window_ref
from test_gpu_window import CLUSTER, TENSOR_CORE, WindowCase

pytestmark = pytest.mark.gpu


# (the rows per KV head reach every kernel: CUDA cores, the position-major
# tensor-core kernel with 32 and 64 rows to a block, the prompt kernel)
@pytest.mark.parametrize("d,G,rows,P", [(128, 4, 1, 64), (512, 4, 1, 512), (128, 8, 4, 512), (128, 8, 8, 37), (256, 4, 3, 64),
                                        (512, 8, 4, 64), (128, 4, 100, 512), (128, 3, 40, 37), (256, 4, 40, 64)])
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.09, 0.09])
def test_plain_calls(d, G, rows, P, scale):
    import verify_paged_gqa_b200 as tf
    c = WindowCase([rows + 900, rows, 1030], rows, 1 << 20, 0, d=d, G=G, P=P, seed=d + rows)
    c.scale = scale
    fn = tf.tf_paged_attn_decode if rows == 1 else tf.tf_paged_attn_verify if rows <= 8 else tf.tf_paged_attn_prompt
    out = torch.full(c.q.shape, float("nan"), dtype=torch.float32, device="cuda")
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")
    fn(c.k_pool, c.v_pool, c.table, c.lens, c.q, scale, out, ws, c.max_len)
    assert tf.tf_workspace_status(ws) == 0
    for s in range(3):
        ref, bound = window_ref.attend(c.q[s], c.k[s], c.v[s], c.max_len, 0, scale)
        # (the plain calls keep P's two bf16 parts by truncation, 2^-14 of it,
        # where the bound has 2^-17)
        room = bound + 2.0 ** -14 * c.v[s].double().abs().amax()
        assert ((out[s].double() - ref).abs() <= room).all(), s


@pytest.mark.parametrize("d,G,rows,P", [(128, 4, 1, 64), (128, 8, 4, 512), (128, 8, 8, 37), (256, 4, 3, 64), (512, 8, 4, 64),
                                        (128, 4, 100, 512), (128, 3, 40, 37)])
@pytest.mark.parametrize("scale", [0.0, -0.09])
@pytest.mark.parametrize("window,sinks", [(300, 4), (1, 0)])
def test_sliding_windows(d, G, rows, P, scale, window, sinks):
    c = WindowCase([rows + 900, rows, 1030], rows, window, sinks, d=d, G=G, P=P, seed=d + rows)
    c.scale = scale
    c.check(c.call())
    c.check(c.call(kernel=TENSOR_CORE))
    c.check(c.call(kernel=CLUSTER))


@pytest.mark.parametrize("scale", [0.0, -0.03])
def test_long_windows_of_prompt_chunks(scale):
    """The form that folds its sums."""
    c = WindowCase([9000], 100, 6000, 4, P=64, seed=6)
    c.scale = scale
    c.check(c.call(kernel=TENSOR_CORE))
