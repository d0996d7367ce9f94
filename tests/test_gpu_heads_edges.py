"""Query/key preparation at the edges of its arguments."""
import pytest
import torch

from test_gpu_heads import freqs, make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (64, "fp32")])
def test_infinite_gradient_past_the_rotated_part_stays_where_it_is(fa, interleaved, d, dtype):
    """There y = x, so dx = dy, element by element."""
    q, k, _, _ = make(1, 2, 1, 5, d, dtype, False, "packed", 8)
    turns = fa.rope_turns(freqs(32), DEV)
    dy = [torch.randn_like(t.contiguous()) for t in (q, k)]
    clean = fa.qk_norm_rope_backward(*dy, q, k, turns, interleaved=interleaved)
    for t in (dy[0], clean[0]):
        t[0, 1, 3, 40] = float("inf")
    for t in (dy[1], clean[1]):
        t[0, 0, 2, 63] = float("-inf")
    got = fa.qk_norm_rope_backward(*dy, q, k, turns, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
