"""The block operators at their edges: the largest sizes they take, infinities in
queries, fp16 gradients far from one, non-finite rows beside masked ones, every
way out of the weight gradient, outputs in place of inputs, scratch sizes."""
import pytest
import torch

from mixed_precision_gb300 import block

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


# ---------------------------------------------------------------------------
# Weight gradient
# ---------------------------------------------------------------------------

def test_weight_grad_of_the_widest_rows():
    """2^30 columns: two rows of codes are further apart than 32 bits reach."""
    tokens, n_in = 64, 1 << 30
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    codes = torch.arange(tokens, device="cuda") % 7 - 3
    q = torch.empty(tokens, n_in, dtype=torch.int8, device="cuda")
    q.copy_(codes.to(torch.int8)[:, None].expand_as(q))
    scales = torch.full((tokens, n_in // 32), 127, dtype=torch.uint8, device="cuda")
    dy = torch.zeros(tokens, 8, dtype=BF16, device="cuda")[:, :1]
    dy[:, 0] = torch.arange(tokens, device="cuda") % 5 - 1
    dw = block.weight_grad(dy, block.PackedActivation(tokens, n_in, q=q, scales=scales))
    want = float((dy[:, 0].double() * codes).sum())  # small whole numbers: exact
    assert bool((dw == want).all())
    block.check()
