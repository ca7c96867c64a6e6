"""The expert layer's operators and the scaled products at their edges: sums that
would be lost in truncated additions, the largest sizes, offsets that no routing
makes, the smallest choices."""
import pytest
import torch

import _experts_ref as ref
from _block_ref import U, close
from mixed_precision_gb300 import experts
from test_gpu_experts import offsets_of

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


# ---------------------------------------------------------------------------
# Truncated additions
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("product", ["forward", "input_grad", "weight_grad"])
def test_small_terms_behind_a_large_one(product, dtype):
    """1 + U + 4094 terms of 1.5 * 2^-28: 16 of them are 0.75 steps of an fp32 number next to 1, which a
    truncated addition drops. All together lift the sum 2.3e-5 above the border between two 16-bit results;
    runs of 1024 terms may lose (64 + 4 + 16) * 2^-23 = 1.0e-5."""
    k, n, m = 4096, 40, 72
    left = torch.full((n, k), 2.0 ** -14, dtype=dtype, device="cuda")
    right = torch.full((m, k), 1.5 * 2.0 ** -14, dtype=dtype, device="cuda")
    left[:, :2], right[:, 0], right[:, 1] = 1.0, 1.0, U[dtype]
    want, size = left.double() @ right.double().t(), left.double() @ right.double().t()
    tol = ref.product_tol(k, size, want, dtype, dtype, run=1024)
    if product == "forward":
        got = experts.forward(left, right[None], offsets_of([n]))
    elif product == "input_grad":
        got = experts.input_grad(left, right.t().contiguous()[None], offsets_of([n]))
    else:
        got = experts.weight_grad(left.t().contiguous(), right.t().contiguous(), offsets_of([k]))[0]
    close(got, want, tol, product)
