"""Arguments that are no tensors are refused by their names, on the CPU."""
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb

X = torch.zeros(4, 64, dtype=torch.bfloat16)
IDS = torch.zeros(4, 2, dtype=torch.int32)


@pytest.mark.parametrize("name,call", [
    ("expert_ids", lambda v: fb.moe_sort(v, 4)), ("x", lambda v: fb.moe_dispatch(v, IDS)),
    ("row_of", lambda v: fb.moe_dispatch(X, v)), ("q", lambda v: fb.moe_dispatch_fp8(v, X, IDS, IDS)),
    ("rows", lambda v: fb.moe_combine(v, IDS)), ("dy", lambda v: fb.moe_combine_backward(v, X, IDS, X)),
    ("x", lambda v: fb.residual_norm(v)), ("x_out", lambda v: fb.residual_norm_backward(v)),
    ("gradient 1", lambda v: fb.grad_norm([X, v])), ("gradient 0", lambda v: fb.clip_grad_norm([v], 1.0)),
    ("output 1", lambda v: fb.grad_table([X, X], [X, v]))])
@pytest.mark.parametrize("value", [None, 3, [[1.0]], X.float().numpy()])
def test_no_tensor(name, call, value):
    with pytest.raises(TypeError, match=f"^{name} must be a tensor"):
        call(value)
