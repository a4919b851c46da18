"""Calls at the edges of what the operators around the layer take, on tensor metadata:
a call that is allowed gets as far as the question of its device.  No GPU."""

import pytest
import torch

from mixture_experts_moe_amd import binding as B


def meta(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("K", [1, 64])
def test_experts_of_one_weight_row(K):
    """Experts of one row may lie any distance apart that rows may; they may not overlap."""
    def call(w):
        B.moe_linear_i8(meta(8, K, dtype=torch.int8), meta(8), w, meta(4),
                        offsets=meta(5, dtype=torch.int32))
    with pytest.raises(ValueError, match="on the GPU"):
        call(meta(4, 5, K, dtype=torch.int8)[:, :1])
    with pytest.raises(ValueError, match="dense rows and experts"):
        call(meta(4, 5, K, dtype=torch.int8)[:, :2])
    with pytest.raises(ValueError, match="rows overlap"):
        call(meta(1, 1, K, dtype=torch.int8).expand(4, 1, K))
