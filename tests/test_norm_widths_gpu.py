"""The channels-first block norm at a width of every size of block, and between them."""
import pytest
import torch

from tests.test_norm_gpu import (FULL, TYPES, backward, check_backward, check_forward, forward, gpu,
                                 make)

pytestmark = pytest.mark.gpu
WIDTHS = [(1, 64, 40), (2, 65, 33), (1, 96, 64), (2, 97, 20), (1, 160, 17), (1, 193, 64), (1, 256, 31),
          (2, 300, 17), (1, 384, 36), (1, 385, 16), (2, 600, 9), (1, 768, 20), (1, 769, 5), (1, 1024, 18)]


@pytest.mark.parametrize("dtype, ytype", TYPES)
@pytest.mark.parametrize("B, D, L", WIDTHS)
def test_widths(B, D, L, dtype, ytype):
    t = make(B * L, D, L, FULL, dtype, ytype, True, seed=D, grad=True)
    y, n = forward(gpu(t), L, layer=True)
    check_forward(t, L, y, n, True, 1e-6)
    check_backward(t, L, backward(gpu(t), L, FULL, layer=True), True, 1e-6)
    m = dict(gpu(t))  # off 16 bytes: element by element
    for k in ("h", "z", "residual", "y", "dy", "dn"):
        b = torch.empty(m[k].numel() + 1, dtype=m[k].dtype, device="cuda")
        m[k] = b[1:].view(m[k].shape).copy_(m[k])
    y, n = forward(m, L, layer=True)
    check_forward(t, L, y, n, True, 1e-6)
    check_backward(t, L, backward(m, L, FULL, layer=True), True, 1e-6)
