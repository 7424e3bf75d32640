"""Which tensors the bindings of the operators around the activation copy (CPU)."""
import torch

from ffn_gated_activation_b200 import block


def test_gradients_are_copied_only_where_rows_are_misaligned():
    base = torch.zeros(6, 40, dtype=torch.bfloat16)  # rows of 80 bytes, on 16
    assert base.data_ptr() % 16 == 0
    for t in (base, base[:, :32], base[:, 8:40], base.view(2, 3, 40)[:, :, :16], base[:1, :8], base[:0], base[2:3]):
        assert block.aligned_rows(t) is t
    odd = torch.zeros(6, 36, dtype=torch.bfloat16)  # of 72
    for t in (base[:, 4:36], odd[:, :32], odd.view(2, 3, 36)[:, :, :32], odd[1:2, :32]):
        c = block.aligned_rows(t)
        assert c is not t and c.is_contiguous() and c.data_ptr() % 16 == 0 and torch.equal(c, t)
    assert block.aligned_rows(odd[:1, :32]).shape == (1, 32) and block.aligned_rows(odd.view(-1)[:32]).data_ptr() == odd.data_ptr()
