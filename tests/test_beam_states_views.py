"""xpress_beam_reorder copies memory: tensors that stand for the conjugate of theirs are refused."""
import pytest
import torch

from vocab_wide_add_amd import native


@pytest.mark.gpu
@pytest.mark.parametrize("count", [1, 70])        # from tensors in the host module, and in Python
def test_conjugate_states(count):
    src = torch.tensor([2, 0, 5], dtype=torch.int32, device="cuda")
    old = torch.randn(4, 6, dtype=torch.complex64, device="cuda")
    new = [torch.full((3, 6), 7.0, dtype=torch.complex64, device="cuda") for _ in range(count)]
    with pytest.raises(ValueError, match="conjugate"):
        native.xpress_beam_reorder([(old.conj(), x) for x in new], src)
    with pytest.raises(ValueError, match="conjugate"):
        native.xpress_beam_reorder([(old, x.conj()) for x in new], src)
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in new)
    native.xpress_beam_reorder([(old.conj().resolve_conj(), x) for x in new], src)
    torch.cuda.synchronize()
    for x in new:
        assert torch.equal(x[:2], old[[2, 0]].conj()) and (x[2] == 0).all()
