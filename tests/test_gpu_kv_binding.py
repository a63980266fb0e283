"""What the paged-cache calls' Python side refuses beyond types and shapes."""
import pytest

pytestmark = pytest.mark.gpu


def test_trained_weights_are_refused_unless_no_gradient_is_asked_for(fk):
    import torch

    q, k = torch.randn(3, 4, 64, device="cuda"), torch.randn(3, 2, 64, device="cuda")
    w = torch.rand(64, device="cuda")
    par = torch.nn.Parameter(w.clone())
    rope, pos = torch.rand(9, 64, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    turn = torch.nn.Parameter(rope.clone())
    want = fk.fk_qk_norm_rope(q, k, None, w, w, rope=rope, positions=pos)
    for ws, r, name in (((par, w), rope, "q_weight"), ((w, par), rope, "k_weight"), ((w, w), turn, "rope")):
        with pytest.raises(ValueError, match=f"{name} requires grad"):
            fk.fk_qk_norm_rope(q, k, None, *ws, rope=r, positions=pos)
        with torch.no_grad():
            got = fk.fk_qk_norm_rope(q, k, None, *ws, rope=r, positions=pos)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
