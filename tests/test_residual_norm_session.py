"""The residual norm's session calls without a GPU: arguments that contradict each other."""
import pytest

torch = pytest.importorskip("torch")


def test_no_norm_takes_no_place_for_its_result(lib):
    """pre_norm = False with an h asks for two things at once (the norm was computed all the same)."""
    from context_document_masked_gb300.session import CPAttention
    s = object.__new__(CPAttention)
    x = torch.zeros(64, 32)
    with pytest.raises(ValueError, match="pre_norm"):
        s.residual_norm(x, pre_norm=False, x_out=x, h=x)
