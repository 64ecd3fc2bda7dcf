"""What the session makes for a call, without a GPU: the library's call is replaced by one that notes its arguments."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def session(lib, monkeypatch):
    from context_document_masked_gb300.session import CPAttention
    s = object.__new__(CPAttention)
    s.T, s.hq, s.hkv, s.d, s.device, s.scale = 24, 4, 2, 64, torch.device("cpu"), 0.0
    s.kbuf = s.vbuf = s.ws = s.dplan = None
    s.calls = []
    monkeypatch.setattr(lib, "attn_bwd", lambda *a, **kw: s.calls.append((a, kw)))
    return s


def test_new_gradients_have_memory_of_their_own(session):
    """One can be kept, saved or freed without the other."""
    dq, dk, dv = session.backward(None, None, None, None, None, None)
    for t, heads in ((dq, 4), (dk, 2), (dv, 2)):
        assert t.shape == (24, heads, 64) and t.dtype == torch.float32 and t.is_contiguous()
        assert t.untyped_storage().nbytes() == 4 * t.numel() and t._base is None
    assert len({t.untyped_storage().data_ptr() for t in (dq, dk, dv)}) == 3
    assert not dk.any() and not dv.any()


def test_given_gradients(session):
    """Set to zero, or as they are; a missing one is new and zero."""
    for zero in (True, False):
        dk = torch.ones(24, 2, 64)
        _, got, dv = session.backward(None, None, None, None, None, None, dk=dk, zero_kv_grads=zero)
        assert got is dk and bool(dk.any()) != zero and not dv.any()
        dv = torch.ones(24, 2, 64)
        _, dk, got = session.backward(None, None, None, None, None, None, dv=dv, zero_kv_grads=zero)
        assert got is dv and bool(dv.any()) != zero and not dk.any()
