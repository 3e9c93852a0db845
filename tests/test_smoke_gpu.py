"""The smoke run launches both attention kernels, whatever the library would choose for its sizes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_smoke_runs_both_attention_kernels(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import q4_dequant_gemv_gb300 as q4k
    call, forms = q4k.paged_attention, []

    def noted(*a, **kw):
        forms.append(kw.get("form"))
        return call(*a, **kw)

    monkeypatch.setattr(q4k, "paged_attention", noted, raising=False)
    __graft_entry__.smoke()
    assert "many" in forms and any(f and f != "many" for f in forms)
