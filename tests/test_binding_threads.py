"""The binding's first calls from two threads (no GPU: a stand-in for the library)."""
import threading
import types

import pytest

from gated_linear_attention_ddts_b200 import _binding


def test_two_threads_may_call_first(monkeypatch):
    """A second thread that comes while the first is still declaring the entry
    points finds the one that it asks for."""
    begun, go_on = threading.Event(), threading.Event()
    first = threading.current_thread().ident
    names = []

    class Library:
        def __getitem__(self, name):
            if threading.current_thread().ident == worker.ident:
                names.append(name)
                if len(names) == 2:  # the first one may be declared, the others are not yet
                    begun.set()
                    assert go_on.wait(20)
            return types.SimpleNamespace(name=name)

    monkeypatch.setattr(_binding, "_packed", {})
    monkeypatch.setattr(_binding, "load", Library)
    got = []
    worker = threading.Thread(target=lambda: got.append(_binding._load_packed("rdm_ssm_step")))
    worker.start()
    try:
        assert begun.wait(20)
        assert threading.current_thread().ident == first
        assert _binding._load_packed("rdm_ska_q8_decode").name == "rdm_ska_q8_decode"
    finally:
        go_on.set()
        worker.join(20)
    assert [f.name for f in got] == ["rdm_ssm_step"]
    with pytest.raises(KeyError):
        _binding._load_packed("rdm_no_such_entry")
