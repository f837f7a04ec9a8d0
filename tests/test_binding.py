"""The binding's short way (csrc/dn_call.cpp) is made for one torch: without it, or with one made
for another, the calls go the general way and the library builds."""
import os

import pytest
import torch

import deltanet_chunkwise_delta_b200 as dn
from deltanet_chunkwise_delta_b200 import _lib as L
from deltanet_chunkwise_delta_b200 import build as B


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()
    L.load()


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """No short way loaded, its file at a place of the test's own."""
    monkeypatch.setattr(B, "CALL", str(tmp_path / "dn_call.so"))
    monkeypatch.setattr(L, "_call", None)
    return tmp_path


def general():
    """The calls get as far as the general way's own checks."""
    with pytest.warns(RuntimeWarning, match="dn_call"):
        c = L._short()
    assert c.scan_step(1, 2, 3, 4, 5) is None and L._short() is c
    x = torch.zeros(1, 4, 64)
    with pytest.raises(ValueError):
        dn.deltanet_scan_fwd(x, x)
    with pytest.raises(ValueError):
        dn.deltanet_norm_fwd(x, torch.ones(64))


def test_missing(elsewhere):
    general()


def test_made_for_another_torch(elsewhere):
    for so, abi in ((b"", None), (b"", "torch 0.0.0 cpython-312"), (b"not a module", B.abi())):
        (elsewhere / "dn_call.so").write_bytes(so)
        if abi:
            (elsewhere / "dn_call.abi").write_text(abi)
        L._call = None
        general()


def test_the_build_goes_on_without_it(elsewhere, monkeypatch, capsys):
    made = []
    monkeypatch.setattr(B, "_build_lib", lambda verbose: made.append(1))
    monkeypatch.setenv("CXX", os.fspath(elsewhere / "no-compiler"))
    (elsewhere / "dn_call.so").write_bytes(b"old")
    assert B.build(force=True) == B.LIB and made == [1]
    assert not os.path.exists(B.CALL) and "not built" in capsys.readouterr().err
    assert B.build() == B.LIB and made == [1]           # tried again, the library left alone
    monkeypatch.setenv("CXX", "false")                  # a compiler that fails (no Python headers)
    B.build()
    assert not B.call_usable()


def test_it_is_made_again_for_another_torch(elsewhere, monkeypatch):
    made = []
    monkeypatch.setattr(B, "_build_lib", lambda verbose: pytest.fail("the library is up to date"))
    monkeypatch.setattr(B, "_build_call", lambda verbose: made.append(1))
    monkeypatch.setattr(B, "stale", lambda: False)
    (elsewhere / "dn_call.so").write_bytes(b"x")
    (elsewhere / "dn_call.abi").write_text(B.abi())
    B.build()
    assert made == [] and B.call_usable()
    (elsewhere / "dn_call.abi").write_text(B.abi() + "1")
    assert not B.call_usable()
    B.build()
    assert made == [1]
