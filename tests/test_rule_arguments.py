"""A rule of routing by groups is made of its arguments' values at the time of the call (CPU only)."""
import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def mx():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp4_expert_gb300 as mx
    return mx


def _struct(mx, monkeypatch, **kw):
    """The rule that a call hands to the library (a fake of its entry)."""
    got = {}

    def fake(logits, T, E, k, bias, rule, idx, w, stream):
        r = rule._obj
        got.update({n: getattr(r, n) for n, _ in r._fields_})
        return 0
    monkeypatch.setattr(mx.lib, "moe_route_groups", fake)
    monkeypatch.setattr(mx, "_ptr", lambda *a: None)
    monkeypatch.setattr(mx, "_stream", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    mx.moe_route_groups(torch.zeros((2, 64)), 2, **kw)
    return got


@pytest.mark.parametrize("make", [lambda v: torch.tensor(v), lambda v: np.array(v)])
def test_values_that_change_in_place(mx, monkeypatch, make):
    scale, renormalise, n_groups = make(2.5), make(True), make(4)
    first = _struct(mx, monkeypatch, scale=scale, renormalise=renormalise, n_groups=n_groups)
    assert (first["scale"], first["renormalise"], first["n_groups"]) == (2.5, 1, 4)
    scale[...] = 5.0
    renormalise[...] = False
    n_groups[...] = 8
    second = _struct(mx, monkeypatch, scale=scale, renormalise=renormalise, n_groups=n_groups)
    assert (second["scale"], second["renormalise"], second["n_groups"]) == (5.0, 0, 8)


def test_zeros_of_both_signs(mx, monkeypatch):
    assert [str(_struct(mx, monkeypatch, scale=s)["scale"]) for s in (0.0, -0.0, 0.0)] == ["0.0", "-0.0", "0.0"]


def test_counts_are_whole_numbers(mx, monkeypatch):
    assert _struct(mx, monkeypatch, n_groups=8)["n_groups"] == 8
    with pytest.raises(TypeError):
        _struct(mx, monkeypatch, n_groups=8.0)
