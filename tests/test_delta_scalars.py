"""qk_scale and eps are read at every call of the gated delta rule and of the
head norm, also where they are tensors that change in place.  The binding's
argument marshalling alone: nothing here launches a kernel."""
import pytest

import xlstm_mlstm_chunkwise_amd as mt

torch = pytest.importorskip("torch")


@pytest.fixture
def calls(monkeypatch):
    """Descriptors of the calls that would be launched, on CPU tensors."""
    seen = []
    monkeypatch.setattr(mt, "_call", lambda where, dev, desc, *args: seen.append(desc._obj))
    monkeypatch.setattr(mt, "_delta_inputs", lambda q, k, v, *rest: (*q.shape, v.shape[-1]))
    monkeypatch.setattr(mt, "_norm_input", lambda x: x.shape)
    monkeypatch.setattr(mt, "_bytes_of", lambda need, workspace, dev: (torch.empty(0), 0))
    return seen


def _inputs():
    x, g = torch.zeros(1, 2, 5, 64), torch.zeros(1, 2, 5)
    return x, g


def test_a_scale_that_changes_in_place(calls):
    x, g = _inputs()
    scale = torch.tensor(0.5)
    for value in (0.5, 0.25, 0.125):
        scale.fill_(value)
        mt.mlstm_delta_fw(x, x, x, g, g, qk_scale=scale)
        mt.mlstm_delta_bw(x, x, x, g, g, x, qk_scale=scale)
        assert [d.qk_scale for d in calls] == [value] * 2
        calls.clear()


def test_a_scale_that_changes_before_the_backward_pass(calls):
    x, g = _inputs()
    x.requires_grad_(True)
    scale = torch.tensor(0.5)
    H = mt.mlstm_delta(x, x, x, g, g, qk_scale=scale)
    scale.fill_(0.25)
    H.sum().backward()
    assert [d.qk_scale for d in calls] == [0.5, 0.5]


def test_an_eps_that_changes_in_place(calls):
    x, _ = _inputs()
    eps = torch.tensor(0.5)
    for value in (0.5, 0.25):
        eps.fill_(value)
        mt.head_norm_fw(x, eps=eps)
        mt.head_norm_bw(x, x.transpose(1, 2).contiguous(), eps=eps)
        assert [d.eps for d in calls] == [value] * 2
        calls.clear()


def test_an_eps_that_changes_before_the_backward_pass(calls):
    x, _ = _inputs()
    x.requires_grad_(True)
    eps = torch.tensor(0.5)
    y = mt.head_norm(x, eps=eps)
    eps.fill_(0.25)
    y.sum().backward()
    assert [d.eps for d in calls] == [0.5, 0.5]
