"""optimizer.AdamW's checkpoints, on the CPU: the plan of a list is made on the
host, so that everything but step() runs without a GPU."""
import pytest
import torch

from mxfp8_block_scaled_04_amd import training as T
from mxfp8_block_scaled_04_amd.optimizer import AdamW


@pytest.fixture(autouse=True)
def cpu_tensors(monkeypatch):
    monkeypatch.setattr(T, "_same_device", lambda *tensors: None)


def _make(weights=None, **kwargs):
    weights = weights or [torch.ones(300), torch.ones(4).bfloat16()]
    return AdamW(weights, [torch.zeros(300), torch.zeros(4)], **{"lr": 1e-2, "weight_decay": [0.1, 0.0], **kwargs})


def test_parameters_are_updated_outside_of_autograd():
    """Weights that require gradients: their masters, checkpoints and loading
    belong to no graph, and the parameter keeps its memory."""
    p, q = (torch.nn.Parameter(torch.ones(n, dtype=d)) for n, d in ((300, torch.float32), (4, torch.bfloat16)))
    opt = _make([p, q])
    assert opt.weights[0].data_ptr() == p.data_ptr() and not opt.masters[1].requires_grad
    saved = opt.state_dict()
    assert not any(t.requires_grad for t in saved.values())
    saved["weights.0"].fill_(5.0)
    saved["masters.1"].fill_(6.0)
    opt.load_state_dict(saved)
    assert (p == 5).all() and (opt.masters[1] == 6).all()
    assert p.requires_grad and p.is_leaf and q.requires_grad and q.is_leaf


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("name,value", [("betas", (0.9, 0.999)), ("betas", (0.8, 0.95)), ("eps", 1e-6),
                                        ("max_norm", 1.0), ("max_norm", float("inf")), ("weight_decay", 0.1),
                                        ("weight_decay", [0.1, 0.2])])
def test_a_state_saved_with_other_settings_is_refused(bits, name, value):
    """A later step would be another one without a word."""
    saved = _make(state_bits=bits).state_dict()
    other = _make(state_bits=bits, **{name: value})
    other.m[0].fill_(3)
    with pytest.raises(ValueError, match=name):
        other.load_state_dict(saved)
    assert (other.m[0].float() == 3).all()  # nothing was loaded
    other.load_state_dict(other.state_dict())


def test_the_learning_rate_and_states_are_loaded():
    a, b = _make(max_norm=1.0), _make(max_norm=1.0, lr=1e-3)
    a.m[0].fill_(2.0)
    a.steps[0] = 7
    saved = a.state_dict()
    assert all(isinstance(t, torch.Tensor) for t in saved.values())
    b.load_state_dict(saved)
    assert (b.m[0] == 2).all() and b.steps.tolist() == [7, 0] and float(b.lr) == float(torch.tensor(1e-2))


def test_a_state_without_settings_is_taken_as_it_is():
    """Tensors of another origin, or saved before the settings were kept."""
    a, b = _make(), _make(eps=1e-6)
    b.load_state_dict({k: t for k, t in a.state_dict().items() if k not in ("betas", "eps", "max_norm", "weight_decay")})
    with pytest.raises(ValueError):
        b.load_state_dict({k: t for k, t in a.state_dict().items() if k != "eps"})
    with pytest.raises(ValueError):
        b.load_state_dict({**a.state_dict(), "more": torch.zeros(1)})
