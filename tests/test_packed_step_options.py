"""Options of the packed step that do not go together are refused before any buffer is made (CPU)."""
import pytest

import __graft_entry__ as entry


@pytest.fixture(scope="module")
def ps():
    entry.build()
    from tensor_transformer_layer_way_gb300 import packed_step
    return packed_step


def _step(ps, **options):
    w = ps.init_weights(1, 128, 128, 2, 1, 64, 256, device="cpu")
    return ps.PackedStep(w, 128, 2, n_q=2, n_kv=1, d=64, device="cpu", **options)


def test_sinks_need_a_window(ps):
    with pytest.raises(ValueError, match="window"):
        _step(ps, sinks=4)
    _step(ps, sinks=0)
    _step(ps, sinks=4, window=16)


def test_the_example_refuses_sinks_without_a_window(ps, monkeypatch):
    weights = ps.init_weights
    monkeypatch.setattr(ps, "init_weights", lambda *a, **k: weights(*a, **dict(k, device="cpu")))
    with pytest.raises(ValueError, match="window"):
        ps.main(steps=1, sinks=4)


@pytest.mark.parametrize("head_norm", [False, True])
def test_positions_need_a_rotation(ps, head_norm):
    """Without one they would be dropped; with one they go on to the kernels (which take no CPU tensors)."""
    import torch
    positions = torch.zeros(1, 128, dtype=torch.int32)
    w = ps.init_weights(1, 128, 128, 2, 1, 64, 256, head_norm=head_norm, device="cpu")
    step = ps.PackedStep(w, 128, 2, n_q=2, n_kv=1, d=64, device="cpu")
    for call in (lambda: step.forward(None, None, None, positions), lambda: step.backward(None, None, positions)):
        with pytest.raises(ValueError, match="rotation"):
            call()
