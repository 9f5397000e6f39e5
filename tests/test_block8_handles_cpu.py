"""Life of e4m3 weight handles on the host, with the library's calls stubbed."""
import copy
import types

import pytest
import torch

import int8_quantized_matmul_outlier_b200 as m


@pytest.fixture
def freed(monkeypatch):
    """The handles that were given back."""
    gone = []
    monkeypatch.setattr(m, "_lib", types.SimpleNamespace(int8mm_block_free=gone.append))
    return gone


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy])
def test_a_handle_is_given_back_once_by_its_last_holder(freed, how):
    w = m.BlockWeight(77, 128, 64, torch.device("cuda", 0))
    layers = [m.LinearBlock8bit(w)]
    layers += [how(layers[0]), how(how(layers[0]))]
    assert all(l._w.handle == 77 for l in layers)
    del w
    while layers:
        assert freed == []
        layers.pop(0)
    assert freed == [77]
