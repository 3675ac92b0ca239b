"""device.ExpertLayer on the host: on which device its calls are made, and what it refuses."""
import contextlib

import pytest
import torch

from sparse_mla_decode_front_b200 import device

E, HIDDEN, WIDTH, ALL, K, T = 4, 256, 128, 64, 2, 3


def tensors():
    e4m3 = lambda *s: torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn)
    return dict(gamma=torch.ones(HIDDEN, dtype=torch.bfloat16),
                router_weights=torch.zeros(HIDDEN, ALL, dtype=torch.bfloat16), w_up=e4m3(E, 2 * WIDTH, HIDDEN),
                w_up_scales=torch.ones(E, 2, 2), w_down=e4m3(E, HIDDEN, WIDTH), w_down_scales=torch.ones(E, 2, 1),
                top_k=K, router_bias=torch.zeros(ALL, dtype=torch.bfloat16))


@pytest.fixture
def calls(monkeypatch):
    """(the device made current, or None; the call) of every call, none of them run."""
    made, current = [], [None]

    @contextlib.contextmanager
    def make_current(dev):
        before, current[0] = current[0], dev
        yield
        current[0] = before
    monkeypatch.setattr(torch.cuda, "device", make_current)
    record = lambda name: lambda *a, **k: made.append((current[0], name))
    for name in ("mla_rmsnorm_router_topk", "mla_get_device_status"):
        monkeypatch.setattr(device.api, name, record(name))
    for name in ("mla_moe_sort", "mla_moe_gather", "mla_fp8_grouped_matmul", "mla_fp8_quantize", "mla_moe_combine"):
        monkeypatch.setattr(device.experts, name, record(name))
    return made


def test_every_call_is_made_on_the_layers_device(calls):
    # the router's call and the status take the current device and its stream, which need not be the layer's
    layer = device.ExpertLayer(T, **tensors())
    layer.run(torch.zeros(T, HIDDEN, dtype=torch.bfloat16))
    layer.device_status()
    assert [name for _, name in calls] == [
        "mla_rmsnorm_router_topk", "mla_moe_sort", "mla_moe_gather", "mla_fp8_grouped_matmul", "mla_fp8_quantize",
        "mla_fp8_grouped_matmul", "mla_moe_combine", "mla_get_device_status"]
    assert all(dev == layer.out.device for dev, _ in calls)


def test_hidden_states_of_another_device_are_refused(calls):
    layer = device.ExpertLayer(T, **tensors())
    with pytest.raises(ValueError, match="hidden_states is on meta"):
        layer.run(torch.zeros(T, HIDDEN, dtype=torch.bfloat16, device="meta"))
    assert not calls


@pytest.mark.parametrize("name", ["gamma", "router_weights", "router_bias", "w_up", "w_up_scales", "w_down_scales"])
def test_weights_of_another_device_are_refused(name):
    t = tensors()
    t[name] = t[name].to("meta")
    with pytest.raises(ValueError, match=f"{name} is on meta"):
        device.ExpertLayer(T, **t)
