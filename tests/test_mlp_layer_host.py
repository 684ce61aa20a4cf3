"""The MLP branch's own bookkeeping without a GPU: the library's launching calls
are replaced by recorders."""
import numpy as np
import pytest
import torch

import halo_sharded_conv_amd as hsc
from halo_sharded_conv_amd import mlp_layer

LAUNCHES = ("st_rmsnorm", "st_rmsnorm_backward", "st_linear", "st_linear_backward", "st_mx8_store", "st_mx8_load")


@pytest.fixture
def events(monkeypatch):
    log = []
    for n in LAUNCHES:
        monkeypatch.setattr(mlp_layer, n, lambda *a, _n=n, **kw: log.append((_n, a, kw)))
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: log.append(("synchronize", a, {})))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(mlp_layer, "_stream", lambda s: hsc.ctypes.c_void_p(s or 0), raising=False)
    return log


def names(log):
    return [e[0] for e in log]


def make(spatial=(4, 6), shards=((2, 2), (6,)), channels=32, hidden=64, **kw):
    return mlp_layer.ShardedMLP(spatial, shards, channels, hidden, device="cpu", **kw)


@pytest.mark.parametrize("args,kw,status", [
    (((4, 6), ((2, 3), (6,))), {}, 2), (((4, 6), ((4,),)), {}, 2), (((4, 6), ((2, 2), (6,))), dict(batch=2), 4),
    (((4, 6), ((4,), (6,))), dict(act="tanh"), 1), (((4, 6), ((4,), (6,))), dict(kept="fp8"), 1),
    (((4, 6), ((4,), (6,))), dict(products="f16"), 1), (((4, 6), ((4,), (6,))), dict(hidden=0), 1),
])
def test_refusals(events, args, kw, status):
    with pytest.raises(hsc.ShardConvError) as e:
        make(*args, **kw)
    assert e.value.status == status


def test_shards_in_the_order_of_the_plans(events):
    """Cells of the shards as a plan of the same volume numbers them."""
    layer = make((4, 6), ((1, 3), (2, 4)))
    plan = hsc.st_plan_shards(2, 1, 32, (4, 6), ((1, 3), (2, 4)), (0, 0), "f32")
    assert [b - a for a, b in zip(layer.starts, layer.starts[1:])] == hsc._cells(plan)


def test_weights_are_waited_for_and_stay_in_place(events):
    layer = make()
    assert names(events)[-1] == "synchronize"
    events.clear()
    w = dict(w_up=np.ones((64, 32)), w_down=np.ones((32, 64)), b_up=np.ones(64), b_down=np.ones(32), gamma=np.ones(32))
    layer.set_weights(**w)
    assert names(events) == ["synchronize", "synchronize"]
    at = [t.data_ptr() for t in (layer.w_up, layer.w_down, layer.b_up, layer.b_down, layer.gamma)]
    layer.set_weights(**{**w, "gamma": 2 * np.ones(32)})
    assert at == [t.data_ptr() for t in (layer.w_up, layer.w_down, layer.b_up, layer.b_down, layer.gamma)]
    assert float(layer.gamma[0]) == 2
    for bad in (dict(w_up=np.ones((32, 64))), dict(b_up=np.ones(32)), dict(gamma=np.ones(64))):
        with pytest.raises(hsc.ShardConvError):
            layer.set_weights(**{**w, **bad})


def test_steps(events):
    layer = make(kept="mx8")
    x, dy = torch.zeros(24, 32), torch.zeros(24, 32)
    events.clear()
    layer.forward(x, stream=7)
    assert names(events) == ["st_rmsnorm", "st_mx8_store", "st_linear", "st_linear"]
    assert events[-1][2]["residual"] is layer.total and events[2][2]["pre"] is layer.pre8
    events.clear()
    layer.backward(dy, stream=7)
    assert names(events) == ["synchronize", "st_mx8_load", "st_linear_backward", "st_linear_backward", "st_rmsnorm_backward"]
    assert all(e[2].get("stream", e[1][-1]) == 7 for e in events[1:])
    events.clear()
    layer.backward(dy)
    assert "synchronize" not in names(events)


def test_capture_without_backward_buffers(events, monkeypatch):
    layer = make()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(hsc.ShardConvError):
        layer.backward(torch.zeros(24, 32), stream=7)


def test_shared_scratch(events):
    a = make(kept="mx8")
    b = make(kept="mx8", scratch=a)
    assert b.h is a.h and b.total is a.total and b.pre8 is not a.pre8 and b.normed8 is not a.normed8
    b.alloc_backward()
    assert a.grads is b.grads is not None
    with pytest.raises(hsc.ShardConvError):
        make(scratch=make())
    with pytest.raises(hsc.ShardConvError):
        make(kept="mx8", hidden=96, scratch=a)
