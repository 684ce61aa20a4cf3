"""The attention branch's own bookkeeping without a GPU: the library's launching
calls are replaced by recorders, the plans are the library's."""
import numpy as np
import pytest
import torch

import halo_sharded_conv_amd as hsc
from halo_sharded_conv_amd import attention_layer

LAUNCHES = ("st_layernorm_sharded", "st_conv_sharded", "st_rope_axes", "st_attention_packed", "st_conv_wgrad",
            "st_conv_dgrad_weights", "st_attention_packed_backward", "st_layernorm_backward", "st_plan_positions")


@pytest.fixture
def events(monkeypatch):
    """Names of the launches and "synchronize", in order, with their arguments."""
    log = []
    for n in LAUNCHES:
        monkeypatch.setattr(attention_layer, n, lambda *a, _n=n, **kw: log.append((_n, a, kw)))
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: log.append(("synchronize", a, {})))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(attention_layer, "_stream", lambda s: hsc.ctypes.c_void_p(s or 0), raising=False)
    return log


def names(log):
    return [e[0] for e in log]


def make(spatial=(4, 6), shards=((2, 2), (6,)), channels=32, heads=2, kv_heads=1, head_dim=16):
    return attention_layer.ShardedAttention(spatial, shards, channels, heads, kv_heads, head_dim, device="cpu")


def test_buffers_are_ready_for_any_stream(events):
    """Steps may run on a stream that is not the current one: everything the
    constructor and set_weights queue is waited for."""
    layer = make()
    assert names(events)[-1] == "synchronize"
    events.clear()
    layer.set_weights(np.ones((64, 32)), np.ones((32, 32)), np.ones(32), np.zeros(32))
    assert names(events) == ["synchronize", "synchronize"]     # older steps have read, later ones see


def test_weights_stay_in_place(events):
    """A captured graph keeps their addresses, and no step reads a freed buffer."""
    layer = make()
    layer.set_weights(np.ones((64, 32)), np.ones((32, 32)), np.ones(32), np.zeros(32))
    at = [t.data_ptr() for t in (layer.w_qkv, layer.w_out, layer.gamma, layer.beta)]
    layer.set_weights(np.ones((64, 32)), np.ones((32, 32)), 2 * np.ones(32), np.ones(32))
    assert at == [t.data_ptr() for t in (layer.w_qkv, layer.w_out, layer.gamma, layer.beta)]
    assert float(layer.gamma[0]) == 2 and float(layer.beta[0]) == 1


def test_first_backward_on_a_stream_of_its_own(events, monkeypatch):
    layer = make()
    x, dy = torch.zeros(24, 32), torch.zeros(24, 32, dtype=torch.bfloat16)
    events.clear()
    layer.backward(x, dy, stream=7)
    assert names(events)[0] == "synchronize" and names(events).count("synchronize") == 1
    events.clear()
    grads = layer.grads
    layer.backward(x, dy, stream=7)
    assert "synchronize" not in names(events) and layer.grads is grads
    # inside a capture nothing can be waited for
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    other = make()
    with pytest.raises(hsc.ShardConvError):
        other.backward(x, dy, stream=7)
    events.clear()
    other.backward(x, dy)
    assert "synchronize" not in names(events)


@pytest.mark.parametrize("spatial,shards", [((9, 15), ((5, 4), (15,))), ((9, 7), ((5, 4), (4, 3))),
                                            ((5, 7, 9), ((2, 3), (7,), (9,)))])
def test_odd_shards_have_aligned_buffers(events, spatial, shards):
    layer = make(spatial, shards, channels=40)
    launch = next(e for e in events if e[0] == "st_plan_positions")
    assert all(t.data_ptr() % 16 == 0 for t in launch[1][1])
    events.clear()
    t = layer.tokens
    layer.forward(torch.zeros(t, 40))
    layer.backward(torch.zeros(t, 40), torch.zeros(t, 40, dtype=torch.bfloat16))
    lists = [b for e in events for b in e[1] if isinstance(b, list) and torch.is_tensor(b[0])]
    assert len(lists) > 10 and all(b.data_ptr() % 16 == 0 for shard in lists for b in shard)


def test_widths_whose_packed_shards_are_not_aligned(events):
    with pytest.raises(hsc.ShardConvError) as e:
        make((9, 15), ((5, 4), (15,)), channels=36)
    assert e.value.status == 7
    make((9, 16), ((5, 4), (16,)), channels=36)            # the shards of this cut do
    make((9, 15), ((9,), (15,)), channels=36)              # and so does a single one


def test_upstream_gradient_of_another_type(events):
    """An fp32 dy is refused, not read as bf16 bits."""
    layer = make()
    x = torch.zeros(24, 32)
    events.clear()
    with pytest.raises(hsc.ShardConvError) as e:
        layer.backward(x, torch.zeros(24, 32))
    assert e.value.status == 1 and not [n for n in names(events) if n != "synchronize"]
    layer.backward(x, torch.zeros(24, 32, dtype=torch.int16))  # bf16 bits


@pytest.mark.parametrize("which", [0, 1])
def test_backward_convs_are_both_checked(events, monkeypatch, which):
    """An input-gradient conv that the library does not have shows as a
    workspace of zero bytes, whichever of the two it is."""
    layer = make()
    real = [layer.norm_plan, layer.joint_plan]
    ask = attention_layer.st_conv_workspace_bytes
    monkeypatch.setattr(attention_layer, "st_conv_workspace_bytes",
                        lambda plan, *a: 0 if plan is real[which] else ask(plan, *a))
    with pytest.raises(hsc.ShardConvError) as e:
        layer.alloc_backward()
    assert e.value.status == 4 and layer.grads is None


def test_weights_of_another_shape(events):
    """A transposed matrix has the right size and the wrong meaning."""
    layer = make()
    w_qkv, w_out = np.ones((64, 32)), np.ones((32, 32))
    layer.set_weights(w_qkv.reshape(64, 32, 1, 1), w_out.reshape(-1))
    for bad in (dict(w_qkv=w_qkv.T), dict(w_qkv=np.ones((64, 31))), dict(w_out=np.ones(1)), dict(gamma=np.ones(31)),
                dict(beta=np.ones(1))):
        with pytest.raises(hsc.ShardConvError) as e:
            layer.set_weights(**{**dict(w_qkv=w_qkv, w_out=w_out), **bad})
        assert e.value.status == 2, bad
