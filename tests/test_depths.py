"""Depths that share one layer, chained without copies: a depth's output is the next one's x, and
a depth's dx the dout of the one before."""
import pytest
import torch

import top_routing_expert_moe_gb300 as moe
from tests.test_checkpoint import layer_case

CFG = dict(T=16, d=128, f=128, E=2, k=1)


@pytest.fixture
def calls(monkeypatch):
    """The binding without its launches: the tensors that each entry point is given."""
    made, real = [], moe._call

    def call(name, *a):
        if name.endswith(("capacity", "size", "pitch", "bytes")):      # asks, launches nothing
            return real(name, *a)
        made.append((name, a))

    for m in (moe, moe.mx8):
        monkeypatch.setattr(m, "_p", lambda t: t)
        monkeypatch.setattr(m, "_s", lambda s: 0)
        monkeypatch.setattr(m, "_call", call)
    monkeypatch.setattr(moe.mx8._Numbers, "ptrs", property(lambda self: (self.codes, self.scales)))
    monkeypatch.setattr(moe.MoECheckpoint, "keep_y", lambda self, y, stream=None: None)
    return made


def cpu_weights():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    return dict(W_r=z(128, 2), W_up=z(2, 128, 128), W_down=z(2, 128, 128))


def lies_in(t, owned):
    return t.untyped_storage().data_ptr() == owned.untyped_storage().data_ptr()


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("where", ["out", "part of out", "y_perm", "dx"])
def test_rows_in_the_layers_own_memory_are_kept_apart(calls, kept, where):
    cfg = moe.MoEConfig(**CFG)
    layer = moe.MoELayer(cfg, "cpu")
    ck = moe.MoECheckpoint(cfg, "cpu") if kept else None
    x = {"out": layer.out, "part of out": layer.out[:], "y_perm": layer.y_perm[:16], "dx": layer.grads()["dx"]}[where]
    x.copy_(torch.arange(16 * 128).reshape(16, 128) % 251)
    rows = x.clone()
    layer.forward(x, **cpu_weights(), checkpoint=ck)
    x.zero_()                                        # as the layer's own kernels write there
    seen = (ck.inputs if kept else layer._inputs)[0]
    assert torch.equal(seen, rows)
    for name, a in calls:
        if name in ("moe_route", "moe_permute"):
            assert a[1] is seen
    fresh = torch.zeros(16, 128, dtype=torch.bfloat16)
    layer.forward(fresh, **cpu_weights(), checkpoint=ck)
    assert (ck.inputs if kept else layer._inputs)[0] is fresh        # others are not copied


def test_each_depth_keeps_a_copy_of_its_own(calls):
    cfg = moe.MoEConfig(**CFG)
    layer = moe.MoELayer(cfg, "cpu")
    cks = [moe.MoECheckpoint(cfg, "cpu") for _ in range(3)]
    x = torch.zeros(16, 128, dtype=torch.bfloat16)
    for i, ck in enumerate(cks):
        x = layer.forward(x, **cpu_weights(), checkpoint=ck)
        x.fill_(i + 1)
    assert [float(ck.inputs[0].float().mean()) for ck in cks] == [0, 1, 2]
    assert not lies_in(cks[1].inputs[0], cks[2].inputs[0])


def test_a_forward_that_raised_leaves_no_backward(calls, monkeypatch):
    """Its first launches have written over what the backward of the one before needs."""
    layer, w = moe.MoELayer(moe.MoEConfig(**CFG), "cpu"), cpu_weights()
    x = torch.zeros(16, 128, dtype=torch.bfloat16)
    layer.forward(x, **w)
    layer.backward(x)

    def ffn(*a, **kw):
        raise moe.MoEError(moe.ERR_INVALID_ARG, "moe_grouped_ffn")
    monkeypatch.setattr(moe, "moe_grouped_ffn", ffn)
    with pytest.raises(moe.MoEError):
        layer.forward(x, **w)
    with pytest.raises(RuntimeError, match="forward"):
        layer.backward(x)


def test_a_checkpoint_on_another_device_is_refused():
    layer, ck = moe.MoELayer(moe.MoEConfig(**CFG), "cpu"), moe.MoECheckpoint(moe.MoEConfig(**CFG), "meta")
    x = torch.zeros(16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on meta, the layer on cpu"):
        layer.forward(x, **cpu_weights(), checkpoint=ck)
    with pytest.raises(ValueError, match="on meta, the layer on cpu"):
        layer.backward(x, checkpoint=ck)


def test_rows_that_are_no_tensor_are_refused_as_other_arguments_are():
    layer = moe.MoELayer(moe.MoEConfig(**CFG), "cpu")
    with pytest.raises(TypeError, match="expected a torch tensor"):
        layer.forward([1.0], **cpu_weights())


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [False, True])
def test_a_chain_without_copies(swiglu):
    """Bit for bit what three layers with copies in between give."""
    T, d, f, E, k = 300, 128, 256, 4, 2
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, ffn=moe.SWIGLU if swiglu else moe.SILU)
    x, _, dout = layer_case(T, d, f, E, k, swiglu, 1)
    ws = [layer_case(T, d, f, E, k, swiglu, 2 + i)[1] for i in range(3)]

    def depths(layers, apart):
        cks, h = [moe.MoECheckpoint(cfg) for _ in ws], x
        for layer, w, c in zip(layers, ws, cks):
            h = apart(layer.forward(h, **w, checkpoint=c))
        got, dy = [h.clone()], dout
        for layer, c in reversed(list(zip(layers, cks))):
            g = layer.backward(dy, checkpoint=c)
            got += [t.clone() for t in g.values() if t is not None]
            dy = apart(g["dx"])
        return got

    want = depths([moe.MoELayer(cfg) for _ in ws], lambda t: t.clone())
    one = moe.MoELayer(cfg)
    graph = torch.cuda.CUDAGraph()
    for a, b in zip(want, depths([one] * 3, lambda t: t)):
        assert torch.equal(a, b)
    with torch.cuda.graph(graph):
        got = depths([one] * 3, lambda t: t)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and moe.last_device_status() == 0


@pytest.mark.gpu
def test_the_plain_layer_on_its_own_output():
    T, d, f, E, k = 300, 128, 256, 4, 2
    x, w, dout = layer_case(T, d, f, E, k, True, 5)
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k, ffn=moe.SWIGLU)
    other, layer = moe.MoELayer(cfg), moe.MoELayer(cfg)
    want_out = other.forward(other.forward(x, **w).clone(), **w)
    want = other.backward(dout)
    out = layer.forward(layer.forward(x, **w), **w)
    assert torch.equal(out, want_out)
    for n, t in layer.backward(dout).items():
        assert t is None or torch.equal(t, want[n]), n


@pytest.mark.gpu
def test_the_copy_is_made_on_the_given_stream():
    """Queued behind work on that stream, with nothing on the current one to wait for."""
    T, d, f, E, k = 300, 128, 256, 4, 2
    cfg = moe.MoEConfig(T=T, d=d, f=f, E=E, k=k)
    x, w, dout = layer_case(T, d, f, E, k, False, 3)

    def chain(layer, stream, apart):
        cks = [moe.MoECheckpoint(cfg) for _ in range(3)]
        h = x
        for c in cks:
            h = apart(layer.forward(h, **w, checkpoint=c, stream=stream))
        dy = dout
        for c in reversed(cks):
            g = layer.backward(dy, checkpoint=c, stream=stream)
            dy = apart(g["dx"])
        return h, g

    want_h, want = chain(moe.MoELayer(cfg), None, lambda t: t.clone())
    want = {n: t.clone() for n, t in want.items() if t is not None}
    big = torch.randn(4096, 4096, device="cuda")
    s = torch.cuda.Stream()
    layer = moe.MoELayer(cfg)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            big @ big                                  # the stream is busy while the calls are made
    h, g = chain(layer, s, lambda t: t)
    s.synchronize()
    assert torch.equal(h, want_h) and all(torch.equal(g[n], t) for n, t in want.items())
    assert moe.last_device_status() == 0
