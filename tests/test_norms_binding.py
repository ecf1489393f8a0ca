"""What the binding of layer norm, dropout and the residual join does with streams, devices and buffers that are lent to it:
no GPU, with a stand-in for the library, the streams, the devices and the allocator."""

import contextlib
import inspect
from types import SimpleNamespace

import pytest
import torch

BF16, F32, I64 = torch.bfloat16, torch.float32, torch.int64


class DeviceTensor(torch.Tensor):
    """A CPU tensor that says it is on a device (0, or the one it is told), and notes the streams it is recorded on."""
    is_cuda = True

    def get_device(self):
        return self.__dict__.get("place", 0)

    def record_stream(self, stream):
        self.__dict__.setdefault("recorded", []).append(stream)


def tensor(*shape, dtype=F32, place=0):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(DeviceTensor)
    t.__dict__["place"] = place
    return t


@pytest.fixture
def box(monkeypatch):
    from contrastive_late_interaction_gb300 import build
    build.build()
    from contrastive_late_interaction_gb300 import _binding as b, _norms as n
    x = SimpleNamespace(caller=SimpleNamespace(cuda_stream=11), side=SimpleNamespace(cuda_stream=22), device=0, made=[],
                        launched=[], b=b, n=n)
    x.current = x.caller

    @contextlib.contextmanager
    def on(stream):
        before, x.current = x.current, stream
        yield
        x.current = before

    @contextlib.contextmanager
    def at(device):
        before, x.device = x.device, device
        yield
        x.device = before

    def noting(make):
        def call(*args, **kw):
            kw["device"] = "cpu"
            t = make(*args, **kw).as_subclass(DeviceTensor)
            x.made.append((x.current, t))
            return t
        return call

    def packed(args):
        x.launched.append((int.from_bytes(args[-8:], "little"), x.device))
        return 0

    monkeypatch.setattr(n, "_VERBS", {k: (packed, pack) for k, (_, pack) in n._VERBS.items()})
    monkeypatch.setattr(n, "_current_device", lambda: x.device)
    monkeypatch.setattr(b, "_raw_stream", lambda t: x.current.cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: x.current)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "device", at)
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, noting(getattr(torch, name)))
    return x


def calls():
    """A call of every verb, on small inputs."""
    x, y, seed, v = tensor(300, 8, dtype=BF16), tensor(300, 8, dtype=BF16), tensor(2, dtype=I64), tensor(8)
    return {
        "layer_norm": ((x,), dict(gain=v, bias=v)),
        "layer_norm_backward": ((x, y), dict(gain=v, bias=v)),
        "dropout": ((x, 0.1, seed), {}),
        "dropout_backward": ((x, 0.1, seed), {}),
        "dropout_layer_norm": ((x, y, 0.1, seed), dict(gain=v, bias=v)),
        "dropout_layer_norm_backward": ((x, y, 0.1, seed), dict(d_sum=y, gain=v, bias=v)),
    }


def test_every_verb_is_the_packages_and_covered(box):
    import contrastive_late_interaction_gb300 as cli
    from contrastive_late_interaction_gb300 import _NORM_NAMES
    verbs = {v for v in _NORM_NAMES if "stream" in inspect.signature(getattr(box.n, v)).parameters}
    assert verbs == set(calls()) == set(box.n._VERBS)
    for v in _NORM_NAMES:
        assert getattr(cli, v) is getattr(box.n, v)


def test_memory_of_a_call_is_its_streams(box):
    for name, (args, kw) in calls().items():
        for stream, want in ((box.side, 22), (None, 11)):
            box.made.clear(), box.launched.clear()
            made = getattr(box.n, name)(*args, **kw, stream=stream)
            assert box.launched == [(want, 0)], name
            assert box.made and all(s is (stream or box.caller) for s, _ in box.made), name
            for t in made.values():   # a result of another stream is not reused before the caller's has passed it
                assert t.__dict__.get("recorded") == ([box.caller] if stream else None), name
            assert box.current is box.caller


def test_a_call_on_another_device_runs_there(box):
    for name, (args, kw) in calls().items():
        for t in (*args, *kw.values()):
            if isinstance(t, torch.Tensor):
                t.__dict__["place"] = 1
        box.launched.clear()
        getattr(box.n, name)(*args, **kw)
        assert box.launched == [(11, 1)] and box.device == 0, name


def test_tensors_of_two_devices_are_refused(box):
    for name, (args, kw) in calls().items():
        tensors = [t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)]
        for t in {id(t): t for t in tensors}.values():
            if len({id(u) for u in tensors}) == 1:
                continue
            t.__dict__["place"] = 1
            with pytest.raises(box.b.InvalidArgumentError, match="device"):
                getattr(box.n, name)(*args, **kw)
            t.__dict__["place"] = 0
    assert not box.launched


def test_lent_buffers(box):
    """Outputs and workspaces in host memory, of another type or shape, or with gaps, are refused before the launch."""
    b = box.b
    for name, (args, kw) in calls().items():
        verb = getattr(box.n, name)
        made = verb(*args, **kw)
        box.launched.clear()
        for key, t in made.items():
            with pytest.raises(b.InvalidArgumentError):
                verb(*args, **kw, out={key: torch.zeros(*t.shape, dtype=t.dtype)})
            with pytest.raises(b.InvalidArgumentError):
                verb(*args, **kw, out={key: tensor(*t.shape, dtype=torch.float64)})
            with pytest.raises(b.ShapeMismatchError):
                verb(*args, **kw, out={key: tensor(*(s + 1 for s in t.shape), dtype=t.dtype)})
            with pytest.raises(b.InvalidArgumentError, match="device"):
                verb(*args, **kw, out={key: tensor(*t.shape, dtype=t.dtype, place=1)})
            mine = tensor(*t.shape, dtype=t.dtype)
            assert verb(*args, **kw, out={key: mine})[key] is mine
            box.launched.clear()
        if "workspace" in inspect.signature(verb).parameters:
            for bad, error in ((torch.zeros(1 << 20, dtype=torch.uint8), b.InvalidArgumentError),
                               (tensor(1 << 20, dtype=torch.uint8)[::2], b.ShapeMismatchError),
                               (tensor(1 << 20, dtype=torch.uint8, place=1), b.InvalidArgumentError)):
                with pytest.raises(error):
                    verb(*args, **kw, workspace=bad)
        assert not box.launched, name


def test_what_is_not_wanted_is_not_made(box):
    x, seed = tensor(4, 8, dtype=BF16), tensor(2, dtype=I64)
    r = box.n.layer_norm_backward(x, x)
    assert r["d_gain"] is None and r["d_bias"] is None and len(box.made) == 1     # no workspace either
    box.made.clear()
    r = box.n.layer_norm_backward(x, x, gain=tensor(8))
    assert len(box.made) == 2                                                     # none over few rows
    box.made.clear()
    r = box.n.dropout_layer_norm(x, x, 0.1, seed, want_sum=False)
    assert r["sum"] is None and len(box.made) == 1
    box.made.clear()
    r = box.n.dropout_layer_norm_backward(x, x, 0.1, seed, want_d_x=False)
    assert r["d_x"] is None and len(box.made) == 1


def test_types_beside_each_other(box):
    x, f = tensor(4, 8, dtype=BF16), tensor(4, 8)
    assert box.n.layer_norm(f)["output"].dtype is F32
    assert box.n.layer_norm(f, dtype=BF16)["output"].dtype is BF16
    assert box.n.layer_norm_backward(f, x)["d_x"].dtype is F32
    seed = tensor(2, dtype=I64)
    r = box.n.dropout_layer_norm(x, f, 0.1, seed)
    assert r["sum"].dtype is F32 and r["output"].dtype is BF16
    r = box.n.dropout_layer_norm_backward(f, x, 0.1, seed)
    assert r["d_residual"].dtype is F32 and r["d_x"].dtype is BF16
    for bad in (lambda: box.n.layer_norm(x, dtype=F32), lambda: box.n.layer_norm_backward(x, f),
                lambda: box.n.dropout_layer_norm(f, x, 0.1, seed)):
        with pytest.raises(box.b.UnsupportedError):
            bad()
