"""What the binding does with streams, and with buffers that are lent to it: no GPU, with a stand-in for the library, the
streams and the allocator that notes which stream was current."""

import contextlib
import inspect
from types import SimpleNamespace

import pytest
import torch

BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


class DeviceTensor(torch.Tensor):
    """A CPU tensor that says it is on a device, and notes the streams it is recorded on."""
    is_cuda = True

    def record_stream(self, stream):
        self.__dict__.setdefault("recorded", []).append(stream)


def tensor(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(DeviceTensor)


class Box:
    """The stand-ins' state: the current stream, the streams of allocations, the streams of launches."""

    def __init__(self):
        self.caller, self.side = SimpleNamespace(cuda_stream=11), SimpleNamespace(cuda_stream=22)
        self.current, self.made, self.launched = self.caller, [], []


@pytest.fixture
def box(monkeypatch):
    from contrastive_late_interaction_gb300 import build
    build.build()
    from contrastive_late_interaction_gb300 import _binding as b
    x = Box()

    @contextlib.contextmanager
    def on(stream):
        before, x.current = x.current, stream
        yield
        x.current = before

    def noting(make):
        def call(*args, **kw):
            kw["device"] = "cpu"
            t = make(*args, **kw).as_subclass(DeviceTensor)
            x.made.append((x.current, t))
            return t
        return call

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_workspace_bytes"):
                    return 4096
                if name == "cli_status_name":
                    return b"refused"
                a = args[0]._obj if hasattr(args[0], "_obj") else None
                while a is not None and not hasattr(a, "stream"):
                    a = getattr(a, "base", None) or a.args
                x.launched.append(a.stream if a is not None else args[3].value)
                return 0
            return call

    def packed(args):
        x.launched.append(int.from_bytes(args[-8:], "little"))
        return 0

    monkeypatch.setattr(b, "lib", Library())
    monkeypatch.setattr(b, "_ROTARY", {k: packed for k in b._ROTARY})
    monkeypatch.setattr(b, "_ATTENTION", {k: (packed, lambda a: 4096) for k in b._ATTENTION})
    monkeypatch.setattr(b, "_raw_stream", lambda *a: (a[0] if len(a) == 2 and a[0] is not None else x.current).cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: x.current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", on)
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, noting(getattr(torch, name)))
    x.b = b
    return x


def calls(b):
    """A call of every verb that takes a stream, on small inputs."""
    e, one = tensor(4, 8, dtype=BF16), tensor(1)
    edges = (tensor(5, dtype=I64), tensor(0, dtype=I32))
    scores, off = tensor(4, 4), tensor(3, dtype=I64)
    tape = (e, off, e, off)
    q, table, gain = tensor(4, 2, 8, dtype=BF16), tensor(9, 4, 2), tensor(8)
    lse = tensor(4, 2)
    return {
        "selftest_bounded_wait": dict(),
        "pair_loss_sigmoid_fwd_bwd": dict(a=(e, one, one, edges)),
        "pair_loss_sigmoid_groups_fwd_bwd": dict(a=(e, tensor(4, dtype=I32), one, one, edges)),
        "pair_loss_sigmoid_matryoshka_fwd_bwd": dict(a=(e, [8], one, one, edges)),
        "pair_loss_sigmoid_scores_fwd_bwd": dict(a=(scores, one, one, edges)),
        "pair_loss_scores_fwd_bwd": dict(a=("ranked", scores, one, one, edges)),
        "maxsim_scores": dict(a=tape),
        "maxsim_scores_named": dict(a=(*tape, edges)),
        "maxsim_backward": dict(a=(*tape, tensor(2, 4, dtype=I32), scores)),
        "maxsim_backward_named": dict(a=(*tape, tensor(2, 4, dtype=I32), scores, edges)),
        "rotary_table": dict(a=(9, 8)),
        "rotary_heads": dict(a=(q, table), k=dict(k=q)),
        "rotary_heads_backward": dict(a=(q, table), k=dict(d_k=q)),
        "norm_rotary_heads": dict(a=(q, table), k=dict(k=q)),
        "norm_rotary_heads_backward": dict(a=(q, q, table), k=dict(q_gain=gain, k=q, d_k=q, k_gain=gain)),
        "cross_attention": dict(a=(q, off, q, q, off)),
        "cross_attention_backward": dict(a=(q, off, q, q, off, q, lse, q)),
    }


def verbs():
    from contrastive_late_interaction_gb300 import _BINDING_NAMES
    from contrastive_late_interaction_gb300 import _binding as b
    return sorted(n for n in _BINDING_NAMES if callable(getattr(b, n)) and inspect.isfunction(getattr(b, n))
                  and "stream" in inspect.signature(getattr(b, n)).parameters)


def test_every_verb_with_a_stream_is_covered(box):
    assert verbs() == sorted(calls(box.b))


def test_memory_of_a_call_on_a_stream_is_that_streams(box):
    """Scratch that a verb drops goes back to the stream that its kernels run on, and results are made there too."""
    for name, c in calls(box.b).items():
        box.made.clear(), box.launched.clear()
        made = getattr(box.b, name)(*c.get("a", ()), **c.get("k", {}), stream=box.side)
        assert box.launched == [22], name
        assert box.made and all(s is box.side for s, _ in box.made), name
        for t in made.values():
            if t is not None:   # and are not reused before the caller's stream has passed them
                assert t.__dict__.get("recorded") == [box.caller], name
        assert box.current is box.caller


def test_memory_of_a_call_without_a_stream_is_the_current_ones(box):
    for name, c in calls(box.b).items():
        box.made.clear(), box.launched.clear()
        getattr(box.b, name)(*c.get("a", ()), **c.get("k", {}))
        assert box.launched == [11], name
        assert box.made and all(s is box.caller for s, _ in box.made), name


def test_lent_buffers_are_device_memory(box):
    """A workspace, a status or an output in host memory, or a workspace with gaps, is refused before the launch."""
    b = box.b
    host, gaps = torch.ones(8192, dtype=torch.uint8), tensor(16384, dtype=torch.uint8)[::2]
    for name, c in calls(b).items():
        takes = inspect.signature(getattr(b, name)).parameters
        call = lambda **kw: getattr(b, name)(*c.get("a", ()), **c.get("k", {}), **kw)  # noqa: E731
        box.launched.clear()
        if "workspace" in takes:
            with pytest.raises(b.InvalidArgumentError, match="workspace"):
                call(workspace=host)
            with pytest.raises(b.ShapeMismatchError, match="workspace"):
                call(workspace=gaps)
        if "device_status" in takes:
            with pytest.raises(b.InvalidArgumentError, match="device_status"):
                call(device_status=torch.ones(1, dtype=torch.int32))
        if "out" in takes:
            for key, t in call().items():
                if t is not None and key != "device_status":
                    with pytest.raises(b.InvalidArgumentError):
                        call(out={key: torch.ones(*t.shape, dtype=t.dtype)})
            box.launched.clear()
        assert not box.launched, name


def test_a_lent_workspace_counts_in_bytes(box):
    b = box.b
    q, off = tensor(4, 2, 8, dtype=BF16), tensor(3, dtype=I64)
    seen = []
    b._ATTENTION["cross_attention"] = (lambda a: seen.append(int.from_bytes(a[-24:-16], "little")) or 0, lambda a: 0)
    b.cross_attention(q, off, q, q, off, workspace=tensor(512))
    assert seen == [2048]


def test_the_packages_names_follow_the_binding(box, monkeypatch):
    """A name replaced in the binding is the package's too, whether it was looked up before or not."""
    import contrastive_late_interaction_gb300 as cli
    assert cli.rotary_table is box.b.rotary_table
    other = lambda *a: None  # noqa: E731
    monkeypatch.setattr(box.b, "rotary_table", other)
    assert cli.rotary_table is other


def test_what_a_call_cannot_do_without_is_asked_for(box):
    b = box.b
    q, off = tensor(4, 2, 8, dtype=BF16), tensor(3, dtype=I64)
    with pytest.raises(b.InvalidArgumentError):
        b.cross_attention_backward(q, off, q, q, off, q, None, q)     # a forward without want_lse gives None
    with pytest.raises(b.InvalidArgumentError):
        b.cross_attention(q, off, q, q, None)
    assert not box.launched
