"""The training operators' binding on the CPU: what it makes of its arguments and which streams it orders. The
tensors only claim to be on the device and the calls of the library are recorded, not made."""
import gc
import weakref

import pytest
import torch

import gram_hash_embedding_gb300 as geng


class OnDevice(torch.Tensor):
    """A host tensor that says it is a CUDA tensor and notes the streams it is marked as used on."""

    is_cuda = True

    def record_stream(self, stream):
        self.__dict__.setdefault("streams", []).append(stream.cuda_stream)


def on_device(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


class Stream:
    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def wait_event(self, event):
        self.log.append(("wait", self.cuda_stream, event.of))


@pytest.fixture
def device(monkeypatch):
    """torch.cuda's streams, as far as a prepared call uses them; `log` has what happened in order."""
    geng.build()

    class Device:
        log, capturing = [], False

        def use(self, handle):
            self.current = Stream(handle, self.log)

    d = Device()
    d.log = []
    d.use(10)

    class Event:
        def record(self):
            self.of = d.current.cuda_stream
            d.log.append(("record", self.of))

    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: d.current)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: d.capturing)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: Stream(handle, d.log))
    monkeypatch.setattr(geng, "_current_stream_handle", lambda: d.current.cuda_stream)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).as_subclass(OnDevice))

    class Lib:
        real = geng._lib()
        engram_grad_norm_workspace = staticmethod(real.engram_grad_norm_workspace)

        @staticmethod
        def engram_grad_clip(*args):
            d.log.append(("call", args[-1]))
            return geng.OK
        engram_grad_norm = engram_grad_clip

    monkeypatch.setattr(geng, "_lib", Lib)
    return d


def _marked(clip):
    """of the norm and the workspace: the streams they are marked as used on"""
    return [t.__dict__.get("streams", []) for t in (clip.norm, clip._keep[-1])]


@pytest.mark.parametrize("given", [None, "object", "handle"])
def test_prepared_clip_orders_its_memory(device, given):
    """Its norm and workspace may still be in use by the constructing stream, and their calls on another
    stream may outlast the object: the other stream waits once, and both tensors are marked as used on it."""
    stream = {None: None, "object": Stream(20, device.log), "handle": 20}[given]
    clip = geng.PreparedGradClip([on_device(5)], 1.0, stream=stream)
    if given is None:
        clip()
        assert device.log[-1] == ("call", 10) and _marked(clip) == [[], []]  # the constructing stream needs neither
        device.use(20)
    for _ in range(2):
        clip()
    waits = [e for e in device.log if e[0] == "wait"]
    assert waits == [("wait", 20, 10)] and _marked(clip) == [[20], [20]]
    assert device.log.index(waits[0]) < device.log.index(("call", 20)) and device.log[-1] == ("call", 20)
    if given is None:
        device.use(30)
        device.capturing = True
        clip()  # a capture cannot wait for what is outside it
        device.capturing = False
        assert device.log[-1] == ("call", 30) and len([e for e in device.log if e[0] == "wait"]) == 1
        clip()
        assert device.log[-2:] == [("wait", 30, 10), ("call", 30)]


def test_prepared_clip_leaves_a_given_norm_alone(device):
    norm = on_device()
    clip = geng.PreparedGradClip([on_device(5)], 1.0, norm=norm)
    device.use(20)
    assert clip() is norm and _marked(clip) == [[], [20]]


def test_prepared_clip_keeps_its_tensors(device):
    """Their addresses are marshalled, so they stay whatever the caller does with the lists that were passed."""
    grads, outs = [on_device(5, 2), on_device(3)], [on_device(5, 2), on_device(3)]
    counts = [on_device(1, dtype=torch.int64), None]
    kept = [weakref.ref(t) for t in grads + outs + counts[:1]]
    clip = geng.PreparedGradClip(grads, 1.0, out=outs, counts=counts)
    grads.clear()
    outs.clear()
    counts[0] = None
    gc.collect()
    assert all(r() is not None for r in kept)
    clip()
    del clip
    gc.collect()
    assert all(r() is None for r in kept)


def test_prepared_lookup_keeps_its_tensors(device, monkeypatch):
    """The same for the prepared hash + lookup."""
    monkeypatch.setattr(geng, "engram_state_layout", lambda state: dict(
        n_layers=2, max_ngram=2, n_heads=1, head_dim=16, block=16, scale_dtype=geng.SCALE_F32))
    monkeypatch.setattr(geng._lib, "engram_hash_lookup", staticmethod(lambda *args: geng.OK), raising=False)
    ids, start = on_device(1, 4, dtype=torch.int64), on_device(1, dtype=torch.int32)
    W = [on_device(7, 16, dtype=torch.uint8) for _ in range(2)]
    S = [on_device(7, 1) for _ in range(2)]
    out = [on_device(4, 16, dtype=torch.bfloat16) for _ in range(2)]
    kept = [weakref.ref(t) for t in W + S + out]
    call = geng.PreparedHashLookup(1, ids, start, W, S, out)
    for ts in (W, S, out):
        ts.clear()
    gc.collect()
    assert all(r() is not None for r in kept)
    call()


def test_empty_gradient_with_a_count():
    """What engram_embed_grad returns for an empty batch, grad [0, dim] and a count, goes into the norm and the
    clip like any other; an empty gradient without rows is still refused."""
    count = on_device(1, dtype=torch.int64)
    arr, n = geng._tensor_list([on_device(0, 128), on_device(3)], None, [count, None])
    assert n == 2 and list(arr[3::6]) == [0, 3]
    assert arr[2] == count.data_ptr() and arr[4] & 0xffffffff == 128
    with pytest.raises(ValueError, match="must be"):
        geng._tensor_list([on_device(0)], None, [count])


def _both_forms(device, monkeypatch, idx, dout, dim):
    """(the sparse form's grad, the width that each form passes to the library) for arguments of these shapes"""
    seen = []
    monkeypatch.setattr(geng._lib, "engram_embed_grad_workspace", geng._lib.real.engram_embed_grad_workspace, raising=False)
    for name in ("engram_embed_grad", "engram_embed_grad_dense"):
        monkeypatch.setattr(geng._lib, name, staticmethod(lambda *a: seen.append(a[8]) or geng.OK), raising=False)
    idx, dout = on_device(*idx, dtype=torch.int64), on_device(*dout)
    grad = geng.engram_embed_grad(idx, dout, 9)[1]
    geng.engram_embed_grad_dense(idx, dout, on_device(9, dim))
    return grad, seen


@pytest.mark.parametrize("idx,dout,dim", [((0, 3), (0, 48), 16), ((0, 3), (0, 3, 16), 16), ((0,), (0, 16), 16), ((0, 5, 7), (0, 5, 7, 8), 8),
                                          ((0, 5, 7), (0, 280), 8), ((4, 0), (4, 0, 16), 16), ((0,), (0,), 1), ((0, 1), (0, 16), 16)])
def test_empty_batch_has_the_width_of_a_full_one(device, monkeypatch, idx, dout, dim):
    """The same layouts with and without tokens: rows as wide, in both forms of the gradient."""
    full = [tuple(2 if n == 0 else n for n in shape) for shape in (idx, dout)]
    for shapes in ((idx, dout), full):
        grad, seen = _both_forms(device, monkeypatch, *shapes, dim)
        assert grad.shape[1] == dim and seen == [dim, dim], shapes


@pytest.mark.parametrize("idx,dout", [((0, 3), (0, 47)), ((0, 3), (0,)), ((2, 3), (0, 48)), ((0, 3), (2, 48)), ((0, 3), (0, 0)), ((0,), ()),
                                      ((2, 3), (2, 47))])
def test_gradients_that_do_not_fit_their_ids(device, monkeypatch, idx, dout):
    with pytest.raises(ValueError, match="does not hold one row"):
        _both_forms(device, monkeypatch, idx, dout, 16)


def test_clip_without_a_bound_is_refused(device):
    """engram_grad_clip with max_norm None is no call for the norm alone (PreparedGradClip's None is)."""
    with pytest.raises(TypeError, match="max_norm"):
        geng.engram_grad_clip([on_device(5)], None)
    assert device.log == []
    geng.engram_grad_clip([on_device(5)], 1.0)
    geng.engram_grad_norm([on_device(5)])
    geng.PreparedGradClip([on_device(5)], None)()
    assert [e[0] for e in device.log if e[0] == "call"] == ["call"] * 3


@pytest.mark.parametrize("shape", [(2, 2 ** 32), (1, 2 ** 32 + 5), (2, 2 ** 31), (3, 2 ** 20, 2 ** 12)])
def test_counted_rows_too_long_for_the_library(shape):
    """A row length is a 32-bit field beside the tensor's type; a longer one would run into it."""
    long_rows = torch.empty(shape, device="meta", dtype=torch.bfloat16).as_subclass(OnDevice)
    count = on_device(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="rows of"):
        geng._tensor_list([long_rows], None, [count])
    assert geng._tensor_list([long_rows], None, [None])[1] == 1  # without a count it is a flat list of values
    assert geng._tensor_list([torch.empty((2, 2 ** 31 - 1), device="meta").as_subclass(OnDevice)], None, [count])[1] == 1


def test_sizes_beyond_the_librarys_fields(device):
    """Widths, columns and copies are 32-bit arguments; a larger one is refused, not cut to its low bits."""
    meta = lambda *shape, dtype=torch.float32: torch.empty_strided(
        shape, [torch.Size(shape[i + 1:]).numel() for i in range(len(shape))], device="meta", dtype=dtype).as_subclass(OnDevice)
    idx, wide = on_device(1, 1, dtype=torch.int64), 2 ** 32 + 8
    many = meta(1, wide, dtype=torch.int64)
    for call in (lambda: geng.engram_embed(idx, meta(1, wide), out=meta(1, 1, wide)),
                 lambda: geng.engram_embed(many, on_device(1, 8), out=meta(1, wide, 8)),
                 lambda: geng.engram_embed_grad(idx, meta(1, wide), 1, grad=meta(1, wide)),
                 lambda: geng.engram_embed_grad_dense(idx, meta(1, wide), meta(1, wide)),
                 lambda: geng.engram_gate_grad(*[meta(1, 1, wide, dtype=torch.bfloat16)] + [meta(1, 2 * wide, dtype=torch.bfloat16)] +
                                               [meta(1, wide, dtype=torch.bfloat16)] * 2 + [meta(1, 1, wide, dtype=torch.bfloat16)])):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
