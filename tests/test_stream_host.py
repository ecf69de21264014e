"""CPU: with `stream=` given, what a call makes comes from that stream's memory.

The caller's stream may still work on memory that its own pool hands out again,
and the other stream does not wait for that.  Streams, allocations and the
library are stand-ins here: recorded is which stream was current when the memory
behind each pointer of the launch was made."""
import contextlib
import ctypes
import types

import pytest
import torch

from bit_fp8_attention_means_gb300 import vc
from paged_case import Case


class Stream:
    """-1 is the device that CPU tensors report."""

    def __init__(self, handle, index=-1):
        self.cuda_stream, self.device = handle, types.SimpleNamespace(index=index)

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream


@pytest.fixture
def world(monkeypatch):
    """The current stream, the launches, the makers of memory (pointer -> stream), the recorded uses."""
    w = {"current": Stream(1), "launches": [], "made": {}, "used": []}

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                if name.endswith("workspace"):
                    return 4096
                w["launches"].append((name, args))
                return 0
            return entry

    @contextlib.contextmanager
    def use(stream):
        before, w["current"] = w["current"], stream
        try:
            yield
        finally:
            w["current"] = before

    def recording(make):
        def wrapper(*args, **kw):
            t = make(*args, **{k: "cpu" if k == "device" and v == -1 else v for k, v in kw.items()})
            w["made"][t.data_ptr()] = w["current"].cuda_stream
            return t
        return wrapper

    library = Library()
    monkeypatch.setattr(vc, "lib", lambda: library)
    monkeypatch.setattr(vc, "_need_cuda", lambda dev: None)
    vc._attn_paged_bytes.cache_clear()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w["current"])
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: w["current"].cuda_stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w["used"].append((t.data_ptr(), s.cuda_stream)), raising=False)
    for name in ("empty", "empty_like", "empty_strided", "zeros"):
        monkeypatch.setattr(torch, name, recording(getattr(torch, name)))
    yield w
    vc._attn_paged_bytes.cache_clear()


def pointers(args):
    return {int(a.value if isinstance(a, ctypes.c_void_p) else a) for a in args
            if isinstance(a, ctypes.c_void_p) and a.value or isinstance(a, int) and a > 1 << 20}


def on_side(w, call, made):
    """Runs call(stream=side): one launch, there, with `made` new tensors, all of that stream's memory, of which
    those returned are recorded as used by the caller's stream."""
    side = Stream(2)
    w["made"].clear()
    out = call(stream=side)
    (name, args), = w["launches"]
    w["launches"].clear()
    handle = args[13 if name == "vc_attn_fwd_debug" else -1]
    handle = handle.value if isinstance(handle, ctypes.c_void_p) else handle
    assert handle == 2, name
    new = pointers(args) & set(w["made"])
    assert len(new) == made and all(w["made"][p] == 2 for p in new), name
    outs = [t for t in (out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,)) if t is not None]
    assert all((t.data_ptr(), 1) in w["used"] for t in outs if t.data_ptr() in new), name
    assert w["current"].cuda_stream == 1
    return out


def test_paged_calls_make_their_memory_on_the_given_stream(world):
    c = Case(n=[2], kv=[5], H=2)
    cache, args = c.cache(), c.args("cpu")
    on_side(world, lambda stream: vc.vc_cache_append(c.K, c.V, cache, *args, stream=stream), 0)
    on_side(world, lambda stream: vc.vc_cache_read(cache, *args, 2, stream=stream), 2)
    on_side(world, lambda stream: vc.vc_cache_read(cache, *args, 2, K=torch.zeros_like(c.K), stream=stream), 1)
    O, lse = on_side(world, lambda stream: vc.vc_attn_paged(c.Q, cache, *args, stream=stream), 3)
    ws = torch.zeros(4096, dtype=torch.uint8)
    got = on_side(world, lambda stream: vc.vc_attn_paged(c.Q, cache, *args, O=O, lse=lse, workspace=ws, stream=stream), 0)
    assert got[0] is O and got[1] is lse
    # the current stream, given or not: no detour
    for stream in (None, Stream(1)):
        vc.vc_attn_paged(c.Q, cache, *args, stream=stream)
        assert world["launches"].pop()[1][-1] == 1


def test_whole_sequence_calls_make_their_memory_on_the_given_stream(world):
    x = torch.zeros((1, 256, 2, 64), dtype=torch.bfloat16)
    shape = vc.shape_of(x)
    cent, labels, perm = on_side(world, lambda stream: vc.vc_cluster(x, 4, 1, stream=stream), 4)
    on_side(world, lambda stream: vc.vc_cluster(x, 4, 1, True, cent, labels, perm, stream=stream, block_fill=1), 1)
    qz = on_side(world, lambda stream: vc.vc_quantize(x, x, x, perm, stream=stream), 8)
    on_side(world, lambda stream: vc.vc_quantize(x, x, x, perm, out=qz, vbits=4, stream=stream), 1)
    for fn in (vc.vc_quantize_ex, vc.vc_quantize_staged):
        on_side(world, lambda stream: fn(x, x, x, hadamard=1, stream=stream), 8)
    O = on_side(world, lambda stream: vc.vc_attn_fwd(qz, shape, stream=stream), 1)
    on_side(world, lambda stream: vc.vc_attn_fwd(qz, shape, O=O, exact_margin=2.0, stream=stream), 0)
    on_side(world, lambda stream: vc.vc_attn_fwd(qz, shape, debug=(0, 0), stream=stream), 3)
    values = torch.zeros(8)
    on_side(world, lambda stream: vc.vc_debug_e4m3_encode(values, stream=stream), 1)


def test_stream_of_another_device_is_refused(world):
    c = Case(n=[2], kv=[5], H=2)
    cache, args = c.cache(), c.args("cpu")
    for call in (lambda s: vc.vc_cache_append(c.K, c.V, cache, *args, stream=s), lambda s: vc.vc_cache_read(cache, *args, 2, stream=s),
                 lambda s: vc.vc_attn_paged(c.Q, cache, *args, stream=s)):
        with pytest.raises(ValueError, match="device"):
            call(Stream(3, 1))
    assert not world["launches"]
