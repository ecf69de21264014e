"""CPU: with `stream=` given, what the rotary, page and shared-prefix calls make comes from that stream's memory (the
stand-ins of test_stream_host.py)."""
import pytest
import torch

from bit_fp8_attention_means_gb300 import vc
from paged_case import Case
from test_stream_host import Stream, on_side, world  # noqa: F401


@pytest.fixture(autouse=True)
def fresh_sizes():
    """What stands in for the library gives other workspace sizes: none of them is kept."""
    for f in (vc._attn_shared_bytes, vc._reserve_bytes):
        f.cache_clear()
    yield
    for f in (vc._attn_shared_bytes, vc._reserve_bytes):
        f.cache_clear()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_new_calls_make_their_memory_on_the_given_stream(world):  # noqa: F811
    c = Case(n=[2], kv=[5], H=2)
    cache, args, rope = c.cache(), c.args("cpu"), vc.make_rope(64, device="cpu")
    pool, pos = vc.alloc_pool(c.pages, "cpu"), ints(1, 2)
    on_side(world, lambda stream: vc.vc_rope(c.Q, rope, pos=pos, stream=stream), 1)
    on_side(world, lambda stream: vc.vc_rope(c.Q, rope, cu=args[0], kv_len=args[1], out=c.Q, stream=stream), 0)
    on_side(world, lambda stream: vc.vc_rope(c.Q.transpose(0, 1).contiguous().transpose(0, 1), rope, pos=pos, stream=stream), 1)
    on_side(world, lambda stream: vc.vc_cache_append_rope(c.Q, c.K, c.V, cache, *args, rope, stream=stream), 1)
    on_side(world, lambda stream: vc.vc_cache_append_rope(None, c.K, c.V, cache, *args, rope, pos=pos, stream=stream), 0)
    on_side(world, lambda stream: vc.vc_pages_reserve(cache, pool, *args, 2, stream=stream), 1)
    ws = torch.zeros(4096, dtype=torch.uint8)
    on_side(world, lambda stream: vc.vc_pages_reserve(cache, pool, *args, 2, workspace=ws, stream=stream), 0)
    on_side(world, lambda stream: vc.vc_pages_compact(cache, pool, args[2], stream=stream), 2)
    on_side(world, lambda stream: vc.vc_pages_compact(cache, pool, args[2], used=ints(0), workspace=ws, stream=stream), 0)
    new = torch.zeros((1, 3), dtype=torch.int32)
    on_side(world, lambda stream: vc.vc_pages_fork(cache, pool, args[2], args[1], ints(0), new, ints(0), stream=stream), 0)
    on_side(world, lambda stream: vc.vc_pages_trim(cache, pool, args[2], args[1], ints(0), stream=stream), 0)
    on_side(world, lambda stream: vc.vc_cache_copy(cache, cache, ints(0), ints(1), stream=stream), 0)
    groups = ints(0, 1), ints(3)
    O, lse = on_side(world, lambda stream: vc.vc_attn_paged_shared(c.Q, cache, *args, *groups, stream=stream), 3)
    on_side(world, lambda stream: vc.vc_attn_paged_shared(c.Q, cache, *args, *groups, O=O, lse=lse, workspace=ws, stream=stream), 0)
    # the current stream, given or not: no detour
    for stream in (None, Stream(1)):
        vc.vc_attn_paged_shared(c.Q, cache, *args, *groups, stream=stream)
        assert world["launches"].pop()[1][-1] == 1


def test_stream_of_another_device_is_refused(world):  # noqa: F811
    c = Case(n=[2], kv=[5], H=2)
    cache, args, rope, pool = c.cache(), c.args("cpu"), vc.make_rope(64, device="cpu"), vc.alloc_pool(c.pages, "cpu")
    new = torch.zeros((1, 3), dtype=torch.int32)
    for call in (lambda s: vc.vc_rope(c.Q, rope, pos=ints(1, 2), stream=s), lambda s: vc.vc_cache_append_rope(c.Q, c.K, c.V, cache, *args, rope, stream=s),
                 lambda s: vc.vc_pages_reserve(cache, pool, *args, 2, stream=s), lambda s: vc.vc_pages_compact(cache, pool, args[2], stream=s),
                 lambda s: vc.vc_pages_fork(cache, pool, args[2], args[1], ints(0), new, ints(0), stream=s),
                 lambda s: vc.vc_pages_trim(cache, pool, args[2], args[1], ints(0), stream=s), lambda s: vc.vc_cache_copy(cache, cache, ints(0), ints(1), stream=s),
                 lambda s: vc.vc_attn_paged_shared(c.Q, cache, *args, ints(0, 1), ints(3), stream=s)):
        with pytest.raises(ValueError, match="device"):
            call(Stream(3, 1))
    assert not world["launches"]
