"""The Python binding's own behaviour, without a GPU: CUDA calls, streams and allocations are stand-ins."""

import contextlib
import types

import pytest
import torch

import kv_cache_decode_attn_b200 as kv


class Allocations:
    """Streams (None: the current one) that torch.empty was called on."""

    def __init__(self, monkeypatch):
        self.on, stack = [], [None]

        @contextlib.contextmanager
        def stream(s):
            stack.append(s)
            yield
            stack.pop()

        def empty(*shape, dtype=None, device=None):
            self.on.append(stack[-1])
            return torch.zeros(shape if len(shape) > 1 else shape[0], dtype=dtype)

        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default",))
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0))
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(torch, "empty", empty)


class Launches:
    """The library: sizes are its own, every other call succeeds and does nothing."""

    def __getattr__(self, name):
        return getattr(_lib, name) if name.endswith("_bytes") else lambda *a: kv.ATTN_OK


_lib = kv.lib
_q, _o = torch.zeros(2, 1, 8, 128), torch.zeros(2, 1, 8, 128)
_cache, _pool = torch.zeros(2, 64, 2, 128), torch.zeros(9, 16, 2, 128)
_n, _scale = torch.zeros(2, dtype=torch.int32), torch.ones(2)
_table, _prefix = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)


@pytest.mark.parametrize("stream,used", [(None, None), (7, ("external", 7)), (0, ("default",))])
@pytest.mark.parametrize("call", [
    lambda s: kv.attn_decode(_q, _cache, _cache, _n, _o, stream=s),
    lambda s: kv.attn_decode_fp8(_q, _cache, _cache, _scale, _scale, _n, _o, stream=s),
    lambda s: kv.attn_decode_window(_q, _cache, _cache, _n, _o, 9, stream=s),
    lambda s: kv.attn_decode_window_fp8(_q, _cache, _cache, _scale, _scale, _n, _o, 9, stream=s),
    lambda s: kv.attn_decode_shared(_q, _pool, _pool, _n, _table, _prefix, _o, stream=s),
    lambda s: kv.attn_decode_shared_fp8(_q, _pool, _pool, _scale, _scale, _n, _table, _prefix, _o, stream=s),
    lambda s: kv.rope_table(8, 64, stream=s),
], ids=["decode", "decode_fp8", "window", "window_fp8", "shared", "shared_fp8", "rope_table"])
def test_calls_allocate_on_the_stream_they_launch_on(monkeypatch, call, stream, used):
    """A workspace of the current stream's pool would be handed out again there while another stream's
    kernels still write their partials to it."""
    made = Allocations(monkeypatch)
    monkeypatch.setattr(kv, "lib", Launches())
    monkeypatch.setattr(kv, "_marshal", Launches())
    monkeypatch.setattr(kv, "_here", lambda t, s: (0, s or 0))
    monkeypatch.setattr(kv, "_dev", lambda *a: 0)
    monkeypatch.setattr(kv, "_codes", lambda *a: 0)
    monkeypatch.setattr(kv, "_out_dtype", lambda o: 0)
    monkeypatch.setattr(kv, "_raw_stream", None)
    call(stream)
    assert made.on == [used]
