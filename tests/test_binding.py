"""The Python binding's own behaviour, without a GPU: CUDA calls, streams and allocations are stand-ins."""

import contextlib
import importlib.util
import os
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


def build_script():
    path = os.path.join(os.path.dirname(kv.__file__), "build.py")
    spec = importlib.util.spec_from_file_location("kvattn_build_under_test", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_binding_is_built_again_for_another_torch_or_python(monkeypatch, tmp_path):
    """The compiled binding is of one torch's and one Python's interface, whatever the files' times say."""
    b = build_script()
    monkeypatch.setattr(b, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(b, "MARSHAL_KEY", str(tmp_path / "key"))
    built = []

    def compiler(cmd, check):
        built.append([a for a in cmd if a.startswith("-DKVATTN_BUILT_FOR")])
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b.subprocess, "run", compiler)
    b.build_binding()
    b.build_binding()
    assert len(built) == 1 and built[0] == [f'-DKVATTN_BUILT_FOR="{b.binding_key()}"']
    version = b.importlib.metadata.version
    monkeypatch.setattr(b.importlib.metadata, "version", lambda name: "9.9" if name == "torch" else version(name))
    b.build_binding()
    b.build_binding()
    assert len(built) == 2 and "torch 9.9" in built[1][0]
    config = b.sysconfig.get_config_var
    monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else config(name))
    b.build_binding()
    assert len(built) == 3
    os.utime(b.MARSHAL, (1, 1))     # older than its sources
    b.build_binding()
    assert len(built) == 4
    os.remove(b.MARSHAL_KEY)
    b.build_binding()
    assert len(built) == 5


def test_a_binding_of_another_torch_is_refused(monkeypatch):
    assert kv._marshal.built_for.startswith(f"torch {torch.__version__}")
    monkeypatch.setattr(torch, "__version__", "1.0")
    with pytest.raises(ImportError, match="torch 1.0"):
        kv._load_marshal()


def test_shapes_are_refused_by_value_without_a_workspace(monkeypatch):
    """The sizes of the call's own workspace come from the arguments before the compiled checks see them."""
    monkeypatch.setattr(kv, "_here", lambda t, s: (0, 0))
    for q, cache, table, prefix in [(_q[0], _pool, _table, _prefix), (_q, _pool[0], _table, _prefix),
                                    (_q, _pool, _table[0], _prefix), (_q, _pool, None, _prefix),
                                    (_q, _pool, _table, None), (_q, _pool, _table, _prefix[None])]:
        with pytest.raises(ValueError):
            kv.attn_decode_shared(q, cache, cache, _n, table, prefix, _o)
        with pytest.raises(ValueError):
            kv.attn_decode_shared_fp8(q, cache, cache, _scale, _scale, _n, table, prefix, _o)
    for q, cache, table in [(_q[0], _cache, None), (_q, _cache[0], None), (_q, _pool, _table[0])]:
        with pytest.raises(ValueError):
            kv.attn_decode_window(q, cache, cache, _n, _o, 9, page_table=table)
        with pytest.raises(ValueError):
            kv.attn_decode_window_fp8(q, cache, cache, _scale, _scale, _n, _o, 9, page_table=table)
