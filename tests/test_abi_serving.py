"""Argument checks of the window, shared-prefix and norm-rotate-append calls (CPU: they return
before anything touches a device), and the sizes of their workspaces."""

import pytest
import torch

import kv_cache_decode_attn_b200 as kv

P, BIG = 256, 1 << 40     # a fake, aligned, never dereferenced pointer; a size above any workspace
INVALID, UNSUPPORTED, WORKSPACE = kv.ATTN_ERR_INVALID_ARG, kv.ATTN_ERR_UNSUPPORTED, kv.ATTN_ERR_WORKSPACE


def caller(fn, names, defaults):
    def call(**kw):
        a = dict(defaults, **kw)
        assert set(kw) <= set(defaults)
        return fn(*[a[n] for n in names.split()], None)
    return call


prefill_window = caller(kv.lib.attn_prefill_window, "q k v o od lse B Hq Hkv N d scale window sinks",
                        dict(q=P, k=P, v=P, o=P, od=0, lse=None, B=2, Hq=4, Hkv=2, N=9, d=64, scale=0.1, window=4, sinks=1))
chunk_window = caller(kv.lib.attn_prefill_cache_window,
                      "q k v sl pt mb nb cap o od lse B Nq Hq Hkv d scale window sinks",
                      dict(q=P, k=P, v=P, sl=P, pt=None, mb=0, nb=0, cap=100, o=P, od=0, lse=None, B=2, Nq=10, Hq=8, Hkv=2,
                           d=128, scale=0.1, window=4, sinks=1))
_decode = dict(q=P, k=P, v=P, ks=P, vs=P, sl=P, pt=None, mb=0, nb=0, cap=100, msk=0, o=P, od=0, lse=None, B=2, T=1, Hq=8,
               Hkv=2, d=128, scale=0.1, window=4, sinks=1, ns=0, ws=P, wsb=BIG)
decode_window = caller(kv.lib.attn_decode_window,
                       "q k v sl pt mb nb cap msk o od lse B T Hq Hkv d scale window sinks ns ws wsb", _decode)
decode_window_fp8 = caller(kv.lib.attn_decode_window_fp8,
                           "q k v ks vs sl pt mb nb cap msk o od lse B T Hq Hkv d scale window sinks ns ws wsb", _decode)
_shared = dict(q=P, k=P, v=P, ks=P, vs=P, sl=P, pt=P, mb=8, nb=50, pre=P, npre=3, msk=0, o=P, od=0, lse=None, B=2, T=1,
               Hq=8, Hkv=2, d=128, scale=0.1, causal=1, ns=0, ws=P, wsb=BIG)
shared = caller(kv.lib.attn_decode_shared, "q k v sl pt mb nb pre npre msk o od lse B T Hq Hkv d scale causal ns ws wsb",
                _shared)
shared_fp8 = caller(kv.lib.attn_decode_shared_fp8,
                    "q k v ks vs sl pt mb nb pre npre msk o od lse B T Hq Hkv d scale causal ns ws wsb", _shared)
_rope = dict(kc=P, vc=P, q=1 << 20, k=1 << 21, v=1 << 22, qs=512, ks=256, vs=256, qo=1 << 23, ko=1 << 24, ksc=P, vsc=P,
             qw=P, kw=P, eps=1e-6, rope=P, rows=100, rot=128, il=0, pos=P, pt=None, mb=0, nb=0, cap=100, B=2, T=3, Hq=4,
             Hkv=2, d=128)
qk = caller(kv.lib.qk_norm_rope, "q k qs ks qo ko qw kw eps rope rows rot il pos B T Hq Hkv d", _rope)
append = caller(kv.lib.kv_append_norm_rope,
                "kc vc q k v qs ks vs qo qw kw eps rope rows rot il pos pt mb nb cap B T Hq Hkv d", _rope)
append_fp8 = caller(kv.lib.kv_append_norm_rope_fp8,
                    "kc vc q k v qs ks vs qo ksc vsc qw kw eps rope rows rot il pos pt mb nb cap B T Hq Hkv d", _rope)


@pytest.mark.parametrize("call", [prefill_window, chunk_window, decode_window, decode_window_fp8])
def test_window_rejects_bad_arguments(call):
    assert call(window=0) == INVALID
    assert call(window=-5) == INVALID
    assert call(sinks=-1) == INVALID
    assert call(q=None) == INVALID
    assert call(q=P + 8) == INVALID
    assert call(Hkv=3) == INVALID
    assert call(B=0) == INVALID
    assert call(od=2) == INVALID
    assert call(scale=float("inf")) == INVALID
    assert call(d=96) == UNSUPPORTED


@pytest.mark.parametrize("call", [decode_window, decode_window_fp8])
def test_decode_window_rejects_bad_arguments(call):
    assert call(sl=None) == INVALID
    assert call(cap=0) == INVALID
    assert call(msk=101) == INVALID
    assert call(T=4, msk=3) == INVALID
    assert call(ns=-1) == INVALID
    assert call(pt=P, mb=0, nb=3) == INVALID
    assert call(Hq=256, Hkv=1) == UNSUPPORTED
    assert call(pt=P, mb=(1 << 26) + 1, nb=1, msk=(1 << 30) + 1) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE
    assert call(wsb=8) == WORKSPACE
    assert call(ws=P + 4) == WORKSPACE
    assert decode_window_fp8(ks=None) == INVALID
    assert decode_window_fp8(d=64) == UNSUPPORTED


def test_chunk_window_rejects_bad_arguments():
    assert chunk_window(cap=9) == INVALID
    assert chunk_window(pt=P, mb=1, nb=4, Nq=17) == INVALID
    assert chunk_window(cap=(1 << 30) + 1) == UNSUPPORTED
    assert chunk_window(pt=P, mb=(1 << 26) + 1, nb=4) == UNSUPPORTED
    assert prefill_window(N=(1 << 30) + 1, B=1, Hq=1, Hkv=1) == UNSUPPORTED


@pytest.mark.parametrize("call", [shared, shared_fp8])
def test_shared_rejects_bad_arguments(call):
    assert call(q=None) == INVALID
    assert call(pt=None) == INVALID             # a shared prefix needs pages
    assert call(pre=None) == INVALID
    assert call(npre=-1) == INVALID
    assert call(npre=9) == INVALID              # more shared blocks than table columns
    assert call(npre=8) == INVALID              # no room for the new token
    assert call(T=4, msk=51) == INVALID         # 48 shared + 4 new tokens above the bound
    assert call(msk=129) == INVALID
    assert call(Hkv=3) == INVALID
    assert call(causal=2) == INVALID
    assert call(ns=-1) == INVALID
    assert call(scale=0.0) == INVALID
    assert call(d=80) == UNSUPPORTED
    assert call(Hq=256, Hkv=1) == UNSUPPORTED
    assert call(B=1 << 20, T=16) == UNSUPPORTED
    assert call(nb=1 << 28) == UNSUPPORTED
    assert call(k=P + 2) == INVALID
    assert call(ws=None) == WORKSPACE
    assert call(wsb=100) == WORKSPACE
    assert call(npre=0, wsb=100) == WORKSPACE   # nothing shared: plain decode's rules
    assert shared_fp8(vs=None) == INVALID
    assert shared_fp8(d=64) == UNSUPPORTED


@pytest.mark.parametrize("call", [qk, append, append_fp8])
def test_norm_rope_rejects_bad_arguments(call):
    assert call(q=None) == INVALID
    assert call(k=None) == INVALID
    assert call(qo=None) == INVALID
    assert call(B=0) == INVALID
    assert call(T=0) == INVALID
    assert call(rope=None) == INVALID               # rot_dim without a table
    assert call(rot=0) == INVALID                   # a table without rot_dim
    assert call(rows=0) == INVALID
    assert call(rot=144) == INVALID                 # above d
    assert call(rot=24) == UNSUPPORTED              # not a multiple of 16
    assert call(d=96, rot=16) == UNSUPPORTED
    assert call(il=2) == INVALID
    assert call(eps=0.0) == INVALID
    assert call(eps=float("nan")) == INVALID
    assert call(qs=504) == INVALID                  # below Hq * d
    assert call(ks=260) == INVALID                  # not a multiple of 8
    assert call(qs=1 << 62) == INVALID
    assert call(q=(1 << 20) + 2) == INVALID
    assert call(qw=P + 2) == INVALID
    assert call(B=1 << 20, T=1 << 12) == UNSUPPORTED
    assert call(qo=(1 << 20) + 256) == INVALID      # overlaps q without being it
    assert call(qo=1 << 21) == INVALID              # is k
    assert call(qo=1 << 20, qs=1024) == INVALID     # in place needs contiguous rows


@pytest.mark.parametrize("call", [append, append_fp8])
def test_append_norm_rope_rejects_bad_arguments(call):
    assert call(kc=None) == INVALID
    assert call(v=None) == INVALID
    assert call(pos=None) == INVALID
    assert call(cap=0) == INVALID
    assert call(pt=P, mb=0, nb=3) == INVALID
    assert call(kc=P + 4) == INVALID
    assert call(qo=1 << 22) == INVALID              # is v
    assert append_fp8(ksc=None) == INVALID


def test_qk_norm_rope_output_overlap():
    assert qk(ko=None) == INVALID
    assert qk(ko=1 << 23) == INVALID                # both outputs in one place
    assert qk(ko=(1 << 21) + 16) == INVALID
    assert qk(ko=1 << 20) == INVALID                # is q


def test_rope_table_rejects_bad_arguments():
    f = kv.lib.rope_table_fill
    assert f(None, 4, 64, 1e4, None) == INVALID
    assert f(P, 0, 64, 1e4, None) == INVALID
    assert f(P, 4, 63, 1e4, None) == INVALID
    assert f(P, 4, 0, 1e4, None) == INVALID
    assert f(P, 4, 64, 0.0, None) == INVALID
    assert f(P, 4, 64, float("inf"), None) == INVALID


def test_window_workspace_follows_the_window_not_the_length():
    w = kv.attn_decode_window_workspace_bytes
    a = w(16, 1, 32, 8, 128, 32768, 1024, 4)
    assert a == w(16, 1, 32, 8, 128, 1 << 20, 1024, 4) < kv.attn_decode_workspace_bytes(16, 1, 32, 8, 128, 32768)
    # a window past the length needs what plain decode needs
    assert w(16, 1, 32, 8, 128, 32768, 1 << 30, 0) == kv.attn_decode_workspace_bytes(16, 1, 32, 8, 128, 32768)
    assert w(16, 1, 32, 8, 128, 32768, 2 ** 31 - 1, 2 ** 31 - 1) == kv.attn_decode_workspace_bytes(16, 1, 32, 8, 128, 32768)
    for bad in (dict(window=0), dict(sinks=-1), dict(T=0), dict(max_seqlen_k=0), dict(max_seqlen_k=(1 << 30) + 1), dict(d=80)):
        args = dict(B=2, T=1, Hq=8, Hkv=2, d=128, max_seqlen_k=1000, window=64, sinks=0)
        args.update(bad)
        assert w(**args) == 0


def test_shared_workspace():
    w = kv.attn_decode_shared_workspace_bytes
    assert w(4, 1, 8, 2, 128, 1000, 0) == kv.attn_decode_workspace_bytes(4, 1, 8, 2, 128, 1000)
    n = w(64, 1, 32, 8, 128, 32768 + 2048, 2048)
    # the prefix's partial rows and the own parts' both fit
    assert n >= 64 * 32 * (128 + 1) * 4 + kv.attn_decode_workspace_bytes(64, 1, 32, 8, 128, 2048)
    for bad in (dict(prefix_blocks=63), dict(prefix_blocks=-1), dict(B=0), dict(d=72), dict(B=1 << 20, T=16),
                dict(max_seqlen_k=(1 << 30) + 1), dict(num_splits=-1), dict(prefix_blocks=1 << 27)):
        args = dict(B=2, T=1, Hq=8, Hkv=2, d=128, max_seqlen_k=1000, prefix_blocks=10, num_splits=0)
        args.update(bad)
        assert w(**args) == 0


def test_bindings_refuse_host_tensors_and_wrong_shapes():
    bf = dict(dtype=torch.bfloat16)
    q, c, o = torch.zeros(1, 1, 4, 64, **bf), torch.zeros(1, 8, 2, 64, **bf), torch.zeros(1, 1, 4, 64)
    n = torch.ones(1, dtype=torch.int32)
    table = torch.zeros(1, 4, dtype=torch.int32)
    for call in (lambda: kv.attn_prefill_window(q, q, q, o, 4),
                 lambda: kv.attn_decode_window(q, c, c, n, o, 4),
                 lambda: kv.attn_prefill_cache_window(q, c, c, n, o, 4),
                 lambda: kv.attn_decode_window(q, c, c, torch.ones(2, dtype=torch.int32), o, 4),
                 lambda: kv.attn_decode_window(q, torch.zeros(2, 8, 2, 64, **bf), torch.zeros(2, 8, 2, 64, **bf), n, o, 4),
                 lambda: kv.attn_prefill_window(q, q, q, o, 1 << 31),
                 lambda: kv.attn_decode_shared(q, c, c, n, table, table[0, :1], o),
                 lambda: kv.qk_norm_rope(q, q, q, q, None),
                 lambda: kv.kv_append_norm_rope(c, c, q, q, q, q, None, n),
                 lambda: kv.rope_table_fill(torch.zeros(4, 64))):
        with pytest.raises(ValueError):
            call()
