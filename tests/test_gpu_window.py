"""GPU parity of the sliding-window calls (window plus first tokens that stay visible) against
the fp64 oracle, through the public wrappers.

Tolerance of o, per element: the probabilities enter the second product rounded to bf16 (half
a step: 2^-8 of the value; 2^-11 in f16 for FP8 caches) while their sum is kept in fp32, so
|error| <= 2^-8 * sum_j p_j |v_j| / sum_j p_j, the attention over |v|.  A score's error is below
2^-14 absolute (|scale * q k| sums below 32, fp32 sums of d / 16 matrix steps, each off by less
than 2^-21 of them) and the base-2 exponential's is smaller; both weigh on |v| the same way, so
2^-12 is added for numerator and denominator together.  bf16 outputs add their half step.  The
LSE sees only the score and exponential errors and fp32 logarithms: 2^-12 + 2^-20 |lse|."""

import math

import numpy as np
import pytest
import torch

import synth
from oracle import fp8 as ofp8
from oracle import gather_paged, serving

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("kv_cache_decode_attn_b200")
from tests.gpu_util import f64, to_dev_i32  # noqa: E402


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    kv.attn_get_device_status(clear=True)
    yield
    assert kv.attn_get_device_status(clear=True) == 0


def check(o, lse, ref, weight, what=""):
    """ref = (o, lse); weight = the attention over |v|."""
    g = f64(o)
    tol = (2.0 ** -8 + 2.0 ** -12) * weight
    if o.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref[0]) + tol)
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    over = np.abs(g - ref[0]) - tol
    assert (over <= 0).all(), f"{what}: o off by {np.abs(g - ref[0]).max()} at {np.argwhere(over > 0)[:4].tolist()}"
    gl = f64(lse)
    assert np.isfinite(gl).all(), f"{what}: non-finite lse"
    err = np.abs(gl - ref[1])
    assert (err <= 2.0 ** -12 + 2.0 ** -20 * np.abs(ref[1])).all(), f"{what}: lse off by {err.max()}"


def host_cache(case, lens):
    """The K and V the case's caches stand for, [B, max(lens), Hkv, d] float64."""
    out = []
    for cache, pool, scale in ((case.k_cache, case.k_pool, case.k_scale), (case.v_cache, case.v_pool, case.v_scale)):
        x = (pool if case.paged else cache).cpu()
        x = ofp8.e4m3_decode(x.numpy()) * np.asarray(scale, np.float64)[:, None] if case.fp8 else f64(x)
        out.append(gather_paged(x, case.page_table, lens) if case.paged else x)
    return out


def poison(case, lens, T, window, sinks):
    """NaN in every cached key and value no query sees, -1 in the page table's entries of blocks
    wholly between the first tokens and the first query's window."""
    bad = 0x7F if case.fp8 else float("nan")
    caches = (case.k_pool, case.v_pool) if case.paged else (case.k_cache, case.v_cache)
    for b, L in enumerate(lens):
        seen = np.zeros((-(-int(caches[0].shape[1] if not case.paged else case.page_table.shape[1] * 16) // 16)) * 16, bool)
        m = serving.window_mask(T, L, window, sinks).any(axis=0)
        seen[:L] = m
        if case.paged:
            table = case.page_table
            for blk in range(table.shape[1]):
                if table[b, blk] < 0:
                    continue
                keep = seen[blk * 16:blk * 16 + 16]
                rows = torch.as_tensor(np.flatnonzero(~keep), device=caches[0].device)
                for c in caches:
                    c[int(table[b, blk])].index_fill_(0, rows, bad)
            w0 = max(0, L - T - window + 1) // 16
            table[b, -(-sinks // 16):max(w0, -(-sinks // 16))] = -1
        else:
            cap = caches[0].shape[1]
            rows = torch.as_tensor(np.flatnonzero(~seen[:cap]), device=caches[0].device)
            for c in caches:
                c[b].index_fill_(0, rows, bad)


def run(case, lens, T, Hq, Hkv, d, window, sinks, o_dtype=torch.float32, fn="decode", **kw):
    B, dev = len(lens), case.q.device
    table = None if case.page_table is None else to_dev_i32(case.page_table)
    kc, vc = (case.k_pool, case.v_pool) if case.paged else (case.k_cache, case.v_cache)
    o = torch.full((B, T, Hq, d), float("nan"), dtype=o_dtype, device=dev)
    lse = torch.full((B, Hq, T), float("nan"), device=dev)
    if fn == "chunk":
        kv.attn_prefill_cache_window(case.q, kc, vc, to_dev_i32(lens), o, window, sinks, lse=lse, page_table=table, **kw)
    elif case.fp8:
        ks, vs = (torch.as_tensor(s, device=dev) for s in (case.k_scale, case.v_scale))
        kv.attn_decode_window_fp8(case.q, kc, vc, ks, vs, to_dev_i32(lens), o, window, sinks, lse=lse, page_table=table,
                                  **kw)
    else:
        kv.attn_decode_window(case.q, kc, vc, to_dev_i32(lens), o, window, sinks, lse=lse, page_table=table, **kw)
    return o, lse


def parity(T, Hq, Hkv, d, window, sinks, lens, kind, seed, fn="decode", **kw):
    lens = [max(L, T) for L in lens]
    case = synth.decode_inputs(len(lens), T, Hq, Hkv, d, 0, 0, seed=seed, device="cuda", paged=kind != "contig",
                               lengths=[L - T for L in lens], capacity=max(lens) + 7, spare_blocks=2,
                               fp8=kind.startswith("fp8"))
    host = host_cache(case, lens)     # before the poison; the oracle reads seen keys only
    poison(case, lens, T, window, sinks)
    o, lse = run(case, lens, T, Hq, Hkv, d, window, sinks, fn=fn, **kw)
    scale = kw.get("scale", 1.0 / math.sqrt(d))
    q = f64(case.q)
    ref = serving.attention_window(q, *host, scale, lens, window, sinks)
    weight = serving.attention_window(q, host[0], np.abs(host[1]), scale, lens, window, sinks)[0]
    check(o, lse, ref, weight, f"{kind} T={T} window={window} sinks={sinks}")


LENS = [1, 2, 15, 16, 17, 64, 65, 130, 300, 1000, 2111]
MASKS = [(1, 0), (1, 1), (5, 4), (16, 16), (17, 0), (64, 33), (100, 4), (500, 1), (1000, 2000), (4000, 3)]


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("kind,T,Hq,Hkv,d", [("contig", 1, 8, 2, 128), ("paged", 1, 16, 2, 64), ("contig", 3, 4, 1, 64),
                                             ("paged", 2, 16, 2, 128),
                                             ("contig", 8, 8, 2, 128), ("paged", 8, 6, 2, 64), ("paged", 20, 16, 2, 128),
                                             ("fp8", 1, 8, 1, 128), ("fp8", 3, 10, 2, 128), ("fp8", 4, 8, 1, 128),
                                             ("fp8", 5, 8, 1, 128), ("fp8", 33, 8, 1, 128)])
def test_decode_window_parity(kind, T, Hq, Hkv, d, window, sinks):
    """Every decode kernel (warp-level bf16, FP8 of 8, 16 and 32 rows, tensor-core bf16 and FP8 with
    one and several row tiles), lengths from one key on."""
    parity(T, Hq, Hkv, d, window, sinks, LENS, kind, seed=40 + T + Hq + d)


@pytest.mark.parametrize("num_splits", [1, 3, 16])
@pytest.mark.parametrize("kind,T", [("contig", 1), ("paged", 6), ("fp8", 1), ("fp8", 6)])
def test_decode_window_splits_and_bf16_out(kind, T, num_splits):
    parity(T, 8, 1, 128, 700, 20, [40, 699, 740, 3000], kind, seed=60 + T, num_splits=num_splits,
           o_dtype=torch.bfloat16, scale=0.11)


@pytest.mark.parametrize("kind", ["contig", "paged"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (60, 4), (300, 17), (1 << 30, 0), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_decode_window_of_many_tokens_runs_the_prefill_form(kind, window, sinks):
    """256 and more new tokens, and windows and sinks up to the largest argument."""
    parity(260, 4, 2, 64, window, sinks, [260, 300, 900], kind, seed=80)
    parity(2, 4, 2, 64, window, sinks, [2, 300, 900], kind, seed=81)


def test_decode_window_many_sequences_balanced_and_not():
    """The tensor-core form with 128 sequences (balanced split) and 129 (fixed chunks)."""
    for B in (128, 129):
        lens = [8 + 13 * (i % 40) for i in range(B)]
        parity(8, 8, 2, 128, 100, 4, lens, "paged", seed=90)


@pytest.mark.parametrize("kind,T,Hq,Hkv,d", [("paged", 1, 150, 150, 64), ("contig", 1, 128, 1, 128), ("paged", 3, 128, 1, 64),
                                             ("fp8", 1, 40, 1, 128), ("fp8", 2, 128, 1, 128), ("contig", 1, 1, 1, 64)])
@pytest.mark.parametrize("window,sinks", [(90, 3), (2500, 40)])
def test_decode_window_head_layouts(kind, T, Hq, Hkv, d, window, sinks):
    """More KV heads than SMs, up to 128 query heads of one KV head (several row tiles), a single head."""
    parity(T, Hq, Hkv, d, window, sinks, [3, 70, 2700, 4001], kind, seed=95)


@pytest.mark.parametrize("kind,T,Hq", [("paged", 1, 4), ("contig", 3, 8), ("fp8", 1, 4), ("fp8", 5, 8)])
def test_decode_window_many_sequences_even_shares_and_not(kind, T, Hq):
    """The warp-level forms with 128 sequences (even shares of the tiles) and 129 (chunks), a window too
    long for one CTA per sequence; the latter's short ones have a share of a tile or two."""
    for B in (128, 129):
        lens = [T + 37 * (i % 50) ** 2 % 3000 for i in range(B)]
        parity(T, Hq, 2, 128, 2900, 7, lens, kind, seed=91)


@pytest.mark.parametrize("kind", ["contig", "paged", "fp8"])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (8, 16, 2)])
def test_wide_window_is_plain_decode(kind, T, Hq, Hkv):
    """A window that covers every key gives attn_decode's bits: same chunks, same order."""
    d, lens = 128, [T, 100, 777, 2500]
    case = synth.decode_inputs(4, T, Hq, Hkv, d, 0, 0, seed=33, device="cuda", paged=kind != "contig",
                               lengths=[L - T for L in lens], fp8=kind == "fp8")
    o, lse = run(case, lens, T, Hq, Hkv, d, 1 << 20, 0)
    table = None if case.page_table is None else to_dev_i32(case.page_table)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    if kind == "fp8":
        ks, vs = (torch.as_tensor(s, device="cuda") for s in (case.k_scale, case.v_scale))
        kv.attn_decode_fp8(case.q, case.k_pool, case.v_pool, ks, vs, to_dev_i32(lens), o2, lse2, page_table=table)
    else:
        kc, vc = (case.k_pool, case.v_pool) if case.paged else (case.k_cache, case.v_cache)
        kv.attn_decode(case.q, kc, vc, to_dev_i32(lens), o2, lse2, page_table=table)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 3, 64)])
def test_prefill_window_parity(N, Hq, Hkv, d):
    q, k, v = synth.prefill_inputs(2, Hq, Hkv, N, d, seed=N + d, device="cuda")
    for window, sinks in ((1, 0), (1, 3), (50, 0), (128, 1), (129, 128), (300, 40), (10, 5000), (5000, 0)):
        for dtype in (torch.float32, torch.bfloat16):
            o = torch.full((2, N, Hq, d), float("nan"), dtype=dtype, device="cuda")
            lse = torch.full((2, Hq, N), float("nan"), device="cuda")
            kv.attn_prefill_window(q, k, v, o, window, sinks, lse=lse)
            scale = d ** -0.5
            lens = [N, N]
            ref = serving.attention_window(f64(q), f64(k), f64(v), scale, lens, window, sinks)
            weight = serving.attention_window(f64(q), f64(k), np.abs(f64(v)), scale, lens, window, sinks)[0]
            check(o, lse, ref, weight, f"N={N} window={window} sinks={sinks} {dtype}")


@pytest.mark.parametrize("kind", ["contig", "paged"])
@pytest.mark.parametrize("Nq,Hq,Hkv,d", [(1, 8, 2, 128), (100, 4, 2, 64), (257, 4, 1, 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (200, 0), (600, 130), (4000, 0)])
def test_prefill_cache_window_parity(kind, Nq, Hq, Hkv, d, window, sinks):
    parity(Nq, Hq, Hkv, d, window, sinks, [Nq, Nq + 1, 400, 1500], kind, seed=70 + Nq, fn="chunk")


def test_window_calls_replay_in_a_graph_with_new_lengths():
    """Captured once, replayed with other lengths and contents: the replay reads them anew."""
    T, Hq, Hkv, d, window, sinks = 1, 8, 2, 128, 64, 4
    lens = [10, 200, 900]
    case = synth.decode_inputs(3, T, Hq, Hkv, d, 0, 0, seed=5, device="cuda", paged=True, lengths=[L - T for L in lens])
    table, seqlens = to_dev_i32(case.page_table), to_dev_i32(lens)
    o, lse = torch.empty(3, T, Hq, d, device="cuda"), torch.empty(3, Hq, T, device="cuda")
    ws = kv.decode_window_workspace(3, T, Hq, Hkv, d, max(lens), window, sinks)

    def call():
        kv.attn_decode_window(case.q, case.k_pool, case.v_pool, seqlens, o, window, sinks, lse=lse, page_table=table,
                              max_seqlen_k=max(lens), workspace=ws)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    host = host_cache(case, lens)
    for now in (lens, [1, 17, 899], [3, 64, 500]):
        seqlens.copy_(to_dev_i32(now))
        case.q.normal_()
        o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        q = f64(case.q)
        ref = serving.attention_window(q, *host, d ** -0.5, now, window, sinks)
        weight = serving.attention_window(q, host[0], np.abs(host[1]), d ** -0.5, now, window, sinks)[0]
        check(o, lse, ref, weight)


def test_window_calls_on_two_streams():
    """Two calls in flight on streams of their own, each with its own workspace."""
    T, Hq, Hkv, d = 2, 16, 2, 128
    lens = [500, 3000, 2000]
    case = synth.decode_inputs(3, T, Hq, Hkv, d, 0, 0, seed=6, device="cuda", lengths=[L - T for L in lens])
    host, q = host_cache(case, lens), f64(case.q)
    seqlens = to_dev_i32(lens)
    outs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    masks = [(100, 4), (2500, 0)]
    bufs = [(torch.empty(3, T, Hq, d, device="cuda"), torch.empty(3, Hq, T, device="cuda"),
             kv.decode_window_workspace(3, T, Hq, Hkv, d, max(lens), *m)) for m in masks]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, m, (o, lse, ws) in zip(streams, masks, bufs):
            kv.attn_decode_window(case.q, case.k_cache, case.v_cache, seqlens, o, *m, lse=lse, max_seqlen_k=max(lens),
                                  workspace=ws, stream=s)
    torch.cuda.synchronize()
    for m, (o, lse, _) in zip(masks, bufs):
        ref = serving.attention_window(q, *host, d ** -0.5, lens, *m)
        weight = serving.attention_window(q, host[0], np.abs(host[1]), d ** -0.5, lens, *m)[0]
        check(o, lse, ref, weight)


@pytest.mark.parametrize("T,kind", [(1, "contig"), (1, "fp8"), (8, "paged"), (300, "paged")])
def test_window_length_errors(T, kind):
    """A length below T or above max_seqlen_k: NaN rows and ATTN_DEV_SEQLEN, the others exact."""
    Hq, Hkv, d, window, sinks = 8, 2, 128, 90, 4
    lens = [max(T, 50), T + 700, T + 800]
    case = synth.decode_inputs(3, T, Hq, Hkv, d, 0, 0, seed=8, device="cuda", paged=kind != "contig",
                               lengths=[L - T for L in lens], fp8=kind == "fp8")
    host = host_cache(case, lens)
    o, lse = run(case, [T - 1, lens[1], lens[2]], T, Hq, Hkv, d, window, sinks, max_seqlen_k=lens[2] - 1)
    assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_SEQLEN
    assert torch.isnan(o[0]).all() and torch.isnan(o[2]).all()
    assert torch.isnan(lse[0]).all() and torch.isnan(lse[2]).all()
    q = f64(case.q)[1:2]
    ref = serving.attention_window(q, host[0][1:], host[1][1:], d ** -0.5, lens[1:2], window, sinks)
    weight = serving.attention_window(q, host[0][1:], np.abs(host[1][1:]), d ** -0.5, lens[1:2], window, sinks)[0]
    check(o[1:2], lse[1:2], ref, weight)


@pytest.mark.parametrize("T", [1, 8, 300])
def test_window_bad_page_entry_is_flagged(T):
    lens = [T + 400]
    case = synth.decode_inputs(1, T, 8, 2, 128, 0, 0, seed=9, device="cuda", paged=True, lengths=[400])
    case.page_table[0, lens[0] // 16 - 2] = 1 << 20
    run(case, lens, T, 8, 2, 128, 64, 4)
    assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_PAGE_ID


def test_other_current_device_is_refused(monkeypatch):
    """Tensors of another device than the current one would reach its stream and status word."""
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="device"):
        kv.attn_prefill_window(q, q, q, torch.zeros(1, 4, 2, 64, device="cuda"), 3)
