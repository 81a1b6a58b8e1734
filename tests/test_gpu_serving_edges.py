"""GPU tests of what the calls do at the edges of their arguments and of how they are used."""

import numpy as np
import pytest
import torch

import synth
from oracle import serving

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("kv_cache_decode_attn_b200")
from tests.gpu_util import f64, to_dev_i32  # noqa: E402
from tests.test_gpu_window import check, host_cache  # noqa: E402


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    kv.attn_get_device_status(clear=True)
    yield
    assert kv.attn_get_device_status(clear=True) == 0


# ------------------------------------------------------------------------------- streams of their own
@pytest.mark.parametrize("as_handle", [False, True])
def test_calls_on_another_stream_make_their_own_workspace_there(as_handle):
    """Launched on a stream that is held up, without a workspace, while the current stream allocates and
    writes: the outputs are those of a call with a workspace of its own."""
    B, Hq, Hkv, d, blocks = 4, 32, 8, 128, 80
    lens = [16 * blocks + n for n in (5, 300, 64, 900)]
    case = synth.decode_inputs(B, 1, Hq, Hkv, d, 0, 0, seed=3, device="cuda", paged=True, lengths=[L - 1 for L in lens])
    fp8 = synth.decode_inputs(B, 1, Hq, Hkv, d, 0, 0, seed=4, device="cuda", paged=True, lengths=[L - 1 for L in lens],
                              fp8=True)
    t, n, most = to_dev_i32(case.page_table), to_dev_i32(lens), max(lens)
    t8 = to_dev_i32(fp8.page_table)
    t[:, :blocks], t8[:, :blocks] = t[0, :blocks].clone(), t8[0, :blocks].clone()
    p, p8 = t[0, :blocks].contiguous(), t8[0, :blocks].contiguous()
    bf, e4 = (case.q, case.k_pool, case.v_pool), (fp8.q, fp8.k_pool, fp8.v_pool)
    scales = [torch.as_tensor(s, device="cuda") for s in (fp8.k_scale, fp8.v_scale)]
    sizes = (B, 1, Hq, Hkv, d, most)
    plain, window = kv.decode_workspace(*sizes), kv.decode_window_workspace(*sizes, 900, 4)
    shared = kv.decode_shared_workspace(*sizes, blocks)
    calls = [
        (plain, lambda o, **kw: kv.attn_decode(*bf, n, o, page_table=t, max_seqlen_k=most, **kw)),
        (plain, lambda o, **kw: kv.attn_decode_fp8(*e4, *scales, n, o, page_table=t8, max_seqlen_k=most, **kw)),
        (window, lambda o, **kw: kv.attn_decode_window(*bf, n, o, 900, 4, page_table=t, max_seqlen_k=most, **kw)),
        (window, lambda o, **kw: kv.attn_decode_window_fp8(*e4, *scales, n, o, 900, 4, page_table=t8, max_seqlen_k=most,
                                                           **kw)),
        (shared, lambda o, **kw: kv.attn_decode_shared(*bf, n, t, p, o, max_seqlen_k=most, **kw)),
        (shared, lambda o, **kw: kv.attn_decode_shared_fp8(*e4, *scales, n, t8, p8, o, max_seqlen_k=most, **kw)),
    ]
    side = torch.cuda.Stream()
    for ws, call in calls:
        want, got = torch.empty(B, 1, Hq, d, device="cuda"), torch.empty(B, 1, Hq, d, device="cuda")
        call(want, workspace=ws)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        call(got, stream=side.cuda_stream if as_handle else side)
        taken = [torch.full_like(ws, 0xFF) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert all(bool((x == 0xFF).all()) for x in taken)


def test_an_angle_table_made_on_another_stream():
    want = kv.rope_table(3000, 128)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    del_me = torch.full((3000, 128), 7.0, device="cuda")     # written late, its memory free at once
    del del_me
    got = kv.rope_table(3000, 128, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


# ------------------------------------------------------------------------- graphs beside eager calls
@pytest.mark.parametrize("cached", [False, True])
@pytest.mark.parametrize("windowed", [False, True])
def test_a_captured_prefill_runs_beside_eager_ones(windowed, cached):
    """A captured prefill replays on one stream while far more eager ones than a library could keep queues
    for run on another: no launch's items are another's."""
    Hq, Hkv, d = 16, 2, 64

    def case(B, N, seed):
        q, k, v = synth.prefill_inputs(B, Hq, Hkv, N, d, seed=seed, device="cuda")
        n = to_dev_i32([N] * B)
        mask = (70, 4) if windowed else ()

        def go(o):
            if cached:
                fn = kv.attn_prefill_cache_window if windowed else kv.attn_prefill_cache
                fn(q, k, v, n, o, *mask)
            else:
                fn = kv.attn_prefill_window if windowed else kv.attn_prefill
                fn(q, k, v, o, *mask)
        want = torch.full_like(q, float("nan"), dtype=torch.float32)
        go(want)
        return go, want

    long, short = case(4, 2000, 1), case(1, 300, 2)     # 512 items, and 32
    o = torch.empty_like(long[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        long[0](o)
    outs = [torch.empty_like(short[1]) for _ in range(8)]
    side = torch.cuda.Stream()
    for round_ in range(3):
        o.fill_(float("nan"))
        for x in outs:
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                g.replay()
        for i in range(1100):
            short[0](outs[i % 8])
        torch.cuda.synchronize()
        assert torch.equal(o, long[1])
        assert all(torch.equal(x, short[1]) for x in outs)


@pytest.mark.parametrize("windowed", [False, True])
def test_prefills_of_many_items_on_several_streams(windowed):
    """Four launches of more items than SMs at once: each output is whole."""
    q, k, v = synth.prefill_inputs(3, 20, 4, 1200, 128, seed=5, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(4)]
    mask = (300, 4) if windowed else ()
    fn = kv.attn_prefill_window if windowed else kv.attn_prefill
    want = torch.empty_like(q, dtype=torch.float32)
    fn(q, k, v, want, *mask)
    outs = [torch.full_like(want, float("nan")) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            fn(q, k, v, o, *mask, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


# ---------------------------------------------------------------- first tokens whose scores are -inf
def overflowing(q, k, sinks):
    """Value 0 of every head: its product with a first token's overflows fp32 to -inf, with any other key's is 0."""
    q[..., 0] = 1e20
    k[..., 0] = 0.0
    k[:, :sinks, :, 0] = -1e20


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sinks", [1, 4, 16, 50, 64, 100])
@pytest.mark.parametrize("N,Hq,B", [(700, 4, 2), (900, 24, 2)])      # one and two query tiles per item
def test_first_tokens_with_infinite_scores_drop_out(d, sinks, N, Hq, B):
    """A first token at -inf weighs nothing, whichever tile holds it.  Rows that see nothing else have no
    finite score and are left out."""
    window, Hkv = 90, 2
    q, k, v = synth.prefill_inputs(B, Hq, Hkv, N, d, seed=sinks + d, device="cuda")
    overflowing(q, k, sinks)
    o = torch.full((B, N, Hq, d), float("nan"), device="cuda")
    lse = torch.full((B, Hq, N), float("nan"), device="cuda")
    kv.attn_prefill_window(q, k, v, o, window, sinks, lse=lse)
    args = f64(q), f64(k)
    ref = serving.attention_window(*args, f64(v), d ** -0.5, [N] * B, window, sinks)
    weight = serving.attention_window(*args, np.abs(f64(v)), d ** -0.5, [N] * B, window, sinks)[0]
    check(o[:, sinks:], lse[:, :, sinks:], (ref[0][:, sinks:], ref[1][:, :, sinks:]), weight[:, sinks:])


@pytest.mark.parametrize("T", [1, 8, 300])
@pytest.mark.parametrize("paged", [False, True])
def test_cached_first_tokens_with_infinite_scores_drop_out(T, paged):
    """The same over a cache: every decode form, and the chunk's."""
    Hq, Hkv, d, window, sinks, lens = 16, 2, 128, 100, 4, [700 + T, 1500 + T]
    case = synth.decode_inputs(2, T, Hq, Hkv, d, 0, 0, seed=T, device="cuda", paged=paged, lengths=[L - T for L in lens])
    case.q[..., 0] = 1e20
    kc, vc = (case.k_pool, case.v_pool) if paged else (case.k_cache, case.v_cache)
    kc[..., 0] = 0.0
    for b in range(2):
        if paged:
            kc[int(case.page_table[b, 0]), :sinks, :, 0] = -1e20
        else:
            kc[b, :sinks, :, 0] = -1e20
    host, q = host_cache(case, lens), f64(case.q)
    ref = serving.attention_window(q, *host, d ** -0.5, lens, window, sinks)
    weight = serving.attention_window(q, host[0], np.abs(host[1]), d ** -0.5, lens, window, sinks)[0]
    table = to_dev_i32(case.page_table) if paged else None
    for call in (kv.attn_decode_window, kv.attn_prefill_cache_window):
        o = torch.full((2, T, Hq, d), float("nan"), device="cuda")
        lse = torch.full((2, Hq, T), float("nan"), device="cuda")
        call(case.q, kc, vc, to_dev_i32(lens), o, window, sinks, lse=lse, page_table=table)
        check(o, lse, ref, weight)


# ------------------------------------------------------------------------------- NaN scores
@pytest.mark.parametrize("num_splits", [0, 1, 7])
@pytest.mark.parametrize("windowed", [False, True])
@pytest.mark.parametrize("kind,T,Hq,Hkv,d", [("contig", 1, 8, 1, 128), ("paged", 1, 4, 2, 64), ("paged", 2, 16, 2, 128),
                                             ("contig", 8, 8, 2, 128), ("fp8", 1, 8, 1, 128), ("fp8", 2, 12, 1, 128),
                                             ("fp8", 4, 8, 1, 128), ("fp8", 33, 8, 1, 128)])
def test_a_row_with_nan_scores_is_nan_in_both_outputs(kind, T, Hq, Hkv, d, windowed, num_splits):
    """NaN in one query row: that row's output and LSE are NaN, not an LSE of -inf (a row without keys);
    the other rows are exact."""
    lens = [T + 40, T + 1900]
    case = synth.decode_inputs(2, T, Hq, Hkv, d, 0, 0, seed=T, device="cuda", paged=kind != "contig",
                               lengths=[L - T for L in lens], fp8=kind == "fp8")
    host, q = host_cache(case, lens), f64(case.q)
    window, sinks = (300, 5) if windowed else (1 << 30, 0)
    ref = serving.attention_window(q, *host, d ** -0.5, lens, window, sinks)
    weight = serving.attention_window(q, host[0], np.abs(host[1]), d ** -0.5, lens, window, sinks)[0]
    case.q[1, T - 1, Hq - 1, 3] = float("nan")
    table = to_dev_i32(case.page_table) if case.paged else None
    kc, vc = (case.k_pool, case.v_pool) if case.paged else (case.k_cache, case.v_cache)
    scales = [torch.as_tensor(s, device="cuda") for s in (case.k_scale, case.v_scale)] if case.fp8 else []
    o = torch.zeros(2, T, Hq, d, device="cuda")
    lse = torch.zeros(2, Hq, T, device="cuda")
    kw = dict(lse=lse, page_table=table, num_splits=num_splits)
    if windowed:
        fn = kv.attn_decode_window_fp8 if case.fp8 else kv.attn_decode_window
        fn(case.q, kc, vc, *scales, to_dev_i32(lens), o, window, sinks, **kw)
    else:
        fn = kv.attn_decode_fp8 if case.fp8 else kv.attn_decode
        fn(case.q, kc, vc, *scales, to_dev_i32(lens), o, **kw)
    assert torch.isnan(o[1, T - 1, Hq - 1]).all()
    assert torch.isnan(lse[1, Hq - 1, T - 1])
    o[1, T - 1, Hq - 1] = torch.as_tensor(ref[0][1, T - 1, Hq - 1])
    lse[1, Hq - 1, T - 1] = float(ref[1][1, Hq - 1, T - 1])
    check(o, lse, ref, weight)


@pytest.mark.parametrize("splits", [34, 70])
@pytest.mark.parametrize("T,d", [(1, 128), (1, 64), (8, 128)])
def test_nan_in_a_late_chunk_behind_an_empty_one(splits, T, d):
    """More than 32 chunks, the first 32 with scores of -inf and one after them with a NaN key: the merged
    LSE is NaN as the output is."""
    L = 64 * splits
    case = synth.decode_inputs(1, T, 8, 2, d, 0, 0, seed=4, device="cuda", lengths=[L - T])
    case.q[..., 0] = 1e20
    case.k_cache[..., 0] = 0.0
    case.k_cache[0, :32 * 64, :, 0] = -1e20
    case.k_cache[0, 32 * 64 + 5] = float("nan")
    o, lse = torch.zeros(1, T, 8, d, device="cuda"), torch.zeros(1, 8, T, device="cuda")
    kv.attn_decode(case.q, case.k_cache, case.v_cache, to_dev_i32([L]), o, lse, num_splits=splits)
    assert torch.isnan(o).all() and torch.isnan(lse).all()


# ---------------------------------------------------------------------- invalid lengths, every form
@pytest.mark.parametrize("via", ["plain", "wide window", "no prefix"])
@pytest.mark.parametrize("num_splits", [0, 3])
@pytest.mark.parametrize("kind,T,Hq,Hkv", [("contig", 8, 16, 2), ("paged", 8, 16, 2), ("paged", 40, 16, 2), ("fp8", 8, 16, 2),
                                           ("paged", 1, 16, 2), ("fp8", 1, 16, 2)])
def test_invalid_lengths_are_flagged_by_plain_decode_too(kind, T, Hq, Hkv, num_splits, via):
    """What attn_decode states, on the tensor-core kernel as on the others, and through the calls that end in
    it: a window that hides nothing, a shared prefix of no blocks."""
    if via == "no prefix" and kind == "contig":
        pytest.skip("sharing needs pages")
    lens = [T + 50, T + 300]
    case = synth.decode_inputs(2, T, Hq, Hkv, 128, 0, 0, seed=T, device="cuda", paged=kind != "contig",
                               lengths=[L - T for L in lens], fp8=kind == "fp8")
    table = to_dev_i32(case.page_table) if case.paged else None
    kc, vc = (case.k_pool, case.v_pool) if case.paged else (case.k_cache, case.v_cache)
    scales = [torch.as_tensor(s, device="cuda") for s in (case.k_scale, case.v_scale)] if case.fp8 else []
    for wrong in ([T - 1, lens[1]], [lens[0], max(lens) + 1]):
        o, lse = torch.zeros(2, T, Hq, 128, device="cuda"), torch.zeros(2, Hq, T, device="cuda")
        n, kw = to_dev_i32(wrong), dict(lse=lse, max_seqlen_k=max(lens), num_splits=num_splits)
        bad = 0 if wrong[0] < T else 1
        if via == "plain":
            fn = kv.attn_decode_fp8 if case.fp8 else kv.attn_decode
            fn(case.q, kc, vc, *scales, n, o, page_table=table, **kw)
        elif via == "wide window":
            fn = kv.attn_decode_window_fp8 if case.fp8 else kv.attn_decode_window
            fn(case.q, kc, vc, *scales, n, o, 1 << 20, 0, page_table=table, **kw)
        else:
            fn = kv.attn_decode_shared_fp8 if case.fp8 else kv.attn_decode_shared
            fn(case.q, kc, vc, *scales, n, table, table[0, :0], o, **kw)
        assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_SEQLEN
        assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all()
        assert torch.isfinite(o[1 - bad]).all() and torch.isfinite(lse[1 - bad]).all()


# ------------------------------------------------------------------- arguments of the wrong kind
@pytest.mark.parametrize("missing", ["k_scale", "v_scale", "both"])
def test_fp8_calls_need_their_scales(missing):
    """Without scales an FP8 call is refused, over a bf16 cache too: it would run as the bf16 call."""
    q = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    o, n, table = torch.zeros(1, 1, 4, 128, device="cuda"), to_dev_i32([5]), to_dev_i32([[0, 1]])
    new = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
    scale = torch.ones(2, device="cuda")
    ks, vs = None if missing != "v_scale" else scale, None if missing != "k_scale" else scale
    for dtype in (torch.bfloat16, torch.uint8):
        c = torch.zeros(2, 16, 2, 128, dtype=dtype, device="cuda")
        calls = [lambda: kv.attn_decode_window_fp8(q, c, c, ks, vs, n, o, 3, page_table=table),
                 lambda: kv.attn_decode_shared_fp8(q, c, c, ks, vs, to_dev_i32([20]), table, table[0, :1], o),
                 lambda: kv.kv_append_norm_rope_fp8(c, c, q, new, new, torch.zeros_like(q), ks, vs, None, n,
                                                    page_table=table)]
        for call in calls:
            with pytest.raises(ValueError, match="scale"):
                call()
        assert not c.any() and not o.any()


def test_empty_tensors_are_not_none():
    """An empty pos0, angle table or lse is a mistake of shape, not the default."""
    q = torch.ones(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, rope = torch.zeros_like(q), kv.rope_table(8, 64)
    nothing = torch.empty(0, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="pos0"):
        kv.qk_norm_rope(q, q, out, torch.zeros_like(q), rope, pos0=nothing)
    for shape in ((0, 64), (8, 0), (0, 0)):
        with pytest.raises(ValueError, match="rope"):
            kv.qk_norm_rope(q, q, out, torch.zeros_like(q), torch.empty(shape, device="cuda"))
    o = torch.zeros(1, 2, 4, 64, device="cuda")
    for shape in ((0,), (1, 4, 0), (0, 4, 2)):
        with pytest.raises(ValueError, match="lse"):
            kv.attn_prefill_window(q, q, q, o, 3, lse=torch.empty(shape, device="cuda"))
    assert not out.any() and not o.any()


def test_items_of_one_query_tile_follow_one_another():
    """A windowed prefill of fewer one-tile items than SMs, beside a long one that holds the SMs: its CTAs then
    take several items each."""
    long = synth.prefill_inputs(4, 32, 8, 4096, 128, seed=6, device="cuda")
    lo = torch.empty_like(long[0])
    q, k, v = synth.prefill_inputs(1, 14, 2, 1200, 128, seed=7, device="cuda")       # 5 x 14 x 2 <= 148
    want = torch.empty_like(q, dtype=torch.float32)
    kv.attn_prefill_window(q, k, v, want, 300, 4)
    outs = [torch.full_like(want, float("nan")) for _ in range(6)]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for o in outs:
        kv.attn_prefill(*long, lo, stream=a)
        kv.attn_prefill_window(q, k, v, o, 300, 4, stream=b)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_the_first_cuda_call_of_a_host_thread():
    """A thread that has not used the device has no context of it yet; each call works as its first one."""
    import threading

    d = 128
    q, k, v = synth.prefill_inputs(2, 16, 2, 300, d, seed=1, device="cuda")
    case = synth.decode_inputs(3, 4, 16, 2, d, 0, 0, seed=2, device="cuda", paged=True, lengths=[100, 900, 2500])
    fp8 = synth.decode_inputs(3, 1, 16, 2, d, 0, 0, seed=3, device="cuda", paged=True, lengths=[100, 900, 2500], fp8=True)
    n, n8 = to_dev_i32([104, 904, 2504]), to_dev_i32([101, 901, 2501])
    t, t8 = to_dev_i32(case.page_table), to_dev_i32(fp8.page_table)
    t[:, :4] = t[0, :4].clone()
    bf, e4 = (case.q, case.k_pool, case.v_pool), (fp8.q, fp8.k_pool, fp8.v_pool)
    scales = [torch.as_tensor(s, device="cuda") for s in (fp8.k_scale, fp8.v_scale)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    calls = [
        (q, lambda o: kv.attn_prefill(q, k, v, o)),
        (q, lambda o: kv.attn_prefill_window(q, k, v, o, 100, 4)),
        (case.q, lambda o: kv.attn_prefill_cache(*bf, n, o, page_table=t)),
        (case.q, lambda o: kv.attn_decode(*bf, n, o, page_table=t, workspace=ws)),
        (fp8.q, lambda o: kv.attn_decode_fp8(*e4, *scales, n8, o, page_table=t8, workspace=ws)),
        (case.q, lambda o: kv.attn_decode_window(*bf, n, o, 700, 4, page_table=t, workspace=ws)),
        (fp8.q, lambda o: kv.attn_decode_window_fp8(*e4, *scales, n8, o, 700, 4, page_table=t8, workspace=ws)),
        (case.q, lambda o: kv.attn_decode_shared(*bf, n, t, t[0, :4], o, workspace=ws)),
    ]
    for like, call in calls:
        want, got = (torch.full_like(like, float("nan"), dtype=torch.float32) for _ in range(2))
        call(want)
        torch.cuda.synchronize()
        failed = []

        def work():
            try:
                call(got)
            except Exception as e:
                failed.append(e)

        th = threading.Thread(target=work)
        th.start()
        th.join()
        torch.cuda.synchronize()
        assert not failed and torch.equal(got, want)


def test_calls_from_several_host_threads():
    """Four threads, each on a stream of its own, without workspaces: each gets what it gets alone."""
    import threading

    Hq, Hkv, d = 16, 2, 128
    cases, wants = [], []
    for i in range(4):
        q, k, v = synth.prefill_inputs(2, Hq, Hkv, 500 + 40 * i, d, seed=i, device="cuda")
        case = synth.decode_inputs(3, 1 + 3 * i, Hq, Hkv, d, 0, 0, seed=10 + i, device="cuda", paged=True,
                                   lengths=[100, 900, 2500 + i])
        n, t = to_dev_i32([L + 1 + 3 * i for L in (100, 900, 2500 + i)]), to_dev_i32(case.page_table)
        cases.append((q, k, v, case, n, t))

    def run(i, stream, outs):
        q, k, v, case, n, t = cases[i]
        kv.attn_prefill_window(q, k, v, outs[0], 100, 4, stream=stream)
        kv.attn_prefill(q, k, v, outs[1], stream=stream)
        kv.attn_decode_window(case.q, case.k_pool, case.v_pool, n, outs[2], 700, 4, page_table=t, stream=stream)
        kv.attn_decode(case.q, case.k_pool, case.v_pool, n, outs[3], page_table=t, stream=stream)

    def outputs(i):
        return [torch.full_like(x, float("nan"), dtype=torch.float32) for x in (cases[i][0],) * 2 + (cases[i][3].q,) * 2]

    for i in range(4):
        wants.append(outputs(i))
        run(i, None, wants[i])
    torch.cuda.synchronize()
    got, failed = [[outputs(i) for _ in range(10)] for i in range(4)], []
    torch.cuda.synchronize()

    def work(i):
        try:
            s = torch.cuda.Stream()
            for outs in got[i]:
                run(i, s, outs)
            s.synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed
    for i in range(4):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, wants[i]))
