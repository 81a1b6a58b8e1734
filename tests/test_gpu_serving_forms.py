"""GPU parity of the forms of the windowed and shared-prefix calls that long inputs take: windowed
prefill in items of two query tiles (many items per SM, tile B with all, some and no rows), a shared
prefix read once for the batch (three launches) where test_gpu_shared.py's short prefixes are read by
each sequence, and FP8 caches under the bound that f16 probabilities allow.  Each test states or asks
which form it takes.  Against the definitions in 64 bits, evaluated by elementary torch operations.

Tolerances of o as derived in test_gpu_window.py, with the cache's own rounding of the probabilities:
2^-8 (bf16) or 2^-11 (f16, FP8 caches) of the attention over |v|, 2^-12 for scores and exponentials,
a half step more for bf16 outputs.  f16 probabilities below 2^-14 are subnormal and off by up to
2^-25 each; a row's probabilities are taken relative to a reference that no score exceeds by more
than 2^8 and that is one of its scores, so their sum is at least exp(lse - max score), and the
subnormals weigh 2^-25 sum_j |v_j| / exp(lse - max score) on the row.  q in f16 is exact from 2^-14
on; below, off by up to 2^-25, at most 2^-19 in a score here: part of the 2^-12."""

import numpy as np
import pytest
import torch

import synth
from oracle import fp8 as ofp8
from oracle import serving

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("kv_cache_decode_attn_b200")
from tests.gpu_util import f64, to_dev_i32  # noqa: E402

EVERY = 1 << 30   # a window that hides nothing


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    kv.attn_get_device_status(clear=True)
    yield
    assert kv.attn_get_device_status(clear=True) == 0


def seen_keys(T, L, window, sinks, causal=True):
    p = torch.arange(L - T, L, device="cuda")[:, None]
    j = torch.arange(L, device="cuda")[None, :]
    if not causal:
        return torch.ones(T, L, dtype=torch.bool, device="cuda")
    return (j <= p) & ((j > p - window) | (j < sinks))


def attention64(q, k, v, lens, window=EVERY, sinks=0, scale=None, causal=True):
    """q [B, T, Hq, d], k and v one [L_b, Hkv, d] per sequence, float64 on the GPU: o, lse, the attention
    over |v|, and sum_j |v_j| / exp(lse - max score)."""
    B, T, Hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    o, weight, small = (torch.empty(B, T, Hq, d, dtype=torch.float64, device="cuda") for _ in range(3))
    lse = torch.empty(B, Hq, T, dtype=torch.float64, device="cuda")
    for b, L in enumerate(lens):
        seen = seen_keys(T, L, window, sinks, causal)
        used = seen.any(dim=0).nonzero()[:, 0]      # what no query sees may hold anything
        kb, vb, m = k[b][used], v[b][used], seen[:, used]
        G = Hq // kb.shape[1]
        for h in range(Hq):
            s = q[b, :, h].double() @ kb[:, h // G].double().T * scale
            s = s.masked_fill(~m, -torch.inf)
            top = s.max(dim=1, keepdim=True).values
            e = torch.exp(s - top)
            z = e.sum(dim=1, keepdim=True)
            vv = vb[:, h // G].double()
            o[b, :, h] = e @ vv / z
            weight[b, :, h] = e @ vv.abs() / z
            small[b, :, h] = m.double() @ vv.abs() / z
            lse[b, h] = (top + z.log())[:, 0]
    return o, lse, weight, small


def check(o, lse, ref, fp8=False, rows=slice(None), what=""):
    ro, rl, weight, small = (x[rows] for x in ref)
    tol = (2.0 ** -11 + 2.0 ** -12) * weight + 2.0 ** -25 * small if fp8 else (2.0 ** -8 + 2.0 ** -12) * weight
    if o.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ro.abs() + tol)
    g, gl = o[rows].double(), lse[rows].double()
    assert torch.isfinite(g).all() and torch.isfinite(gl).all(), f"{what}: non-finite"
    over = (g - ro).abs() - tol
    assert (over <= 0).all(), f"{what}: o off by {(g - ro).abs().max()} at {(over > 0).nonzero()[:4].tolist()}"
    err = (gl - rl).abs()
    assert (err <= 2.0 ** -12 + 2.0 ** -20 * rl.abs()).all(), f"{what}: lse off by {err.max()}"


def launches(call):
    """Kernels that a call launches."""
    from cuda.bindings import runtime

    call()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    err, _, n = runtime.cudaGraphGetNodes(runtime.cudaGraph_t(g.raw_cuda_graph()))
    assert int(err) == 0
    return n


# ------------------------------------------------------------ windowed prefill, two query tiles an item
def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def two_tile_items(N, Hq, B):
    """The rule of run_prefill (csrc/prefill.cu): items of two query tiles where as many of one tile
    would be more than the SMs.  Returns their number."""
    n = -(-N // 256) * Hq * B
    assert 2 * n > sms(), "these sizes take the form of one query tile an item"
    return n


WINDOWS = [(1, 0), (1, 3), (100, 0), (130, 4), (127, 64), (300, 65), (129, 128), (256, 300), (600, 130), (2000, 0),
           (40, 5000)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("B,N,Hq,Hkv,d", [
    (2, 1100, 16, 4, 128),    # 160 items on 148 SMs; the last item's tile B has no rows
    (3, 640, 32, 8, 64),      # 288 items, the same with 128 rows in its tile A
    (2, 900, 24, 24, 64),     # 192 items, four rows in the last tile B
    (5, 257, 16, 1, 128),     # 160 items, half of them one row
    (1, 1500, 13, 13, 128),   # fewer items than SMs
])
def test_prefill_window_in_items_of_two_tiles(B, N, Hq, Hkv, d, window, sinks):
    two_tile_items(N, Hq, B)
    q, k, v = synth.prefill_inputs(B, Hq, Hkv, N, d, seed=N + d, device="cuda")
    ref = attention64(q, k, v, [N] * B, window, sinks)
    for dtype in (torch.float32, torch.bfloat16):
        o = torch.full((B, N, Hq, d), float("nan"), dtype=dtype, device="cuda")
        lse = torch.full((B, Hq, N), float("nan"), device="cuda")
        kv.attn_prefill_window(q, k, v, o, window, sinks, lse=lse)
        check(o, lse, ref, what=f"window={window} sinks={sinks} {dtype}")


def hide(case, lens, T, window, sinks):
    """The case's K and V as [L, Hkv, d] per sequence; then NaN in every cached row no query sees, and -1 in
    the page table's entries between the first tokens' blocks and the first query's window."""
    ks, vs = [], []
    for b, L in enumerate(lens):
        at = torch.arange(L, device="cuda")
        if case.paged:
            row = to_dev_i32(case.page_table[b]).long()
            pick = lambda c: c[row[at // 16], at % 16].clone()
        else:
            pick = lambda c: c[b, :L].clone()
        kc, vc = (case.k_pool, case.v_pool) if case.paged else (case.k_cache, case.v_cache)
        ks.append(pick(kc))
        vs.append(pick(vc))
        dead = torch.ones(-(-L // 16) * 16 if case.paged else kc.shape[1], dtype=torch.bool, device="cuda")
        dead[:L] = ~seen_keys(T, L, window, sinks).any(dim=0)
        rows = dead.nonzero()[:, 0]
        for c in (kc, vc):
            if case.paged:
                c[row[rows // 16], rows % 16] = float("nan")
            else:
                c[b, rows] = float("nan")
        if case.paged:
            first = -(-sinks // 16)
            case.page_table[b, first:max(max(0, L - T - window + 1) // 16, first)] = -1
    return ks, vs


@pytest.mark.parametrize("kind", ["contig", "paged"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (128, 64), (200, 0), (300, 65), (600, 130), (90, 300), (4000, 3)])
@pytest.mark.parametrize("T,Hq,Hkv,d", [(300, 32, 8, 128), (520, 16, 2, 64), (257, 12, 12, 128)])
def test_chunk_window_in_items_of_two_tiles(kind, T, Hq, Hkv, d, window, sinks):
    lens = [T, T + 1, T + 600, 3 * T + 37]
    two_tile_items(T, Hq, 4)
    case = synth.decode_inputs(4, T, Hq, Hkv, d, 0, 0, seed=T, device="cuda", paged=kind == "paged",
                               lengths=[L - T for L in lens], capacity=max(lens) + 7, spare_blocks=2)
    ks, vs = hide(case, lens, T, window, sinks)
    ref = attention64(case.q, ks, vs, lens, window, sinks)
    table = to_dev_i32(case.page_table) if case.paged else None
    kc, vc = (case.k_pool, case.v_pool) if case.paged else (case.k_cache, case.v_cache)
    for call in (kv.attn_prefill_cache_window, kv.attn_decode_window):   # 256 and more tokens: the same kernel
        o = torch.full((4, T, Hq, d), float("nan"), device="cuda")
        lse = torch.full((4, Hq, T), float("nan"), device="cuda")
        call(case.q, kc, vc, to_dev_i32(lens), o, window, sinks, lse=lse, page_table=table)
        check(o, lse, ref, what=f"{call.__name__} window={window} sinks={sinks}")


# --------------------------------------------------------------- shared prefix, read once for the batch
def shared_case(B, T, Hq, Hkv, d, prefix_blocks, own, seed, fp8=False):
    """Pools, scales (or none), the true table and the lengths; K and V as [L, Hkv, d] per sequence."""
    lens = [16 * prefix_blocks + n for n in own]
    blocks = [-(-n // 16) for n in own]
    total = prefix_blocks + sum(blocks) + 2
    perm = synth.block_permutation(total, seed)
    table = np.full((B, prefix_blocks + max(blocks)), -1, dtype=np.int32)
    table[:, :prefix_blocks] = perm[:prefix_blocks]
    at = prefix_blocks
    for b, n in enumerate(blocks):
        table[b, prefix_blocks:prefix_blocks + n] = perm[at:at + n]
        at += n
    q = synth.normal_bf16((B, T, Hq, d), seed + 1, "cuda")
    if fp8:
        scales = [torch.as_tensor(synth.kv_scales(Hkv, seed + i), device="cuda") for i in (2, 3)]
        pools = [synth.normal_e4m3_codes((total, 16, Hkv, d), f64(s), seed + i, "cuda") for i, s in zip((4, 5), scales)]
    else:
        scales = []
        pools = [synth.normal_bf16((total, 16, Hkv, d), seed + i, "cuda") for i in (4, 5)]
    return q, pools, scales, table, lens


def gathered(pools, scales, table, lens):
    """K and V per sequence, float64."""
    out = []
    for i, pool in enumerate(pools):
        x = torch.as_tensor(ofp8.e4m3_decode(pool.cpu().numpy()), device="cuda") * scales[i].double()[:, None] if scales \
            else pool.double()
        out.append([x[to_dev_i32(table[b]).long()[:-(-L // 16)]].flatten(0, 1)[:L] for b, L in enumerate(lens)])
    return out


def shared(q, pools, scales, n, t, p, o, lse, **kw):
    fn = kv.attn_decode_shared_fp8 if scales else kv.attn_decode_shared
    fn(q, *pools, *scales, n, t, p, o, lse=lse, **kw)


def outputs(B, T, Hq, d):
    return (torch.full((B, T, Hq, d), float("nan"), device="cuda"), torch.full((B, Hq, T), float("nan"), device="cuda"))


FORMS = [pytest.param(12, 1, id="read by each"), pytest.param(1300, 3, id="read once")]


@pytest.mark.parametrize("blocks,kernels", FORMS)
def test_shared_prefix_with_a_bad_scale(blocks, kernels):
    """One head's scale is no number (K's, then V's): its rows are NaN, the other head's exact."""
    q, pools, scales, table, lens = shared_case(6, 1, 8, 2, 128, blocks, [3, 40, 17, 900, 64, 1], seed=11, fp8=True)
    ref = attention64(q, *gathered(pools, scales, table, lens), lens)
    n, t, p = to_dev_i32(lens), to_dev_i32(table), to_dev_i32(table[0, :blocks])
    for which in (0, 1):
        for value in (float("nan"), 0.0, -1.0, float("inf")):
            wrong = [s.clone() for s in scales]
            wrong[which][0] = value
            o, lse = outputs(6, 1, 8, 128)
            shared(q, pools, wrong, n, t, p, o, lse)
            assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_SCALE
            assert torch.isnan(o[:, :, :4]).all() and torch.isnan(lse[:, :4]).all()
            good = tuple(x[:, 4:] if x.dim() == 3 else x[:, :, 4:] for x in ref)
            check(o[:, :, 4:], lse[:, 4:], good, fp8=True)
    assert launches(lambda: shared(q, pools, scales, n, t, p, o, lse)) >= kernels


@pytest.mark.parametrize("blocks,kernels", FORMS)
@pytest.mark.parametrize("fp8", [False, True])
def test_shared_prefix_past_the_lengths(blocks, kernels, fp8):
    """NaN behind every length, in the last block and in blocks of the table past it."""
    own = [5, 16, 37, 470]
    q, pools, scales, table, lens = shared_case(4, 1, 8, 2, 128, blocks, own, seed=9, fp8=fp8)
    kh, vh = gathered(pools, scales, table, lens)
    for b, L in enumerate(lens):
        if L % 16:
            for c in pools:
                c[int(table[b, L // 16]), L % 16:] = 0x7F if fp8 else float("nan")
    hidden = table.copy()
    hidden[:, :blocks] = -1
    for b, L in enumerate(lens):
        hidden[b, -(-L // 16):] = -5
    n, t, p = to_dev_i32(lens), to_dev_i32(hidden), to_dev_i32(table[0, :blocks])
    o, lse = outputs(4, 1, 8, 128)

    def go():
        shared(q, pools, scales, n, t, p, o, lse)

    assert launches(go) >= kernels
    o.fill_(float("nan"))
    go()
    check(o, lse, attention64(q, kh, vh, lens), fp8)


@pytest.mark.parametrize("blocks,kernels", FORMS)
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (2, 16, 2), (8, 8, 2)])
def test_shared_prefix_on_two_streams_in_both_forms(blocks, kernels, T, Hq, Hkv):
    """Two calls in flight, each on a stream and with a workspace of its own."""
    d, own = 128, [T + x for x in (4, 299, 63, 19, 899, 0)]
    sides = []
    for seed in (31, 32):
        q, pools, scales, table, lens = shared_case(6, T, Hq, Hkv, d, blocks, own, seed)
        n, t, p = to_dev_i32(lens), to_dev_i32(table), to_dev_i32(table[0, :blocks])
        ws = kv.decode_shared_workspace(6, T, Hq, Hkv, d, max(lens), blocks)
        sides.append((q, pools, scales, n, t, p, *outputs(6, T, Hq, d), dict(max_seqlen_k=max(lens), workspace=ws),
                      attention64(q, *gathered(pools, scales, table, lens), lens)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for (*args, kw, _), s in zip(sides, streams):
            shared(*args, stream=s, **kw)
    torch.cuda.synchronize()
    for *args, kw, ref in sides:
        check(args[6], args[7], ref)
    *args, kw, _ = sides[0]
    assert launches(lambda: shared(*args, **kw)) >= kernels


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,fp8", [(1, 8, 2, False), (1, 8, 2, True), (4, 16, 2, False), (8, 16, 2, True)])
@pytest.mark.parametrize("blocks,kernels", FORMS)
def test_shared_prefix_directly_behind_its_writer(blocks, kernels, T, Hq, Hkv, fp8, captured):
    """kv_append_norm_rope writes the queries, K and V that the shared call, launched right behind it in the
    stream or the same graph, reads: in the form of three launches the own keys' launch waits for the
    writer only through the prefix's.  Several steps, the lengths growing on the device in between."""
    B, d, steps = 5, 128, 4
    own = [T, 16, 31, 100, 900]
    q, pools, scales, table, _ = shared_case(B, T, Hq, Hkv, d, blocks, [n + T * steps for n in own], 21, fp8)
    lens = [16 * blocks + n - T for n in own]
    qkv = torch.empty(B, T, (Hq + 2 * Hkv) * d, dtype=torch.bfloat16, device="cuda")
    qn, kn, vn = [x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], dim=-1)]
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    most = max(lens) + T * steps
    rope, at, n = kv.rope_table(most, d), to_dev_i32(lens), to_dev_i32([L + T for L in lens])
    t, p = to_dev_i32(table), to_dev_i32(table[0, :blocks])
    q_out = torch.empty(B, T, Hq, d, dtype=torch.bfloat16, device="cuda")
    o, lse = outputs(B, T, Hq, d)
    ws = kv.decode_shared_workspace(B, T, Hq, Hkv, d, most, blocks)

    def append():
        fn = kv.kv_append_norm_rope_fp8 if fp8 else kv.kv_append_norm_rope
        fn(*pools, qn, kn, vn, q_out, *scales, rope, at, page_table=t, q_weight=w, k_weight=w)

    def attend():
        shared(q_out, pools, scales, n, t, p, o, lse, max_seqlen_k=most, workspace=ws)

    def step():
        append()
        attend()
        at.add_(T)
        n.add_(T)

    run = step
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    for i in range(steps):
        qkv.normal_()
        o.fill_(float("nan"))
        for c in pools:      # what the writer has to put there, and nothing else does
            for b, L in enumerate(lens):
                for j in range(L + T * i, L + T * (i + 1)):
                    c[int(table[b, j // 16]), j % 16] = 0x7F if fp8 else float("nan")
        run()
        torch.cuda.synchronize()
        now = [L + T * (i + 1) for L in lens]
        pos = np.asarray(now)[:, None] - T + np.arange(T)
        qr = serving.norm_rotate(f64(qn), np.ones(d), 1e-6, pos, d)
        assert np.abs(f64(q_out) - qr).max() <= (2.0 ** -8 + 2.0 ** -16) * np.abs(qr).max()
        ref = attention64(q_out, *gathered(pools, scales, table, now), now)
        check(o, lse, ref, fp8, what=f"step {i}")
    n.copy_(to_dev_i32(now))
    assert launches(attend) >= kernels


def test_forked_sequences_behind_a_long_prompt():
    """A long prompt written once, forked by the block pool and decoded: each fork's own blocks and the
    prompt's, read once for the batch."""
    B, Hq, Hkv, d, prompt = 6, 8, 2, 128, 20000 + 5
    host = kv.BlockPool(-(-prompt // 16) + 2 * B)
    pools = [torch.zeros(host.num_blocks, 16, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    parent = host.create()
    host.reserve(parent, prompt)
    width = -(-prompt // 16) + 2
    table, _ = host.page_table([parent], width)
    k, v = (synth.normal_bf16((1, prompt, Hkv, d), s, "cuda") for s in (1, 2))
    kv.kv_append(*pools, k, v, to_dev_i32([0]), page_table=table.cuda())
    seqs = [parent] + [host.fork(parent) for _ in range(B - 1)]
    shared_blocks = prompt // 16
    keys = [k[0]] * B, [v[0]] * B
    for step in range(3):
        for s in seqs:
            for src, dst in host.reserve(s, 1):
                kv.copy_blocks(*pools, to_dev_i32([src]), to_dev_i32([dst]))
        t = host.page_table(seqs, width)[0].cuda()
        q = synth.normal_bf16((B, 1, Hq, d), 10 + step, "cuda")
        new = [synth.normal_bf16((B, 1, Hkv, d), s + step, "cuda") for s in (20, 30)]
        kv.kv_append(*pools, *new, to_dev_i32([prompt + step] * B), page_table=t)
        keys = tuple([torch.cat([x[b], y[b]]) for b in range(B)] for x, y in zip(keys, new))
        lens = [prompt + step + 1] * B
        o, lse = outputs(B, 1, Hq, d)
        n, p = to_dev_i32(lens), t[0, :shared_blocks].contiguous()
        shared(q, pools, [], n, t, p, o, lse)
        check(o, lse, attention64(q, *keys, lens), what=f"step {step}")
        assert launches(lambda: shared(q, pools, [], n, t, p, o, lse)) == 3


# ------------------------------------------------------------- FP8 caches under the bound of f16 weights
@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 3), (500, 20), (3000, 0), (EVERY, 0)])
@pytest.mark.parametrize("num_splits", [0, 5])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 1), (2, 12, 3), (3, 10, 2), (4, 8, 1), (5, 8, 1), (33, 8, 1), (2, 128, 1)])
def test_fp8_window_within_the_f16_bound(T, Hq, Hkv, num_splits, window, sinks):
    """At most 8, 16 and 32 rows per KV head (warp-level kernels), and the tensor-core form."""
    lens = [max(T, n) for n in (1, 16, 65, 300, 1000, 2700)]
    case = synth.decode_inputs(len(lens), T, Hq, Hkv, 128, 0, 0, seed=T + Hq, device="cuda", paged=True,
                               lengths=[L - T for L in lens], fp8=True)
    scales = [torch.as_tensor(s, device="cuda", dtype=torch.float32) for s in (case.k_scale, case.v_scale)]
    k, v = gathered([case.k_pool, case.v_pool], scales, case.page_table, lens)
    o, lse = outputs(len(lens), T, Hq, 128)
    kv.attn_decode_window_fp8(case.q, case.k_pool, case.v_pool, *scales, to_dev_i32(lens), o, window, sinks, lse=lse,
                              page_table=to_dev_i32(case.page_table), num_splits=num_splits)
    check(o, lse, attention64(case.q, k, v, lens, window, sinks), fp8=True)


@pytest.mark.parametrize("B,T,Hq,Hkv,blocks", [(4, 1, 8, 2, 20), (4, 1, 8, 2, 1300), (24, 1, 8, 2, 400), (20, 2, 16, 2, 300),
                                               (6, 8, 16, 2, 200), (3, 3, 8, 1, 40)])
def test_fp8_shared_prefix_within_the_f16_bound(B, T, Hq, Hkv, blocks):
    q, pools, scales, table, lens = shared_case(B, T, Hq, Hkv, 128, blocks, [T + 37 * b % 500 for b in range(B)], 50, True)
    o, lse = outputs(B, T, Hq, 128)
    shared(q, pools, scales, to_dev_i32(lens), to_dev_i32(table), to_dev_i32(table[0, :blocks]), o, lse)
    check(o, lse, attention64(q, *gathered(pools, scales, table, lens), lens), fp8=True)


# -------------------------------------------------------------------------------- the same bits each time
def test_calls_repeat_their_bits():
    """No sum depends on the order in which CTAs run: work queues and launches beside one another included."""
    q, k, v = synth.prefill_inputs(2, 24, 8, 900, 128, seed=1, device="cuda")
    case = synth.decode_inputs(6, 4, 16, 2, 128, 0, 0, seed=2, device="cuda", lengths=[5, 100, 900, 3000, 40, 2000])
    sh = shared_case(6, 1, 8, 2, 128, 1300, [5, 300, 64, 20, 900, 1], seed=3)
    n, t, p = to_dev_i32(sh[4]), to_dev_i32(sh[3]), to_dev_i32(sh[3][0, :1300])
    lens = to_dev_i32([L + 4 for L in (5, 100, 900, 3000, 40, 2000)])
    first = None
    for _ in range(6):
        got = [torch.empty_like(q, dtype=torch.float32), torch.empty_like(case.q, dtype=torch.float32), *outputs(6, 1, 8, 128)]
        kv.attn_prefill_window(q, k, v, got[0], 200, 4)
        kv.attn_decode_window(case.q, case.k_cache, case.v_cache, lens, got[1], 1000, 4)
        shared(sh[0], sh[1], sh[2], n, t, p, got[2], got[3])
        torch.cuda.synchronize()
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


# -------------------------------------------------------------------- offsets that do not fit in 32 bits
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_far_into_a_large_pool(fp8):
    """Blocks of a pool whose last elements lie past 2^31 elements and 2^32 bytes: written by the append, read by
    windowed and shared-prefix decode and by a windowed chunk."""
    B, Hq, Hkv, d = 3, 16, 8, 128
    total = (1 << (18 if fp8 else 17)) + 300          # blocks of 16 * 8 * 128 elements
    dtype = torch.uint8 if fp8 else torch.bfloat16
    pools = [torch.zeros(total, 16, Hkv, d, dtype=dtype, device="cuda") for _ in "kv"]
    scales = [torch.full((Hkv,), s, device="cuda") for s in (0.03, 0.02)] if fp8 else []
    blocks, shared_blocks, T = 40, 20, 280
    table = torch.stack([torch.cat([torch.arange(total - 1, total - 1 - shared_blocks, -1),
                                    torch.arange(blocks - shared_blocks) + total - 200 + 60 * b]) for b in range(B)])
    t = table.to(torch.int32).cuda()
    lens = [blocks * 16 - 9, blocks * 16, 500]
    qkv = synth.normal_bf16((B, 16 * blocks, (Hq + 2 * Hkv) * d), 3, "cuda")
    q, k, v = [x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], dim=-1)]
    k[:, :16 * shared_blocks], v[:, :16 * shared_blocks] = k[0, :16 * shared_blocks].clone(), v[0, :16 * shared_blocks].clone()
    rope, at = kv.rope_table(16 * blocks, d), to_dev_i32([0] * B)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty(B, 16 * blocks, Hq, d, dtype=torch.bfloat16, device="cuda")
    append = kv.kv_append_norm_rope_fp8 if fp8 else kv.kv_append_norm_rope
    append(*pools, q, k, v, q_out, *scales, rope, at, page_table=t, q_weight=w, k_weight=w)
    got = [pool[t[b].long()].flatten(0, 1) for pool in pools for b in range(B)]
    if fp8:
        got = [torch.as_tensor(ofp8.e4m3_decode(x.cpu().numpy()), device="cuda") * s.double()[:, None]
               for x, s in zip(got, [scales[0]] * B + [scales[1]] * B)]
    else:
        assert all(torch.equal(x, v[b]) for b, x in enumerate(got[B:]))
        kr = serving.norm_rotate(f64(k), np.ones(d), 1e-6, np.tile(np.arange(16 * blocks), (B, 1)), d)
        assert all(np.abs(f64(x) - kr[b]).max() <= (2.0 ** -8 + 2.0 ** -16) * np.abs(kr[b]).max()
                   for b, x in enumerate(got[:B]))
    ks, vs = ([x[:L] for x, L in zip(side, lens)] for side in (got[:B], got[B:]))
    n, p = to_dev_i32(lens), t[0, :shared_blocks].contiguous()
    qd = q_out[:, -1:].contiguous()
    o, lse = outputs(B, 1, Hq, d)
    fn = kv.attn_decode_window_fp8 if fp8 else kv.attn_decode_window
    fn(qd, *pools, *scales, n, o, 200, 4, lse=lse, page_table=t)
    check(o, lse, attention64(qd, ks, vs, lens, 200, 4), fp8, what="window")
    for num_splits in (0, 2):
        o, lse = outputs(B, 1, Hq, d)
        shared(qd, pools, scales, n, t, p, o, lse, num_splits=num_splits)
        check(o, lse, attention64(qd, ks, vs, lens), fp8, what="shared")
    if not fp8:
        qc = q_out[:, -T:].contiguous()
        o, lse = outputs(B, T, Hq, d)
        kv.attn_prefill_cache_window(qc, *pools, n, o, 200, 4, lse=lse, page_table=t)
        check(o, lse, attention64(qc, ks, vs, lens, 200, 4), what="chunk")


def test_rows_far_into_a_large_contiguous_cache():
    """The same for a contiguous cache of more than 2^31 elements."""
    B, Hq, Hkv, d, cap = 2, 16, 8, 128, (1 << 20) + 64
    kc, vc = (torch.zeros(B, cap, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    lens = [cap - 20, cap]
    k, v = (synth.normal_bf16((B, 2000, Hkv, d), s, "cuda") for s in (1, 2))
    q = synth.normal_bf16((B, 2000, Hq, d), 3, "cuda")
    start = [L - 2000 for L in lens]
    q_out, w = torch.empty_like(q), torch.ones(d, dtype=torch.bfloat16, device="cuda")
    rope = kv.rope_table(cap, d)
    kv.kv_append_norm_rope(kc, vc, q, k, v, q_out, rope, to_dev_i32(start), q_weight=w, k_weight=w)
    pos = np.asarray(start)[:, None] + np.arange(2000)
    kr = serving.norm_rotate(f64(k), np.ones(d), 1e-6, pos, d)
    n = to_dev_i32(lens)
    for b in range(B):
        x = f64(kc[b, start[b]:lens[b]])
        assert np.abs(x - kr[b]).max() <= (2.0 ** -8 + 2.0 ** -16) * np.abs(kr[b]).max()
        assert torch.equal(vc[b, start[b]:lens[b]], v[b])
    for T, call in ((1, kv.attn_decode_window), (8, kv.attn_decode_window), (300, kv.attn_prefill_cache_window)):
        qt = q_out[:, -T:].contiguous()
        o, lse = outputs(B, T, Hq, d)
        call(qt, kc, vc, n, o, 900, 0, lse=lse)
        # the last 2000 positions stand for the sequence: the window does not reach past them
        ref = attention64(qt, [kc[b, start[b]:lens[b]] for b in range(B)], [vc[b, start[b]:lens[b]] for b in range(B)],
                          [2000] * B, 900, 0)
        check(o, lse, ref, what=f"T={T}")
