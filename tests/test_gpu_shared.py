"""GPU parity of decode over a batch that shares a prefix, against the fp64 oracle's plain paged
decode (tolerances as derived in test_gpu_window.py), and of the serving step that the window,
shared-prefix and norm-rotate-append calls make together."""

import math

import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import fp8 as ofp8
from oracle import serving

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("kv_cache_decode_attn_b200")
from tests.gpu_util import f64, to_dev_i32  # noqa: E402
from tests.test_gpu_window import check  # noqa: E402


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    kv.attn_get_device_status(clear=True)
    yield
    assert kv.attn_get_device_status(clear=True) == 0


def make(B, T, Hkv, Hq, d, prefix_blocks, own, seed, fp8=False):
    """Pools, the true table (prefix in every row) and the lengths of sequences with own[b] >= T
    keys behind the prefix."""
    lens = [16 * prefix_blocks + L for L in own]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    nblk = [-(-L // 16) for L in own]
    total = prefix_blocks + sum(nblk) + 2
    perm = synth.block_permutation(total, seed)
    table = np.full((B, prefix_blocks + max(nblk)), -1, dtype=np.int32)
    table[:, :prefix_blocks] = perm[:prefix_blocks]
    at = prefix_blocks
    for b, n in enumerate(nblk):
        table[b, prefix_blocks:prefix_blocks + n] = perm[at:at + n]
        at += n
    q = synth.normal_bf16((B, T, Hq, d), seed + 1, "cuda")
    if fp8:
        ks, vs = synth.kv_scales(Hkv, seed + 2), synth.kv_scales(Hkv, seed + 3)
        kp, vp = (synth.normal_e4m3_codes((total, 16, Hkv, d), s, seed + i, "cuda") for i, s in ((4, ks), (5, vs)))
        return q, kp, vp, ks, vs, table, lens
    kp, vp = (synth.normal_bf16((total, 16, Hkv, d), seed + i, "cuda") for i in (4, 5))
    return q, kp, vp, None, None, table, lens


def reference(q, kp, vp, ks, vs, table, lens, scale, causal=True):
    kh, vh = (f64(kp), f64(vp)) if ks is None else \
        (ofp8.e4m3_decode(kp.cpu().numpy()) * np.asarray(ks, np.float64)[:, None],
         ofp8.e4m3_decode(vp.cpu().numpy()) * np.asarray(vs, np.float64)[:, None])
    ref = oracle.decode_paged(f64(q), kh, vh, table, lens, scale, causal)
    weight = oracle.decode_paged(f64(q), kh, np.abs(vh), table, lens, scale, causal)[0]
    return ref, weight


def call(q, kp, vp, ks, vs, table, lens, prefix_blocks, o_dtype=torch.float32, **kw):
    B, T, Hq, d = q.shape
    prefix = to_dev_i32(table[0, :prefix_blocks])
    hidden = table.copy()
    hidden[:, :prefix_blocks] = -1          # the shared columns are not read
    o = torch.full((B, T, Hq, d), float("nan"), dtype=o_dtype, device="cuda")
    lse = torch.full((B, Hq, T), float("nan"), device="cuda")
    if ks is None:
        kv.attn_decode_shared(q, kp, vp, to_dev_i32(lens), to_dev_i32(hidden), prefix, o, lse=lse, **kw)
    else:
        kv.attn_decode_shared_fp8(q, kp, vp, torch.as_tensor(ks, device="cuda"), torch.as_tensor(vs, device="cuda"),
                                  to_dev_i32(lens), to_dev_i32(hidden), prefix, o, lse=lse, **kw)
    return o, lse


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hkv,d,prefix_blocks,own", [
    (1, 1, 8, 2, 128, 1, [1]),                                  # one sequence, one block, one own key
    (2, 1, 4, 4, 64, 3, [1, 40]),                               # one row per KV head and sequence
    (3, 2, 8, 2, 128, 40, [2, 16, 300]),
    (5, 1, 16, 2, 128, 130, [1, 15, 16, 17, 700]),              # 40 prefix rows per KV head
    (7, 4, 8, 1, 128, 33, [4, 5, 64, 65, 100, 1000, 6]),        # 224 prefix rows: two row tiles
    (40, 1, 8, 1, 64, 9, [1 + 7 * i for i in range(40)]),
    (33, 1, 6, 2, 128, 70, [1 + 20 * (i % 9) for i in range(33)]),   # odd group size
    (2, 300, 2, 1, 128, 20, [300, 401]),                        # long own parts, many new tokens
])
def test_shared_prefix_parity(fp8, B, T, Hq, Hkv, d, prefix_blocks, own):
    if fp8 and d != 128:
        pytest.skip("FP8 caches are built for d = 128")
    args = make(B, T, Hkv, Hq, d, prefix_blocks, own, seed=100 + B, fp8=fp8)
    ref, weight = reference(*args, 1.0 / math.sqrt(d))
    for dtype in (torch.float32, torch.bfloat16):
        o, lse = call(*args, prefix_blocks, o_dtype=dtype)
        check(o, lse, ref, weight, f"B={B} T={T}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hkv,d,prefix_blocks,own", [
    (24, 1, 8, 2, 128, 400, [1 + 13 * i for i in range(24)]),          # 96 prefix rows: the tensor-core kernel
    (20, 2, 16, 2, 128, 300, [2 + 7 * i for i in range(20)]),          # 320 rows: several row tiles, 16 own rows
    (5, 1, 6, 2, 128, 1500, [1, 16, 17, 100, 640]),                    # 15 rows: the warp-level kernels
    (2, 1, 8, 2, 128, 4000, [5, 300]),                                 # 8 rows
    (30, 1, 4, 2, 64, 500, [1 + 29 * i for i in range(30)]),
    (20, 8, 16, 2, 128, 300, [8 + 31 * i for i in range(20)]),         # 64 own rows: tensor cores there too
])
def test_long_shared_prefix_parity(fp8, B, T, Hq, Hkv, d, prefix_blocks, own):
    """Prefixes long enough that they are read once for the batch (short ones are read by each sequence)."""
    if fp8 and d != 128:
        pytest.skip("FP8 caches are built for d = 128")
    args = make(B, T, Hkv, Hq, d, prefix_blocks, own, seed=200 + B, fp8=fp8)
    ref, weight = reference(*args, 1.0 / math.sqrt(d))
    for causal in (True, False):
        o, lse = call(*args, prefix_blocks, causal=causal)
        if not causal:
            ref, weight = reference(*args, 1.0 / math.sqrt(d), False)
        check(o, lse, ref, weight, f"B={B} T={T} causal={causal}")
    # a length short of prefix + T, and a block outside the pool
    lens = list(args[6])
    short = list(args)
    short[6] = [16 * prefix_blocks + T - 1] + lens[1:]
    o, lse = call(*short, prefix_blocks, causal=False)
    assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_SEQLEN
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    check(o[1:], lse[1:], (ref[0][1:], ref[1][1:]), weight[1:])
    table = args[5].copy()
    table[0, prefix_blocks // 2] = -7
    bad = list(args)
    bad[5] = table
    call(*bad, prefix_blocks)
    assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_PAGE_ID


@pytest.mark.parametrize("num_splits", [1, 3, 40])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fp8", [False, True])
def test_shared_prefix_splits(num_splits, causal, fp8):
    args = make(6, 3, 2, 8, 128, 50, [3, 9, 100, 64, 400, 33], seed=7, fp8=fp8)
    ref, weight = reference(*args, 0.1, causal)
    o, lse = call(*args, 50, num_splits=num_splits, causal=causal, scale=0.1)
    check(o, lse, ref, weight)


def test_no_shared_blocks_is_plain_decode():
    args = make(4, 2, 2, 8, 128, 0, [2, 30, 500, 64], seed=8)
    o, lse = call(*args, 0)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    q, kp, vp, _, _, table, lens = args
    kv.attn_decode(q, kp, vp, to_dev_i32(lens), o2, lse2, page_table=to_dev_i32(table))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_shared_prefix_ignores_what_lies_past_the_lengths():
    args = make(3, 1, 2, 8, 128, 4, [5, 16, 37], seed=9)
    q, kp, vp, _, _, table, lens = args
    ref, weight = reference(*args, 128 ** -0.5)
    for b, L in enumerate(lens):
        if L % 16:
            for c in (kp, vp):
                c[int(table[b, L // 16]), L % 16:] = float("nan")
    o, lse = call(*args, 4)
    check(o, lse, ref, weight)


@pytest.mark.parametrize("T", [1, 8])
def test_shared_prefix_length_and_page_errors(T):
    args = list(make(3, T, 2, 8, 128, 10, [T, 50, 80], seed=10))
    ref, weight = reference(*args, 128 ** -0.5)
    good = list(args[6])
    args[6] = [160 + T - 1, good[1], good[2]]         # sequence 0: fewer keys than prefix + T
    o, lse = call(*args, 10)
    assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_SEQLEN
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    check(o[1:], lse[1:], (ref[0][1:], ref[1][1:]), weight[1:])
    args[6] = good
    args[5] = args[5].copy()
    args[5][0, 3] = 1 << 20                           # a block of the prefix outside the pool
    call(*args, 10)
    assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_PAGE_ID


def test_shared_prefix_bad_scale_is_flagged():
    args = list(make(2, 1, 2, 8, 128, 5, [3, 40], seed=11, fp8=True))
    args[3] = np.array([np.nan, 0.02], np.float32)
    o, lse = call(*args, 5)
    assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_SCALE
    assert torch.isnan(o[:, :, :4]).all() and not torch.isnan(o[:, :, 4:]).any()


@pytest.mark.parametrize("blocks", [30, 1200])   # read by each sequence, and once for the batch
def test_shared_prefix_replays_in_a_graph(blocks):
    args = make(5, 1, 2, 8, 128, blocks, [9, 100, 64, 20, 300], seed=12)
    q, kp, vp, _, _, table, lens = args
    t, p, n = to_dev_i32(table), to_dev_i32(table[0, :blocks]), to_dev_i32(lens)
    o, lse = torch.empty(5, 1, 8, 128, device="cuda"), torch.empty(5, 8, 1, device="cuda")
    ws = kv.decode_shared_workspace(5, 1, 8, 2, 128, max(lens), blocks)

    def go():
        kv.attn_decode_shared(q, kp, vp, n, t, p, o, lse=lse, max_seqlen_k=max(lens), workspace=ws)

    go()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for shift in (0, 3, 8):
        now = [L - shift for L in lens]
        n.copy_(to_dev_i32(now))
        q.normal_()
        o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref, weight = reference(q, kp, vp, None, None, table, now, 128 ** -0.5)
        check(o, lse, ref, weight)


@pytest.mark.parametrize("fp8", [False, True])
def test_serving_step_of_forked_sequences(fp8):
    """A prompt written once, forked by the block pool, and decoded for several steps: norm, rotation
    and append of each new token, then attention over the shared prefix, and over a window."""
    B, Hq, Hkv, d, prompt, steps, rot, eps = 4, 8, 2, 128, 70, 3, 64, 1e-6
    n_blocks = 64
    host = kv.BlockPool(n_blocks)
    shape = (n_blocks, 16, Hkv, d)
    kp, vp = (torch.zeros(shape, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in "kv")
    scales = ()
    if fp8:
        scales = tuple(torch.as_tensor(synth.kv_scales(Hkv, s), device="cuda") for s in (1, 2))
    qw, kw = (synth.normal_bf16((d,), s, "cuda") * 0.1 + 1 for s in (3, 4))
    rope = kv.rope_table(256, rot)
    # what each sequence's cache should hold, from the oracle
    keys = [np.zeros((0, Hkv, d)) for _ in range(B)]
    vals = [np.zeros((0, Hkv, d)) for _ in range(B)]

    def append(seqs, lens, T, seed):
        n = len(seqs)
        table = host.page_table(seqs, 8)[0].cuda()
        qkv = synth.normal_bf16((n, T, (Hq + 2 * Hkv) * d), seed, "cuda")
        q = qkv[..., :Hq * d].unflatten(-1, (Hq, d))
        k = qkv[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d))
        v = qkv[..., (Hq + Hkv) * d:].unflatten(-1, (Hkv, d))
        q_out = torch.empty(n, T, Hq, d, dtype=torch.bfloat16, device="cuda")
        at = to_dev_i32(lens)
        more = dict(page_table=table, q_weight=qw, k_weight=kw, eps=eps)
        if fp8:
            kv.kv_append_norm_rope_fp8(kp, vp, q, k, v, q_out, *scales, rope, at, **more)
        else:
            kv.kv_append_norm_rope(kp, vp, q, k, v, q_out, rope, at, **more)
        pos = np.asarray(lens)[:, None] + np.arange(T)
        qr = serving.norm_rotate(f64(q), f64(qw), eps, pos, rot)
        assert np.abs(f64(q_out) - qr).max() <= (2.0 ** -8 + 2.0 ** -16) * np.abs(qr).max()
        return q_out, serving.norm_rotate(f64(k), f64(kw), eps, pos, rot), f64(v), table

    def stored(table, b, L):
        """Sequence b's cache rows as the pools hold them."""
        out = []
        for pool, s in ((kp, 0), (vp, 1)):
            x = ofp8.e4m3_decode(pool.cpu().numpy()) * f64(scales[s])[:, None] if fp8 else f64(pool)
            out.append(oracle.gather_paged(x, table.cpu().numpy()[b:b + 1], [L])[0])
        return out

    step = 2.0 ** -4 if fp8 else 2.0 ** -8
    parent = host.create()
    host.reserve(parent, prompt)
    _, k0, v0, _ = append([parent], [0], prompt, 10)
    seqs = [parent] + [host.fork(parent) for _ in range(B - 1)]
    for b in range(B):
        keys[b], vals[b] = k0[0], v0[0]
    shared = prompt // 16
    for i in range(steps):
        L = prompt + i
        for s in seqs:
            for src, dst in host.reserve(s, 1):
                kv.copy_blocks(kp, vp, to_dev_i32([src]), to_dev_i32([dst]))
        q_out, k1, v1, table = append(seqs, [L] * B, 1, 20 + i)
        for b in range(B):
            keys[b], vals[b] = np.concatenate([keys[b], k1[b]]), np.concatenate([vals[b], v1[b]])
            got = stored(table, b, L + 1)
            for g, want in zip(got, (keys[b], vals[b])):
                assert (np.abs(g - want) <= step * 1.001 * np.abs(want) + 2.0 ** -10 / 16).all()
        lens = [L + 1] * B
        o, lse = torch.empty(B, 1, Hq, d, device="cuda"), torch.empty(B, Hq, 1, device="cuda")
        kc = np.stack([stored(table, b, L + 1)[0] for b in range(B)])
        vc = np.stack([stored(table, b, L + 1)[1] for b in range(B)])
        qh = f64(q_out)
        if fp8:
            kv.attn_decode_shared_fp8(q_out, kp, vp, *scales, to_dev_i32(lens), table, table[0, :shared], o, lse=lse)
        else:
            kv.attn_decode_shared(q_out, kp, vp, to_dev_i32(lens), table, table[0, :shared], o, lse=lse)
        check(o, lse, oracle.decode(qh, kc, vc, lens, d ** -0.5, True),
              oracle.decode(qh, kc, np.abs(vc), lens, d ** -0.5, True)[0], f"step {i}")
        o.fill_(float("nan"))
        if fp8:
            kv.attn_decode_window_fp8(q_out, kp, vp, *scales, to_dev_i32(lens), o, 20, 4, lse=lse, page_table=table)
        else:
            kv.attn_decode_window(q_out, kp, vp, to_dev_i32(lens), o, 20, 4, lse=lse, page_table=table)
        check(o, lse, serving.attention_window(qh, kc, vc, d ** -0.5, lens, 20, 4),
              serving.attention_window(qh, kc, np.abs(vc), d ** -0.5, lens, 20, 4)[0], f"window step {i}")


def test_serving_steps_in_one_graph():
    """Norm-rotate-append, then attention over a window and over the shared prefix, captured once and
    replayed while the lengths grow on the device: each call sees what the one before it wrote."""
    B, Hq, Hkv, d, prefix_blocks, steps, window, sinks = 5, 8, 2, 128, 40, 6, 700, 4
    own = [1, 16, 31, 100, 900]
    q, kp, vp, _, _, table, lens = make(B, 1, Hkv, Hq, d, prefix_blocks, [L + steps for L in own], seed=21)
    lens = [16 * prefix_blocks + L for L in own]
    qkv = torch.empty(B, 1, (Hq + 2 * Hkv) * d, dtype=torch.bfloat16, device="cuda")
    qn, kn, vn = [x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], dim=-1)]
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    rope, at, n = kv.rope_table(4096, d), to_dev_i32(lens), to_dev_i32([L + 1 for L in lens])
    t, p = to_dev_i32(table), to_dev_i32(table[0, :prefix_blocks])
    q_out = torch.empty(B, 1, Hq, d, dtype=torch.bfloat16, device="cuda")
    o = [torch.empty(B, 1, Hq, d, device="cuda") for _ in range(2)]
    lse = [torch.empty(B, Hq, 1, device="cuda") for _ in range(2)]
    most = max(lens) + steps
    ws = kv.decode_window_workspace(B, 1, Hq, Hkv, d, most, window, sinks)
    ws2 = kv.decode_shared_workspace(B, 1, Hq, Hkv, d, most, prefix_blocks)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.kv_append_norm_rope(kp, vp, qn, kn, vn, q_out, rope, at, page_table=t, q_weight=w, k_weight=w)
        kv.attn_decode_window(q_out, kp, vp, n, o[0], window, sinks, lse=lse[0], page_table=t, max_seqlen_k=most,
                              workspace=ws)
        kv.attn_decode_shared(q_out, kp, vp, n, t, p, o[1], lse=lse[1], max_seqlen_k=most, workspace=ws2)
        at.add_(1)
        n.add_(1)
    for step in range(steps):
        qkv.normal_()
        g.replay()
        torch.cuda.synchronize()
        now = [L + step + 1 for L in lens]
        pos = np.asarray(now)[:, None] - 1
        qr = serving.norm_rotate(f64(qn), np.ones(d), 1e-6, pos, d)
        assert np.abs(f64(q_out) - qr).max() <= (2.0 ** -8 + 2.0 ** -16) * np.abs(qr).max()
        kc, vc = (oracle.gather_paged(f64(x), table, now) for x in (kp, vp))
        new = serving.norm_rotate(f64(kn), np.ones(d), 1e-6, pos, d)[:, 0]
        for b in range(B):
            assert np.abs(kc[b, now[b] - 1] - new[b]).max() <= (2.0 ** -8 + 2.0 ** -16) * np.abs(new[b]).max()
            assert np.array_equal(vc[b, now[b] - 1], f64(vn)[b, 0])
        qh = f64(q_out)
        check(o[0], lse[0], serving.attention_window(qh, kc, vc, d ** -0.5, now, window, sinks),
              serving.attention_window(qh, kc, np.abs(vc), d ** -0.5, now, window, sinks)[0], f"window, step {step}")
        check(o[1], lse[1], oracle.decode(qh, kc, vc, now, d ** -0.5, True),
              oracle.decode(qh, kc, np.abs(vc), now, d ** -0.5, True)[0], f"shared, step {step}")


def test_shared_prefix_on_two_streams():
    """Two calls in flight, each with a workspace of its own."""
    args = [make(6, 1, 2, 8, 128, 60, [5, 300, 64, 20, 900, 1], seed=s) for s in (31, 32)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    bufs = []
    for q, kp, vp, _, _, table, lens in args:
        bufs.append((to_dev_i32(lens), to_dev_i32(table), to_dev_i32(table[0, :60]), torch.empty(6, 1, 8, 128, device="cuda"),
                     torch.empty(6, 8, 1, device="cuda"), kv.decode_shared_workspace(6, 1, 8, 2, 128, max(lens), 60)))
    torch.cuda.synchronize()
    for _ in range(5):
        for (q, kp, vp, *_), (n, t, p, o, lse, ws), s in zip(args, bufs, streams):
            kv.attn_decode_shared(q, kp, vp, n, t, p, o, lse=lse, max_seqlen_k=16 * 60 + 900, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for a, (_, _, _, o, lse, _) in zip(args, bufs):
        ref, weight = reference(*a, 128 ** -0.5)
        check(o, lse, ref, weight)
