"""GPU parity of the per-head norm, rotation and append in one pass against the fp64 oracle.

Tolerance of a bf16 output y, per element: its half step 2^-8 |y|, and fp32 arithmetic on values
up to |a| + |b| of its pair: the mean of 128 squares and the inverse square root cost below 2^-20
relative, the two roundings of each product and sum and the table's fp32 cosines 2^-22 more, so
2^-19 (|a| + |b|) covers both.  An e4m3 code adds half its step: 2^-4 |y|, or 2^-10 of the scale
below the normal range.  V and FP8 codes of V are kv_append's bits."""

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

EPS = 1e-6


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    kv.attn_get_device_status(clear=True)
    yield
    assert kv.attn_get_device_status(clear=True) == 0


def projection(B, T, Hq, Hkv, d, seed, fused=True):
    """q, k, v as views of one projection output, or contiguous."""
    qkv = synth.normal_bf16((B, T, (Hq + 2 * Hkv) * d), seed, "cuda")
    out = [x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], dim=-1)]
    return out if fused else [x.contiguous() for x in out]


def weights(d, seed):
    return [(synth.normal_bf16((d,), seed + i, "cuda").float() * 0.2 + 1).to(torch.bfloat16) for i in range(2)]


def tolerance(x, w, ref, pos, rot, interleaved):
    """2^-8 |y| + 2^-19 (|a| + |b|), the pair's values taken before the rotation."""
    y = np.abs(serving.head_norm(f64(x), None if w is None else f64(w), EPS))
    pair = y.copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        pair[..., a] = pair[..., b] = y[..., a] + y[..., b]
    return 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * pair


def check(got, x, w, pos, rot, interleaved, theta=10000.0, what=""):
    ref = serving.norm_rotate(f64(x), None if w is None else f64(w), EPS, pos, rot, theta, interleaved)
    err = np.abs(f64(got) - ref)
    assert (err <= tolerance(x, w, ref, pos, rot, interleaved)).all(), f"{what}: off by {err.max()}"
    return ref


ROT = [(128, 128, False), (128, 64, False), (128, 128, True), (128, 48, True), (128, 16, False), (64, 64, False),
       (64, 32, True), (64, 16, False), (128, 0, False), (64, 0, True), (128, 112, False)]


@pytest.mark.parametrize("d,rot,interleaved", ROT)
@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (3, 5, 6, 2), (2, 33, 8, 8), (3, 1333, 9, 2), (3, 4099, 9, 2)])
def test_qk_norm_rope_parity(d, rot, interleaved, B, T, Hq, Hkv):
    start = [0, 7, 100000][:B]
    rope = kv.rope_table(max(start) + T, rot) if rot else None
    pos = np.asarray(start)[:, None] + np.arange(T)
    for fused in (True, False):
        for norm in (True, False):
            q, k, _ = projection(B, T, Hq, Hkv, d, seed=d + T, fused=fused)
            qw, kw = weights(d, 9) if norm else (None, None)
            q_out = torch.empty(B, T, Hq, d, dtype=torch.bfloat16, device="cuda")
            k_out = torch.empty(B, T, Hkv, d, dtype=torch.bfloat16, device="cuda")
            kv.qk_norm_rope(q, k, q_out, k_out, rope, q_weight=qw, k_weight=kw, eps=EPS, interleaved=interleaved,
                            pos0=to_dev_i32(start))
            check(q_out, q, qw, pos, rot, interleaved, what="q")
            check(k_out, k, kw, pos, rot, interleaved, what="k")


def test_norm_of_one_side_only_and_positions_from_zero():
    q, k, _ = projection(2, 9, 4, 2, 64, seed=3)
    qw, _ = weights(64, 4)
    q_out, k_out = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(k.shape, dtype=q.dtype, device="cuda")
    kv.qk_norm_rope(q, k, q_out, k_out, kv.rope_table(9, 64), q_weight=qw, eps=EPS)
    pos = np.tile(np.arange(9), (2, 1))
    check(q_out, q, qw, pos, 64, False)
    check(k_out, k, None, pos, 64, False)


def test_qk_norm_rope_in_place():
    q, k, _ = projection(2, 9, 4, 2, 128, seed=5, fused=False)
    q0, k0 = q.clone(), k.clone()
    qw, kw = weights(128, 4)
    kv.qk_norm_rope(q, k, q, k, kv.rope_table(9, 128), q_weight=qw, k_weight=kw, eps=EPS)
    pos = np.tile(np.arange(9), (2, 1))
    check(q, q0, qw, pos, 128, False)
    check(k, k0, kw, pos, 128, False)


def test_extreme_rows():
    """Zero rows stay zero; rows of tiny, large and mixed size keep the relative accuracy (squares of
    up to 1e30 and the mean of 128 of them stay inside fp32); a NaN stays in its own row."""
    d = 128
    q, k, _ = projection(1, 6, 2, 1, d, seed=6, fused=False)
    q[0, 0] = 0
    q[0, 1] *= 1e15
    q[0, 2] *= 1e-15
    q[0, 3, 0, 0] = 3e4
    q[0, 4, 1, 5] = float("nan")
    qw, kw = weights(d, 4)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    kv.qk_norm_rope(q, k, q_out, k_out, kv.rope_table(6, d), q_weight=qw, k_weight=kw, eps=EPS)
    assert (q_out[0, 0] == 0).all()
    assert torch.isnan(q_out[0, 4, 1]).all() and not torch.isnan(q_out[0, 4, 0]).any()
    pos = np.arange(6)[None]
    q[0, 4, 1] = 0
    q_out[0, 4, 1] = 0
    check(q_out, q, qw, pos, d, False)
    check(k_out, k, kw, pos, d, False)


@pytest.mark.parametrize("theta,rot", [(10000.0, 128), (500000.0, 128), (10000.0, 2), (1e6, 6)])
def test_rope_table_values(theta, rot):
    """Every entry is the 64-bit value rounded once to fp32 (half a step: 2^-24 relative), the angle
    itself good to 2^-50 of it (2^-30 at the last row)."""
    rows = 1 << 16
    t = kv.rope_table(rows, rot, theta=theta)
    p = np.concatenate([np.arange(64), np.arange(64, rows, 997), [rows - 1]])
    a = p[:, None] * theta ** (-np.arange(0, rot, 2) / rot)
    ref = np.concatenate([np.cos(a), np.sin(a)], axis=1)
    got = t.cpu().numpy().astype(np.float64)[p]
    assert (np.abs(got - ref) <= 2.0 ** -24 * np.abs(ref) + 2.0 ** -30).all()


def cache_for(kind, lens, T, Hkv, d, seed):
    case = synth.decode_inputs(len(lens), T, Hkv, Hkv, d, 0, 0, seed=seed, device="cuda", paged=kind != "contig",
                               lengths=lens, capacity=max(lens) + T + 3, spare_blocks=2, fp8=kind == "fp8")
    return case, ((case.k_pool, case.v_pool) if case.paged else (case.k_cache, case.v_cache))


@pytest.mark.parametrize("kind", ["contig", "paged", "fp8", "fp8contig"])
@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (64, 32, True)])
@pytest.mark.parametrize("T", [1, 4, 37, 1501, 3203])
def test_append_norm_rope_parity(kind, d, rot, interleaved, T):
    """q_out and the new rows are right and nothing else of the cache changes; few tokens and many (one,
    two and four per warp), whole groups of them or not."""
    Hq, Hkv, lens = 6, 2, [0, 1, 15, 16, 300]
    if T > 1000:
        Hq, lens = (18, [0, 16, 301]) if d == 64 else (6, [1, 16, 301])
    B = len(lens)
    fp8 = kind.startswith("fp8")
    case = synth.decode_inputs(B, T, Hkv, Hkv, d, 0, 0, seed=20 + T, device="cuda", paged=kind in ("paged", "fp8"),
                               lengths=lens, capacity=max(lens) + T + 3, spare_blocks=2, fp8=fp8)
    kc, vc = (case.k_pool, case.v_pool) if case.paged else (case.k_cache, case.v_cache)
    before = [c.clone() for c in (kc, vc)]
    q, k, v = projection(B, T, Hq, Hkv, d, seed=21)
    qw, kw = weights(d, 22)
    rope = kv.rope_table(max(lens) + T, rot)
    table = None if case.page_table is None else to_dev_i32(case.page_table)
    q_out = torch.empty(B, T, Hq, d, dtype=torch.bfloat16, device="cuda")
    more = dict(page_table=table, q_weight=qw, k_weight=kw, eps=EPS, interleaved=interleaved)
    at = to_dev_i32(lens)
    ks = vs = None
    if fp8:
        ks, vs = (torch.as_tensor(s, device="cuda") for s in (case.k_scale, case.v_scale))
        kv.kv_append_norm_rope_fp8(kc, vc, q, k, v, q_out, ks, vs, rope, at, **more)
    else:
        kv.kv_append_norm_rope(kc, vc, q, k, v, q_out, rope, at, **more)
    pos = np.asarray(lens)[:, None] + np.arange(T)
    check(q_out, q, qw, pos, rot, interleaved, what="q")
    k_ref = serving.norm_rotate(f64(k), f64(kw), EPS, pos, rot, interleaved=interleaved)
    tol = tolerance(k, kw, k_ref, pos, rot, interleaved)
    # V as kv_append writes it, K too apart from its new rows
    k2, v2 = (c.clone() for c in before)
    if fp8:
        kv.kv_append_fp8(k2, v2, k.contiguous(), v.contiguous(), ks, vs, at, page_table=table)
    else:
        kv.kv_append(k2, v2, k.contiguous(), v.contiguous(), at, page_table=table)
    assert torch.equal(vc, v2)
    new = torch.zeros(kc.shape[:2], dtype=torch.bool, device="cuda")
    for b in range(B):
        p = torch.arange(lens[b], lens[b] + T)
        row = (torch.as_tensor(case.page_table[b])[p // 16].long(), p % 16) if case.paged else (torch.full_like(p, b), p)
        row = tuple(r.cuda() for r in row)
        new[row] = True
        got = kc[row].cpu()
        if fp8:
            s = np.asarray(case.k_scale, np.float64)[:, None]
            y = ofp8.e4m3_decode(got.numpy()) * s
            want = np.clip(k_ref[b], -448 * s, 448 * s)
            limit = (tol[b] - 2.0 ** -8 * np.abs(k_ref[b])) + 2.0 ** -4 * np.abs(want) * 1.001 + 2.0 ** -10 * s
        else:
            y, want, limit = f64(got), k_ref[b], tol[b]
        assert (np.abs(y - want) <= limit).all(), b
    assert torch.equal(kc[~new], before[0][~new])


def test_append_fp8_saturates_and_keeps_nan():
    """A key beyond 448 scales saturates, a NaN key gives the NaN code in its own row."""
    d = 128
    case, (kc, vc) = cache_for("fp8", [5, 20], 1, 1, d, 3)
    q, k, v = projection(2, 1, 1, 1, d, seed=4, fused=False)
    k[0] *= 1000.0
    k[1, 0, 0, 3] = float("nan")
    ks, vs = (torch.as_tensor(s, device="cuda") for s in (case.k_scale, case.v_scale))
    kv.kv_append_norm_rope_fp8(kc, vc, q, k, v, torch.empty_like(q), ks, vs, None, to_dev_i32([5, 20]),
                               page_table=to_dev_i32(case.page_table))
    row = [kc[int(case.page_table[b, p // 16]), p % 16, 0].cpu().numpy() for b, p in ((0, 5), (1, 20))]
    assert np.array_equal(row[0], ofp8.quantize_rows(f64(k[0, 0]), case.k_scale)[0])
    assert (row[0] & 0x7F == 0x7E).any()
    assert row[1][3] & 0x7F == 0x7F and (np.delete(row[1], 3) & 0x7F != 0x7F).all()


def test_append_range_position_and_page_errors():
    d, Hq, Hkv = 128, 4, 2
    q, k, v = projection(3, 2, Hq, Hkv, d, seed=8)
    kc = torch.zeros(3, 40, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    q_out = torch.empty(3, 2, Hq, d, dtype=torch.bfloat16, device="cuda")
    # beyond the cache: that token is left out, q is still written
    kv.kv_append_norm_rope(kc, vc, q, k, v, q_out, kv.rope_table(64, d), to_dev_i32([0, 39, 10]))
    assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_APPEND_RANGE
    assert torch.isfinite(q_out).all()
    assert [int((c[:, :, 0].abs().sum(-1) > 0).sum()) for c in (kc, vc)] == [5, 5]
    # a position outside the angle table: NaN queries, cache as it was; V too
    kc.zero_(), vc.zero_()
    kv.kv_append_norm_rope(kc, vc, q, k, v, q_out, kv.rope_table(11, d), to_dev_i32([0, -1, 10]))
    assert kv.attn_get_device_status(clear=True) & kv.ATTN_DEV_POSITION
    nan = torch.isnan(q_out).all(-1).all(-1)
    assert nan.tolist() == [[False, False], [True, False], [False, True]]
    assert int((kc[:, :, 0].abs().sum(-1) > 0).sum()) == int((vc[:, :, 0].abs().sum(-1) > 0).sum()) == 4
    # a block outside the pool
    pool = torch.zeros(4, 16, Hkv, d, dtype=torch.bfloat16, device="cuda")
    kv.kv_append_norm_rope(pool, pool.clone(), q, k, v, q_out, kv.rope_table(64, d), to_dev_i32([0, 0, 0]),
                           page_table=to_dev_i32([[0], [4], [-1]]))
    assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_PAGE_ID
    assert int((pool[:, :, 0].abs().sum(-1) > 0).sum()) == 2
    # the dense form outside its table
    k_out = torch.empty(3, 2, Hkv, d, dtype=torch.bfloat16, device="cuda")
    kv.qk_norm_rope(q, k, q_out, k_out, kv.rope_table(3, d), pos0=to_dev_i32([0, 2, 1]))
    assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_POSITION
    assert torch.isnan(q_out[1, 1]).all() and torch.isnan(k_out[1, 1]).all()
    assert torch.isfinite(q_out[[0, 2]]).all() and torch.isfinite(k_out[[0, 2]]).all()


def test_append_bad_scale_is_flagged():
    case, (kc, vc) = cache_for("fp8", [5], 1, 2, 128, 3)
    before = kc.clone()
    q, k, v = projection(1, 1, 2, 2, 128, seed=4)
    bad = torch.tensor([0.0, float("inf")], device="cuda")
    kv.kv_append_norm_rope_fp8(kc, vc, q, k, v, torch.empty(q.shape, dtype=q.dtype, device="cuda"), bad, bad, None,
                               to_dev_i32([5]), page_table=to_dev_i32(case.page_table))
    assert kv.attn_get_device_status(clear=True) == kv.ATTN_DEV_SCALE
    assert torch.equal(kc, before)


def test_norm_rope_replays_in_a_graph_on_its_stream():
    B, T, Hq, Hkv, d = 3, 1, 4, 2, 128
    q, k, v = projection(B, T, Hq, Hkv, d, seed=8)
    kc = torch.zeros(B, 50, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    q_out = torch.empty(B, T, Hq, d, dtype=torch.bfloat16, device="cuda")
    lens, rope = to_dev_i32([0, 5, 20]), kv.rope_table(64, d)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        kv.kv_append_norm_rope(kc, vc, q, k, v, q_out, rope, lens)
        lens.add_(1)
    for step in range(3):
        q.normal_()
        g.replay()
        torch.cuda.synchronize()
        pos = np.asarray([0, 5, 20])[:, None] + step
        check(q_out, q, None, pos, d, False)
    assert lens.tolist() == [3, 8, 23]
    assert int((vc[:, :, 0].abs().sum(-1) > 0).sum()) == 9
