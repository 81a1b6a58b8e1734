"""Cases of the attention operators next to the plain prefill and decode calls:

* ``rope``           per-head RMS norm of queries and keys with the position rotation, in the pass
                     that writes the new tokens' K and V (into a contiguous, paged or FP8 cache, or
                     dense for a whole prompt);
* ``window_decode``  decode of T new tokens that see a sliding window and a few first tokens;
* ``window_prefill`` the same mask over a whole prompt, and ``window_chunk`` over a prompt chunk
                     appended to a cache;
* ``shared``         decode of a batch whose sequences share a long prefix held once in the cache.

``run`` computes them from elementary torch operations where ``own`` is false, and through the
framework's entry points where it is true.  Sizes are this repository's workloads (GPT-2-small and
Llama-3.1-8B head layouts, 16-token pages) and generic ones.
"""

import math

import torch

own = False

PAGE = 16


def _framework():
    import kv_cache_decode_attn_b200 as kv

    return kv


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 16 sequences: the new token's q, k, v come as views of a fused projection
        dict(name="rope_append_decode", op="rope", cache="paged", B=16, T=1, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, lo=1024, hi=32768),
        # four new tokens per sequence (speculative verify) into an FP8 cache
        dict(name="rope_append_fp8_verify", op="rope", cache="fp8", B=8, T=4, Hq=64, Hkv=8, d=128, rot=128,
             interleaved=False, lo=4096, hi=16384),
        # a whole prompt batch, dense, half of each head rotated in adjacent pairs (d = 64 heads)
        dict(name="rope_dense_d64_partial", op="rope", cache="dense", B=8, T=1023, Hq=12, Hkv=12, d=64, rot=32,
             interleaved=True, lo=0, hi=0),
        # four 4096-token prompts written to a contiguous cache
        dict(name="rope_append_prompt", op="rope", cache="contig", B=4, T=4096, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, lo=0, hi=0),
        # one token per sequence, window of 1024, four sinks, contiguous cache
        dict(name="window_decode_contig", op="window_decode", cache="contig", B=16, T=1, Hq=32, Hkv=8, d=128,
             window=1024, sinks=4, lo=1024, hi=32768),
        # a long FP8 cache behind a page table, window of 8192
        dict(name="window_decode_fp8", op="window_decode", cache="fp8", B=8, T=1, Hq=64, Hkv=8, d=128,
             window=8192, sinks=16, lo=16384, hi=65536),
        # speculative verify with a window: 32 query rows per KV head
        dict(name="window_verify_paged", op="window_decode", cache="paged", B=8, T=4, Hq=64, Hkv=8, d=128,
             window=4096, sinks=5, lo=32768, hi=65536),
        # prompts of the Llama layout with a window
        dict(name="window_prefill_gqa", op="window_prefill", B=2, Hq=32, Hkv=8, N=4096, d=128, window=1024, sinks=4),
        # short odd prompts of the GPT-2 layout
        dict(name="window_prefill_d64_odd", op="window_prefill", B=8, Hq=12, Hkv=12, N=1023, d=64, window=255,
             sinks=0),
        # a 512-token chunk appended to cached prefixes
        dict(name="window_chunk_paged", op="window_chunk", cache="paged", B=4, T=512, Hq=32, Hkv=8, d=128,
             window=4096, sinks=64, lo=4096, hi=16384),
        # a few parallel samples of one prompt
        dict(name="shared_few", op="shared", cache="paged", B=4, T=1, Hq=32, Hkv=8, d=128, prefix=1024, lo=1, hi=100),
        # many requests behind one long system prompt
        dict(name="shared_long", op="shared", cache="paged", B=64, T=1, Hq=32, Hkv=8, d=128, prefix=32768, lo=33,
             hi=2048),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges: decode batches of 1 to 64 sequences, prompts of 1 to 4096
    tokens, windows of 1 to 8192, prefixes of 16 to 32768 tokens, both head sizes, all cache layouts.
    None needs more work than the largest listed one."""
    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        c = _any(rng)
        if all(work(c)[k] <= most[k] for k in most):
            return c


def _any(rng):
    op = rng.choice(["rope", "window_decode", "window_prefill", "window_chunk", "shared"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    if op == "rope":
        cache = rng.choice(["dense", "contig", "paged", "fp8"])
        T = _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(64, 16384 // T)))
        lo = _log_int(rng, 1, 8192)
        return dict(op=op, cache=cache, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2]),
                    interleaved=rng.random() < 0.3, lo=lo, hi=lo + _log_int(rng, 1, 8192))
    if op == "window_decode":
        cache = rng.choice(["contig", "paged", "fp8"])
        T = rng.choice([1, 1, 2, 3, 4, 7, 8])
        window, sinks = _log_int(rng, 1, 8192), rng.choice([0, 1, 4, 16, 33])
        lo = max(T, _log_int(rng, 16, 32768))
        return dict(op=op, cache=cache, B=_log_int(rng, 1, 16), T=T, Hq=Hq, Hkv=Hkv, d=128 if cache == "fp8" else d,
                    window=window, sinks=sinks, lo=lo, hi=lo + _log_int(rng, 1, 16384))
    if op == "window_prefill":
        N = _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(16, (2 << 20) // (N * N + 1), 64 // Hq)))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, N=N, d=d, window=_log_int(rng, 1, 4096),
                    sinks=rng.choice([0, 1, 4, 100]))
    if op == "window_chunk":
        T = _log_int(rng, 32, 512)
        lo = T + _log_int(rng, 16, 8192)
        return dict(op=op, cache=rng.choice(["contig", "paged"]), B=_log_int(rng, 1, 4), T=T, Hq=min(Hq, 32 // Hkv * Hkv),
                    Hkv=Hkv, d=d, window=_log_int(rng, 16, 4096), sinks=rng.choice([0, 4, 64]), lo=lo,
                    hi=lo + _log_int(rng, 1, 4096))
    cache = rng.choice(["paged", "paged", "fp8"])
    T = rng.choice([1, 1, 1, 2, 4])
    prefix = PAGE * _log_int(rng, 1, 2048)
    lo = T + _log_int(rng, 1, 512)
    return dict(op=op, cache=cache, B=max(1, _log_int(rng, 2, 64) // T), T=T, Hq=Hkv * min(4, Hq // Hkv), Hkv=Hkv,
                d=128 if cache == "fp8" else d, prefix=prefix, lo=lo, hi=lo + _log_int(rng, 1, 1024))


def _lengths(c):
    """The batch's lengths, evenly spread over [lo, hi] (which sequence has which is the seed's choice)."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [lo + (hi - lo) * i // max(1, B - 1) for i in range(B)]


# ------------------------------------------------------------------ inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _pool(g, cache, *shape, Hkv):
    """Cache contents: N(0, 1) in bf16, or e4m3 codes of about N(0, 1) under one scale per KV head."""
    if cache != "fp8":
        return _normal(g, *shape), None
    scale = torch.rand(Hkv, generator=g, device="cuda") * (3 / 64) + 1 / 64
    x = _normal(g, *shape)
    x = (x / scale.to(torch.bfloat16)[:, None]).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return x, scale


def _table(g, blocks, width):
    """A page table whose sequences own `blocks[b]` blocks each, physical ids permuted; unused entries -1."""
    total = sum(blocks)
    perm = torch.randperm(total, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((len(blocks), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def _order(g, lens):
    at = torch.randperm(len(lens), generator=g, device="cuda").tolist()
    return [lens[i] for i in at]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _rope_table(rows, rot):
    """Cosines, then sines, of position * 10000^(-2 i / rot): angles in 64 bits, rounded once."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, d, Hq, Hkv, B = c["op"], c["d"], c["Hq"], c["Hkv"], c["B"]
    s = {"c": c, "scale": d ** -0.5}
    if op == "window_prefill":
        N = c["N"]
        s.update(q=_normal(g, B, N, Hq, d), k=_normal(g, B, N, Hkv, d), v=_normal(g, B, N, Hkv, d))
        s.update(o=torch.empty_like(s["q"]), lse=torch.empty(B, Hq, N, device="cuda"))
        return s
    T = c["T"]
    if op == "rope":
        lens = _order(g, _lengths(c))
        qkv = _normal(g, B, T, (Hq + 2 * Hkv) * d)      # the projection's output; q, k, v are views of it
        s["q"] = qkv[..., :Hq * d].unflatten(-1, (Hq, d))
        s["k"] = qkv[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d))
        s["v"] = qkv[..., (Hq + Hkv) * d:].unflatten(-1, (Hkv, d))
        s["qw"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
        s["kw"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
        s["rope"] = _rope_table(max(lens) + T, c["rot"])
        s["q_out"] = torch.empty(B, T, Hq, d, dtype=torch.bfloat16, device="cuda")
        s["lens"], s["eps"] = _i32(lens), 1e-6
        if c["cache"] == "dense":
            s["k_out"] = torch.empty(B, T, Hkv, d, dtype=torch.bfloat16, device="cuda")
            return s
        s["ks"] = s["vs"] = s["table"] = None
        if c["cache"] == "contig":
            cap = max(lens) + T
            s["kc"], s["vc"] = (torch.zeros(B, cap, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
            return s
        blocks = [-(-(L + T) // PAGE) for L in lens]
        s["table"], total = _table(g, blocks, max(blocks))
        kind = torch.bfloat16 if c["cache"] == "paged" else torch.float8_e4m3fn
        s["kc"], s["vc"] = (torch.zeros(total, PAGE, Hkv, d, device="cuda", dtype=torch.bfloat16).to(kind) for _ in "kv")
        if c["cache"] == "fp8":
            s["ks"], s["vs"] = (torch.rand(Hkv, generator=g, device="cuda") * (3 / 64) + 1 / 64 for _ in "kv")
        return s
    s["q"] = _normal(g, B, T, Hq, d)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(B, Hq, T, device="cuda")
    lens = _order(g, _lengths(c))
    if op == "shared":
        n = c["prefix"] // PAGE
        own_blocks = [-(-L // PAGE) for L in lens]      # blocks past the shared prefix
        suffix, total = _table(g, own_blocks, max(own_blocks))
        perm = torch.randperm(total + n, generator=g, device="cuda", dtype=torch.int32)
        moved = torch.where(suffix >= 0, perm[suffix.clamp(min=0).long()], suffix)
        s["table"] = torch.cat([perm[total:].expand(B, n), moved], dim=1).contiguous()
        s["kc"], s["ks"] = _pool(g, c["cache"], total + n, PAGE, Hkv, d, Hkv=Hkv)
        s["vc"], s["vs"] = _pool(g, c["cache"], total + n, PAGE, Hkv, d, Hkv=Hkv)
        s["lens"] = _i32([c["prefix"] + L for L in lens])
        s["max_len"] = c["prefix"] + max(lens)
        return s
    s["lens"], s["max_len"] = _i32(lens), max(lens)
    if c["cache"] == "contig":
        s["table"] = s["ks"] = s["vs"] = None
        s["kc"], s["vc"] = (_normal(g, B, max(lens), Hkv, d) for _ in "kv")
        return s
    blocks = [-(-L // PAGE) for L in lens]
    s["table"], total = _table(g, blocks, max(blocks))
    s["kc"], s["ks"] = _pool(g, c["cache"], total, PAGE, Hkv, d, Hkv=Hkv)
    s["vc"], s["vs"] = _pool(g, c["cache"], total, PAGE, Hkv, d, Hkv=Hkv)
    return s


# ------------------------------------------------------------------ the plain forms
def _norm_rotate(x, weight, table, positions, eps, rot, interleaved):
    """x [B, T, H, d] in fp32: x * rsqrt(mean(x^2) + eps) * weight, then the first `rot` elements of
    each head rotated by the angles of its token's position."""
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()
    cos, sin = table[positions].unsqueeze(2).split(rot // 2, dim=-1)        # [B, T, 1, rot / 2]
    r = x[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r.split(rot // 2, dim=-1)
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([r, x[..., rot:]], dim=-1)


def _slots(s, positions):
    """Rows of the caches viewed as [rows, Hkv, d] that hold these positions [B, n]."""
    if s["table"] is None:
        return positions + torch.arange(positions.shape[0], device="cuda")[:, None] * s["kc"].shape[1]
    blocks = s["table"].long().gather(1, positions // PAGE)
    return blocks * PAGE + positions % PAGE


def _rows(cache, scale, slots):
    """Cached rows at `slots` in fp32, [..., Hkv, d]."""
    x = cache.view(-1, *cache.shape[2:])
    x = x.view(torch.uint8)[slots].view(cache.dtype) if scale is not None else x[slots]
    x = x.float()
    return x if scale is None else x * scale[:, None]


def _attend(q, k, v, visible, scale):
    """q [B, T, Hq, d], k/v [B, n, Hkv, d] fp32, visible [B or 1, T, n] -> o in bf16, lse [B, Hq, T]."""
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    q = q.float().view(B, T, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)      # [B, Hkv, G, T, d]
    s = (q @ k.permute(0, 2, 3, 1).unsqueeze(2)) * scale                    # [B, Hkv, G, T, n]
    s = s.masked_fill(~visible[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = (s - m).exp()
    z = p.sum(-1, keepdim=True)
    o = (p @ v.permute(0, 2, 1, 3).unsqueeze(2)) / z
    lse = (m + z.log()).squeeze(-1).reshape(B, Hq, T)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, d).to(torch.bfloat16), lse


def _seen(query_pos, key_pos, window, sinks):
    """Whether the query at a position sees the key at another: the last `window` positions up to its
    own, and the first `sinks`."""
    return (key_pos <= query_pos) & ((key_pos > query_pos - window) | (key_pos < sinks))


def _plain_rope(s):
    c = s["c"]
    B, T = c["B"], c["T"]
    pos = s["lens"].long()[:, None] + torch.arange(T, device="cuda")
    q, k = (_norm_rotate(s[n], s[n + "w"], s["rope"], pos, s["eps"], c["rot"], c["interleaved"]) for n in "qk")
    q = q.to(torch.bfloat16)
    if c["cache"] == "dense":
        return q, k.to(torch.bfloat16)
    slots = _slots(s, pos).reshape(-1)
    k, v = k.flatten(0, 1), s["v"].flatten(0, 1)
    if c["cache"] == "fp8":
        k = (k / s["ks"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        v = (v.float() / s["vs"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["kc"].view(torch.uint8).view(-1, c["Hkv"], c["d"])[slots] = k.view(torch.uint8)
        s["vc"].view(torch.uint8).view(-1, c["Hkv"], c["d"])[slots] = v.view(torch.uint8)
    else:
        s["kc"].view(-1, c["Hkv"], c["d"])[slots] = k.to(torch.bfloat16)
        s["vc"].view(-1, c["Hkv"], c["d"])[slots] = v
    return q, s["kc"], s["vc"]


def _plain_window_decode(s):
    """Only the sinks and the last window + T - 1 positions of each sequence are gathered."""
    c = s["c"]
    T, window, sinks = c["T"], c["window"], c["sinks"]
    L = s["lens"].long()[:, None]
    n_win = min(window + T - 1, s["max_len"])
    first = torch.arange(min(sinks, s["max_len"]), device="cuda").expand(c["B"], -1)
    last = L - n_win + torch.arange(n_win, device="cuda")
    last = torch.where(last >= sinks, last, -1)          # positions already among the sinks, or before 0
    key_pos = torch.cat([torch.where(first < L, first, -1), last], dim=1)
    slots = _slots(s, key_pos.clamp(min=0))
    query_pos = L - T + torch.arange(T, device="cuda")
    visible = _seen(query_pos[:, :, None], key_pos[:, None], window, sinks) & (key_pos[:, None] >= 0)
    return _attend(s["q"], _rows(s["kc"], s["ks"], slots), _rows(s["vc"], s["vs"], slots), visible, s["scale"])


def _plain_window_prefill(s):
    c = s["c"]
    pos = torch.arange(c["N"], device="cuda")
    visible = _seen(pos[:, None], pos[None], c["window"], c["sinks"])[None]
    return _attend(s["q"], s["k"].float(), s["v"].float(), visible, s["scale"])


def _plain_window_chunk(s):
    c = s["c"]
    L = s["lens"].long()[:, None]
    key_pos = torch.arange(s["max_len"], device="cuda").expand(c["B"], -1)
    slots = _slots(s, torch.minimum(key_pos, L - 1))
    query_pos = L - c["T"] + torch.arange(c["T"], device="cuda")
    visible = _seen(query_pos[:, :, None], key_pos[:, None], c["window"], c["sinks"])
    return _attend(s["q"], _rows(s["kc"], s["ks"], slots), _rows(s["vc"], s["vs"], slots), visible, s["scale"])


def _plain_shared(s):
    """The prefix's rows are gathered once and meet the queries of every sequence; each sequence's own
    rows meet its queries; one softmax over both."""
    c = s["c"]
    B, T, Hq, Hkv, d, P = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"], c["prefix"]
    L = s["lens"].long()[:, None]
    n = s["max_len"] - P
    pos = torch.arange(P, device="cuda")
    pre = s["table"][0].long()[pos // PAGE] * PAGE + pos % PAGE
    kp, vp = _rows(s["kc"], s["ks"], pre), _rows(s["vc"], s["vs"], pre)                 # [P, Hkv, d]
    key_pos = P + torch.arange(n, device="cuda").expand(B, -1)
    slots = _slots(s, torch.minimum(key_pos, L - 1))
    ko, vo = _rows(s["kc"], s["ks"], slots), _rows(s["vc"], s["vs"], slots)             # [B, n, Hkv, d]
    query_pos = L - T + torch.arange(T, device="cuda")
    visible = key_pos[:, None] <= query_pos[:, :, None]                                 # [B, T, n]
    q = s["q"].float().view(B, T, Hkv, Hq // Hkv, d)
    sp = torch.einsum("btghd,pgd->bghtp", q, kp) * s["scale"]
    so = torch.einsum("btghd,bngd->bghtn", q, ko) * s["scale"]
    so = so.masked_fill(~visible[:, None, None], -math.inf)
    m = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    pp, po = (sp - m).exp(), (so - m).exp()
    z = pp.sum(-1, keepdim=True) + po.sum(-1, keepdim=True)
    o = (torch.einsum("bghtp,pgd->bghtd", pp, vp) + torch.einsum("bghtn,bngd->bghtd", po, vo)) / z
    lse = (m + z.log()).squeeze(-1).reshape(B, Hq, T)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, d).to(torch.bfloat16), lse


# ------------------------------------------------------------------ the framework's calls
def _own_rope(s):
    kv, c = _framework(), s["c"]
    if c["cache"] == "dense":
        kv.qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["rope"], q_weight=s["qw"], k_weight=s["kw"],
                        eps=s["eps"], interleaved=c["interleaved"], pos0=s["lens"])
        return s["q_out"], s["k_out"]
    if c["cache"] == "fp8":
        kv.kv_append_norm_rope_fp8(s["kc"], s["vc"], s["q"], s["k"], s["v"], s["q_out"], s["ks"], s["vs"], s["rope"],
                                   s["lens"], page_table=s["table"], q_weight=s["qw"], k_weight=s["kw"],
                                   eps=s["eps"], interleaved=c["interleaved"])
    else:
        kv.kv_append_norm_rope(s["kc"], s["vc"], s["q"], s["k"], s["v"], s["q_out"], s["rope"], s["lens"],
                               page_table=s["table"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"],
                               interleaved=c["interleaved"])
    return s["q_out"], s["kc"], s["vc"]


def _own_window_decode(s):
    kv, c = _framework(), s["c"]
    if "ws" not in s:
        s["ws"] = kv.decode_window_workspace(c["B"], c["T"], c["Hq"], c["Hkv"], c["d"], s["max_len"], c["window"],
                                             c["sinks"])
    more = dict(lse=s["lse"], page_table=s["table"], max_seqlen_k=s["max_len"], workspace=s["ws"])
    if c["cache"] == "fp8":
        kv.attn_decode_window_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["lens"], s["o"], c["window"],
                                  c["sinks"], **more)
    else:
        kv.attn_decode_window(s["q"], s["kc"], s["vc"], s["lens"], s["o"], c["window"], c["sinks"], **more)
    return s["o"], s["lse"]


def _own_window_prefill(s):
    kv, c = _framework(), s["c"]
    kv.attn_prefill_window(s["q"], s["k"], s["v"], s["o"], c["window"], c["sinks"], lse=s["lse"])
    return s["o"], s["lse"]


def _own_window_chunk(s):
    kv, c = _framework(), s["c"]
    kv.attn_prefill_cache_window(s["q"], s["kc"], s["vc"], s["lens"], s["o"], c["window"], c["sinks"], lse=s["lse"],
                                 page_table=s["table"])
    return s["o"], s["lse"]


def _own_shared(s):
    kv, c = _framework(), s["c"]
    n = c["prefix"] // PAGE
    if "ws" not in s:
        s["ws"] = kv.decode_shared_workspace(c["B"], c["T"], c["Hq"], c["Hkv"], c["d"], s["max_len"], n)
    more = dict(lse=s["lse"], max_seqlen_k=s["max_len"], workspace=s["ws"])
    prefix = s["table"][0, :n]
    if c["cache"] == "fp8":
        kv.attn_decode_shared_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["lens"], s["table"], prefix, s["o"],
                                  **more)
    else:
        kv.attn_decode_shared(s["q"], s["kc"], s["vc"], s["lens"], s["table"], prefix, s["o"], **more)
    return s["o"], s["lse"]


_PLAIN = {"rope": _plain_rope, "window_decode": _plain_window_decode, "window_prefill": _plain_window_prefill,
          "window_chunk": _plain_window_chunk, "shared": _plain_shared}
_OWN = {"rope": _own_rope, "window_decode": _own_window_decode, "window_prefill": _own_window_prefill,
        "window_chunk": _own_window_chunk, "shared": _own_shared}


def run(state):
    return (_OWN if own else _PLAIN)[state["c"]["op"]](state)


# ------------------------------------------------------------------ work
def _window_pairs(first, last, window, sinks):
    """(query, key) pairs of the queries at positions first .. last, and the keys any of them sees."""
    pairs = 0
    for p in range(first, last + 1):
        lo = max(0, p - window + 1)
        pairs += p + 1 - lo + min(sinks, lo)
    lo = max(0, first - window + 1)
    return pairs, last + 1 - lo + min(sinks, lo)


def work(case):
    c = case
    d, Hq, Hkv, B, op = c["d"], c["Hq"], c["Hkv"], c["B"], c["op"]
    if op == "window_prefill":
        pairs, _ = _window_pairs(0, c["N"] - 1, c["window"], c["sinks"])
        return {"bytes": B * c["N"] * (2 * (2 * Hq + 2 * Hkv) * d + 4 * Hq), "flops": 4 * d * Hq * B * pairs}
    T = c["T"]
    eb = 1 if c["cache"] == "fp8" else 2
    if op == "rope":
        dense = c["cache"] == "dense"
        read = 2 * (Hq + (1 if dense else 2) * Hkv) * d
        written = 2 * Hq * d + (2 * Hkv * d if dense else 2 * Hkv * d * eb)
        angles = 4 * c["rot"] * (min(B * T, c["hi"] + T))
        return {"bytes": B * T * (read + written) + angles + 4 * d + 4 * B, "flops": 7 * B * T * (Hq + Hkv) * d}
    lens = _lengths(c)
    io = B * T * Hq * (4 * d + 4) + 4 * B
    if op == "shared":
        keys = c["prefix"] + sum(lens)
        pairs = B * T * c["prefix"] + sum(T * L - T * (T - 1) // 2 for L in lens)
    else:
        both = [_window_pairs(L - T, L - 1, c["window"], c["sinks"]) for L in lens]
        pairs, keys = sum(p for p, _ in both), sum(k for _, k in both)
    pages = 0 if c["cache"] == "contig" else 4 * (keys // PAGE)
    return {"bytes": keys * Hkv * d * eb * 2 + io + pages, "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------ 64 bits
def _exact_rows(s, name, b, positions):
    """K or V rows of sequence b at a list of positions in 64 bits, [n, Hkv, d]."""
    cache, scale = s[name + "c"], s[name + "s"]
    p = torch.as_tensor(positions, device="cuda", dtype=torch.long)
    if s["table"] is None:
        x = cache[b].index_select(0, p)
    else:
        raw = cache.view(torch.uint8) if scale is not None else cache
        x = raw[s["table"][b].long()[torch.div(p, PAGE, rounding_mode="floor")], torch.remainder(p, PAGE)]
        x = x.view(cache.dtype)
    x = x.to(torch.float64)
    return x if scale is None else x * scale.to(torch.float64).reshape(-1, 1)


def _exact_heads(q, k, v, hidden, scale):
    """q [T, Hq, d], k/v [n, Hkv, d], hidden [T, n]; one query head at a time."""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    o = torch.empty(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(Hq, T, dtype=torch.float64, device="cuda")
    for h in range(Hq):
        x = scale * torch.mm(q[:, h].double(), k[:, h // G].T)
        x[hidden] = -math.inf
        lse[h] = torch.logsumexp(x, 1)
        o[:, h] = torch.mm(torch.exp(x - lse[h][:, None]), v[:, h // G])
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    op, B, d = c["op"], c["B"], c["d"]
    if op == "rope":
        T, rot = c["T"], c["rot"]
        half = rot // 2
        first = [2 * i if c["interleaved"] else i for i in range(half)]
        second = [2 * i + 1 if c["interleaved"] else i + half for i in range(half)]
        freq = torch.tensor([10000.0 ** (-2 * i / rot) for i in range(half)], dtype=torch.float64, device="cuda")
        pos = s["lens"].double().reshape(B, 1) + torch.arange(T, device="cuda").double()
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[:, :, None, None] * freq)
        out = []
        for n in "qk":
            x = s[n].double()
            x = x / (x.pow(2).sum(-1, keepdim=True) / d + s["eps"]).sqrt() * s[n + "w"].double()
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            out.append(x)
        if c["cache"] == "dense":
            return tuple(out)
        caches = []
        for new, name in ((out[1], "k"), (s["v"].double(), "v")):
            cache = s[name + "c"].double()
            if c["cache"] == "fp8":
                # the stored codes stand for these values before their rounding to 8 bits
                new = (new / s[name + "s"].double().reshape(-1, 1)).clamp(-448, 448)
            for b in range(B):
                p = torch.arange(T, device="cuda") + int(s["lens"][b])
                if s["table"] is None:
                    cache[b, p] = new[b]
                else:
                    cache[s["table"][b].long()[p // PAGE], p % PAGE] = new[b]
            caches.append(cache)
        return (out[0], *caches)
    os, lses = [], []
    for b in range(B):
        if op == "window_prefill":
            L = T = c["N"]
            keys = list(range(L))
            k, v = s["k"][b].double(), s["v"][b].double()
        else:
            L, T = int(s["lens"][b]), c["T"]
            keys = list(range(L))
            if op == "window_decode":
                start = max(c["sinks"], L - T - c["window"] + 1)
                keys = keys[:c["sinks"]] + keys[start:]
            k, v = _exact_rows(s, "k", b, keys), _exact_rows(s, "v", b, keys)
        j = torch.as_tensor(keys, device="cuda")
        i = torch.arange(L - T, L, device="cuda")[:, None]
        hidden = j > i
        if op != "shared":
            hidden = hidden | ((i - j >= c["window"]) & (j >= c["sinks"]))
        o, lse = _exact_heads(s["q"][b], k, v, hidden, s["scale"])
        os.append(o)
        lses.append(lse)
    return torch.stack(os), torch.stack(lses)
