"""What is measured of the 8-bit key/value cache (written, read back, attended)
and of the token log probabilities: the cases, their inputs, their plain forms
in torch, their 64-bit definitions and the work each cannot do without.

A cache holds codes [B, N, kv heads * head size] (int8 in -127..127, or e4m3)
and one scale per block of tokens and head [B, blocks, kv heads], a power of
two (0 for a block of zeros).  Writing rows into a block gives the block the
smallest power of two s >= 2^-126 with max |v| <= qmax * s over its new and its
remaining rows, and every row the codes round(v / s), ties to even.
"""
import math

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # the fill that starts a decode: every row of a 32 x 128 layer's K and V is written, then read back
        dict(name="cache-fill-n1024-int8", op="cache", B=1, N=1024, kv=32, hd=128, k=1024, block=64,
             fmt="int8", dtype="bf16"),
        # one cached step of a batched decode: 16 % of the rows, scattered, into a cache already full
        dict(name="cache-step-b8-n2048-e4m3", op="cache", B=8, N=2048, kv=32, hd=128, k=328, block=64,
             fmt="e4m3", dtype="bf16"),
        # a small fp32 layer, where launches count; the last block is cut by N
        dict(name="cache-step-small-f32", op="cache", B=2, N=71, kv=4, hd=64, k=16, block=16,
             fmt="int8", dtype="f32"),
        # one cached layer step at 512 tokens, a quarter of the rows refreshed
        dict(name="attn-n512-k128-int8", op="attn", B=1, N=512, heads=32, kv=32, hd=128, k=128, block=64,
             fmt="int8", dtype="bf16", ragged=False),
        # the widest layer of a batched decode, 25 % of 2048 tokens: bound by the products
        dict(name="attn-b8-n2048-k512-e4m3", op="attn", B=8, N=2048, heads=32, kv=32, hd=128, k=512, block=64,
             fmt="e4m3", dtype="bf16", ragged=False),
        # a padded batch (an empty and a one-token sequence among them), shared heads, odd sizes
        dict(name="attn-ragged-b5-n1537-k61-int8", op="attn", B=5, N=1537, heads=16, kv=4, hd=64, k=61, block=32,
             fmt="int8", dtype="bf16", ragged=True),
        # one token at a time over long caches with shared heads: bound by the cache's bytes
        dict(name="attn-one-token-b4-n65536-int8", op="attn", B=4, N=65536, heads=32, kv=8, hd=128, k=1, block=128,
             fmt="int8", dtype="bf16", ragged=False),
        # the same on one short sequence, where latency counts; seven query heads to a kv head
        dict(name="attn-one-token-n1000-e4m3", op="attn", B=1, N=1000, heads=14, kv=2, hd=128, k=1, block=16,
             fmt="e4m3", dtype="bf16", ragged=False),
        # fp32 queries of a small layer
        dict(name="attn-f32-n256-k40-int8", op="attn", B=2, N=256, heads=4, kv=4, hd=64, k=40, block=64,
             fmt="int8", dtype="f32", ragged=False),
        # two tokens unmasked in a step: two rows of fp32 logits
        dict(name="logp-r2-v126464", op="logp", rows=2, V=126464, pad=0, top=8, dtype="f32", masked=False),
        # every still-masked position of a 1024-token sequence, for confidence- or entropy-based unmasking
        dict(name="logp-r768-v126464", op="logp", rows=768, V=126464, pad=0, top=4, dtype="f32", masked=False),
        # bf16 logits of an odd vocabulary in padded rows, part of it masked out, many equal values
        dict(name="logp-r130-v32003-bf16", op="logp", rows=130, V=32003, pad=5, top=20, dtype="bf16", masked=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "attn", "attn", "logp"])
    if op == "logp":
        V = _log_int(rng, 1000, 130000)
        rows = _log_int(rng, 1, min(1024, 97000000 // V))
        return dict(op=op, rows=rows, V=V, pad=rng.choice([0, 0, 1, 3, 61]), top=rng.choice([0, 1, 2, 5, 8, 20, 32]),
                    dtype=rng.choice(["f32", "bf16"]), masked=rng.random() < 0.5)
    fmt = rng.choice(["int8", "e4m3"])
    block = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "cache":
        hd = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8, 32])
        N = _log_int(rng, 17, 2048)
        k, B = _log_int(rng, 1, N), _log_int(rng, 1, 8)
        while B > 1 and B * (N + k) * kv * hd * ESIZE[dtype] > 8 * (2048 + 328) * 4096 * 2:
            B //= 2  # no more than the batched decode's step
        return dict(op=op, B=B, N=N, kv=kv, hd=hd, k=k, block=block, fmt=fmt, dtype=dtype)
    if dtype == "f32":
        hd, kv, group = 64, rng.choice([1, 2, 4]), rng.choice([1, 2, 4])
        N = _log_int(rng, 1, 1024)
        k = _log_int(rng, 1, 128)
        B = _log_int(rng, 1, 4)
    else:
        hd = rng.choice([64, 128])
        kv, group = rng.choice([(1, 8), (2, 7), (4, 4), (8, 4), (32, 1), (16, 1), (4, 2)])
        if rng.random() < 0.5:
            N, k, B = _log_int(rng, 1, 2048), _log_int(rng, 1, 512), _log_int(rng, 1, 8)
        else:
            N, k, B = _log_int(rng, 1000, 65536), _log_int(rng, 1, 4), _log_int(rng, 1, 4)
        while kv * group * hd % 256:  # a layer's width is a multiple of 256 in bf16
            group *= 2
        N = min(N, 4 * 65536 * 8 * 128 // (B * kv * hd))  # no more than the long caches
    return dict(op=op, B=B, N=N, heads=kv * group, kv=kv, hd=hd, k=k, block=block, fmt=fmt, dtype=dtype,
                ragged=rng.random() < 0.4)


def _lens(case):
    """Tokens of each sequence: all N, or a padded batch with a full, an empty and a one-token sequence in it."""
    B, N = case["B"], case["N"]
    if not case["ragged"]:
        return [N] * B
    return [[N, 0, 1, (2 * N) // 3, max(1, N - 1)][b % 5] for b in range(B)]


# ------------------------------------------------------------------ inputs

def _pow2_scale(A, qmax):
    """Smallest power of two s >= 2^-126 with A <= qmax * s, 0 where A is 0 (A float32, exact)."""
    m, e = torch.frexp(A)
    mq, eq = math.frexp(qmax)
    t = e - eq + (m > mq).to(e.dtype)
    s = torch.ldexp(torch.ones_like(A), t.clamp(min=-126))
    return torch.where(A > 0, s, torch.zeros_like(s))


def _blocks(N, block):
    return (N + block - 1) // block


def _per_row(scale, N, block):
    return scale.repeat_interleave(block, dim=1)[:, :N]


def _quantise(v, block, fmt):
    """Codes and scales of values v [B, N, kv, hd] (float32), every block anew."""
    B, N, kv, hd = v.shape
    nb = _blocks(N, block)
    a = v.abs().amax(-1)
    a = torch.nn.functional.pad(a, (0, 0, 0, nb * block - N)).view(B, nb, block, kv).amax(2)
    s = _pow2_scale(a, QMAX[fmt])
    sr = _per_row(s, N, block)[..., None]
    y = torch.where(sr > 0, v / torch.where(sr > 0, sr, torch.ones_like(sr)), torch.zeros_like(v))
    codes = torch.round(y).to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)
    return codes, s


def _values(g, B, N, kv, hd, dtype, spread):
    """Keys or values as a layer makes them: a few wide channels, tokens of different sizes."""
    chan = torch.exp(0.5 * torch.randn((1, 1, kv, hd), generator=g, device="cuda"))
    tok = torch.exp(spread * torch.randn((B, N, 1, 1), generator=g, device="cuda"))
    return (torch.randn((B, N, kv, hd), generator=g, device="cuda") * chan * tok).to(DTYPE[dtype])


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "logp":
        rows, V, ld = case["rows"], case["V"], case["V"] + case["pad"]
        x = torch.randn((rows, ld), generator=g, device="cuda")
        # from flat rows to rows in which one token has nearly all of the probability
        x *= 0.5 + 4.0 * torch.rand((rows, 1), generator=g, device="cuda")
        if case["masked"]:
            x[torch.rand((rows, ld), generator=g, device="cuda") < 0.3] = -math.inf
        tok = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
        best = x[:, :V].argmax(-1).to(torch.int32)
        tok = torch.where(torch.rand((rows,), generator=g, device="cuda") < 0.5, best, tok)
        return {"logits": x.to(DTYPE[case["dtype"]])[:, :V], "tok": tok}
    B, N, kv, hd, k, block, fmt = (case[n] for n in ("B", "N", "kv", "hd", "k", "block", "fmt"))
    kc, ks = _quantise(_values(g, B, N, kv, hd, case["dtype"], 0.3).float(), block, fmt)
    vc, vs = _quantise(_values(g, B, N, kv, hd, case["dtype"], 0.5).float(), block, fmt)
    st = {"kc": kc, "ks": ks, "vc": vc, "vs": vs}
    if case["op"] == "cache":
        # the rows of a step: which, and their new keys and values
        st["idx"] = torch.rand((B, N), generator=g, device="cuda").argsort(-1)[:, :k].sort(-1)[0].to(torch.int32)
        st["k_rows"] = _values(g, B, k, kv, hd, case["dtype"], 0.4)
        st["v_rows"] = _values(g, B, k, kv, hd, case["dtype"], 0.6)
    else:
        q = torch.randn((B, k, case["heads"], hd), generator=g, device="cuda")
        q *= torch.exp(0.7 * torch.randn((B, k, case["heads"], 1), generator=g, device="cuda"))
        st["q"] = q.to(DTYPE[case["dtype"]])
        st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        from adaptive_hidden_state_b200 import spa
        dt = spa.SPA_BF16 if case["dtype"] == "bf16" else spa.SPA_F32
        if case["op"] == "logp":
            heads, hd, B, N = 2, 128, 1, 1
        else:
            hd, B, N = case["hd"], case["B"], min(case["N"], 8192)
            heads = case.get("heads", case["kv"])
            while dt == spa.SPA_BF16 and heads * hd % 256:
                heads *= 2
        desc = spa.LayerDesc(d=heads * hd, n_heads=heads, head_dim=hd, ffn=128, r=1, dtype=dt, rms_eps=1e-5,
                             rope_theta=1e4)
        st["spa"], st["ws"] = spa, spa.Workspace(desc, B, N)
        if case["op"] == "logp":
            rows, top = case["rows"], case["top"]
            st["out"] = [torch.empty((rows,), device="cuda"), torch.empty((rows,), device="cuda"),
                         torch.empty((rows, top), dtype=torch.int32, device="cuda"),
                         torch.empty((rows, top), device="cuda")]
        else:
            N, kv = case["N"], case["kv"]
            c = spa.Q8Cache(B, N, kv, hd, block=case["block"],
                            fmt=spa.SPA_Q8_INT8 if case["fmt"] == "int8" else spa.SPA_Q8_E4M3)
            c.k.copy_(st.pop("kc").view(B, N, kv * hd))
            c.v.copy_(st.pop("vc").view(B, N, kv * hd))
            c.k_scale.copy_(st.pop("ks"))
            c.v_scale.copy_(st.pop("vs"))
            st["cache"] = c
            if case["op"] == "cache":
                st["out"] = [torch.empty((B, N, kv, hd), dtype=DTYPE[case["dtype"]], device="cuda") for _ in range(2)]
            else:
                st["out"] = torch.empty_like(st["q"])
    return st


# ------------------------------------------------------------------ one pass

def _write_plain(codes, scale, rows, idx, block, fmt):
    """Rows idx of a cache written in place; the whole cache's values afterwards (float32)."""
    B, N, kv, hd = codes.shape
    nb = _blocks(N, block)
    v = codes.float() * _per_row(scale, N, block)[..., None]
    v.scatter_(1, idx.long()[:, :, None, None].expand(-1, -1, kv, hd), rows.float())
    c2, s2 = _quantise(v, block, fmt)
    hit = torch.zeros((B, nb), dtype=torch.bool, device=v.device)
    hit.scatter_(1, idx.long() // block, True)
    scale.copy_(torch.where(hit[:, :, None], s2, scale))
    hr = hit.repeat_interleave(block, dim=1)[:, :N, None, None]
    codes.view(torch.uint8).copy_(torch.where(hr, c2.view(torch.uint8), codes.view(torch.uint8)))
    return codes.float() * _per_row(scale, N, block)[..., None]


def _attention_plain(q, kc, ks, vc, vs, lens, block):
    B, k, heads, hd = q.shape
    N, kv = kc.shape[1], kc.shape[2]
    K = (kc.float() * _per_row(ks, N, block)[..., None]).permute(0, 2, 1, 3)
    V = (vc.float() * _per_row(vs, N, block)[..., None]).permute(0, 2, 1, 3)
    x = q.float().view(B, k, kv, heads // kv, hd).permute(0, 2, 1, 3, 4).reshape(B, kv, -1, hd)
    s = torch.matmul(x, K.transpose(-1, -2)) / math.sqrt(hd)
    keep = torch.arange(N, device=q.device)[None] < lens[:, None]
    s = s.masked_fill(~keep[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, V) / torch.where(l > 0, l, torch.ones_like(l))
    return o.view(B, kv, k, heads // kv, hd).permute(0, 2, 1, 3, 4).reshape(B, k, heads, hd).to(q.dtype)


def _logp_plain(logits, tok, top):
    x = logits.float()
    m = x.amax(-1, keepdim=True)
    t = x - m
    e = torch.exp(t)
    S = e.sum(-1, keepdim=True)
    logS = torch.log(S)
    logp = (t - logS).gather(1, tok.long()[:, None])[:, 0]
    entropy = (logS - torch.where(e > 0, e * t, torch.zeros_like(e)).sum(-1, keepdim=True) / S)[:, 0]
    v, i = torch.sort(x, dim=-1, descending=True, stable=True)
    v, i = v[:, :top], i[:, :top]
    gone = v == -math.inf
    return [logp, entropy, torch.where(gone, -1, i).to(torch.int32), (v - m) - logS]


def run(st):
    case = st["case"]
    if own:
        spa = st["spa"]
        if case["op"] == "cache":
            spa.spa_q8_write(st["ws"], st["cache"], st["k_rows"], st["v_rows"], idx=st["idx"])
            spa.spa_q8_read(st["ws"], st["cache"], st["out"][0], st["out"][1])
        elif case["op"] == "attn":
            spa.spa_q8_attention(st["ws"], st["q"], st["cache"], st["out"],
                                 lens=st["lens"] if case["ragged"] else None)
        else:
            spa.spa_token_logprobs(st["ws"], st["logits"], st["tok"], *st["out"])
        return st["out"]
    if case["op"] == "cache":
        dt = DTYPE[case["dtype"]]
        return [_write_plain(st["kc"], st["ks"], st["k_rows"], st["idx"], case["block"], case["fmt"]).to(dt),
                _write_plain(st["vc"], st["vs"], st["v_rows"], st["idx"], case["block"], case["fmt"]).to(dt)]
    if case["op"] == "attn":
        return _attention_plain(st["q"], st["kc"], st["ks"], st["vc"], st["vs"], st["lens"], case["block"])
    return _logp_plain(st["logits"], st["tok"], case["top"])


# ------------------------------------------------------------------ 64 bits

def _round_code(y, fmt):
    """y (float64, within the format's range) to the nearest value of the format, ties to even."""
    if fmt == "int8":
        return torch.round(y)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(y / step) * step


def _exact_cache(codes, scale, rows, idx, block, fmt):
    out = torch.empty(codes.shape, dtype=torch.float64, device=codes.device)
    for b in range(codes.shape[0]):
        for j in range(scale.shape[1]):
            r0, r1 = j * block, min((j + 1) * block, codes.shape[1])
            out[b, r0:r1] = codes[b, r0:r1].to(torch.float64) * scale[b, j].to(torch.float64)[None, :, None]
        new = out[b].clone()
        new[idx[b].long()] = rows[b].to(torch.float64)
        for j in torch.unique(idx[b].long() // block).tolist():
            v = new[j * block:(j + 1) * block]
            A = v.abs().amax((0, 2))
            t = torch.ceil(torch.log2(A / QMAX[fmt])).clamp(min=-126.0)
            t = torch.where(A > QMAX[fmt] * torch.exp2(t), t + 1.0, t)
            t = torch.where((t > -126.0) & (A <= QMAX[fmt] * torch.exp2(t - 1.0)), t - 1.0, t)
            s = torch.where(A > 0, torch.exp2(t), torch.ones_like(t))[None, :, None]
            out[b, j * block:(j + 1) * block] = _round_code(v / s, fmt) * s
    return out


def _exact_attention(st, case):
    B, k, heads, hd = st["q"].shape
    group, block = heads // case["kv"], case["block"]
    out = torch.zeros((B, k, heads, hd), dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        blk = torch.arange(n, device="cuda") // block
        for h in range(heads):
            kh = h // group
            K = st["kc"][b, :n, kh].to(torch.float64) * st["ks"][b, blk, kh].to(torch.float64)[:, None]
            V = st["vc"][b, :n, kh].to(torch.float64) * st["vs"][b, blk, kh].to(torch.float64)[:, None]
            a = torch.softmax(st["q"][b, :, h].to(torch.float64) @ K.T / hd ** 0.5, -1)
            out[b, :, h] = a @ V
    return out


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "cache":
        return [_exact_cache(st["kc"], st["ks"], st["k_rows"], st["idx"], case["block"], case["fmt"]),
                _exact_cache(st["vc"], st["vs"], st["v_rows"], st["idx"], case["block"], case["fmt"])]
    if case["op"] == "attn":
        return _exact_attention(st, case)
    rows, top = case["rows"], case["top"]
    logp = torch.empty((rows,), dtype=torch.float64, device="cuda")
    ent = torch.empty_like(logp)
    ids = torch.empty((rows, top), dtype=torch.int32, device="cuda")
    tlp = torch.empty((rows, top), dtype=torch.float64, device="cuda")
    for r in range(rows):
        x = st["logits"][r].to(torch.float64)
        lp = torch.log_softmax(x, -1)
        logp[r] = lp[st["tok"][r].long()]
        ent[r] = -torch.xlogy(lp.exp(), lp.exp()).sum()
        order = torch.argsort(-x, stable=True)[:top]
        ids[r] = torch.where(x[order] == -math.inf, torch.full_like(order, -1), order).to(torch.int32)
        tlp[r] = lp[order]
    return [logp, ent, ids, tlp]


# ------------------------------------------------------------------ work

def work(case):
    es = ESIZE[case["dtype"]]
    if case["op"] == "logp":
        rows, V, top = case["rows"], case["V"], case["top"]
        # per logit: subtract, exponential, two sums, one product
        return {"bytes": rows * V * es + rows * (4 + 8) + rows * top * 8, "flops": 5 * rows * V}
    B, N, kv, hd, k = (case[n] for n in ("B", "N", "kv", "hd", "k"))
    scales = 2 * B * _blocks(N, case["block"]) * kv * 4
    if case["op"] == "cache":
        # rows and indices in, their codes out; the cache's codes in (the remaining rows set a block's scale),
        # every row out; one division or product an element
        rows, cells = 2 * B * k * kv * hd, 2 * B * N * kv * hd
        return {"bytes": rows * (es + 1) + B * k * 4 + cells * (1 + es) + 2 * scales, "flops": rows + cells}
    keys, d = sum(_lens(case)), case["heads"] * hd
    return {"bytes": 2 * B * k * d * es + 2 * keys * kv * hd + scales, "flops": 4 * keys * k * d}
