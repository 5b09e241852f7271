"""GPU tests of spa_token_logprobs against log-softmax in 64 bits.

Tolerance.  S = sum e^(x-m) is a sum of positive fp32 terms: V / 256 of them
one after the other in a thread at most, then a tree, each addition 2^-24; a
term is e^(x-m) with x - m rounded (2^-24 |x-m|), its product with log2 e
rounded, and the exponential's own 2^-22.  A term's weight falls as e^-|x-m|,
so |x-m| e^-|x-m| <= 0.37 bounds what the roundings of its argument add.
Relative error of S: rs = (V / 256 + 40) 2^-24 + 2^-21.  log p = (x-m) - log S:
rs + 2^-24 (|x-m| + 2 |log S| + |log p|) + logf's 2^-23 |log S|.  The entropy's
T / S has the relative error 2 rs more."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("adaptive_hidden_state_b200.spa")


@pytest.fixture(scope="module")
def ws():
    return spa.Workspace(spa.LayerDesc(d=256, n_heads=2, head_dim=128, ffn=128, r=1, dtype=spa.SPA_BF16,
                                       rms_eps=1e-5, rope_theta=1e4), 1, 16)


def call(ws, x, tok, top, stream=None):
    rows = x.shape[0]
    lp, ent = (torch.full((rows,), 9.0, device="cuda") for _ in range(2))
    tid = torch.full((rows, top), -9, dtype=torch.int32, device="cuda") if top else None
    tlp = torch.full((rows, top), 9.0, device="cuda") if top else None
    spa.spa_token_logprobs(ws, x, tok, lp, ent, tid, tlp, stream=stream)
    return lp, ent, tid, tlp


def check(ws, x, tok, top):
    got = call(ws, x, tok, top)
    ws.check()
    lp, ent = (t.double().cpu().numpy() for t in got[:2])
    x64 = x.double().cpu().numpy()
    tok = tok.cpu().numpy()
    rows, V = x64.shape
    rs = (V / 256 + 40) * 2.0 ** -24 + 2.0 ** -21
    for r in range(rows):
        row = x64[r]
        m = row.max()
        if m == -np.inf:
            assert lp[r] == -np.inf and ent[r] == 0
            if top:
                assert np.all(got[2][r].cpu().numpy() == -1) and np.all(got[3][r].cpu().numpy() == -np.inf)
            continue
        with np.errstate(over="ignore"):
            d = row - m
            e = np.exp(d)
        S = e.sum()
        T = (e * np.where(e > 0, d, 0.0)).sum()
        logS = np.log(S)

        def tol(v, dv):
            return rs + 2.0 ** -24 * (abs(dv) + 4 * logS + abs(v)) + 1e-12

        ref = d[tok[r]] - logS
        if ref < -3.4e38:
            assert lp[r] < -3.3e38
        else:
            assert abs(lp[r] - ref) <= tol(ref, d[tok[r]]), (r, lp[r], ref)
        h = logS - T / S
        assert abs(ent[r] - h) <= 2 * rs + 2 * rs * abs(T / S) + 2.0 ** -22 * (logS + abs(h)) + 1e-12, (r, ent[r], h)
        if top:
            order = np.lexsort((np.arange(V), -row))[:top]
            order = order[row[order] > -np.inf]
            tid, tlp = got[2][r].cpu().numpy(), got[3][r].double().cpu().numpy()
            n = len(order)
            assert np.array_equal(tid[:n], order), r
            assert np.all(tid[n:] == -1) and np.all(tlp[n:] == -np.inf)
            for i in range(n):
                ref = d[order[i]] - logS
                if ref > -3.4e38:
                    assert abs(tlp[i] - ref) <= tol(ref, d[order[i]])
    return got


def logits(rng, rows, V, dtype, pad=0, mask=0.0, scale=3.0):
    x = torch.from_numpy((scale * rng.standard_normal((rows, V + pad))).astype(np.float32))
    if mask:
        x[torch.from_numpy(rng.random((rows, V + pad)) < mask)] = -float("inf")
    return x.to(dtype).cuda()[:, :V], torch.from_numpy(rng.integers(0, V, rows).astype(np.int32)).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,V,pad,top,mask", [
    (1, 1, 0, 1, 0.0), (3, 2, 1, 4, 0.0), (2, 7, 0, 7, 0.5), (5, 31, 2, 3, 0.0), (4, 255, 1, 32, 0.3),
    (3, 1003, 5, 8, 0.0), (7, 4097, 3, 1, 0.9), (2, 16385, 7, 20, 0.2), (9, 32003, 1, 32, 0.0), (2, 126464, 0, 8, 0.0),
    (700, 515, 1, 2, 0.1), (3, 70001, 0, 0, 0.3)])
def test_against_64_bits(ws, dtype, rows, V, pad, top, mask):
    rng = np.random.default_rng(V + rows)
    x, tok = logits(rng, rows, V, dtype, pad, mask)
    check(ws, x, tok, top)


@pytest.mark.parametrize("offset", [1, 2, 3, 5, 7])
def test_rows_that_start_anywhere(ws, offset):
    """Row starts at every alignment of an element, the row stride odd."""
    rng = np.random.default_rng(offset)
    for dtype in (torch.float32, torch.bfloat16):
        base = torch.from_numpy(rng.standard_normal(6 * 1013 + 16).astype(np.float32)).to(dtype).cuda()
        x = base[offset:offset + 6 * 1013].view(6, 1013)[:, :1009]
        check(ws, x, torch.arange(6, dtype=torch.int32, device="cuda"), 5)
        few = base[offset:offset + 6].view(3, 2)[:, :1]     # rows shorter than their way to an aligned address
        check(ws, few, torch.zeros(3, dtype=torch.int32, device="cuda"), 2)


def test_order_and_ties(ws):
    V = 20011
    rng = np.random.default_rng(1)
    up = torch.arange(V, dtype=torch.float32, device="cuda") / 500      # every element a new best
    rows = torch.stack([up, -up, torch.zeros_like(up), torch.full_like(up, -3e38),
                        torch.from_numpy(rng.integers(0, 3, V).astype(np.float32)).cuda(),
                        torch.from_numpy((rng.random(V) < 1e-3).astype(np.float32)).cuda()])
    for x in (rows, rows.to(torch.bfloat16)):
        for top in (1, 13, 32):
            check(ws, x, torch.full((6,), V - 1, dtype=torch.int32, device="cuda"), top)


def test_masked_rows_and_sharp_rows(ws):
    V, inf = 5000, float("inf")
    x = torch.full((7, V), -inf)
    x[1, 17] = 2.5                        # one token left
    x[2, 4999] = torch.finfo(torch.float32).min            # the lowest value, and nothing else
    x[3] = torch.finfo(torch.float32).min                  # lowest value everywhere
    x[4] = -3.0e38
    x[4, 3] = 3.0e38                      # a difference past the type's range
    x[5] = 0.0
    x[5, 100] = 80.0                      # one sure token
    x[6, ::2] = torch.linspace(-100, 100, 2500)
    tok = torch.tensor([4, 17, 4999, 0, 3, 100, 1], dtype=torch.int32, device="cuda")
    check(ws, x.cuda(), tok, 5)


def test_nan_and_infinity_make_the_row_nan(ws):
    rng = np.random.default_rng(2)
    for bad in (float("nan"), float("inf")):
        for at in (0, 1, 777, 4999):
            x, tok = logits(rng, 3, 5000, torch.float32)
            clean = call(ws, x, tok, 3)
            y = x.clone()
            y[1, at] = bad
            got = call(ws, y, tok, 3)
            assert torch.isnan(got[0][1]) and torch.isnan(got[1][1]) and torch.isnan(got[3][1]).all()
            for g, c in zip(got, clean):
                assert torch.equal(g[[0, 2]], c[[0, 2]])
    x = torch.full((1, 4000), float("nan"), device="cuda")
    got = call(ws, x, torch.zeros(1, dtype=torch.int32, device="cuda"), 2)
    assert torch.isnan(got[0]).all() and torch.isnan(got[1]).all()


def test_token_outside_is_reported(ws):
    rng = np.random.default_rng(3)
    x, _ = logits(rng, 4, 300, torch.bfloat16)
    tok = torch.tensor([0, -1, 300, 299], dtype=torch.int32, device="cuda")
    lp, ent, _, _ = call(ws, x, tok, 0)
    assert ws.status() == -7 and ws.status() == 0
    assert torch.isnan(lp).tolist() == [False, True, True, False] and not torch.isnan(ent).any()


def test_repeats_streams_and_graphs(ws):
    rng = np.random.default_rng(4)
    x, tok = logits(rng, 5, 40000, torch.bfloat16, scale=0.5)   # many equal values
    want = call(ws, x, tok, 32)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(call(ws, x, tok, 32), want))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    lp, ent = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    tid, tlp = torch.empty((5, 32), dtype=torch.int32, device="cuda"), torch.empty((5, 32), device="cuda")
    spa.spa_token_logprobs(ws, x, tok, lp, ent, tid, tlp, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((lp, ent, tid, tlp), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        spa.spa_token_logprobs(ws, x, tok, lp, ent, tid, tlp)
    x.copy_(x.flip(0).clone())
    tok.copy_(tok.flip(0).clone())
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b.flip(0)) for a, b in zip((lp, ent, tid, tlp), want))
    ws.check()
