"""The attention operators against the fp64 oracle.

Tolerances, derived before the first run:
  * Stored codes and scales, ids, and everything read back: equal.
  * A rounding to type t is off by at most eps(t)/2 of the value (bf16 2^-8,
    fp16 2^-11, fp32 2^-24).
  * Queries after norm and rotation: fp32 leaves 2^-19 (|a cos| + |b sin|)
    (see the kernel), then one rounding to the output type.
  * Attention.  Scores are sums of D exact products in fp32: off by at most
    (D + 4) 2^-24 sum|q k| scale (the accumulation, the scaling and the
    subtraction of the maximum), called e; a weight is then off by a factor
    e^(2e), plus 2^-21 of the exponential, plus 2^-11 where it is rounded to
    fp16, plus an absolute 2^-25 of the largest weight there (fp16's smallest
    step; the largest weight is at least 2^-8 after lazy rescaling, so 2^-17
    of it); weighted sums over n keys in fp32 add n 2^-24.  All of these scale
    the softmax-weighted |v| (mag); the output's rounding comes on top.
"""
import numpy as np
import pytest
import torch

import block_quantized_moe_layer_gb300 as pkg
from oracle import attn as oa

pytestmark = pytest.mark.gpu

HEADS = [(64, 4, 192, 64), (32, 8, 128, 128), (16, 16, 64, 32), (6, 2, 256, 64), (5, 1, 64, 0), (3, 3, 128, 16)]


def _np(t):
    return t.detach().double().cpu().numpy()


def _norms(rng, D):
    return [torch.tensor(1 + 0.1 * rng.normal(size=D), dtype=torch.float32, device="cuda") for _ in range(2)]


def _slots(rng, n_pages, P, T):
    return torch.tensor(rng.permutation(n_pages * P)[:T].astype(np.int64), device="cuda")


def _append_check(rng, hq, hk, D, rot, T, P, in_dtype, act, norm=True, interleaved=False, far=100_000, positions=None,
                  x=None, skip=None):
    n_pages = -(-T // P) + 2
    qw, kw = _norms(rng, D) if norm else (None, None)
    at = pkg.Attention(hq, hk, D, P, n_pages, T, 1, far, act=act, rot_dim=rot, interleaved=interleaved, q_norm=qw, k_norm=kw)
    if x is None:
        x = rng.normal(size=(T, hq + 2 * hk, D)) * np.exp(rng.normal(size=(T, 1, 1)))
    x = torch.tensor(x, device="cuda").to(in_dtype)
    q, k, v = x.split([hq, hk, hk], 1)
    pos = rng.integers(0, far, T) if positions is None else np.asarray(positions)
    slots = _slots(rng, n_pages, P, T)
    if skip is not None:
        slots[skip] = -1
    pages = at.pages()
    pages.fill_(0xAB)
    before = pages.clone()
    p32 = torch.tensor(pos.astype(np.int32), device="cuda")
    out = at.append(q, k, v, p32, slots, pages)
    keys, values = at.read(slots, pages)
    at.status()
    f = oa.frequencies(rot)
    want = oa.prepared(_np(q), None if qw is None else _np(qw), pos, rot, f, interleaved)
    plain = oa.prepared(_np(q), None if qw is None else _np(qw), pos, 0, f)
    # |a cos| + |b sin| <= |a| + |b|
    m = np.abs(plain)
    if rot:
        i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        s = m[..., i] + m[..., j]
        m[..., i], m[..., j] = s, s
    tol = 2.0 ** -19 * m + np.abs(want) * (2.0 ** -8 if act == pkg.ACT_BF16 else 2.0 ** -24) * (1 + 2.0 ** -10)
    assert (np.abs(_np(out) - want) <= tol).all()
    kc, ks = oa.quantise(oa.prepared(_np(k), None if kw is None else _np(kw), pos, rot, f, interleaved))
    vc, vs = oa.quantise(_np(v))
    arrays = oa.page_arrays(pages.cpu().numpy(), hk, P, D)
    sl = slots.cpu().numpy()
    keep = sl >= 0
    for (codes, scales), (gc, gs) in (((kc, ks), arrays[:2]), ((vc, vs), arrays[2:])):
        got_c = oa.unpack(gc[sl[keep] // P, :, sl[keep] % P])
        got_s = gs[sl[keep] // P, :, sl[keep] % P]
        assert np.array_equal(got_s, scales[keep]), (got_s != scales[keep]).sum()
        assert np.array_equal(got_c, codes[keep]), (got_c != codes[keep]).sum()
    assert np.array_equal(_np(keys)[keep], oa.dequantise(kc, ks)[keep])
    assert np.array_equal(_np(values)[keep], oa.dequantise(vc, vs)[keep])
    assert (_np(keys)[~keep] == 0).all()
    # nothing else is touched
    untouched = np.ones((n_pages, P), bool)
    untouched[sl[keep] // P, sl[keep] % P] = False
    for g, b in zip(arrays, oa.page_arrays(before.cpu().numpy(), hk, P, D)):
        assert np.array_equal(g.transpose(0, 2, 1, 3)[untouched], b.transpose(0, 2, 1, 3)[untouched])
    at.close()


@pytest.mark.parametrize("hq,hk,D,rot", HEADS)
@pytest.mark.parametrize("T,P", [(1, 16), (4, 64), (67, 32), (300, 128)])
def test_append(hq, hk, D, rot, T, P):
    rng = np.random.default_rng(T * 1000 + D + hq)
    _append_check(rng, hq, hk, D, rot, T, P, torch.bfloat16, pkg.ACT_BF16)


@pytest.mark.parametrize("in_dtype,act", [(torch.float32, pkg.ACT_BF16), (torch.bfloat16, pkg.ACT_F32), (torch.float32, pkg.ACT_F32)])
@pytest.mark.parametrize("hq,hk,D,rot", HEADS[:4])
def test_append_types(hq, hk, D, rot, in_dtype, act):
    _append_check(np.random.default_rng(D), hq, hk, D, rot, 37, 32, in_dtype, act)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_pairs_and_no_norm(norm, interleaved):
    for hq, hk, D, rot in HEADS:
        _append_check(np.random.default_rng(D + rot), hq, hk, D, rot, 50, 64, torch.bfloat16, pkg.ACT_BF16, norm, interleaved)


def test_append_borders():
    """Rows full of values on and next to the borders of codes and scales, at position 0 and far out."""
    rng = np.random.default_rng(5)
    hq, hk, D, T = 4, 2, 128, 64
    x = rng.integers(-14, 15, (T, hq + 2 * hk, D)) / 2.0  # halves: exact ties once amax is 7
    x[:, :, ::16] = 7.0
    x[1::4] *= np.exp2(rng.integers(-20, 8, (T // 4, 1, 1)).astype(float))
    x[2::4] = np.where(rng.random((T // 4, hq + 2 * hk, D)) < 0.5, 0.0, x[2::4] * (1 + 2.0 ** -7))
    x[3::4] = 0
    for norm in (False, True):
        for pos in (np.zeros(T), np.full(T, 99_999), np.arange(T)):
            for t in (torch.bfloat16, torch.float32):
                _append_check(rng, hq, hk, D, 64, T, 16, t, pkg.ACT_BF16, norm, positions=pos.astype(np.int64), x=x)
    # fp32 neighbours of exact ties
    x = x * (1 + rng.integers(-1, 2, x.shape) * 2.0 ** -23)
    _append_check(rng, hq, hk, D, 64, T, 16, torch.float32, pkg.ACT_F32, False, positions=np.zeros(T, np.int64), x=x)


def test_append_many_rows_codes_are_exact():
    _append_check(np.random.default_rng(6), 8, 8, 128, 128, 4096, 64, torch.bfloat16, pkg.ACT_BF16)


def test_append_padding_strides_and_in_place():
    rng = np.random.default_rng(7)
    _append_check(rng, 8, 2, 64, 64, 33, 16, torch.bfloat16, pkg.ACT_BF16, skip=[0, 5, 32])
    # a fused projection with room after each token, head-major keys, and q_out = q
    hq, hk, D, T, P = 8, 2, 64, 19, 16
    at = pkg.Attention(hq, hk, D, P, 4, T, 1, 1000, rot_dim=64)
    big = torch.tensor(rng.normal(size=(T, (hq + hk) * D + 40)), device="cuda").to(torch.bfloat16)
    q = big[:, :hq * D].unflatten(1, (hq, D))
    v = big[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    k = torch.tensor(rng.normal(size=(hk, T, D)), device="cuda").to(torch.bfloat16).transpose(0, 1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = _slots(rng, 4, P, T)
    a, b = at.pages(), at.pages()
    one = at.append(q, k, v, pos, slots, a)
    qc = q.contiguous()
    two = at.append(qc, k.contiguous(), v.contiguous(), pos, slots, b, q_out=qc)
    assert two is qc and torch.equal(one, two) and torch.equal(a, b)


def test_append_special_values():
    hq, hk, D, P = 2, 1, 64, 16
    at = pkg.Attention(hq, hk, D, P, 2, 8, 1, 100, rot_dim=0)
    x = torch.randn(3, hq + 2 * hk, D, device="cuda").to(torch.bfloat16)
    x[0, 2:, 3] = float("inf")
    x[0, 2:, 4] = float("-inf")
    x[1, 2:, 5] = float("nan")
    x[2, 2:, :16] = 3.0e38
    slots = torch.tensor([0, 17, 31], device="cuda")
    pages = at.pages()
    at.append(x[:, :2], x[:, 2:3], x[:, 3:], torch.zeros(3, dtype=torch.int32, device="cuda"), slots, pages)
    keys, values = at.read(slots, pages)
    c, s = oa.quantise(_np(x[:, 2:3]))
    assert np.array_equal(_np(keys), oa.dequantise(c, s)) and np.array_equal(_np(values), oa.dequantise(*oa.quantise(_np(x[:, 3:]))))
    assert keys[0, 0, 3] == 7 * 896 and keys[0, 0, 4] == -8 * 896 and keys[1, 0, 5] == 0


# ---------------------------------------------------------------- attention


def _cache(rng, lens, hk, D, P, spare=3, wild=1.0):
    """Random pages: valid codes and scales everywhere, rows past a sequence's end full of the format's infinities."""
    tables = [-(-n // P) for n in lens]
    n_pages = sum(tables) + spare
    pages = np.full((n_pages, hk * P * D * 9 // 8), 0xFF, np.uint8)
    arrays = oa.page_arrays(pages, hk, P, D)
    order = rng.permutation(n_pages)
    width = max(max(tables), 1) + 2
    table = rng.integers(0, n_pages, (len(lens), width)).astype(np.int32)
    keys, values, used = [], [], 0
    for b, n in enumerate(lens):
        mine = order[used:used + tables[b]]
        used += tables[b]
        table[b, :tables[b]] = mine
        both = []
        for i in (0, 2):
            x = rng.normal(size=(n, hk, D)) * wild
            c, s = oa.quantise(x)
            j = np.arange(n)
            if n:
                arrays[i][mine[j // P], :, j % P] = oa.pack(c)
                arrays[i + 1][mine[j // P], :, j % P] = s
            both.append(oa.dequantise(c, s))
        keys.append(both[0])
        values.append(both[1])
    return torch.tensor(pages, device="cuda"), torch.tensor(table, device="cuda"), keys, values, n_pages


def _forward_check(rng, hq, hk, D, lens, news, P, act=None, window=0, scale=0.0, q_scale=1.5, wild=1.0, stream=None,
                   pad_q=0, extra=0):
    act = pkg.ACT_BF16 if act is None else act
    bf = act == pkg.ACT_BF16
    pages, table, keys, values, n_pages = _cache(rng, lens, hk, D, P, wild=wild)
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    T = int(starts[-1])
    max_len = max(max(lens), 1) + extra
    if max_len > table.shape[1] * P:
        table = torch.nn.functional.pad(table, (0, -(-max_len // P) - table.shape[1]))
    at = pkg.Attention(hq, hk, D, P, n_pages, T, len(lens), max_len, act=act, rot_dim=0, window=window, scale=scale)
    dt = torch.bfloat16 if bf else torch.float32
    big = torch.tensor(rng.normal(size=(T, hq, D + pad_q)) * q_scale, device="cuda").to(dt)
    q = big[..., :D]
    lse = torch.full((T, hq), 7.0, device="cuda")
    out = torch.full((T, hq, D), 7.0, dtype=dt, device="cuda")
    args = (q, pages, torch.tensor(starts, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda"), table,
            max(max(news), 1) + (extra > 0 and max(news) < T), max_len)
    at.forward(*args, out=out, lse=lse, stream=stream)
    torch.cuda.synchronize()
    at.status()
    again = at.forward(*args)
    torch.cuda.synchronize()
    assert torch.equal(out, again)  # the same bits, with and without lse
    got, got_lse, qn = _np(out), _np(lse), _np(q)
    sc = D ** -0.5 if scale == 0.0 else scale
    worst = 0.0
    for b, (n, t) in enumerate(zip(lens, news)):
        sl = slice(starts[b], starts[b + 1])
        want, wl, mag = oa.attention(qn[sl], keys[b], values[b], t, window, sc)
        if t == 0:
            continue
        if n == 0:
            assert (got[sl] == 0).all() and np.isneginf(got_lse[sl]).all()
            continue
        s_abs = sc * np.abs(qn[sl]).max() * np.abs(keys[b]).sum(-1).max()
        e = (D + 4) * 2.0 ** -24 * s_abs
        n_vis = min(n, window) if window else n
        rel = np.expm1(2 * e) + 2.0 ** -20 + n_vis * 2.0 ** -24
        tol = mag * (rel + (2.0 ** -11 if bf else 0)) + np.abs(want) * (2.0 ** -8 if bf else 2.0 ** -23)
        if bf:
            tol += n_vis * 2.0 ** -17 * 2.0 ** -8 * np.abs(values[b]).max()
        err = np.abs(got[sl] - want)
        assert np.isfinite(got[sl]).all()
        assert (err <= tol).all(), (b, float((err - tol).max()), float((err / tol.clip(1e-30)).max()))
        worst = max(worst, float((err / tol.clip(1e-30)).max()))
        seen = np.isfinite(wl)
        assert np.array_equal(np.isneginf(got_lse[sl]), ~seen)
        assert (np.abs(got_lse[sl][seen] - wl[seen]) <= rel + (2.0 ** -11 if bf else 0) + 2.0 ** -22 * (1 + np.abs(wl[seen]))).all()
    at.close()
    return worst


@pytest.mark.parametrize("act", [pkg.ACT_F32, pkg.ACT_BF16])
@pytest.mark.parametrize("hq,hk,D,rot", HEADS)
def test_forward_single_tokens(hq, hk, D, rot, act):
    rng = np.random.default_rng(D + hq)
    for lens, P in [([1], 16), ([2, 15, 16, 17], 16), ([257, 64, 63, 65, 1], 64), ([130, 0, 128, 127, 129], 128), ([1000], 32)]:
        _forward_check(rng, hq, hk, D, lens, [1] * len(lens), P, act)


@pytest.mark.parametrize("act", [pkg.ACT_F32, pkg.ACT_BF16])
@pytest.mark.parametrize("hq,hk,D,rot", HEADS)
def test_forward_verify_batches(hq, hk, D, rot, act):
    rng = np.random.default_rng(D + hq + 1)
    # ragged query counts; a sequence shorter than its queries leaves rows empty
    _forward_check(rng, hq, hk, D, [4, 300, 2, 129], [4, 3, 4, 8], 16, act)
    _forward_check(rng, hq, hk, D, [777, 5, 0], [4, 0, 2], 64, act)


@pytest.mark.parametrize("hq,hk,D,rot", HEADS)
@pytest.mark.parametrize("window", [1, 7, 128, 500])
def test_forward_window(hq, hk, D, rot, window):
    rng = np.random.default_rng(window)
    _forward_check(rng, hq, hk, D, [900, 3, 130], [4, 1, 6], 32, window=window)
    _forward_check(rng, hq, hk, D, [400, 700], [150, 300], 64, window=window)


@pytest.mark.parametrize("hq,hk,D,rot", HEADS)
def test_forward_prompts(hq, hk, D, rot):
    rng = np.random.default_rng(D + hq + 2)
    for lens, news, P in [([200], [200], 64), ([513], [300], 16), ([128, 300, 90], [128, 257, 33], 128), ([260, 1, 40], [129, 1, 40], 32)]:
        _forward_check(rng, hq, hk, D, lens, news, P)


@pytest.mark.parametrize("hq,hk,D,tokens", [(16, 16, 64, 192), (4, 1, 128, 64), (8, 1, 192, 32), (16, 1, 256, 16)])
def test_forward_around_the_row_limit(hq, hk, D, tokens):
    """The most rows of the verify kernel, and one token more."""
    rng = np.random.default_rng(D + tokens)
    for t in (tokens, tokens + 1):
        _forward_check(rng, hq, hk, D, [t + 40, t, 150], [t, t // 2, 1], 32)


def test_forward_long_and_split():
    rng = np.random.default_rng(11)
    _forward_check(rng, 16, 1, 192, [9001], [4], 64)
    _forward_check(rng, 4, 4, 128, [12345], [1], 16)
    _forward_check(rng, 8, 1, 64, [7000, 20], [40, 20], 32)


def test_forward_mixed_prompt_and_single_tokens():
    rng = np.random.default_rng(12)
    _forward_check(rng, 16, 2, 128, [500, 1, 77, 300], [200, 1, 1, 9], 64)


def test_forward_strides_scale_and_loose_bounds():
    rng = np.random.default_rng(13)
    _forward_check(rng, 8, 2, 64, [100, 33], [2, 2], 16, scale=0.3, pad_q=8)
    _forward_check(rng, 16, 1, 128, [300, 40], [30, 9], 16, scale=0.02, pad_q=24, extra=700)
    _forward_check(rng, 16, 1, 192, [300, 40], [3, 2], 64, extra=1500)


def test_forward_peaked_and_flat_scores():
    rng = np.random.default_rng(14)
    for news in ([1], [4], [150]):
        _forward_check(rng, 16, 2, 128, [600], news, 64, q_scale=30.0)  # one key takes nearly all
        _forward_check(rng, 16, 2, 128, [600], news, 64, q_scale=0.0)  # all the same
        _forward_check(rng, 16, 2, 192, [600], news, 64, wild=60.0, q_scale=0.02)  # large cached values


def test_forward_on_another_stream():
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        _forward_check(np.random.default_rng(15), 16, 2, 64, [300, 50], [4, 4], 16)
        _forward_check(np.random.default_rng(15), 16, 2, 64, [300, 250], [100, 4], 16)


def test_forward_rows_of_no_sequence_are_left_alone():
    rng = np.random.default_rng(16)
    pages, table, keys, values, n_pages = _cache(rng, [40, 60], 2, 64, 16)
    at = pkg.Attention(8, 2, 64, 16, n_pages, 10, 2, 64, rot_dim=0)
    q = torch.randn(10, 8, 64, device="cuda").to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 5.0)
    at.forward(q, pages, torch.tensor([2, 4, 7], **i32), torch.tensor([40, 60], **i32), table, 3, 60, out=out)
    at.status()
    assert (out[:2] == 5).all() and (out[7:] == 5).all()
    want, _, mag = oa.attention(_np(q[4:7]), keys[1], values[1], 3)
    assert (np.abs(_np(out[4:7]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag).all()


@pytest.mark.parametrize("D", [64, 192, 256])
@pytest.mark.parametrize("news", [1, 4, 40])
def test_forward_window_with_pages_given_back(D, news):
    """Table entries of pages wholly before every query's window are not looked at."""
    rng = np.random.default_rng(20)
    hq, hk, P, n, window = 16, 1, 16, 700, 100
    pages, table, keys, values, n_pages = _cache(rng, [n], hk, D, P)
    at = pkg.Attention(hq, hk, D, P, n_pages, news, 1, n, rot_dim=0, window=window)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn(news, hq, D, device="cuda").to(torch.bfloat16)
    args = (torch.tensor([0, news], **i32), torch.tensor([n], **i32))
    whole = at.forward(q, pages, *args, table, news, n)
    table[0, :(n - news - window + 1) // P] = -1
    assert torch.equal(at.forward(q, pages, *args, table, news, n), whole)
    at.status()


def test_forward_captured_in_a_graph_follows_its_inputs():
    rng = np.random.default_rng(17)
    pages, table, keys, values, n_pages = _cache(rng, [500, 300], 2, 128, 64)
    at = pkg.Attention(16, 2, 128, 64, n_pages, 8, 2, 512, rot_dim=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn(8, 16, 128, device="cuda").to(torch.bfloat16)
    starts, lens = torch.tensor([0, 4, 8], **i32), torch.tensor([500, 300], **i32)
    out = torch.empty_like(q)
    at.forward(q, pages, starts, lens, table, 4, 512, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        at.forward(q, pages, starts, lens, table, 4, 512, out=out)
    lens.copy_(torch.tensor([123, 64], **i32))
    q.copy_(torch.randn(8, 16, 128, device="cuda"))
    g.replay()
    got = out.clone()
    assert torch.equal(got, at.forward(q, pages, starts, lens, table, 4, 512))
    for b, n in enumerate((123, 64)):
        want, _, mag = oa.attention(_np(q[4 * b:4 * b + 4]), keys[b][:n], values[b][:n], 4)
        assert (np.abs(_np(got[4 * b:4 * b + 4]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag).all()


# ---------------------------------------------------------------- refusals and reports


def test_refusals():
    at = pkg.Attention(8, 2, 64, 16, 4, 10, 2, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.randn(4, 12, 64, device="cuda").to(torch.bfloat16)
    q, k, v = x.split([8, 2, 2], 1)
    pos, slots, pages = torch.arange(4, **i32), torch.arange(4, device="cuda"), at.pages()
    starts, lens, table = torch.tensor([0, 4], **i32), torch.tensor([4], **i32), torch.zeros(1, 4, **i32)
    odd = torch.randn(4 * 12 * 64 + 1, device="cuda").to(torch.bfloat16)[1:].view(4, 12, 64)
    bad = [
        lambda: at.append(q.float(), k, v, pos, slots, pages),
        lambda: at.append(q, k[:3], v, pos, slots, pages),
        lambda: at.append(q[:, :4], k, v, pos, slots, pages),
        lambda: at.append(q, k, v, pos.long(), slots, pages),
        lambda: at.append(q, k, v, pos, slots.int(), pages),
        lambda: at.append(q, k, v, pos, slots, pages[:2]),
        lambda: at.append(odd[:, :8], k, v, pos, slots, pages),  # 2 bytes off a 16-byte boundary
        lambda: at.append(x.transpose(1, 2).contiguous().transpose(1, 2)[:, :8], k, v, pos, slots, pages),
        lambda: at.append(torch.cat([q] * 3), torch.cat([k] * 3), torch.cat([v] * 3), pos.repeat(3), slots.repeat(3), pages),
        lambda: at.forward(q.float(), pages, starts, lens, table, 4, 4),
        lambda: at.forward(q, pages, starts, lens, table, 5, 4),
        lambda: at.forward(q, pages, starts, lens, table, 4, 65),
        lambda: at.forward(q, pages, starts[:1], lens, table, 4, 4),
        lambda: at.forward(q, pages, starts, lens, table[:, :1], 4, 17),
        lambda: at.forward(q, pages, torch.zeros(4, **i32), lens.repeat(3), table.repeat(3, 1), 4, 4),
        lambda: at.forward(q.cpu(), pages, starts, lens, table, 4, 4),
        lambda: at.forward(q, pages, starts, lens, table, 4, 4, out=torch.empty(4, 8, 64, device="cuda")),
        lambda: at.read(slots.int(), pages),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(pkg.MoEError) as e:
            f()
        assert e.value.code == pkg.MOE_EINVAL, i
    at.status()  # none of them reached the GPU
    # empty calls launch nothing
    at.append(q[:0], k[:0], v[:0], pos[:0], slots[:0], pages)
    at.forward(q[:0], pages, starts, lens, table, 0, 4)
    assert at.read(slots[:0], pages)[0].shape == (0, 2, 64)


def test_out_of_range_inputs_are_reported_and_skipped():
    rng = np.random.default_rng(18)
    hq, hk, D, P = 8, 2, 64, 16
    at = pkg.Attention(hq, hk, D, P, 4, 400, 2, 640)
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.randn(4, hq + 2 * hk, D, device="cuda").to(torch.bfloat16)
    q, k, v = x.split([hq, hk, hk], 1)
    pages = at.pages()
    ok = dict(positions=torch.arange(4, **i32), slots=torch.arange(4, device="cuda"))

    def reports(word):
        with pytest.raises(pkg.MoEError) as e:
            at.status()
        assert word in str(e.value) and e.value.code == pkg.MOE_EINVAL
        at.status()  # cleared

    at.append(q, k, v, ok["positions"], torch.tensor([0, 64, 1 << 40, 2], device="cuda"), pages)
    reports("slot")
    assert (at.read(torch.tensor([1], device="cuda"), pages)[0] == 0).all()
    out = at.append(q, k, v, torch.tensor([0, 640, -1, 3], **i32), ok["slots"], pages)
    reports("position")
    assert (out[1:3] == 0).all() and (out[0] != 0).any()
    assert (at.read(torch.tensor([70], device="cuda"), pages)[1] == 0).all()
    reports("slot")
    # a table entry beyond the pages: its tokens are masked
    pages, table, keys, values, n_pages = _cache(rng, [40], hk, D, P, spare=0)
    at2 = pkg.Attention(hq, hk, D, P, n_pages, 400, 2, 640, rot_dim=0)
    for bad in (-1, n_pages, 1 << 30):
        for news in (1, 4, 40):
            t2 = table.clone()
            t2[0, 1] = bad
            qq = torch.randn(news, hq, D, device="cuda").to(torch.bfloat16)
            out = at2.forward(qq, pages, torch.tensor([0, news], **i32), torch.tensor([40], **i32), t2, news, 40)
            with pytest.raises(pkg.MoEError, match="block-table"):
                at2.status()
            gone = np.r_[0:16, 32:40]
            if news <= 8:
                want, _, mag = oa.attention(_np(qq[-1:]), keys[0][gone], values[0][gone], 1)
                assert (np.abs(_np(out[-1:]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag).all()
    # lengths and starts beyond what the call said
    qq = torch.randn(4, hq, D, device="cuda").to(torch.bfloat16)
    for starts, lens in (([0, 9], [40]), ([3, 1], [40]), ([-2, 4], [40]), ([0, 4], [1 << 30]), ([0, 4], [-5])):
        at2.forward(qq, pages, torch.tensor(starts, **i32), torch.tensor(lens, **i32), table, 4, 40)
        with pytest.raises(pkg.MoEError, match="lengths"):
            at2.status()


def test_offsets_past_32_bits():
    """The last of 40,000 pages of 147 KB each lies past 2^32 bytes."""
    hq, hk, D, P = 16, 4, 256, 128
    n_pages = 40_000
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    at = pkg.Attention(hq, hk, D, P, n_pages, 300, 1, 4096, rot_dim=64)
    assert n_pages * at.page_bytes > 1 << 32
    pages = torch.empty(n_pages, at.page_bytes, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(19)
    T = 300
    x = torch.tensor(rng.normal(size=(T, hq + 2 * hk, D)), device="cuda").to(torch.bfloat16)
    q, k, v = x.split([hq, hk, hk], 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[n_pages - 1, 5, n_pages - 2]], **i32)
    j = torch.arange(T, device="cuda")
    slots = table[0][j // P].long() * P + j % P
    qr = at.append(q, k, v, j.int(), slots, pages)
    keys, values = (_np(t) for t in at.read(slots, pages))
    c, s = oa.quantise(oa.prepared(_np(k), None, np.arange(T), 64, oa.frequencies(64)))
    assert np.array_equal(keys, oa.dequantise(c, s))
    for n in (1, 4, 300):
        out = at.forward(qr[T - n:], pages, torch.tensor([0, n], **i32), torch.tensor([T], **i32), table, n, T)
        at.status()
        want, _, mag = oa.attention(_np(qr[T - n:]), keys, values, n)
        assert (np.abs(_np(out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag + 1e-6).all()


@pytest.mark.parametrize("act", [pkg.ACT_F32, pkg.ACT_BF16])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30])
def test_forward_window_beyond_every_length(window, act):
    """Also where queries stand before the first token, at negative positions."""
    rng = np.random.default_rng(23)
    _forward_check(rng, 4, 2, 64, [3, 300], [8, 5], 16, act=act, window=window)
    if act == pkg.ACT_BF16:
        _forward_check(rng, 16, 1, 192, [2, 300], [8, 5], 16, window=window)
        _forward_check(rng, 16, 1, 128, [30, 300], [70, 50], 16, window=window)


@pytest.mark.parametrize("act", [pkg.ACT_F32, pkg.ACT_BF16])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("news", [1, 4, 40])
def test_forward_with_no_cached_token_at_all(D, news, act):
    """max_len = 0: no query sees a key, whichever kernel the row count takes."""
    hq, hk, P = 16, 1, 16
    at = pkg.Attention(hq, hk, D, P, 4, 2 * news, 2, 64, act=act, rot_dim=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn(2 * news, hq, D, device="cuda").to(at.dtype)
    starts, table = torch.tensor([0, news, 2 * news], **i32), torch.full((2, 1), -1, **i32)
    out, lse = torch.full_like(q, 5.0), torch.full((2 * news, hq), 5.0, device="cuda")
    for t in (table, table[:, :0], torch.empty(2, 0, **i32)):
        at.forward(q, at.pages(), starts, torch.tensor([0, 0], **i32), t, news, 0, out=out, lse=lse)
        at.status()
        assert (out == 0).all() and torch.isneginf(lse).all()
        out.fill_(5.0)
        lse.fill_(5.0)
    # a length beyond it is reported, and nothing of it is read
    at.forward(q, at.pages(), starts, torch.tensor([0, 9], **i32), table, news, 0, out=out, lse=lse)
    with pytest.raises(pkg.MoEError, match="lengths"):
        at.status()
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("angle", [2.0 ** -26, 1e-9, 2.0 ** -40])
def test_append_scales_next_to_the_midpoint_of_two_scales(angle):
    """A largest channel within 2^-26 of the midpoint of two neighbouring
    scales, below and above it (a rotation by a small angle puts it there):
    the nearer scale is stored, for every pair of scales."""
    hq, hk, D, P = 1, 1, 64, 16
    b = np.arange(1, oa.KV_MAX_SCALE)
    mid = 3.5 * (oa.scale_of(b) + oa.scale_of(b + 1))  # 8 significant bits: exact in bf16
    T = 2 * len(b)
    k = np.zeros((T, hk, D))
    k[:, 0, 0] = np.repeat(mid, 2)
    k[:, 0, 8] = np.repeat(mid / 2, 2) * np.where(np.arange(T) % 2, -1, 1)  # its partner: below for +, above for -
    k[:, 0, 16:] = np.random.default_rng(0).normal(size=(T, D - 16))
    n_pages = -(-T // P)
    for dtype in (torch.bfloat16, torch.float32):
        at = pkg.Attention(hq, hk, D, P, n_pages, T, 1, 4, rot_dim=16, freq=[angle] * 8)
        kd = torch.tensor(k, device="cuda").to(dtype)
        pos, slots = torch.ones(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda")
        pages = at.pages()
        at.append(kd, kd, kd, pos, slots, pages)
        at.status()
        codes, scales = oa.quantise(oa.prepared(_np(kd), None, np.ones(T), 16, [angle] * 8))
        assert np.array_equal(scales[:, 0, 0], np.repeat(b, 2) + np.arange(T) % 2)  # (the oracle's own choice)
        gc, gs = oa.page_arrays(pages.cpu().numpy(), hk, P, D)[:2]
        sl = np.arange(T)
        assert np.array_equal(gs[sl // P, :, sl % P], scales), (gs[sl // P, :, sl % P] != scales).sum()
        assert np.array_equal(oa.unpack(gc[sl // P, :, sl % P]), codes)


@pytest.mark.parametrize("act,news,lens", [(pkg.ACT_F32, 4, [300, 2]), (pkg.ACT_BF16, 1, [300, 40]), (pkg.ACT_BF16, 1, [9000, 40]),
                                           (pkg.ACT_BF16, 4, [300, 2]), (pkg.ACT_BF16, 4, [9000, 2]), (pkg.ACT_BF16, 70, [300, 50]),
                                           (pkg.ACT_BF16, 70, [9000, 50])])
@pytest.mark.parametrize("hq,hk,D", [(8, 2, 64), (16, 1, 64), (16, 2, 128), (16, 1, 192), (16, 1, 256)])
def test_forward_nan_and_infinite_queries(hq, hk, D, act, news, lens):
    """Their rows are NaN in every kernel (a row without a key stays 0), the
    other rows keep their bits."""
    rng = np.random.default_rng(21)
    P = 16
    pages, table, keys, values, n_pages = _cache(rng, lens, hk, D, P)
    T = 2 * news
    at = pkg.Attention(hq, hk, D, P, n_pages, T, 2, max(lens), act=act, rot_dim=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (pages, torch.tensor([0, news, T], **i32), torch.tensor(lens, **i32), table, news, max(lens))
    q = torch.randn(T, hq, D, device="cuda").to(at.dtype)
    lse, lse_bad = (torch.empty(T, hq, device="cuda") for _ in range(2))
    good = at.forward(q, *args, lse=lse)
    empty = torch.isneginf(lse)  # (rows before the first token of a sequence shorter than its queries)
    bad = q.clone()
    bad[0, 0, 3] = float("nan")
    bad[0, 2, 5] = float("inf")
    bad[news - 1, 1, D - 1] = float("-inf")
    bad[news - 1, hq - 1, 7] = 3.0e38  # finite, with scores beyond fp32
    bad[news - 1, hq - 1, 8] = -3.0e38
    bad[news, 3] = float("nan")
    bad[T - 1, 4, 0] = float("nan")
    rows = torch.zeros(T, hq, dtype=torch.bool, device="cuda")
    for t, h in ((0, 0), (0, 2), (news - 1, 1), (news, 3), (T - 1, 4)):
        rows[t, h] = True
    out = at.forward(bad, *args, lse=lse_bad)
    at.status()
    dead = rows & ~empty
    assert torch.isnan(out[dead]).all(), torch.isnan(out[dead]).all(1)
    assert (out[rows & empty] == 0).all() and torch.isneginf(lse_bad[rows & empty]).all()
    nan = dead.clone()
    nan[0, 2] = nan[news - 1, 1] = False  # (scores of -inf alone have an lse of -inf)
    assert torch.isnan(lse_bad[nan]).all()
    rows[news - 1, hq - 1] = True
    assert torch.equal(out[~rows], good[~rows]) and torch.equal(lse_bad[~rows], lse[~rows])


@pytest.mark.parametrize("act,news", [(pkg.ACT_F32, 1), (pkg.ACT_BF16, 1), (pkg.ACT_BF16, 4), (pkg.ACT_BF16, 70)])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_forward_scores_of_minus_infinity(D, act, news):
    """Keys whose score is -inf have weight 0 beside others; where a row sees
    only such keys its softmax has no value and the row is NaN."""
    hq, hk, P, n = 16, 1, 16, 90
    at = pkg.Attention(hq, hk, D, P, 6, news, 1, 96, act=act, rot_dim=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.ones(n, hk, D, device="cuda")
    k[40:, :, :16] = 0  # (the later keys do not meet the query's infinity: 0 codes would make NaN of it, so it is finite)
    pages, j = at.pages(), torch.arange(n, device="cuda")
    tmp = pkg.Attention(1, hk, D, P, 6, n, 1, 96, rot_dim=0)
    tmp.append(k[:, :1], k, torch.randn_like(k), j.int(), j, pages)
    v = tmp.read(j, pages)[1].float()
    q = torch.zeros(news, hq, D, device="cuda")
    q[:, 0, :16] = -3.0e38  # 16 of them times a key of 1 is beyond fp32
    table = torch.arange(6, **i32)[None]
    args = lambda m: (pages, torch.tensor([0, news], **i32), torch.tensor([m], **i32), table, news, m)
    out = at.forward(q.to(at.dtype), *args(n)).float()
    if news <= 50:  # keys 40.. have score 0: the mean of their values
        want = torch.stack([v[40:n - news + t + 1, 0].mean(0) for t in range(news)])
        assert ((out[:, 0] - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -9).all()
    first = at.forward(q.to(at.dtype)[:news], *args(max(news, 40)))
    at.status()
    seen = min(40, news)
    rows = first[:, 0] if news <= 40 else first[:40, 0]
    assert torch.isnan(rows).all(), seen
    assert torch.isfinite(first[:, 1:]).all()


def test_creation_on_a_side_stream_beside_a_busy_default_stream():
    """The rotation table is made from the frequencies, whatever else is queued on other streams."""
    D, T, far = 256, 64, 1 << 20
    x = torch.randn(T, 3, D, device="cuda")
    q, k, v = x.split([1, 1, 1], 1)
    pos = torch.randint(far, (T,), dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda")
    a = pkg.Attention(1, 1, D, 16, 4, T, 1, far, act=pkg.ACT_F32)
    want = a.append(q, k, v, pos, slots, a.pages())
    big = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for _ in range(4):
            big = big @ big * 1e-2
        b = pkg.Attention(1, 1, D, 16, 4, T, 1, far, act=pkg.ACT_F32, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(b.append(q, k, v, pos, slots, b.pages()), want)
        b.close()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hk,D,rot", HEADS)
def test_append_norm_of_very_large_and_very_small_rows(hq, hk, D, rot, interleaved):
    """Rows whose squares leave the range of fp32 are normalised all the same."""
    rng = np.random.default_rng(22)
    T = 40
    x = rng.normal(size=(T, hq + 2 * hk, D))
    x[0::4] *= 1e22
    x[1::4, ::2] *= 2.0 ** 120  # heads of a token differ
    x[2::4] *= 3e37
    x = np.clip(x, -3.3e38, 3.3e38)
    for dtype, act in ((torch.bfloat16, pkg.ACT_BF16), (torch.float32, pkg.ACT_F32)):
        _append_check(rng, hq, hk, D, rot, T, 32, dtype, act, interleaved=interleaved, x=x)
    # without eps small rows have a norm too (fp32: down to 2^-149, where a channel has few bits)
    x = rng.normal(size=(T, hq + 2 * hk, D))
    x[0::4] *= 1e-22
    x[1::4, ::2] *= 2.0 ** -110
    x[2::4] *= 2.0 ** -124
    f, pos = oa.frequencies(rot), rng.integers(0, 1000, T)
    for dtype in (torch.bfloat16, torch.float32):
        qw, kw = _norms(rng, D)
        at = pkg.Attention(hq, hk, D, 16, 4, T, 1, 1000, act=pkg.ACT_F32, rot_dim=rot, interleaved=interleaved, q_norm=qw, k_norm=kw, eps=0.0)
        t = torch.tensor(x, device="cuda").to(dtype)
        q, k, v = t.split([hq, hk, hk], 1)
        slots, pages = _slots(rng, 4, 16, T), at.pages()
        out = at.append(q, k, v, torch.tensor(pos.astype(np.int32), device="cuda"), slots, pages)
        at.status()
        want = oa.prepared(_np(q), _np(qw), pos, rot, f, interleaved, eps=0.0)
        m = np.abs(oa.prepared(_np(q), _np(qw), pos, 0, f, eps=0.0))
        if rot:
            i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
            s = m[..., i] + m[..., j]
            m[..., i], m[..., j] = s, s
        assert (np.abs(_np(out) - want) <= 2.0 ** -19 * m + 2.0 ** -24 * np.abs(want)).all()
        keys = at.read(slots, pages)[0]
        want = oa.dequantise(*oa.quantise(oa.prepared(_np(k), _np(kw), pos, rot, f, interleaved, eps=0.0)))
        assert np.array_equal(_np(keys), want)
        at.close()


def test_append_norm_of_rows_with_nothing_or_infinities():
    """A zero row without eps is 0/0: NaN, stored as 0; an infinite channel makes NaN of itself and 0 of the others."""
    hq, hk, D = 2, 1, 64
    one = torch.ones(D, device="cuda")
    at = pkg.Attention(hq, hk, D, 16, 1, 3, 1, 4, rot_dim=0, q_norm=one, k_norm=one, eps=0.0)
    x = torch.randn(3, hq + 2 * hk, D, device="cuda").to(torch.bfloat16)
    x[0] = 0
    x[1, :, 5] = float("inf")
    pages, slots = at.pages(), torch.arange(3, device="cuda")
    out = at.append(x[:, :2], x[:, 2:3], x[:, 3:], slots.int(), slots, pages)
    assert torch.isnan(out[0]).all() and torch.isnan(out[1, :, 5]).all() and torch.isfinite(out[2]).all()
    assert (out[1][:, [i for i in range(D) if i != 5]] == 0).all()
    keys = at.read(slots, pages)[0]
    assert (keys[:2] == 0).all() and (keys[2] != 0).any()


def test_results_of_a_given_stream_belong_to_it():
    """Results are allocated on the stream that writes them, not on the current
    one, whose own pending work may still use the memory."""
    hq, hk, D, P, T = 8, 2, 64, 16, 64
    at = pkg.Attention(hq, hk, D, P, 8, T, 1, 100, rot_dim=0)
    x = torch.randn(T, hq + 2 * hk, D, device="cuda").to(torch.bfloat16)
    q, k, v = x.split([hq, hk, hk], 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    pos, slots, pages = torch.arange(T, **i32), torch.arange(T, device="cuda"), at.pages()
    seq = (torch.tensor([0, T], **i32), torch.tensor([T], **i32), torch.arange(4, **i32)[None], T, T)
    logits = torch.randn(64, 1000, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls = (lambda s: [at.append(q, k, v, pos, slots, pages, stream=s)], lambda s: list(at.read(slots, pages, stream=s)),
             lambda s: [at.forward(q, pages, *seq, stream=s)],
             lambda s: list(pkg.token_logprobs(logits, pos, 8, stream=s).values()))
    for i, call in enumerate(calls):
        want = call(None)
        torch.cuda.synchronize()
        keep = [t.clone() for t in want]
        torch.cuda.synchronize()
        freed = {t.data_ptr() for t in want}
        del want  # blocks of the same sizes, free on the current stream
        got = call(side)
        side.synchronize()
        assert not freed & {t.data_ptr() for t in got}, i
        assert all(torch.equal(a, b) for a, b in zip(got, keep))


def test_a_refused_creation_leaves_no_error_behind():
    """A workspace that no GPU holds is refused with MOE_ENOMEM; what is launched next does not see the error."""
    with pytest.raises(pkg.MoEError) as e:
        pkg.Attention(64, 64, 256, 16, 4, 1 << 20, 1, 1 << 27, rot_dim=0)  # (some 9 TB of operand images)
    assert e.value.code == pkg.MOE_ENOMEM
    assert int(torch.arange(5, device="cuda").sum()) == 10
    at = pkg.Attention(4, 2, 64, 16, 4, 4, 1, 64)
    at.status()


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("news", [1, 8, 100])  # 4 rows each: the small, the verify and the prompt kernel
def test_forward_bad_table_entries_mask_their_tokens_in_every_kernel(D, news):
    rng = np.random.default_rng(24 + D)
    hq, hk, P, n = 8, 2, 16, 150
    pages, table, keys, values, n_pages = _cache(rng, [n], hk, D, P, spare=0)
    at = pkg.Attention(hq, hk, D, P, n_pages, news, 1, n, rot_dim=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn(news, hq, D, device="cuda").to(torch.bfloat16)
    for bad in (-1, n_pages, 1 << 30, -(1 << 31), 1 - (1 << 31), 2 ** 31 - 1):
        t2 = table.clone()
        t2[0, 1] = t2[0, 9] = bad  # tokens 16..31 and 144..149
        lse = torch.empty(news, hq, device="cuda")
        out = _np(at.forward(q, pages, torch.tensor([0, news], **i32), torch.tensor([n], **i32), t2, news, n, lse=lse))
        with pytest.raises(pkg.MoEError, match="block-table"):
            at.status()
        for t in range(news):
            pos = n - news + t
            here = np.array([j for j in range(pos + 1) if j // 16 not in (1, 9)])
            want, wl, mag = oa.attention(_np(q[t:t + 1]), keys[0][here], values[0][here], 1)
            assert (np.abs(out[t] - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -9 * mag[0]).all(), (bad, t)
            assert (np.abs(_np(lse[t]) - wl[0]) <= 2.0 ** -9).all()
    # every page absent: no key
    t2 = torch.full_like(table, -1)
    out = at.forward(q, pages, torch.tensor([0, news], **i32), torch.tensor([n], **i32), t2, news, n, lse=lse)
    with pytest.raises(pkg.MoEError, match="block-table"):
        at.status()
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("act", [pkg.ACT_F32, pkg.ACT_BF16])
@pytest.mark.parametrize("news", [1, 8, 100])
def test_forward_lengths_and_starts_beyond_the_call_in_every_kernel(news, act):
    """They are clamped to what the call said, reported, and nothing outside is read or written."""
    rng = np.random.default_rng(25)
    hq, hk, D, P, n = 8, 2, 64, 16, 150
    pages, table, keys, values, n_pages = _cache(rng, [n], hk, D, P, spare=0)
    at = pkg.Attention(hq, hk, D, P, n_pages, news + 6, 1, n, act=act, rot_dim=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn(news + 6, hq, D, device="cuda").to(at.dtype)
    for starts, length, rows, want_len in (([3, news + 3], 1 << 30, (3, news), n), ([3, news + 3], -5, (3, news), 0),
                                           ([-2, news], n, (0, news), n), ([5, 2], n, (0, 0), n),
                                           ([6, 1 << 30], n, (6, news), n), ([1 << 30, 1 << 30], n, (0, 0), n)):
        out = torch.full_like(q, 7.0)
        at.forward(q, pages, torch.tensor(starts, **i32), torch.tensor([length], **i32), table, news, n, out=out)
        with pytest.raises(pkg.MoEError, match="lengths"):
            at.status()
        a, t = rows
        assert (out[:a] == 7).all() and (out[a + t:] == 7).all()
        if t:
            want, _, mag = oa.attention(_np(q[a:a + t]), keys[0][:want_len], values[0][:want_len], t) if want_len else (0.0, 0, 0.0)
            assert (np.abs(_np(out[a:a + t]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag).all(), starts


def test_forward_prompts_in_groups_that_share_the_images():
    """More sequences than the operand images hold at once run group by group, whole and with split row tiles."""
    rng = np.random.default_rng(26)
    hq, hk, D, n = 16, 16, 256, 2000
    tiles = -(-n // 128)
    assert (256 << 20) // (4 * 128 * D) // (hk * tiles) < 9  # the sequences that go at once
    _forward_check(rng, hq, hk, D, [2000, 1, 700, 1999, 300, 1300, 0, 257, 2000], [300, 1, 257, 280, 300, 260, 3, 257, 12], 128)
    # one key/value head: the row tiles of a group do not fill the GPU, so their keys are split
    _forward_check(rng, 4, 1, 256, [9000] + [200] * 9, [65] + [66] * 9, 64, extra=150_000)


@pytest.mark.parametrize("hq,hk,D", [(16, 16, 64), (16, 16, 128)])
def test_forward_prompt_walks_past_its_ring(hq, hk, D):
    """Row tiles that go whole, over more key tiles than the ring of images has stages."""
    rng = np.random.default_rng(27)
    # 16 heads x 5 row tiles of 256 rows = 80 pairs: 76 whole ones, the others split
    _forward_check(rng, hq, hk, D, [2500], [1280], 64)


def test_workspace_of_a_windowed_handle():
    """A prompt's operand images take what its window and chunk can reach, not the longest sequence."""
    kw = dict(n_q_heads=16, n_kv_heads=4, head_dim=192, page_tokens=64, n_pages=8, T_max=256, S_max=1, len_max=131072, rot_dim=0)
    whole = pkg.Attention(**kw).workspace_bytes
    part = pkg.Attention(**kw, window=512).workspace_bytes
    tile = 4 * 2 * 128 * 192 * 2  # 128 tokens of all heads
    assert whole >= 1024 * tile and part <= whole - 1000 * tile
    # and they hold all that a call needs: chunks of T_max tokens far into a sequence, several sequences
    rng = np.random.default_rng(28)
    _forward_check(rng, 8, 2, 64, [3000, 200, 129, 2100], [300, 200, 100, 1], 64, window=100, extra=30_000)
    _forward_check(rng, 16, 2, 256, [2000, 130], [128, 20], 128, window=1, extra=30_000)


@pytest.mark.parametrize("news", [1, 4, 70])  # 16 rows each: the small, the verify and the prompt kernel
@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_forward_waits_run_out_and_the_handle_recovers(D, news):
    """An operand that never arrives ends the launch with MOE_ETIMEOUT; the next one is as before."""
    import time
    rng = np.random.default_rng(29)
    hq, hk, P, lens = 16, 1, 64, [4000, 130]
    pages, table, keys, values, n_pages = _cache(rng, lens, hk, D, P)
    at = pkg.Attention(hq, hk, D, P, n_pages, 2 * news, 2, 4000, rot_dim=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn(2 * news, hq, D, device="cuda").to(torch.bfloat16)
    args = (q, pages, torch.tensor([0, news, 2 * news], **i32), torch.tensor(lens, **i32), table, news, 4000)
    want = at.forward(*args)
    at.status()
    at.inject_timeout(1000)
    t0 = time.perf_counter()
    at.forward(*args)
    with pytest.raises(pkg.MoEError, match="timed out") as e:
        at.status()
    assert e.value.code == pkg.MOE_ETIMEOUT and time.perf_counter() - t0 < 5
    at.status()  # cleared
    for _ in range(2):
        assert torch.equal(at.forward(*args), want)
        at.status()
    with pytest.raises(pkg.MoEError):
        at.inject_timeout(0)
