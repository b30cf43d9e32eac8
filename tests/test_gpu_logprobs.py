"""Token scores against the fp64 oracle.

Tolerance, derived before the first run: z = x - M is off by one fp32 rounding
(2^-24 |z|), e^z by 2^-21 of itself, a thread's sum of at most n terms by n
2^-24 (all terms positive), the logarithm by 2^-22 of ln S + 1; so log
probabilities are within 2^-23 |result| + 2^-20 + n 2^-24, and the entropy,
whose second sum has terms of one sign as well, within the same times (1 +
its value).  n: at most V / 256 + 16 terms a thread, and 16 joins."""
import numpy as np
import pytest
import torch

import block_quantized_moe_layer_gb300 as pkg
from oracle import attn as oa

pytestmark = pytest.mark.gpu


def _check(x, tokens, n_top, dev=None):
    dev = x.cuda() if dev is None else dev
    r = pkg.token_logprobs(dev, torch.tensor(tokens, dtype=torch.int32, device="cuda"), n_top)
    lp, en, ids, tl = oa.scores(x.double().numpy(), tokens, n_top)
    V = x.shape[1]
    t = 2.0 ** -20 + (V / 256 + 32) * 2.0 ** -24
    got = {k: v.cpu().numpy().astype(np.float64) for k, v in r.items()}

    def near(a, b, tol):
        fin = np.isfinite(b)
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isneginf(a), np.isneginf(b))
        assert (np.abs(a - b)[fin] <= tol[fin]).all(), float((np.abs(a - b)[fin] - tol[fin]).max())

    near(got["logprob"], lp, t + 2.0 ** -22 * np.abs(lp))
    near(got["entropy"], en, t * (1 + en))
    near(got["top_logprobs"], tl, t + 2.0 ** -22 * np.abs(tl))
    assert np.array_equal(got["top_ids"].astype(np.int64), ids)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V", [(1, 1), (3, 2), (2, 31), (5, 257), (4, 1000), (2, 4097), (4, 32768), (7, 100_003), (400, 2049), (1, 1 << 20)])
def test_random_rows(n, V, dtype):
    rng = np.random.default_rng(n * 7919 + V)
    x = torch.tensor(rng.normal(size=(n, V)) * 3).to(dtype)
    for n_top in sorted({0, 1, min(V, 5), min(V, 32)}):
        _check(x, rng.integers(0, V, n).tolist(), n_top)


@pytest.mark.parametrize("V", [300, 5000, 40_000])
def test_ties_and_orders(V):
    k = min(32, V)
    _check(torch.zeros(3, V), [0, V - 1, V // 2], k)  # all equal: the lowest ids
    up = torch.arange(V, dtype=torch.float32) / 100
    _check(torch.stack([up, up.flip(0), (up % 0.05)]), [1, 2, 3], k)
    _check((torch.randn(4, V) * 2).round(), [0, 1, 2, 3], k)  # many equal values
    x = torch.zeros(2, V)
    x[0, ::2] = -0.0
    _check(x, [0, 1], k)  # -0 and 0 are equal


def test_masked_rows():
    V = 9000
    x = torch.full((6, V), float("-inf"))
    x[1, 7777] = 3.0  # one token left
    x[2, [5, 4000, 8999]] = torch.tensor([1.0, 1.0, -2.0])
    x[3] = torch.finfo(torch.float32).min  # the type's lowest value everywhere: uniform
    x[4, ::3] = torch.finfo(torch.float32).min
    x[5] = torch.randn(V)
    x[5, 100:8000] = torch.finfo(torch.float32).min
    _check(x, [3, 7777, 8999, 10, 1, 200], 8)
    _check(x, [3, 0, 4000, 10, 3, 50], 32)


def test_large_values_and_bad_tokens():
    V = 5000
    x = torch.randn(4, V) * 3
    x[1] += 1e6
    x[2] *= 1e30
    x[3, 17] = 3e38
    r = pkg.token_logprobs(x.cuda(), torch.tensor([V, -1, int(x[2].argmax()), 17], dtype=torch.int32, device="cuda"), 3)
    lp = r["logprob"].cpu()
    assert torch.isnan(lp[:2]).all() and (lp[2:] == 0).all() and (r["entropy"][2:] == 0).all()
    _check(x, [V, -1, int(x[2].argmax()), 17], 3)


def test_nan_and_inf_rows():
    x = torch.randn(3, 3000)
    x[0, 5] = float("nan")
    x[1, 6] = float("inf")
    x[2] = float("nan")
    r = pkg.token_logprobs(x.cuda(), torch.tensor([1, 1, 1], dtype=torch.int32, device="cuda"), 4)
    assert torch.isnan(r["logprob"]).all() and torch.isnan(r["entropy"]).all()
    best = x[0].nan_to_num(-1e9).argsort(descending=True)[:4].int()
    assert torch.equal(r["top_ids"][0].cpu(), best) and r["top_ids"][1, 0] == 6
    assert (r["top_ids"][2] == -1).all() and torch.isnan(r["top_logprobs"][2]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned_rows(dtype):
    rng = np.random.default_rng(3)
    for off in range(0, 9):
        for V in (1, 5, 700, 4099):
            big = torch.tensor(rng.normal(size=(3, V + 11))).to(dtype)
            dev = big.cuda()
            _check(big[:, off:off + V], rng.integers(0, V, 3).tolist(), min(V, 6), dev=dev[:, off:off + V])


def test_optional_outputs_streams_and_refusals():
    x = torch.randn(4, 3000, device="cuda")
    tok = torch.arange(4, dtype=torch.int32, device="cuda")
    full = pkg.token_logprobs(x, tok, 5)
    r = pkg.token_logprobs(x, None, 5, entropy=False)
    assert r["logprob"] is None and r["entropy"] is None and torch.equal(r["top_ids"], full["top_ids"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y = x * 1.0
        s = pkg.token_logprobs(y, tok, 5)
    st.synchronize()
    assert all(torch.equal(s[k], full[k]) for k in full)
    assert pkg.token_logprobs(x[:0], tok[:0], 5)["top_ids"].shape == (0, 5)
    for f in (lambda: pkg.token_logprobs(x, tok.long()), lambda: pkg.token_logprobs(x.half(), tok),
              lambda: pkg.token_logprobs(x, tok, 33), lambda: pkg.token_logprobs(x.t(), tok),
              lambda: pkg.token_logprobs(x[:, :3], tok, 4), lambda: pkg.token_logprobs(x, tok[:2]),
              lambda: pkg.token_logprobs(x.cpu(), tok)):
        with pytest.raises(pkg.MoEError):
            f()


def _time_us(x, n_top):
    """The best of five times of 10 calls."""
    pkg.token_logprobs(x, None, n_top)
    best = float("inf")
    for _ in range(5):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        torch.cuda.synchronize()
        e[0].record()
        for _ in range(10):
            pkg.token_logprobs(x, None, n_top)
        e[1].record()
        e[1].synchronize()
        best = min(best, e[0].elapsed_time(e[1]) * 100)
    return best


@pytest.mark.parametrize("n,V", [(64, 151_936), (2, 151_936), (300, 32_768)])
def test_masked_and_equal_logits_cost_no_more_than_twice_ordinary_rows(n, V):
    """Rows with few logits left, or of few different values: every element
    ties with the bound of the best, but few can be among them."""
    x = torch.randn(n, V, device="cuda")
    usual = _time_us(x, 20)
    few = torch.full((n, V), float("-inf"), device="cuda")
    few[:, torch.randint(V, (3,)).tolist()] = 1.0
    part = x.clone()
    part[:, V // 3:] = float("-inf")
    for y in (few, part, torch.zeros(n, V, device="cuda"), x.round(), few.to(torch.bfloat16)):
        us = _time_us(y, 20)
        assert us <= 2 * usual + 20, (us, usual)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V", [(1, 151_936), (3, 40_000), (200, 3001), (2, 33)])
def test_masked_and_equal_logits_in_any_place(n, V, dtype):
    rng = np.random.default_rng(V)
    for left in (0, 1, 3, 19, 40):
        x = torch.full((n, V), float("-inf"))
        for i in range(n):
            at = rng.choice(V, min(left, V), replace=False)
            x[i, at] = torch.tensor(rng.integers(-2, 3, len(at)).astype(np.float32))
        _check(x.to(dtype), rng.integers(0, V, n).tolist(), min(V, 20))
    stretch = torch.full((n, V), float("-inf"))
    stretch[:, V // 2:V // 2 + 25] = torch.randn(n, min(25, V - V // 2))
    _check(stretch.to(dtype), [V // 2] * n, min(V, 32))
    _check(torch.full((n, V), 2.0).to(dtype), [0] * n, min(V, 32))
    _check((torch.randn(n, V) * 0.6).round().to(dtype), [1] * n, min(V, 32))
