"""The draw of the next token where little is left: it is always a token that the
target has, whatever the roundings, and its place is right to the documented part
of the row's sum.
"""
import numpy as np
import pytest
import torch

import block_quantized_moe_layer_gb300 as pkg
from tests.test_gpu_verify_sample import _i32

pytestmark = pytest.mark.gpu


def _star(x, kids, uniforms, draft=None):
    """next and n_accepted of trees of a root with one level of children: x [n, V] the roots' rows, kids [n, c], uniforms [n, 1 + c]."""
    n, c = kids.shape
    rows = torch.zeros(n, 1 + c, x.shape[1], device="cuda", dtype=x.dtype)
    rows[:, 0] = x
    drafts = None
    if draft is not None:
        drafts = torch.zeros_like(rows)
        drafts[:, 0] = draft
        drafts = drafts.flatten(0, 1)
    tokens = torch.cat([torch.zeros(n, 1, dtype=torch.int64), kids], 1).flatten()
    r = pkg.verify_sample(rows.flatten(0, 1), _i32(tokens), _i32(([-1] + [0] * c) * n), _i32(range(0, n * (1 + c) + 1, 1 + c)),
                          torch.as_tensor(uniforms, dtype=torch.float32).flatten().cuda(), 1 + c, draft_logits=drafts)
    return r["next"].cpu(), r["n_accepted"].cpu()


@pytest.mark.parametrize("V", [50, 4099])
def test_rejected_drafts_leave_nothing_of_a_range(V):
    """Two improbable drafts side by side among masked tokens; the number 0 asks for the first token that is left."""
    rng = np.random.default_rng(V)
    n = 200
    x = np.full((n, V), -np.inf)
    x[:, V // 2:] = rng.normal(size=(n, V - V // 2))
    x[:, V // 2] = 8
    kids = np.stack([rng.choice(4, 2, replace=False) for _ in range(n)])
    for i in range(n):
        x[i, kids[i]] = rng.uniform(-25, -8, 2)
    u = np.full((n, 3), 0.5)
    u[:, 0] = 0
    nxt, acc = _star(torch.tensor(x, dtype=torch.float32, device="cuda"), torch.tensor(kids), u)
    assert (acc == 0).all() and (nxt == V // 2).all(), nxt


def test_drafts_that_are_nearly_the_target():
    """Rejected drafts of a draft head that is the target's to a part in 10^5: tokens whose rest is about nothing come first."""
    rng = np.random.default_rng(3)
    n, V = 3000, 40
    for noise in (1e-5, 1e-3):
        x = rng.normal(size=(n, V))
        y = x + noise * rng.normal(size=(n, V))
        x[:, 30] -= 3.0  # the draft that the target hardly has
        x[:, 36] = 2.0
        x, y = (torch.tensor(v, dtype=torch.float32, device="cuda") for v in (x, y))
        kids = torch.full((n, 1), 30)
        u = np.full((n, 2), 0.97)
        u[:, 0] = 0
        nxt, acc = _star(x, kids, u, y)
        p, q = (torch.softmax(v.double(), 1).cpu() for v in (x, y))
        some = acc == 0
        assert some.float().mean() > 0.9 and (nxt >= 0).all()
        at = nxt[some].long()[:, None]
        # what it has left, p - q, is not below nothing by more than roundings
        assert (p[some].gather(1, at) - q[some].gather(1, at) >= -(2.0 ** -32)).all()


@pytest.mark.parametrize("blocks", [1, 16])
@pytest.mark.parametrize("V,low", [(1 << 22, 39.0), (1 << 22, 36.3), (1 << 20, 41.0), (1 << 24, 38.0), (1 << 24, 43.0)])
def test_a_broad_rest_of_a_long_row(V, low, blocks):
    """A rejected chosen draft that held all but a rest of tokens of 2^-low of it each: one of them is drawn, and the
    mass before it, of the row's sum, is right to 2^-32 (to 2^-30 above 2^22 tokens)."""
    x = torch.full((V,), -low * float(np.log(2.0)), dtype=torch.float64)
    top = V // 3
    x[top] = 0
    x = x.float()
    w = torch.exp(x.double())
    w[top] = 0
    rest = float(w.sum())
    near = (2.0 ** -32 if V <= 1 << 22 else 2.0 ** -30) * (1 + rest)
    if rest < 2.0 ** -23:
        pytest.skip("no fp32 number rejects the draft")
    mass = torch.cumsum(w, 0)
    n = 160 if blocks == 1 else 1  # (sequences without nodes fill the GPU)
    rows = torch.stack([x, torch.zeros_like(x)]).cuda()
    one = float(np.nextafter(np.float32(1), np.float32(0)))
    for u0 in (0.0, 0.1, 0.37, 0.5, 0.8, one):
        r = pkg.verify_sample(rows, _i32([0, top]), _i32([-1, 0]), _i32([0] + [2] * n), torch.tensor([u0, one], device="cuda"), 2)
        nxt = int(r["next"][0])
        assert int(r["n_accepted"][0]) == 0 and 0 <= nxt < V and nxt != top
        t = float(np.float32(u0)) * rest
        before, through = float(mass[nxt] - w[nxt]), float(mass[nxt])
        assert before - near <= t <= through + near, (u0, nxt, (before - t) / near, (t - through) / near)


@pytest.mark.parametrize("blocks", [1, 16])
def test_equal_tokens_of_a_long_row(blocks):
    """A likely token and a broad rest of equal ones, of 2^-36.3 of it: the place of the number among them."""
    V, near = 1 << 22, 2.0 ** -32
    x = torch.full((V,), -36.3 * float(np.log(2.0)), dtype=torch.float64)
    x[V - 1] = 0
    x = x.float()
    w = torch.exp(x.double())
    w /= w.sum()
    mass = torch.cumsum(w, 0)
    n = 160 if blocks == 1 else 1
    for part in (0.01, 0.3, 0.5, 0.77, 0.999):
        u = float(np.float32(part * float(mass[V - 2])))
        r = pkg.verify_sample(x[None].cuda(), _i32([0]), None, _i32([0] + [1] * n), torch.tensor([u], device="cuda"), 1)
        nxt = int(r["next"][0])
        assert float(mass[nxt] - w[nxt]) - near <= u <= float(mass[nxt]) + near, (part, nxt, (u - float(mass[nxt])) / near)
