"""Sampled verification at the borders of what its definition says."""
import numpy as np
import pytest
import torch

import block_quantized_moe_layer_gb300 as pkg
from tests.test_gpu_verify_sample import _i32, _peaked

pytestmark = pytest.mark.gpu


def test_a_millionth_is_greedy():
    """The fp32 number 1e-6 is below 1e-6: as temperature 0, drawn drafts and all."""
    rng = np.random.default_rng(44)
    n = 30
    x = torch.tensor(_peaked(rng, 3 * n, 200), dtype=torch.float32, device="cuda")
    y = torch.tensor(_peaked(rng, 3 * n, 200), dtype=torch.float32, device="cuda")
    tokens = torch.stack([x[::3].argmax(1) * 0, y[::3].argmax(1), x[::3].argmax(1)], 1).flatten().to(torch.int32)
    u = torch.rand(3 * n, device="cuda")
    for drafts in (None, y):
        a, b, c = (pkg.verify_sample(x, tokens, _i32([-1, 0, 0] * n), _i32(range(0, 3 * n + 1, 3)), u, 3, draft_logits=drafts,
                                     temperature=torch.full((n,), t, device="cuda")) for t in (0.0, 1e-6, 1e-7))
        assert all(torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]) for k in a)
        assert (a["n_accepted"] == 1).all() and (a["path"][:, 1] == 2).sum() > n // 2
