"""Host-side refusals of the attention and scoring entry points (no GPU needed)."""
import ctypes

import pytest

import block_quantized_moe_layer_gb300 as pkg


@pytest.fixture(scope="module")
def lib():
    from block_quantized_moe_layer_gb300 import _build
    _build.build()
    return pkg.lib()


def test_attention_entry_points_reject_bad_arguments_on_host(lib):
    assert lib.moe_attn_page_bytes(4, 192, 64) == 4 * 64 * 192 * 9 // 8
    for bad in ((0, 192, 64), (4, 80, 64), (4, 192, 48), (2000, 64, 16)):
        assert lib.moe_attn_page_bytes(*bad) == 0
    out = ctypes.c_void_p()
    good = dict(n_q_heads=64, n_kv_heads=4, head_dim=192, page_tokens=64, n_pages=10, rot_dim=64, T_max=4, S_max=1,
                len_max=100, eps=1e-6)
    for change in (dict(n_q_heads=63), dict(n_q_heads=0), dict(n_kv_heads=0), dict(head_dim=96), dict(page_tokens=8),
                   dict(n_pages=0), dict(rot_dim=24), dict(rot_dim=208), dict(rot_dim=-16), dict(interleaved=2),
                   dict(window=-1), dict(act_dtype=2), dict(T_max=0), dict(S_max=0), dict(S_max=70000), dict(len_max=0),
                   dict(eps=-1.0), dict(eps=float("nan")), dict(scale=-1.0), dict(scale=float("inf")),
                   dict(rope_base=-1.0)):
        d = pkg.MoeAttnDesc(**{**good, **change})
        assert lib.moe_attn_create(ctypes.byref(d), None, ctypes.byref(out)) == pkg.MOE_EINVAL, change
        assert b"moe_attn_create" in lib.moe_last_error()
    assert lib.moe_attn_create(None, None, ctypes.byref(out)) == pkg.MOE_EINVAL
    assert out.value is None
    assert lib.moe_attn_append(None, None, None, None, 0, None, None, None, 1, None, None, None) == pkg.MOE_EINVAL
    assert lib.moe_attn_read(None, None, None, 1, None, None, None) == pkg.MOE_EINVAL
    assert lib.moe_attn_forward(None, None, 0, 0, None, None, None, None, 1, 1, 1, 1, 1, None, None, None) == pkg.MOE_EINVAL
    assert lib.moe_attn_status(None, None) == pkg.MOE_EINVAL
    # token scores: dtype, sizes, n_top, stride, NULL pointers
    for args in ((7, 10, 1, 10, 0), (1, 10, -1, 10, 0), (1, 10, 1, 0, 0), (1, 10, 1, 10, 11), (1, 100, 1, 100, 33),
                 (1, 9, 2, 10, 0), (1, 10, 1, 10, 0)):
        dtype, stride, n, V, top = args
        assert lib.moe_token_logprobs(None, dtype, stride, n, V, None, top, None, None, None, None, None) == pkg.MOE_EINVAL
    assert lib.moe_token_logprobs(None, 1, 10, 0, 10, None, 0, None, None, None, None, None) == pkg.MOE_OK


def test_timeout_hook_rejects_a_missing_handle(lib):
    assert lib.moe_attn_inject_timeout(None, 1000) == pkg.MOE_EINVAL
    assert b"moe_attn_inject_timeout" in lib.moe_last_error()
