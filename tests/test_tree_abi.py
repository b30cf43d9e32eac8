"""Host-side refusals of the tree operators' entry points (no GPU needed)."""
import pytest

import block_quantized_moe_layer_gb300 as pkg


@pytest.fixture(scope="module")
def lib():
    from block_quantized_moe_layer_gb300 import _build
    _build.build()
    return pkg.lib()


def test_attention_and_commit_reject_a_missing_handle(lib):
    assert lib.moe_attn_forward_tree(None, None, 0, 0, None, None, None, None, 1, 4, 1, 4, 4, 1, None, None, None) == pkg.MOE_EINVAL
    assert b"moe_attn_forward_tree" in lib.moe_last_error()
    assert lib.moe_attn_forward_tree(None, None, 0, 0, None, None, None, None, 1, 4, 1, 70, 65, 1, None, None, None) == pkg.MOE_EINVAL
    assert b"64" in lib.moe_last_error()
    assert lib.moe_attn_commit(None, None, None, None, None, 1, None, 1, 1, 1, None, None) == pkg.MOE_EINVAL
    assert b"moe_attn_commit" in lib.moe_last_error()


def test_verify_sample_rejects_bad_arguments_on_host(lib):
    def call(logits=16, dtype=1, stride=10, draft=None, dstride=10, V=10, tokens=16, parents=None, starts=16, n_seqs=1, n_nodes=4,
             max_nodes=4, uniforms=16, temperature=None, replacement=0, path=16, acc=16, nxt=16):
        return lib.mtp_verify_sample(logits, dtype, stride, draft, dstride, V, tokens, parents, starts, n_seqs, n_nodes, max_nodes,
                                     uniforms, temperature, replacement, path, acc, nxt, None)
    for change in (dict(dtype=2), dict(V=0), dict(V=2 ** 24 + 1), dict(n_seqs=-1), dict(n_nodes=-1), dict(max_nodes=0), dict(max_nodes=65),
                   dict(replacement=2), dict(stride=9), dict(draft=16, dstride=9), dict(logits=None), dict(tokens=None), dict(starts=None),
                   dict(uniforms=None), dict(path=None), dict(acc=None), dict(nxt=None), dict(logits=18), dict(draft=17)):
        assert call(**change) == pkg.MOE_EINVAL, change
        assert b"mtp_verify_sample" in lib.moe_last_error()
    assert call(n_seqs=0) == pkg.MOE_OK
