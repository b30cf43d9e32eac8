"""Pins of the attention oracle against closed forms."""
import numpy as np

from oracle import attn as oa


def test_scales_are_the_top_bits_of_half_precision():
    b = np.arange(oa.KV_MAX_SCALE + 1)
    half = (b.astype(np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(oa.scale_of(b), half)
    assert oa.scale_of(198) == 896.0 and (np.diff(half) > 0).all()


def test_pack_is_nibbles_of_words_and_round_trips():
    c = np.arange(16, dtype=np.uint8).reshape(1, 16)
    w = oa.pack(c).view("<u4")
    # channels 0..7 -> nibbles 0, 4, 1, 5, 2, 6, 3, 7
    assert w[0, 0] == 0x75316420
    assert np.array_equal(oa.unpack(oa.pack(c)), c)
    r = np.random.default_rng(0).integers(0, 16, (3, 5, 64)).astype(np.uint8)
    assert np.array_equal(oa.unpack(oa.pack(r)), r)


def test_quantise_hand_built_blocks():
    x = np.zeros((1, 16))
    c, b = oa.quantise(x)
    assert (c == 8).all() and b[0, 0] == 0
    x[0, :5] = [7.0, -7.0, 0.5, 1.5, 2.5]  # d = 1: halves go to the even code
    c, b = oa.quantise(x)
    assert oa.scale_of(b[0, 0]) == 1.0 and list(c[0, :5]) == [15, 1, 8, 10, 10]
    x[0, 0] = 1e9  # saturates
    c, b = oa.quantise(x)
    assert b[0, 0] == 198 and c[0, 0] == 15
    # 7.4375 / 7 = 1.0625, the midpoint of 1 (byte 120) and 1.125: the even byte
    x[:] = 0
    x[0, 0] = 7.4375
    assert oa.quantise(x)[1][0, 0] == 120
    # the midpoint of 1.125 (byte 121) and 1.25 (byte 122): the even byte again
    x[0, 0] = 7 * 1.1875
    assert oa.quantise(x)[1][0, 0] == 122
    rng = np.random.default_rng(1)
    r = rng.normal(size=(50, 64))
    c, b = oa.quantise(r)
    d = np.repeat(oa.scale_of(b), 16, -1)
    inside = (r >= -8.5 * d) & (r <= 7.5 * d)
    assert (np.abs(oa.dequantise(c, b) - r)[inside] <= 0.5 * d[inside] + 1e-15).all() and inside.mean() > 0.99


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(2)
    f = oa.frequencies(32)
    for inter in (False, True):
        x = rng.normal(size=(2, 1, 64))
        y = oa.prepared(x, None, [5, 9], 32, f, inter)
        assert np.allclose((x ** 2).sum(-1), (y ** 2).sum(-1))
        z = oa.prepared(x, None, [105, 109], 32, f, inter)
        assert np.isclose((y[0] * y[1]).sum(), (z[0] * z[1]).sum())
        assert np.array_equal(x[..., 32:], y[..., 32:])


def test_attention_closed_forms():
    rng = np.random.default_rng(3)
    v = rng.normal(size=(9, 2, 64))
    k = np.zeros((9, 2, 64))
    q = rng.normal(size=(3, 4, 64))
    o, lse, _ = oa.attention(q, k, v, 3)  # equal scores: the mean of the visible values
    assert np.allclose(o[0, 0], v[:7, 0].mean(0)) and np.allclose(o[2, 3], v[:, 1].mean(0))
    assert np.allclose(lse[1], np.log(8))
    o, lse, _ = oa.attention(q, k, v, 3, window=1)
    assert np.allclose(o[1, 2], v[7, 1]) and np.allclose(lse, 0)
    o, lse, _ = oa.attention(q, k[:1], v[:1], 3)  # one cached token, three queries: the first two see nothing
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(o[2, 0], v[0, 0])


def test_scores_closed_forms():
    lp, en, ids, tl = oa.scores(np.zeros((1, 8)), [3], 3)
    assert np.isclose(lp[0], -np.log(8)) and np.isclose(en[0], np.log(8)) and list(ids[0]) == [0, 1, 2]
    x = np.full((2, 5), -np.inf)
    x[1, 4] = 2.0
    lp, en, ids, tl = oa.scores(x, [0, 4], 2)
    assert np.isneginf(lp[0]) and lp[1] == 0 and en[0] == 0 and en[1] == 0 and ids[1, 0] == 4
