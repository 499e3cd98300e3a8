"""Pins of the oracle's token sampling and 8-bit cache: closed forms, brute
force and invariants (CPU only)."""
import numpy as np
import pytest

from oracle import kv8, sample
from oracle.quant import e4m3_decode


def test_greedy_is_argmax_lowest_index():
    z = [0.5, 2.0, 2.0, -1.0]
    for u in (0.0, 0.5, 0.999):
        assert sample.sample_row(z, u, temperature=0.0) == (1, 0.0)


def test_plain_draw_is_the_inverse_cdf_of_the_softmax():
    z = np.log([0.1, 0.2, 0.3, 0.4])
    for u, i in ((0.0, 0), (0.09, 0), (0.11, 1), (0.29, 1), (0.31, 2), (0.61, 3)):
        t, lp = sample.sample_row(z, u)
        assert t == i and lp == pytest.approx(z[i], abs=1e-12)


def test_cutoffs_keep_prefixes_with_ties_to_the_lowest_index():
    z = np.array([1.0, 3.0, 2.0, 3.0, 2.0])
    kept = lambda **kw: list(np.flatnonzero(sample.kept(z, **kw)))  # noqa: E731
    assert kept(top_k=1) == [1]
    assert kept(top_k=3) == [1, 2, 3]
    assert kept(min_p=1.0) == [1, 3]
    assert kept(min_p=np.exp(-1.0) * 0.999) == [1, 2, 3, 4]
    assert kept(top_p=0.0) == [1]
    assert kept(top_p=1.0) == [0, 1, 2, 3, 4]
    # four equal tokens: half the mass is exactly two of them
    assert list(np.flatnonzero(sample.kept([1.0] * 4, top_p=0.5))) == [0, 1]
    # top-p acts on what top-k left
    assert kept(top_k=2, top_p=0.5) == [1]


def test_masked_rows():
    assert sample.sample_row([-np.inf, np.nan], 0.3) == (-1, -np.inf)
    assert sample.sample_row([-np.inf, 0.0, np.nan], 0.9) == (1, 0.0)
    t, lp = sample.sample_row([np.inf, 0.0, np.inf], 0.6)
    assert t == 2 and lp == pytest.approx(np.log(0.5))


def test_scale_is_the_least_power_of_two_that_holds_the_rows():
    assert kv8.scale_for([448.0]) == 1.0
    assert kv8.scale_for([448.01]) == 2.0
    assert kv8.scale_for([224.0, -3.0]) == 0.5
    assert kv8.scale_for([np.inf, np.nan, 1.75]) == 2.0 ** -8
    assert kv8.scale_for([0.0]) == 2.0 ** -126
    for a in 2.0 ** np.random.default_rng(0).uniform(-60, 60, 200):
        s = kv8.scale_for([a])
        assert a <= 448 * s and a > 448 * s / 2


def test_append_error_is_half_a_step_and_order_hardly_matters():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((100, 16)) * 2.0 ** rng.uniform(-4, 4, (100, 1))
    runs = []
    for cuts in ([100], [1] * 100, [33, 1, 40, 26]):
        c, s, p = np.full((128, 16), 0x7F, np.uint8), np.ones(4), 0
        for n in cuts:
            kv8.append(c, s, p, x[p:p + n])
            p += n
        runs.append((c, s))
        y = kv8.decode(c, s, 100)
        smax = np.repeat(s, 32)[:100, None]
        # a half step of E4M3, twice where a grown scale rounded again
        assert np.all(np.abs(y - x) <= 2 * np.maximum(np.abs(x) * 2.0 ** -4, smax * 2.0 ** -10))
        assert np.all(c[100:] == 0x7F)
    for c, s in runs[1:]:
        assert np.array_equal(s, runs[0][1])
        d = e4m3_decode(c[:100]) - e4m3_decode(runs[0][0][:100])
        assert np.all(np.abs(d) <= 2.0 ** -9)   # one subnormal step at most


def test_attend_closed_forms():
    k = np.zeros((5, 4))
    v = np.arange(20.0).reshape(5, 4)
    q = np.ones((2, 4))
    o, _ = kv8.attend(q, k, v, 0, 1.0)
    assert np.allclose(o, v.mean(0))
    o, _ = kv8.attend(q, k, v, 2, 1.0)
    assert np.allclose(o, v[3:].mean(0))
    o, _ = kv8.attend(q, k[:0], v[:0], 0, 1.0)
    assert np.all(o == 0)


def test_kv8_model_holds_codes_and_stays_near_the_model():
    """Sliding-window layers are untouched; a full layer's entries are the
    decoded codes of the bf16 rows; an 8-bit cache changes logits, but little;
    and decoding token by token equals one call up to a subnormal step."""
    from oracle import Model
    from synthetic import TINY, make_prompt, make_weights
    w = make_weights(TINY, seed=0)
    toks = make_prompt(TINY, 1, 70)
    ref = Model(TINY, w, kv_mode="per_loop")
    z0 = ref.forward(toks, 2, all_logits=True)
    m = kv8.Kv8Model(TINY, w, kv_mode="per_loop")
    z1 = m.forward(toks, 2, all_logits=True)
    d = np.abs(z1 - z0).max()
    assert 1e-4 < d < 0.2
    full = [i for i, t in enumerate(TINY.layer_types) if t == 1]
    assert {k[0] for k in m.codes} == set(full) and full
    (i, slot, kind, b, h), (c, s) = next(iter(m.codes.items()))
    assert np.array_equal(m.cache[i, slot][kind][b, h, :70], kv8.decode(c, s, 70))
    m2 = kv8.Kv8Model(TINY, w, kv_mode="per_loop")
    m2.forward(toks[:, :37], 2)
    for t in range(37, 70):
        z = m2.decode_step(toks[:, t], 2)
    assert np.abs(z - z1[:, -1]).max() < d


def test_round_bf16():
    x = np.array([1.0, 1.00390625, 1.01171875, -3.14159, 1e-3])
    import torch
    want = torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).double().numpy()
    assert np.array_equal(kv8.round_bf16(x), want)
