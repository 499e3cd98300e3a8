"""Token sampling on the GPU against the float64 oracle on the same logits,
options and uniforms: tokens equal, log-probabilities within the rounding of
their f32 result (2^-24 relative) plus 1e-9 for sums of up to 2^18 weights in
64 bits (2^18 * 2^-52 < 1e-10, and the weights' own error)."""
import numpy as np
import pytest
import torch

import looped_ngpt_b200 as lb
from oracle import sample as oracle

pytestmark = pytest.mark.gpu


def run(z, u, T=None, k=None, p=None, mp=None, **kw):
    """GPU and oracle on one batch; options are arrays, one value per row."""
    z, u = np.asarray(z, np.float32), np.asarray(u, np.float32)
    dev = lambda a, dt: None if a is None else torch.tensor(  # noqa: E731
        np.asarray(a), dtype=dt, device="cuda")
    zt = kw.pop("logits", None)
    zt = dev(z, torch.float32) if zt is None else zt
    tok, lp = lb.sample(zt, dev(u, torch.float32),
                        temperature=dev(T, torch.float32), top_k=dev(k, torch.int32),
                        top_p=dev(p, torch.float32), min_p=dev(mp, torch.float32),
                        logprobs=True, **kw)
    tok, lp = tok.cpu().numpy(), lp.cpu().numpy().astype(np.float64)
    f32 = lambda a, b, d: d if a is None else float(np.float32(a[b]))  # noqa: E731
    for b in range(len(z)):
        t, l = oracle.sample_row(z[b], u[b], f32(T, b, 1.0),
                                 0 if k is None else int(k[b]), f32(p, b, 1.0),
                                 f32(mp, b, 0.0))
        assert tok[b] == t, (b, tok[b], t)
        assert lp[b] == l or abs(lp[b] - l) <= 2.0 ** -23 * abs(l) + 1e-9, (b, lp[b], l)
    return tok


def logits(rng, B, V, peak=1.0):
    return (-peak * np.log1p(rng.random((B, V)) * V) + 0.5 * rng.standard_normal((B, V))
            ).astype(np.float32)


@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 1024, 4097, 50257, 131072, 131071])
def test_options(V):
    rng = np.random.default_rng(V)
    B = 24 if V < 50000 else 12
    z = logits(rng, B, V, 1.2)
    u = rng.random(B)
    pick = lambda a: [a[rng.integers(len(a))] for _ in range(B)]  # noqa: E731
    run(z, u)
    run(z, u, T=[0.7] * B, p=[0.9] * B)
    run(z, u, k=[50] * B, p=[0.95] * B, T=[0.8] * B)
    run(z, u, T=pick([0.0, -1.0, 0.3, 1.0, 1.7, 50.0, np.nan]), k=pick([0, -3, 1, 2, 40, 1999, 1 << 30]),
        p=pick([1.0, 1.5, 0.999, 0.9, 0.4, 1e-3, 0.0, -1.0, np.nan]),
        mp=pick([0.0, -1.0, 1e-4, 0.05, 0.5, 1.0, 2.0, np.nan]))


@pytest.mark.parametrize("V", [7, 3000, 40000])
def test_ties_go_to_the_lowest_index(V):
    rng = np.random.default_rng(V)
    B = 16
    z = np.round(rng.standard_normal((B, V)) * 2) / 2      # few distinct values
    z[3] = 1.25                                            # all equal
    z[4] = np.where(rng.random(V) < 0.5, 0.0, -0.0)        # equal despite the sign
    u = rng.random(B)
    run(z, u, k=[max(1, V // 3)] * B)
    run(z, u, p=[0.5] * B)
    run(z, u, p=[0.25] * B, k=[V // 2 + 1] * B, mp=[0.01] * B)
    run(z, u, T=[0.0] * B)


def test_adversarial_ranges():
    """Logits whose cutoffs lie in a tiny part of their range."""
    rng = np.random.default_rng(5)
    V, B = 20011, 12
    z = rng.random((B, V)).astype(np.float32)
    z[0, 17] = 1000.0                       # one outlier, the rest in one bin
    z[1, 11] = -3.0e38
    z[2, 5], z[2, 9] = 3.0e38, -3.0e38
    z[3] = 1.0 + np.arange(V) * 2.0 ** -20  # neighbours
    z[4] = -(2.0 ** -np.linspace(-100, 120, V))      # every binade
    z[5] = 1e-40 * rng.random(V)            # subnormal logits
    z[6] = np.nextafter(np.float32(2), np.float32(3)) - (np.arange(V) % 2) * 2.0 ** -22
    u = rng.random(B)
    for T in (1.0, 1e-3, 1e4, 1e-30):
        run(z, u, T=[T] * B)
        run(z, u, T=[T] * B, k=[1 + 997 * b for b in range(B)])
        run(z, u, T=[T] * B, p=[0.05 + 0.08 * b for b in range(B)])
        run(z, u, T=[T] * B, k=[5000] * B, p=[0.7] * B, mp=[1e-3] * B)


def test_masked_rows_and_special_values():
    rng = np.random.default_rng(7)
    V, B = 5000, 9
    z = logits(rng, B, V)
    z[0] = -np.inf
    z[1] = np.nan
    z[2] = -np.inf
    z[2, 4321] = -5.0                       # one token left
    z[3, ::2] = np.nan
    z[4, 1:] = -np.inf
    z[5, [7, 70, 700]] = np.inf
    z[6, 2500:] = -np.inf
    u = rng.random(B)
    tok = run(z, u)
    assert list(tok[:3]) == [-1, -1, 4321]
    run(z, u, k=[10] * B)
    run(z, u, p=[0.6] * B)
    run(z, u, T=[0.0] * B)
    run(z, u, k=[4000] * B, mp=[0.001] * B)


@pytest.mark.parametrize("T", [1e36, 1e37, 3e38, np.inf])
def test_huge_temperatures_leave_masked_tokens_out(T):
    """m - 44 T leaves f32's range; only finite logits (and +inf) may be drawn."""
    rng = np.random.default_rng(11)
    V, B = 5000, 6
    z = logits(rng, B, V)
    z[:, ::3] = -np.inf
    z[1, 1::3] = np.nan
    z[2, 300:] = -np.inf
    z[3, 44] = np.inf
    z[4, 100:200] = -3.0e38
    z[5, 7], z[5, 8] = 3.0e38, -3.0e38
    u = [0.0, 0.3, 0.999, 0.5, 0.7, 1.0]
    # tokens below e^-44 of the largest weight are not drawn, not even by u = 1
    # (row 5: e^-300 at T = 1e36), which the oracle would do
    z64 = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    m = z64.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        drawn = np.where(((z64 - m) / float(np.float32(T)) < -44) | (z64 < m) & (m == np.inf),
                         -np.inf, z)
    on_gpu = torch.tensor(z, device="cuda")
    for kw in ({}, dict(k=[900] * B), dict(p=[0.6] * B), dict(mp=[0.5] * B, p=[0.9] * B),
               dict(k=[2000] * B, mp=[1e-3] * B, p=[0.8] * B)):
        run(drawn, u, T=[T] * B, logits=on_gpu, **kw)


def test_uniform_at_its_ends():
    rng = np.random.default_rng(8)
    z = logits(rng, 6, 3001)
    z[:, -5:] = -np.inf
    z[:, :3] = -np.inf
    u = [0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, np.nan]
    run(z, u)
    run(z, u, k=[17] * 6)


def test_strided_rows_given_outputs_and_empty_batch():
    rng = np.random.default_rng(9)
    big = torch.full((8, 4100), 1e9, device="cuda")
    z = logits(rng, 4, 4001)
    view = big[1::2, 3:4004]                # rows apart, not 16-byte aligned
    view.copy_(torch.tensor(z))
    tok = torch.full((4,), -7, dtype=torch.int32, device="cuda")
    run(z, rng.random(4), k=[9] * 4, logits=view, tokens=tok)
    run(z, rng.random(4), logits=view)
    t, lp = lb.sample(torch.empty(0, 5, device="cuda"), torch.empty(0, device="cuda"))
    assert t.shape == (0,) and lp is None


@pytest.mark.parametrize("V", [262143, 262144, 262145])
def test_around_the_largest_cluster(V):
    """The longest rows a cluster holds, flat and peaked, and one logit more."""
    rng = np.random.default_rng(V)
    B = 4
    z = np.stack([logits(rng, 1, V, p)[0] for p in (0.0, 0.7, 1.5, 3.0)])
    z[0] = 0.5                              # all equal
    u = rng.random(B)
    for kw in ({}, dict(p=[0.9] * B), dict(k=[50] * B, p=[0.95] * B), dict(k=[200000] * B),
               dict(mp=[0.01] * B, p=[0.5] * B)):
        run(z, u, T=[0.8] * B, **kw)


def test_large_vocabulary():
    """Rows too large for the shared memory of one cluster."""
    rng = np.random.default_rng(10)
    V = 1_000_003
    z = rng.standard_normal((2, V)).astype(np.float32)
    u = rng.random(2)
    run(z, u)
    run(z, u, k=[100_000, 7], p=[0.8, 0.9])
    run(z, u, p=[0.3, 0.99])


def test_frequencies_follow_the_distribution():
    """20000 uniforms on an even grid hit each token within one grid step of
    its probability (the inverse CDF maps the grid onto the borders)."""
    z = np.log(np.array([0.05, 0.4, 0.15, 0.1, 0.3]))
    n = 20000
    u = (torch.arange(n, device="cuda").double() / n).float()
    zt = torch.tensor(z, dtype=torch.float32, device="cuda").expand(n, 5).contiguous()
    tok, _ = lb.sample(zt, u)
    f = np.bincount(tok.cpu().numpy(), minlength=5) / n
    # 1/n per border, and the f32 rounding of logits and uniforms
    assert np.abs(f - np.exp(z)).max() <= 2.0 / n + 1e-6


def test_refusals():
    z = torch.zeros(2, 8, device="cuda")
    u = torch.zeros(2, device="cuda")
    for bad in (dict(logits=z.half()), dict(logits=z[0]), dict(logits=z.t()),
                dict(uniform=u.double()), dict(uniform=u[:1]),
                dict(top_k=u), dict(temperature=u.cpu()), dict(min_p=u[None]),
                dict(logits=z[:1].expand(2, 8)), dict(logits=z[:, :0]),
                dict(tokens=u), dict(logprobs=z)):
        kw = dict(logits=z, uniform=u) | bad
        with pytest.raises(ValueError):
            lb.sample(kw.pop("logits"), kw.pop("uniform"), **kw)


def test_other_stream_and_graph_replay():
    rng = np.random.default_rng(11)
    z = torch.tensor(logits(rng, 3, 9000), device="cuda")
    u = torch.rand(3, device="cuda")
    p = torch.full((3,), 0.8, device="cuda")
    want, lp0 = lb.sample(z, u, top_p=p, logprobs=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, lp1 = lb.sample(z, u, top_p=p, logprobs=True, stream=s)
    s.synchronize()
    assert torch.equal(want, got) and torch.equal(lp0, lp1)
    tok, lp = torch.empty_like(want), torch.empty_like(lp0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lb.sample(z, u, top_p=p, tokens=tok, logprobs=lp)
    for seed in (1, 2):
        z.copy_(torch.tensor(logits(np.random.default_rng(seed), 3, 9000)))
        u.copy_(torch.rand(3))
        g.replay()
        want, lp0 = lb.sample(z, u, top_p=p, logprobs=True)
        assert torch.equal(want, tok) and torch.equal(lp0, lp)


@pytest.mark.parametrize("V", [262144, 262145])
def test_infinite_temperature_and_logits_of_long_rows(V):
    """Tokens at +inf share the row at any temperature, in rows of one cluster
    and in longer ones."""
    rng = np.random.default_rng(12)
    z = logits(rng, 3, V)
    z[0, [5, 70000, 200000]] = np.inf
    z[1, [9, 250000]] = np.inf
    z[1, 11] = -np.inf
    z[2, ::2] = -np.inf
    on_gpu = torch.tensor(z, device="cuda")
    drawn = np.where((z == np.inf) | (z.max(1, keepdims=True) != np.inf), z, -np.inf)
    for u in ([0.1, 0.1, 0.2], [0.5, 0.6, 0.9]):
        for T in (1.0, np.inf):
            run(drawn, u, T=[T] * 3, logits=on_gpu)
            run(drawn, u, T=[T] * 3, p=[0.9] * 3, logits=on_gpu)


@pytest.mark.parametrize("V", [5000, 262145])
def test_tokens_far_below_the_largest_are_not_drawn(V):
    """Weights below e^-44 of the largest: not at the ends of the uniforms
    either, where the oracle would draw them."""
    z = np.zeros((4, V), np.float32)
    z[:2, [0, V - 1]] = -60.0
    z[:2, [1, V - 2]] = -30.0
    z[2:, [0, V - 1]] = -20.0
    z[2:, [1, V - 2]] = -10.0
    T = [1.0, 1.0, 0.4, 0.4]                # -50 and -25
    drawn = z.copy()
    drawn[:, [0, V - 1]] = -np.inf
    u = [0.0, 1.0, 0.0, 1.0]
    on_gpu = torch.tensor(z, device="cuda")
    for kw in ({}, dict(k=[V - 1] * 4), dict(mp=[1e-30] * 4)):
        tok = run(drawn, u, T=T, logits=on_gpu, **kw)
        assert kw.get("k") or list(tok) == [1, V - 2] * 2


def test_long_rows_of_equal_logits():
    """How many of a million equal tokens a top-p keeps is not counted one by
    one."""
    V = 1 << 20
    z = np.zeros((4, V), np.float32)
    z[2:, ::2] = 1.0
    run(z, [0.2, 0.999, 0.4, 1.0], p=[0.5, 0.9, 0.6, 0.95])
    run(z, [0.2, 0.999, 0.4, 1.0], p=[1e-9, 0.0, 1.0 - 2.0 ** -24, 0.3], k=[0, 0, 0, V // 2 + 5])


@pytest.mark.parametrize("T", [1.0, 0.7])
def test_borders_are_off_by_less_than_2_to_the_minus_36(T):
    """Two tokens of weights w and 1: token 0 is drawn for u < w / (1 + w).  Rows
    are picked whose border lies between 2^-36 and 2^-34 of itself from the
    nearest f32 uniform: a relative error of 2^-36 in w (2^-36 / (1 + w) in the
    border) must not change the side; f64 sums and products add 2^-52."""
    rng = np.random.default_rng(13)
    z0 = -rng.uniform(0.01, 20.0, 1 << 22).astype(np.float32)
    w = np.exp(z0.astype(np.longdouble) / np.longdouble(np.float32(T)))
    border = w / (1 + w)
    u = border.astype(np.float32)
    rel = (border - u.astype(np.longdouble)) / border
    pick = np.flatnonzero((np.abs(rel) >= 2.0 ** -36) & (np.abs(rel) <= 2.0 ** -34))
    assert len(pick) > 1000
    z = np.full((len(pick), 3), -np.inf, np.float32)
    z[:, 0], z[:, 1] = z0[pick], 0.0
    past = rel[pick] <= 0                          # u at the border or past it: token 1
    dev = lambda a, dt: torch.tensor(a, dtype=dt, device="cuda")  # noqa: E731
    n, zt, ut = len(pick), dev(z, torch.float32), dev(u[pick], torch.float32)
    Tt = torch.full((n,), T, device="cuda")
    for kw in ({}, dict(top_k=torch.full((n,), 2, dtype=torch.int32, device="cuda")),
               dict(min_p=torch.full((n,), 1e-12, device="cuda"))):
        # (min-p leaves out token 0 where it is lighter than that)
        out = w[pick] < np.float32(1e-12) if "min_p" in kw else False
        want = torch.tensor(past | out).int()
        tok, _ = lb.sample(zt, ut, temperature=Tt, **kw)
        assert torch.equal(tok.cpu(), want), (kw, int((tok.cpu() != want).sum()))
