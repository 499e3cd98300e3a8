"""The model on an 8-bit K/V cache (kv_fmt "e4m3") against the float64 oracle
with the same cache format, and generation with sampling.

Logits: the bound of the bf16 path (tests/gpu_util.py).  It leaves room for
codes that fall to the other side of a rounding border: storing k and v after
a random relative change of 2^-7, twice a bf16 rounding, moves the oracle's
tiny logits by at most 0.008.

Cached values: read from the cache buffer and held against the oracle's k and
v before they are stored: half an E4M3 step (2^-4 of the value, or 2^-10 of
the scale below the normal range) beside the bf16 path's own error, which the
bf16 parity tests bound at the logits; 2^-5 of the row's largest value is
allowed for it here.
"""
import numpy as np
import pytest
import torch

import looped_ngpt_b200 as lb
from oracle.kv8 import Kv8Model, append, decode
from oracle.quant import e4m3_decode
from synthetic import TINY, ModelShape, make_prompt, make_weights
from synthetic.kvgen import kv_rows
from tests.gpu_util import compare

pytestmark = pytest.mark.gpu

# the head layout of the 4B model (16 / 4 heads of 160) at a small width
WIDE = ModelShape(name="wide-heads", d=256, n_q_heads=16, n_kv_heads=4, head_dim=160, ffn=512,
                  vocab=512, n_in=1, n_rec=2, n_out=1, swa_window=16, layer_types=(0, 1, 0, 1))


@pytest.fixture(scope="module")
def tiny():
    w = make_weights(TINY, seed=0)
    return w, lb.DoryModel(TINY, w, device="cuda:0")


@pytest.fixture(autouse=True)
def no_device_error(tiny):
    yield
    assert tiny[1].sync_status() == 0


def run_both(shape, w, gm, B, chunks, k, kv_mode, steps, label):
    T = sum(chunks)
    prompt = make_prompt(shape, B, T, seed=60)
    ref = Kv8Model(shape, w, batch=B, kv_mode=kv_mode)
    cache = gm.new_cache(B, T + steps, max(chunks), kv_mode=kv_mode, max_loops=k, kv_fmt="e4m3")
    ws = gm.workspace(B, max(chunks))
    zg, zr, t0 = [], [], 0
    for c in chunks:
        z, _ = gm.prefill(cache, torch.from_numpy(prompt[:, t0:t0 + c].copy()).cuda(), k, ws,
                          logits_all=True)
        zg.append(z.cpu().numpy())
        zr.append(ref.forward(prompt[:, t0:t0 + c], k, all_logits=True))
        t0 += c
    zg, zr = np.concatenate(zg, 1), np.concatenate(zr, 1)
    tok = np.argmax(zr[:, -1], -1)
    dg, dr = [], []
    for _ in range(steps):
        dr.append(ref.decode_step(tok, k))
        z, _ = gm.decode_step(cache, torch.from_numpy(tok.astype(np.int32)).cuda(), k, ws)
        dg.append(z.cpu().numpy().copy())
        tok = np.argmax(dr[-1], -1)
    compare(zg, zr, f"{label} prefill")
    if steps:
        compare(np.array(dg), np.array(dr), f"{label} decode")
    return cache, ref


@pytest.mark.parametrize("kv_mode", ["per_loop", "last_loop"])
@pytest.mark.parametrize("B,chunks,k", [(1, (61,), 1), (2, (33, 30, 1), 2), (10, (40,), 2),
                                        (1, (1, 1, 70), 4)])
def test_tiny_parity(tiny, kv_mode, B, chunks, k):
    """Batches on the GEMV and the GEMM path, chunks that end inside a block
    and of one token, decode across the borders of blocks and pages."""
    run_both(TINY, tiny[0], tiny[1], B, chunks, k, kv_mode, 5, f"e4m3 {kv_mode} B={B} k={k}")


@pytest.mark.parametrize("hd,G", [(160, 4), (128, 8), (128, 1), (64, 2)])
def test_other_head_layouts(hd, G):
    H = 2 if hd * G * 2 % 256 == 0 else 4
    shape = WIDE if hd == 160 else ModelShape(
        name="heads", d=256, n_q_heads=H * G, n_kv_heads=H, head_dim=hd, ffn=256, vocab=256, n_in=1,
        n_rec=1, n_out=1, swa_window=16, layer_types=(0, 1, 1))
    w = make_weights(shape, seed=3)
    gm = lb.DoryModel(shape, w, device="cuda:0")
    run_both(shape, w, gm, 2, (50, 17), 2, "last_loop", 4, f"e4m3 heads {hd}x{G}")


def pages_of(gm, cache, shape, slot):
    """Codes and scales of one full-attention slot from the cache buffer: a
    256-byte header, the block table, then per slot K, V and (8-bit) their
    scales, each a multiple of 256 bytes."""
    up = lambda n: (n + 255) & ~255  # noqa: E731
    B, P = cache.batch, -(-cache.max_ctx // 64)
    tr = 64
    cap = -(-min(cache.max_ctx, shape.swa_window + cache.max_chunk - 1) // tr) * tr
    at = 256 + up(B * P * 4)
    n_rec = range(shape.n_in, shape.n_in + shape.n_rec)
    for i in range(shape.n_blocks):
        for t in range(slot[1] + 1 if i == slot[0] else
                       (cache.loops if i in n_rec and cache.kv_mode == "per_loop" else 1)):
            if shape.layer_types[i] == 0:
                at += 2 * up(B * shape.n_kv_heads * cap * shape.head_dim * 2)
                continue
            rows = B * P * shape.n_kv_heads
            nb, ns = up(rows * 64 * shape.head_dim), up(rows * 8)
            if (i, t) == slot:
                buf = cache.buf.cpu().numpy()
                code = [buf[at + o:at + o + rows * 64 * shape.head_dim].reshape(
                    B, P, shape.n_kv_heads, 64, shape.head_dim) for o in (0, nb)]
                sc = [buf[at + 2 * nb + o:at + 2 * nb + o + rows * 8].view(np.float32).reshape(
                    B, P, shape.n_kv_heads, 2) for o in (0, ns)]
                return code, sc
            at += 2 * (nb + ns)
    raise AssertionError(slot)


@pytest.mark.parametrize("kv_mode", ["per_loop", "last_loop"])
def test_cache_holds_the_models_rows(tiny, kv_mode):
    w, gm = tiny

    class Seen(Kv8Model):
        stored = {}

        def store_kv(self, i, slot, pos, k, v):
            for kind, x in enumerate((k, v)):
                for t, p in enumerate(pos):
                    self.stored[i, slot, kind, int(p)] = x[:, :, t].copy()
            return super().store_kv(i, slot, pos, k, v)

    B, T, k, steps = 2, 40, 2, 30
    prompt = make_prompt(TINY, B, T, seed=61)
    ref = Seen(TINY, w, batch=B, kv_mode=kv_mode)
    ref.forward(prompt, k)
    cache = gm.new_cache(B, T + steps, T, kv_mode=kv_mode, max_loops=k, kv_fmt="e4m3")
    cache.loops = k
    ws = gm.workspace(B, T)
    gm.prefill(cache, torch.from_numpy(prompt).cuda(), k, ws)
    for j in range(steps):
        tok = np.array([j, 3 * j], dtype=np.int32)
        ref.decode_step(tok, k)
        gm.decode_step(cache, torch.from_numpy(tok).cuda(), k, ws)
    torch.cuda.synchronize()
    gin, grec, gout = TINY.block_groups()
    for i in [b for b, t in enumerate(TINY.layer_types) if t == 1]:
        loops = range(1, k + 1) if i in grec and kv_mode == "per_loop" else [0]
        for s in loops:
            code, sc = pages_of(gm, cache, TINY, (i, s - 1 if s else 0))
            for kind in range(2):
                # [B, P, H, 64, hd] -> [B, H, positions, hd]
                x = e4m3_decode(code[kind]) * np.repeat(sc[kind], 32, axis=3)[..., None]
                x = x.transpose(0, 2, 1, 3, 4).reshape(B, TINY.n_kv_heads, -1, TINY.head_dim)
                scale = np.repeat(sc[kind], 32, axis=3).transpose(0, 2, 1, 3).reshape(
                    B, TINY.n_kv_heads, -1)
                for p in range(T + steps):
                    want = ref.stored[i, s, kind, p]
                    err = np.abs(x[:, :, p] - want)
                    top = np.abs(want).max(-1, keepdims=True)
                    bound = np.maximum(np.abs(want) * 2.0 ** -4, scale[:, :, p, None] * 2.0 ** -10)
                    assert np.all(err <= bound + top * 2.0 ** -5), (i, s, kind, p, err.max())
                    # and the scale is a power of two that the block's rows need
                    m, _ = np.frexp(scale[:, :, p])
                    assert np.all(m == 0.5) and np.all(top[..., 0] <= 460 * scale[:, :, p])


@pytest.mark.parametrize("kv_mode", ["per_loop", "last_loop"])
def test_mixed_loop_counts(tiny, kv_mode):
    w, gm = tiny
    loops, T, steps = (1, 3, 2), 34, 4
    prompt = make_prompt(TINY, 3, T, seed=62)
    rl = torch.tensor(loops, dtype=torch.int32, device="cuda:0")
    cache = gm.new_cache(3, T + steps, T, kv_mode=kv_mode, max_loops=3, kv_fmt="e4m3")
    ws = gm.workspace(3, T)
    zg, _ = gm.prefill_mixed(cache, torch.from_numpy(prompt).cuda(), rl, ws, logits_all=True)
    refs = [Kv8Model(TINY, w, kv_mode=kv_mode) for _ in range(3)]
    zr = np.concatenate([refs[b].forward(prompt[b:b + 1], loops[b], True) for b in range(3)])
    tok = np.argmax(zr[:, -1], -1)
    dg, dr = [], []
    for _ in range(steps):
        dr.append(np.concatenate([refs[b].decode_step(tok[b:b + 1], loops[b]) for b in range(3)]))
        g, _ = gm.decode_step_mixed(cache, torch.from_numpy(tok.astype(np.int32)).cuda(), rl, 3, ws)
        dg.append(g.cpu().numpy().copy())
        tok = np.argmax(dr[-1], -1)
    compare(zg.cpu().numpy(), zr, f"e4m3 mixed prefill {kv_mode}")
    compare(np.array(dg), np.array(dr), f"e4m3 mixed decode {kv_mode}")


def test_prefix_copy_and_reset(tiny):
    """A copied prefix continues like the oracle that ran prefix and suffix as
    two calls; a reset cache starts over as a new one does, bit for bit."""
    w, gm = tiny
    k, Tp, Ts = 2, 45, 10
    prefix, suffix = make_prompt(TINY, 1, Tp, seed=63), make_prompt(TINY, 2, Ts, seed=64)
    src = gm.new_cache(1, 64, Tp, max_loops=k, kv_fmt="e4m3")
    ws1, ws2 = gm.workspace(1, Tp), gm.workspace(2, Tp)
    gm.prefill(src, torch.from_numpy(prefix).cuda(), k, ws1)
    dst = gm.new_cache(2, 128, Tp, max_loops=k, kv_fmt="e4m3")
    dst.copy_prefix_from(src, 0, Tp)
    zg, _ = gm.prefill(dst, torch.from_numpy(suffix).cuda(), k, ws2, logits_all=True)
    ref = Kv8Model(TINY, w, batch=2, kv_mode="last_loop")
    ref.forward(np.repeat(prefix, 2, axis=0), k)
    compare(zg.cpu().numpy(), ref.forward(suffix, k, all_logits=True), "e4m3 prefix copy")
    with pytest.raises(lb.DoryError) as e:
        gm.new_cache(2, 128, Tp, max_loops=k).copy_prefix_from(src, 0, Tp)
    assert e.value.code == -3
    dst.reset()
    new = gm.new_cache(2, 128, Tp, max_loops=k, kv_fmt="e4m3")
    z1, _ = gm.prefill(dst, torch.from_numpy(suffix).cuda(), k, ws2)
    z2, _ = gm.prefill(new, torch.from_numpy(suffix).cuda(), k, ws2)
    assert torch.equal(z1, z2)


@pytest.mark.parametrize("n_ctx", [40, 1000])
def test_synthetic_context_and_eager_launches(tiny, monkeypatch, n_ctx):
    """A cache bound for one-token calls only, filled with synthetic entries,
    decodes like the oracle holding them; replayed graphs give the bits of
    eager launches."""
    w, gm = tiny
    B, seed, k = 2, 2, 2
    ref = Kv8Model(TINY, w, batch=B, kv_mode="last_loop")
    for i in range(TINY.n_blocks):
        K = np.zeros((B, TINY.n_kv_heads, n_ctx, TINY.head_dim))
        V = np.zeros_like(K)
        for b in range(B):
            for h in range(TINY.n_kv_heads):
                for kind, (x, out) in enumerate(zip(kv_rows(TINY, seed, i, 0, b, h,
                                                            np.arange(n_ctx)), (K, V))):
                    out[b, h] = x
                    if TINY.layer_types[i] == 1:
                        cap = -(-n_ctx // 32) * 32
                        c, s = np.zeros((cap, TINY.head_dim), np.uint8), np.zeros(cap // 32)
                        append(c, s, 0, x)
                        ref.codes[i, 0, kind, b, h] = c, s
                        out[b, h] = decode(c, s, n_ctx)
        ref.cache[i, 0] = (K, V)
    ref.n_ctx = n_ctx
    monkeypatch.setenv("DORY_NO_GRAPH", "1")
    eager = lb.DoryModel(TINY, dict(gm.tensors), device="cuda:0")
    runs = []
    for model in (gm, eager):
        cache = model.new_cache(B, n_ctx + 8, 1, max_loops=k, kv_fmt="e4m3")
        cache.fill_synthetic(n_ctx, seed)
        ws = model.workspace(B, 1)
        out = []
        for j in range(6):
            tok = torch.tensor([j, 100 + j], dtype=torch.int32, device="cuda")
            out.append(model.decode_step(cache, tok, k, ws)[0].cpu().numpy().copy())
        runs.append(np.array(out))
    assert np.array_equal(runs[0], runs[1])
    zr = [ref.decode_step(np.array([j, 100 + j]), k) for j in range(6)]
    compare(runs[0], np.array(zr), f"e4m3 synthetic {n_ctx}")


def test_long_context_matches_the_bf16_cache_closely():
    """Wide heads, 20000 cached tokens: the two formats' logits differ by the
    quantisation alone.  Scores are sums of 160 products with independent
    relative errors of at most 2^-4 (2.6% rms), values likewise, averaged over
    20000 keys: far below the bf16 path's own bound."""
    w = make_weights(WIDE, seed=4)
    gm = lb.DoryModel(WIDE, w, device="cuda:0")
    z = {}
    for fmt in ("bf16", "e4m3"):
        cache = gm.new_cache(3, 20010, 1, max_loops=2, kv_fmt=fmt)
        cache.fill_synthetic(20000, seed=5)
        ws = gm.workspace(3, 1)
        tok = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
        for _ in range(3):
            out = gm.decode_step(cache, tok, 2, ws)[0]
        z[fmt] = out.cpu().numpy().copy()
        size = cache.nbytes
    compare(z["e4m3"], z["bf16"], "e4m3 against bf16 at 20000 tokens")
    assert gm.sync_status() == 0
    bf16 = gm.new_cache(3, 20010, 1, max_loops=2).nbytes
    assert size < 0.56 * bf16


def test_cache_format_refusals(tiny):
    w, gm = tiny
    import ctypes
    from looped_ngpt_b200 import _lib
    lib, n = _lib.load(), ctypes.c_int64()
    assert lib.dory_kv_cache_bytes_fmt(gm.handle, 1, 64, 8, 1, 1, 2, ctypes.byref(n)) == -1
    assert lib.dory_kv_cache_bytes_fmt(gm.handle, 4000, 64, 8, 1, 1, 1, ctypes.byref(n)) == -2
    cache = gm.new_cache(1, 64, 8, kv_mode="per_loop", max_loops=4, kv_fmt="e4m3")
    gm.prefill(cache, torch.zeros((1, 8), dtype=torch.int32, device="cuda"), 4, gm.workspace(1, 8))
    with pytest.raises(lb.DoryError) as e:
        gm.spec_decode_step(cache, torch.zeros(1, dtype=torch.int32, device="cuda"), 3, 1, 4,
                            gm.spec_workspace(1, 3))
    assert e.value.code == -2


@pytest.mark.parametrize("kv_fmt", ["bf16", "e4m3"])
def test_generate(tiny, kv_fmt):
    """Greedy generation is the argmax loop; sampled tokens are those that
    lb.sample draws from the same logits, with their log-probabilities."""
    w, gm = tiny
    B, T, n, k = 2, 12, 9, 2
    prompt = torch.from_numpy(make_prompt(TINY, B, T, seed=65)).cuda()
    u = torch.rand(n, B, device="cuda")
    for opts in (dict(), dict(temperature=0.9, top_k=40, top_p=0.95, min_p=0.01),
                 dict(temperature=torch.tensor([0.0, 1.3], device="cuda"), top_k=3)):
        got, lp = gm.generate(prompt, n, k, uniform=u, kv_fmt=kv_fmt, logprobs=True, **opts)
        cache = gm.new_cache(B, T + n, T, max_loops=k, kv_fmt=kv_fmt)
        ws = gm.workspace(B, T)
        full = lambda x, dt: (x if isinstance(x, torch.Tensor)  # noqa: E731
                              else torch.full((B,), x, dtype=dt, device="cuda"))
        z, am = gm.prefill(cache, prompt, k, ws)
        for i in range(n):
            tok, l = lb.sample(z, u[i], full(opts.get("temperature", 0.0), torch.float32),
                               full(opts.get("top_k", 0), torch.int32),
                               full(opts.get("top_p", 1.0), torch.float32),
                               full(opts.get("min_p", 0.0), torch.float32), logprobs=True)
            assert torch.equal(tok, got[:, i]) and torch.equal(l, lp[:, i])
            if not opts:
                assert torch.equal(tok, am) and torch.all(l == 0)
            z, am = gm.decode_step(cache, tok, k, ws)
    assert gm.generate(prompt, 3, k, temperature=1.0).shape == (B, 3)


def test_generate_refusals(tiny):
    _, gm = tiny
    p = torch.from_numpy(make_prompt(TINY, 2, 12, seed=66)).cuda()
    u = torch.rand(3, 2, device="cuda")
    for prompt, kw in ((p.long(), {}), (p.cpu(), {}), (p[0], {}), (p[:, ::2], {}),
                       (p[:, :0], {}), (p, dict(uniform=u[:2])), (p, dict(uniform=u.t()))):
        with pytest.raises(ValueError):
            gm.generate(prompt, 3, 2, **kw)
    assert gm.generate(p, 0, 2).shape == (2, 0)


def test_generate_where_nothing_can_be_drawn(tiny):
    """All logits NaN: every token is -1, the log-probabilities are -inf, and
    no device error is left for a later call to report."""
    w, gm = tiny
    bad = lb.DoryModel(TINY, dict(w, s_z=np.full_like(w["s_z"], np.nan)), device="cuda:0")
    p = torch.from_numpy(make_prompt(TINY, 2, 12, seed=67)).cuda()
    for opts in (dict(), dict(temperature=0.9, top_k=5)):
        tok, lp = bad.generate(p, 4, 2, logprobs=True, **opts)
        assert torch.all(tok == -1) and torch.all(lp == -np.inf)
        assert bad.sync_status() == 0


def test_generate_keeps_the_other_sequences_of_a_batch(tiny, monkeypatch):
    """A sequence that stops is -1 from there on, whatever its later logits
    are; the others go on as they would."""
    _, gm = tiny
    p = torch.from_numpy(make_prompt(TINY, 3, 12, seed=68)).cuda()
    u = torch.rand(6, 3, device="cuda")
    want, wlp = gm.generate(p, 6, 2, uniform=u, temperature=0.9, logprobs=True)
    from looped_ngpt_b200 import model as module
    real, calls = module.sample, []

    def stops(logits, *args, **kw):
        calls.append(None)
        if len(calls) == 3:
            logits = logits.clone()
            logits[1] = -np.inf
        return real(logits, *args, **kw)

    monkeypatch.setattr(module, "sample", stops)
    tok, lp = gm.generate(p, 6, 2, uniform=u, temperature=0.9, logprobs=True)
    for b in (0, 2):
        assert torch.equal(tok[b], want[b]) and torch.equal(lp[b], wlp[b])
    assert torch.equal(tok[1, :2], want[1, :2])
    assert torch.all(tok[1, 2:] == -1) and torch.all(lp[1, 2:] == -np.inf)


def test_generate_refuses_before_anything_is_enqueued(tiny, monkeypatch):
    _, gm = tiny
    p = torch.from_numpy(make_prompt(TINY, 2, 12, seed=69)).cuda()
    u = torch.rand(3, 2, device="cuda")
    monkeypatch.setattr(gm, "prefill", None)       # a call of it would raise TypeError
    f = torch.ones(2, device="cuda")
    for kw in (dict(uniform=u.double()), dict(uniform=u.cpu()), dict(uniform=u.cpu().numpy()),
               dict(temperature=f.double()), dict(temperature=f[:1]), dict(top_k=f),
               dict(top_p=f.cpu()), dict(min_p=f[None])):
        with pytest.raises(ValueError):
            gm.generate(p, 3, 2, **kw)
    monkeypatch.undo()
    # uniforms in any layout
    a = gm.generate(p, 3, 2, uniform=u, temperature=1.0)
    b = gm.generate(p, 3, 2, uniform=u.t().contiguous().t(), temperature=1.0)
    assert torch.equal(a, b)
