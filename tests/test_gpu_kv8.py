"""The 8-bit K/V cache operators on the GPU against the float64 oracle.

append: codes and scales equal bit for bit (every step is exact or one
correctly rounded conversion).

attend: with A = sum_j p_j |v_j| the output may be off by its bf16 rounding,
2^-8 |o| (half a step), and by the rounding of the weights: each p_j to 11
bits (2^-11), and p_j through its f32 score, whose sum of head_dim <= 160
products errs by at most 160 * 2^-24 * sum |q k| * scale, below 2^-12 for the
|scores| <= 16 drawn here; together below 2^-10 A.
"""
import numpy as np
import pytest
import torch

import looped_ngpt_b200 as lb
from oracle import kv8 as oracle
from synthetic import TINY, make_weights

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def model():
    """Any model: its sync_status reads the device's status word."""
    return lb.DoryModel(TINY, make_weights(TINY, seed=0), device="cuda:0")


@pytest.fixture(autouse=True)
def no_device_error(model):
    yield
    assert model.sync_status() == 0


def bf(x):
    """float64 -> the bf16 values a GPU tensor of it holds."""
    return torch.tensor(np.asarray(x), dtype=torch.float32).to(torch.bfloat16)


def pool(rng, B, P, H, hd, extra=3, fill=0x7F):
    """Pages in a shuffled order, all NaN codes (or random bytes)."""
    n = B * P + extra
    table = rng.permutation(n)[:B * P].reshape(B, P).astype(np.int32)
    if fill is None:
        codes = [rng.integers(0, 256, (n, H, 64, hd)).astype(np.uint8) for _ in "kv"]
    else:
        codes = [np.full((n, H, 64, hd), fill, np.uint8) for _ in "kv"]
    return codes, [np.ones((n, H, 2), np.float32) for _ in "kv"], table


def pages_of(codes, scales, table):
    t = lambda a: torch.tensor(a, device=DEV)  # noqa: E731
    return lb.KV8Pages(t(codes[0]), t(codes[1]), t(scales[0]), t(scales[1]), t(table))


@pytest.fixture(params=["pairs", "runs"])
def layout(request, monkeypatch):
    """attend takes a cluster per pair where the block table is short, and
    equal runs over all pairs where it is long: the same pages behind both."""
    if request.param == "runs":
        short = pages_of

        def long(codes, scales, table):
            more = np.zeros((len(table), 5000), np.int32)
            return short(codes, scales, np.concatenate([table, more], axis=1))

        monkeypatch.setitem(globals(), "pages_of", long)
    return request.param


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def seq_view(codes, scales, table, b, h):
    """One sequence's and head's codes [P * 64, hd] and scales [P * 2]."""
    return (np.concatenate([codes[pg, h] for pg in table[b]]),
            np.concatenate([scales[pg, h] for pg in table[b]]).astype(np.float64))


def oracle_append(codes, scales, table, rows, pos, n):
    for kind in range(2):
        for b in range(len(table)):
            for h in range(codes[kind].shape[1]):
                c, s = seq_view(codes[kind], scales[kind], table, b, h)
                oracle.append(c, s, int(pos[b]), rows[kind][b, :n[b], h])
                for i, pg in enumerate(table[b]):
                    codes[kind][pg, h] = c[64 * i:64 * i + 64]
                    scales[kind][pg, h] = s[2 * i:2 * i + 2]


def same_pages(pages, codes, scales):
    torch.cuda.synchronize()
    assert np.array_equal(pages.k.cpu().numpy(), codes[0])
    assert np.array_equal(pages.v.cpu().numpy(), codes[1])
    assert np.array_equal(pages.k_scale.cpu().numpy(), scales[0])
    assert np.array_equal(pages.v_scale.cpu().numpy(), scales[1])


def rows_of(rng, B, T, H, hd, spread=3.0):
    x = rng.standard_normal((2, B, T, H, hd)) * 2.0 ** rng.uniform(-spread, spread, (2, B, T, 1, 1))
    return bf(x)


@pytest.mark.parametrize("hd,H", [(64, 1), (128, 2), (160, 4)])
def test_append_steps(hd, H):
    """Calls of every kind behind one another: single tokens, ragged padded
    batches, empty ones, runs that end inside and at the end of a page."""
    rng = np.random.default_rng(hd)
    B, P = 5, 5
    codes, scales, table = pool(rng, B, P, H, hd)
    pages = pages_of(codes, scales, table)
    pos = np.array([0, 31, 32, 63, 64])
    first = rows_of(rng, B, 64, H, hd)
    pages.append(first[0].cuda(), first[1].cuda(), i32([0] * B), n=i32(pos))
    oracle_append(codes, scales, table, first.double().numpy(), [0] * B, pos)
    same_pages(pages, codes, scales)
    for T, n in ((1, None), (1, None), (40, [40, 0, 1, 33, 17]), (2, [2, 0, 1, 2, 0]),
                 (32, None), (95, [95, 64, 95, 1, 0])):
        x = rows_of(rng, B, T, H, hd)
        pages.append(x[0].cuda(), x[1].cuda(), i32(pos), n=None if n is None else i32(n))
        n = [T] * B if n is None else n
        oracle_append(codes, scales, table, x.double().numpy(), pos, n)
        same_pages(pages, codes, scales)
        pos = pos + np.array(n)


def test_append_over_a_truncated_sequence_and_twice():
    """Writing again from an earlier position: rows behind it are dead, its
    block keeps the older rows; the same call twice changes nothing."""
    rng = np.random.default_rng(2)
    codes, scales, table = pool(rng, 2, 3, 2, 64)
    pages = pages_of(codes, scales, table)
    for pos, T in (([0, 0], 150), ([70, 33], 20), ([70, 33], 20)):
        x = rows_of(np.random.default_rng(T), 2, T, 2, 64, spread=5.0)
        pages.append(x[0].cuda(), x[1].cuda(), i32(pos))
        oracle_append(codes, scales, table, x.double().numpy(), pos, [T, T])
        same_pages(pages, codes, scales)


def test_append_special_values():
    rng = np.random.default_rng(3)
    codes, scales, table = pool(rng, 1, 2, 1, 64)
    pages = pages_of(codes, scales, table)
    x = rng.standard_normal((2, 1, 128, 1, 64))
    x[0, 0, 3, 0, :4] = [np.inf, -np.inf, np.nan, 3.0e38]
    x[0, 0, 32:64] = 0.0                       # a block of zeros, signed ones too
    x[0, 0, 40, 0, 3] = -0.0
    x[0, 0, 64:96] = np.nan
    x[0, 0, 96:128] *= 1e-38                   # subnormal bf16 values
    x[1, 0, :32] = np.inf
    x[1, 0, 32:64] = 448.0
    x[1, 0, 64:96] = 3.3895e38                 # the largest bf16 value
    xb = bf(x)
    pages.append(xb[0].cuda(), xb[1].cuda(), i32([0]))
    oracle_append(codes, scales, table, xb.double().numpy(), [0], [128])
    got = pages.k.cpu().numpy()
    nan = (codes[0] & 0x7F) == 0x7F            # a NaN's sign is free
    assert np.array_equal((got & 0x7F) == 0x7F, nan)
    assert np.array_equal(got[~nan], codes[0][~nan])
    assert np.array_equal(pages.v.cpu().numpy(), codes[1])
    assert np.array_equal(pages.k_scale.cpu().numpy(), scales[0])
    assert np.array_equal(pages.v_scale.cpu().numpy(), scales[1])


def test_append_strided_rows():
    """K and V as slices of one projection output."""
    rng = np.random.default_rng(4)
    B, T, H, hd = 2, 37, 2, 128
    codes, scales, table = pool(rng, B, 2, H, hd)
    pages = pages_of(codes, scales, table)
    fused = bf(rng.standard_normal((B, T, 5 * H * hd))).cuda()
    k = fused[..., H * hd:2 * H * hd].view(B, T, H, hd)
    v = fused[..., 3 * H * hd:4 * H * hd].view(B, T, H, hd)
    pages.append(k, v, i32([5, 0]), n=i32([30, 37]))
    oracle_append(codes, scales, table, [k.double().cpu().numpy(), v.double().cpu().numpy()],
                  [5, 0], [30, 37])
    same_pages(pages, codes, scales)


def filled(rng, lens, P, H, hd, cap=None):
    """A pool whose sequences hold lens[b] rows; everything else NaN codes."""
    B = len(lens)
    codes, scales, table = pool(rng, B, P, H, hd)
    T = max(max(lens), 1)
    x = rows_of(rng, B, T, H, hd, spread=1.0)
    x[0] *= 0.1
    pages = pages_of(codes, scales, table)
    pages.append(x[0].cuda(), x[1].cuda(), i32([0] * B), n=i32(lens))
    codes = [pages.k.cpu().numpy(), pages.v.cpu().numpy()]
    scales = [pages.k_scale.cpu().numpy(), pages.v_scale.cpu().numpy()]
    return pages, codes, scales, table


def check_attend(out, q, codes, scales, table, lens, window, scale):
    out = out.double().cpu().numpy()
    qd = q.double().cpu().numpy()
    B, H = len(table), codes[0].shape[1]
    G = q.shape[1] // H
    for b in range(B):
        for h in range(H):
            kv = []
            for kind in range(2):
                c, s = seq_view(codes[kind], scales[kind], table, b, h)
                kv.append(oracle.decode(c, s, int(lens[b])))
            o, A = oracle.attend(qd[b, h * G:(h + 1) * G], kv[0], kv[1], window, scale)
            err = np.abs(out[b, h * G:(h + 1) * G] - o)
            assert np.all(err <= 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * A), (
                b, h, lens[b], window, float((err / (A + 1e-30)).max()))


@pytest.mark.parametrize("hd,H,G", [(64, 2, 1), (64, 1, 8), (128, 1, 2), (128, 2, 8),
                                    (160, 1, 4), (160, 2, 8), (160, 1, 1)])
def test_attend_lengths_and_windows(hd, H, G, layout):
    rng = np.random.default_rng(hd + G)
    lens = [0, 1, 31, 32, 33, 63, 64, 65, 127, 200, 700]
    pages, codes, scales, table = filled(rng, lens, 11, H, hd)
    q = bf(rng.standard_normal((len(lens), H * G, hd))).cuda()
    for window in (0, 1, 16, 33, 64, 500):
        out = pages.attend(q, i32(lens), window=window)
        check_attend(out, q, codes, scales, table, lens, window, hd ** -0.5)
        assert torch.all(out[0] == 0)
    # a sequence may also use less than it holds
    short = [0, 1, 5, 31, 2, 60, 64, 32, 100, 199, 350]
    check_attend(pages.attend(q, i32(short), scale=-0.3), q, codes, scales, table, short, 0, -0.3)


def test_attend_long_and_many(layout):
    rng = np.random.default_rng(20)
    lens = [9000, 3, 4097]
    pages, codes, scales, table = filled(rng, lens, 141, 1, 160)
    q = bf(rng.standard_normal((3, 4, 160)) * 2).cuda()
    for window in (0, 1024):
        check_attend(pages.attend(q, i32(lens), window=window), q, codes, scales, table, lens,
                     window, 160 ** -0.5)
    lens = [(37 * b) % 130 for b in range(300)]
    pages, codes, scales, table = filled(rng, lens, 3, 2, 64)
    q = bf(rng.standard_normal((300, 4, 64))).cuda()
    check_attend(pages.attend(q, i32(lens)), q, codes, scales, table, lens, 0, 64 ** -0.5)


def test_attend_unlike_scales_and_query_magnitudes(layout):
    """V blocks whose scales differ by 2^60, the larger ones with weight ~0 or
    not; queries from 2^-40 to 2^30 (their scores stay moderate)."""
    rng = np.random.default_rng(21)
    hd, P = 64, 4
    codes, scales, table = pool(rng, 2, P, 1, hd, fill=0x00)
    for c in codes:
        c[...] = rng.integers(0, 0x7E, c.shape)
        c[...] ^= rng.integers(0, 2, c.shape).astype(np.uint8) << 7
    scales[0][...] = 2.0 ** rng.integers(-12, -8, scales[0].shape)
    scales[1][...] = 2.0 ** rng.integers(-30, 30, scales[1].shape)
    lens = [256, 170]
    for mag in (-40, 0, 30):
        q = bf(rng.standard_normal((2, 8, hd)) * 2.0 ** mag).cuda()
        pages = pages_of(codes, scales, table)
        out = pages.attend(q, i32(lens), scale=0.25 * 2.0 ** -mag)
        check_attend(out, q, codes, scales, table, lens, 0, 0.25 * 2.0 ** -mag)
    # the huge block gets no weight: its keys point away from the query
    one = np.zeros((1, 1, hd))
    one[..., 0] = 1.0
    codes[0][...] = 0
    codes[0][table[0, 0], 0, :32, 0] = 0xFE    # -448
    codes[0][table[0, 0], 0, 32:, 0] = 0x38    # 1
    codes[0][table[0, 1:], 0, :, 0] = 0x38
    scales[0][...] = 1.0
    scales[1][...] = 2.0 ** -40
    scales[1][table[0, 0], 0, 0] = 2.0 ** 60
    pages = pages_of(codes, scales, table[:1])
    q = bf(one).cuda()
    check_attend(pages.attend(q, i32([256]), scale=1.0), q, codes, scales, table[:1], [256], 0, 1.0)


def test_attend_small_weights_add_up(layout):
    """One key of weight 1 and 8000 of weight e^-16 each: together they are
    a thousandth of the answer, and none may be lost to rounding."""
    hd, n = 64, 8001
    P = -(-n // 64)
    k = np.zeros((1, n, 1, hd))
    k[0, 0, 0, 0] = 16.0
    v = np.zeros((1, n, 1, hd))
    v[0, 0, 0, :] = 0.0
    v[0, 1:, 0, :] = 448.0
    pages = lb.KV8Pages.empty(1, n, 1, hd)
    pages.append(bf(k).cuda(), bf(v).cuda(), i32([0]))
    q = np.zeros((1, 1, hd))
    q[..., 0] = 1.0
    out = pages.attend(bf(q).cuda(), i32([n]), scale=1.0).double().cpu().numpy()
    w = 8000 * np.exp(-16.0)
    want = 448 * w / (1 + w)
    # bf16 result, and weights of 11 bits
    assert np.all(np.abs(out - want) <= (2.0 ** -8 + 2.0 ** -10) * want)


def test_attend_strided_query_given_buffers_and_streams(layout):
    rng = np.random.default_rng(22)
    lens = [100, 64, 5]
    pages, codes, scales, table = filled(rng, lens, 2, 2, 128)
    fused = bf(rng.standard_normal((3, 3, 8, 128))).cuda()
    q = fused[:, 1]
    out = torch.full((3, 8, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = pages.workspace(8)
    got = pages.attend(q, i32(lens), out=out, ws=ws)
    assert got.data_ptr() == out.data_ptr()
    check_attend(out, q, codes, scales, table, lens, 0, 128 ** -0.5)
    ref = out.clone()
    # two streams at once, each with its own workspace
    ls = i32(lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[pages.attend(q, ls, stream=s) for s in streams] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for pair in outs for o in pair)


def test_threads_with_unlike_strides(layout):
    """Two threads on one cache, each with its own stream and query layout."""
    import sys
    import threading

    rng = np.random.default_rng(25)
    lens = [70, 128, 1]
    pages, codes, scales, table = filled(rng, lens, 2, 2, 64)
    fused = bf(rng.standard_normal((3, 3, 8, 64))).cuda()
    qs = [fused[:, 1], fused[:, 2].contiguous()]
    ls = i32(lens)
    want = [pages.attend(q, ls).clone() for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        outs = [pages.attend(qs[i], ls, stream=streams[i]) for _ in range(200)]
        streams[i].synchronize()
        bad.extend(i for o in outs if not torch.equal(o, want[i]))

    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(before)
    assert not bad


def test_shared_prefix_pages(layout):
    """Two sequences read the same first page and own their last ones."""
    rng = np.random.default_rng(23)
    codes, scales, table = pool(rng, 2, 3, 1, 64)
    table[1, 0] = table[0, 0]
    pages = pages_of(codes, scales, table)
    x = rows_of(rng, 2, 64, 1, 64, spread=1.0)
    pages.append(x[0].cuda(), x[1].cuda(), i32([0, 64]), n=i32([64, 0]))
    y = rows_of(rng, 2, 50, 1, 64, spread=1.0)
    pages.append(y[0].cuda(), y[1].cuda(), i32([64, 64]), n=i32([50, 9]))
    codes = [pages.k.cpu().numpy(), pages.v.cpu().numpy()]
    scales = [pages.k_scale.cpu().numpy(), pages.v_scale.cpu().numpy()]
    q = bf(rng.standard_normal((2, 2, 64))).cuda()
    check_attend(pages.attend(q, i32([114, 73])), q, codes, scales, table, [114, 73], 0, 0.125)


def test_offsets_past_32_bits():
    """The last pages of a pool of more than 2^32 bytes of codes."""
    rng = np.random.default_rng(24)
    H, hd = 8, 160
    n = (1 << 32) // (H * 64 * hd) + 10
    k = torch.empty((n, H, 64, hd), dtype=torch.uint8, device=DEV)
    v = torch.empty_like(k)
    sc = [torch.ones((n, H, 2), device=DEV) for _ in "kv"]
    table = np.array([[n - 1, 3, n - 2]], np.int32)
    pages = lb.KV8Pages(k, v, sc[0], sc[1], i32(table))
    x = rows_of(rng, 1, 150, H, hd, spread=1.0)
    pages.append(x[0].cuda(), x[1].cuda(), i32([0]))
    q = bf(rng.standard_normal((1, 4 * H, hd))).cuda()
    out = pages.attend(q, i32([150]))
    at = torch.tensor([n - 1, 3, n - 2], device=DEV)
    codes = [k[at].cpu().numpy(), v[at].cpu().numpy()]
    scales = [s[at].cpu().numpy() for s in sc]
    check_attend(out, q, codes, scales, np.array([[0, 1, 2]]), [150], 0, hd ** -0.5)
    c0, s0, t0 = [np.zeros_like(c) for c in codes], [np.ones_like(s) for s in scales], np.array([[0, 1, 2]])
    oracle_append(c0, s0, t0, x.double().numpy(), [0], [150])
    for kind in range(2):
        assert np.array_equal(scales[kind][:, :, 0], s0[kind][:, :, 0])
        got = np.concatenate(list(codes[kind]), axis=1)[:, :150]
        assert np.array_equal(got, np.concatenate(list(c0[kind]), axis=1)[:, :150])


def test_bad_pages_positions_and_lengths_are_reported(model):
    """Indexes that fall outside are skipped and reported; nothing else is
    written or read."""
    rng = np.random.default_rng(25)
    codes, scales, table = pool(rng, 3, 2, 1, 64)
    n = codes[0].shape[0]
    assert model.sync_status() == 0
    bad = table.copy()
    bad[0, 0], bad[1, 0] = -1, n
    pages = pages_of(codes, scales, bad)
    x = rows_of(rng, 3, 40, 1, 64)
    pages.append(x[0].cuda(), x[1].cuda(), i32([0, 0, 0]), n=i32([40, 40, 0]))
    same_pages(pages, codes, scales)
    assert model.sync_status() == -7
    pages = pages_of(codes, scales, table)
    for pos, num in ((-1, 5), (100, 40), (0, -1), (0, 41), (2 ** 31 - 1, 40), (128, 1)):
        pages.append(x[0].cuda(), x[1].cuda(), i32([pos, 0, 0]), n=i32([num, 0, 0]))
        same_pages(pages, codes, scales)
        assert model.sync_status() == -7
    pages, codes, scales, table = filled(rng, [128, 128, 128], 2, 1, 64)
    q = bf(rng.standard_normal((3, 2, 64))).cuda()
    out = pages.attend(q, i32([129, -1, 128]))
    assert model.sync_status() == -7
    assert torch.all(out[:2] == 0)
    check_attend(out[2:], q[2:], codes, scales, table[2:], [128], 0, 0.125)
    # a bad page hides its 64 keys
    bad = table.copy()
    bad[0, 1], bad[1, 1] = n + 5, -3
    out = pages_of(codes, scales, bad).attend(q, i32([128, 128, 128]))
    assert model.sync_status() == -7
    check_attend(out, q, codes, scales, table, [64, 64, 128], 0, 0.125)


def test_bad_pages_and_lengths_in_long_tables(model, layout):
    rng = np.random.default_rng(26)
    B = 5
    pages, codes, scales, table = filled(rng, [128] * B, 2, 2, 160)
    q = bf(rng.standard_normal((B, 8, 160))).cuda()
    lens = [128, 128, 10 ** 6, -5, 90]
    bad = table.copy()
    bad[0, 1], bad[1, 0], bad[4, 0], bad[4, 1] = len(codes[0]), -1, -7, 2 ** 31 - 1
    out = pages_of(codes, scales, bad).attend(q, i32(lens))
    assert model.sync_status() == -7
    assert torch.all(out[2:] == 0)
    check_attend(out[:1], q[:1], codes, scales, table[:1], [64], 0, 160 ** -0.5)
    # (the second page alone, as a sequence of its own)
    check_attend(out[1:2], q[1:2], codes, scales, table[1:2, 1:], [64], 0, 160 ** -0.5)


@pytest.mark.parametrize("hd,H,G", [(160, 4, 4), (128, 8, 8), (64, 1, 1), (64, 4, 2)])
def test_attend_pairs_over_the_range(hd, H, G):
    """From one pair to more than a device runs at once, at lengths on both
    sides of every split between thread blocks and warps."""
    rng = np.random.default_rng(hd * G)
    for B in (1, 2, 5, 17, 40):
        lens = [int(x) for x in rng.integers(0, 1200, B)]
        lens[0] = 1200
        pages, codes, scales, table = filled(rng, lens, 19, H, hd)
        q = bf(rng.standard_normal((B, H * G, hd))).cuda()
        for window in (0, 100):
            out = pages.attend(q, i32(lens), window=window)
            check_attend(out, q, codes, scales, table, lens, window, hd ** -0.5)
            again = pages.attend(q, i32(lens), window=window)
            assert torch.equal(out, again)


def test_refusals():
    pages = lb.KV8Pages.empty(2, 100, 2, 64)
    k = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device=DEV)
    pos = i32([0, 0])
    odd = torch.zeros(2, 3, 2, 65, dtype=torch.bfloat16, device=DEV)[..., :64]
    for kw in (dict(k=k.float()), dict(v=k[:1]), dict(k=k[..., :32]), dict(k=odd), dict(pos=pos.long()),
               dict(pos=pos[:1]), dict(n=pos.cpu()), dict(k=k.transpose(1, 3)),
               dict(k=k.new_zeros(2, 129, 2, 64), v=k.new_zeros(2, 129, 2, 64))):
        with pytest.raises(ValueError):
            pages.append(**(dict(k=k, v=k, pos=pos) | kw))
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=DEV)
    for kw in (dict(q=q.float()), dict(q=q[:, :6]), dict(q=q[:1]), dict(lens=pos.long()), dict(window=-1),
               dict(out=q.float()), dict(out=q[:, :4]), dict(q=q.new_zeros(2, 32, 64))):
        with pytest.raises(ValueError):
            pages.attend(**(dict(q=q, lens=pos) | kw))
    with pytest.raises(lb.DoryError):
        pages.attend(q, pos, scale=float("inf"))
    c = pages.k
    for args in ((c, c, pages.k_scale, pages.v_scale[:1], pages.block_table),
                 (c.view(torch.int8), c, pages.k_scale, pages.v_scale, pages.block_table),
                 (c[:, :, :32], c, pages.k_scale, pages.v_scale, pages.block_table),
                 (c, c, pages.k_scale, pages.v_scale, pages.block_table.long()),
                 (c, c, pages.k_scale, pages.v_scale, pages.block_table[:0])):
        with pytest.raises(ValueError):
            lb.KV8Pages(*args)
    pages.append(k[:, :0], k[:, :0], pos)          # an empty call


def test_decode_steps_together_and_captured():
    """A serving step as a user runs it, append, attend and sample, captured
    once into a graph and replayed while the sequences grow (one of them sits
    out every other step), against the same steps by the oracle."""
    rng = np.random.default_rng(26)
    B, H, G, hd, P, V = 3, 2, 4, 64, 3, 900
    codes, scales, table = pool(rng, B, P, H, hd)
    pages = pages_of(codes, scales, table)
    lens = np.array([0, 30, 95])
    first = rows_of(rng, B, 95, H, hd, spread=1.0)
    pages.append(first[0].cuda(), first[1].cuda(), i32([0] * B), n=i32(lens))
    oracle_append(codes, scales, table, first.double().numpy(), [0] * B, lens)
    kbuf = torch.zeros(B, 1, H, hd, dtype=torch.bfloat16, device=DEV)
    vbuf, qbuf = torch.zeros_like(kbuf), torch.zeros(B, H * G, hd, dtype=torch.bfloat16, device=DEV)
    pos, n, after = i32(lens), i32([1] * B), i32(lens)
    zbuf, u = torch.zeros(B, V, device=DEV), torch.zeros(B, device=DEV)
    top_p = torch.full((B,), 0.9, device=DEV)
    W = torch.tensor(rng.standard_normal((H * G * hd, V)), dtype=torch.float32, device=DEV)
    out = torch.zeros_like(qbuf)
    tok = torch.zeros(B, dtype=torch.int32, device=DEV)
    ws = pages.workspace(H * G)

    def step():
        pages.append(kbuf, vbuf, pos, n=n)
        torch.add(pos, n, out=after)
        pages.attend(qbuf, after, out=out, ws=ws)
        torch.matmul(out.view(B, -1).float(), W, out=zbuf)
        lb.sample(zbuf, u, top_p=top_p, tokens=tok)

    n.zero_()
    step()                                          # warm up without a token
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    from oracle import sample as osample
    for i in range(6):
        x = rows_of(rng, B, 1, H, hd, spread=1.0)
        q = bf(rng.standard_normal((B, H * G, hd)))
        cnt = [1, 1, i % 2]
        uu = rng.random(B).astype(np.float32)
        kbuf.copy_(x[0]); vbuf.copy_(x[1]); qbuf.copy_(q)      # noqa: E702
        pos.copy_(i32(lens)); n.copy_(i32(cnt)); u.copy_(torch.tensor(uu))  # noqa: E702
        graph.replay()
        oracle_append(codes, scales, table, x.double().numpy(), lens, cnt)
        lens = lens + cnt
        same_pages(pages, codes, scales)
        check_attend(out, q, codes, scales, table, lens, 0, hd ** -0.5)
        z = zbuf.cpu().numpy()
        for b in range(B):
            assert int(tok[b]) == osample.sample_row(z[b], uu[b], top_p=float(np.float32(0.9)))[0]


def test_threads_on_one_stream(layout):
    """Two threads on one cache and one stream, with the kept workspace."""
    import sys
    import threading

    rng = np.random.default_rng(27)
    lens = [70, 128, 100]
    pages, codes, scales, table = filled(rng, lens, 2, 2, 64)
    qs = [bf(rng.standard_normal((3, 8, 64))).cuda() for _ in range(2)]
    ls = i32(lens)
    want = [pages.attend(q, ls).clone() for q in qs]
    for q, o in zip(qs, want):
        check_attend(o, q, codes, scales, table, lens, 0, 0.125)
    torch.cuda.synchronize()
    bad = []

    def work(i):
        outs = [pages.attend(qs[i], ls) for _ in range(300)]
        torch.cuda.current_stream().synchronize()
        bad.extend(i for o in outs if not torch.equal(o, want[i]))

    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(before)
    assert not bad


def test_one_head_then_more_of_one_buffer(layout):
    """Queries of the same strides with 1 and with 8 heads, in turn."""
    rng = np.random.default_rng(28)
    lens = [100, 64, 5]
    pages, codes, scales, table = filled(rng, lens, 2, 1, 64)
    buf = bf(rng.standard_normal((3, 8, 64))).cuda()
    for G in (1, 8, 1, 2):
        q = buf[:, :G]
        check_attend(pages.attend(q, i32(lens)), q, codes, scales, table, lens, 0, 0.125)


@pytest.mark.parametrize("hd,G", [(64, 2), (160, 4)])
def test_attend_light_blocks_with_large_values(hd, G, layout):
    """Blocks of weight e^-22 to e^-30 whose values are so much larger that
    they make up a good part of the answer, next to ordinary ones in the same
    warp: light and heavy in turn, light first or heavy first."""
    rng = np.random.default_rng(29)
    B, nb = 100, 32
    codes, scales, table = pool(rng, B, nb // 2, 1, hd, fill=0x00)
    a = [22.0, 24.0, 26.0, 28.0, 30.0]                     # E4M3 values
    for b in range(B):
        for j in range(nb):
            pg, half = table[b, j // 2], j % 2
            rows = slice(32 * half, 32 * half + 32)
            k, v = codes[0][pg, 0, rows], codes[1][pg, 0, rows]
            k[:, 1] = rng.integers(0x20, 0x38, 32)         # 1/8 .. 1
            v[...] = rng.integers(0x30, 0x58, v.shape)     # 1/2 .. 16
            v ^= rng.integers(0, 2, v.shape).astype(np.uint8) << 7
            if (j + b) % 2:
                x = a[(j + b) // 2 % 5]
                k[:, 0] = oracle.encode(-x)
                scales[1][pg, 0, half] = 2.0 ** round(x / np.log(2.0))
    pages = pages_of(codes, scales, table)
    q = np.zeros((B, G, hd))
    q[..., 0] = 1.0
    q[..., 1] = rng.uniform(0.1, 1.0, (B, G))
    q = bf(q).cuda()
    check_attend(pages.attend(q, i32([32 * nb] * B), scale=1.0), q, codes, scales, table,
                 [32 * nb] * B, 0, 1.0)


def test_small_weights_add_up_in_both_layouts(layout):
    """8000 keys of weight e^-16 beside one of weight 1 (see
    test_attend_small_weights_add_up), on pages of the layout's table."""
    hd, n = 64, 8001
    P = -(-n // 64)
    codes, scales, table = pool(np.random.default_rng(30), 1, P, 1, hd, fill=0x00)
    pages = pages_of(codes, scales, table)
    k, v = np.zeros((2, 1, n, 1, hd))
    k[0, 0, 0, 0] = 16.0
    v[0, 1:] = 448.0
    pages.append(bf(k).cuda(), bf(v).cuda(), i32([0]))
    q = np.zeros((1, 1, hd))
    q[..., 0] = 1.0
    out = pages.attend(bf(q).cuda(), i32([n]), scale=1.0).double().cpu().numpy()
    w = 8000 * np.exp(-16.0)
    want = 448 * w / (1 + w)
    assert np.all(np.abs(out - want) <= (2.0 ** -8 + 2.0 ** -10) * want)


@pytest.mark.parametrize("hd,H,G", [(64, 2, 4), (160, 4, 4)])
def test_output_in_place_of_the_query(hd, H, G, layout):
    """`out` = q gives the bits of an output of its own."""
    rng = np.random.default_rng(31)
    lens = [0, 1, 200, 700, 33, 64, 1000, 1000]
    pages, codes, scales, table = filled(rng, lens, 16, H, hd)
    q = bf(rng.standard_normal((len(lens), H * G, hd))).cuda()
    for window in (0, 100):
        want = pages.attend(q, i32(lens), window=window)
        mine = q.clone()
        got = pages.attend(mine, i32(lens), window=window, out=mine)
        assert got.data_ptr() == mine.data_ptr() and torch.equal(mine, want)


@pytest.mark.parametrize("spread", [1, 20, 60])
@pytest.mark.parametrize("hd,B,n", [(64, 150, 300), (128, 7, 1000), (160, 40, 96)])
def test_attend_holds_its_stated_bound(hd, B, n, spread, layout):
    """Keys of random codes and steep scores: the heaviest key's values may be
    2^-9 in units where a light one's are 448.  Beside the output's rounding
    (2^-8 |o|) and 11-bit weights (2^-10 A, see the module) a weight may be off
    by 2^-32 of the largest among the blocks whose V scale is at least 1/16 of
    its own block's.  An f32 score is a sum of hd products and errs by at most
    hd 2^-23 sum |q k| scale, which is the relative error of its weight."""
    rng = np.random.default_rng(hd + spread)
    H, G, P, scale = 1, 2, -(-n // 64), 1.0
    codes, scales, table = pool(rng, B, P, H, hd, fill=0x00)
    for c in codes:
        c[...] = rng.integers(0, 0x7F, c.shape)
        c[...] ^= rng.integers(0, 2, c.shape).astype(np.uint8) << 7
    scales[0][...] = 2.0 ** rng.integers(-12, -6, scales[0].shape)
    scales[1][...] = 2.0 ** rng.integers(-spread, spread + 1, scales[1].shape)
    lens = [n] + [int(x) for x in rng.integers(1, n + 1, B - 1)]
    pages = pages_of(codes, scales, table)
    q = bf(rng.standard_normal((B, H * G, hd))).cuda()
    out = pages.attend(q, i32(lens), scale=scale).double().cpu().numpy()
    qd = q.double().cpu().numpy()
    for b in range(B):
        (ck, sk), (cv, sv) = [seq_view(c, s, table, b, 0) for c, s in zip(codes, scales)]
        k, v = oracle.decode(ck, sk, lens[b]), oracle.decode(cv, sv, lens[b])
        o, A = oracle.attend(qd[b], k, v, 0, scale)
        z = scale * (qd[b] @ k.T)
        w = np.exp(z - z.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        nb = -(-lens[b] // 32)
        first = np.arange(nb) * 32
        heaviest = np.maximum.reduceat(w, first, axis=1)             # [G, nb]
        allowed = sv[None, :nb] >= sv[:nb, None] / 16                # [nb, nb]
        ref = np.where(allowed[None], heaviest[:, None, :], 0.0).max(-1)
        lost = 2.0 ** -32 * (ref @ np.add.reduceat(np.abs(v), first, axis=0))
        e = hd * 2.0 ** -23 * scale * (np.abs(qd[b]) @ np.abs(k).T).max(1, keepdims=True)
        bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + e) * A + lost
        err = np.abs(out[b] - o)
        assert np.all(err <= bound), (b, lens[b], float((err / bound).max()))
