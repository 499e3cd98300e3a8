"""Host side of KV8Pages with a stand-in for the library (no GPU): which
strides, sizes and workspaces the entry points get, and in which order calls of
several threads are enqueued."""
import contextlib
import threading
import time

import pytest
import torch

from looped_ngpt_b200 import ops

BF16 = torch.bfloat16


class StandIn:
    """Notes what each call gets.  Attention is enqueued as two launches, with
    time for another thread between them, as outside the interpreter lock."""

    def __init__(self):
        self.strides, self.launches, self.windows = [], [], []

    def dory_kv8_plan(self, c, plan):
        return 0

    def dory_kv8_workspace_bytes(self, c, n_q_heads, out):
        out._obj.value = 512
        return 0

    def dory_kv8_attend(self, c, q, strides, n_q_heads, lens, window, scale, out, ws, nb, st):
        self.strides.append(list(strides))
        self.windows.append(window)
        self.launches.append((ws, "attend", out))
        time.sleep(0.002)
        self.launches.append((ws, "merge", out))
        return 0


@pytest.fixture
def lib(monkeypatch):
    lib = StandIn()
    monkeypatch.setattr(ops, "_cuda", lambda t, name: t.device)
    monkeypatch.setattr(ops, "_here", lambda device: 0)
    monkeypatch.setattr(ops._lib, "load", lambda: lib)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return lib


def pages(heads=1, batch=3):
    return ops.KV8Pages.empty(batch, 64, heads, 64, device="cpu")


def test_threads_on_one_stream_do_not_mix_their_launches(lib):
    """A workspace carries pieces from the attention to the kernel that joins
    them: no other call may use it between the two."""
    p, lens = pages(), torch.zeros(3, dtype=torch.int32)

    def work():
        q = torch.zeros(3, 4, 64, dtype=BF16)
        for _ in range(5):
            p.attend(q, lens)

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(lib.launches) == 30
    for ws in {ws for ws, _, _ in lib.launches}:
        mine = [x for x in lib.launches if x[0] == ws]
        for a, m in zip(mine[::2], mine[1::2]):
            assert (a[1], m[1]) == ("attend", "merge") and a[2] == m[2]


def test_strides_of_one_head_are_not_kept_for_more(lib):
    """A dim of length 1 has no stride of its own, so calls with the same
    strides and another number of heads do not share stride arrays."""
    p, lens = pages(), torch.zeros(3, dtype=torch.int32)
    buf = torch.zeros(3, 8, 64, dtype=BF16)
    p.attend(buf[:, :1], lens)
    p.attend(buf, lens)
    p.attend(buf[:, :1], lens)
    assert lib.strides == [[512, 0], [512, 64], [512, 0]]
    # a head stride that one head does not use, and more do
    odd = torch.zeros(3 * 8 * 68, dtype=BF16).as_strided((3, 8, 64), (544, 68, 1))
    p.attend(odd[:, :1], lens)
    with pytest.raises(ValueError, match="aligned"):
        p.attend(odd, lens)
    assert len(lib.strides) == 4


def test_windows_past_32_bits(lib):
    """A window of the whole cache or more is the whole cache, however large."""
    p, lens = pages(), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=BF16)
    for w in (0, 5, 64, 65, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 70):
        p.attend(q, lens, window=w)
    assert lib.windows == [0, 5] + [64] * 6
    with pytest.raises(ValueError, match="window"):
        p.attend(q, lens, window=-2 ** 32)


def test_sizes_past_32_bits_are_refused(lib):
    """Sizes that the library's 32-bit arguments would cut (no memory behind
    these tensors)."""
    def meta(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="meta")

    for B, V in ((1, 2 ** 31), (1, 2 ** 32 + 5), (2 ** 32 + 1, 3)):
        with pytest.raises(ValueError, match="2\\^31"):
            ops.sample(meta(B, V), meta(B))
    for n, H, B, P in ((2 ** 32 + 2, 1, 1, 2), (2, 1, 2 ** 32 + 1, 1), (2, 1, 1, 2 ** 31)):
        codes, scales = meta(n, H, 64, 64, dtype=torch.uint8), meta(n, H, 2)
        with pytest.raises(ValueError, match="2\\^31"):
            ops.KV8Pages(codes, codes, scales, scales, meta(B, P, dtype=torch.int32))


def test_workspaces_that_do_not_fit(lib):
    """A workspace is bytes in one piece on the cache's device; anything else
    would have the kernels write to memory that is not theirs."""
    p, lens = pages(), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=BF16)
    ws = p.workspace(4)
    for bad in (ws.view(torch.int32), ws.to("meta"), torch.zeros(2 * ws.numel(), dtype=torch.uint8)[::2],
                ws.numpy(), ws.data_ptr()):
        with pytest.raises(ValueError, match="ws"):
            p.attend(q, lens, ws=bad)
    assert not lib.launches
    p.attend(q, lens, ws=ws)
    assert lib.launches[0][0] == ws.data_ptr()


def test_outputs_that_overlap_the_query(lib):
    """`out` may be the query itself (a pair's query has been read when its
    output is written) or lie between its rows, but not on other rows of it."""
    p, lens = pages(heads=2), torch.zeros(3, dtype=torch.int32)
    buf = torch.zeros(2 * 3 * 256, dtype=BF16)
    q = buf[:3 * 256].view(3, 4, 64)
    for at in (8, 64, 256, 512):
        with pytest.raises(ValueError, match="overlap"):
            p.attend(q, lens, out=buf[at:at + 3 * 256].view(3, 4, 64))
    big = torch.zeros(3, 5, 4, 64, dtype=BF16)
    with pytest.raises(ValueError, match="overlap"):
        p.attend(big[:, 1], lens, out=big[0, 1:4])
    assert not lib.launches
    p.attend(q, lens, out=q)
    p.attend(big[:, 1], lens, out=big[0, 2:5])          # before the second row
    p.attend(q, lens, out=torch.zeros_like(q))
    assert len(lib.launches) == 6
