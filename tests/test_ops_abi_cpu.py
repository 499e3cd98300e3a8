"""Arguments that the sampling and 8-bit cache entry points refuse, checked on
the host before any device work (no GPU needed)."""
import ctypes

import pytest
import torch

import looped_ngpt_b200 as lb
from looped_ngpt_b200 import _lib

P = 0x1000                      # a well-aligned address that is never read
S3 = (ctypes.c_int64 * 3)(640, 640, 160)
S2 = (ctypes.c_int64 * 2)(640, 160)


def _kv8(**over):
    v = dict(k=P, v=P, k_scale=P, v_scale=P, block_table=P, n_pages=4,
             pages_per_seq=2, batch=2, n_kv_heads=4, head_dim=160)
    v.update(over)
    return _lib.DoryKv8(**v)


def test_sample_refusals():
    f = _lib.load().dory_sample

    def call(z=P, ld=8, B=1, V=8, u=P, t=P):
        return f(z, ld, B, V, None, None, None, None, u, t, None, None)

    assert call(z=None) == -1 and call(u=None) == -1 and call(t=None) == -1
    assert call(V=0) == -1 and call(ld=7) == -1 and call(B=-1) == -1
    assert call(z=P + 2) == -1
    assert call(B=0) == 0                       # an empty call


@pytest.mark.parametrize("over,code", [
    (dict(k=None), -1), (dict(v_scale=None), -1), (dict(block_table=None), -1),
    (dict(k=P + 8), -1), (dict(v_scale=P + 4), -1), (dict(n_pages=0), -1),
    (dict(batch=0), -1), (dict(pages_per_seq=0), -1), (dict(n_kv_heads=0), -1),
    (dict(head_dim=96), -2), (dict(pages_per_seq=1 << 26), -2),
    (dict(batch=70000), -2), (dict(plan=P + 8), -1),
])
def test_kv8_refuses_a_bad_cache(over, code):
    lib = _lib.load()
    c = ctypes.byref(_kv8(**over))
    n = ctypes.c_int64()
    assert lib.dory_kv8_append(c, P, P, S3, S3, 1, P, None, None) == code
    assert lib.dory_kv8_workspace_bytes(c, 16, ctypes.byref(n)) == code
    assert lib.dory_kv8_plan(c, P) == code
    assert lib.dory_kv8_attend(c, P, S2, 16, P, 0, 1.0, P, P, 1 << 30, None) == code


def test_kv8_append_refusals():
    f = _lib.load().dory_kv8_append
    c = ctypes.byref(_kv8())
    odd = (ctypes.c_int64 * 3)(640, 641, 160)
    assert f(None, P, P, S3, S3, 1, P, None, None) == -1
    assert f(c, None, P, S3, S3, 1, P, None, None) == -1
    assert f(c, P, P + 2, S3, S3, 1, P, None, None) == -1
    assert f(c, P, P, odd, S3, 1, P, None, None) == -1
    assert f(c, P, P, S3, None, 1, P, None, None) == -1
    assert f(c, P, P, S3, S3, 1, None, None, None) == -1
    assert f(c, P, P, S3, S3, -1, P, None, None) == -1
    assert f(c, P, P, S3, S3, 129, P, None, None) == -1   # more than 2 pages
    assert f(c, P, P, S3, S3, 0, P, None, None) == 0      # an empty call


def test_kv8_attend_refusals():
    lib = _lib.load()
    f = lib.dory_kv8_attend
    c = ctypes.byref(_kv8())
    big = 1 << 40
    odd = (ctypes.c_int64 * 2)(640, 161)
    assert f(c, None, S2, 16, P, 0, 1.0, P, P, big, None) == -1
    assert f(c, P + 2, S2, 16, P, 0, 1.0, P, P, big, None) == -1
    assert f(c, P, odd, 16, P, 0, 1.0, P, P, big, None) == -1
    assert f(c, P, S2, 16, None, 0, 1.0, P, P, big, None) == -1
    assert f(c, P, S2, 16, P, -1, 1.0, P, P, big, None) == -1
    assert f(c, P, S2, 16, P, 0, float("nan"), P, P, big, None) == -1
    assert f(c, P, S2, 16, P, 0, 1.0, None, P, big, None) == -1
    assert f(c, P, S2, 18, P, 0, 1.0, P, P, big, None) == -1    # 18 on 4 heads
    assert f(c, P, S2, 12, P, 0, 1.0, P, P, big, None) == -2    # 3 per head
    assert f(c, P, S2, 64, P, 0, 1.0, P, P, big, None) == -2    # 16 per head


def test_kv8_plan_refusals():
    f = _lib.load().dory_kv8_plan
    assert f(None, P) == -1
    assert f(ctypes.byref(_kv8()), None) == -1
    assert f(ctypes.byref(_kv8()), P + 32) == -1
    # 2^31 rows and more
    assert f(ctypes.byref(_kv8(n_pages=1 << 25, n_kv_heads=1)), P) == -2


def test_python_refuses_what_is_not_on_a_gpu():
    z = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        lb.sample(z, torch.zeros(2))
    c = torch.zeros(2, 1, 64, 64, dtype=torch.uint8)
    s = torch.ones(2, 1, 2)
    with pytest.raises(ValueError, match="CUDA"):
        lb.KV8Pages(c, c, s, s, torch.zeros(1, 2, dtype=torch.int32))


def test_sample_refuses_rows_past_its_loops():
    """Rows near 2^31 would carry the kernel's 32-bit loops past their end."""
    f = _lib.load().dory_sample
    for V in (2 ** 30 + 1, 2 ** 31 - 1):
        assert f(P, V, 1, V, None, None, None, None, P, P, None, None) == -2
    assert f(P, 8, 0, 8, None, None, None, None, P, P, None, None) == 0
