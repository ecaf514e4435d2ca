"""Handles know the device that they were made on: a call refuses a cache of
another device, and runs only while its own is current."""
import ctypes
from types import SimpleNamespace

import pytest

i32, i64, vp, f64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_double


class Kv(ctypes.Structure):  # struct qg_kv of qg_attn_api.cu
    _fields_ = [("kind", i32), ("pages", i64), ("page_size", i32), ("page_shift", i32),
                ("heads", i32), ("dim", i32), ("device", i32), ("sms", i32), ("pool", vp),
                ("err", vp)]


class Rope(ctypes.Structure):  # struct qg_rope
    _fields_ = [("i", i32 * 4), ("f", f64 * 6), ("mscale", ctypes.c_float), ("device", i32),
                ("sms", i32), ("freq", vp)]


class Attn(ctypes.Structure):  # struct qg_attn
    _fields_ = [("i", i32 * 5), ("max_len", i64), ("device", i32), ("sms", i32), ("p", vp * 5)]


@pytest.fixture(scope="module")
def qg():
    from skinny_gemm_q4_gb300 import build, qgemv
    build.build()
    qgemv.load()
    return qgemv


def test_caches_of_another_device_are_refused(qg):
    """Made-up handles of two devices; no pointer of theirs is looked at."""
    lib, P = qg.load(), 4096
    kv = Kv(kind=0, pages=4, page_size=16, page_shift=4, heads=2, dim=64, device=1, sms=1,
            pool=P, err=P)
    attn = Attn(max_len=64, device=0, sms=1)
    attn.i[:] = [4, 2, 64, 4, 1]
    args = qg.QgAttnArgs(cache=ctypes.addressof(kv), q=P, out=P, q_start=P, kv_len=P, page_table=P,
                         table_width=4, N=1, B=1, max_q=1, scale=1.0)
    assert lib.qgemv_attn_run(ctypes.addressof(attn), ctypes.byref(args), None) == -1
    assert "device" in qg.qgemv_last_error()
    rope = Rope(device=0, sms=1, freq=P)
    rope.i[:] = [64, 64, 0, 0]
    args = qg.QgRopeArgs(N=1, q_heads=4, kv_heads=2, q=P, q_out=P, k=P, positions=P,
                         cache=ctypes.addressof(kv), slots=P, v=P)
    assert lib.qgemv_rope_run(ctypes.addressof(rope), ctypes.byref(args), None) == -1
    assert "device" in qg.qgemv_last_error()


def test_caches_are_made_on_their_pools_device(qg, monkeypatch):
    import torch
    current = [0]

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.before, current[0] = current[0], self.d

        def __exit__(self, *_):
            current[0] = self.before

    made = []
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(qg, "qgemv_kv_create", lambda *a: made.append(current[0]))
    pool = SimpleNamespace(is_cuda=True, dtype=torch.uint8, is_contiguous=lambda: True,
                           dim=lambda: 2, shape=(3, qg.qgemv_kv_page_bytes(0, 16, 2, 64)),
                           data_ptr=lambda: 4096, device=1)
    qg.KVCache(0, pool, 16, 2, 64)
    assert made == [1] and current == [0]


@pytest.mark.gpu
def test_calls_while_another_device_is_current_are_refused(qg):
    """(With one GPU at hand, the handle is made to say that it is another's.)"""
    import torch
    c = qg.KVCache.new(qg.KV_F16, 2, 16, 2, 64)
    k = torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda")
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    ints = torch.zeros(2, dtype=torch.int32, device="cuda")
    r, a = qg.Rope(64), qg.Attn(2, 2, 64, 1, 16, 1)
    rope = qg.make_rope_call(k, k, ints[:1])
    attn = qg.make_attn_call(c, k, torch.empty_like(k), ints, ints[:1], ints.view(1, 2), 1)
    runs = [(lambda: c.write(k, k, slots), (Kv.from_address(c.c),)),
            (lambda: c.read(slots), (Kv.from_address(c.c),)),
            (lambda: r.run(rope), (Rope.from_address(r.r),)),
            (lambda: a.run(attn), (Kv.from_address(c.c), Attn.from_address(a.a)))]
    for run, handles in runs:
        run()
        for h in handles:
            assert h.device == 0
            h.device = 7
        with pytest.raises(qg.QgemvError) as e:
            run()
        for h in handles:
            h.device = 0
        assert e.value.status == -1 and "device" in str(e.value)
    torch.cuda.synchronize()
