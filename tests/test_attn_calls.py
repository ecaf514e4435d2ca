"""What the binding refuses before a call reaches the library (no GPU needed:
CPU tensors that say they are on one, and handles that are never used)."""
from types import SimpleNamespace

import pytest
import torch


class Fake:
    """A CPU tensor that a call takes for one on the GPU."""

    def __init__(self, t):
        self.t = t

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self.t, name)


def half(*shape):
    return Fake(torch.zeros(shape, dtype=torch.float16))


def ints(*shape, dtype=torch.int32):
    return Fake(torch.zeros(shape, dtype=dtype))


@pytest.fixture(scope="module")
def qg():
    from skinny_gemm_q4_gb300 import build, qgemv
    build.build()
    qgemv.load()
    return qgemv


@pytest.fixture
def cache(qg):
    class Cache(qg.KVCache):
        def __init__(self):
            self.kv_heads, self.head_dim = 2, 64
            self.c = 4096  # an address that nothing may look at

        def close(self):
            self.c = None

    return Cache()


def attn_call(qg, cache, N=1, H=4, D=64, **change):
    args = dict(q=half(N, H, D), out=half(N, H, D), q_start=ints(2), kv_len=ints(1),
                page_table=ints(1, 3), max_q=N)
    return qg.make_attn_call(cache, **{**args, **change})


def test_broadcast_tokens_are_refused(qg, cache):
    """Tokens that share their storage (stride 0) are not taken for contiguous
    ones, which lie beyond it."""
    wide = Fake(torch.zeros((1, 4, 64), dtype=torch.float16).expand(3, 4, 64))
    flat = Fake(torch.zeros((1, 256), dtype=torch.float16).expand(3, 256))
    kv = Fake(torch.zeros((1, 2, 64), dtype=torch.float16).expand(3, 2, 64))
    for bad in (dict(q=wide), dict(out=wide), dict(out=flat)):
        with pytest.raises(ValueError):
            attn_call(qg, cache, N=3, **bad)
    for q, k, more in ((wide, half(3, 2, 64), {}), (half(3, 4, 64), kv, {}),
                       (half(3, 4, 64), half(3, 2, 64), dict(q_out=wide)),
                       (half(3, 4, 64), half(3, 2, 64),
                        dict(cache=cache, slots=ints(3, dtype=torch.int64), v=kv))):
        with pytest.raises(ValueError):
            qg.make_rope_call(q, k, ints(3), **more)
    slots = ints(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        cache.write(kv, half(3, 2, 64), slots)
    with pytest.raises(ValueError):
        cache.read(slots, half(3, 2, 64), kv)
    attn_call(qg, cache, N=1, q=Fake(torch.zeros((1, 4, 64), dtype=torch.float16).expand(1, 4, 64)))
    assert attn_call(qg, cache, N=3).args.q_stride == 256


def test_calls_of_other_heads_than_the_handle_are_refused(qg, cache):
    """A call carries no head sizes of its own to the library, which goes by the
    handle's: single tokens of fewer or smaller heads would be read past
    their end."""
    def refused(handle, call):
        with pytest.raises(qg.QgemvError) as e:
            handle.run(call, stream=SimpleNamespace(cuda_stream=0))
        return e.value.status == -1 and "heads" in str(e.value)

    a = object.__new__(qg.Attn)
    a.a = None
    for a.heads in ((32, 64), (4, 128), (2, 64)):
        for N in (1, 2):
            assert refused(a, attn_call(qg, cache, N, 4, 64))
    r = object.__new__(qg.Rope)
    r.r, r.head_dim = None, 128
    for N in (1, 2):
        assert refused(r, qg.make_rope_call(half(N, 4, 64), half(N, 2, 64), ints(N)))
    with pytest.raises(ValueError):  # other heads than the cache's
        attn_call(qg, cache, D=128)
    for slots in (None, ints(1, dtype=torch.int64)):
        with pytest.raises(ValueError):  # a cache, and no slots or no values
            qg.make_rope_call(half(1, 4, 64), half(1, 2, 64), ints(1), cache=cache, slots=slots)


def test_calls_on_a_closed_cache_are_refused(qg, cache):
    """A prepared call keeps the address of its cache's handle; once that is
    closed, it does not go back to it."""
    calls = [(qg.Attn, attn_call(qg, cache)),
             (qg.Rope, qg.make_rope_call(half(1, 4, 64), half(1, 2, 64), ints(1), cache=cache,
                                         slots=ints(1, dtype=torch.int64), v=half(1, 2, 64)))]
    cache.close()
    for cls, call in calls:
        h = object.__new__(cls)
        h.a = h.r = None
        h.heads, h.head_dim = (4, 64), 64
        with pytest.raises(qg.QgemvError) as e:
            h.run(call, stream=SimpleNamespace(cuda_stream=0))
        assert e.value.status == -1 and "closed" in str(e.value)


def test_stream_without_torchs_private_queries(qg, monkeypatch):
    """Where torch has no raw-stream query, its public one gives the stream."""
    monkeypatch.setattr(qg, "_raw_stream", None)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=77))
    assert qg._stream_ptr() == 77 and qg._stream_ptr(SimpleNamespace(cuda_stream=5)) == 5
