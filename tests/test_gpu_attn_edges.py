"""Edges of the attention side on the GPU: values, lengths, masks and handles
that the ordinary sizes do not reach.  Tolerances as in test_gpu_attn.py."""
import numpy as np
import pytest

import attn_plain as ap
from gpu_util import torch
from test_gpu_attn import KINDS, Batch, check, dev, half_ulp, qg  # noqa: F401  (qg: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Ts,Ls", [([9, 1, 5], [3, 1, 300]), ([60, 45, 20], [20, 2, 130])])
def test_attn_widest_window(qg, kind, causal, Ts, Ls):
    """The largest window hides nothing, for requests with more new tokens than
    context too: the bits of a call without a window."""
    b = Batch(qg, kind, 64, 16, 2, 1, Ts, Ls, seed=21)
    want = b.check(causal, 0)
    for window in (2 ** 31 - 1, 2 ** 30, 400):
        got = b.run(causal, window)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("kind", [ap.Q8, ap.Q4])
@pytest.mark.parametrize("D,heads", [(128, 3), (64, 5)])
def test_rows_that_are_not_finite_read_back_as_nan(qg, kind, D, heads):
    """A NaN or an infinity makes its row (one token of one head) NaN; the rows
    beside it keep their bits."""
    t = torch()
    rng = np.random.default_rng(22)
    N, page = 24, 16
    x = [rng.normal(size=(N, heads, D)).astype(np.float16) for _ in range(2)]
    bad = [y.copy() for y in x]
    hit = [np.zeros((N, heads), bool) for _ in range(2)]
    for w in range(2):
        for i, v in enumerate((np.nan, np.inf, -np.inf)):
            for d in (0, 31, D - 1):
                n, h = rng.integers(N), rng.integers(heads)
                bad[w][n, h, d], hit[w][n, h] = v, True
        bad[w][5, 1], hit[w][5, 1] = np.nan, True
        bad[w][6, 0], hit[w][6, 0] = -np.inf, True
        bad[w][7, 0, 3:5], hit[w][7, 0] = (np.inf, np.nan), True
    slots = dev(rng.permutation(2 * page)[:N].astype(np.int64))
    c = qg.KVCache.new(kind, 2, page, heads, D)
    c.write(dev(x[0]), dev(x[1]), slots)
    clean = [o.cpu().numpy() for o in c.read(slots)]
    c.write(dev(bad[0]), dev(bad[1]), slots)
    for got, want, h in zip(c.read(slots), clean, hit):
        got = got.cpu().numpy()
        assert np.all(np.isnan(got[h])) and np.array_equal(got[~h], want[~h])
    # a NaN under the norm, written by the rotation's pass
    r = qg.Rope(D)
    k = rng.normal(size=(N, heads, D)).astype(np.float16)
    k[3, 1, 7] = np.nan
    ones = t.ones(D, device="cuda")
    r.run(qg.make_rope_call(dev(k), dev(k), dev(np.arange(N, dtype=np.int32)), k_weight=ones,
                            cache=c, slots=slots, v=dev(x[1])))
    got = c.read(slots)[0].cpu().numpy()
    hit = np.zeros((N, heads), bool)
    hit[3, 1] = True
    assert np.all(np.isnan(got[hit])) and np.all(np.isfinite(got[~hit]))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 3, 40])
@pytest.mark.parametrize("which", [0, 1])
def test_attn_over_a_nan_is_nan(qg, kind, T, which):
    """A key or value of NaN reaches every row that sees it, in whatever form it
    is cached, and no row of a context that ends before it."""
    b = Batch(qg, kind, 128, 16, 4, 1, [T], [200], seed=23)
    at = 200 - T  # seen by all new tokens, the last before them
    want = b.run()
    rows = np.ones((1, 1, 128), np.float16)
    kv = [rows.copy(), rows.copy()]
    kv[which][:] = np.nan
    b.cache.write(dev(kv[0]), dev(kv[1]), dev(b.slots[at:at + 1]))
    out, _ = b.run()
    assert np.all(np.isnan(out)) and np.all(np.isfinite(want[0]))
    b.Ls = [at]
    out, lse = b.run()
    assert np.all(np.isfinite(out)) and np.all(np.isfinite(lse))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Ts,Ls", [([1] * 20, [1] * 20), ([8, 8, 8], [8, 9, 200]),
                                   ([40, 33], [40, 90])])
def test_attn_small_queries(qg, kind, Ts, Ls):
    """Queries at fp16's smallest normal numbers, with a scale that makes scores
    of ordinary size of them: every bit of q counts.  (Over one key the log
    of the sum is the score.)"""
    b = Batch(qg, kind, 128, 16, 4, 1, Ts, Ls, seed=24)
    b.q = (b.q.astype(np.float64) * 2.0 ** -13).astype(np.float16)
    b.check(scale=2.0 ** 10)


def test_status_waits_for_every_stream(qg):
    """The status calls see what was enqueued before them on a stream that
    does not wait for the null stream."""
    t = torch()
    c = qg.KVCache.new(qg.KV_Q8, 2, 16, 1, 64)
    k = t.ones((1, 1, 64), dtype=t.float16, device="cuda")
    slots = dev(np.array([1 << 20], np.int64))
    a = qg.Attn(1, 1, 64, 1, 32, 1)
    o = t.empty_like(k)
    call = qg.make_attn_call(c, k, o, dev(np.array([0, 1], np.int32)),
                             dev(np.array([16], np.int32)), dev(np.array([[1 << 20]], np.int32)), 1)
    big = t.ones((8192, 8192), dtype=t.float16, device="cuda")
    side = t.cuda.Stream()
    with t.cuda.stream(side):
        big @ big
    t.cuda.synchronize()
    for run, status in ((lambda: c.write(k, k, slots, stream=side), c.status),
                        (lambda: a.run(call, stream=side), a.status)):
        run()  # (a kernel's first launch may wait by itself)
        assert status(clear=True) == 8 and status() == 0
        with t.cuda.stream(side):
            for _ in range(20):  # some 10 ms
                big @ big
            run()
        assert status(clear=True) == 8 and status() == 0


@pytest.mark.parametrize("args", [(8, 2, 64, 2048, 65536), (32, 8, 128, 128, 128),
                                  (4, 4, 128, 64, 4096, 64), (32, 8, 128, 4096, 8192, 1)])
def test_attn_workspace_is_what_a_call_can_need(qg, args):
    """No more device memory than the header states."""
    t = torch()
    H, Hkv, D, tokens, length, batch = (*args, args[3])[:6]
    few = max(1, min(tokens, 32 * Hkv // H))
    rows = min(tokens, batch * few) * H * (length // 512 + 48)
    parts = 256 * t.cuda.get_device_properties(0).multi_processor_count
    stated = rows * (4 * D + 8) * (length > 64)
    stated += parts * (4 * D + 8) * (tokens * H // Hkv > 32 and length >= 512)
    qg.Attn(1, 1, 64, 1, 16, 1)  # the library's own start-up
    t.cuda.synchronize()
    before = t.cuda.mem_get_info()[0]
    a = qg.Attn(*args)
    used = before - t.cuda.mem_get_info()[0]
    assert used <= stated + 5 * (2 << 20)  # five allocations, in pages of 2 MiB
    a.close()


@pytest.mark.parametrize("kind", [ap.F16, ap.Q4])
def test_attn_partial_results_of_ragged_and_full_calls(qg, kind):
    """Few rows of several pieces, with as many tokens as requests times the
    most of one (8 each) and with fewer: the same bits for the same rows."""
    b = Batch(qg, kind, 64, 16, 4, 1, [8, 8, 8], [700, 1300, 90], seed=28)
    out, lse = b.check()
    b.Ts = [8, 1, 3]
    keep = np.r_[0:8, 15:16, 21:24]  # the last tokens of each request
    b.q, b.start = b.q[keep], np.array([0, 8, 9, 12], np.int32)
    got, gl = b.run()
    assert np.array_equal(got, out[keep]) and np.array_equal(gl, lse[keep])


def test_attn_few_rows_beside_many_tokens(qg):
    """A batch of single tokens as large as the handle's tokens, and a handle
    whose default batch is its tokens."""
    t = torch()
    B = 96
    b = Batch(qg, ap.Q8, 64, 16, 4, 2, [1] * B, [1 + (37 * i) % 500 for i in range(B)], seed=29)
    want = b.run()
    a = qg.Attn(4, 2, 64, B, 4096)
    o = t.empty((B, 4, 64), dtype=t.float16, device="cuda")
    a.run(qg.make_attn_call(b.cache, dev(b.q), o, dev(b.start), dev(np.array(b.Ls, np.int32)),
                            dev(b.table), 1))
    assert a.status() == 0 and np.array_equal(o.cpu().numpy(), want[0])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,L", [(1, 16384), (1, 16385), (2, 16896), (8, 33001)])
def test_attn_few_rows_over_long_contexts(qg, kind, T, L):
    """Contexts that reach the largest pieces (512 tokens from 16384 on), whole
    and behind windows that begin inside one and at its edge."""
    b = Batch(qg, kind, 64, 64, 4, 1, [T], [L], seed=25)
    b.check()
    if L > 16896:
        for window in (L - 16384, 600, 16000):
            b.check(window=window)


@pytest.mark.parametrize("kind", KINDS)
def test_attn_chunks_of_many_requests(qg, kind):
    """More requests of many rows than a warp has lanes, empty ones and single
    tokens among them."""
    Ts = [9 + (7 * i) % 40 if i % 6 else i % 2 for i in range(75)]
    Ls = [T + (13 * i) % 90 for i, T in enumerate(Ts)]
    Batch(qg, kind, 64, 16, 4, 1, Ts, Ls, seed=26).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Ts,Ls", [([40], [40]), ([130], [700]), ([33, 1, 64], [400, 90, 64]),
                                   ([1, 1], [1, 130])])
@pytest.mark.parametrize("window", [0, 50])
def test_attn_handle_wider_than_the_contexts(qg, kind, Ts, Ls, window):
    """A handle and a page table for far longer contexts than the call's: the
    keys' parts, most of them empty, are joined all the same."""
    t = torch()
    b = Batch(qg, kind, 128, 16, 4, 1, Ts, Ls, seed=27)
    N = sum(Ts)
    wide = np.full((len(Ts), 2048), -1, np.int32)
    wide[:, :b.table.shape[1]] = b.table
    o, ls = t.empty((N, 4, 128), dtype=t.float16, device="cuda"), t.empty((N, 4), device="cuda")
    a = qg.Attn(4, 1, 128, 256, 32768, len(Ts))
    a.run(qg.make_attn_call(b.cache, dev(b.q), o, dev(b.start), dev(np.array(Ls, np.int32)),
                            dev(wide), max(Ts), window=window, lse=ls))
    assert a.status() == 0
    o, ls = o.cpu().numpy(), ls.cpu().numpy()
    few, lse = b.run(window=window)
    for i, (T, L) in enumerate(zip(Ts, Ls)):
        n = slice(b.start[i], b.start[i + 1])
        ref, rl, mag = ap.attention(b.q[n], b.K[i], b.V[i], T, L, 128 ** -0.5, True, window)
        vmax = np.abs(b.V[i]).max()
        check(o[n], ref, half_ulp(ref) + 2.0 ** -10 * mag + L * 2.0 ** -24 * vmax, f"request {i}")
        if 4 * T <= 32:  # few rows: the same bits whatever the handle's limits
            assert np.array_equal(o[n], few[n]) and np.array_equal(ls[n], lse[n])
