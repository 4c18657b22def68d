"""The paged calls where it is odd: keys, values and queries that are no numbers, the largest batch,
fp32 projections with 128-dimensional heads, calls from several threads."""
import threading

import pytest
import torch

from long_context_prefill_dca_b200 import q1m
from long_context_prefill_dca_b200.layer import PagedCache
from tests import paged_reference as R
from tests import test_gpu_paged as P
from tests.test_gpu_paged import cache_of, cumulative, i32

pytestmark = pytest.mark.gpu
NAN = float("nan")


def place(c, b, j):
    return int(c.table[b, j // c.page]), j % c.page


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---- no numbers in visible places -----------------------------------------------------------
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("w,lens,at", [
    (R.G2, [40, 3000, 1], [(1, 0), (1, 1500), (1, 2999), (0, 17)]),            # few pairs: cut over CTAs
    (R.G3_D64, [70 + b for b in range(120)], [(60, 0), (60, 129), (119, 100)]),  # many: whole, joined in a CTA
], ids=["cut", "whole"])
def test_decode_nan_reaches_its_pair_alone(w, lens, at, what, out_dtype):
    c = R.Case(w, lens, 16, 3)
    q, ln = c.queries(len(lens)).cuda(), i32(lens)
    cache = cache_of(c, out_dtype)
    lse, clean_lse = (torch.empty(w.n_q_heads, len(lens), device="cuda") for _ in range(2))
    clean = cache.decode(q, ln, lse=clean_lse)
    pages = cache.k_pages if what == "k" else cache.v_pages
    for b, j in at:
        page, row = place(c, b, j)
        g = w.n_kv_heads - 1
        old = pages[page, g, row, 5].clone()
        pages[page, g, row, 5] = NAN
        out = cache.decode(q, ln, lse=lse)
        assert q1m.status_poll() == 0
        pages[page, g, row, 5] = old
        hit = torch.zeros(len(lens), w.n_q_heads, dtype=torch.bool, device="cuda")
        hit[b, g * w.group:] = True
        if what == "k":
            assert out[hit].isnan().all() and lse.T[hit].isnan().all()
        else:
            assert out[hit][:, 5].isnan().all()
            assert same_bits(out[hit][:, :5], clean[hit][:, :5]) and same_bits(lse, clean_lse)
        assert same_bits(out[~hit], clean[~hit]) and same_bits(lse.T[~hit], clean_lse.T[~hit])


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("w,lens,new,window,sinks,at", [
    (R.G2, [700, 300], [650, 300], 0, 0, [(0, 0), (0, 300), (0, 699), (1, 130)]),
    (R.G7, [1700, 40], [1000, 40], 300, 64, [(0, 3), (0, 500), (0, 1100), (0, 1699)]),
    (R.G3_D64, [9000], [3], 0, 0, [(0, 0), (0, 5000), (0, 8998)]),                  # one row tile, cut
], ids=["full", "window", "few"])
def test_prefill_nan_key_reaches_the_rows_that_see_it(w, lens, new, window, sinks, at, out_dtype):
    c = R.Case(w, lens, 32, 3)
    n, cu = sum(new), [0]
    for m in new:
        cu.append(cu[-1] + m)
    q, ln, cud = c.queries(n).cuda(), i32(lens), i32(cu)
    cache = cache_of(c, out_dtype)
    lse, clean_lse = (torch.empty(w.n_q_heads, n, device="cuda") for _ in range(2))
    clean = cache.prefill(q, ln, cud, window, sinks, lse=clean_lse)
    assert clean.isfinite().all()
    for b, j in at:
        page, row = place(c, b, j)
        g = w.n_kv_heads - 1
        old = cache.k_pages[page, g, row, 7].clone()
        cache.k_pages[page, g, row, 7] = NAN
        out = cache.prefill(q, ln, cud, window, sinks, lse=lse)
        assert q1m.status_poll() == 0
        cache.k_pages[page, g, row, 7] = old
        hit = torch.zeros(n, w.n_q_heads, dtype=torch.bool, device="cuda")
        pos = torch.arange(lens[b] - new[b], lens[b], device="cuda")
        sees = (pos >= j) & ((pos - j < window) if window and j >= sinks else True)
        hit[cu[b]:cu[b + 1], g * w.group:] = sees[:, None]
        assert out[hit].isnan().all() and lse.T[hit].isnan().all()
        assert same_bits(out[~hit], clean[~hit]) and same_bits(lse.T[~hit], clean_lse.T[~hit])


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("w", [R.G2, R.G7], ids=["g2", "g7"])
def test_shared_nan_key_reaches_the_sequences_that_see_it(w, out_dtype):
    prefix, lens = 1024, [1030, 1024, 500, 1300, 0] + [1100] * 40
    c = R.Case(w, lens, 64, 3, prefix=prefix)
    q, ln, pre = c.queries(len(lens)).cuda(), i32(lens), c.prefix_table.cuda()
    cache = cache_of(c, out_dtype)
    lse, clean_lse = (torch.empty(w.n_q_heads, len(lens), device="cuda") for _ in range(2))
    clean = cache.decode_shared(q, ln, pre, prefix, lse=clean_lse)
    g = w.n_kv_heads - 1
    for b, j in ((None, 0), (None, 600), (None, 1023), (3, 1299), (20, 1050)):
        page, row = (int(c.prefix_table[j // 64]), j % 64) if b is None else place(c, b, j)
        old = cache.k_pages[page, g, row, 7].clone()
        cache.k_pages[page, g, row, 7] = NAN
        out = cache.decode_shared(q, ln, pre, prefix, lse=lse)
        assert q1m.status_poll() == 0
        cache.k_pages[page, g, row, 7] = old
        hit = torch.zeros(len(lens), w.n_q_heads, dtype=torch.bool, device="cuda")
        for s, m in enumerate(lens):
            hit[s, g * w.group:] = m > j and (b is None or s == b)
        assert out[hit].isnan().all() and lse.T[hit].isnan().all()
        assert same_bits(out[~hit], clean[~hit]) and same_bits(lse.T[~hit], clean_lse.T[~hit])


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_nan_value_stays_in_its_dimension_head_and_sequences(out_dtype):
    """Prefill and shared prefix: the rows that see it get it. Rows in front of it may (a weight of 0
    times NaN): those of a row tile, 256 rows of 7 heads or up to 38 tokens, one of which sees some
    key of its 128-key tile. No other dimension, head or sequence gets it."""
    w, prefix, lens, new = R.G7, 256, [900, 700, 256], [400, 300, 1]
    c = R.Case(w, lens, 32, 3, prefix=prefix)
    cache, ln, pre, cu = cache_of(c, out_dtype), i32(lens), c.prefix_table.cuda(), cumulative(new)
    qp, qd, g = c.queries(701).cuda(), c.queries(3).cuda(), 1
    for j, call, x, first in ((650, lambda q: cache.prefill(q, ln, cu), qp, 150),
                              (700, lambda q: cache.decode_shared(q, ln, pre, prefix), qd, 0)):
        clean = call(x)
        page, row = place(c, 0, j)
        old = cache.v_pages[page, g, row, 5].clone()
        cache.v_pages[page, g, row, 5] = NAN
        out = call(x)
        assert q1m.status_poll() == 0
        cache.v_pages[page, g, row, 5] = old
        last = 400 if x is qp else 1
        assert out[first:last, g * w.group:, 5].isnan().all()
        may = torch.zeros_like(out, dtype=torch.bool)
        may[j // 128 * 128 - (lens[0] - new[0]) - 37 if x is qp else 0:last, g * w.group:, 5] = True
        assert same_bits(out[~may], clean[~may])


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_nan_queries_stay_in_their_rows(out_dtype):
    """A query that is no number is reported, and its row alone holds it."""
    w, lens, new = R.G2, [700, 300], [300, 2]
    c = R.Case(w, lens, 32, 3, prefix=256)
    cache, ln, pre = cache_of(c, out_dtype), i32(lens), c.prefix_table.cuda()
    q, qd, cu = c.queries(302).cuda(), c.queries(2).cuda(), i32([0, 300, 302])
    for x, row, call in ((q, 130, lambda x: cache.prefill(x, ln, cu)), (qd, 1, lambda x: cache.decode(x, ln)),
                         (qd, 0, lambda x: cache.decode_shared(x, ln, pre, 256))):
        clean = call(x)
        assert q1m.status_poll() == 0
        y = x.clone()
        y[row, 2, 9] = NAN
        out = call(y)
        assert q1m.status_poll() == -6 and q1m.status_poll() == 0
        hit = torch.zeros(x.shape[:2], dtype=torch.bool, device="cuda")
        hit[row, 2] = True
        assert out[hit].isnan().all() and same_bits(out[~hit], clean[~hit])


# ---- sizes ----------------------------------------------------------------------------------
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_the_largest_batch(out_dtype):
    w, batch = R.G2, q1m.MAX_PAGED_BATCH
    lens = [(7 * b) % 45 for b in range(batch)]
    lens[1000] = 900
    c, q, cache = P.decode_case(w, lens, 16, 20, 3, out_dtype)
    lse = torch.empty(w.n_q_heads, batch, device="cuda")
    out = cache.decode(q.cuda(), i32(lens), 20, 3, lse=lse)
    torch.cuda.synchronize()
    q1m.check_status()
    P.decode_check(c, q, out, lse, 20, 3, out_dtype)
    new = [min(n, b % 3) for b, n in enumerate(lens)]
    n = sum(new)
    qp, cu = c.queries(n), cumulative(new)
    got = cache.prefill(qp.cuda(), i32(lens), cu, 20, 3)
    q1m.check_status()
    at = 0
    for b, m in enumerate(new):
        if m and b % 5 == 0 or b == 1000:
            ref, _ = R.attend(w, qp[at + m - 1:at + m], [lens[b] - 1], c.kc[b], c.vc[b], 20, 3)
            tol, _ = R.bounds(w, qp[at + m - 1:at + m], c.kc[b], c.vc[b], out_dtype == "bf16")
            R.check(w, got[at + m - 1:at + m], None, ref, None, tol, 0, out_dtype == "bf16")
        at += m
    table = torch.arange(3 * batch, dtype=torch.int32, device="cuda").view(batch, 3)
    pages = torch.zeros(3 * batch, w.n_kv_heads, 16, w.head_dim, dtype=torch.float16, device="cuda")
    cache = PagedCache(w, pages, pages.clone(), table)
    lens = [b % 49 for b in range(batch)]
    new = [min(m, (b * 5) % 7) for b, m in enumerate(lens)]
    x = torch.randn(sum(new) + 9, w.n_kv_heads, w.head_dim, device="cuda").bfloat16()
    cache.append(x, x, i32(lens), cumulative(new))
    torch.cuda.synchronize()
    q1m.check_status()
    want = torch.zeros(batch, 48, w.n_kv_heads, w.head_dim, dtype=torch.float16, device="cuda")
    at = 0
    for b, m in enumerate(new):
        want[b, lens[b] - m:lens[b]] = x[at:at + m].half()
        at += m
    got = cache.v_pages.view(batch, 3, w.n_kv_heads, 16, w.head_dim).transpose(2, 3).reshape(want.shape)
    assert torch.equal(got, want)


def test_append_f32_with_128_dimensions():
    P.test_append_writes_the_prefill_rotation(R.G2.with_(in_dtype="f32"), 32, [5, 700, 33], [5, 450, 1])
    P.test_append_writes_the_prefill_rotation(R.G5, 64, [1, 64, 65, 300], [1, 1, 1, 1])


# ---- threads --------------------------------------------------------------------------------
def test_calls_from_several_threads():
    """Threads with streams of their own share a cache: results are those of calls one by one."""
    lens = [900, 17, 1300]
    c, q, cache = P.decode_case(R.G2, lens, 16, 0, 0, "f32")
    qd, ln, cu, n = q.cuda(), i32(lens), cumulative(lens), sum(lens)
    qp = c.queries(n).cuda()
    want = cache.decode(qd, ln), cache.decode(qd, ln, 100, 4), cache.prefill(qp, ln, cu)
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got = cache.decode(qd, ln), cache.decode(qd, ln, 100, 4), cache.prefill(qp, ln, cu)
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        bad.append("differs")
        except Exception as e:      # noqa: BLE001  (a thread's failure is the test's)
            bad.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    q1m.check_status()
    assert not bad
