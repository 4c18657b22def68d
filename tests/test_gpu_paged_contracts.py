"""What the paged calls promise beside their results: a table's own width, malformed token
offsets, memory and streams, lengths beyond the table, sums that keep their precision."""
import time

import numpy as np
import pytest
import torch

from long_context_prefill_dca_b200 import q1m
from long_context_prefill_dca_b200.layer import PagedCache
from oracle import dca_vs as O
from tests import paged_reference as R

pytestmark = pytest.mark.gpu

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_a_sliced_table_ends_at_its_own_width():
    """A table that is a slice of a larger one: the parent's entries beside it (here all valid pages)
    are not the sequence's. A length or a new position behind the slice latches the page fault in
    every call, no page outside the slice changes, and the other sequence is right."""
    w, page, width = R.G2, 32, 6
    lens = [page * width, 150]
    c = R.Case(w, lens, page, 7, prefix=128)
    spare = 100
    g = torch.Generator().manual_seed(1)
    more = torch.randn(spare, w.n_kv_heads, page, w.head_dim, generator=g).half()
    k, v = torch.cat([c.k, more]).cuda(), torch.cat([c.v, more]).cuda()
    big = (c.n_pages + torch.arange(4 * 20) % spare).view(4, 20).int()
    own = c.table[:, :width]
    big[1:3, 4:4 + width] = torch.where((own >= 0) & (own < c.n_pages), own, c.n_pages)
    big = big.cuda()
    cache = PagedCache(w, k, v, big[1:3, 4:4 + width], "f32")
    inside = torch.unique(big[1:3, 4:4 + width]).cpu()
    outside = torch.ones(c.n_pages + spare, dtype=torch.bool)
    outside[inside.long()] = False
    before = k.cpu().view(torch.int16).clone(), v.cpu().view(torch.int16).clone()
    q = c.queries(2)
    ref, _ = R.attend(w, q[1:], [149], c.kc[1], c.vc[1])
    tol, _ = R.bounds(w, q[1:], c.kc[1], c.vc[1], False)
    qd, pre = q.cuda(), c.prefix_table.cuda()
    for over in (1, page, 5 * page):
        ln = i32([lens[0] + over, 150])
        for call in (lambda: cache.decode(qd, ln), lambda: cache.prefill(qd, ln, i32([0, 1, 2])),
                     lambda: cache.decode_shared(qd, ln, pre, 128)):
            out = call()
            assert q1m.status_poll() == -8 and q1m.status_poll() == 0
            R.check(w, out[1:], None, ref, None, tol, 0, False)
    x = torch.randn(2, w.n_kv_heads, w.head_dim, generator=g).bfloat16().cuda()
    for over in (1, page, 5 * page):
        cache.append(x, x, i32([lens[0] + over, 150]))
        assert q1m.status_poll() == -8 and q1m.status_poll() == 0
    assert torch.equal(v[int(big[2, 4 + 149 // page]), :, 149 % page], x[1].half())
    for now, old in zip((k, v), before):
        assert torch.equal(now.cpu().view(torch.int16)[outside], old[outside])
        same = now.cpu().view(torch.int16) == old
        assert int((~same).any(-1).any(-1).any(-1).sum()) == 1     # sequence 1's page alone
    cache.decode(qd, i32(lens))
    cache.append(x, x, i32(lens))
    assert q1m.status_poll() == 0


@pytest.mark.parametrize("batch,cu", [
    (2, [0, 30, 61]), (2, [1, 30, 60]), (2, [0, 40, 30]), (2, [0, -5, 60]), (2, [30, 30, 60]),
    (300, [0] * 299 + [60, 50]), (300, [0, 60] + [55] + [60] * 298), (1, [0, 1 << 30]), (1, [-7, 60]),
], ids=lambda x: None)
def test_append_rejects_malformed_token_offsets(batch, cu):
    """Nothing is written, whichever entry is wrong (every table entry is a valid page here)."""
    w, page = R.G2, 16
    n_pages = 8 * batch
    k = torch.full((n_pages, w.n_kv_heads, page, w.head_dim), 3.0, dtype=torch.float16, device="cuda")
    v = k.clone()
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").view(batch, 8)
    cache = PagedCache(w, k, v, table, "f32")
    x = torch.randn(60, w.n_kv_heads, w.head_dim, device="cuda").bfloat16()
    cache.append(x, x, i32([60] * batch), i32(cu))
    assert q1m.status_poll() == -1 and q1m.status_poll() == 0
    assert (k == 3).all() and (v == 3).all()
    good = [0] * batch + [60]
    cache.append(x, x, i32([60] * batch), i32(good))
    assert q1m.status_poll() == 0
    at = table[-1].long()
    assert torch.equal(v[at].transpose(1, 2).reshape(128, w.n_kv_heads, w.head_dim)[:60], x.half())


def test_a_new_cache_can_be_used_on_any_stream_at_once():
    """The angles that the constructor computes are there for the first call, whatever stream that
    uses and whatever was queued before them."""
    w = R.G2
    c = R.Case(w, [300], 16, 2)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(300, w.n_kv_heads, w.head_dim, generator=g).bfloat16().cuda()
    ln, cu, table = i32([300]), i32([0, 300]), c.table.cuda()
    want = PagedCache(w, c.k.cuda(), c.v.cuda(), table)
    want.append(x, x, ln, cu)
    k, v = c.k.cuda(), c.v.cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    stale = torch.zeros_like(want.table)              # what the new table's memory holds before
    del stale
    torch.cuda._sleep(200_000_000)
    cache = PagedCache(w, k, v, table)
    cache.append(x, x, ln, cu, stream=side)
    torch.cuda.synchronize()
    q1m.check_status()
    at = c.table[0, :19].long()
    assert torch.equal(k[at, :, :4].view(torch.int16), want.k_pages[at, :, :4].view(torch.int16))
    assert torch.equal(k.view(torch.int16), want.k_pages.view(torch.int16))


def delayed(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(400_000_000)


def reuse(t, value):
    """Memory of t's size and type, taken again and again, with `value` in it."""
    return [torch.full_like(t, value) for _ in range(4)]


def test_inputs_may_be_dropped_once_a_call_on_another_stream_is_queued():
    """Keys, values, queries, lengths, offsets and a replaced page table whose last reference goes
    while the work still waits on `stream`."""
    w = R.G2
    lens, new = [300, 40], [200, 40]
    c = R.Case(w, lens, 16, 2)
    g = torch.Generator().manual_seed(3)
    x0 = torch.randn(240, w.n_kv_heads, w.head_dim, generator=g).bfloat16().cuda()
    q0 = c.queries(240).cuda()
    table = c.table.clone()
    table[(table < 0) | (table >= c.n_pages)] = 0
    want = PagedCache(w, c.k.cuda(), c.v.cuda(), table.cuda())
    want.append(x0, x0, i32(lens), i32([0, 200, 240]))
    want_p = want.prefill(q0, i32(lens), i32([0, 200, 240]))
    want_d = want.decode(q0[:2], i32(lens))
    cache = PagedCache(w, c.k.cuda(), c.v.cuda(), table.cuda())
    side = torch.cuda.Stream()
    for t in (x0, q0, i32(lens)):                     # kernels are loaded before anything waits
        reuse(t, 1), t.clone()
    torch.cuda.synchronize()
    delayed(side)
    x, q, q2, ln, cu = x0.clone(), q0.clone(), q0[:2].clone(), i32(lens), i32([0, 200, 240])
    torch.cuda.current_stream().synchronize()         # the copies are there; the side stream still sleeps
    cache.append(x, x, ln, cu, stream=side)
    got_p = cache.prefill(q, ln, cu, stream=side)
    got_d = cache.decode(q2, ln, stream=side)
    cache.set_page_table(torch.zeros_like(cache.page_table))
    junk = []
    del x
    junk += reuse(x0, 7.0)
    del q
    junk += reuse(q0, 7.0)
    del q2
    junk += reuse(q0[:2].clone(), 7.0)
    del ln, cu
    junk += reuse(i32(lens), 1) + reuse(i32([0, 200, 240]), 0)
    junk += reuse(cache.page_table, 1)
    torch.cuda.synchronize()
    q1m.check_status()
    assert torch.equal(cache.k_pages.view(torch.int16), want.k_pages.view(torch.int16))
    assert torch.equal(cache.v_pages.view(torch.int16), want.v_pages.view(torch.int16))
    assert torch.equal(got_p, want_p) and torch.equal(got_d, want_d)


def test_outputs_of_another_stream_may_be_dropped_once_their_use_is_queued():
    """A result from `stream`, read on the caller's stream: its memory is not given to the next call on
    `stream` before that."""
    w, lens = R.G2, [300, 40]
    c = R.Case(w, lens, 16, 2)
    cache = PagedCache(w, c.k.cuda(), c.v.cuda(), c.table.cuda())
    qa, qb = c.queries(2).cuda(), c.queries(2).cuda()
    ln, cu, pre = i32(lens), i32([0, 1, 2]), None
    side = torch.cuda.Stream()
    for call in (lambda q: cache.decode(q, ln, stream=side), lambda q: cache.prefill(q, ln, cu, stream=side)):
        torch.cuda.synchronize()
        want = call(qa)
        torch.cuda.synchronize()
        kept = want.clone()
        del want
        torch.cuda.synchronize()
        out = call(qa)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(100_000_000)
        used = out.clone()                            # waits on the caller's stream
        del out
        later = [call(qb) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(used, kept)
        del later
    q1m.check_status()


def test_shared_prefix_cuts_a_length_beyond_the_table_as_a_whole():
    """Both parts of a shared-prefix step, the prefix's and the sequence's own, see the same
    (cut) position when a length is more than its table row holds."""
    w, page, prefix = R.G2, 16, 512
    c = R.Case(w, [544, 530], page, 7, prefix=prefix)
    table = c.table[:, :544 // page].clone()
    table[(table < 0) | (table >= c.n_pages)] = c.prefix_table[0]
    cache = PagedCache(w, c.k.cuda(), c.v.cuda(), table.contiguous().cuda(), "f32")
    q, pre = c.queries(2).cuda(), c.prefix_table.cuda()
    want = cache.decode_shared(q, i32([544, 530]), pre, prefix)
    assert q1m.status_poll() == 0
    for over in (545, 1000, 2 ** 30, 2 ** 31 - 1):
        got = cache.decode_shared(q, i32([over, 530]), pre, prefix)
        assert q1m.status_poll() == -8 and q1m.status_poll() == 0
        assert torch.equal(got, want), over


# ---- sums over many keys --------------------------------------------------------------------
# Values of one sign, so that what an accumulator loses adds up. The bound, relative to the result:
# a key tile's products are 2 to 16 dependent accumulation steps, each of which cuts at most 2^-23 of
# the sum so far: 2^-20 in the mean. The n / 32 tile sums (weights, and weights times values) are
# rounded to nearest: n / 32 <= 1,024 steps of a partial sum, sqrt(1024 / 3) 2^-24 rms = 1.1e-6. The
# weights' errors (2^-22 and 2^-21 S 2^-22 ...) average out over the keys, as their sign is the key's
# own. 2^-20 + 1.1e-6 = 2.1e-6: 2^-18.8. One accumulator for all keys is cut in one direction at
# every step: 1e-4 of the result at 131,000 keys of a pair, 1.2e-5 at 16,000 (measured).
SUM_BOUND = 2.0 ** -18.8


def one_signed(w, n, page, seed, extra=0):
    g = torch.Generator().manual_seed(seed)
    n_pages = -(-n // page)
    k = torch.randn(n_pages + extra, w.n_kv_heads, page, w.head_dim, generator=g).half()
    v = (0.5 + torch.rand(n_pages + extra, w.n_kv_heads, page, w.head_dim, generator=g)).half()
    rows = lambda t: t[:n_pages].permute(0, 2, 1, 3).reshape(n_pages * page, w.n_kv_heads, w.head_dim)[:n]  # noqa: E731
    return k, v, rows(k), rows(v), g


def assert_unbiased(got, ref):
    rel = (got.double().cpu().numpy() - ref) / ref
    assert abs(rel.mean()) <= SUM_BOUND, rel.mean()
    assert np.sqrt((rel ** 2).mean()) <= SUM_BOUND, np.sqrt((rel ** 2).mean())
    return rel


@pytest.mark.parametrize("w,n", [(R.G8, 131_000), (R.G3_D64, 70_001)], ids=["g8-d128", "g3-d64"])
def test_decode_f32_sums_of_whole_pairs(w, n):
    """More (sequence, KV head) pairs than SMs: a pair's keys stay in one CTA, 1/8 of them in one
    warp's accumulator. All sequences are the same pages."""
    batch, page = 330 // w.n_kv_heads, 128
    k, v, kr, vr, g = one_signed(w, n, page, 5)
    table = torch.arange(k.shape[0], dtype=torch.int32).expand(batch, -1).contiguous()
    cache = PagedCache(w, k.cuda(), v.cuda(), table.cuda(), "f32")
    q = (0.3 * torch.randn(batch, w.n_q_heads, w.head_dim, generator=g)).to(DTYPE[w.in_dtype])
    out = cache.decode(q.cuda(), i32([n] * batch))
    torch.cuda.synchronize()
    q1m.check_status()
    for b in (0, batch // 2, batch - 1):
        ref, _ = R.attend(w, q[b:b + 1], [n - 1], kr, vr)
        assert_unbiased(out[b:b + 1], ref)


def test_prefill_f32_sums_of_whole_row_tiles():
    w, n, new, page = R.G8, 18_000, 2_400, 64
    k, v, kr, vr, g = one_signed(w, n, page, 6)
    table = torch.arange(k.shape[0], dtype=torch.int32).view(1, -1)
    cache = PagedCache(w, k.cuda(), v.cuda(), table.cuda(), "f32")
    q = (0.3 * torch.randn(new, w.n_q_heads, w.head_dim, generator=g)).to(DTYPE[w.in_dtype])
    out = cache.prefill(q.cuda(), i32([n]), i32([0, new]))
    torch.cuda.synchronize()
    q1m.check_status()
    for r in (0, 7, 1_201, new - 1):
        ref, _ = R.attend(w, q[r:r + 1], [n - new + r], kr, vr)
        assert_unbiased(out[r:r + 1], ref)


def test_shared_prefix_f32_sums_of_the_largest_batch():
    """Q1M_MAX_PAGED_BATCH sequences behind a shared prefix, a few keys of their own each."""
    w, prefix, page, batch = R.G8, 18_048, 64, q1m.MAX_PAGED_BATCH
    k, v, kr, vr, g = one_signed(w, prefix, page, 7, extra=batch)
    shared = prefix // page
    table = torch.full((batch, shared + 1), -1, dtype=torch.int32)
    table[:, shared] = shared + torch.arange(batch)
    pre = torch.arange(shared, dtype=torch.int32).cuda()
    cache = PagedCache(w, k.cuda(), v.cuda(), table.cuda(), "f32")
    q = (0.3 * torch.randn(batch, w.n_q_heads, w.head_dim, generator=g)).to(DTYPE[w.in_dtype])
    lens = [prefix + 1 + b % page for b in range(batch)]
    out = cache.decode_shared(q.cuda(), i32(lens), pre, prefix)
    torch.cuda.synchronize()
    q1m.check_status()
    for b in (0, 777, batch - 1):
        m = lens[b] - prefix
        kk = torch.cat([kr, k[shared + b, :, :m].transpose(0, 1)])
        vv = torch.cat([vr, v[shared + b, :, :m].transpose(0, 1)])
        ref, _ = R.attend(w, q[b:b + 1], [lens[b] - 1], kk, vv)
        assert_unbiased(out[b:b + 1], ref)


def test_an_empty_table_serves_an_empty_batch():
    w = R.G2
    c = R.Case(w, [40], 16)
    cache = PagedCache(w, c.k.cuda(), c.v.cuda(), c.table.cuda()[:0], "bf16")
    z = torch.empty(0, w.n_kv_heads, w.head_dim, dtype=torch.bfloat16, device="cuda")
    zq = torch.empty(0, w.n_q_heads, w.head_dim, dtype=torch.bfloat16, device="cuda")
    none, before = torch.empty(0, dtype=torch.int32, device="cuda"), q1m.launch_count()
    cache.append(z, z, none)
    cache.append(z, z, none, i32([0]))
    assert cache.decode(zq, none).shape == (0, 4, 128)
    assert cache.decode_shared(zq, none, i32([0] * 8), 128).shape[0] == 0
    assert cache.prefill(zq, none, i32([0])).shape[0] == 0
    assert q1m.launch_count() == before


@pytest.mark.parametrize("fault", [-1, -6, -7, -8])
def test_a_timeout_behind_an_unpolled_fault_is_reported_and_ends_the_other_waits(fault):
    """20 waits of half a second each that nothing completes, behind a fault that nobody polled: the
    first runs out, the others end at once, and both codes are reported, one a poll."""
    q1m.check_status()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert q1m.selftest_timeout_behind(fault, 20, 1_000_000_000) == -5
    assert time.perf_counter() - t0 < 5
    assert q1m.status_poll() == fault and q1m.status_poll() == 0
    c = R.Case(R.G2, [300], 16, 2)
    cache, q = PagedCache(c.w, c.k.cuda(), c.v.cuda(), c.table.cuda()), c.queries(1)
    out = cache.decode(q.cuda(), i32([300]))
    q1m.check_status()
    ref, _ = R.attend(c.w, q, [299], c.kc[0], c.vc[0])
    tol, _ = R.bounds(c.w, q, c.kc[0], c.vc[0], False)
    R.check(c.w, out, None, ref, None, tol, 0, False)


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_shared_prefix_behind_a_table_narrower_than_it(out_dtype):
    """Sequences that end inside the prefix need no table entries for the rest of it."""
    w, page, prefix, lens = R.G2, 16, 512, [150, 100, 1]
    c = R.Case(w, lens, page, 9, prefix=prefix)
    narrow = torch.full((3, 10), -1, dtype=torch.int32, device="cuda")
    cache = PagedCache(w, c.k.cuda(), c.v.cuda(), narrow, out_dtype)
    q = c.queries(3)
    out = cache.decode_shared(q.cuda(), i32(lens), c.prefix_table.cuda(), prefix)
    torch.cuda.synchronize()
    q1m.check_status()
    for b, ln in enumerate(lens):
        ref, _ = R.attend(w, q[b:b + 1], [ln - 1], c.kc[b], c.vc[b])
        tol, _ = R.bounds(w, q[b:b + 1], c.kc[b], c.vc[b], out_dtype == "bf16")
        R.check(w, out[b:b + 1], None, ref, None, tol, 0, out_dtype == "bf16")


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_waits_that_run_out_at_once_leave_nothing_behind(out_dtype):
    """A wait budget of one cycle: calls may give up (the status says so) at any of their waits; no
    copy or MMA outlives its CTA, nothing unset is used as an address, and with the default budget
    the same buffers give the results that they gave before."""
    w, lens, prefix = R.G2, [5000, 700, 1300, 0], 384
    c = R.Case(w, lens, 32, 5, prefix=prefix)
    cache, ln, pre, new = PagedCache(w, c.k.cuda(), c.v.cuda(), c.table.cuda(), out_dtype), i32(lens), c.prefix_table.cuda(), 600
    q, qp, cu = c.queries(4).cuda(), c.queries(2 * new + 100).cuda(), i32([0, new, 2 * new, 2 * new + 100, 2 * new + 100])
    calls = [lambda: cache.decode(q, ln), lambda: cache.decode(q, ln, 300, 7), lambda: cache.decode_shared(q, ln, pre, prefix),
             lambda: cache.prefill(qp, ln, cu), lambda: cache.prefill(qp, ln, cu, 200, 5)]
    want = [f() for f in calls]
    q1m.check_status()
    try:
        q1m.set_wait_budget(1)
        for f in calls:
            f()
            assert q1m.status_poll() in (0, -5)
    finally:
        q1m.set_wait_budget(0)
    assert q1m.status_poll() == 0
    for f, x in zip(calls, want):
        assert torch.equal(f(), x)
    q1m.check_status()
