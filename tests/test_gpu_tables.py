"""GPU tests of pa_extend_tables and pa_release_tables against a row-by-row
implementation in plain Python: whole numbers, so everything is equal."""
import numpy as np
import pytest
import torch

from paged_kv_cache_429_b200 import (BlockPool, pa_extend_tables, pa_get_device_error,
                                     pa_release_tables)

pytestmark = pytest.mark.gpu

B = 16
OUT_OF_BLOCKS, LENGTH, FREE, BLOCK = 0x20, 0x40, 0x80, 0x10


@pytest.fixture(autouse=True)
def _clean():
    pa_get_device_error()
    yield
    pa_get_device_error()


def plain_extend(tables, lens, new, free, count, T, nb):
    """(tables, lens, count, slots, positions, query_start, flags)."""
    tables, lens = tables.copy(), lens.astype(np.int64)
    S, W = tables.shape
    slots, pos = np.full(T, -1, np.int64), np.zeros(T, np.int32)
    start = np.zeros(S + 1, np.int64)
    need = [-(-int(a + n) // B) - -(-int(a) // B) for a, n in zip(lens, new)]
    flags = 0
    if S and (lens.min() < 0 or new.min() < 0 or (lens + new).max() > W * B):
        flags |= LENGTH
    elif int(new.sum()) > T:
        flags |= LENGTH
    if count < 0 or count > len(free):
        flags |= FREE
    if not flags and sum(need) > count:
        flags |= OUT_OF_BLOCKS
    if flags:
        return tables, lens, count, slots, pos, start, flags
    t = 0
    for s in range(S):
        start[s] = t
        old = -(-int(lens[s]) // B)
        for i in range(need[s]):
            count -= 1
            tables[s, old + i] = free[count]
        for p in range(int(lens[s]), int(lens[s] + new[s])):
            b = int(tables[s, p // B])
            if 0 <= b < nb:
                slots[t] = b * B + p % B
            else:
                flags |= BLOCK
            pos[t] = p
            t += 1
    start[S] = t
    return tables, lens + new, count, slots, pos, start, flags


def plain_release(tables, lens, rel, free, count, keep, nb):
    free, lens = free.copy(), lens.astype(np.int64)
    S, W = tables.shape
    flags = 0
    if any(r and (a < 0 or a > W * B) for a, r in zip(lens, rel)):
        flags |= LENGTH
    held = 0 if flags else sum(max(-(-int(a) // B) - keep, 0) for a, r in zip(lens, rel) if r)
    if count < 0 or count > len(free) or (not flags and count + held > len(free)):
        flags |= FREE
    if flags:
        return free, lens, count, flags
    for s in range(S):
        if not rel[s]:
            continue
        for j in range(keep, -(-int(lens[s]) // B)):
            free[count] = tables[s, j]
            flags |= 0 if 0 <= tables[s, j] < nb else BLOCK
            count += 1
        lens[s] = min(int(lens[s]), keep * B)
    return free, lens, count, flags


def dev(a, dt=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).cuda()


def state(seed, S, W, max_len, nb_spare=40):
    """Tables whose rows hold distinct blocks of a shuffled pool, and the rest as a free stack."""
    g = np.random.default_rng(seed)
    lens = g.integers(0, max_len + 1, S)
    held = -(-lens // B)
    nb = int(held.sum()) + nb_spare
    ids = g.permutation(nb)
    tables = np.full((S, W), -1, np.int32)
    k = 0
    for s in range(S):
        tables[s, :held[s]] = ids[k:k + held[s]]
        k += held[s]
    free = np.concatenate([ids[k:], np.full(k, -7)]).astype(np.int32)
    return g, tables, lens, free, nb - k, nb


def run_extend(tables, lens, new, free, count, T, nb, inplace=False, offset=0):
    t, ln, nw, fr, ct = dev(tables), dev(lens), dev(new), dev(free), dev([count])
    lo = ln if inplace else torch.full_like(ln, -99)
    co = ct if inplace else torch.full_like(ct, -99)
    # outputs at odd offsets inside larger buffers: neighbours must stay
    sl = torch.full((T + offset + 3,), -5, dtype=torch.int64, device="cuda")
    ps = torch.full((T + offset + 3,), -5, dtype=torch.int32, device="cuda")
    qs = torch.full((len(lens) + 1,), -5, dtype=torch.int32, device="cuda")
    pa_extend_tables(t, ln, nw, fr, ct, lo, co, sl[offset:offset + T], ps[offset:offset + T], qs, num_blocks=nb)
    torch.cuda.synchronize()
    for x in (sl, ps):
        assert torch.all(x[:offset] == -5) and torch.all(x[offset + T:] == -5)
    np.testing.assert_array_equal(fr.cpu().numpy(), free)      # only read
    if not inplace:
        np.testing.assert_array_equal(ln.cpu().numpy(), lens)
        assert int(ct) == count
    return [x.cpu().numpy() for x in (t, lo, co, sl[offset:offset + T], ps[offset:offset + T], qs)]


def check_extend(got, want):
    t, lo, co, sl, ps, qs = got
    tables, lens, count, slots, pos, start, flags = want
    np.testing.assert_array_equal(t, tables)
    np.testing.assert_array_equal(lo, lens)
    assert int(co[0]) == count
    np.testing.assert_array_equal(sl, slots)
    np.testing.assert_array_equal(ps, pos)
    np.testing.assert_array_equal(qs, start)
    assert pa_get_device_error() == flags


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("S,W,max_len,new_hi,pad", [
    (1, 1, 0, 16, 0),          # one empty row, one block
    (1, 4, 15, 1, 5),          # a row whose next token may end a block
    (3, 8, 100, 28, 1),
    (33, 16, 200, 1, 7),       # a decode step
    (130, 20, 150, 170, 301),  # prompts
    (1024, 4, 40, 3, 0),       # a thread a row
    (1025, 4, 40, 3, 0),       # and one more
    (5000, 3, 40, 8, 13),
    (2, 700, 20, 11000, 3),    # two long prompts
])
def test_extend_equals_the_plain_form(S, W, max_len, new_hi, pad, inplace):
    for seed in range(2):
        g, tables, lens, free, count, nb = state(seed, S, W, max_len)
        new = np.minimum(g.integers(0, new_hi + 1, S), W * B - lens)
        need = int((-(-(lens + new) // B) - -(-lens // B)).sum())
        extra = np.arange(nb, nb + max(0, need - count), dtype=np.int32)
        free = np.concatenate([free[:count], extra, free[count:]])
        count += len(extra)
        nb += len(extra)
        T = int(new.sum()) + pad
        want = plain_extend(tables, lens, new, free, count, T, nb)
        assert want[-1] == 0
        check_extend(run_extend(tables, lens, new, free, count, T, nb, inplace, offset=seed), want)


def test_extend_the_most_rows():
    S, W = 16384, 2
    g, tables, lens, free, count, nb = state(5, S, W, 31, nb_spare=20000)
    new = np.minimum(g.integers(0, 2, S), W * B - lens)
    want = plain_extend(tables, lens, new, free, count, S, nb)
    check_extend(run_extend(tables, lens, new, free, count, S, nb), want)


def test_extend_without_rows_or_tokens():
    got = run_extend(np.empty((0, 4), np.int32), np.empty(0, np.int64), np.empty(0, np.int64),
                     np.arange(5, dtype=np.int32), 3, 6, 5)
    check_extend(got, plain_extend(np.empty((0, 4), np.int32), np.empty(0, np.int64), np.empty(0, np.int64),
                                   np.arange(5, dtype=np.int32), 3, 6, 5))
    g, tables, lens, free, count, nb = state(1, 9, 8, 60)
    got = run_extend(tables, lens, np.zeros(9, np.int64), free, count, 0, nb)
    check_extend(got, plain_extend(tables, lens, np.zeros(9, np.int64), free, count, 0, nb))


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("what", ["blocks", "row", "tokens", "negative_new", "negative_len", "count_low",
                                  "count_high", "long_len"])
def test_extend_is_all_or_nothing(what, inplace):
    g, tables, lens, free, count, nb = state(3, 70, 12, 100)
    new = np.full(70, 3)
    T = 70 * 3 + 4
    if what == "blocks":
        count = 2
    elif what == "row":
        new[41] = 12 * B - lens[41] + 1
    elif what == "tokens":
        T = 70 * 3 - 1
    elif what == "negative_new":
        new[69] = -1
    elif what == "negative_len":
        lens[0] = -5
    elif what == "count_low":
        count = -1
    elif what == "count_high":
        count = len(free) + 1
    elif what == "long_len":
        lens[7] = 2 ** 31 - 2
    want = plain_extend(tables, lens, new, free, count, T, nb)
    assert want[-1] != 0 and np.all(want[3] == -1)
    check_extend(run_extend(tables, lens, new, free, count, T, nb, inplace), want)


def test_extend_sums_past_32_bits_are_refused():
    """Rows whose token counts add up to 2^32 + 2: a 32-bit sum would see 2."""
    W = 2 ** 26
    S = 5
    lens = np.zeros(S, np.int64)
    new = np.array([2 ** 30] * 4 + [2])
    # the table is never touched: nothing is done
    t = torch.zeros((S, 1), dtype=torch.int32, device="cuda")
    from paged_kv_cache_429_b200 import _lib
    ln, nw, fr, ct = dev(lens), dev(new), dev(np.arange(64)), dev([64])
    sl = torch.zeros(8, dtype=torch.int64, device="cuda")
    ps, qs = torch.ones(8, dtype=torch.int32, device="cuda"), torch.ones(S + 1, dtype=torch.int32, device="cuda")
    rc = _lib.lib().pa_extend_tables(t.data_ptr(), W, ln.data_ptr(), nw.data_ptr(), fr.data_ptr(), 64, ct.data_ptr(),
                                     ln.data_ptr(), ct.data_ptr(), sl.data_ptr(), ps.data_ptr(), qs.data_ptr(), S, 8,
                                     16, 64, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert int(ct) == 64 and torch.all(sl == -1) and torch.all(qs == 0) and torch.all(ln == 0)
    assert pa_get_device_error() == LENGTH


def test_extend_flags_ids_outside_the_pool():
    g, tables, lens, free, count, nb = state(4, 6, 8, 90)
    lens[:] = [5, 33, 40, 1, 16, 90]
    new = np.full(6, 14)
    tables[1, 2] = nb          # row 1's partly filled block
    free[count - 1] = -3       # the first block popped
    want = plain_extend(tables, lens, new, free, count, 90, nb)
    assert want[-1] == BLOCK
    check_extend(run_extend(tables, lens, new, free, count, 90, nb), want)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("S,W,max_len,share,keep", [
    (1, 1, 16, 1.0, 0), (1, 1, 0, 1.0, 0), (40, 20, 320, 0.3, 0), (40, 20, 320, 0.5, 4), (40, 20, 320, 1.0, 20),
    (40, 20, 320, 0.9, 1000), (1025, 6, 96, 0.5, 1), (5000, 3, 48, 0.7, 0), (16384, 2, 32, 0.5, 0),
    (3, 600, 9600, 1.0, 2), (0, 4, 4, 1.0, 0),
])
def test_release_equals_the_plain_form(S, W, max_len, share, keep, inplace):
    g, tables, lens, free, count, nb = state(11, S, W, max_len)
    rel = (g.random(S) < share) * g.integers(-2, 3, S)  # any non-zero value ends a row
    fr, ln, ct, tb = dev(free), dev(lens), dev([count]), dev(tables)
    lo = ln if inplace else torch.full_like(ln, -9)
    co = ct if inplace else torch.full_like(ct, -9)
    pa_release_tables(tb, ln, dev(rel), fr, ct, lo, co, keep_blocks=keep, num_blocks=nb)
    torch.cuda.synchronize()
    wf, wl, wc, flags = plain_release(tables, lens, rel, free, count, keep, nb)
    assert flags == 0
    np.testing.assert_array_equal(fr.cpu().numpy(), wf)
    np.testing.assert_array_equal(lo.cpu().numpy(), wl)
    assert int(co) == wc
    np.testing.assert_array_equal(tb.cpu().numpy(), tables)
    assert pa_get_device_error() == 0


@pytest.mark.parametrize("what", ["full", "count_low", "count_high", "length", "bad_id"])
def test_release_refuses_on_the_device(what):
    g, tables, lens, free, count, nb = state(12, 20, 8, 120)
    lens[3] = 77
    rel = np.ones(20, np.int64)
    if what == "full":
        free = free[:count + 5]
    elif what == "count_low":
        count = -2
    elif what == "count_high":
        count = len(free) + 1
    elif what == "length":
        lens[3] = 8 * B + 1
    elif what == "bad_id":
        tables[3, 1] = nb + 4
    fr, ln, ct = dev(free), dev(lens), dev([count])
    pa_release_tables(dev(tables), ln, dev(rel), fr, ct, ln, ct, num_blocks=nb)
    torch.cuda.synchronize()
    wf, wl, wc, flags = plain_release(tables, lens, rel, free, count, 0, nb)
    assert flags != 0
    np.testing.assert_array_equal(fr.cpu().numpy(), wf)
    np.testing.assert_array_equal(ln.cpu().numpy(), wl)
    assert int(ct) == wc
    assert pa_get_device_error() == flags


def test_steps_in_a_graph_follow_the_host_pool():
    """Decode steps captured once and replayed, rows ended and restarted
    between replays: lengths and block counts equal a host pool's that does
    the same, no block is held twice, and none is lost."""
    S, W, NB = 24, 12, 260
    pool = BlockPool(NB)
    for s in range(S):
        pool.add_seq(s)
    g = np.random.default_rng(0)
    tables = torch.full((S, W), -1, dtype=torch.int32, device="cuda")
    lens, count = dev(np.zeros(S)), dev([NB])
    free = dev(g.permutation(NB))
    new, rel = dev(np.ones(S)), dev(np.zeros(S))
    T = 3 * S
    slots = torch.empty(T, dtype=torch.int64, device="cuda")
    pos, qs = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(S + 1, dtype=torch.int32, device="cuda")

    def step():
        pa_release_tables(tables, lens, rel, free, count, lens, count)
        pa_extend_tables(tables, lens, new, free, count, lens, count, slots, pos, qs)

    rel0 = rel.clone()
    new.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()   # nothing ends, nothing comes: only warms the launches
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(60):
        n = g.integers(0, 4, S)
        r = (g.random(S) < 0.08).astype(np.int64)
        cur = np.array([pool.seq_len(s) for s in range(S)])
        r[cur + 3 > W * B] = 1
        for s in range(S):
            if r[s]:
                pool.free_seq(s)
                pool.add_seq(s)
            if n[s]:
                pool.append(s, int(n[s]))
        new.copy_(dev(n))
        rel.copy_(dev(r))
        graph.replay()
        torch.cuda.synchronize()
        want = np.array([pool.seq_len(s) for s in range(S)])
        np.testing.assert_array_equal(lens.cpu().numpy(), want)
        assert int(count) == pool.num_free
        tb, k = tables.cpu().numpy(), int(count)
        held = np.concatenate([tb[s, :-(-int(want[s]) // B)] for s in range(S)] + [free.cpu().numpy()[:k]])
        assert len(np.unique(held)) == NB == len(held)
        sl = slots.cpu().numpy()
        total = int(n.sum())
        assert np.all(sl[total:] == -1) and len(np.unique(sl[:total])) == total
        at = 0
        for s in range(S):
            for p in range(int(want[s] - n[s]), int(want[s])):
                assert sl[at] == tb[s, p // B] * B + p % B and int(pos[at]) == p
                at += 1
    assert pa_get_device_error() == 0
    del graph
    assert torch.count_nonzero(rel0) == 0


def uneven(g, S, long):
    """Rows of 0, 1, 2, 3 and many tokens beside one another, in runs."""
    kinds = g.choice(6, S, p=[0.3, 0.2, 0.15, 0.1, 0.1, 0.15])
    return np.where(kinds < 4, kinds, g.integers(4, long, S))


@pytest.mark.parametrize("S,long,pad,offset", [
    (64, 40, 0, 0),        # one CTA
    (90, 130, 3, 1),       # about 2048 tokens, outputs off their alignment
    (700, 200, 17, 0),     # a large call whose threads meet up to four rows
    (3000, 90, 1, 3),
])
def test_extend_rows_of_uneven_lengths(S, long, pad, offset):
    g, tables, lens, free, count, nb = state(S + long, S, 24, 150, nb_spare=S * 16)
    new = uneven(g, S, long)
    new = np.minimum(new, 24 * B - lens)
    T = int(new.sum()) + pad
    got = run_extend(tables, lens, new, free, count, T, nb, offset=offset)
    check_extend(got, plain_extend(tables, lens, new, free, count, T, nb))


@pytest.mark.parametrize("tokens", [2047, 2048, 2049, 4096, 4097])
def test_extend_where_the_calls_split(tokens):
    """The two sides of the one-CTA rule give the same."""
    g, tables, lens, free, count, nb = state(tokens, 5, 200, 600, nb_spare=400)
    new = np.full(5, tokens // 5)
    new[2] += tokens - int(new.sum())
    got = run_extend(tables, lens, new, free, count, tokens, nb)
    check_extend(got, plain_extend(tables, lens, new, free, count, tokens, nb))


@pytest.mark.parametrize("keep", [0, 2])
@pytest.mark.parametrize("S,W", [(64, 128), (64, 130), (700, 24), (3000, 9)])
def test_release_rows_of_uneven_lengths(S, W, keep):
    g = np.random.default_rng(S + W + keep)
    blocks = np.minimum(uneven(g, S, W + 1), W)
    lens = np.maximum(blocks * B - g.integers(0, B, S), 0)
    held = -(-lens // B)
    nb = int(held.sum()) + 3
    tables = np.full((S, W), -1, np.int32)
    ids = g.permutation(nb)
    for s, e in enumerate(np.cumsum(held)):
        tables[s, :held[s]] = ids[e - held[s]:e]
    rel = (g.random(S) < 0.8).astype(np.int32)
    free = np.full(nb + 5, -7, np.int32)
    fr, ct, ln = dev(free), dev([2]), dev(lens)
    pa_release_tables(dev(tables), ln, dev(rel), fr, ct, ln, ct, keep_blocks=keep, num_blocks=nb)
    want, wl, wc, flags = plain_release(tables, lens, rel, free, 2, keep, nb)
    np.testing.assert_array_equal(fr.cpu().numpy(), want)
    np.testing.assert_array_equal(ln.cpu().numpy(), wl)
    assert int(ct) == wc and pa_get_device_error() == flags == 0


def test_calls_behind_one_another_see_each_others_results():
    """Large calls in place, without a synchronisation between: the next
    call's first launch must find the last one's lengths and count."""
    g, tables, lens, free, count, nb = state(5, 600, 40, 60, nb_spare=30000)
    t, ln, fr, ct = dev(tables), dev(lens), dev(free), dev([count])
    news = [g.integers(0, 30, 600) for _ in range(8)]
    rels = [(g.random(600) < 0.3).astype(np.int32) for _ in range(8)]
    T = 20000
    sl = torch.empty(T, dtype=torch.int64, device="cuda")
    ps, qs = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(601, dtype=torch.int32, device="cuda")
    dn, dr = [dev(n) for n in news], [dev(r) for r in rels]
    torch.cuda.synchronize()
    for n, r in zip(dn, dr):
        pa_extend_tables(t, ln, n, fr, ct, ln, ct, sl, ps, qs, num_blocks=nb)
        pa_release_tables(t, ln, r, fr, ct, ln, ct, num_blocks=nb)
    for n, r in zip(news, rels):
        tables, lens, count, slots, pos, start, flags = plain_extend(tables, lens, n, free, count, T, nb)
        assert flags == 0
        free, lens, count, flags = plain_release(tables, lens, r, free, count, 0, nb)
        assert flags == 0
    np.testing.assert_array_equal(t.cpu().numpy(), tables)
    np.testing.assert_array_equal(ln.cpu().numpy(), lens)
    np.testing.assert_array_equal(fr.cpu().numpy()[:count], free[:count])
    np.testing.assert_array_equal(sl.cpu().numpy(), slots)
    np.testing.assert_array_equal(ps.cpu().numpy(), pos)
    assert int(ct) == count and pa_get_device_error() == 0


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("what", ["blocks", "row", "tokens", "negative_new", "negative_len", "count_low",
                                  "count_high", "long_len", "two"])
def test_large_extends_are_all_or_nothing(what, inplace):
    """The same refusals where the call is two launches (more than 2048 tokens)."""
    S, W = 700, 12
    g, tables, lens, free, count, nb = state(6, S, W, 100, nb_spare=1500)
    new = np.full(S, 5)
    T = S * 5 + 9
    if what in ("blocks", "two"):
        count = int((-(-(lens + new) // B) - -(-lens // B)).sum()) - 1
    if what in ("row", "two"):
        new[699] = W * B - lens[699] + 1
    if what == "tokens":
        T = S * 5 - 1
    elif what == "negative_new":
        new[350] = -1
    elif what == "negative_len":
        lens[0] = -5
    elif what == "count_low":
        count = -1
    elif what == "count_high":
        count = len(free) + 1
    elif what == "long_len":
        lens[7] = 2 ** 31 - 2
    want = plain_extend(tables, lens, new, free, count, T, nb)
    assert want[-1] not in (0, BLOCK) and np.all(want[3] == -1)
    check_extend(run_extend(tables, lens, new, free, count, T, nb, inplace), want)


def test_a_large_extend_takes_the_last_block():
    S, W = 700, 12
    g, tables, lens, free, count, nb = state(6, S, W, 100, nb_spare=1500)
    new = np.full(S, 5)
    need = int((-(-(lens + new) // B) - -(-lens // B)).sum())
    want = plain_extend(tables, lens, new, free, need, S * 5, nb)
    assert want[-1] == 0 and want[2] == 0
    check_extend(run_extend(tables, lens, new, free, need, S * 5, nb), want)


def test_a_large_extend_flags_ids_outside_the_pool():
    S, W = 700, 12
    g, tables, lens, free, count, nb = state(6, S, W, 100, nb_spare=1500)
    new = np.full(S, 5)
    lens[1] = 33
    tables[1, 2] = nb          # a partly filled block
    free[count - 2] = -3       # the second block popped
    want = plain_extend(tables, lens, new, free, count, S * 5 + 1, nb)
    assert want[-1] == BLOCK
    check_extend(run_extend(tables, lens, new, free, count, S * 5 + 1, nb), want)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("what", ["full", "count_low", "count_high", "length", "negative", "bad_id", "fits"])
def test_large_releases_refuse_on_the_device(what, inplace):
    """Where the call is two launches (a bound of more than 8192 blocks)."""
    S, W = 700, 14
    g, tables, lens, free, count, nb = state(14, S, W, W * B)
    lens[3] = 77
    rel = (g.random(S) < 0.9).astype(np.int64)
    rel[[3, 699]] = 1
    held = int(sum(-(-int(a) // B) for a, r in zip(lens, rel) if r))
    if what in ("full", "fits"):
        free = free[:count + held - (what == "full")]
    elif what == "count_low":
        count = -2
    elif what == "count_high":
        count = len(free) + 1
    elif what == "length":
        lens[699] = W * B + 1
    elif what == "negative":
        lens[3] = -1
    elif what == "bad_id":
        tables[3, 1] = nb + 4
    fr, ln, ct = dev(free), dev(lens), dev([count])
    lo = ln if inplace else torch.full_like(ln, -9)
    co = ct if inplace else torch.full_like(ct, -9)
    pa_release_tables(dev(tables), ln, dev(rel), fr, ct, lo, co, num_blocks=nb)
    torch.cuda.synchronize()
    wf, wl, wc, flags = plain_release(tables, lens, rel, free, count, 0, nb)
    assert (flags != 0) == (what != "fits")
    np.testing.assert_array_equal(fr.cpu().numpy(), wf)
    np.testing.assert_array_equal(lo.cpu().numpy(), wl)
    assert int(co) == wc
    assert pa_get_device_error() == flags


def test_tables_of_more_than_2_to_31_entries():
    """Rows that start past 2^31 entries of the table, one CTA and two launches."""
    W = (1 << 27) - 9               # columns: just below the most
    S = -(-(1 << 31) // W) + 2      # 19 rows, the last ones past 2^31
    tables = torch.full((S, W), -1, dtype=torch.int32, device="cuda")
    lens = np.zeros(S, np.int64)
    lens[S - 1], lens[S - 2], lens[3] = 16 * (W - 200) + 5, 33, 1
    tables[S - 2, :2] = 14
    tables[S - 1, W - 200], tables[S - 2, 2], tables[3, 0] = 11, 12, 13
    for new_tokens in (17, 2100):
        new = np.zeros(S, np.int64)
        new[S - 1], new[S - 2], new[3] = new_tokens, 20, 0
        need = int((-(-(lens + new) // B) - -(-lens // B)).sum())
        ln, fr, ct = dev(lens), dev(np.arange(100, 100 + need)), dev([need])
        T = int(new.sum()) + 3
        sl = torch.empty(T, dtype=torch.int64, device="cuda")
        ps, qs = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(S + 1, dtype=torch.int32, device="cuda")
        pa_extend_tables(tables, ln, dev(new), fr, ct, ln, ct, sl, ps, qs, num_blocks=1000)
        torch.cuda.synchronize()
        assert pa_get_device_error() == 0 and int(ct) == 0
        np.testing.assert_array_equal(ln.cpu().numpy(), lens + new)
        stack, at, got = list(range(100, 100 + need)), 0, sl.cpu().numpy()
        for s in range(S):
            ids = {int(lens[s]) // B: {S - 1: 11, S - 2: 12, 3: 13}.get(s)}
            for p in range(int(lens[s]), int(lens[s] + new[s])):
                if p % B == 0:
                    ids[p // B] = stack.pop()
                    assert int(tables[s, p // B]) == ids[p // B]
                assert got[at] == ids[p // B] * B + p % B and int(ps[at]) == p
                at += 1
        assert np.all(got[at:] == -1)
        # and back: a small bound keeps every block but the row's last ones
        rel = np.zeros(S, np.int64)
        rel[S - 1] = 1
        keep = int(lens[S - 1]) // B + 1
        fr2, ct2, l2 = dev(np.full(need + 2, -7)), dev([1]), torch.empty_like(ln)
        c2 = torch.empty_like(ct2)
        pa_release_tables(tables, ln, dev(rel), fr2, ct2, l2, c2, keep_blocks=keep, num_blocks=1000)
        torch.cuda.synchronize()
        n = -(-int(lens[S - 1] + new[S - 1]) // B) - keep
        assert int(c2) == 1 + n and pa_get_device_error() == 0
        np.testing.assert_array_equal(fr2.cpu().numpy()[1:1 + n], tables[S - 1, keep:keep + n].cpu().numpy())
        assert int(l2[S - 1]) == keep * B
        # without a bound two launches; the row before, whole
        rel[:] = 0
        rel[S - 2] = 1
        fr2, ct2 = dev(np.full(9, -7)), dev([2])
        pa_release_tables(tables, ln, dev(rel), fr2, ct2, l2, c2, num_blocks=1000)
        torch.cuda.synchronize()
        assert int(c2) == 6 and int(l2[S - 2]) == 0 and pa_get_device_error() == 0
        np.testing.assert_array_equal(fr2.cpu().numpy()[2:6], tables[S - 2, :4].cpu().numpy())


def test_large_calls_captured_and_replayed():
    """Both two-launch calls in place in one graph, other rows each time, a
    refused step among them."""
    g, tables, lens, free, count, nb = state(7, 600, 40, 60, nb_spare=30000)
    t, ln, fr, ct = dev(tables), dev(lens), dev(free), dev([count])
    T = 12000
    sl = torch.empty(T, dtype=torch.int64, device="cuda")
    ps, qs = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(601, dtype=torch.int32, device="cuda")
    new, rel = dev(np.zeros(600)), dev(np.zeros(600))

    def step():
        pa_extend_tables(t, ln, new, fr, ct, ln, ct, sl, ps, qs, num_blocks=nb)
        pa_release_tables(t, ln, rel, fr, ct, ln, ct, num_blocks=nb)

    step()                       # of nothing: loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(6):
        n, r = g.integers(0, 30, 600), (g.random(600) < 0.3).astype(np.int32)
        if i == 3:
            n[5] = 40 * B        # past its table
        new.copy_(dev(n))
        rel.copy_(dev(r))
        graph.replay()
        torch.cuda.synchronize()
        tables, lens, count, slots, pos, start, flags = plain_extend(tables, lens, n, free, count, T, nb)
        assert (flags == LENGTH) == (i == 3)
        assert pa_get_device_error() == flags
        free, lens, count, flags = plain_release(tables, lens, r, free, count, 0, nb)
        assert flags == 0
        for got, want in ((t, tables), (ln, lens), (sl, slots), (ps, pos), (qs, start), (ct, [count])):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        np.testing.assert_array_equal(fr.cpu().numpy()[:count], free[:count])
    del graph
