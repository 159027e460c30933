"""GPU tests of the serving-step operators used together.

A step of a serving loop whose requests share a system prompt, all on the
device: finished rows give their blocks back (pa_release_tables), every row
gets its next token's block and slot (pa_extend_tables), the queries and
keys are rotated and cached (pa_rope_and_cache), and the batch decodes
behind its shared prefix (pa_decode_shared_prefix). It is captured as one
CUDA graph and replayed; a row-by-row model on the host follows it.
"""
import numpy as np
import pytest
import torch

import oracle
import synth
import paged_kv_cache_429_b200 as pa
from paged_kv_cache_429_b200.batch import DecodeBatch
from parity_harness import (assert_cache_equal, max_abs_err, oracle_caches, oracle_decode, to_u8,
                            to_u16)

pytestmark = pytest.mark.gpu

B = 16


@pytest.fixture(autouse=True)
def _clean():
    pa.pa_get_device_error()
    yield
    pa.pa_get_device_error()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_serving_steps(fp8):
    S, HQ, HKV, D, W, NB, PRE = 19, 16, 4, 128, 12, 150, 5
    g = torch.Generator(device="cuda").manual_seed(3)
    rng = np.random.default_rng(4)
    rnd = lambda *n: torch.randn(n, generator=g, device="cuda").to(torch.bfloat16)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    ks, vs = (0.02, 0.01) if fp8 else (1.0, 1.0)
    inv, scale = pa.pa_rope_frequencies(D, 10000.0, pa.PA_ROPE_BANDS, factor=8.0, original_max_position=64,
                                        high=4.0, device="cuda")
    sentinel = synth.SENTINEL_FP8 if fp8 else synth.SENTINEL_BF16
    kc = torch.full((NB, HKV, B, D), sentinel, dtype=torch.uint8 if fp8 else torch.int16, device="cuda")
    kc = kc if fp8 else kc.view(torch.bfloat16)
    vc = kc.clone()

    # the host pool hands out the prefix and, as one reserved sequence, the
    # blocks of the device's free stack
    pool = pa.BlockPool(NB, shuffle_seed=1)
    pool.add_seq(0)
    pslots, _ = pool.append(0, PRE * B)
    pool.add_seq(1)
    pool.append(1, (NB - PRE) * B)
    ids, _ = pool.block_tables([0, 1], NB - PRE)
    prefix, stack = ids[0, :PRE], ids[1]
    qkv = rnd(PRE * B, HQ + 2 * HKV, D)
    out_q = torch.empty((PRE * B, HQ, D), dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_and_cache(out_q, qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], kc, vc,
                         torch.from_numpy(pslots).cuda(), torch.arange(PRE * B, dtype=torch.int32, device="cuda"),
                         inv, rope_scale=scale, k_scale=ks, v_scale=vs)

    tables = i32(np.full((S, W), -1))
    tables[:, :PRE] = i32(prefix)
    lens, count, free = i32(np.full(S, PRE * B)), i32([NB - PRE]), i32(stack)
    new, rel = i32(np.ones(S)), i32(np.zeros(S))
    slots, pos = torch.empty(S, dtype=torch.int64, device="cuda"), i32(np.zeros(S))
    start = i32(np.zeros(S + 1))
    qkv = rnd(S, HQ + 2 * HKV, D)
    q = torch.empty((S, HQ, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((S, HQ, D), device="cuda")
    group, blocks = i32([0, S]), i32([PRE])

    def step():
        pa.pa_release_tables(tables, lens, rel, free, count, lens, count, keep_blocks=PRE, num_blocks=NB)
        pa.pa_extend_tables(tables, lens, new, free, count, lens, count, slots, pos, start, num_blocks=NB)
        pa.pa_rope_and_cache(q, qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], kc, vc, slots, pos, inv,
                             rope_scale=scale, k_scale=ks, v_scale=vs)
        pa.pa_decode_shared_prefix(out, q, kc, vc, tables, lens, W * B, group, blocks, PRE, D ** -0.5,
                                   max_suffix_len=(W - PRE) * B, k_scale=ks, v_scale=vs)

    state = [t.clone() for t in (tables, lens, count, free, kc.view(torch.uint8), vc.view(torch.uint8))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((tables, lens, count, free, kc.view(torch.uint8), vc.view(torch.uint8)), state):
        t.copy_(s)

    m_tables = np.tile(np.concatenate([prefix, np.full(W - PRE, -1)]), (S, 1))
    m_lens, m_free = np.full(S, PRE * B), list(stack)
    for i in range(45):
        ended = rng.random(S) < 0.04
        ended |= m_lens + 1 > W * B
        for s in np.flatnonzero(ended):
            m_free += [int(m_tables[s, j]) for j in range(PRE, -(-int(m_lens[s]) // B))]
            m_lens[s] = PRE * B
        want_slots = []
        for s in range(S):
            j, off = divmod(int(m_lens[s]), B)
            if off == 0:
                m_tables[s, j] = m_free.pop()
            want_slots.append(int(m_tables[s, j]) * B + off)
            m_lens[s] += 1
        rel.copy_(i32(ended))
        qkv.copy_(rnd(S, HQ + 2 * HKV, D))
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(lens.cpu().numpy(), m_lens)
        assert int(count) == len(m_free)
        np.testing.assert_array_equal(free.cpu().numpy()[:len(m_free)], m_free)
        np.testing.assert_array_equal(slots.cpu().numpy(), want_slots)
        np.testing.assert_array_equal(pos.cpu().numpy(), m_lens - 1)
        tb = tables.cpu().numpy()
        for s in range(S):
            n = -(-int(m_lens[s]) // B)
            np.testing.assert_array_equal(tb[s, :n], m_tables[s, :n])
        if i % 9 == 8:   # the decode, against the oracle on the rotated queries and the cache as they stand
            to = to_u8 if fp8 else to_u16
            ref = oracle.paged_decode(to_u16(q), to(kc), to(vc), m_tables.astype(np.int32), m_lens.astype(np.int32),
                                      D ** -0.5, kv_dtype=oracle.KV_FP8_E4M3 if fp8 else oracle.KV_BF16, k_scale=ks,
                                      v_scale=vs)
            got = out.double().cpu().numpy()
            assert np.all(np.isfinite(got))
            assert np.linalg.norm(got - ref) <= 2e-5 * np.linalg.norm(ref)
            # the rotated queries, against the formula (half a step of bf16, and fp32's roundings on the pair)
            x = qkv[:, :HQ].double()
            ang = torch.outer(pos.double(), inv)[:, None]
            a, b = x[..., :D // 2], x[..., D // 2:]
            want = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1) * scale
            mag = torch.cat([a.abs() + b.abs()] * 2, -1) * scale
            assert torch.all((q.double() - want).abs() <= want.abs() * 2.0 ** -8 + mag * 2.0 ** -20)
    assert pa.pa_get_device_error() == 0
    del graph


def test_prefix_workload_step_shared():
    """The prefix workload (256 forked sequences, copy-on-write) decoded as
    one group: 32 sequences against the oracle, all against the plain decode."""
    b = DecodeBatch.build(synth.WORKLOADS["prefix"], 0, "cuda:0")
    b.out.fill_(float("nan"))
    b.step_shared()
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    shared = b.out.clone()
    assert torch.all(torch.isfinite(shared))
    b.decode()
    # both within their roundings of the same values (two 16-bit halves of each weight: 2^-17)
    assert float((shared - b.out).norm()) <= 2e-5 * float(b.out.norm())
    sub = np.random.default_rng(1).choice(b.w.num_seqs, 8, replace=False)
    kc, vc = oracle_caches(b, subset=sub)
    assert_cache_equal(b, kc, vc, subset=sub)
    ref = oracle_decode(b, kc, vc, subset=sub)
    assert max_abs_err(shared, ref, subset=sub) <= 5e-5


@pytest.mark.parametrize("name", ["tiny", "gqa_fp8"])
def test_step_shared_without_a_prefix(name):
    b = DecodeBatch.build(synth.WORKLOADS[name], 1, "cuda:0")
    b.step_shared()
    shared = b.out.clone()
    b.decode(partition_size=0)
    # the plain fp8 decode keeps about 9 bits of each weight
    assert float((shared - b.out).norm()) <= (2e-3 if b.w.kv_fp8 else 2e-5) * float(b.out.norm())
    assert pa.pa_get_device_error() == 0


def small(dtype=torch.bfloat16):
    S, HQ, HKV, D, NB = 5, 8, 2, 64, 30
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *n: torch.randn(n, generator=g, device="cuda").to(torch.bfloat16)
    cache = lambda: (rnd(NB, HKV, B, D).float().clamp(-400, 400).to(dtype) if dtype == torch.float8_e4m3fn
                     else rnd(NB, HKV, B, D))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    return S, HQ, HKV, D, NB, rnd, cache, i32


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_explicit_stream_and_workspace_give_the_same(dtype):
    """A given stream or workspace goes another way through the binding."""
    S, HQ, HKV, D, NB, rnd, cache, i32 = small(dtype)
    fp8 = dtype != torch.bfloat16
    ks, vs = (0.02, 0.03) if fp8 else (1.0, 1.0)
    k, v = cache(), cache()
    perm = torch.randperm(NB, device="cuda").to(torch.int32)
    tables = perm[:S * 6].view(S, 6).clone()
    tables[:, :2] = tables[0, :2]
    lens, free, count = i32([33, 90, 32, 40, 95]), perm.clone(), i32([NB])
    results = []
    for stream in (None, torch.cuda.current_stream()):
        t, kc, vc, f = tables.clone(), k.clone(), v.clone(), free.clone()
        lo, co, rel = torch.empty_like(lens), torch.empty_like(count), i32([0, 1, 0, 0, 3])
        sl = torch.empty(9, dtype=torch.int64, device="cuda")
        ps, qs = torch.empty(9, dtype=torch.int32, device="cuda"), torch.empty(S + 1, dtype=torch.int32, device="cuda")
        pa.pa_extend_tables(t, lens, i32([2, 1, 0, 3, 1]), f, count, lo, co, sl, ps, qs, num_blocks=NB, stream=stream)
        l2, c2 = torch.empty_like(lens), torch.empty_like(count)
        big = torch.cat([f, torch.zeros_like(f)])
        pa.pa_release_tables(t, lo, rel, big, co, l2, c2, keep_blocks=2, num_blocks=NB, stream=stream)
        g = torch.Generator(device="cuda").manual_seed(9)
        x = torch.randn((9, HQ + 2 * HKV, D), generator=g, device="cuda").to(torch.bfloat16)
        inv, _ = pa.pa_rope_frequencies(32, device="cuda")
        qo = torch.empty((9, HQ, D), dtype=torch.bfloat16, device="cuda")
        pa.pa_rope_and_cache(qo, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], kc, vc, sl, ps, inv, interleaved=True,
                             k_scale=ks, v_scale=vs, stream=stream)
        out = torch.empty((S, HQ, D), device="cuda")
        n = pa.pa_decode_shared_prefix_workspace_size(S, HQ, HKV, D, 1, 2, 80)
        ws = None if stream is None else torch.empty(n, dtype=torch.uint8, device="cuda")
        pa.pa_decode_shared_prefix(out, qo[:S].contiguous(), kc, vc, t, lo, 96, i32([0, S]), i32([2]), 2, 0.125,
                                   max_suffix_len=80, k_scale=ks, v_scale=vs, workspace=ws, stream=stream)
        torch.cuda.synchronize()
        assert pa.pa_get_device_error() == 0
        results.append([y.view(torch.uint8).clone() if y.dtype == dtype and fp8 else y.clone()
                        for y in (t, lo, co, sl, ps, qs, big, l2, c2, qo, kc, vc, out)])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_the_binding_says_what_is_wrong():
    S, HQ, HKV, D, NB, rnd, cache, i32 = small()
    k, v, q = cache(), cache(), rnd(S, HQ, D)
    out = torch.empty((S, HQ, D), device="cuda")
    t, lens, gs, pb = i32([[0, 1]] * S), i32([20] * S), i32([0, S]), i32([1])

    def dec(**kw):
        a = dict(out=out, q=q, k=k, v=v, t=t, lens=lens, gs=gs, pb=pb, scale=0.125, ws=None)
        a.update(kw)
        return pa.pa_decode_shared_prefix(a["out"], a["q"], a["k"], a["v"], a["t"], a["lens"], 32, a["gs"], a["pb"], 1,
                                          a["scale"], workspace=a["ws"])
    dec()
    with pytest.raises(TypeError, match="out: dtype"):
        dec(out=out.double())
    with pytest.raises(ValueError, match="q must be contiguous"):
        dec(q=rnd(S, D, HQ).transpose(1, 2))
    with pytest.raises(ValueError, match="CUDA device"):
        dec(lens=lens.cpu())
    with pytest.raises(ValueError, match="shape mismatch"):
        dec(out=torch.empty((S + 1, HQ, D), device="cuda"))
    with pytest.raises(ValueError, match="group_start"):
        dec(gs=i32([0, 2, S]))
    with pytest.raises(ValueError, match="rows"):
        dec(lens=i32([20] * (S - 1)))
    with pytest.raises(TypeError, match="v_cache"):
        dec(v=v.view(torch.uint8)[..., :D].contiguous())
    with pytest.raises(pa.PagedAttentionError, match="PA_ERR_INVALID_ARG"):
        dec(scale=float("nan"))
    with pytest.raises(pa.PagedAttentionError, match="PA_ERR_WORKSPACE"):
        dec(ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="torch.Tensor"):
        dec(t=[[0, 1]] * S)
    inv, _ = pa.pa_rope_frequencies(64, device="cuda")
    slots, kv = torch.arange(S, device="cuda"), rnd(S, HKV, D)
    with pytest.raises(ValueError, match="key / value"):
        pa.pa_rope_and_cache(q.clone(), q, kv[:, :1], kv[:, :1], k, v, slots, lens, inv)
    with pytest.raises(TypeError, match="inv_freq"):
        pa.pa_rope_and_cache(q.clone(), q, kv, kv, k, v, slots, lens, inv.float())
    with pytest.raises(pa.PagedAttentionError, match="PA_ERR_UNSUPPORTED"):
        pa.pa_rope_and_cache(q.clone(), q, kv, kv, k, v, slots, lens, inv[:12])
    with pytest.raises(ValueError, match="free_count"):
        pa.pa_release_tables(t, lens, lens, t.view(-1), i32([1, 2]), lens, i32([0]))
    with pytest.raises(ValueError, match="positions"):
        pa.pa_extend_tables(t, lens, lens, t.view(-1), i32([1]), lens, i32([0]), slots, lens[:3], i32([0] * (S + 1)))
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0


def test_numbers_outside_their_range_are_refused():
    """Through the extension and, with a stream given, through ctypes."""
    S, HQ, HKV, D, NB, rnd, cache, i32 = small()
    k, q = cache(), rnd(S, HQ, D)
    out = torch.empty((S, HQ, D), device="cuda")
    t, lens, zero, one = i32([[0, 1]] * S), i32([20] * S), i32([0] * S), i32([1])
    free, slots, qs = i32([5, 6, 7]), torch.arange(S, device="cuda"), i32([0] * (S + 1))
    for stream in (None, torch.cuda.current_stream()):
        for nb in (0, -1, -7):
            with pytest.raises(pa.PagedAttentionError, match="PA_ERR_INVALID_ARG"):
                pa.pa_extend_tables(t, lens, zero, free, one, lens, one, slots, zero, qs, num_blocks=nb, stream=stream)
            with pytest.raises(pa.PagedAttentionError, match="PA_ERR_INVALID_ARG"):
                pa.pa_release_tables(t, lens, zero, free, one, lens, one, num_blocks=nb, stream=stream)
        with pytest.raises(pa.PagedAttentionError, match="PA_ERR_INVALID_ARG"):
            pa.pa_release_tables(t, lens, zero, free, one, lens, one, keep_blocks=-1, stream=stream)
        for big in (2**31, 2**32 + 5, -2**40):
            with pytest.raises(OverflowError, match="num_blocks"):
                pa.pa_extend_tables(t, lens, zero, free, one, lens, one, slots, zero, qs, num_blocks=big, stream=stream)
            with pytest.raises(OverflowError, match="keep_blocks"):
                pa.pa_release_tables(t, lens, zero, free, one, lens, one, keep_blocks=big, stream=stream)
            with pytest.raises(OverflowError, match="max_suffix_len"):
                pa.pa_decode_shared_prefix(out, q, k, k, t, lens, 32, i32([0, S]), one, 1, 0.1, max_suffix_len=big,
                                           stream=stream)
        # numbers of numpy are numbers
        pa.pa_decode_shared_prefix(out, q, k, k, t, lens, np.int64(32), i32([0, S]), one, np.int32(1), np.float32(0.1),
                                   max_suffix_len=np.int64(16), k_scale=np.float32(1), stream=stream)
        pa.pa_release_tables(t, lens, zero, free, one, lens, one, keep_blocks=np.int64(1), num_blocks=np.int32(NB),
                             stream=stream)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0 and lens.tolist() == [20] * S and one.tolist() == [1]


def test_tensors_of_more_than_2_to_31_columns_are_refused():
    """A table of 2^32 + 8 columns is not one of 8."""
    S, HQ, HKV, D, NB, rnd, cache, i32 = small()
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 17 GB of device memory")
    k, q = cache(), rnd(1, HQ, D)
    out = torch.empty((1, HQ, D), device="cuda")
    wide = torch.empty((1, 2**32 + 8), dtype=torch.int32, device="cuda")
    lens, zero, one = i32([20]), i32([0]), i32([1])
    free, slots, qs = i32([5, 6, 7]), torch.arange(1, device="cuda"), i32([0, 0])
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(OverflowError, match="block_tables"):
            pa.pa_extend_tables(wide, lens, zero, free, one, lens, one, slots, zero, qs, num_blocks=NB, stream=stream)
        with pytest.raises(OverflowError, match="block_tables"):
            pa.pa_release_tables(wide, lens, zero, free, one, lens, one, num_blocks=NB, stream=stream)
        with pytest.raises(OverflowError, match="block_tables"):
            pa.pa_decode_shared_prefix(out, q, k, k, wide, lens, 32, i32([0, 1]), one, 1, 0.1, max_suffix_len=32,
                                       stream=stream)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0


def test_an_expanded_workspace_is_refused():
    S, HQ, HKV, D, NB, rnd, cache, i32 = small()
    k, q = cache(), rnd(S, HQ, D)
    out = torch.full((S, HQ, D), 7.0, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for bad in (ws[:1].expand(1 << 20), torch.empty((1 << 20, 2), dtype=torch.uint8, device="cuda")[:, 0], ws.cpu()):
        with pytest.raises(ValueError, match="workspace"):
            pa.pa_decode_shared_prefix(out, q, k, k, i32([[0, 1]] * S), i32([20] * S), 32, i32([0, S]), i32([1]), 1, 0.1,
                                       max_suffix_len=16, workspace=bad)
    assert torch.all(out == 7.0)


def test_a_new_batch_is_captured_at_its_first_step_shared():
    warm = DecodeBatch.build(synth.WORKLOADS["tiny"], 3, "cuda:0")
    want = warm.step_shared().clone()      # loads the kernels, and says what comes out
    b = DecodeBatch.build(synth.WORKLOADS["tiny"], 3, "cuda:0")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step_shared()
    for _ in range(2):
        b.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.out, want)
    assert pa.pa_get_device_error() == 0
    del graph
