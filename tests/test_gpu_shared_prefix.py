"""GPU tests of pa_decode_shared_prefix against the fp64 oracle of the plain
decode on the same caches and tables.

Tolerance, derived from the arithmetic. A score is a sum of head_dim exact
products kept in fp32: with at most 10 roundings of a running sum, 2^-23
each (the tensor core may truncate), it is off by 10 * 2^-23 * Z, where Z is
the largest sm_scale * sum |q k| over the data. A weight exp(z) is off
relatively by that, by 2^-21 of the exponential and its argument, and by
2^-17 of its own split into two 16-bit halves; sums over n tokens add one
rounding per 128 tokens and about 16 more. Numerator and denominator each
carry the error, so against outputs that are averages of values at most
max|v|:
    |err| <= 2 max|v| (10 * 2^-23 Z + 2^-21 (1 + Z / 8) + 2^-17 + (n / 128 + 16) 2^-23).
(2^-21 Z / 8: the argument z * log2 e, |z| <= Z, is rounded twice in fp32.)
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from paged_kv_cache_429_b200 import (pa_decode, pa_decode_shared_prefix,
                                     pa_decode_shared_prefix_workspace_size, pa_get_device_error)
from parity_harness import to_u16, to_u8

pytestmark = pytest.mark.gpu

B = 16
CLAMP, BLOCK, GROUP = 0x4, 0x10, 0x100


@pytest.fixture(autouse=True)
def _clean():
    pa_get_device_error()
    yield
    pa_get_device_error()
    torch.cuda.empty_cache()


class Batch:
    """Groups of `sizes` sequences behind `prefixes` blocks, suffix lengths
    `suf` (of every sequence, in order); stale slots and unused blocks NaN."""

    def __init__(self, hq, hkv, d, sizes, prefixes, suf, fp8=False, seed=0, spread=1.0, tail=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed * 977 + 5)
        S = sum(sizes) + tail
        suf = np.asarray(suf, np.int64)
        assert len(suf) == S
        of = np.repeat(np.arange(len(sizes) + 1), list(sizes) + [tail])
        pre = np.array(list(prefixes) + [0])[of]
        lens = np.maximum(pre * B + suf, 0)
        own = -(-np.maximum(suf, 0) // B)
        shared = [p if n else 0 for p, n in zip(prefixes, sizes)]
        nb = int(sum(shared) + own.sum()) + 9
        ids = np.random.default_rng(seed).permutation(nb)
        W = max(1, int((pre + own).max()))
        tables = np.full((S, W), -1, np.int32)
        firsts = np.cumsum([0] + shared)
        k = int(sum(shared))
        for s in range(S):
            if of[s] < len(sizes):
                tables[s, :pre[s]] = ids[firsts[of[s]]:firsts[of[s]] + pre[s]]
            tables[s, pre[s]:pre[s] + own[s]] = ids[k:k + own[s]]
            k += own[s]
        self.S, self.hq, self.hkv, self.d, self.fp8 = S, hq, hkv, d, fp8
        self.lens, self.tables, self.pre, self.nb = lens, tables, pre, nb
        self.start, self.blocks = np.cumsum([0] + list(sizes)), np.array(prefixes, np.int64)
        self.max_suffix = max(1, int(suf.max()))
        self.ks, self.vs = (0.0125, 0.01) if fp8 else (1.0, 1.0)
        self.q = (torch.randn((S, hq, d), generator=g, device="cuda") * spread).to(torch.bfloat16)
        shape = (nb, hkv, B, d)
        self.vmax = 0.0
        self.scale = d ** -0.5

        def cache(scale):
            x = torch.randn(shape, generator=g, device="cuda")
            self.vmax = float(x.abs().max())
            return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else x.to(torch.bfloat16)
        self.k, self.v = cache(self.ks), cache(self.vs)
        # what no sequence's token owns holds NaN
        owned = np.zeros((nb, B), bool)
        for s in range(S):
            for j in range(-(-int(lens[s]) // B)):
                owned[tables[s, j], :max(0, min(B, int(lens[s]) - B * j))] = True
            for j in range(int(pre[s])):
                owned[tables[s, j]] = True    # a prefix belongs to the cache whoever is short of it
        bad = torch.from_numpy(~owned).cuda()[:, None, :, None]
        for t in (self.k, self.v):
            u = t.view(torch.uint8) if fp8 else t.view(torch.int16)
            u.copy_(torch.where(bad, torch.full_like(u, synth.SENTINEL_FP8 if fp8 else synth.SENTINEL_BF16), u))

    def dev(self, a):
        return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()

    def run(self, out=None, q=None, **kw):
        out = torch.full((self.S, self.hq, self.d), float("nan"), device="cuda") if out is None else out
        a = dict(max_len=max(int(self.lens.max()), 0), max_prefix=int(max(list(self.blocks) + [0])),
                 max_suffix_len=self.max_suffix, start=self.start, blocks=self.blocks, tables=self.tables,
                 lens=self.lens, workspace=None, stream=None)
        a.update(kw)
        return pa_decode_shared_prefix(
            out, self.q if q is None else q, self.k, self.v, self.dev(a["tables"]), self.dev(a["lens"]), a["max_len"],
            self.dev(a["start"]), self.dev(a["blocks"]), a["max_prefix"], self.scale,
            max_suffix_len=a["max_suffix_len"], k_scale=self.ks, v_scale=self.vs, workspace=a["workspace"],
            stream=a["stream"])

    def oracle(self, lens=None, tables=None, subset=None, k=None, v=None):
        to = to_u8 if self.fp8 else to_u16
        return oracle.paged_decode(to_u16(self.q), to(self.k if k is None else k), to(self.v if v is None else v),
                                   self.tables if tables is None else tables,
                                   (self.lens if lens is None else lens).astype(np.int32), self.scale,
                                   kv_dtype=oracle.KV_FP8_E4M3 if self.fp8 else oracle.KV_BF16, k_scale=self.ks,
                                   v_scale=self.vs, seq_subset=subset)

    def tol(self):
        # Z: sm_scale sum |q k| <= sm_scale |q| |k| (Cauchy-Schwarz on the largest rows)
        kk = self.k.float().nan_to_num(0.0) * self.ks
        Z = abs(self.scale) * float(self.q.float().norm(dim=-1).max()) * float(kk.norm(dim=-1).max())
        n = max(int(self.lens.max()), 1)
        return 2 * self.vmax * (10 * 2.0 ** -23 * Z + 2.0 ** -21 * (1 + Z / 8) + 2.0 ** -17
                                + (n / 128 + 16) * 2.0 ** -23)

    def check(self, out, subset=None, **kw):
        ref = self.oracle(subset=subset, **kw)
        got = out.double().cpu().numpy()
        if subset is not None:
            got, ref = got[subset], ref[subset]
        assert np.all(np.isfinite(got))
        err = np.abs(got - ref)
        assert err.max() <= self.tol(), (err.max(), self.tol())
        # and as a whole: the errors of many weights do not line up
        norm = np.linalg.norm(ref)
        assert np.linalg.norm(err) <= 2e-5 * norm + 1e-30


def suffixes(seed, n, lo, hi):
    return np.random.default_rng(seed + 100).integers(lo, hi + 1, n)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,sizes,prefixes,lo,hi", [
    (1, 1, 64, [1], [1], 1, 1),
    (8, 8, 64, [4], [16], 1, 64),          # one head per KV head
    (8, 8, 128, [3], [7], 1, 40),          # a prefix that ends inside a key tile
    (8, 2, 128, [5], [8], 0, 33),          # exactly one key tile; sequences without a suffix
    (32, 8, 128, [9], [9], 1, 100),
    (16, 1, 128, [20], [33], 1, 20),       # the widest group: several row tiles
    (7, 1, 64, [37], [5], 0, 17),          # seven heads: rows do not fill a tile
    (5, 1, 128, [130], [12], 1, 5),
    (12, 4, 64, [3, 1, 8], [4, 9, 1], 0, 50),   # three groups
    (8, 8, 128, [300], [20], 1, 8),        # more than two row tiles of one head each
    (4, 4, 64, [2], [600], 1, 30),         # a long prefix, split over several CTAs
    (64, 8, 128, [6], [300], 1, 700),      # long suffixes of few sequences
])
def test_matches_the_oracle(hq, hkv, d, sizes, prefixes, lo, hi, fp8):
    b = Batch(hq, hkv, d, sizes, prefixes, suffixes(len(sizes), sum(sizes), lo, hi), fp8=fp8, seed=hq + d)
    out = b.run()
    torch.cuda.synchronize()
    b.check(out)
    assert pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("spread", [6.0, 24.0])
def test_peaked_scores(spread, fp8):
    b = Batch(8, 2, 128, [11], [40], suffixes(3, 11, 0, 300), fp8=fp8, seed=2, spread=spread)
    b.check(b.run())
    assert pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [-0.11, 0.0, 1e-3])
def test_any_finite_scale(scale, fp8):
    """A negative scale turns the order of the scores around, zero makes all
    weights equal; a prefix that ends inside a key tile is masked either way."""
    b = Batch(8, 2, 128, [7], [13], suffixes(9, 7, 0, 90), fp8=fp8, seed=21)
    b.scale = scale
    b.check(b.run())
    assert pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_without_tokens_short_rows_and_rows_of_no_group(fp8):
    """L = 0 inside and outside groups (zeros), L inside the prefix, an empty
    group, a group with an empty prefix, and three sequences behind the last
    group."""
    sizes, prefixes = [6, 0, 4, 2], [10, 5, 0, 3]
    suf = [5, 1, 0, 20, 17, 3, 9, 40, 1, 16, 2, 2, 33, 7, 100]
    b = Batch(8, 2, 128, sizes, prefixes, suf, fp8=fp8, seed=9, tail=3)
    lens = b.lens.copy()
    lens[1], lens[2], lens[3], lens[6], lens[13] = 0, 1, 77, 0, 0   # rows 1-3 end inside the prefix
    b.lens = lens
    out = b.run()
    torch.cuda.synchronize()
    assert torch.count_nonzero(out[[1, 6, 13]]) == 0
    b.check(out)
    assert pa_get_device_error() == 0


def test_without_groups_it_is_the_plain_decode():
    b = Batch(32, 8, 128, [], [], suffixes(1, 7, 1, 900), tail=7, seed=4)
    out = b.run(max_prefix=0)
    b.check(out)
    b2 = Batch(32, 8, 128, [7], [0], suffixes(1, 7, 1, 900), seed=4)
    b2.check(b2.run())
    assert pa_get_device_error() == 0


def test_agrees_with_pa_decode():
    b = Batch(32, 8, 128, [20, 12], [70, 30], suffixes(8, 32, 1, 400), seed=6)
    out = b.run()
    ref = torch.empty_like(out)
    pa_decode(ref, b.q, b.k, b.v, b.dev(b.tables), b.dev(b.lens), int(b.lens.max()), b.d ** -0.5)
    assert float((out - ref).abs().max()) <= 2 * b.tol()


def test_loose_bounds_change_nothing():
    """Bounds well above the lengths (another split of the work) and a
    workspace of NaN from another call."""
    b = Batch(16, 4, 128, [10, 3], [21, 6], suffixes(5, 13, 0, 90), seed=12)
    ref = b.run()
    n = pa_decode_shared_prefix_workspace_size(b.S, b.hq, b.hkv, b.d, 2, 500, 9000)
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    tables = np.full((b.S, 900), -1, np.int32)
    tables[:, :b.tables.shape[1]] = b.tables
    out = b.run(max_len=14000, max_prefix=500, max_suffix_len=9000, workspace=ws, tables=tables)
    b.check(ref)
    b.check(out)
    assert pa_get_device_error() == 0


def test_lengths_beyond_their_bounds_are_cut_and_flagged():
    b = Batch(8, 2, 64, [5], [4], [10, 50, 3, 20, 30], seed=13)
    cut = np.minimum(b.lens, 4 * B + 20)
    out = b.run(max_suffix_len=20)
    assert pa_get_device_error() == CLAMP
    b.check(out, lens=cut)
    out = b.run(max_len=70)
    assert pa_get_device_error() == CLAMP
    b.check(out, lens=np.minimum(b.lens, 70))
    lens = b.lens.copy()
    lens[2] = -4
    out = b.run(lens=lens)
    assert pa_get_device_error() == CLAMP
    b.check(out, lens=np.maximum(lens, 0))


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_block_ids_read_zeros(fp8):
    b = Batch(8, 2, 128, [6], [11], suffixes(2, 6, 20, 60), fp8=fp8, seed=14)
    tables = b.tables.copy()
    tables[0, 3], tables[0, 10] = -1, b.nb         # the prefix is read from the first row
    tables[2, 11], tables[4, 12] = b.nb + 1000, -7
    out = b.run(tables=tables)
    assert pa_get_device_error() == BLOCK
    # the oracle sees an added block of zeros in their place
    zero = tables.copy()
    zero[zero >= b.nb] = b.nb
    for s in range(6):
        zero[s, 3] = zero[s, 10] = b.nb
        n = -(-int(b.lens[s]) // B)
        zero[s, :n][zero[s, :n] < 0] = b.nb
    pad = lambda t: torch.cat([t.view(torch.uint8), torch.zeros_like(t[:1]).view(torch.uint8)]).view(t.dtype)
    b.check(out, tables=zero, k=pad(b.k), v=pad(b.v))


@pytest.mark.parametrize("start,blocks", [
    ([0, 4, 2, 9], [3, 3, 3]),             # not ascending
    ([-5, 3, 6, 100], [3, 3, 3]),          # outside the batch
    ([0, 3, 6, 9], [3, -2, 1000]),         # prefixes outside their bound
])
def test_bad_groups_never_fault(start, blocks):
    b = Batch(8, 4, 64, [3, 3, 3], [3, 3, 3], [20] * 9, seed=15)
    out = b.run(start=np.array(start), blocks=np.array(blocks))
    torch.cuda.synchronize()
    assert pa_get_device_error() & GROUP
    assert out.shape == (9, 8, 64)


def test_repeated_calls_are_bit_identical():
    b = Batch(32, 8, 128, [40], [90], suffixes(4, 40, 0, 300), seed=16)
    first = b.run().clone()
    for _ in range(3):
        assert torch.equal(b.run(), first)


def test_captured_beside_eager_and_on_two_streams():
    """Two captured graphs with a workspace each, an eager call between their
    replays, and two calls at once on two streams."""
    b = Batch(32, 8, 128, [16], [64], suffixes(4, 16, 1, 200), seed=17)
    c = Batch(32, 8, 128, [9], [20], suffixes(5, 9, 1, 100), seed=18)
    want = [x.run().clone() for x in (b, c)]
    args = [(x.dev(x.tables), x.dev(x.lens), x.dev(x.start), x.dev(x.blocks)) for x in (b, c)]
    outs = [torch.zeros_like(w) for w in want]

    def call(i, x, stream=None):
        t, l, s, p = args[i]
        pa_decode_shared_prefix(outs[i], x.q, x.k, x.v, t, l, int(x.lens.max()), s, p, int(x.blocks.max()),
                                x.d ** -0.5, max_suffix_len=x.max_suffix, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i, x in enumerate((b, c)):
            call(i, x)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for i, x in enumerate((b, c)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, x)
        graphs.append(g)
    for o in outs:
        o.zero_()
    for _ in range(2):
        for g in graphs:
            g.replay()
        eager = b.run()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, want[0])
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for i, (x, st) in enumerate(((b, side), (c, other))):
        with torch.cuda.stream(st):   # the call's own workspace belongs to its stream
            call(i, x)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    del graphs
    assert pa_get_device_error() == 0


def test_rows_behind_the_batch_stay():
    b = Batch(8, 2, 128, [5], [9], suffixes(6, 5, 1, 60), seed=19)
    big = torch.full((b.S + 3, b.hq, b.d), 7.0, device="cuda")
    b.run(out=big[:b.S])
    torch.cuda.synchronize()
    assert torch.all(big[b.S:] == 7.0)
    b.check(big[:b.S])


def test_a_cache_of_more_than_2_to_31_elements():
    """Blocks whose rows start past 2^31 elements of the cache."""
    hkv, d = 8, 128
    nb = (1 << 31) // (hkv * B * d) + 300
    b = Batch(16, hkv, d, [6], [12], suffixes(7, 6, 1, 80), seed=20)
    small_k, small_v, n = b.k, b.v, b.nb
    b.k = torch.zeros((nb, hkv, B, d), dtype=torch.bfloat16, device="cuda")
    b.v = torch.zeros((nb, hkv, B, d), dtype=torch.bfloat16, device="cuda")
    b.k[nb - n:] = small_k
    b.v[nb - n:] = small_v
    tables = np.where(b.tables >= 0, b.tables + nb - n, -1).astype(np.int32)
    out = b.run(tables=tables)
    torch.cuda.synchronize()
    assert pa_get_device_error() == 0
    b.k, b.v = small_k, small_v
    b.check(out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bound", [2**31 - 1, 2**31 - 130, 2**30])
def test_loose_bounds_near_32_bits(bound, fp8):
    """Enough sequences that a suffix is one part, as long as its bound."""
    b = Batch(8, 8, 64, [100, 28], [3, 2], suffixes(11, 128, 0, 400), fp8=fp8, seed=22)
    out = b.run(max_len=bound, max_suffix_len=bound)
    b.check(out)
    assert pa_get_device_error() == 0


def reference(b):
    """All rows by the formula, in 64 bits on the GPU: (S, Hq, D)."""
    out = torch.zeros((b.S, b.hq, b.d), dtype=torch.float64, device="cuda")
    tables = torch.from_numpy(b.tables).cuda().long()
    for s in range(b.S):
        n = int(b.lens[s])
        if n == 0:
            continue
        ids = tables[s, :-(-n // B)]

        def rows(t, scale):
            x = t.view(torch.uint8)[ids].view(torch.float8_e4m3fn) if b.fp8 else t[ids]
            return x.double().transpose(0, 1).reshape(b.hkv, -1, b.d)[:, :n] * scale
        z = torch.bmm(b.q[s].double().view(b.hkv, -1, b.d), rows(b.k, b.ks).transpose(1, 2)) * b.scale
        out[s] = torch.bmm(torch.softmax(z, -1), rows(b.v, b.vs)).reshape(b.hq, b.d)
    return out


def tiles_of_a_part(b):
    """Key tiles of a part of the longest prefix, from the workspace's size:
    a record of head_dim values, a maximum and a sum a row and part."""
    size = lambda g: pa_decode_shared_prefix_workspace_size(b.S, b.hq, b.hkv, b.d, g, int(b.blocks.max()), b.max_suffix)
    parts = round((size(len(b.blocks)) - size(0)) / (b.S * b.hq * (4 * b.d + 8)))
    return -(-(-(-int(b.blocks.max()) // 8)) // parts)


def slope(b, nats, period, seed):
    """Scores that rise by `nats` from key tile to key tile of a part, for
    every other sequence, and fall for the rest: queries +-u plus noise, keys
    of the prefixes a multiple of u plus noise."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *n: torch.randn(n, generator=g, device="cuda")
    u = torch.where(rnd(b.d) > 0, 1.0, -1.0)
    sign = torch.where(torch.arange(b.S, device="cuda") % 2 == 0, 1.0, -1.0)[:, None, None]
    b.q = (sign * u + 0.5 * rnd(b.S, b.hq, b.d)).to(torch.bfloat16)
    step = nats / (b.d * b.scale)              # of one tile, as a multiple of u
    b.ks = 0.025 if b.fp8 else 1.0             # the largest key stays below 448 codes
    for first, n in zip(b.start, b.blocks):
        ids = torch.from_numpy(b.tables[first, :n]).cuda().long()
        tile = torch.arange(int(n), device="cuda") // 8 % period
        x = (tile - (period - 1) / 2)[:, None, None, None] * step * u + 0.5 * rnd(len(ids), b.hkv, B, b.d)
        assert float(x.abs().max()) / b.ks < (448 if b.fp8 else 1e30)
        b.k[ids] = (x / b.ks).to(torch.float8_e4m3fn) if b.fp8 else x.to(torch.bfloat16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nats", [0.0, 0.7, 7.0])
@pytest.mark.parametrize("hq,hkv,d,sizes,prefixes,tiles", [
    (32, 32, 64, [150, 140, 10], [320, 313, 47], 14),   # two query tiles and, in the last group, one
    (32, 32, 128, [40, 3, 1, 128], [320, 200, 9, 320], 14),   # one query tile everywhere
    (64, 8, 128, [150], [320], 14),                     # eight heads; the last CTA's second tile part full
    (28, 4, 64, [300], [317], 10),                      # seven heads; a part that ends inside a key tile
    (32, 32, 128, [260], [256], 16),                    # the longest parts
])
def test_parts_of_many_key_tiles(hq, hkv, d, sizes, prefixes, tiles, nats, fp8):
    """Rings that go round, table entries past the first 32, and scores that
    pass the running reference again and again (by up to 7 nats, 10 in log2,
    a tile: far over the 2^15 of E4M3 and, within a part, the 2^60 of bf16)."""
    b = Batch(hq, hkv, d, sizes, prefixes, suffixes(hq + d, sum(sizes), 0, 30), fp8=fp8, seed=23)
    assert tiles_of_a_part(b) == tiles
    if nats:
        slope(b, nats, tiles, seed=24)
    out = b.run()
    torch.cuda.synchronize()
    assert pa_get_device_error() == 0
    err = (out.double() - reference(b)).abs()
    assert bool(torch.isfinite(out).all())
    assert float(err.max()) <= b.tol(), (float(err.max()), b.tol())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("groups", [31, 32, 33, 64, 65, 100, 1100])
def test_more_groups_than_a_warp(groups, fp8):
    """Parallel samples: groups of 0 to 4 sequences, some without a prefix,
    and sequences of no group behind them."""
    g = np.random.default_rng(groups)
    sizes = g.integers(0, 5 if groups < 1000 else 2, groups)
    sizes[[0, groups - 1]] = [2, 3]
    prefixes = g.integers(0, 13, groups)
    b = Batch(8, 2, 64, list(sizes), list(prefixes), suffixes(groups, int(sizes.sum()) + 5, 0, 40), fp8=fp8, seed=25,
              tail=5)
    out = b.run()
    torch.cuda.synchronize()
    b.check(out)
    assert pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_clamped_groups_give_the_same_values(fp8):
    """Prefixes outside their bound are clamped, a group that passes the
    batch's ends is cut there: every sequence still attends to its context."""
    b = Batch(8, 4, 64, [3, 3, 3], [3, 3, 3], suffixes(26, 9, 1, 60), fp8=fp8, seed=26)
    for start, blocks, suffix in (([0, 3, 6, 9], [3, -2, 1000], 3 * B + b.max_suffix),
                                  ([-5, 3, 6, 100], [3, 3, 3], b.max_suffix)):
        out = b.run(start=np.array(start), blocks=np.array(blocks), max_prefix=3, max_suffix_len=suffix)
        torch.cuda.synchronize()
        assert pa_get_device_error() == GROUP
        b.check(out)


def test_sequences_beside_overlapping_groups_are_right():
    """[3, 7), [7, 5) and [5, 9) overlap, which is flagged; the group in front
    of them and the sequences of no group keep their values."""
    b = Batch(8, 4, 64, [3, 6], [4, 3], suffixes(27, 12, 1, 60), seed=27, tail=3)
    out = b.run(start=np.array([0, 3, 7, 5, 9]), blocks=np.array([4, 3, 3, 3]))
    torch.cuda.synchronize()
    assert pa_get_device_error() & GROUP
    b.check(out, subset=np.array([0, 1, 2, 9, 10, 11]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), 3.0e38])
def test_padded_rows_hold_anything(junk, fp8):
    """Rows without tokens, in the middle of a group and behind the last one,
    whose queries are what an earlier step left: zeros come out, and nothing
    of them reaches the other rows of their tiles. A live row of such queries
    spoils itself alone."""
    b = Batch(16, 4, 128, [21, 9], [70, 25], suffixes(28, 34, 0, 60), fp8=fp8, seed=28, tail=4)
    empty, spoilt = [3, 11, 20, 22, 31, 33], 7
    b.lens[empty] = 0
    b.q[empty] = junk
    b.q[spoilt] = float("nan")
    out = b.run()
    torch.cuda.synchronize()
    assert torch.count_nonzero(out[empty]) == 0 and bool(torch.isnan(out[spoilt]).all())
    live = np.array([s for s in range(b.S) if s != spoilt])
    b.q[empty + [spoilt]] = 1.0       # for the oracle and the tolerance
    b.check(out, subset=live)
    assert pa_get_device_error() == 0
