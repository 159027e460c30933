"""GPU tests of pa_rope_and_cache against the formula in 64 bits.

Tolerances, derived from the arithmetic: the kernel forms a cos - b sin in
fp32 from cosines and sines off by at most 2 ulp (2^-23), of an angle that
is off by at most 2^-23.3 radians (a 24-bit fraction of half a turn) plus
2^-53 * |position| * 2 pi / 2 (the 64-bit frequency; 2^-21.4 at 2^31), with
two products, a sum and the scale rounded: together below
2^-20 (|a| + |b|) rope_scale. Then one rounding: half a step, 2^-8 of the
value (bf16) or 2^-4 (E4M3; 2^-10 below its normal range) on the quotient
by the scale, whose own division adds 2^-24.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

from paged_kv_cache_429_b200 import (pa_get_device_error, pa_reshape_and_cache, pa_rope_and_cache,
                                     pa_rope_frequencies, PA_ROPE_YARN)

pytestmark = pytest.mark.gpu

B = 16
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510")


@pytest.fixture(autouse=True)
def _clean():
    pa_get_device_error()
    yield
    pa_get_device_error()


def angles(positions, inv):
    """positions x inv reduced to one turn, the product taken exactly."""
    out = np.empty((len(positions), len(inv)))
    for j, f in enumerate(inv):
        fr = Fraction(float(f))
        for i, p in enumerate(positions):
            out[i, j] = float(fr * int(p) % TWO_PI)
    return out


def rotated(x, ang, rot, interleaved, scale):
    """(value, |a| + |b| of its pair) in 64 bits; x [T][H][D]."""
    x = x.astype(np.float64)
    y, mag = x.copy(), np.zeros_like(x)
    c, s = np.cos(ang)[:, None] * scale, np.sin(ang)[:, None] * scale
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (np.abs(a) + np.abs(b)) * abs(scale)
    return y, mag


def case(T, hq, hkv, d, seed, fp8, fused, nb=None, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qkv = (torch.randn((T, hq + 2 * hkv, d), generator=g, device="cuda") * spread).to(torch.bfloat16)
    q, k, v = qkv.split([hq, hkv, hkv], dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = nb or -(-T // B) + 3
    slots = torch.randperm(nb * B, generator=g, device="cuda")[:T].clone()
    dt = torch.uint8 if fp8 else torch.int16
    kc = torch.full((nb, hkv, B, d), 0x55, dtype=dt, device="cuda")
    kc = kc if fp8 else kc.view(torch.bfloat16)
    return q, k, v, kc, kc.clone(), slots


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def check(q, k, v, kc, vc, slots, positions, inv, rot, interleaved, scale, fp8, ks, vs, q_out, kc0):
    T, hq, d = q.shape
    hkv = k.shape[1]
    ang = angles(positions.cpu().numpy(), inv.cpu().numpy())
    want, mag = rotated(q.float().cpu().numpy(), ang, rot, interleaved, scale)
    got = q_out.float().cpu().double().numpy()
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + mag * 2.0 ** -20)
    # the caches: values, and unrotated keys, byte for byte as pa_reshape_and_cache writes them
    rk, rv = kc0.clone(), kc0.clone()
    pa_reshape_and_cache(k.contiguous(), v.contiguous(), rk, rv, slots, k_scale=ks, v_scale=vs)
    np.testing.assert_array_equal(raw(vc), raw(rv))
    np.testing.assert_array_equal(raw(kc[..., rot:]), raw(rk[..., rot:]))
    sl = slots.cpu().numpy()
    live = sl >= 0
    flat = lambda c: c.transpose(1, 2).reshape(-1, hkv, d)
    untouched = np.setdiff1d(np.arange(flat(kc).shape[0]), sl[live])
    np.testing.assert_array_equal(raw(flat(kc)[untouched]), raw(flat(kc0)[untouched]))
    want, mag = rotated(k.float().cpu().numpy(), ang, rot, interleaved, scale)
    rows = flat(kc)[torch.from_numpy(sl[live]).cuda()]
    if fp8:
        got = rows.view(torch.float8_e4m3fn).float().cpu().double().numpy()
        y, m = want[live] / ks, mag[live] / ks
        edge = np.abs(y) * 2.0 ** -4 + 2.0 ** -10 + np.abs(y) * 2.0 ** -23 + m * 2.0 ** -20
        y = np.clip(y, -448, 448)
    else:
        got, y = rows.float().cpu().double().numpy(), want[live]
        edge = np.abs(y) * 2.0 ** -8 + mag[live] * 2.0 ** -20
    assert np.all(np.abs(got - y) <= edge)
    assert pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,rot,fused", [
    (1, 1, 1, 64, 64, False),
    (1, 32, 8, 128, 128, True),
    (3, 7, 1, 128, 16, True),
    (4, 8, 8, 64, 32, False),
    (5, 4, 2, 128, 48, True),
    (33, 5, 5, 64, 64, True),
    (130, 14, 2, 128, 112, True),
    (257, 3, 3, 128, 128, False),
])
def test_matches_the_formula(T, hq, hkv, d, rot, fused, interleaved, fp8):
    q, k, v, kc, vc, slots = case(T, hq, hkv, d, T, fp8, fused)
    pos = torch.randint(0, 131072, (T,), device="cuda", dtype=torch.int32,
                        generator=torch.Generator(device="cuda").manual_seed(T + 1))
    inv, scale = pa_rope_frequencies(rot, device="cuda")
    ks, vs = (0.0125, 0.011) if fp8 else (1.0, 1.0)
    kc0 = kc.clone()
    out = torch.full((T, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    pa_rope_and_cache(out, q, k, v, kc, vc, slots, pos, inv, interleaved=interleaved, rope_scale=scale, k_scale=ks,
                      v_scale=vs)
    torch.cuda.synchronize()
    check(q, k, v, kc, vc, slots, pos, inv, rot, interleaved, scale, fp8, ks, vs, out, kc0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_any_position_and_a_stretched_table(interleaved):
    pos = torch.tensor([0, 1, -1, 2, 4095, 131071, -131071, 1 << 20, (1 << 24) + 1, -(1 << 31), (1 << 31) - 1],
                       dtype=torch.int32, device="cuda")
    T = len(pos)
    q, k, v, kc, vc, slots = case(T, 4, 2, 128, 9, False, True)
    inv, scale = pa_rope_frequencies(128, 10000.0, PA_ROPE_YARN, factor=16.0, original_max_position=4096,
                                     device="cuda")
    assert scale > 1.2
    kc0 = kc.clone()
    out = torch.empty((T, 4, 128), dtype=torch.bfloat16, device="cuda")
    pa_rope_and_cache(out, q, k, v, kc, vc, slots, pos, inv, interleaved=interleaved, rope_scale=scale)
    torch.cuda.synchronize()
    check(q, k, v, kc, vc, slots, pos, inv, 128, interleaved, scale, False, 1.0, 1.0, out, kc0)


def test_negative_and_large_frequencies():
    """Any finite table: turns beyond a whole one, negative ones, zero."""
    inv = torch.tensor([0.0, -0.5, 7.5, 100.0, -6.2, 3.14159, 1e-9, 1.0], dtype=torch.float64, device="cuda")
    T = 40
    q, k, v, kc, vc, slots = case(T, 2, 2, 64, 3, False, True)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 11
    kc0 = kc.clone()
    out = torch.empty((T, 2, 64), dtype=torch.bfloat16, device="cuda")
    pa_rope_and_cache(out, q, k, v, kc, vc, slots, pos, inv)
    torch.cuda.synchronize()
    check(q, k, v, kc, vc, slots, pos, inv, 16, False, 1.0, False, 1.0, 1.0, out, kc0)


@pytest.mark.parametrize("fp8", [False, True])
def test_padding_and_slots_outside_the_pool(fp8):
    T = 50
    q, k, v, kc, vc, slots = case(T, 4, 2, 128, 21, fp8, True)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 7
    inv, _ = pa_rope_frequencies(64, device="cuda")
    ks, vs = (0.02, 0.02) if fp8 else (1.0, 1.0)
    kc0 = kc.clone()
    slots[45:] = -1
    slots[3] = -7
    out = torch.empty((T, 4, 128), dtype=torch.bfloat16, device="cuda")
    pa_rope_and_cache(out, q, k, v, kc, vc, slots, pos, inv, k_scale=ks, v_scale=vs)
    check(q, k, v, kc, vc, slots, pos, inv, 64, False, 1.0, fp8, ks, vs, out, kc0)
    # past the pool: skipped and flagged, everything else as before
    kc1, vc1 = kc0.clone(), kc0.clone()
    slots[10] = kc.shape[0] * B
    slots[11] = 1 << 40
    pa_rope_and_cache(out, q, k, v, kc1, vc1, slots, pos, inv, k_scale=ks, v_scale=vs)
    assert pa_get_device_error() == 0x1
    slots[10:12] = -1
    kc2, vc2 = kc0.clone(), kc0.clone()
    pa_rope_and_cache(out, q, k, v, kc2, vc2, slots, pos, inv, k_scale=ks, v_scale=vs)
    assert np.array_equal(raw(kc1), raw(kc2)) and np.array_equal(raw(vc1), raw(vc2))


def test_saturation_nan_and_infinity_follow_the_cache_write():
    """Position 0 rotates by nothing: keys are stored as pa_reshape_and_cache
    stores them, at the ends of E4M3 too."""
    T = 16
    q, k, v, kc, vc, slots = case(T, 2, 2, 64, 31, True, False, spread=300.0)
    k[0, 0, 5] = float("nan")
    v[1, 1, 6] = float("inf")
    k[2, 0, 7] = 3e38
    inv, _ = pa_rope_frequencies(64, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    rk, rv = kc.clone(), kc.clone()
    out = torch.empty_like(q)
    pa_rope_and_cache(out, q, k, v, kc, vc, slots, pos, inv, k_scale=0.5, v_scale=0.5)
    pa_reshape_and_cache(k, v, rk, rv, slots, k_scale=0.5, v_scale=0.5)
    np.testing.assert_array_equal(raw(vc), raw(rv))
    # b * sin 0 = NaN * 0 reaches the partner of a NaN only
    same = raw(kc) == raw(rk)
    partner = slots[0].item()
    bad = np.argwhere(~same)
    assert len(bad) <= 1 and all(tuple(x) == (partner // B, 0, partner % B, 5 + 32) for x in bad)
    assert torch.equal(out, q)


def test_in_place_other_stream_and_repeat():
    T = 300
    q, k, v, kc, vc, slots = case(T, 8, 4, 128, 41, False, False)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    inv, _ = pa_rope_frequencies(128, device="cuda")
    out = torch.empty_like(q)
    pa_rope_and_cache(out, q, k, v, kc, vc, slots, pos, inv)
    k1, v1 = kc.clone(), vc.clone()
    kc.fill_(0.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa_rope_and_cache(q, q, k, v, kc, vc, slots, pos, inv, stream=side)   # q_out is q
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(q, out)
    live = torch.zeros(kc.shape[0] * B, dtype=torch.bool, device="cuda")
    live[slots] = True
    rows = lambda c: c.transpose(1, 2).reshape(-1, 4, 128)[live]
    assert torch.equal(rows(kc), rows(k1)) and torch.equal(vc, v1)
    assert pa_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("extra,hq,hkv,d,rot,fused", [
    (0, 2, 1, 64, 64, False),       # the fewest prompt tokens, whole CTAs
    (1, 7, 1, 128, 128, True),      # one token in the last CTA
    (2, 5, 5, 64, 48, True),
    (3, 4, 2, 128, 16, True),
    (517, 32, 8, 128, 128, True),   # several batches of units a CTA
])
def test_prompts_match_the_formula(extra, hq, hkv, d, rot, fused, interleaved, fp8):
    """From ten tokens an SM on a CTA takes four tokens whole; padding and
    skipped tokens stand anywhere among them."""
    T = 10 * torch.cuda.get_device_properties(0).multi_processor_count + extra
    q, k, v, kc, vc, slots = case(T, hq, hkv, d, T, fp8, fused)
    slots[T - T // 50:] = -1
    slots[torch.arange(0, 90, 7, device="cuda")] = -3
    pos = torch.randint(0, 131072, (T,), device="cuda", dtype=torch.int32,
                        generator=torch.Generator(device="cuda").manual_seed(T + 1))
    inv, scale = pa_rope_frequencies(rot, 10000.0, PA_ROPE_YARN, factor=16.0, original_max_position=4096,
                                     device="cuda")
    ks, vs = (0.0125, 0.011) if fp8 else (1.0, 1.0)
    kc0 = kc.clone()
    vc0 = vc.clone()
    out = torch.full((T, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    kw = dict(interleaved=interleaved, rope_scale=scale, k_scale=ks, v_scale=vs)
    pa_rope_and_cache(out, q, k, v, kc, vc, slots, pos, inv, **kw)
    torch.cuda.synchronize()
    check(q, k, v, kc, vc, slots, pos, inv, rot, interleaved, scale, fp8, ks, vs, out, kc0)
    # in place, and tokens past the pool (one in each place of a CTA) skipped and flagged
    past = torch.tensor([8, 13, 18, 23], device="cuda")
    slots[past] = kc.shape[0] * B + past
    k2, v2, q2 = kc0.clone(), vc0.clone(), q.contiguous().clone()
    pa_rope_and_cache(q2, q2, k, v, k2, v2, slots, pos, inv, **kw)
    assert pa_get_device_error() == 0x1 and torch.equal(q2, out)
    slots[past] = -1
    k3, v3 = kc0.clone(), vc0.clone()
    pa_rope_and_cache(q2, q, k, v, k3, v3, slots, pos, inv, **kw)
    assert np.array_equal(raw(k2), raw(k3)) and np.array_equal(raw(v2), raw(v3))
    assert pa_get_device_error() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_large_frequencies_at_far_positions(interleaved):
    """The product is reduced with the frequency's full 53 bits and both of
    1 / 2 pi's doubles: 2^-104 of an angle of up to 2^62 radians, far below the
    tolerance's 2^-20."""
    inv = torch.tensor([1.0, -7.5, 100.0, 12345.678, -1e6, 2.0 ** 31 + 0.37, 3e-7, 3.14159265], dtype=torch.float64,
                       device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    far = torch.randint(-2 ** 31, 2 ** 31, (190,), device="cuda", generator=g).to(torch.int32)
    ends = torch.tensor([-2 ** 31, 2 ** 31 - 1, -2 ** 31 + 1, 2 ** 30, -2 ** 30, 131071, 1, 0, -1, 2 ** 24 + 1],
                        dtype=torch.int32, device="cuda")
    pos = torch.cat([far, ends])
    T = len(pos)
    q, k, v, kc, vc, slots = case(T, 4, 2, 64, 51, False, True)
    kc0 = kc.clone()
    out = torch.empty((T, 4, 64), dtype=torch.bfloat16, device="cuda")
    pa_rope_and_cache(out, q, k, v, kc, vc, slots, pos, inv, interleaved=interleaved)
    torch.cuda.synchronize()
    check(q, k, v, kc, vc, slots, pos, inv, 16, interleaved, 1.0, False, 1.0, 1.0, out, kc0)


@pytest.mark.parametrize("tokens", [5, 1500])
def test_offsets_past_32_bits(tokens):
    """Slots past 2^31 elements of a cache, and tokens so far apart that the
    last one starts past 2^31 elements of their tensor."""
    hkv, d = 8, 128
    nb = (1 << 31) // (hkv * B * d) + 200
    kc = torch.zeros((nb, hkv, B, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    heads, stride = 16 + 2 * hkv, (1 << 31) // (tokens - 1) // 8 * 8 + 8
    g = torch.Generator(device="cuda").manual_seed(61)
    rows = torch.randn((tokens, heads, d), generator=g, device="cuda").to(torch.bfloat16)
    far = torch.empty(stride * (tokens - 1) + heads * d, dtype=torch.bfloat16, device="cuda")
    far = far.as_strided((tokens, heads, d), (stride, d, 1))
    far.copy_(rows)
    first = nb * B - 2 * tokens       # in the last blocks
    slots = first + 2 * torch.randperm(tokens, generator=g, device="cuda")
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    inv, _ = pa_rope_frequencies(d, device="cuda")
    out = torch.empty((tokens, 16, d), dtype=torch.bfloat16, device="cuda")
    pa_rope_and_cache(out, far[:, :16], far[:, 16:16 + hkv], far[:, 16 + hkv:], kc, vc, slots, pos, inv)
    torch.cuda.synchronize()
    # the same tokens close together, into the cache's last blocks alone
    low = first // B
    k2, v2 = torch.zeros_like(kc[low:]), torch.zeros_like(vc[low:])
    out2 = torch.empty_like(out)
    pa_rope_and_cache(out2, rows[:, :16], rows[:, 16:16 + hkv], rows[:, 16 + hkv:], k2, v2, slots - low * B, pos, inv)
    assert torch.equal(out, out2) and torch.equal(kc[low:], k2) and torch.equal(vc[low:], v2)
    assert int(torch.count_nonzero(k2)) > 0 and int(torch.count_nonzero(kc[:low])) == 0
    assert pa_get_device_error() == 0
