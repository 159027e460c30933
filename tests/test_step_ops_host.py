"""Host side of the serving-step operators (no GPU): the frequency table of
pa_rope_and_cache against its formulas, and what the entry points refuse
before anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_429_b200 as pa
from paged_kv_cache_429_b200 import _lib

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x100000  # aligned non-null address; never dereferenced by these calls


# ------------------------------------------------------------- frequencies

def plain_frequencies(r, base, scaling, factor, n, low, high):
    """The formulas of pa.h, one component at a time."""
    if scaling == pa.PA_ROPE_BASE:
        base = base * factor ** (r / (r - 2))
    out = []
    for i in range(r // 2):
        f = base ** (-2 * i / r)
        if scaling == pa.PA_ROPE_LINEAR:
            f = f / factor
        elif scaling == pa.PA_ROPE_BANDS:
            turns = n / (2 * math.pi / f)
            if turns <= low:
                f = f / factor
            elif turns < high:
                x = (turns - low) / (high - low)
                f = x * f + (1 - x) * f / factor
        elif scaling == pa.PA_ROPE_YARN:
            at = lambda t: r * math.log(n / (t * 2 * math.pi)) / (2 * math.log(base))
            a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), r - 1)
            x = min(max((i - a) / max(b - a, 1e-3), 0), 1)
            f = (1 - x) * f + x * f / factor
        out.append(f)
    return np.array(out), (0.1 * math.log(factor) + 1 if scaling == pa.PA_ROPE_YARN else 1.0)


@pytest.mark.parametrize("r", [4, 16, 48, 64, 128])
@pytest.mark.parametrize("scaling,kw", [
    (pa.PA_ROPE_NONE, {}),
    (pa.PA_ROPE_LINEAR, dict(factor=4.0)),
    (pa.PA_ROPE_BASE, dict(factor=8.0)),
    (pa.PA_ROPE_BANDS, dict(factor=8.0, original_max_position=8192, low=1.0, high=4.0)),
    (pa.PA_ROPE_YARN, dict(factor=16.0, original_max_position=4096, low=1.0, high=32.0)),
    (pa.PA_ROPE_YARN, dict(factor=1.0, original_max_position=4096)),
])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies_follow_their_formulas(r, scaling, kw, base):
    inv, scale = pa.pa_rope_frequencies(r, base, scaling, **kw)
    want, want_scale = plain_frequencies(r, base, scaling, kw.get("factor", 1.0),
                                         kw.get("original_max_position", 0.0), kw.get("low", 1.0),
                                         kw.get("high", 32.0))
    assert inv.dtype == torch.float64 and inv.shape == (r // 2,)
    # a few roundings of 64-bit pow, log and products
    np.testing.assert_allclose(inv.numpy(), want, rtol=1e-14, atol=0)
    assert scale == pytest.approx(want_scale, rel=2 ** -23)


def test_base_scaling_keeps_the_ends():
    """The slowest component is divided by the factor, the fastest kept."""
    plain, _ = pa.pa_rope_frequencies(64, 10000.0)
    inv, _ = pa.pa_rope_frequencies(64, 10000.0, pa.PA_ROPE_BASE, factor=8.0)
    assert float(inv[0]) == 1.0
    assert float(inv[-1]) == pytest.approx(float(plain[-1]) / 8.0, rel=1e-12)


@pytest.mark.parametrize("args", [
    dict(rotary_dim=0), dict(rotary_dim=-2), dict(rotary_dim=7), dict(base=1.0), dict(base=float("nan")),
    dict(scaling=5), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("inf")),
    dict(scaling=2, rotary_dim=2, factor=2.0),
    dict(scaling=3, factor=8.0, original_max_position=0.0),
    dict(scaling=3, factor=8.0, original_max_position=8192, low=0.0, high=4.0),
    dict(scaling=4, factor=8.0, original_max_position=8192, low=4.0, high=4.0),
])
def test_frequencies_refuse_bad_arguments(args):
    a = dict(rotary_dim=64, base=10000.0, scaling=0)
    a.update(args)
    with pytest.raises(pa.PagedAttentionError, match="PA_ERR_INVALID_ARG"):
        pa.pa_rope_frequencies(a.pop("rotary_dim"), a.pop("base"), a.pop("scaling"), **a)


def test_frequencies_need_both_outputs():
    scale = ctypes.c_float()
    out = (ctypes.c_double * 32)()
    lib = _lib.lib()
    assert lib.pa_rope_frequencies(None, ctypes.byref(scale), 64, 1e4, 0, 1.0, 0.0, 1.0, 2.0) == INVALID
    assert lib.pa_rope_frequencies(out, None, 64, 1e4, 0, 1.0, 0.0, 1.0, 2.0) == INVALID
    assert lib.pa_rope_frequencies(out, ctypes.byref(scale), 64, 1e4, 0, 1.0, 0.0, 1.0, 2.0) == OK


# ----------------------------------------------------------------- refusals

@pytest.mark.parametrize("kw,expect", [
    (dict(T=0), OK),
    (dict(T=-1), INVALID),
    (dict(B=32), UNSUPPORTED),
    (dict(D=80, qs=640, ks=640, vs_=640), UNSUPPORTED),
    (dict(rot=0), INVALID),
    (dict(rot=24), UNSUPPORTED),          # not a multiple of 16
    (dict(rot=144), UNSUPPORTED),         # wider than the head
    (dict(scale=float("nan")), INVALID),
    (dict(qs=1016), INVALID),             # rows overlap
    (dict(ks=1028), INVALID),             # not a multiple of 8
    (dict(q_out=None), INVALID),
    (dict(pos=None), INVALID),
    (dict(inv=None), INVALID),
    (dict(inv=FAKE + 4), INVALID),
    (dict(key=FAKE + 8), INVALID),
    (dict(k=FAKE + 8), INVALID),
    (dict(dtype=1, ksc=0.0), INVALID),
    (dict(dtype=1, vsc=float("inf")), INVALID),
    (dict(dtype=2), INVALID),
    (dict(q_out=FAKE, qs=2048), INVALID),  # in place needs one row length
    (dict(NB=0), INVALID),
])
def test_rope_rejects_bad_arguments_on_host(kw, expect):
    a = dict(q_out=FAKE + 0x100000, q=FAKE, key=FAKE, value=FAKE, k=FAKE, v=FAKE, slots=FAKE, pos=FAKE, inv=FAKE,
             rot=128, il=0, scale=1.0, qs=1024, ks=1024, vs_=1024, T=4, Hq=8, Hkv=8, D=128, B=16, NB=64, dtype=0,
             ksc=1.0, vsc=1.0, stream=None)
    a.update(kw)
    assert _lib.lib().pa_rope_and_cache(*a.values()) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(B=8), UNSUPPORTED),
    (dict(S=16385), UNSUPPORTED),
    (dict(W=1 << 27), UNSUPPORTED),
    (dict(S=-1), INVALID),
    (dict(T=-1), INVALID),
    (dict(W=-1), INVALID),
    (dict(NB=0), INVALID),
    (dict(cap=-1), INVALID),
    (dict(bt=None), INVALID),
    (dict(lens=None), INVALID),
    (dict(new=None), INVALID),
    (dict(free=None), INVALID),
    (dict(count=None), INVALID),
    (dict(count_out=None), INVALID),
    (dict(slots=None), INVALID),
    (dict(qs=None), INVALID),
    (dict(slots=FAKE + 4), INVALID),
    (dict(pos=FAKE + 2), INVALID),
])
def test_extend_rejects_bad_arguments_on_host(kw, expect):
    a = dict(bt=FAKE, W=8, lens=FAKE, new=FAKE, free=FAKE, cap=64, count=FAKE, lens_out=FAKE, count_out=FAKE,
             slots=FAKE, pos=FAKE, qs=FAKE, S=4, T=16, B=16, NB=64, stream=None)
    a.update(kw)
    assert _lib.lib().pa_extend_tables(*a.values()) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(B=8), UNSUPPORTED),
    (dict(S=16385), UNSUPPORTED),
    (dict(W=1 << 27), UNSUPPORTED),
    (dict(keep=-1), INVALID),
    (dict(S=-1), INVALID),
    (dict(rel=None), INVALID),
    (dict(free=None), INVALID),
    (dict(lens_out=None), INVALID),
    (dict(count=FAKE + 2), INVALID),
])
def test_release_rejects_bad_arguments_on_host(kw, expect):
    a = dict(bt=FAKE, W=8, lens=FAKE, rel=FAKE, free=FAKE, cap=64, count=FAKE, lens_out=FAKE, count_out=FAKE,
             keep=0, S=4, B=16, NB=64, stream=None)
    a.update(kw)
    assert _lib.lib().pa_release_tables(*a.values()) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(S=0), OK),                       # empty batch: nothing to launch
    (dict(S=-1), INVALID),
    (dict(G=-1), INVALID),
    (dict(G=65536), UNSUPPORTED),
    (dict(maxb=1 << 27), UNSUPPORTED),
    (dict(maxp=-1), INVALID),
    (dict(maxs=-1), INVALID),
    (dict(B=8), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED),
    (dict(Hq=12, Hkv=8), UNSUPPORTED),
    (dict(Hq=32, Hkv=1), UNSUPPORTED),
    (dict(dtype=9), INVALID),
    (dict(dtype=1, ks=0.0), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(NB=0), INVALID),
    (dict(gs=None), INVALID),
    (dict(pb=None), INVALID),
    (dict(out=FAKE + 4), INVALID),
    (dict(q=None), INVALID),
    (dict(cl=None), INVALID),
    (dict(ws=None), WORKSPACE),
    (dict(wsb=255), WORKSPACE),
    (dict(ws=FAKE + 128), WORKSPACE),      # not 256-byte aligned
])
def test_shared_prefix_rejects_bad_arguments_on_host(kw, expect):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, dtype=0, ks=1.0, vs=1.0, bt=FAKE, maxb=8, cl=FAKE, maxctx=128,
             gs=FAKE, pb=FAKE, G=1, maxp=4, maxs=64, S=2, Hq=8, Hkv=8, D=128, B=16, NB=64, scale=0.1, ws=FAKE, wsb=1 << 30,
             stream=None)
    a.update(kw)
    assert _lib.lib().pa_decode_shared_prefix(*a.values()) == expect


def test_shared_prefix_workspace_grows_with_its_bounds():
    f = _lib.lib().pa_decode_shared_prefix_workspace_size
    assert f(64, 64, 8, 128, 1, 2048, 1024) > f(64, 64, 8, 128, 1, 0, 1024) > 0
    # one part of a suffix and none of a prefix: o and (m, l), 256-byte aligned
    assert f(256, 8, 8, 128, 0, 0, 100) == 256 * 8 * (512 + 8)
    assert f(0, 8, 8, 128, 0, 0, 100) == 0
    assert f(4, 9, 8, 128, 1, 4, 100) == 0      # not a whole group
    assert f(4, 8, 8, 128, 1, -1, 100) == 0
    assert f(4, 32, 1, 128, 1, 4, 100) == 0     # a group of 32


def test_binding_refuses_host_tensors_and_wrong_shapes():
    S, HQ, HKV, D, NB = 2, 4, 2, 64, 8
    bf = torch.bfloat16
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)
    q, kv = torch.empty(S, HQ, D, dtype=bf), torch.empty(S, HKV, D, dtype=bf)
    cache = torch.empty(NB, HKV, 16, D, dtype=bf)
    slots, inv = torch.zeros(S, dtype=torch.int64), torch.ones(D // 2, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.pa_rope_and_cache(q, q, kv, kv, cache, cache, slots, i32(S), inv)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.pa_extend_tables(i32(S, 4), i32(S), i32(S), i32(NB), i32(1), i32(S), i32(1), slots, i32(S), i32(S + 1))
    with pytest.raises(ValueError, match="CUDA device"):
        pa.pa_release_tables(i32(S, 4), i32(S), i32(S), i32(NB), i32(1), i32(S), i32(1))
    # the row check: a token's heads must be contiguous, tokens may be apart
    with pytest.raises(ValueError, match="heads must be contiguous"):
        pa._need_rows(torch.empty(S, 2 * HQ, D, dtype=bf)[:, ::2], "q")
    with pytest.raises(ValueError, match="heads must be contiguous"):
        pa._need_rows(torch.empty(S, HQ, 2 * D, dtype=bf)[..., ::2], "q")
    with pytest.raises(TypeError, match="dtype"):
        pa._need_rows(torch.empty(S, HQ, D), "q")
    fused = torch.empty(S, 3 * HQ, D, dtype=bf)
    with pytest.raises(ValueError, match="CUDA device"):  # only its place is wrong
        pa._need_rows(fused[:, HQ:2 * HQ], "key")


def test_shared_prefix_bounds_near_32_bits():
    """Loose bounds up to 2^31 - 1: a suffix bound only makes the parts long,
    a prefix bound past what a grid holds is refused."""
    most, limit = 2**31 - 1, 65535 * 128
    f = _lib.lib().pa_decode_shared_prefix_workspace_size
    assert f(128, 8, 8, 128, 0, 0, most) == 2 * 128 * 8 * (512 + 8)
    assert f(1, 8, 8, 128, 1, limit, 16) == (65535 + 1) * 8 * (512 + 8)
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, dtype=0, ks=1.0, vs=1.0, bt=FAKE, maxb=8, cl=FAKE, maxctx=most,
             gs=FAKE, pb=FAKE, G=1, maxp=limit, maxs=most, S=1, Hq=8, Hkv=8, D=128, B=16, NB=64, scale=0.1, ws=FAKE,
             wsb=256, stream=None)
    assert _lib.lib().pa_decode_shared_prefix(*a.values()) == WORKSPACE
    for maxp in (limit + 1, most - 7, most - 6, most):
        assert f(1, 8, 8, 128, 1, maxp, 16) == 0
        a["maxp"] = maxp
        assert _lib.lib().pa_decode_shared_prefix(*a.values()) == UNSUPPORTED
        assert f(1, 8, 8, 128, 0, maxp, 16) == 8 * 512 + 256   # without groups it bounds nothing


@pytest.mark.parametrize("scaling,high", [(pa.PA_ROPE_BANDS, 4.0), (pa.PA_ROPE_YARN, 32.0)])
def test_the_upper_bound_goes_by_the_scaling(scaling, high):
    kw = dict(factor=8.0, original_max_position=8192)
    inv, scale = pa.pa_rope_frequencies(128, 500000.0, scaling, **kw)
    want, want_scale = plain_frequencies(128, 500000.0, scaling, 8.0, 8192, 1.0, high)
    np.testing.assert_allclose(inv.numpy(), want, rtol=1e-14, atol=0)
    assert scale == pytest.approx(want_scale, rel=2 ** -23)
    given, _ = pa.pa_rope_frequencies(128, 500000.0, scaling, high=high, **kw)
    assert torch.equal(inv, given)


@pytest.mark.parametrize("big", [2**31, 2**32 + 64, -2**31 - 1])
def test_sizes_past_32_bits_raise(big):
    """Nothing is cut to its lower 32 bits on the way into the library."""
    with pytest.raises(OverflowError, match="rotary_dim"):
        pa.pa_rope_frequencies(big)
    with pytest.raises(OverflowError, match="scaling"):
        pa.pa_rope_frequencies(64, 10000.0, big)
    names = ("num_seqs", "num_q_heads", "num_kv_heads", "head_dim", "num_groups", "max_prefix_blocks",
             "max_suffix_len")
    for i, name in enumerate(names):
        a = [4, 8, 8, 64, 1, 4, 100]
        a[i] = big
        with pytest.raises(OverflowError, match=name):
            pa.pa_decode_shared_prefix_workspace_size(*a)


@pytest.mark.parametrize("kw", [dict(slots=FAKE + 4), dict(slots=FAKE + 1), dict(pos=FAKE + 2)])
def test_rope_rejects_misaligned_arrays(kw):
    a = dict(q_out=FAKE + 0x100000, q=FAKE, key=FAKE, value=FAKE, k=FAKE, v=FAKE, slots=FAKE, pos=FAKE, inv=FAKE,
             rot=128, il=0, scale=1.0, qs=1024, ks=1024, vs_=1024, T=4, Hq=8, Hkv=8, D=128, B=16, NB=64, dtype=0,
             ksc=1.0, vsc=1.0, stream=None)
    a.update(kw)
    assert _lib.lib().pa_rope_and_cache(*a.values()) == INVALID


@pytest.mark.parametrize("kw", [dict(bt=FAKE + 2), dict(cl=FAKE + 1), dict(gs=FAKE + 2), dict(pb=FAKE + 3)])
def test_shared_prefix_rejects_misaligned_arrays(kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, dtype=0, ks=1.0, vs=1.0, bt=FAKE, maxb=8, cl=FAKE, maxctx=128,
             gs=FAKE, pb=FAKE, G=1, maxp=4, maxs=64, S=2, Hq=8, Hkv=8, D=128, B=16, NB=64, scale=0.1, ws=None, wsb=0,
             stream=None)
    a.update(kw)
    assert _lib.lib().pa_decode_shared_prefix(*a.values()) == INVALID


def test_binding_refuses_workspaces_that_hold_less_than_they_say():
    with pytest.raises(ValueError, match="contiguous"):
        pa._need_workspace(torch.empty(1, dtype=torch.uint8).expand(1 << 20), -1)
    with pytest.raises(ValueError, match="contiguous"):
        pa._need_workspace(torch.empty(512, 2, dtype=torch.uint8)[:, 0], -1)
    with pytest.raises(ValueError, match="device"):
        pa._need_workspace(torch.empty(512, dtype=torch.uint8), 0)
    with pytest.raises(TypeError, match="torch.Tensor"):
        pa._need_workspace(np.empty(512, np.uint8), 0)
    pa._need_workspace(torch.empty(512, dtype=torch.uint8), -1)


@pytest.mark.parametrize("r,base,factor", [(4, 10000.0, 1e153), (64, 1e300, 1e9), (6, 1e4, 1e250)])
def test_a_stretched_base_past_64_bits_is_refused(r, base, factor):
    with pytest.raises(pa.PagedAttentionError, match="PA_ERR_INVALID_ARG"):
        pa.pa_rope_frequencies(r, base, pa.PA_ROPE_BASE, factor=factor)
    inv, _ = pa.pa_rope_frequencies(r, 10000.0, pa.PA_ROPE_BASE, factor=1e100)
    assert bool(torch.all(torch.isfinite(inv) & (inv > 0)))
