"""Cases for the serving-step operators: block tables and slot maps built on
the GPU (extend, release), rotary positions with the cache write (rope), and
decode attention over a shared prefix (shared).

`run` computes each operator either in its plain form (elementary torch
operations) or, where `own` is true, through the package's entry points.
"""
import math

import torch

own = False

BS = 16  # tokens of a cache block


# --------------------------------------------------------------------- cases

def _rope(name, tokens, hq, hkv, d, rot, fp8=False, interleaved=False, scaling="none", prompts=False,
          fused=True, max_pos=2048):
    c = dict(op="rope", tokens=tokens, hq=hq, hkv=hkv, d=d, rot=rot, fp8=fp8, interleaved=interleaved,
             scaling=scaling, prompts=prompts, fused=fused, max_pos=max_pos)
    return dict(c, name=name) if name else c


def _extend(name, seqs, width, max_len, prompts):
    c = dict(op="extend", seqs=seqs, width=width, max_len=max_len, prompts=prompts)
    return dict(c, name=name) if name else c


def _release(name, seqs, width, share, keep):
    c = dict(op="release", seqs=seqs, width=width, share=share, keep=keep)
    return dict(c, name=name) if name else c


def _shared(name, seqs, hq, hkv, d, prefix, groups, lo, hi, fp8=False, heavy=False):
    c = dict(op="shared", seqs=seqs, hq=hq, hkv=hkv, d=d, prefix=prefix, groups=groups, lo=lo, hi=hi, fp8=fp8,
             heavy=heavy)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of the 64-sequence, 32-head workload: one new token each, views of the fused projection
        _rope("rope_decode_mha", 64, 32, 32, 128, 128),
        # one decode step of the fp8 GQA workload, positions stretched for long contexts
        _rope("rope_decode_gqa_fp8", 128, 32, 8, 128, 128, fp8=True, scaling="yarn", max_pos=131072),
        # sixteen prompts of up to 2048 tokens in one prefill
        _rope("rope_prompts", 32768, 32, 8, 128, 128, prompts=True, scaling="bands", max_pos=2048),
        # an odd number of prompt tokens, small heads, interleaved pairs in half of each head, separate tensors
        _rope("rope_partial_ragged", 1037, 8, 8, 64, 32, interleaved=True, prompts=True, fused=False, max_pos=65536),
        # a decode step of the serving loop's largest batch: one token for each of 128 requests
        _extend("extend_decode", 128, 128, 2047, False),
        # a large admission beside decoding requests: two thousand rows, prompts of up to 4096 tokens
        _extend("extend_admit", 2000, 256, 4096, True),
        # a few of the loop's 128 requests end in a step and leave a shared prefix behind
        _release("release_few", 128, 128, 0.05, 4),
        # a drained batch: most of two thousand rows give their blocks back
        _release("release_most", 2000, 256, 0.9, 0),
        # smallest decode: four sequences behind a 16-block prompt
        _shared("shared_tiny", 4, 8, 8, 64, 16, 1, 1, 64),
        # 256 sequences, 40 heads, a 62-block system prompt, long-tailed private parts
        _shared("shared_prompt_mha", 256, 40, 40, 128, 62, 1, 1, 2048, heavy=True),
        # 64 sequences, 64 query heads on 8 KV heads, behind one 32768-token document
        _shared("shared_long_gqa", 64, 64, 8, 128, 2048, 1, 1, 1024),
        # three long documents in an fp8 cache, questions of up to 500 tokens behind them
        _shared("shared_docs_gqa_fp8", 130, 32, 8, 128, 1024, 3, 1, 500, fp8=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "extend", "release", "shared", "shared"])
    if op == "rope":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8, 32])
        hq = hkv * (rng.choice([1, 2, 4, 7, 8]) if hkv <= 8 else 1)
        prompts = rng.random() < 0.5
        return _rope("", _log(rng, 64, 20000) if prompts else _log(rng, 1, 512), hq, hkv, d,
                     rng.choice([d, d, d // 2, 16, 48]), fp8=rng.random() < 0.4, interleaved=rng.random() < 0.4,
                     scaling=rng.choice(["none", "linear", "bands", "yarn"]), prompts=prompts,
                     fused=rng.random() < 0.7, max_pos=rng.choice([2048, 65536, 131072, 1000000]))
    if op == "extend":
        width = _log(rng, 8, 256)
        return _extend("", _log(rng, 1, 2000), width, rng.randint(16, 16 * width), rng.random() < 0.5)
    if op == "release":
        return _release("", _log(rng, 1, 2000), _log(rng, 4, 256), round(rng.uniform(0.01, 1.0), 3), rng.choice([0, 0, 1, 3]))
    fp8 = rng.random() < 0.4
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8, 16])
    seqs = _log(rng, 1, 200)
    prefix = min(_log(rng, 1, 2048), 8388608 // (seqs * hq))
    return _shared("", seqs, hq, hkv, d, prefix, rng.randint(1, min(4, seqs)), rng.choice([0, 1]),
                   _log(rng, 16, 1024), fp8=fp8)


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(lo, hi, shape, g):
    """Uniform whole numbers of [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int64)


def _inv_freq(rot, scaling):
    """Angles per position, in 64 bits, and the factor on cos and sin.

    linear: positions divided by 4. bands: fast components kept, slow ones
    divided by 8, a ramp between (a wavelength against an original context
    of 8192). yarn: the ramp over the components that turn 32 times and
    once in an original context of 4096, stretched 16 times, with the
    attention factor 0.1 ln 16 + 1."""
    base = 500000.0 if scaling == "bands" else 10000.0
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = base ** (-i / rot)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "bands":
        ramp = ((8192.0 * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f * (ramp + (1 - ramp) / 8.0), 1.0
    if scaling == "yarn":
        def at(turns):
            return rot * math.log(4096.0 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * ((1 - ramp) + ramp / 16.0), 0.1 * math.log(16.0) + 1.0
    return f, 1.0


def _prepare_rope(c, seed):
    g = _gen(seed)
    T, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["d"]
    heads = hq + 2 * hkv
    qkv = _randn((T, heads, d), g).to(torch.bfloat16)
    parts = qkv.split([hq, hkv, hkv], dim=1)
    q, k, v = parts if c["fused"] else (p.contiguous() for p in parts)
    if c["prompts"]:  # several prompts one behind the other, each from a position of its own on (chunks)
        nb = -(-T // BS) + 32
        t = torch.arange(T, device="cuda")
        cut = max(1, min(T, c["max_pos"] // 2))
        start = _ints(0, max(0, c["max_pos"] - cut - 1), (T // cut + 1,), g)
        positions = start[t // cut] + t % cut
        blocks = torch.randperm(nb, generator=g, device="cuda")
        slots = blocks[t // BS] * BS + t % BS
    else:
        nb = T + 32
        positions = _ints(0, c["max_pos"] - 1, (T,), g)
        blocks = torch.randperm(nb, generator=g, device="cuda")[:T]
        slots = blocks * BS + positions % BS
    pad = T // 50  # rows behind the last sequence of a padded batch
    if pad:
        slots[T - pad:] = -1
    inv, factor = _inv_freq(c["rot"], c["scaling"])
    # one block more than the pool has: the plain form writes the padding there
    room = (nb + 1, hkv, BS, d)
    dt = torch.float8_e4m3fn if c["fp8"] else torch.bfloat16
    return dict(c=c, q=q, k=k, v=v, nb=nb, positions=positions.to(torch.int32), slots=slots,
                inv_freq=inv.cuda(), factor=float(factor), q_out=torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda"),
                k_room=torch.zeros(room, device="cuda").to(dt), v_room=torch.zeros(room, device="cuda").to(dt),
                k_scale=0.0125 if c["fp8"] else 1.0, v_scale=0.01 if c["fp8"] else 1.0)


def _prepare_extend(c, seed):
    g = _gen(seed)
    S, W = c["seqs"], c["width"]
    cap = min(c["max_len"], W * BS)
    if c["prompts"]:
        total = _ints(1, cap, (S,), g)
        lens = torch.where(torch.rand(S, generator=g, device="cuda") < 0.4, total - 1, torch.zeros_like(total))
        new = total - lens
        new[_ints(0, S - 1, (max(1, S // 16),), g)] = 0  # rows that wait in this step
    else:
        lens = _ints(0, cap - 1, (S,), g)
        new = torch.ones_like(lens)
    old = -(-lens // BS)
    need = -(-(lens + new) // BS) - old
    held, wanted = int(old.sum()), int(need.sum())
    nb = held + wanted + 64
    ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(W, device="cuda")[None]
    first = (torch.cumsum(old, 0) - old)[:, None]
    tables = torch.where(j < old[:, None], ids[(first + j).clamp(max=nb - 1)], ids.new_full((), -1))
    count = nb - held
    free = torch.cat([ids[held:], ids.new_full((held,), -1)])
    # the token bound of a padded batch: about a tenth more than the rows have on average, and one long row
    T = int(0.33 * S * cap) + cap + 64 if c["prompts"] else S + S // 16
    e = lambda n, dt: torch.empty(n, dtype=dt, device="cuda")  # noqa: E731
    return dict(c=c, tables=tables.contiguous(), lens=lens.to(torch.int32), new=new.to(torch.int32), free=free,
                count=torch.tensor([count], dtype=torch.int32, device="cuda"), T=T, lens_out=e(S, torch.int32),
                count_out=e(1, torch.int32), slots=e(T, torch.int64), positions=e(T, torch.int32),
                query_start=e(S + 1, torch.int32))


def _prepare_release(c, seed):
    g = _gen(seed)
    S, W, keep = c["seqs"], c["width"], min(c["keep"], c["width"])
    lens = _ints(0, W * BS, (S,), g)
    held = (-(-lens // BS) - keep).clamp(min=0)
    nb = S * W + keep + 100
    ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(W, device="cuda")[None]
    first = (torch.cumsum(held, 0) - held)[:, None]
    mine = ids[(keep + first + j - keep).clamp(0, nb - 1)]
    tables = torch.where(j < keep, ids[j.clamp(max=nb - 1)], mine)
    tables = torch.where(j < -(-lens // BS)[:, None], tables, tables.new_full((), -1))
    n = int(held.sum())
    free = torch.cat([ids[keep + n:], ids.new_full((keep + n,), -1)])
    return dict(c=c, keep=keep, tables=tables.contiguous(), lens=lens.to(torch.int32),
                mask=(torch.rand(S, generator=g, device="cuda") < c["share"]).to(torch.int32), free=free,
                count=torch.tensor([nb - keep - n], dtype=torch.int32, device="cuda"),
                lens_out=torch.empty(S, dtype=torch.int32, device="cuda"),
                count_out=torch.empty(1, dtype=torch.int32, device="cuda"))


def _shared_lengths(c):
    """Suffix lengths and the groups' first sequences, from the sizes alone (so that `work` knows them)."""
    S, G = c["seqs"], c["groups"]
    g = torch.Generator()
    g.manual_seed(S * 1000003 + c["hi"] * 101 + c["prefix"])
    if c["heavy"]:  # lognormal with a median of 300 tokens
        n = torch.exp(math.log(300.0) + torch.randn(S, generator=g, dtype=torch.float64)).round().to(torch.int64)
    else:
        n = torch.randint(c["lo"], c["hi"] + 1, (S,), generator=g)
    n = n.clamp(c["lo"], c["hi"])
    cuts = [round(S * (i / G) ** 1.5) for i in range(G + 1)]  # groups of different sizes
    prefix = [max(1, round(c["prefix"] / (1 + 0.7 * i))) for i in range(G)]
    return n, cuts, prefix


def _prepare_shared(c, seed):
    g = _gen(seed)
    S, hq, hkv, d = c["seqs"], c["hq"], c["hkv"], c["d"]
    n, cuts, prefix = _shared_lengths(c)
    n = n.cuda()
    group_start = torch.tensor(cuts, dtype=torch.int64, device="cuda")
    pblocks = torch.tensor(prefix, dtype=torch.int64, device="cuda")
    of = torch.searchsorted(group_start, torch.arange(S, device="cuda"), right=True) - 1
    lens = pblocks[of] * BS + n
    own_blocks = -(-n // BS)
    shared_blocks = sum(prefix)
    nb = int((shared_blocks + int(own_blocks.sum())) * 1.1) + 8
    ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    W = int((-(-lens // BS)).max())
    j = torch.arange(W, device="cuda")[None]
    pre_first = (torch.cumsum(pblocks, 0) - pblocks)[of][:, None]
    own_first = (shared_blocks + torch.cumsum(own_blocks, 0) - own_blocks)[:, None]
    p = pblocks[of][:, None]
    tables = torch.where(j < p, ids[(pre_first + j).clamp(max=nb - 1)], ids[(own_first + j - p).clamp(0, nb - 1)])
    tables = torch.where(j < p + own_blocks[:, None], tables, tables.new_full((), -1))
    shape = (nb, hkv, BS, d)
    scale = (0.0125, 0.01) if c["fp8"] else (1.0, 1.0)

    def cache(sc):
        x = _randn(shape, g)
        return (x / sc).clamp(-448, 448).to(torch.float8_e4m3fn) if c["fp8"] else x.to(torch.bfloat16)

    kc, vc = cache(scale[0]), cache(scale[1])
    # slots behind a sequence's last token hold whatever an earlier request left: NaN here
    r = torch.arange(S, device="cuda")
    last = tables[r, ((lens - 1) // BS).clamp(min=0)].long()
    stale = (torch.arange(BS, device="cuda")[None] >= ((lens - 1) % BS + 1)[:, None]) & (n > 0)[:, None]
    nan = 0x7F if c["fp8"] else 0x7FC0
    for t in (kc, vc):
        u = t.view(torch.uint8) if c["fp8"] else t.view(torch.int16)
        u[last] = torch.where(stale[:, None, :, None], u.new_full((), nan), u[last])
    return dict(c=c, q=_randn((S, hq, d), g).to(torch.bfloat16), kc=kc, vc=vc, tables=tables.contiguous(),
                lens=lens.to(torch.int32), max_len=int(lens.max()), group_start=group_start.to(torch.int32),
                pblocks=pblocks.to(torch.int32), max_prefix=max(prefix), of=of, rank=r - group_start[of],
                most=max(b - a for a, b in zip(cuts, cuts[1:])), max_suffix=max(1, int(own_blocks.max())),
                out=torch.empty((S, hq, d), dtype=torch.float32, device="cuda"), k_scale=scale[0], v_scale=scale[1],
                sm_scale=d ** -0.5, suffix_len=max(1, int(n.max())))


def prepare(case, seed):
    return {"rope": _prepare_rope, "extend": _prepare_extend, "release": _prepare_release,
            "shared": _prepare_shared}[case["op"]](case, seed)


# --------------------------------------------------------------- plain forms

def _rotated(x, cos, sin, rot, interleaved):
    """x [T][H][d] in 32 bits, its first `rot` elements of each head turned."""
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _plain_rope(s):
    c = s["c"]
    angle = s["positions"].double()[:, None] * s["inv_freq"][None]
    cos = (angle.cos() * s["factor"]).float()[:, None]
    sin = (angle.sin() * s["factor"]).float()[:, None]
    q = _rotated(s["q"], cos, sin, c["rot"], c["interleaved"]).to(torch.bfloat16)
    k = _rotated(s["k"], cos, sin, c["rot"], c["interleaved"])
    slots = torch.where(s["slots"] < 0, s["nb"] * BS, s["slots"])
    block, off = slots // BS, slots % BS
    if c["fp8"]:
        k = (k / s["k_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (s["v"].float() / s["v_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["k_room"].view(torch.uint8)[block, :, off] = k
        s["v_room"].view(torch.uint8)[block, :, off] = v
    else:
        s["k_room"][block, :, off] = k.to(torch.bfloat16)
        s["v_room"][block, :, off] = s["v"]
    return {"q": q, "k": s["k_room"][: s["nb"]], "v": s["v_room"][: s["nb"]]}


def _plain_extend(s):
    S, W, T = s["c"]["seqs"], s["c"]["width"], s["T"]
    lens, new, free, count = s["lens"].long(), s["new"].long(), s["free"], s["count"].long()
    old = (lens + BS - 1) // BS
    now = (lens + new + BS - 1) // BS
    need = now - old
    first = torch.cumsum(need, 0) - need
    ends = torch.cumsum(new, 0)
    fine = (need.sum() <= count) & (now.max() <= W) & (ends[-1] <= T) & (lens.min() >= 0) & (new.min() >= 0)
    j = torch.arange(W, device="cuda")[None]
    taken = free[(count - 1 - (first[:, None] + j - old[:, None])).clamp(0, free.numel() - 1)]
    tables = torch.where((j >= old[:, None]) & (j < now[:, None]) & fine, taken, s["tables"])
    t = torch.arange(T, device="cuda")
    row = torch.searchsorted(ends, t, right=True).clamp(max=S - 1)
    live = (t < ends[-1]) & fine
    p = torch.where(live, lens[row] + t - (ends - new)[row], 0)
    slots = torch.where(live, tables[row, (p // BS).clamp(max=W - 1)].long() * BS + p % BS, -1)
    start = torch.cat([ends.new_zeros(1), ends]) * fine
    return {"tables": tables, "lens": torch.where(fine, lens + new, lens).to(torch.int32),
            "count": torch.where(fine, count - need.sum(), count).to(torch.int32), "slots": slots,
            "positions": p.to(torch.int32), "start": start.to(torch.int32)}


def _plain_release(s):
    keep, tables = s["keep"], s["tables"]
    lens, count, go = s["lens"].long(), s["count"].long(), s["mask"] != 0
    held = torch.where(go, ((lens + BS - 1) // BS - keep).clamp(min=0), 0)
    first = torch.cumsum(held, 0) - held
    j = torch.arange(s["c"]["width"], device="cuda")[None] - keep
    live = (j >= 0) & (j < held[:, None])
    nb = s["free"].numel()
    to = torch.where(live, count + first[:, None] + j, nb)
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    free[to.reshape(-1)] = tables.reshape(-1)
    return {"free": free[:nb], "count": (count + held.sum()).to(torch.int32),
            "lens": torch.where(go, lens.clamp(max=keep * BS), lens).to(torch.int32)}


def _plain_shared(s):
    c = s["c"]
    S, hq, hkv, d, G = c["seqs"], c["hq"], c["hkv"], c["d"], c["groups"]
    grp = hq // hkv
    q = s["q"].float().view(S, hkv, grp, d) * (s["sm_scale"] * s["k_scale"])
    lens, of, pblocks, tables = s["lens"].long(), s["of"], s["pblocks"].long(), s["tables"].long()

    def rows(cache, blocks):  # [...][n] block ids -> [...][hkv][16 n][d] in 32 bits
        x = cache.view(torch.uint8)[blocks].view(torch.float8_e4m3fn) if c["fp8"] else cache[blocks]
        return x.float().movedim(-3, -4).flatten(-3, -2)

    # the prefixes: each group's sequences against its first blocks, once
    P = s["max_prefix"]
    pre = tables[s["group_start"].long()[:-1], :P].clamp(min=0)
    qg = q.new_zeros((G, s["most"], hkv, grp, d))
    qg[of, s["rank"]] = q
    qg = qg.movedim(1, 2).flatten(2, 3)                                  # [G][hkv][most grp][d]
    z1 = qg @ rows(s["kc"], pre).transpose(-1, -2)
    seen = torch.arange(P * BS, device="cuda")[None] < pblocks[:, None] * BS
    z1 = z1.masked_fill(~seen[:, None, None], -torch.inf)
    # the private parts, a padded gather
    j = torch.arange(s["max_suffix"], device="cuda")[None] + pblocks[of][:, None]
    mine = torch.gather(tables, 1, j.clamp(max=tables.shape[1] - 1)).clamp(min=0)
    live = (torch.arange(s["max_suffix"] * BS, device="cuda")[None] < (lens - pblocks[of] * BS)[:, None])[:, None]
    z2 = (q @ rows(s["kc"], mine).transpose(-1, -2)).masked_fill(~live[:, :, None], -torch.inf)
    m1 = z1.amax(-1).view(G, hkv, s["most"], grp).movedim(2, 1)[of, s["rank"]]
    m = torch.maximum(m1, z2.amax(-1))
    mg = m.new_zeros((G, s["most"], hkv, grp))
    mg[of, s["rank"]] = m
    e1 = torch.exp(z1 - mg.movedim(1, 2).reshape(G, hkv, -1, 1))
    e2 = torch.exp(z2 - m[..., None])
    v1 = rows(s["vc"], pre).masked_fill(~seen[:, None, :, None], 0.0)
    o1 = (e1 @ v1).view(G, hkv, s["most"], grp, d).movedim(2, 1)[of, s["rank"]]
    l1 = e1.sum(-1).view(G, hkv, s["most"], grp).movedim(2, 1)[of, s["rank"]]
    v2 = rows(s["vc"], mine).masked_fill(~live[..., None], 0.0)
    o = (o1 + e2 @ v2) / (l1 + e2.sum(-1))[..., None] * s["v_scale"]
    return o.reshape(S, hq, d)


# ------------------------------------------------------------------- a pass

def run(state):
    s, op = state, state["c"]["op"]
    if own:
        import paged_kv_cache_429_b200 as pa
        if op == "rope":
            k, v = s["k_room"][: s["nb"]], s["v_room"][: s["nb"]]
            pa.pa_rope_and_cache(s["q_out"], s["q"], s["k"], s["v"], k, v, s["slots"], s["positions"], s["inv_freq"],
                                 interleaved=s["c"]["interleaved"], rope_scale=s["factor"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"])
            return {"q": s["q_out"], "k": k, "v": v}
        if op == "extend":
            pa.pa_extend_tables(s["tables"], s["lens"], s["new"], s["free"], s["count"], s["lens_out"], s["count_out"],
                                s["slots"], s["positions"], s["query_start"])
            return {"tables": s["tables"], "lens": s["lens_out"], "count": s["count_out"], "slots": s["slots"],
                    "positions": s["positions"], "start": s["query_start"]}
        if op == "release":
            pa.pa_release_tables(s["tables"], s["lens"], s["mask"], s["free"], s["count"], s["lens_out"],
                                 s["count_out"], keep_blocks=s["keep"])
            return {"free": s["free"], "count": s["count_out"], "lens": s["lens_out"]}
        pa.pa_decode_shared_prefix(s["out"], s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["max_len"],
                                   s["group_start"], s["pblocks"], s["max_prefix"], s["sm_scale"],
                                   max_suffix_len=s["suffix_len"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"]
    return {"rope": _plain_rope, "extend": _plain_extend, "release": _plain_release, "shared": _plain_shared}[op](s)


# ------------------------------------------------------------- 64-bit values

def _exact_rope(case, seed):
    s = _prepare_rope(case, seed)
    c, half = s["c"], s["c"]["rot"] // 2
    x = torch.outer(s["positions"].double(), s["inv_freq"])
    turn = torch.polar(torch.full_like(x, s["factor"]), x)[:, None]      # complex numbers of length `factor`

    def turned(t):
        t = t.double()
        y = t.clone()
        if c["interleaved"]:
            z = torch.view_as_complex(t[..., : c["rot"]].reshape(*t.shape[:2], half, 2).contiguous()) * turn
            y[..., : c["rot"]] = torch.view_as_real(z).reshape(*t.shape[:2], c["rot"])
        else:
            z = torch.complex(t[..., :half].contiguous(), t[..., half: c["rot"]].contiguous()) * turn
            y[..., :half], y[..., half: c["rot"]] = z.real, z.imag
        return y

    slots = s["slots"]
    kept = slots >= 0

    def cached(t, scale):
        room = torch.zeros((s["nb"] * BS, c["hkv"], c["d"]), dtype=torch.float64, device="cuda")
        room[slots[kept]] = (t / scale).clamp(-448, 448)[kept] if c["fp8"] else t[kept]
        return room.view(s["nb"], BS, c["hkv"], c["d"]).transpose(1, 2)

    return {"q": turned(s["q"]), "k": cached(turned(s["k"]), s["k_scale"]), "v": cached(s["v"].double(), s["v_scale"])}


def _exact_shared(case, seed):
    s = _prepare_shared(case, seed)
    c = s["c"]
    hkv, d = c["hkv"], c["d"]
    out = torch.zeros((c["seqs"], c["hq"], d), dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):  # sequence by sequence, its whole context gathered
        if n == 0:
            continue
        b = s["tables"][i, : -(-n // BS)].long()
        k, v = (t[b].double().transpose(0, 1).reshape(hkv, -1, d)[:, :n]
                if not c["fp8"] else
                t.view(torch.uint8)[b].view(torch.float8_e4m3fn).double().transpose(0, 1).reshape(hkv, -1, d)[:, :n]
                for t in (s["kc"], s["vc"]))
        z = torch.bmm(s["q"][i].double().view(hkv, -1, d), k.transpose(1, 2)) * s["k_scale"] * s["sm_scale"]
        out[i] = torch.bmm(torch.softmax(z, -1), v).reshape(-1, d) * s["v_scale"]
    return out


def exact(case, seed):
    """Extend and release give whole numbers only: they have no such values."""
    if case["op"] == "rope":
        return _exact_rope(case, seed)
    return _exact_shared(case, seed) if case["op"] == "shared" else None


# ---------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "rope":
        elements = c["tokens"] * c["d"]
        eb = 1 if c["fp8"] else 2
        return {"bytes": elements * (2 * (c["hq"] + 2 * c["hkv"]) + 2 * c["hq"] + 2 * eb * c["hkv"]) + 12 * c["tokens"],
                "flops": 3 * c["tokens"] * c["rot"] * (c["hq"] + c["hkv"])}
    if c["op"] == "extend":
        # lengths in and out; a slot, a position and a sixteenth of a table entry for a token
        cap = min(c["max_len"], c["width"] * BS)
        tokens = c["seqs"] * (cap / 2 * 0.6 + 0.4 if c["prompts"] else 1)
        return {"bytes": 16 * c["seqs"] + tokens * (12 + 8 / BS), "flops": 0}
    if c["op"] == "release":
        return {"bytes": 12 * c["seqs"] + c["seqs"] * c["share"] * (c["width"] / 2) * 8, "flops": 0}
    n, cuts, prefix = _shared_lengths(c)
    eb = 1 if c["fp8"] else 2
    kv = (int(n.sum()) + BS * sum(prefix)) * c["hkv"] * c["d"] * 2 * eb
    total = int(n.sum()) + sum(BS * p * (b - a) for p, a, b in zip(prefix, cuts, cuts[1:]))
    return {"bytes": kv + c["seqs"] * c["hq"] * c["d"] * 6 + total // 4,
            "flops": 4 * c["hq"] * c["d"] * total}
