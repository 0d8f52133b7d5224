"""Rotary positions with several axes and linear attention with a decay for each head: cases, plain forms, calls.

Each case is one call of a serving step on one GPU.  ``run`` computes it either with elementary torch operations in
32 bits (``own`` false) or with the library's call (``own`` true); both take what ``prepare`` makes.

  rotary   q and k rotated by positions on one to three axes, from a packed projection; with ``write`` the
           rotated k and v go to a paged pool (bf16 or e4m3) in the same call
  decode   linear attention of one new token per sequence over its fp32 state, which it updates
  prefill  linear attention of a ragged batch of prompt chunks and single-token rows, with their states
"""
import math

import torch

own = False

BLOCK = 16  # tokens of a pool block


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of four users on a small grouped-query shape: latency only.
        dict(name="rotary 4 tokens 32/8x64", op="rotary", tokens=4, hq=32, hkv=8, d=64, rot=64, axes=1,
             interleaved=False, adjacent=False, write="bf16", far=100000),
        # A 2,048-token step budget of text beside images: time, height and width sections, keys into the cache.
        dict(name="rotary 2048 tokens 3 axes", op="rotary", tokens=2048, hq=16, hkv=8, d=128, rot=128, axes=3,
             interleaved=True, adjacent=False, write="bf16", far=4096),
        # A mixed batch of 1,568 rows into an 8-bit pool.
        dict(name="rotary 1568 tokens e4m3", op="rotary", tokens=1568, hq=16, hkv=8, d=128, rot=128, axes=3,
             interleaved=False, adjacent=False, write="e4m3", far=32768),
        # Many image patches (height and width axes) of a multi-head shape, half of the dims rotated, no cache.
        dict(name="rotary 16381 patches 2 axes", op="rotary", tokens=16381, hq=40, hkv=40, d=128, rot=64, axes=2,
             interleaved=False, adjacent=True, write="no", far=1024),
        # One user's single token: latency.
        dict(name="decode 1x16/16x128", op="decode", seqs=1, hq=16, hkv=16, d=128),
        # The 34 users whose contexts fill a small card, grouped query heads.
        dict(name="decode 34x16/8x128", op="decode", seqs=34, hq=16, hkv=8, d=128),
        # A full serving batch of a multi-head shape.
        dict(name="decode 128x40/40x128", op="decode", seqs=128, hq=40, hkv=40, d=128),
        # Narrow heads, four q heads to a state.
        dict(name="decode 61x32/8x64", op="decode", seqs=61, hq=32, hkv=8, d=64),
        # One short prompt of a new request.
        dict(name="prefill 300 16/8x128", op="prefill", lens="300", past=0, hq=16, hkv=8, d=128, packed=True),
        # A step that mixes three 512-token chunks of long prompts with 32 single-token rows.
        dict(name="prefill mixed 3x512+32", op="prefill", lens="512*3+1*32", past=1024, hq=16, hkv=8, d=128,
             packed=True),
        # Ragged prompts admitted together, narrow heads.
        dict(name="prefill ragged 12 32/8x64", op="prefill",
             lens="1500+37+640+129+1000+64+2+333+1211+18+777+450", past=0, hq=32, hkv=8, d=64, packed=False),
        # One long document.
        dict(name="prefill 16384 16/16x128", op="prefill", lens="16384", past=0, hq=16, hkv=16, d=128, packed=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "decode", "prefill"])
    d = rng.choice([64, 128])
    g = rng.choice([1, 2, 4, 8])
    if op == "rotary":
        hkv = _spread(rng, 1, 40 // g)
        t = min(_spread(rng, 1, 16381), 16381 * 80 // (hkv * (g + 2)))
        axes = rng.choice([1, 2, 3])
        return dict(op=op, tokens=t, hq=hkv * g, hkv=hkv, d=d, rot=rng.choice([d, d // 2]), axes=axes,
                    interleaved=axes > 1 and rng.random() < 0.5, adjacent=rng.random() < 0.3,
                    write=rng.choice(["no", "bf16", "e4m3"]), far=_spread(rng, 256, 1000000))
    if op == "decode":
        hkv = _spread(rng, 1, 40 // g)
        return dict(op=op, seqs=_spread(rng, 1, 128), hq=hkv * g, hkv=hkv, d=d)
    hkv = _spread(rng, 1, 16 // g)
    total = _spread(rng, 16, 16000)
    lens = []
    for _ in range(rng.choice([1, 2, 5, 9])):
        lens.append(max(1, min(total, _spread(rng, 1, 16000))))
        total -= lens[-1]
        if total < 1:
            break
    # the plain form pads every sequence to the longest
    while len(lens) > 1 and len(lens) * max(lens) ** 2 > 16000 ** 2:
        lens.remove(max(lens))
    ones = rng.choice([0, 0, 7, 19])
    if ones and (len(lens) + ones) * max(lens) ** 2 <= 16000 ** 2:
        lens += [1] * ones
    rng.shuffle(lens)
    return dict(op=op, lens="+".join(map(str, lens)), past=rng.choice([0, 1, 1000]), hq=hkv * g, hkv=hkv, d=d,
                packed=rng.random() < 0.5)


def _lens(case):
    got = []
    for part in case["lens"].split("+"):
        n, _, times = part.partition("*")
        got += [int(n)] * int(times or 1)
    return got


def _sections(case):
    """Pairs of each axis: the first takes what the others leave."""
    pairs, axes = case["rot"] // 2, case["axes"]
    return [pairs - (axes - 1) * (pairs // axes)] + [pairs // axes] * (axes - 1)


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rotary":
        t = case["tokens"]
        moved = t * ((hq + hkv) * d * 2 + hq * d * 2 + 4 * case["axes"]) + case["rot"] * 2
        if case["write"] == "no":
            moved += t * hkv * d * 2
        else:
            moved += t * (hkv * d * 2 + 2 * hkv * d * (2 if case["write"] == "bf16" else 1) + 4)
        return {"bytes": moved, "flops": t * (hq + hkv) * case["rot"] * 3}
    lens = [1] * case["seqs"] if case["op"] == "decode" else _lens(case)
    t, n = sum(lens), len(lens)
    states = n * hkv * d * d * 4
    reads = case["op"] == "decode" or case["past"] > 0
    moved = states * (2 if reads else 1) + t * ((hq + 2 * hkv) * d * 2 + hq * d * 4) + hkv * 4 + n * 16
    return {"bytes": moved, "flops": t * (hq + hkv) * 2 * d * d}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def whole(hi, *shape):
        return torch.randint(0, hi, shape, generator=gen, device=dev, dtype=torch.int32)

    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = dict(case=case)
    if case["op"] == "rotary":
        t = case["tokens"]
        qkv = normal(t, hq + 2 * hkv, d)  # the projection's output: q, k and v side by side
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
        # Text runs along the first axis; the others hold the places inside an image.
        s["positions"] = whole(case["far"], case["axes"], t)
        pair = torch.arange(case["rot"] // 2, device=dev, dtype=torch.float64)
        s["inv_freq"] = torch.pow(10000.0, -2.0 * pair / case["rot"]).float()
        s["sections"] = _sections(case)
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
        if case["write"] == "no":
            s["k_out"] = torch.empty((t, hkv, d), dtype=torch.bfloat16, device=dev)
            return s
        blocks = (t * 5 // 4 + BLOCK - 1) // BLOCK + 1
        s["slots"] = torch.randperm(blocks * BLOCK, generator=gen, device=dev)[:t].to(torch.int32)
        if case["write"] == "bf16":
            s["k_pool"], s["v_pool"] = normal(blocks, hkv, BLOCK, d), normal(blocks, hkv, BLOCK, d)
            s["k_scale"] = s["v_scale"] = None
        else:
            # codes below 0x7f: finite
            s["k_pool"] = whole(0x7F, blocks, hkv, BLOCK, d).to(torch.uint8)
            s["v_pool"] = whole(0x7F, blocks, hkv, BLOCK, d).to(torch.uint8)
            s["k_scale"], s["v_scale"] = 0.0123, 0.0171
        return s
    lens = [1] * case["seqs"] if case["op"] == "decode" else _lens(case)
    n, t = len(lens), sum(lens)
    past = 1000 if case["op"] == "decode" else case["past"]
    if case.get("packed"):
        qkv = normal(t, hq + 2 * hkv, d)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
    else:
        s.update(q=normal(t, hq, d), k=normal(t, hkv, d), v=normal(t, hkv, d))
    # Decays from one token to hundreds of tokens over the heads.
    head = torch.arange(1, hkv + 1, device=dev, dtype=torch.float32)
    s["log_decay"] = -torch.exp2(-8.0 * head / hkv) * (0.9 + 0.2 * torch.rand(hkv, generator=gen, device=dev))
    # The states before the step, then those after it: a sequence reads one of the first n and writes one of the last.
    s["states"] = 4.0 * normal(2 * n, hkv, d, d, dtype=torch.float32)
    s["slots"] = torch.randperm(n, generator=gen, device=dev).to(torch.int32)
    s["new_slots"] = (n + torch.randperm(n, generator=gen, device=dev)).to(torch.int32)
    s["context_lens"] = torch.tensor([past + x for x in lens], dtype=torch.int32, device=dev)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty((t, hq, d), dtype=torch.float32, device=dev)
    if case["op"] == "prefill":
        starts = [0]
        for x in lens:
            starts.append(starts[-1] + x)
        s["start_host"] = torch.tensor(starts, dtype=torch.int32)
        s["start"] = s["start_host"].to(dev)
        s["longest"] = max(lens)
        if own:
            import paged_kv_cache_291_gb300 as pkv
            s["workspace"] = pkv.new_workspace(pkv.linear_prefill_workspace_size(n, t, hq, hkv, d), dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"rotary": _rotary, "decode": _decode, "prefill": _prefill}[s["case"]["op"]](s)


def _axis_of_pair(sections, interleaved, dev):
    """The axis of each pair: section by section, or dealt to the axes in turn while they have pairs left."""
    turn = torch.cat([torch.arange(n, device=dev) * (len(sections) if interleaved else 0) + a
                      for a, n in enumerate(sections)])
    axis = torch.cat([torch.full((n,), a, device=dev) for a, n in enumerate(sections)])
    return axis[torch.argsort(turn, stable=True)] if interleaved else axis


def _turn(x, cos, sin, case):
    """x [tokens][heads][d] in 32 bits, rotated by cos and sin [tokens][1][pairs]."""
    r, p = case["rot"], case["rot"] // 2
    if case["adjacent"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :p], x[..., p:r]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., r:]), -1)


def _codes(x, scale):
    inv = torch.ones((), device=x.device) / scale
    return (x * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _rotary(s):
    case = s["case"]
    write = case["write"]
    if own:
        import paged_kv_cache_291_gb300 as pkv
        how = dict(sections=s["sections"], interleaved_axes=case["interleaved"], adjacent_pairs=case["adjacent"],
                   q_out=s["q_out"])
        if write == "no":
            return pkv.rotary(s["q"], s["k"], s["positions"], s["inv_freq"], k_out=s["k_out"], **how)
        q_out = pkv.rotary_cache_write(s["k_pool"], s["v_pool"], s["q"], s["k"], s["v"], s["slots"], s["positions"],
                                       s["inv_freq"], k_scale=s["k_scale"], v_scale=s["v_scale"], **how)
    else:
        axis = _axis_of_pair(s["sections"], case["interleaved"], s["q"].device)
        # far positions: the angle in 64 bits
        angle = s["positions"].double()[axis].t() * s["inv_freq"].double()
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        q_out, k_out = _turn(s["q"].float(), cos, sin, case).bfloat16(), _turn(s["k"].float(), cos, sin, case)
        if write == "no":
            return q_out, k_out.bfloat16()
        block, row = s["slots"].long() // BLOCK, s["slots"].long() % BLOCK
        if write == "bf16":
            s["k_pool"][block, :, row] = k_out.bfloat16()
            s["v_pool"][block, :, row] = s["v"]
        else:
            s["k_pool"][block, :, row] = _codes(k_out, s["k_scale"])
            s["v_pool"][block, :, row] = _codes(s["v"].float(), s["v_scale"])
    if write == "e4m3":
        return q_out, s["k_pool"].view(torch.float8_e4m3fn), s["v_pool"].view(torch.float8_e4m3fn)
    return q_out, s["k_pool"], s["v_pool"]


def _decode(s):
    n = s["q"].shape[0]
    if own:
        import paged_kv_cache_291_gb300 as pkv
        out = pkv.linear_decode_attention(s["states"], s["log_decay"], s["q"], s["k"], s["v"], s["slots"],
                                          s["context_lens"], s["scale"], new_slots=s["new_slots"], out=s["out"])
        return out, s["states"][n:]
    hkv, d = s["case"]["hkv"], s["case"]["d"]
    new = s["states"][s["slots"].long()] * torch.exp(s["log_decay"])[:, None, None]
    new = new + s["k"].float()[..., :, None] * s["v"].float()[..., None, :]
    s["states"][s["new_slots"].long()] = new
    out = torch.matmul(s["q"].float().view(n, hkv, -1, d), new) * s["scale"]
    return out.reshape(n, -1, d), s["states"][n:]


def _prefill(s):
    n = s["slots"].shape[0]
    if own:
        import paged_kv_cache_291_gb300 as pkv
        out = pkv.linear_prefill_attention(s["states"], s["log_decay"], s["q"], s["k"], s["v"], s["start"], s["slots"],
                                           s["context_lens"], s["scale"], new_slots=s["new_slots"], out=s["out"],
                                           workspace=s["workspace"], query_start_loc_host=s["start_host"])
        return out, s["states"][n:]
    hq, hkv, d, dev = s["case"]["hq"], s["case"]["hkv"], s["case"]["d"], s["q"].device
    tokens, longest = s["q"].shape[0], s["longest"]
    place = torch.arange(longest, device=dev)
    count = s["start"][1:] - s["start"][:-1]
    inside = (place < count[:, None])[:, :, None, None]
    rows = (s["start"][:-1, None] + place).clamp(max=tokens - 1).long()
    # padded: q [n][hkv][group][longest][d], k and v [n][hkv][1][longest][d]
    q = s["q"].float()[rows].view(n, longest, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    k = torch.where(inside, s["k"].float()[rows], 0.0).transpose(1, 2)[:, :, None]
    v = torch.where(inside, s["v"].float()[rows], 0.0).transpose(1, 2)[:, :, None]
    g = s["log_decay"][:, None, None]
    ago = place[:, None] - place
    decay = torch.where(ago >= 0, torch.exp(g * ago), 0.0)
    fresh = (s["context_lens"] == count)[:, None, None, None]
    before = torch.where(fresh, 0.0, s["states"][s["slots"].long()])
    score = torch.matmul(q, k.transpose(-1, -2))
    score *= decay[:, None]
    out = torch.matmul(score, v)
    del score, decay
    out += torch.matmul(q * torch.exp(g * (place[:, None] + 1))[:, None], before[:, :, None])
    out *= s["scale"]
    left = count[:, None, None, None] - 1 - place[:, None]
    weight = torch.where(left >= 0, torch.exp(g * left), 0.0)
    after = torch.matmul((k[:, :, 0] * weight).transpose(-1, -2), v[:, :, 0])
    after += before * torch.exp(g * count[:, None, None, None])
    s["states"][s["new_slots"].long()] = after
    row = torch.arange(tokens, device=dev, dtype=torch.int32)
    seq = torch.searchsorted(s["start"], row, right=True) - 1
    out = out.reshape(n, hq, longest, d)[seq, :, (row - s["start"][seq]).long()]
    return out, s["states"][n:]


# ---------------------------------------------------------------- from the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] == "rotary":
        # Each pair as a complex number, times exp(i angle).
        owners, left = [], list(s["sections"])
        while sum(left):
            for a in range(len(left)):
                take = min(left[a], 1 if case["interleaved"] else left[a])
                owners += [a] * take
                left[a] -= take
        angle = torch.stack([s["positions"][a].double() * s["inv_freq"][i].double() for i, a in enumerate(owners)], -1)
        unit = torch.polar(torch.ones_like(angle), angle)[:, None]

        def turned(x):
            y, p = x.double(), case["rot"] // 2
            at = torch.arange(p, device=x.device)
            first, second = (2 * at, 2 * at + 1) if case["adjacent"] else (at, at + p)
            z = torch.complex(y[..., first], y[..., second]) * unit
            y[..., first], y[..., second] = z.real, z.imag
            return y

        if case["write"] == "no":
            return turned(s["q"]), turned(s["k"])
        pools = []
        for name, rows in (("k", turned(s["k"])), ("v", s["v"].double())):
            pool = s[name + "_pool"]
            if case["write"] == "e4m3":
                pool = pool.view(torch.float8_e4m3fn)
                rows = (rows / s[name + "_scale"]).clamp(-448.0, 448.0)
            pool = pool.double().transpose(1, 2).reshape(-1, hkv, d)  # by slot
            pool[s["slots"].long()] = rows
            pools.append(pool.view(-1, BLOCK, hkv, d).transpose(1, 2))
        return turned(s["q"]), pools[0], pools[1]
    # The recurrence, token by token, every sequence at once.
    lens = [1] * case["seqs"] if case["op"] == "decode" else _lens(case)
    n, t = len(lens), sum(lens)
    count = torch.tensor(lens, device=s["q"].device)
    start = torch.cumsum(count, 0) - count
    lam = torch.exp(s["log_decay"].double())[:, None, None]
    state = s["states"][s["slots"].long()].double()
    state[s["context_lens"] == count] = 0.0
    out = torch.empty((t, hq, d), dtype=torch.float64, device=s["q"].device)
    for i in range(max(lens)):
        live = torch.tensor([j for j in range(n) if lens[j] > i], device=s["q"].device) if n > 1 else slice(None)
        at = start[live] + i
        k, v, q = s["k"][at].double(), s["v"][at].double(), s["q"][at].double()
        now = state[live] * lam + k[..., :, None] * v[..., None, :]
        state[live] = now
        out[at] = torch.matmul(q.view(-1, hkv, hq // hkv, d), now).reshape(-1, hq, d) * s["scale"]
    after = s["states"].double()
    after[s["new_slots"].long()] = state
    return out, after[n:]
