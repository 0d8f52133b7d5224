"""A paged cache held in 8 bits with a scale for each block and kv head: cases, plain forms, calls.

Each case is one call of a serving step on one GPU.  ``run`` computes it either with elementary torch operations in
32 bits (``own`` false; sums over a context in 64) or with the library's call (``own`` true); both take what
``prepare`` makes.

  append   the step's new k and v rows quantised into the last blocks of their sequences; a block whose scale grows
           has its earlier rows quantised again
  read     rows of the cache back as bf16, in order
  decode   attention of one new token per sequence over its context
  prefill  causal attention of prompt chunks over their context, beside single-token rows
"""
import math

import torch

own = False

BLOCK = 16  # tokens of a pool block
LARGEST = {"int8": 127.0, "e4m3": 448.0}
LEAST = 2.0 ** -100  # of a scale


# ---------------------------------------------------------------- cases
# new, past: new rows of each sequence and rows it has before them.  "512*3" is 512 three times, "300~4096*31" 31
# numbers spread over that range.

def listed():
    return [
        # A decode step of 34 users on a small card: one row each, most into a block that holds rows already.
        dict(name="append 34 rows 8x128 int8", op="append", kind="int8", new="1*34", past="600~679*34", hkv=8, d=128),
        # A step that mixes three prompt chunks with 32 single rows.
        dict(name="append 3x512+32 8x128 e4m3", op="append", kind="e4m3", new="512*3+1*32", past="1024*3+300~4096*32",
             hkv=8, d=128),
        # Prompts of a multi-head shape admitted together, ragged.
        dict(name="append 16381 rows 40x128 int8", op="append", kind="int8", new="4099+37+8000+1+2500+1744",
             past="0*3+5+0+333", hkv=40, d=128),
        # One user's cache handed to other code.
        dict(name="read 640 rows 8x128 int8", op="read", kind="int8", new="640", past="0", hkv=8, d=128),
        # Long contexts of a multi-head shape, read back from the middle on.
        dict(name="read 30000 rows 40x128 e4m3", op="read", kind="e4m3", new="8191*3+5000+427", past="0+17*2+100+0",
             hkv=40, d=128),
        # Four short contexts, narrow heads, four q heads to a kv head: latency only.
        dict(name="decode 4 32/8x64 e4m3", op="decode", kind="e4m3", new="1*4", past="0+16+99+511", hq=32, hkv=8,
             d=64),
        # The 34 users whose contexts fill a small card.
        dict(name="decode 34x640 16/8x128 int8", op="decode", kind="int8", new="1*34", past="639*34", hq=16, hkv=8,
             d=128),
        # A multi-head shape, 64 ordinary contexts beside four long ones.
        dict(name="decode 68 40/40x128 int8", op="decode", kind="int8", new="1*68", past="127~2047*64+32767*4", hq=40,
             hkv=40, d=128),
        # Ragged contexts, eight q heads to a kv head.
        dict(name="decode 31 64/8x128 e4m3", op="decode", kind="e4m3", new="1*31", past="300~4096*31", hq=64, hkv=8,
             d=128),
        # One short prompt of a new request, narrow heads.
        dict(name="prefill 300 32/8x64 e4m3", op="prefill", kind="e4m3", new="300", past="0", hq=32, hkv=8, d=64),
        # The mixed step: three 512-token chunks of long prompts and 32 single-token rows.
        dict(name="prefill 3x512+32 16/8x128 int8", op="prefill", kind="int8", new="512*3+1*32",
             past="1024*3+300~4096*32", hq=16, hkv=8, d=128),
        # The last 2,048 tokens of a 16,384-token document.
        dict(name="prefill 2048 16/8x128 e4m3", op="prefill", kind="e4m3", new="2048", past="14336", hq=16, hkv=8,
             d=128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "prefill"])
    d = rng.choice([64, 128])
    kind = rng.choice(["int8", "e4m3"])
    g = rng.choice([1, 2, 4, 8])
    hkv = _spread(rng, 1, 40 // g)
    heads = dict(hq=hkv * g, hkv=hkv) if op in ("decode", "prefill") else dict(hkv=hkv)
    if op == "decode":
        n = _spread(rng, 1, 128)
        room = 200000 * 40 * 128 // (hkv * d) // n  # rows of a context, so that all stay below the largest case
        past = [min(room, _spread(rng, 1, 32768)) - 1 for _ in range(n)]
        new = [1] * n
    elif op == "prefill":
        new, past = [], []
        for _ in range(rng.choice([1, 2, 4, 7])):
            new.append(_spread(rng, 2, 2048))
            past.append(rng.choice([0, _spread(rng, 1, 14336)]))
        for _ in range(rng.choice([0, 0, 3, 17])):
            new.append(1)
            past.append(_spread(rng, 1, 4096))
        # the plain form pads every sequence to the longest
        while len(new) > 1 and len(new) * max(new) * max(map(sum, zip(new, past))) * hkv * g > 2 ** 29:
            at = max(range(len(new)), key=lambda i: new[i] * (new[i] + past[i]))
            del new[at], past[at]
        while max(new) * max(map(sum, zip(new, past))) * hkv * g > 2 ** 29:
            new, past = [max(1, x // 2) for x in new], [x // 2 for x in past]
    else:
        n = _spread(rng, 1, 128)
        total = _spread(rng, n, 16000)
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        new = [b - a for a, b in zip([0] + cuts, cuts + [total])]  # some without rows
        past = [rng.choice([0, _spread(rng, 1, 4096)]) for _ in range(n)]
    both = list(zip(new, past))
    rng.shuffle(both)
    return dict(op=op, kind=kind, new="+".join(str(x) for x, _ in both), past="+".join(str(x) for _, x in both),
                d=d, **heads)


def _numbers(text):
    got = []
    for part in text.split("+"):
        what, _, times = part.partition("*")
        lo, _, hi = what.partition("~")
        lo, hi, times = int(lo), int(hi or lo), int(times or 1)
        got += [lo + int((hi - lo) * (i * 0.6180339887 % 1.0)) for i in range(times)]
    return got


def _blocks(rows):
    return -(-rows // BLOCK)


def work(case):
    new, past = _numbers(case["new"]), _numbers(case["past"])
    hkv, d = case["hkv"], case["d"]
    t = sum(new)
    touched = sum(_blocks(n + p) - p // BLOCK for n, p in zip(new, past) if n)
    if case["op"] in ("append", "read"):
        # bf16 rows on one side, codes and scales on the other.  A full block's scale is only written, the codes of
        # rows that keep their scale are not touched.
        return {"bytes": t * hkv * d * 2 * 3 + touched * (8 * hkv + 4) + len(new) * 8, "flops": 4 * t * hkv * d}
    hq = case["hq"]
    blocks = sum(_blocks(n + p) for n, p in zip(new, past))
    keys = sum(n + p for n, p in zip(new, past))
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    moved = keys * hkv * d * 2 + blocks * (8 * hkv + 4) + t * hq * d * (2 + 4) + len(new) * 8
    return {"bytes": moved, "flops": pairs * hq * d * 4}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    hkv, d = case["hkv"], case["d"]
    new, past = _numbers(case["new"]), _numbers(case["past"])
    lens = [n + p for n, p in zip(new, past)]
    n, t = len(new), sum(new)
    used = [_blocks(x) for x in lens]
    # blocks scattered over a pool a fifth larger than what the sequences hold
    pool = sum(used) * 6 // 5 + 1
    ids = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    wide = max(used)
    tables = torch.zeros((n, wide), dtype=torch.int32, device=dev)
    inside = torch.arange(wide, device=dev) < torch.tensor(used, device=dev)[:, None]
    tables[inside] = ids[:sum(used)]
    s = dict(case=case, block_tables=tables, longest=max(lens), rows=t, most=max(new))
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    s["start_host"] = torch.tensor(starts, dtype=torch.int32)
    s["start"] = s["start_host"].to(dev)
    s["context_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    # codes as rows of a normal distribution leave them, scales that differ between blocks and heads
    largest = LARGEST[case["kind"]]
    for name in ("k_pool", "v_pool"):
        codes = normal(pool, hkv, BLOCK, d, dtype=torch.float32)
        codes.mul_(largest / 3.0).clamp_(-largest, largest)
        s[name] = codes.round_().to(torch.int8) if case["kind"] == "int8" else codes.to(torch.float8_e4m3fn)
        del codes
    s["block_scales"] = torch.exp(0.3 * normal(pool, hkv, 2, dtype=torch.float32)) * (2.5 / largest)
    if case["op"] == "append":
        qkv = normal(t, 3 * hkv, d)  # the projection's output: q, k and v side by side
        s.update(k=qkv[:, hkv:2 * hkv], v=qkv[:, 2 * hkv:])
        return s
    if case["op"] == "read":
        s["k_out"] = torch.empty((t, hkv, d), dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty((t, hkv, d), dtype=torch.bfloat16, device=dev)
        return s
    s["q"] = normal(t, case["hq"], d)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty((t, case["hq"], d), dtype=torch.float32, device=dev)
    if own:
        import paged_kv_cache_291_gb300 as pkv
        if case["op"] == "decode":
            need = pkv.decode_workspace_size(n, case["hq"], hkv, d, s["longest"])
        else:
            need = pkv.prefill_workspace_size(n, t, case["hq"], hkv, d, s["longest"])
        s["workspace"] = pkv.new_workspace(need, dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"append": _append, "read": _read, "decode": _decode, "prefill": _prefill}[s["case"]["op"]](s)


def _row_places(s):
    """Sequence and position of each new row."""
    row = torch.arange(s["rows"], device=s["start"].device)
    seq = torch.searchsorted(s["start"].long(), row, right=True) - 1
    return seq, s["context_lens"].long()[seq] - s["start"].long()[seq + 1] + row


def _codes(x, kind):
    """The codes nearest to x, ties to the even one."""
    if kind == "int8":
        return x.round().clamp(-127.0, 127.0).to(torch.int8)
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _append(s):
    kind, pools = s["case"]["kind"], (s["k_pool"], s["v_pool"])
    if own:
        import paged_kv_cache_291_gb300 as pkv
        pkv.cache_append(s["k_pool"], s["v_pool"], s["block_scales"], s["k"], s["v"], s["start"], s["context_lens"],
                         s["block_tables"])
        return s["k_pool"], s["v_pool"], s["block_scales"]
    seq, pos = _row_places(s)
    block = s["block_tables"].long()[seq, pos // BLOCK]
    touched, unit = torch.unique(block, return_inverse=True)
    dev = block.device
    first = torch.full(touched.shape, BLOCK, device=dev).scatter_reduce(0, unit, pos % BLOCK, "amin")
    kept = torch.arange(BLOCK, device=dev) < first[:, None]  # rows that were there
    hkv, d = s["k"].shape[1:]
    one = torch.ones((), device=dev)
    for which, x in enumerate((s["k"], s["v"])):
        rows = torch.zeros((touched.shape[0], BLOCK, hkv, d), device=dev)
        rows[unit, pos % BLOCK] = x.float()
        rows = rows.transpose(1, 2)
        old = torch.where(first[:, None] > 0, s["block_scales"][touched, :, which], 0.0)
        scale = torch.maximum(old, rows.abs().amax((2, 3)) * (one / LARGEST[kind])).clamp(min=LEAST)
        inv = one / scale
        before = pools[which][touched]
        again = _codes(before.float() * (old * inv)[..., None, None], kind)
        before = torch.where((scale > old)[..., None, None] & kept[:, None, :, None], again.view(torch.uint8),
                             before.view(torch.uint8)).view(again.dtype)
        pools[which][touched] = before
        s["block_scales"][touched, :, which] = scale
        pools[which].view(torch.uint8)[block, :, pos % BLOCK] = _codes(
            x.float() * inv[unit][..., None], kind).view(torch.uint8)
    return s["k_pool"], s["v_pool"], s["block_scales"]


def _read(s):
    if own:
        import paged_kv_cache_291_gb300 as pkv
        return pkv.cache_read(s["k_pool"], s["v_pool"], s["start"], s["context_lens"], s["block_tables"], s["rows"],
                              block_scales=s["block_scales"], k_out=s["k_out"], v_out=s["v_out"])
    seq, pos = _row_places(s)
    block = s["block_tables"].long()[seq, pos // BLOCK]
    scales = s["block_scales"][block][..., None]
    k = s["k_pool"].view(torch.uint8)[block, :, pos % BLOCK].view(s["k_pool"].dtype).float() * scales[:, :, 0]
    v = s["v_pool"].view(torch.uint8)[block, :, pos % BLOCK].view(s["v_pool"].dtype).float() * scales[:, :, 1]
    return k.bfloat16(), v.bfloat16()


def _blocks_of(s, blocks, which):
    """Pool blocks as 32-bit values [..., hkv, BLOCK, d]."""
    pool = s["v_pool"] if which else s["k_pool"]
    codes = pool.view(torch.uint8)[blocks].view(pool.dtype).float()
    return codes.mul_(s["block_scales"][blocks][..., which, None, None])


def _decode(s):
    n = s["q"].shape[0]
    if own:
        import paged_kv_cache_291_gb300 as pkv
        return pkv.decode_attention(s["k_pool"], s["v_pool"], s["q"], s["block_tables"], s["context_lens"],
                                    s["longest"], s["scale"], out=s["out"], workspace=s["workspace"],
                                    block_scales=s["block_scales"])
    # All sequences' blocks in one list, joined by the running maximum and sum of a softmax.
    hq, hkv, d = s["case"]["hq"], s["case"]["hkv"], s["case"]["d"]
    lens = s["context_lens"].long()
    seq, at = ((torch.arange(s["block_tables"].shape[1], device=lens.device) * BLOCK) < lens[:, None]).nonzero(
        as_tuple=True)
    blocks = s["block_tables"].long()[seq, at]
    q = s["q"].float().view(n, hkv, hq // hkv, d)[seq]
    score = torch.matmul(q, _blocks_of(s, blocks, 0).transpose(-1, -2)) * s["scale"]
    there = at[:, None] * BLOCK + torch.arange(BLOCK, device=lens.device) < lens[seq][:, None]
    score = torch.where(there[:, None, None], score, -math.inf)
    most = torch.full((n, hkv, hq // hkv), -math.inf, device=lens.device)
    most = most.scatter_reduce(0, seq[:, None, None].expand(-1, hkv, hq // hkv), score.amax(-1), "amax")
    weight = torch.exp(score - most[seq][..., None])
    total = torch.zeros(most.shape, dtype=torch.float64, device=lens.device)
    total.index_add_(0, seq, weight.double().sum(-1))
    out = torch.zeros((n, hkv, hq // hkv, d), dtype=torch.float64, device=lens.device)
    out.index_add_(0, seq, torch.matmul(weight, _blocks_of(s, blocks, 1)).double())
    return (out / total[..., None]).float().view(n, hq, d)


def _prefill(s):
    if own:
        import paged_kv_cache_291_gb300 as pkv
        return pkv.chunked_prefill_attention(s["k_pool"], s["v_pool"], s["q"], s["start"], s["context_lens"],
                                             s["block_tables"], s["longest"], s["scale"], out=s["out"],
                                             workspace=s["workspace"], query_start_loc_host=s["start_host"],
                                             block_scales=s["block_scales"])
    hq, hkv, d = s["case"]["hq"], s["case"]["hkv"], s["case"]["d"]
    n, dev = s["context_lens"].shape[0], s["q"].device
    # padded: q [n][hkv][group][most][d], keys and values [n][hkv][1][blocks * BLOCK][d]
    place = torch.arange(s["most"], device=dev)
    start, lens = s["start"].long(), s["context_lens"].long()
    rows = (start[:-1, None] + place).clamp(max=s["rows"] - 1)
    q = s["q"].float()[rows].view(n, s["most"], hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    key = torch.arange(s["block_tables"].shape[1] * BLOCK, device=dev)
    pos = (lens - (start[1:] - start[:-1]))[:, None] + place
    k = _blocks_of(s, s["block_tables"].long(), 0).transpose(1, 2).reshape(n, hkv, 1, -1, d)
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    score.masked_fill_((key > pos[..., None])[:, None, None], -math.inf)
    score -= score.amax(-1, keepdim=True)
    score.exp_()
    total = score.sum(-1, keepdim=True)
    v = _blocks_of(s, s["block_tables"].long(), 1).transpose(1, 2).reshape(n, hkv, 1, -1, d)
    v = torch.where((key < lens[:, None])[:, None, None, :, None], v, 0.0)
    out = (torch.matmul(score, v) / total).reshape(n, hq, s["most"], d)
    row = torch.arange(s["rows"], device=dev)
    seq = torch.searchsorted(start, row, right=True) - 1
    return out[seq, :, row - start[seq]]


# ---------------------------------------------------------------- from the definition, in 64 bits

def _values(pool):
    return pool.double() if pool.dtype == torch.int8 else pool.float().double()


def _nearest(y, kind):
    """The value of the code nearest to y (both in 64 bits), by the spacing of the codes around it."""
    if kind == "int8":
        return torch.round(y).clamp(-127, 127)
    place = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(place - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    hkv, d, kind = case["hkv"], case["d"], case["kind"]
    new, past = _numbers(case["new"]), _numbers(case["past"])
    tables = s["block_tables"].tolist()
    starts = s["start_host"].tolist()
    scales = s["block_scales"].double()
    if case["op"] == "append":
        # Block by block.  A scale is stored in 32 bits, and so is what a code is chosen from: both are rounded here.
        pools = [_values(s["k_pool"]), _values(s["v_pool"])]
        inv_largest = torch.tensor(1.0 / LARGEST[kind], dtype=torch.float32).double().item()
        for i, table in enumerate(tables):
            at, end, row = past[i], past[i] + new[i], starts[i]
            while at < end:
                b, r = table[at // BLOCK], at % BLOCK
                count = min(BLOCK - r, end - at)
                for which, x in enumerate((s["k"], s["v"])):
                    fresh = x[row:row + count].double().transpose(0, 1)
                    wanted = (fresh.abs().amax((1, 2)) * inv_largest).float().double().clamp(min=LEAST)
                    old = scales[b, :, which] if r else torch.zeros_like(wanted)
                    scale = torch.maximum(old, wanted)
                    inv = (1.0 / scale).float().double()
                    if r:
                        ratio = (old * inv).float().double()[:, None, None]
                        again = _nearest((pools[which][b, :, :r] * ratio).float().double(), kind)
                        grown = (scale > old)[:, None, None]
                        pools[which][b, :, :r] = torch.where(grown, again, pools[which][b, :, :r])
                    pools[which][b, :, r:r + count] = _nearest((fresh * inv[:, None, None]).float().double(), kind)
                    scales[b, :, which] = scale
                at, row = at + count, row + count
        return pools[0], pools[1], scales

    def rows_of(i, which, first):
        """Rows from `first` on of sequence i's context, [heads][rows][d]."""
        end = past[i] + new[i]
        ids = s["block_tables"][i, :_blocks(end)].long()
        pool = s["v_pool"] if which else s["k_pool"]
        held = pool.view(torch.uint8)[ids].view(pool.dtype)
        held = _values(held) * scales[ids, :, which][..., None, None]
        return held.transpose(0, 1).reshape(hkv, -1, d)[:, first:end]

    if case["op"] == "read":
        return tuple(torch.cat([rows_of(i, which, past[i]).transpose(0, 1) for i in range(len(new))])
                     for which in (0, 1))
    hq = case["hq"]
    out = torch.empty((s["rows"], hq, d), dtype=torch.float64, device=s["q"].device)
    for i in range(len(new)):
        if not new[i]:
            continue
        q = s["q"][starts[i]:starts[i + 1]].double()
        k, v = rows_of(i, 0, 0), rows_of(i, 1, 0)
        later = torch.ones((new[i], past[i] + new[i]), dtype=torch.bool, device=q.device).triu(past[i] + 1)
        for h in range(hq):
            score = (q[:, h] @ k[h * hkv // hq].t() * s["scale"]).masked_fill(later, -math.inf)
            out[starts[i]:starts[i + 1], h] = torch.softmax(score, -1) @ v[h * hkv // hq]
    return out
