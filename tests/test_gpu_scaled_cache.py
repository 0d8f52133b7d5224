"""GPU parity of pkv_cache_append, pkv_cache_read and the block moves of 8-bit
pools with a scale per block and head.  Codes and scales are bit-exact: the
definition rounds each fp32 operation once.  Rows read back are the bf16
nearest to the fp32 product, bit-exact too."""
import numpy as np
import pytest
import torch

from oracle import scaled as S
from scaled_batch import Batch, bf16_rows, to_dev, to_host

pytestmark = pytest.mark.gpu

KINDS = [np.int8, np.uint8]


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_291_gb300 as p
    p.load()
    p.get_error()
    return p


def append_and_check(pkv, b, kn, vn, kt, vt, **kw):
    k, v, sc, start, lens, tables = b.dev()
    pkv.cache_append(k, v, sc, kt, vt, start, lens, tables, **kw)
    torch.cuda.synchronize()
    S.append(b.k, b.v, b.scales, kn, vn, b.start, b.lens, b.tables)
    assert np.array_equal(sc.cpu().numpy(), b.scales, equal_nan=True)
    assert np.array_equal(to_host(k), b.k) and np.array_equal(to_host(v), b.v)


BATCHES = [
    ([1], [0]), ([1], [1]), ([1], [15]), ([1], [16]), ([16], [0]), ([17], [0]), ([3], [14]), ([100], [7]),
    ([1] * 34, list(range(600, 634))), ([0, 5, 0, 33, 1, 0], [3, 0, 0, 15, 31, 16]),
    ([1, 40, 0, 2, 129, 1, 1, 16], [0, 3, 9, 15, 0, 300, 17, 32]), ([1] * 70 + [50] * 3, [5] * 73),
    ([2] * 1100, [i % 37 for i in range(1100)]),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,past", BATCHES)
def test_append(pkv, kind, new, past):
    hkv, d = (3, 128) if len(new) % 2 else (8, 64)
    b = Batch(len(new) + new[0], kind, new, past, hkv, d, empty=True)
    rng = np.random.default_rng(7)
    kn, kt = bf16_rows(rng, b.T, hkv, d)
    vn, vt = bf16_rows(rng, b.T, hkv, d, size=30.0)
    append_and_check(pkv, b, kn, vn, kt, vt)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,d", [(1, 64), (1, 128), (5, 128), (13, 64), (40, 128)])
def test_append_packed_projection(pkv, kind, hkv, d):
    """k and v are views of one projection; rows behind the last sequence stay out."""
    b = Batch(hkv, kind, [4, 30, 1], [0, 9, 47], hkv, d, empty=True)
    x, t = bf16_rows(np.random.default_rng(8), b.T + 5, 4 * hkv, d)
    cut = slice(hkv, 2 * hkv), slice(2 * hkv, 3 * hkv)
    append_and_check(pkv, b, x[:, cut[0]], x[:, cut[1]], t[:, cut[0]], t[:, cut[1]])
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_append_step_by_step(pkv, kind):
    """40 decode steps with growing rows: the block's scale grows time after time."""
    rng = np.random.default_rng(9)
    b = Batch(3, kind, [40, 40], [0, 11], 2, 64, empty=True)
    k, v, sc, _, _, tables = b.dev()
    starts = np.array([0, 1, 2], np.int32)
    for i in range(40):
        lens = np.array([i + 1, 11 + i + 1], np.int32)
        kn, kt = bf16_rows(rng, 2, 2, 64, size=1.2 ** (i % 16))
        vn, vt = bf16_rows(rng, 2, 2, 64, size=0.8 ** i)
        pkv.cache_append(k, v, sc, kt, vt, torch.from_numpy(starts).cuda(), torch.from_numpy(lens).cuda(), tables)
        S.append(b.k, b.v, b.scales, kn, vn, starts, lens, b.tables)
    assert np.array_equal(sc.cpu().numpy(), b.scales, equal_nan=True)
    assert np.array_equal(to_host(k), b.k) and np.array_equal(to_host(v), b.v)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [0.0, 1e-37, 2.0 ** -101, 1e-20, 1e30, 3e38])
def test_append_extreme_sizes(pkv, kind, size):
    b = Batch(4, kind, [20, 1], [0, 20], 2, 64, empty=True)
    x = np.clip(np.random.default_rng(10).standard_normal((21, 2, 64)) / 3, -1, 1) * size
    x = S.bf16_values(S.to_bf16_bits(x.astype(np.float32)))
    t = torch.from_numpy(x).bfloat16().cuda()
    append_and_check(pkv, b, x, -x, t, -t)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_append_values_that_are_not_finite(pkv, kind):
    b = Batch(5, kind, [18, 3], [0, 30], 2, 64, empty=True)
    x, _ = bf16_rows(np.random.default_rng(11), b.T, 2, 64)
    x[3, 0, 5], x[3, 1, 9], x[17, 0, 1], x[19, 1, 63] = np.inf, -np.inf, np.nan, np.nan
    x[16:18, 1] = np.inf  # nothing finite in that block and head
    t = torch.from_numpy(x).bfloat16().cuda()
    append_and_check(pkv, b, x, x, t, t)
    err, detail = pkv.get_error()
    assert err == 9 and detail in (0, 1)


@pytest.mark.parametrize("kind", KINDS)
def test_append_infinities_under_a_large_scale(pkv, kind):
    """An infinity is the largest code even where the block's scale passes the largest bf16 by far."""
    b = Batch(8, kind, [2, 1], [5, 0], 2, 64, empty=True)
    b.scales[b.tables[0, 0]] = 2.0 ** 122
    x, _ = bf16_rows(np.random.default_rng(14), 3, 2, 64)
    x[0, 0, 3], x[1, 1, 60], x[2, 1, 7] = np.inf, -np.inf, np.inf
    t = torch.from_numpy(x).bfloat16().cuda()
    append_and_check(pkv, b, x, -x, t, -t)
    assert pkv.get_error()[0] == 9


@pytest.mark.parametrize("kind", KINDS)
def test_append_products_next_to_ties(pkv, kind):
    """Codes of x (1 / scale) as fp32 rounds that product, over many scales."""
    b = Batch(9, kind, [1600], [0], 4, 128, empty=True)
    rng = np.random.default_rng(15)
    kn, kt = bf16_rows(rng, 1600, 4, 128, size=1.0 + np.arange(1600)[:, None, None] / 16)
    vn, vt = bf16_rows(rng, 1600, 4, 128)
    append_and_check(pkv, b, kn, vn, kt, vt)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_append_bad_sequences(pkv, kind):
    """Sequences and blocks out of range store nothing and are reported; the others are stored."""
    for spoil, detail in ((lambda b: b.lens.__setitem__(1, 2), 1), (lambda b: b.lens.__setitem__(1, 16 * 9 + 1), 1),
                          (lambda b: b.lens.__setitem__(0, -5), 0), (lambda b: b.tables.__setitem__((2, 0), b.nb), 2),
                          (lambda b: b.tables.__setitem__((2, 0), -1), 2),
                          (lambda b: b.start.__setitem__(3, b.T + 1), 2)):
        b = Batch(6, kind, [3, 7, 5], [0, 20, 2], 2, 64, empty=True)
        kn, kt = bf16_rows(np.random.default_rng(12), b.T, 2, 64)
        spoil(b)
        append_and_check(pkv, b, kn, kn, kt, kt)
        assert pkv.get_error() == (9, detail)


@pytest.mark.parametrize("kind", KINDS)
def test_append_a_bad_scale_of_earlier_rows(pkv, kind):
    b = Batch(7, kind, [1, 1], [5, 5], 1, 64, empty=True)
    b.scales[b.tables[1, 0], 0, 1] = np.inf
    kn, kt = bf16_rows(np.random.default_rng(13), 2, 1, 64)
    append_and_check(pkv, b, kn, kn, kt, kt)
    assert pkv.get_error() == (9, 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,past", BATCHES)
def test_read(pkv, kind, new, past):
    hkv, d = (8, 64) if len(new) % 2 else (3, 128)
    b = Batch(len(new) + past[0], kind, new, past, hkv, d)
    k, v, sc, start, lens, tables = b.dev()
    gk, gv = pkv.cache_read(k, v, start, lens, tables, b.T, block_scales=sc)
    wk, wv = S.read(b.k, b.v, b.scales, b.start, b.lens, b.tables, b.T)
    for got, want in ((gk, wk), (gv, wv)):
        assert np.array_equal(got.view(torch.int16).cpu().numpy().view(np.uint16), S.to_bf16_bits(want))
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("d", [64, 128])
def test_read_pools_without_block_scales(pkv, d):
    b = Batch(20, np.uint8, [33, 4], [0, 50], 3, d)
    k, v, sc, start, lens, tables = b.dev()
    gk, gv = pkv.cache_read(k, v, start, lens, tables, b.T, k_scale=0.37, v_scale=2.5)
    for scale, got, pool in ((0.37, gk, b.k), (2.5, gv, b.v)):
        want = S.read(pool, pool, np.full_like(b.scales, scale), b.start, b.lens, b.tables, b.T)[0]
        assert np.array_equal(got.view(torch.int16).cpu().numpy().view(np.uint16), S.to_bf16_bits(want))
    bits = np.random.default_rng(1).integers(0, 65536, (2,) + b.k.shape, dtype=np.uint16)  # every bf16 pattern
    pools = [torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16) for x in bits]
    gk, gv = pkv.cache_read(*pools, start, lens, tables, b.T)
    for got, x in ((gk, bits[0]), (gv, bits[1])):
        want = np.concatenate([x[b.tables[s][np.arange(b.past[s], b.lens[s]) // 16], :,
                                 np.arange(b.past[s], b.lens[s]) % 16] for s in range(2)])
        assert np.array_equal(got.view(torch.int16).cpu().numpy().view(np.uint16), want)
    assert pkv.get_error()[0] == 0


def test_read_bad_sequences(pkv):
    b = Batch(21, np.int8, [3, 20, 18], [0, 20, 2], 2, 64)
    b.lens[1] = 19                      # shorter than its rows
    b.tables[2, 1] = b.nb + 5           # rows 16.. of its context
    b.scales[b.tables[0, 0], 1, 0] = 0  # counts as 2^-100
    k, v, sc, start, lens, tables = b.dev()
    out = [torch.full((b.T + 2, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gk, gv = pkv.cache_read(k, v, start, lens, tables, b.T + 2, block_scales=sc, k_out=out[0], v_out=out[1])
    assert gk is out[0] and gv is out[1] and pkv.get_error()[0] == 9
    wk, wv = S.read(b.k, b.v, b.scales, b.start, b.lens, b.tables, b.T)
    for got, want in ((gk, wk), (gv, wv)):
        got = got.float().cpu().numpy()
        assert np.all(got[b.T:] == 7.0)
        assert np.array_equal(got[:b.T], S.bf16_values(S.to_bf16_bits(np.nan_to_num(want))))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_copy_and_swap_take_the_scales_along(pkv, kind, hkv):
    b = Batch(22, kind, [64, 64], [0, 0], hkv, 64)
    k, v, sc, *_ = b.dev()
    held = [int(x) for x in b.tables.reshape(-1)[:8]]
    free = [x for x in range(b.nb) if x not in held]
    pkv.copy_blocks(k, v, torch.tensor([held[1], -1, held[4]], dtype=torch.int32, device="cuda"),
                    torch.tensor([free[0], 0, free[2]], dtype=torch.int32, device="cuda"), block_scales=sc)
    slab = 2 * hkv * 16 * 64 + (8 * hkv + 15) // 16 * 16
    host = torch.zeros((4, slab), dtype=torch.uint8).pin_memory()
    blocks = torch.tensor([held[2], -1, held[7]], dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 1, 0], dtype=torch.int32, device="cuda")
    pkv.swap_out(k, v, blocks, slots, host, block_scales=sc)
    back = torch.tensor([held[0], free[1]], dtype=torch.int32, device="cuda")
    pkv.swap_in(k, v, back, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), host, block_scales=sc)
    torch.cuda.synchronize()
    for to, frm in ((free[0], held[1]), (free[2], held[4])):
        b.k[to], b.v[to], b.scales[to] = b.k[frm], b.v[frm], b.scales[frm]
    first, last = [(x[held[2]].copy(), x[held[7]].copy()) for x in (b.k, b.v, b.scales)], (held[0], free[1])
    for pool, (h2, h7) in zip((b.k, b.v, b.scales), first):
        pool[last[0]], pool[last[1]] = h7, h2
    assert np.array_equal(to_host(k), b.k) and np.array_equal(to_host(v), b.v)
    assert np.array_equal(sc.cpu().numpy(), b.scales, equal_nan=True)
    assert not host[1].any() and not host[2].any() and pkv.get_error()[0] == 0


def test_refusals_of_the_binding(pkv):
    b = Batch(23, np.int8, [4], [0], 2, 64)
    k, v, sc, start, lens, tables = b.dev()
    new = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    args = dict(k_pool=k, v_pool=v, block_scales=sc, k_new=new, v_new=new, query_start_loc=start, context_lens=lens,
                block_tables=tables)
    for bad in (dict(block_scales=None), dict(block_scales=sc[:-1]), dict(block_scales=sc.half()),
                dict(k_new=new.half()), dict(k_new=new[:3]), dict(v_new=new[:, :1]), dict(k_new=new.transpose(0, 1)),
                dict(context_lens=lens.long()), dict(query_start_loc=start[:1]), dict(block_tables=tables[0]),
                dict(v_pool=v.view(torch.uint8)), dict(k_pool=k.float(), v_pool=v.float()), dict(k_new=new.cpu()),
                dict(k_pool=k.view(torch.bfloat16), v_pool=v.view(torch.bfloat16)),
                dict(k_pool=k[:, :, :, ::2], v_pool=v[:, :, :, ::2])):
        with pytest.raises((TypeError, ValueError, AttributeError)):
            pkv.cache_append(**(args | bad))
    with pytest.raises(ValueError):
        pkv.cache_read(k, v, start, lens, tables, 4, k_scale=1.0, v_scale=1.0, block_scales=sc)
    with pytest.raises(ValueError):
        pkv.cache_read(to_dev(b.k.view(np.uint8)), to_dev(b.v.view(np.uint8)), start, lens, tables, 4)
    with pytest.raises(TypeError):
        pkv.cache_read(to_dev(b.k.view(np.int8)), to_dev(b.v.view(np.int8)), start, lens, tables, 4, k_scale=1.0,
                       v_scale=1.0)
    assert pkv.get_error()[0] == 0


def test_append_and_read_in_a_graph_and_on_another_stream(pkv):
    rng = np.random.default_rng(14)
    b = Batch(24, np.uint8, [5, 1], [0, 40], 2, 128, empty=True)
    k, v, sc, start, lens, tables = b.dev()
    kn, kt = bf16_rows(rng, b.T, 2, 128)
    vn, vt = bf16_rows(rng, b.T, 2, 128)
    out = [torch.empty((b.T, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        pkv.cache_append(k, v, sc, kt, vt, start, lens, tables)
        pkv.cache_read(k, v, start, lens, tables, b.T, k_out=out[0], v_out=out[1], block_scales=sc)
    for size in (1.0, 4.0):  # other rows in the same buffers
        kt.copy_(torch.from_numpy(size * kn))
        vt.copy_(torch.from_numpy(size * vn))
        graph.replay()
        S.append(b.k, b.v, b.scales, size * kn, size * vn, b.start, b.lens, b.tables)
        torch.cuda.synchronize()
        assert np.array_equal(to_host(k), b.k) and np.array_equal(to_host(v), b.v)
        want = S.read(b.k, b.v, b.scales, b.start, b.lens, b.tables, b.T)
        for got, w in zip(out, want):
            assert np.array_equal(got.view(torch.int16).cpu().numpy().view(np.uint16), S.to_bf16_bits(w))
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.stream(side):
        pkv.cache_append(k, v, sc, kt, vt, start, lens, tables)
    a, c = pkv.cache_read(k, v, start, lens, tables, b.T, block_scales=sc, stream=side)
    side.synchronize()
    assert torch.equal(a, out[0]) and torch.equal(c, out[1]) and pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_offsets_past_32_bits(pkv, kind):
    """Pools of 4.3 GB: blocks whose bytes lie beyond 2^32."""
    hkv, d, nb = 40, 128, 2 ** 32 // (40 * 16 * 128) + 64
    k = torch.zeros((nb, hkv, 16, d), dtype=torch.int8 if kind == np.int8 else torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    sc = torch.ones((nb, hkv, 2), dtype=torch.float32, device="cuda")
    rng = np.random.default_rng(15)
    tables = np.array([[nb - 1, 5, nb - 30]], np.int32)
    kn, kt = bf16_rows(rng, 40, hkv, d)
    vn, vt = bf16_rows(rng, 40, hkv, d)
    start, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 40], [40]))
    t = torch.from_numpy(tables).cuda()
    pkv.cache_append(k, v, sc, kt, vt, start, lens, t)
    gk, gv = pkv.cache_read(k, v, start, lens, t, 40, block_scales=sc)
    small = [np.zeros((3, hkv, 16, d), kind), np.zeros((3, hkv, 16, d), kind), np.ones((3, hkv, 2), np.float32)]
    S.append(*small, kn, vn, [0, 40], [40], [[0, 1, 2]])
    at = torch.from_numpy(tables[0].astype(np.int64)).cuda()
    assert np.array_equal(k[at].cpu().numpy(), small[0]) and np.array_equal(v[at].cpu().numpy(), small[1])
    assert np.array_equal(sc[at].cpu().numpy(), small[2])
    want = S.read(*small, [0, 40], [40], [[0, 1, 2]], 40)
    for got, w in zip((gk, gv), want):
        assert np.array_equal(got.view(torch.int16).cpu().numpy().view(np.uint16), S.to_bf16_bits(w))
    assert int(k[6:nb - 30].count_nonzero()) == 0 and pkv.get_error()[0] == 0
