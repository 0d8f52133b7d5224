"""GPU parity of decode and chunked prefill over 8-bit pools with a scale per
block and head, against the float64 oracle; the tolerance is derived in
scaled_batch.attention_tolerance."""
import numpy as np
import pytest
import torch

from oracle import scaled as S
from scaled_batch import NAN_CODE, Batch, attention_tolerance, bf16_rows, to_dev

pytestmark = pytest.mark.gpu

KINDS = [np.int8, np.uint8]


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_291_gb300 as p
    p.load()
    p.get_error()
    return p


def check(b, got, q, scale):
    exact = S.attention(b.k, b.v, b.scales, q, b.start, b.lens, b.tables, scale)
    held = np.concatenate([b.tables[s, :-(-int(n) // 16)] for s, n in enumerate(b.lens)]).astype(int)
    tol = attention_tolerance(exact, int(b.lens.max()), b.scales[held])
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    over = np.abs(got - exact[0]) / np.maximum(tol, 1e-300)
    assert over.max() <= 1, f"{over.max():.3g} of the tolerance at {np.unravel_index(over.argmax(), over.shape)}"


def decode(pkv, b, q, scale, **kw):
    k, v, sc, _, lens, tables = b.dev()
    return pkv.decode_attention(k, v, q, tables, lens, int(b.lens.max()), scale, block_scales=sc, **kw)


def prefill(pkv, b, q, scale, **kw):
    k, v, sc, start, lens, tables = b.dev()
    return pkv.chunked_prefill_attention(k, v, q, start, lens, tables, int(b.lens.max()), scale,
                                         query_start_loc_host=b.start, block_scales=sc, **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,hkv", [(1, 1), (1, 5), (2, 3), (4, 2), (8, 1), (8, 3)])
def test_decode_head_shapes(pkv, kind, d, g, hkv):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 47, 64, 100, 129, 300, 0, 511, 640]
    b = Batch(g * 10 + hkv, kind, [1] * len(lens), [n - 1 for n in lens], hkv, d)
    q, qt = bf16_rows(b.rng, b.T, g * hkv, d)
    check(b, decode(pkv, b, qt, d ** -0.5), q, d ** -0.5)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("part", [0, 1, 2, 3, 7, 50])
def test_decode_split_contexts(pkv, kind, part):
    b = Batch(part, kind, [1] * 5, [2999, 0, 700, 33, 1], 2, 128)
    q, qt = bf16_rows(b.rng, b.T, 4, 128)
    first = decode(pkv, b, qt, 0.1, partition_blocks=part)
    check(b, first, q, 0.1)
    assert torch.equal(first, decode(pkv, b, qt, 0.1, partition_blocks=part))
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_decode_many_sequences(pkv, kind):
    lens = [(i * 37) % 211 for i in range(700)]
    b = Batch(1, kind, [1] * 700, [n - 1 for n in lens], 1, 64)
    q, qt = bf16_rows(b.rng, b.T, 2, 64)
    check(b, decode(pkv, b, qt, 0.125), q, 0.125)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size,spread,scale", [(1.0, 4.0, 0.05), (2.0 ** -90, 0.5, 1.0), (1e30, 0.5, 1e-31), (1.0, 0.5, 3.0)])
def test_scales_far_apart(pkv, kind, size, spread, scale):
    """Blocks whose scales differ by factors of hundreds, tiny and huge caches, weights on single keys."""
    b = Batch(2, kind, [1, 70, 1], [300, 40, 16], 2, 128, size=size, spread=spread)
    q, qt = bf16_rows(b.rng, b.T, 4, 128)
    check(b, prefill(pkv, b, qt, scale), q, scale)
    one = Batch(3, kind, [1] * 4, [100, 0, 31, 600], 2, 64, size=size, spread=spread)
    q, qt = bf16_rows(one.rng, one.T, 4, 64)
    check(one, decode(pkv, one, qt, scale), q, scale)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_blocks_of_zeros(pkv, kind):
    """Appended zeros have the least scale; a context of zeros gives zeros."""
    b = Batch(4, kind, [1, 40], [40, 8], 2, 64)
    for s in range(2):
        blocks = b.tables[s, :2] if s else b.tables[s, :3]
        b.k[blocks[0]], b.v[blocks[0]], b.scales[blocks[0]] = 0, 0, 2.0 ** -100
        if not s:
            b.v[blocks], b.scales[blocks, :, 1] = 0, 2.0 ** -100
    q, qt = bf16_rows(b.rng, b.T, 4, 64)
    got = prefill(pkv, b, qt, 0.125)
    check(b, got, q, 0.125)
    assert not got[0].any() and pkv.get_error()[0] == 0


PREFILLS = [
    ([2], [0]), ([3], [14]), ([16], [0]), ([17], [16]), ([127], [1]), ([128], [0]), ([129], [0]), ([130], [250]),
    ([300], [0]), ([5, 1, 64, 0, 1, 200], [0, 30, 64, 7, 0, 513]), ([140, 2, 1, 260], [900, 0, 128, 3]),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,g,hkv", [(64, 1, 2), (64, 4, 1), (128, 1, 1), (128, 2, 2), (128, 8, 1)])
@pytest.mark.parametrize("new,past", PREFILLS)
def test_prefill(pkv, kind, d, g, hkv, new, past):
    b = Batch(sum(new) + d + g, kind, new, past, hkv, d)
    q, qt = bf16_rows(b.rng, b.T, g * hkv, d)
    check(b, prefill(pkv, b, qt, d ** -0.5), q, d ** -0.5)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_a_large_weight_far_back(pkv, kind):
    """The running maximum moves late and early; a NaN code behind the context stays out."""
    for place in (0, 200, 399):
        b = Batch(place, kind, [150, 1], [250, 399], 1, 128, spread=0.1)
        q = np.zeros((151, 2, 128), np.float32)
        q[...] = S.bf16_values(S.to_bf16_bits(b.rng.standard_normal((151, 2, 128)).astype(np.float32)))
        for s in range(2):
            block = b.tables[s, place // 16]
            b.k[block, 0, place % 16] = S.encode((40 * np.sign(q[-1, 0])).astype(np.float32), b.k)
        qt = torch.from_numpy(q).bfloat16().cuda()
        check(b, prefill(pkv, b, qt, 0.3), q, 0.3)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (-0.1, 1.0), (0.1, 2.0 ** -120), (2.0 ** -100, 2.0 ** -100), (-0.0, 1.0)])
def test_factors_of_any_sign_and_size(pkv, kind, d, scale, size):
    """Weights that are all equal, a negative scale, q rows that vanish: what is masked stays out."""
    b = Batch(8, kind, [70, 1, 1], [35, 0, 400], 2, d)
    q, qt = bf16_rows(b.rng, b.T, 4, d, size=size)
    check(b, prefill(pkv, b, qt, scale), q, scale)
    one = Batch(9, kind, [1] * 5, [5, 0, 33, 700, 47], 2, d)
    q, qt = bf16_rows(one.rng, one.T, 4, d, size=size)
    check(one, decode(pkv, one, qt, scale), q, scale)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_a_scale_or_rows_of_nan(pkv, kind):
    """NaN in every row that it reaches, and in no other."""
    b = Batch(11, kind, [150, 1], [10, 400], 2, 64)
    q, qt = bf16_rows(b.rng, b.T, 4, 64)
    assert prefill(pkv, b, qt, float("nan")).isnan().all()
    for spoil in (float("nan"), float("inf")):
        qn = qt.clone()
        qn[70, 1, 5] = qn[150, 3, 60] = spoil
        got = prefill(pkv, b, qn, 0.1)
        nan = torch.zeros_like(got, dtype=torch.bool)
        nan[70, 1] = nan[150, 3] = True
        assert torch.equal(got.isnan(), nan)
    one = Batch(12, kind, [1] * 2, [30, 500], 2, 64)
    q, qt = bf16_rows(one.rng, 2, 4, 64)
    assert decode(pkv, one, qt, float("nan")).isnan().all()
    qt[1, 2, 7] = float("nan")
    got = decode(pkv, one, qt, 0.1).isnan()
    assert got[1, 2].all() and int(got.sum()) == 64
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [8, 13, 14, 15, 16, 17, 18, 20, 24, 40, 100])
def test_scores_of_any_size(pkv, kind, sign, power):
    """One key far above the rest (scores of 40 and 96, or -96 and -40, times 2^power): its V row comes out.

    The others' weights are at most e^(-56 * 2^8) = 0 of it; its own weight
    cancels but for its two fp16 terms (2^-22), the products and sums with
    others' zeros lose nothing, and the quotient's roundings (V's scale, its
    reciprocal and log2, sum, inverse, product) are below 2^-20."""
    high, low = (96, 40) if sign > 0 else (40, 96)
    for place in (0, 150, 329):
        b = Batch(place, kind, [40, 1], [290, 329], 1, 128, spread=0.5)
        b.scales[..., 0] = 1
        for s in range(2):
            for j in range(330):
                b.k[b.tables[s, j // 16], 0, j % 16] = 0
                row = np.array([high if j == place else low], np.float32)
                b.k[b.tables[s, j // 16], 0, j % 16, :1] = S.encode(row, b.k)
        q = np.zeros((41, 2, 128), np.float32)
        q[..., 0] = sign * 2.0 ** power
        block = b.tables[:, place // 16]
        rows = S.values(b.v[block, 0, place % 16]).astype(np.float64) * b.scales[block, 0, 1:].astype(np.float64)
        sees = np.array([[j >= place] for j in range(290, 330)])
        got = prefill(pkv, b, torch.from_numpy(q).bfloat16().cuda(), 1.0).double().cpu().numpy()
        for s, part in enumerate((got[:40], got[40:])):
            want = np.broadcast_to(rows[s], part.shape)
            ok = np.abs(part - want) <= 2.0 ** -19 * np.abs(want)
            if s == 0:
                ok |= ~sees[..., None]
            assert ok.all()
        k, v, sc, _, lens, tables = b.dev()
        one = torch.from_numpy(q[:2]).bfloat16().cuda()
        got = pkv.decode_attention(k, v, one, tables, lens, 330, 1.0, block_scales=sc).double().cpu().numpy()
        want = np.broadcast_to(rows[:, None], got.shape)
        assert np.all(np.abs(got - want) <= 2.0 ** -19 * np.abs(want))
    assert pkv.get_error()[0] == 0


def test_e4m3_nan_codes_inside_a_context(pkv):
    """A NaN code in K or V of a visible row reaches the heads that read it, and no others."""
    for which in (0, 1):
        b = Batch(30, np.uint8, [20, 1, 1], [30, 60, 60], 2, 64)
        for s in (0, 1):
            (b.v if which else b.k)[b.tables[s, 2], 1, 3, 5] = NAN_CODE[np.uint8]  # position 35
        q, qt = bf16_rows(b.rng, b.T, 4, 64)
        got = prefill(pkv, b, qt, 0.125).cpu().numpy()
        nan = np.isnan(got)
        seen = np.zeros(got.shape, bool)
        seen[5:21, 2:] = True  # rows at positions 35.. of sequence 0, and sequence 1's row
        if which:
            seen[..., :5] = seen[..., 6:] = False
        assert np.array_equal(nan, seen)
    assert pkv.get_error()[0] == 0


def test_bad_arguments_found_on_the_device(pkv):
    """A scale out of range counts as 2^-100, a block id out of range as block 0, a long context as the longest."""
    for spoil in (lambda b: b.scales.__setitem__((b.tables[1, 0], 0, 0), -1.0),
                  lambda b: b.scales.__setitem__((b.tables[1, 1], 0, 1), np.nan)):
        b = Batch(31, np.int8, [1, 30, 1], [5, 9, 50], 1, 64)
        spoil(b)
        q, qt = bf16_rows(b.rng, b.T, 2, 64)
        check(b, prefill(pkv, b, qt, 0.125), q, 0.125)
        assert pkv.get_error() == (9, 1)
    b = Batch(32, np.int8, [1, 30, 1], [5, 9, 50], 1, 64)
    b.scales[0] = 1.0
    b.k[0], b.v[0] = 3, 3
    b.tables[2, 1] = b.nb
    q, qt = bf16_rows(b.rng, b.T, 2, 64)
    got = prefill(pkv, b, qt, 0.125)
    assert pkv.get_error() == (9, 2)
    b.tables[2, 1] = 0
    check(b, got, q, 0.125)
    k, v, sc, start, lens, tables = b.dev()
    lens[0] = 10 ** 9
    got = pkv.decode_attention(k, v, qt[:3], tables, lens, int(b.lens.max()), 0.125, block_scales=sc)
    assert pkv.get_error()[0] == 9 and got.shape == (3, 2, 64)
    lens[1] = 12  # shorter than its rows: zero rows
    lens[0] = 6
    got = pkv.chunked_prefill_attention(k, v, qt, start, lens, tables, int(b.lens.max()), 0.125,
                                        query_start_loc_host=b.start, block_scales=sc)
    assert pkv.get_error() == (9, 1) and not got[1:31].any() and got[0].any() and got[31].any()


@pytest.mark.parametrize("kind", KINDS)
def test_other_entry_points(pkv, kind):
    """Shared blocks are attended per sequence; the call without a workspace; out in page-locked memory."""
    b = Batch(33, kind, [1] * 3, [95, 110, 64], 2, 128)
    b.tables[1:, :4] = b.tables[0, :4]
    q, qt = bf16_rows(b.rng, b.T, 4, 128)
    want = decode(pkv, b, qt, 0.1)
    check(b, want, q, 0.1)
    k, v, sc, start, lens, tables = b.dev()
    got = pkv.decode_attention_shared_prefix(k, v, qt, tables, lens, int(b.lens.max()), 4, 0.1, block_scales=sc)
    assert torch.equal(got, want)
    host = torch.empty(want.shape).pin_memory()
    decode(pkv, b, qt, 0.1, out=host)
    torch.cuda.synchronize()
    assert torch.equal(host, want.cpu())
    import ctypes
    c = pkv._cache(k, v, block_scales=sc)
    out = torch.empty_like(want)
    P = ctypes.c_void_p
    st = pkv.load().pkv_decode_attention_static(
        ctypes.byref(c), P(qt.data_ptr()), 4, P(tables.data_ptr()), tables.shape[1], P(lens.data_ptr()), 3,
        int(b.lens.max()), ctypes.c_float(0.1), P(out.data_ptr()), P(torch.cuda.current_stream().cuda_stream))
    assert st == 0 and torch.equal(out, want) and pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_graphs_that_share_a_workspace(pkv, kind):
    """Two captured batches on one workspace, replayed in turn, with other queries and lengths in their buffers."""
    many = Batch(34, kind, [1] * 6, [500, 3, 90, 0, 16, 250], 2, 64)
    mixed = Batch(35, kind, [1, 130, 1], [700, 40, 15], 2, 64)
    ws = pkv.new_workspace(max(pkv.decode_workspace_size(6, 4, 2, 64, 501),
                               pkv.prefill_workspace_size(3, 132, 4, 2, 64, 701)))
    todo = []
    for b, mixed_batch in ((many, False), (mixed, True)):
        k, v, sc, start, lens, tables = b.dev()
        q, qt = bf16_rows(b.rng, b.T, 4, 64)
        out = torch.empty((b.T, 4, 64), device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if mixed_batch:
                pkv.chunked_prefill_attention(k, v, qt, start, lens, tables, int(b.lens.max()), 0.125, out=out,
                                              workspace=ws, query_start_loc_host=b.start, block_scales=sc)
            else:
                pkv.decode_attention(k, v, qt, tables, lens, int(b.lens.max()), 0.125, out=out, workspace=ws,
                                     block_scales=sc)
        todo.append((b, graph, q, qt, out, lens, (k, v, sc, start, tables)))
    for turn in range(3):
        for b, graph, q, qt, out, lens, _ in todo:
            q = S.bf16_values(S.to_bf16_bits(b.rng.standard_normal(q.shape).astype(np.float32)))
            qt.copy_(torch.from_numpy(q))
            if turn == 2:
                b.lens[0] -= 37
                lens.copy_(torch.from_numpy(b.lens))
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            check(b, out, q, 0.125)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_a_serving_loop(pkv, kind, d):
    """Blocks handed out on the device, a prompt in chunks, a fork with copy-on-write, decode steps: append and
    attention over what it left, against the oracle over the oracle's own pools."""
    rng = np.random.default_rng(36)
    hkv, hq, nb = 2, 4, 24
    blocks = pkv.Blocks(nb, 4, 8)
    host = [np.zeros((nb, hkv, 16, d), kind), np.zeros((nb, hkv, 16, d), kind), np.full((nb, hkv, 2), np.nan, np.float32)]
    k, v, sc = to_dev(host[0]), to_dev(host[1]), torch.from_numpy(host[2]).cuda()
    steps = [[50, 0, 7, 0], [20, 0, 1, 0], "fork"] + [[1, 1, 1, 0]] * 14
    for rows in steps:
        if rows == "fork":
            blocks.fork(*(torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0], [1])))
            continue
        start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        st, T = torch.from_numpy(start).cuda(), int(start[-1])
        kn, kt = bf16_rows(rng, T, hkv, d, size=1.1)
        vn, vt = bf16_rows(rng, T, hkv, d)
        q, qt = bf16_rows(rng, T, hq, d)
        _, src, dst, _ = blocks.append(st, T)
        pkv.copy_blocks(k, v, src, dst, check_host=False, block_scales=sc)
        pkv.cache_append(k, v, sc, kt, vt, st, blocks.context_lens, blocks.block_tables)
        got = pkv.chunked_prefill_attention(k, v, qt, st, blocks.context_lens, blocks.block_tables, 128, d ** -0.5,
                                            query_start_loc_host=start, block_scales=sc)
        for a, c in zip(src.tolist(), dst.tolist()):
            if a >= 0:
                for x in host:
                    x[c] = x[a]
        lens, tables = blocks.context_lens.cpu().numpy(), blocks.block_tables.cpu().numpy()
        S.append(*host, kn, vn, start, lens, tables)
        assert np.array_equal(sc.cpu().numpy(), host[2], equal_nan=True)
        exact = S.attention(*host, q, start, lens, tables, d ** -0.5)
        tol = attention_tolerance(exact, int(lens.max()), host[2][np.isfinite(host[2])])
        assert np.all(np.abs(got.double().cpu().numpy() - exact[0]) <= tol)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,g,d", [(4, 1, 64), (2, 8, 128)])
def test_decode_more_blocks_than_a_cut_of_equal_ranges_needs(pkv, kind, hkv, g, d):
    """Enough work that short contexts count for more than their blocks (pairs then hold units without keys)."""
    lens = [(i * 193) % 700 for i in range(150 * 4 // hkv)] + [9000, 1, 0, 16]
    b = Batch(40, kind, [1] * len(lens), [n - 1 for n in lens], hkv, d)
    q, qt = bf16_rows(b.rng, b.T, g * hkv, d)
    got = decode(pkv, b, qt, d ** -0.5)
    check(b, got, q, d ** -0.5)
    assert torch.equal(got, decode(pkv, b, qt, d ** -0.5)) and pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_offsets_past_32_bits(pkv, kind):
    """Pools of 4.3 GB, the contexts in blocks beyond 2^32 bytes."""
    hkv, d = 40, 128
    b = Batch(41, kind, [1, 20, 300], [100, 5, 40], hkv, d)
    nb = 2 ** 32 // (hkv * 16 * d) + 64
    k = torch.zeros((nb, hkv, 16, d), dtype=torch.int8 if kind == np.int8 else torch.uint8, device="cuda")
    v, sc = torch.zeros_like(k), torch.ones((nb, hkv, 2), device="cuda")
    ids = torch.arange(nb - b.nb, nb, device="cuda")
    k[ids], v[ids], sc[ids] = (torch.from_numpy(x).cuda() for x in (b.k, b.v, b.scales))
    q, qt = bf16_rows(b.rng, b.T, hkv, d)
    _, _, _, start, lens, tables = b.dev()
    got = pkv.chunked_prefill_attention(k, v, qt, start, lens, tables + (nb - b.nb), int(b.lens.max()), 0.1,
                                        query_start_loc_host=b.start, block_scales=sc)
    check(b, got, q, 0.1)
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_calls_on_two_streams(pkv, kind):
    """Two batches at once, each with a workspace of its own."""
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    todo = []
    for i in range(2):
        b = Batch(42 + i, kind, [1] * 9 + [150], [50 * n for n in range(9)] + [400], 2, 128)
        q, qt = bf16_rows(b.rng, b.T, 4, 128)
        todo.append((b, q, qt, b.dev(), torch.from_numpy(b.start)))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, (b, _, qt, (k, v, sc, start, lens, tables), host) in enumerate(todo):
            outs[i].append(pkv.chunked_prefill_attention(k, v, qt, start, lens, tables, int(b.lens.max()), 0.1,
                                                         query_start_loc_host=host, block_scales=sc, stream=sides[i]))
    torch.cuda.synchronize()
    for (b, q, *_), got in zip(todo, outs):
        check(b, got[0], q, 0.1)
        assert all(torch.equal(got[0], x) for x in got[1:])
    assert pkv.get_error()[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_rows_into_page_locked_host_memory(pkv, kind, d):
    """A page-locked out gets the same bits as one on the device, tiles whose O is moved out between included."""
    b = Batch(41, kind, [200, 1, 37], [400, 50, 900], 2, d)
    q, qt = bf16_rows(b.rng, b.T, 4, d)
    host = torch.full((b.T, 4, d), -1.0).pin_memory()
    want = prefill(pkv, b, qt, 0.1)
    prefill(pkv, b, qt, 0.1, out=host)
    torch.cuda.synchronize()
    assert torch.equal(host, want.cpu())
    one = Batch(42, kind, [1] * 3, [700, 3, 90], 2, d)
    q, qt = bf16_rows(one.rng, 3, 4, d)
    host = torch.full((3, 4, d), -1.0).pin_memory()
    want = decode(pkv, one, qt, 0.1)
    decode(pkv, one, qt, 0.1, out=host)
    torch.cuda.synchronize()
    assert torch.equal(host, want.cpu()) and pkv.get_error()[0] == 0


def test_rows_that_the_call_does_not_have(pkv):
    """Device row starts that differ from the host's and leave the call's rows are reported; nothing is read or
    written there, and the other sequences are right."""
    for at, detail in (((3, 33), 2), ((1, 3), 1)):
        b = Batch(44, np.int8, [1, 30, 1], [5, 9, 50], 1, 64)
        q, qt = bf16_rows(b.rng, b.T, 2, 64)
        k, v, sc, start, lens, tables = b.dev()
        start[at[0]] = at[1]
        if detail == 2:
            start[2] = 32  # the last sequence's row is behind the rows
        guard = torch.full((b.T + 8, 2, 64), 5.0, device="cuda")
        got = pkv.chunked_prefill_attention(k, v, qt, start, lens, tables, int(b.lens.max()), 0.125, out=guard[:b.T],
                                            query_start_loc_host=b.start, block_scales=sc)
        if detail == 2:
            assert pkv.get_error() == (9, 2)
            exact = S.attention(b.k, b.v, b.scales, q, b.start, b.lens, b.tables, 0.125)[0]
            assert np.abs(got[0].cpu().numpy() - exact[0]).max() < 1e-4
        assert torch.all(guard[b.T:] == 5.0)
        pkv.get_error()


def test_an_expired_wait_is_reported_and_the_next_call_is_right(pkv):
    b = Batch(45, np.uint8, [1] * 3, [39, 299, 1499], 2, 128)
    q, qt = bf16_rows(b.rng, b.T, 4, 128)
    ws = pkv.new_workspace(pkv.decode_workspace_size(3, 4, 2, 128, 1500))
    out = torch.full((3, 4, 128), 7.0, device="cuda")
    pkv.test_arm_decode_stall(1)
    decode(pkv, b, qt, 0.1, out=out, workspace=ws)
    torch.cuda.synchronize()
    status, detail = pkv.get_error()
    assert status == 10 and detail in (2, 3)
    assert torch.all(out == 7.0) and int(ws.count_nonzero()) == 0
    check(b, decode(pkv, b, qt, 0.1, out=out, workspace=ws), q, 0.1)
    assert pkv.get_error()[0] == 0


def test_refusals_of_the_binding(pkv):
    b = Batch(46, np.int8, [1, 3], [4, 5], 2, 64)
    k, v, sc, start, lens, tables = b.dev()
    _, q = bf16_rows(b.rng, 4, 4, 64)
    args = dict(k_pool=k, v_pool=v, q=q[:2], block_tables=tables, context_lens=lens, max_context_len=8, scale=0.1,
                block_scales=sc)
    for bad in (dict(block_scales=sc[1:]), dict(block_scales=sc.double()), dict(q=q[:2].half()), dict(q=q[:2].float()),
                dict(q=q[:2, :, :32]), dict(q=q[:2].transpose(0, 1)), dict(k_scale=1.0), dict(context_lens=lens[:1]),
                dict(block_tables=tables[0]), dict(block_tables=tables.long()), dict(v_pool=v[1:]),
                dict(v_pool=v.view(torch.uint8)), dict(out=torch.empty((2, 4, 64), dtype=torch.bfloat16, device="cuda")),
                dict(out=torch.empty((3, 4, 64), device="cuda")), dict(out=torch.empty((2, 4, 64)))):
        with pytest.raises((TypeError, ValueError)):
            pkv.decode_attention(**(args | bad))
    for bad in (dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")), dict(max_context_len=-1)):
        with pytest.raises(pkv.PKVError):
            pkv.decode_attention(**(args | bad))
    args = dict(k_pool=k, v_pool=v, q=q, query_start_loc=start, context_lens=lens, block_tables=tables,
                max_context_len=8, scale=0.1, block_scales=sc)
    for bad in (dict(query_start_loc=start[:2]), dict(query_start_loc_host=b.start[:2]), dict(q=q.half()),
                dict(out=torch.empty((3, 4, 64), device="cuda")), dict(context_lens=lens.long())):
        with pytest.raises((TypeError, ValueError)):
            pkv.chunked_prefill_attention(**(args | bad))
    with pytest.raises(pkv.PKVError):
        pkv.chunked_prefill_attention(**(args | dict(query_start_loc_host=b.start + 1)))
    assert pkv.get_error()[0] == 0
