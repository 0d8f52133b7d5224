"""GPU parity of linear attention (recurrent and chunked) against the fp64
oracle.

Tolerance, derived: every term of an output or state element passes through a
bounded number of fp32 roundings: up to four for each token it is carried over
(the decay pair, the update, the products that stand for them in the chunked
form) and fewer than forty for the products, sums and factors of its own
chunk.  The error is thus at most (40 + 4 rows) 2^-24 times the same sum over
absolute values, which the oracle gives for |q|, |k|, |v| and |S|.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import assert_close, dev_tensor
from oracle import linear as L
from oracle import rotary as R
import pkv_workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_291_gb300 as p
    p.load()
    return p


def f64(t):
    return t.float().double().cpu().numpy()


class Batch:
    """A ragged batch: lens new tokens each; past[s] tokens before them."""

    def __init__(self, seed, lens, past, hq, hkv, d, packed=True, spare=3, pad_rows=0, separate=True):
        rng = np.random.default_rng(seed)
        self.lens, S, T = lens, len(lens), sum(lens)
        self.T, self.hq, self.hkv, self.d = T, hq, hkv, d
        self.qsl = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.ctx = (np.array(lens) + np.array(past)).astype(np.int32)
        n = 2 * S + spare
        perm = rng.permutation(n).astype(np.int32)
        self.slots, self.new = perm[:S].copy(), perm[S:2 * S].copy() if separate else None
        self.g = -np.exp(rng.uniform(np.log(1e-3), np.log(1.0), hkv)).astype(np.float32)
        self.scale = float(d) ** -0.5
        self.S0 = (3 * rng.standard_normal((n, hkv, d, d))).astype(np.float32)
        # states that no sequence reads must not matter
        read = {int(self.slots[s]) for s in range(S) if past[s] > 0}
        for i in range(n):
            if i not in read:
                self.S0[i] = np.nan
        x = torch.from_numpy(rng.standard_normal((T + pad_rows, hq + 2 * hkv, d)).astype(np.float32)).bfloat16().cuda()
        x[T:] = float("nan")
        if packed:
            self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        else:
            self.q, self.k, self.v = (t.contiguous() for t in (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]))
        self.states = dev_tensor(self.S0)

    def args(self):
        return (self.states, dev_tensor(self.g), self.q, self.k, self.v)

    def prefill(self, pkv, **kw):
        new = dev_tensor(self.new) if self.new is not None else None
        return pkv.linear_prefill_attention(*self.args(), dev_tensor(self.qsl), dev_tensor(self.slots),
                                            dev_tensor(self.ctx), self.scale, new_slots=new,
                                            query_start_loc_host=self.qsl, **kw)

    def decode(self, pkv, **kw):
        new = dev_tensor(self.new) if self.new is not None else None
        return pkv.linear_decode_attention(*self.args(), dev_tensor(self.slots), dev_tensor(self.ctx), self.scale,
                                           new_slots=new, **kw)

    def oracle(self, absolute=False):
        a = np.abs if absolute else (lambda x: x)
        return L.attend(a(self.S0), self.g, *(a(f64(x)[:self.T]) for x in (self.q, self.k, self.v)), self.qsl,
                        self.slots, self.ctx, self.scale, self.new)

    def check(self, out, what=""):
        want, after = self.oracle()
        bound, bound_after = self.oracle(absolute=True)
        c = (40 + 4 * np.repeat(np.array(self.lens), self.lens)) * 2.0 ** -24
        err = np.abs(f64(out)[:self.T] - want)
        assert np.all(err <= c[:, None, None] * bound + 1e-37), f"{what}: out off by {np.max(err):.3g}"
        got = self.states.double().cpu().numpy()
        stored = set()
        new = self.new if self.new is not None else self.slots
        for s, n in enumerate(self.lens):
            if n > 0 and 0 <= new[s] < len(got):
                i = int(new[s])
                if not np.array_equal(after[i], self.S0[i].astype(np.float64), equal_nan=True):
                    stored.add(i)
                    e = np.abs(got[i] - after[i])
                    assert np.all(e <= (40 + 4 * n) * 2.0 ** -24 * bound_after[i] + 1e-37), f"{what}: state {s}"
        for i in range(len(got)):
            if i not in stored:
                assert np.array_equal(got[i].astype(np.float32), self.S0[i], equal_nan=True), f"{what}: slot {i}"


HEADS = [(1, 1, 64), (4, 2, 128), (8, 2, 64), (8, 1, 128), (3, 3, 128), (16, 8, 64)]


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("seqs", [1, 5])
def test_decode(pkv, hq, hkv, d, seqs, packed):
    past = [0 if s % 3 == 2 else 10 + s for s in range(seqs)]
    b = Batch(hq * d + seqs, [1] * seqs, past, hq, hkv, d, packed=packed)
    out = b.decode(pkv)
    assert pkv.get_error() == (0, 0)
    b.check(out, "decode")


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (2, 2, 64)])
def test_decode_in_place_steps_follow_the_recurrence(pkv, hq, hkv, d):
    """Twenty steps on the same slots equal the oracle over twenty tokens."""
    n, S = 20, 3
    whole = Batch(21, [n] * S, [0] * S, hq, hkv, d, packed=False, separate=False)
    for t in range(n):
        rows = torch.arange(S, device="cuda") * n + t
        out = pkv.linear_decode_attention(whole.states, dev_tensor(whole.g), whole.q[rows], whole.k[rows],
                                          whole.v[rows], dev_tensor(whole.slots),
                                          torch.full((S,), t + 1, dtype=torch.int32, device="cuda"), whole.scale)
    want, _ = whole.oracle()
    bound, _ = whole.oracle(absolute=True)
    last = whole.qsl[1:] - 1
    assert np.all(np.abs(f64(out) - want[last]) <= (40 + 4 * n) * 2.0 ** -24 * bound[last])
    assert pkv.get_error() == (0, 0)


def test_decode_padding_skips_and_stores_nowhere(pkv):
    b = Batch(22, [1] * 7, [5, 5, 5, 0, 0, 9, 9], 4, 2, 64)
    b.ctx[1] = 0            # padding
    b.slots[2] = -1         # no state to go on from
    b.slots[3] = -7         # fresh: its slot is not read
    b.new[4] = -1           # fresh, not stored
    b.new[5] = -1           # goes on, not stored
    out = b.decode(pkv)
    assert pkv.get_error() == (0, 0)
    want, after = b.oracle()
    want[1] = 0
    bound, _ = b.oracle(absolute=True)
    assert np.all(np.abs(f64(out) - want) <= 44 * 2.0 ** -24 * bound)
    assert torch.all(out[1] == 0) and torch.all(out[2] == 0) and torch.all(out[3] != 0)
    got = b.states.double().cpu().numpy()
    for s in (0, 3, 6):
        assert np.allclose(got[b.new[s]], after[b.new[s]], rtol=1e-5, atol=1e-5)
    for s in (1, 2):
        assert np.array_equal(got[b.new[s]].astype(np.float32), b.S0[b.new[s]], equal_nan=True)


@pytest.mark.parametrize("field,value", [("slots", 17), ("new", 17), ("ctx", -1)])
def test_decode_out_of_range_is_reported_and_zero(pkv, field, value):
    b = Batch(23, [1] * 3, [5] * 3, 2, 1, 64, spare=11)
    getattr(b, field)[1] = value
    out = b.decode(pkv)
    assert pkv.get_error() == (9, 1)
    assert torch.all(out[1] == 0) and torch.all(torch.isfinite(out)) and torch.any(out[2] != 0)
    want, _ = b.oracle()
    assert np.allclose(f64(out)[[0, 2]], want[[0, 2]], rtol=1e-4, atol=1e-4)
    got = b.states.cpu().numpy()
    untouched = [i for i in range(17) if i not in (b.new[0], b.new[2])]
    assert np.array_equal(got[untouched], b.S0[untouched], equal_nan=True)


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_shared_stored_slots_are_reported(pkv, form):
    for kind in ("two stores", "store and read"):
        b = Batch(24, [1, 1, 90] if form == "prefill" else [1] * 3, [5] * 3, 2, 1, 64)
        b.new[0] = b.new[2] if kind == "two stores" else b.slots[2]
        getattr(b, form)(pkv)
        st, detail = pkv.get_error()
        assert st == 6 and detail in (0, 2)
    # many readers of one slot are fine
    b = Batch(25, [1, 1, 90] if form == "prefill" else [1] * 3, [5] * 3, 2, 1, 64)
    b.slots[:] = b.slots[0]
    out = getattr(b, form)(pkv)
    assert pkv.get_error() == (0, 0)
    b.check(out, "one state for all")


@pytest.mark.parametrize("lens", [[1], [2], [70]])
def test_decays_at_and_past_their_ends(pkv, lens):
    """0 keeps everything, -inf nothing; a positive or NaN decay counts as 0
    and is reported."""
    b = Batch(26, lens, [3], 4, 4, 64)
    b.g = np.array([0.0, -np.inf, -1e30, -1e-9], np.float32)
    out = b.prefill(pkv)
    assert pkv.get_error() == (0, 0)
    b.check(out, "decay ends")
    for bad in (0.25, np.nan):
        b = Batch(27, lens, [3], 4, 4, 64)
        b.g[2] = bad
        out = b.prefill(pkv)
        assert pkv.get_error() == (9, 2)
        b.g[2] = 0.0
        b.check(out, "decay out of range")


PREFILLS = [
    ([1], [0]), ([1], [9]), ([2], [0]), ([3, 1, 5], [0, 4, 9]), ([63], [0]), ([64], [0]), ([65], [7]),
    ([128, 1, 127], [0, 3, 1]), ([129], [64]), ([300], [0]), ([0, 17, 0, 200, 1], [3, 0, 0, 50, 1]),
    ([700, 16, 33], [0, 100, 0]),
]


@pytest.mark.parametrize("lens,past", PREFILLS)
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (4, 2, 64)])
def test_prefill(pkv, lens, past, hq, hkv, d):
    b = Batch(30 + len(lens), lens, past, hq, hkv, d)
    out = b.prefill(pkv)
    assert pkv.get_error() == (0, 0)
    b.check(out, "prefill")


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("packed", [True, False])
def test_prefill_heads_and_strides(pkv, hq, hkv, d, packed):
    b = Batch(40, [130, 20, 1], [0, 6, 6], hq, hkv, d, packed=packed, separate=False)
    out = b.prefill(pkv)
    assert pkv.get_error() == (0, 0)
    b.check(out, "heads")


def test_prefill_many_short_sequences(pkv):
    rng = np.random.default_rng(41)
    lens = [int(x) for x in rng.integers(0, 40, 70)]
    b = Batch(42, lens, [int(x) for x in rng.integers(0, 3, 70)], 2, 2, 64)
    b.check(b.prefill(pkv), "many")
    assert pkv.get_error() == (0, 0)


def test_prefill_long_prompt_is_cut_and_joined(pkv):
    """A prompt long enough to be split over the SMs, one head."""
    for seed, hq, hkv, d, past in ((43, 1, 1, 128, 0), (44, 2, 1, 64, 11)):
        b = Batch(seed, [4100], [past], hq, hkv, d)
        b.check(b.prefill(pkv), "long prompt")
        assert pkv.get_error() == (0, 0)


def test_prefill_chunks_equal_one_call(pkv):
    """A prompt taken in slices ends in the state of one call (to rounding)."""
    b = Batch(45, [500], [0], 4, 2, 128, packed=False, separate=False)
    want, after = b.oracle()
    bound, bound_after = b.oracle(absolute=True)
    outs, at = [], 0
    for n in (200, 1, 64, 235):
        outs.append(pkv.linear_prefill_attention(
            b.states, dev_tensor(b.g), b.q[at:at + n], b.k[at:at + n], b.v[at:at + n],
            dev_tensor(np.array([0, n], np.int32)), dev_tensor(b.slots),
            dev_tensor(np.array([at + n], np.int32)), b.scale))
        at += n
    assert np.all(np.abs(f64(torch.cat(outs)) - want) <= 2040 * 2.0 ** -24 * bound)
    i = int(b.slots[0])
    assert np.all(np.abs(b.states[i].double().cpu().numpy() - after[i]) <= 2040 * 2.0 ** -24 * bound_after[i])


def test_prefill_padding_rows_and_bad_neighbours_stay_apart(pkv):
    """Rows behind the last sequence are left alone, and NaN or infinite
    rows of one sequence do not reach another, whichever side they are on."""
    lens = [100, 70, 65]
    b = Batch(46, lens, [0, 5, 0], 4, 2, 64, pad_rows=50)
    clean_oracle, _ = b.oracle()
    bound, _ = b.oracle(absolute=True)
    b.k[100:170] = float("nan")
    b.v[100:170] = float("inf")
    b.q[100:170] = float("nan")
    out = torch.full((b.T + 50, 4, 64), 7.0, device="cuda")
    b.prefill(pkv, out=out)
    assert pkv.get_error() == (0, 0)
    assert torch.all(out[b.T:] == 7)
    got = f64(out)
    for r0, r1 in ((0, 100), (170, 235)):
        assert np.all(np.abs(got[r0:r1] - clean_oracle[r0:r1]) <= 440 * 2.0 ** -24 * bound[r0:r1])
    assert not np.isfinite(got[100:170]).any()
    for s in (0, 2):
        assert torch.isfinite(b.states[int(b.new[s])]).all()


@pytest.mark.parametrize("n", [1, 5, 90])
def test_prefill_refuses_per_sequence(pkv, n):
    """A context shorter than the rows, a slot past the pool: zero rows, no
    store, the others as usual."""
    for field, value in (("ctx", n - 1), ("slots", 99), ("new", 99)):
        b = Batch(47, [20, n, 90], [4, 4, 0], 2, 1, 64)
        getattr(b, field)[1] = value
        out = b.prefill(pkv)
        assert pkv.get_error() == (9, 1)
        assert torch.all(out[20:20 + n] == 0)
        b.check(out, field)


def test_prefill_guards(pkv):
    """Nothing is written outside out, the stored states and the workspace."""
    b = Batch(48, [300, 1, 40], [0, 2, 2], 4, 2, 128)
    need = pkv.linear_prefill_workspace_size(3, 341, 4, 2, 128)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    full = torch.full((341 + 2, 4, 128), 7.0, device="cuda")
    b.prefill(pkv, out=full[1:-1], workspace=ws[:need])
    assert pkv.get_error() == (0, 0)
    assert torch.all(ws[need:] == 0xA5) and torch.all(full[0] == 7) and torch.all(full[-1] == 7)
    b.check(full[1:-1], "guards")


def test_prefill_is_reproducible_and_workspace_needs_no_clearing(pkv):
    a = Batch(49, [2500, 3, 100], [0, 9, 2], 2, 1, 128)
    ws = torch.full((pkv.linear_prefill_workspace_size(3, 2603, 2, 1, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    first = a.prefill(pkv, workspace=ws).clone()
    states = a.states.clone()
    for _ in range(3):
        assert torch.equal(a.prefill(pkv, workspace=ws), first)
    assert torch.equal(a.states.view(torch.int32), states.view(torch.int32))


def test_replayed_graph_takes_new_inputs(pkv):
    """A captured prefill and decode step replay on changed inputs, and an
    eager call in between disturbs neither."""
    b = Batch(50, [150, 1, 30], [0, 4, 4], 4, 2, 128, packed=False)
    other = Batch(51, [150, 1, 30], [0, 4, 4], 4, 2, 128, packed=False)
    dev = [dev_tensor(x) for x in (b.g, b.qsl, b.slots, b.ctx, b.new)]
    ws = torch.empty(pkv.linear_prefill_workspace_size(3, 181, 4, 2, 128), dtype=torch.uint8, device="cuda")
    out = torch.zeros((181, 4, 128), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.linear_prefill_attention(b.states, dev[0], b.q, b.k, b.v, dev[1], dev[2], dev[3], b.scale,
                                     new_slots=dev[4], out=out, workspace=ws, query_start_loc_host=b.qsl)
    other.prefill(pkv)
    for name in ("q", "k", "v"):
        getattr(b, name).copy_(getattr(other, name))
    graph.replay()
    torch.cuda.synchronize()
    assert pkv.get_error() == (0, 0)
    b.check(out, "replay")


def test_two_streams_at_once(pkv):
    batches = [Batch(52 + i, [900, 1, 60], [0, 2, 2], 4, 4, 64) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in batches]
    outs = []
    torch.cuda.synchronize()
    for _ in range(3):
        outs = []
        for b, st in zip(batches, streams):
            with torch.cuda.stream(st):
                outs.append(b.prefill(pkv))
    torch.cuda.synchronize()
    assert pkv.get_error() == (0, 0)
    for b, out in zip(batches, outs):
        b.check(out, "streams")


def test_out_in_page_locked_memory(pkv):
    b = Batch(54, [1] * 4, [3] * 4, 4, 2, 64)
    out = torch.zeros((4, 4, 64)).pin_memory()
    b.decode(pkv, out=out)
    torch.cuda.synchronize()
    b.check(out, "pinned")
    b = Batch(55, [100, 1], [3, 3], 4, 2, 64)
    out = torch.zeros((101, 4, 64)).pin_memory()
    b.prefill(pkv, out=out)
    torch.cuda.synchronize()
    b.check(out, "pinned prefill")


def test_states_past_two_gigabytes(pkv):
    """Slots whose offsets pass 32 bits: 5.4 GB of states."""
    n, hkv, d = 10240, 8, 128
    states = torch.zeros((n, hkv, d, d), device="cuda")
    b = Batch(56, [1, 90], [4, 4], 8, 8, 128)
    src = dev_tensor(b.S0)
    states[n - 1], states[n - 2] = src[int(b.slots[0])], src[int(b.slots[1])]
    small = b.prefill(pkv).clone()
    slots = dev_tensor(np.array([n - 1, n - 2], np.int32))
    out = pkv.linear_prefill_attention(states, dev_tensor(b.g), b.q, b.k, b.v, dev_tensor(b.qsl), slots,
                                       dev_tensor(b.ctx), b.scale)
    assert pkv.get_error() == (0, 0)
    assert torch.equal(out, small)
    assert torch.equal(states[n - 1], b.states[int(b.new[0])])
    assert torch.equal(states[n - 2], b.states[int(b.new[1])])


def test_prefill_more_sequences_than_a_range_lists(pkv):
    """300 one- and two-chunk sequences on one head: ranges are held to the
    128 segments a CTA lists."""
    rng = np.random.default_rng(70)
    lens = [int(x) for x in rng.integers(12, 90, 300)]
    b = Batch(71, lens, [int(x) for x in rng.integers(0, 2, 300) * 5], 1, 1, 64)
    b.check(b.prefill(pkv), "300 sequences")
    assert pkv.get_error() == (0, 0)


def test_prefill_joins_more_ranges_than_are_listed_at_once(pkv):
    """100,000 tokens of one head: 1,563 chunks in more than the 128 ranges
    that the join lists at once, with a decay slow enough to carry a state
    over many of them.  Tolerance: a term meets no more than 28 half steps per
    chunk (twelve truncating sums of the tensor cores, a whole step each, and
    four roundings of the decay), four per join (at most 152), and forty in its
    own chunk."""
    b = Batch(72, [100000], [4], 1, 1, 64)
    b.g[:] = -2e-4
    out = b.prefill(pkv)
    assert pkv.get_error() == (0, 0)
    want, after = b.oracle()
    bound, bound_after = b.oracle(absolute=True)
    c = (40 + 28 * 1563 + 4 * 152) * 2.0 ** -24
    assert np.all(np.abs(f64(out) - want) <= c * bound)
    i = int(b.new[0])
    assert np.all(np.abs(b.states[i].double().cpu().numpy() - after[i]) <= c * bound_after[i])


def test_prefill_more_keys_and_values_than_the_cache_keeps(pkv):
    """44 MB of K and V, cut into ranges: the first of their two readings asks
    for another cache policy."""
    b = Batch(73, [2700], [0], 64, 64, 64)
    b.check(b.prefill(pkv), "2,700 tokens of 64 heads")
    assert pkv.get_error() == (0, 0)


@pytest.mark.parametrize("seed", range(6))
def test_prefill_random_batches(pkv, seed):
    """Batches whose ranges begin and end anywhere in the sequences."""
    rng = np.random.default_rng(80 + seed)
    group, d = [(1, 128), (2, 64), (4, 128), (8, 64), (2, 128), (4, 64)][seed]
    hkv = int(rng.integers(1, 4))
    lens = [int(np.exp(rng.uniform(0, np.log(700)))) for _ in range(int(rng.integers(1, 9)))]
    past = [int(x) for x in rng.integers(0, 2, len(lens)) * 9]
    b = Batch(90 + seed, lens, past, group * hkv, hkv, d, packed=bool(seed % 2), separate=bool(seed % 3))
    b.check(b.prefill(pkv), f"lens {lens}")
    assert pkv.get_error() == (0, 0)


@pytest.mark.parametrize("n,hq,d", [(5, 2, 64), (150, 2, 64), (150, 1, 128)])
def test_values_that_are_not_finite_keep_their_place(pkv, n, hq, d):
    """A NaN or infinite v element reaches its own column from its own token
    on; a NaN q row its own outputs; a NaN k row all outputs from its token
    on.  Nothing earlier changes."""
    b = Batch(100, [n], [3], hq, 1, d, packed=False)
    want, _ = b.oracle()
    bound, _ = b.oracle(absolute=True)
    c = (40 + 4 * n) * 2.0 ** -24
    t = n * 2 // 3
    clean = {x: getattr(b, x).clone() for x in "qkv"}

    def run(name, index, value):
        for x in "qkv":
            getattr(b, x).copy_(clean[x])
        getattr(b, name)[index] = value
        out = f64(b.prefill(pkv))
        assert pkv.get_error() == (0, 0)
        return out

    def same(got, sel):
        assert np.all(np.abs(got[sel] - want[sel]) <= c * bound[sel])

    for value in (float("nan"), float("inf")):
        out = run("v", (t, 0, 7), value)
        same(out, np.s_[:t])
        assert not np.isfinite(out[t:, :, 7]).any()
        others = [e for e in range(d) if e != 7]
        same(out, np.s_[:, :, others])
        assert not torch.isfinite(b.states[int(b.new[0]), 0, :, 7]).any()
        assert torch.isfinite(b.states[int(b.new[0]), 0, :, 8]).all()
    out = run("q", (t, 0), float("nan"))
    assert np.isnan(out[t, 0]).all()
    out[t, 0] = want[t, 0]
    same(out, np.s_[:])
    out = run("k", (t, 0), float("nan"))
    same(out, np.s_[:t])
    assert np.isnan(out[t:]).all()


@pytest.mark.parametrize("lens,devices", [
    ([100, 100], ([0, 170, 200], [0, 100, 130], [0, 100, 900], [0, -5, 200])),
    ([64, 64], ([0, 64, 67],)),      # the host saw no short sequence
    ([3, 4], ([0, 3, 60],)),         # the host saw short ones only
])
def test_device_lengths_that_are_not_the_hosts_are_reported(pkv, lens, devices):
    b = Batch(101, lens, [0, 0], 2, 1, 64, pad_rows=60)
    for device in devices:
        pkv.linear_prefill_attention(*b.args(), dev_tensor(np.array(device, np.int32)), dev_tensor(b.slots),
                                     dev_tensor(b.ctx), b.scale, new_slots=dev_tensor(b.new),
                                     query_start_loc_host=b.qsl)
        st, _ = pkv.get_error()
        assert st == 9, device


def test_calls_on_a_stream_of_the_callers(pkv):
    """The stream argument, and torch's current stream."""
    st = torch.cuda.Stream()
    for explicit in (True, False):
        a, b = Batch(108, [1] * 3, [2] * 3, 2, 1, 64), Batch(109, [90, 2], [0, 3], 2, 1, 64)
        torch.cuda.synchronize()
        with torch.cuda.stream(st if not explicit else torch.cuda.default_stream()):
            kw = dict(stream=st) if explicit else {}
            out_a, out_b = a.decode(pkv, **kw), b.prefill(pkv, **kw)
        torch.cuda.synchronize()
        assert pkv.get_error() == (0, 0)
        a.check(out_a, "decode")
        b.check(out_b, "prefill")


def test_prefill_group_dealt_to_several_ctas_stores_the_state_once(pkv):
    """Few heads and a short prompt: the q heads of a state go to CTAs of their own."""
    b = Batch(102, [80], [4], 8, 1, 64, separate=False)
    b.check(b.prefill(pkv), "dealt")
    assert pkv.get_error() == (0, 0)


def test_two_graphs_on_one_workspace(pkv):
    """Graphs that share a workspace replay one after the other."""
    a, b = (Batch(103 + i, [700, 3, 60], [0, 4, 4], 2, 1, 128, packed=False) for i in range(2))
    ws = torch.empty(pkv.linear_prefill_workspace_size(3, 763, 2, 1, 128), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros((763, 2, 128), device="cuda") for _ in range(2)]
    graphs = []
    torch.cuda.synchronize()
    for x, out in ((a, outs[0]), (b, outs[1])):
        dev = [dev_tensor(y) for y in (x.g, x.qsl, x.slots, x.ctx, x.new)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.linear_prefill_attention(x.states, dev[0], x.q, x.k, x.v, dev[1], dev[2], dev[3], x.scale,
                                         new_slots=dev[4], out=out, workspace=ws, query_start_loc_host=x.qsl)
        graphs.append((g, dev))
    for g, _ in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    assert pkv.get_error() == (0, 0)
    a.check(outs[0], "first graph")
    b.check(outs[1], "second graph")


def test_decode_many_sequences_and_heads(pkv):
    b = Batch(105, [1] * 150, [0 if s % 5 == 0 else s for s in range(150)], 5, 5, 64)
    b.check(b.decode(pkv), "150 sequences")
    assert pkv.get_error() == (0, 0)


def test_slow_decay_keeps_its_accuracy_over_many_steps(pkv):
    """3,000 single-token steps of a head that forgets 1/10,000 a step: a
    factor rounded to fp32 once would be off by 2^-25 a step, 9e-5 at the
    end; the pair keeps the recurrence at its own roundings, which are
    independent: 2^-24 times the root of the steps, 3.3e-6, of the norm."""
    steps, d = 3000, 64
    rng = np.random.default_rng(106)
    S0 = rng.standard_normal((1, 1, d, d)).astype(np.float32)
    states = dev_tensor(S0)
    g = np.array([-1.00007e-4], np.float32)
    zero = torch.zeros((1, 1, d), dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    gd = dev_tensor(g)
    for _ in range(steps):
        pkv.linear_decode_attention(states, gd, zero, zero, zero, slots, ctx, 1.0)
    want = S0.astype(np.float64) * np.exp(float(g[0]) * steps)
    err = np.linalg.norm(states.double().cpu().numpy() - want) / np.linalg.norm(want)
    assert err <= 2.0 ** -24 * np.sqrt(steps), err


def test_binding_refuses_what_it_cannot_pass_on(pkv):
    b = Batch(107, [1] * 3, [2] * 3, 2, 1, 64)
    args = list(b.args()) + [dev_tensor(b.slots), dev_tensor(b.ctx)]
    for i, bad, kind in ((0, b.states.double(), TypeError), (0, b.states[:, :, :32], ValueError),
                         (1, dev_tensor(np.zeros(2, np.float32)), ValueError), (2, b.q.float(), TypeError),
                         (3, b.k[:2], ValueError), (4, b.v.cpu(), ValueError), (5, args[5].long(), TypeError),
                         (6, args[6][:2], ValueError)):
        broken = list(args)
        broken[i] = bad
        with pytest.raises(kind):
            pkv.linear_decode_attention(*broken, b.scale)
    with pytest.raises(ValueError):
        pkv.linear_decode_attention(*args, b.scale, out=torch.zeros((3, 2, 32), device="cuda"))
    with pytest.raises(ValueError):
        pkv.linear_decode_attention(*args, b.scale, out=torch.zeros((3, 2, 64)))
    with pytest.raises(ValueError):
        pkv.linear_prefill_attention(*args[:5], dev_tensor(np.array([0, 1, 3], np.int32)), args[5], args[6], b.scale)
    with pytest.raises(pkv.PKVError) as e:
        pkv.linear_prefill_attention(*args[:5], dev_tensor(b.qsl), args[5], args[6], b.scale,
                                     workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 7

def test_hybrid_layers_prefill_then_decode(pkv):
    """A two-layer step as a hybrid stack runs it: rotary, then softmax
    attention over the paged cache in one layer and linear attention over the
    states in the other; a mixed batch, then single tokens."""
    hq, hkv, d = 8, 4, 128
    lens, past = [130, 1, 40], [0, 20, 16]
    w = W.make_paged("hybrid", 60, hq, hkv, d, [lens[s] + past[s] for s in range(3)], lens)
    b = Batch(61, lens, past, hq, hkv, d, packed=True, separate=False)
    T = b.T
    f = (10000.0 ** (-np.arange(64) / 64.0)).astype(np.float32)
    how = dict(sections=[24, 20, 20], interleaved=True)
    rng = np.random.default_rng(62)
    pos = rng.integers(0, 300, (3, T)).astype(np.int32)
    k_pool, v_pool = dev_tensor(w.k_pool), dev_tensor(w.v_pool)
    qr = pkv.rotary_cache_write(k_pool, v_pool, b.q, b.k, b.v, dev_tensor(w.slot_mapping), dev_tensor(pos),
                                dev_tensor(f), sections=how["sections"], interleaved_axes=True)
    soft = pkv.chunked_prefill_attention(k_pool, v_pool, qr, dev_tensor(w.query_start_loc),
                                         dev_tensor(w.context_lens), dev_tensor(w.block_tables), w.max_context_len,
                                         w.scale, query_start_loc_host=w.query_start_loc)
    ql, kl = pkv.rotary(b.q, b.k, dev_tensor(pos), dev_tensor(f), sections=how["sections"], interleaved_axes=True)
    assert torch.equal(ql, qr)
    v = b.v
    b.q, b.k = ql, kl
    out = b.prefill(pkv)
    assert pkv.get_error() == (0, 0)
    # the attention oracles take the turned rows that the calls made
    b.check(out, "linear layer")
    w.q, w.k_new = ql.cpu().view(torch.int16).numpy().view(np.uint16), kl.cpu().view(torch.int16).numpy().view(np.uint16)
    w.v_new = v.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)
    kp, vp, ref = oracle.run_step(w)
    assert np.array_equal(k_pool.cpu().view(torch.int16).numpy().view(np.uint16), kp)
    assert_close(soft.cpu().numpy(), ref, "softmax layer")
    # one more token for every sequence, on the states and positions that follow
    S1 = b.states.double().cpu().numpy()
    x = torch.from_numpy(rng.standard_normal((3, hq + 2 * hkv, d)).astype(np.float32)).bfloat16().cuda()
    pos1 = rng.integers(300, 400, (3, 3)).astype(np.int32)
    q1, k1 = pkv.rotary(x[:, :hq], x[:, hq:hq + hkv], dev_tensor(pos1), dev_tensor(f), sections=how["sections"],
                        interleaved_axes=True)
    want_q = R.rotate(f64(x[:, :hq]), pos1, f, **how)
    assert np.all(np.abs(f64(q1) - want_q) <= 2.0 ** -8 * np.abs(want_q) + 2.0 ** -18)
    ctx1 = b.ctx + 1
    out1 = pkv.linear_decode_attention(b.states, dev_tensor(b.g), q1, k1, x[:, hq + hkv:], dev_tensor(b.slots),
                                       dev_tensor(ctx1), b.scale)
    args = (b.g, f64(q1), f64(k1), f64(x[:, hq + hkv:]), [0, 1, 2, 3], b.slots, ctx1, b.scale)
    want, _ = L.attend(S1, *args)
    bound, _ = L.attend(np.abs(S1), b.g, *(np.abs(a) for a in args[1:4]), *args[4:])
    assert np.all(np.abs(f64(out1) - want) <= 44 * 2.0 ** -24 * bound)
    assert pkv.get_error() == (0, 0)
