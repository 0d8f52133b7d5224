"""Linear attention over prompt chunks that replace their states in place.

The call reads a sequence's state and stores its new one from different
thread blocks: a sequence is cut over several, and a group's q heads may be
dealt to several.  Where both are one slot, the results are those of the same
batch with separate slots, bit for bit: the same sums of the same inputs.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import dev_tensor
from test_gpu_linear import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_291_gb300 as p
    p.load()
    return p


def run(pkv, b, new, states, **kw):
    out = pkv.linear_prefill_attention(states, dev_tensor(b.g), b.q, b.k, b.v, dev_tensor(b.qsl), dev_tensor(b.slots),
                                       dev_tensor(b.ctx), b.scale, new_slots=new, query_start_loc_host=b.qsl, **kw)
    return out, states


def assert_in_place_equals_separate(pkv, b, what="", runs=3):
    """new_slots left out, naming the same slots, and naming them for every
    other sequence, against separate slots for all."""
    want, after = run(pkv, b, dev_tensor(b.new), dev_tensor(b.S0))
    assert pkv.get_error() == (0, 0)
    same = dev_tensor(b.slots)
    some = np.where(np.arange(len(b.lens)) % 2 == 0, b.slots, b.new)
    for name, new, to in (("left out", None, b.slots), ("the same", same, b.slots), ("some", dev_tensor(some), some)):
        for _ in range(runs):
            out, states = run(pkv, b, new, dev_tensor(b.S0))
            assert pkv.get_error() == (0, 0)
            assert torch.equal(out, want), f"{what}: out, new_slots {name}"
            for s, n in enumerate(b.lens):
                if n:
                    assert torch.equal(states[int(to[s])], after[int(b.new[s])]), f"{what}: state {s}, {name}"


# Each batch has a sequence whose first chunks come late in one block's list
# and whose last come early in another's.
CUT = [
    ([1800, 2000, 1700], 16, 16, 128),
    ([1283, 1092, 453, 1107], 16, 16, 128),
    ([500, 300, 640], 16, 8, 128),
    ([300, 5, 900, 1, 450], 8, 4, 64),
    ([2000, 130, 1900, 64, 700], 32, 8, 64),
]


@pytest.mark.parametrize("lens,hq,hkv,d", CUT)
def test_cut_sequences_in_place(pkv, lens, hq, hkv, d):
    b = Batch(200 + len(lens), lens, [5 + s for s in range(len(lens))], hq, hkv, d)
    assert_in_place_equals_separate(pkv, b, "cut")


def test_cut_sequences_in_place_against_the_oracle(pkv):
    b = Batch(210, [500, 300, 640], [3, 9, 4], 16, 8, 128, separate=False)
    b.check(b.prefill(pkv), "in place")
    assert pkv.get_error() == (0, 0)


@pytest.mark.parametrize("seed", range(8))
def test_random_batches_in_place(pkv, seed):
    """Chunks of 16 to 2,000 tokens, some of them fresh sequences."""
    rng = np.random.default_rng(220 + seed)
    hq, hkv, d = [(16, 8, 128), (16, 16, 128), (32, 8, 64), (8, 2, 128)][seed % 4]
    lens = [int(np.exp(rng.uniform(np.log(16), np.log(2000)))) for _ in range(int(rng.integers(2, 9)))]
    past = [int(x) for x in rng.integers(0, 4, len(lens))]
    assert_in_place_equals_separate(pkv, Batch(230 + seed, lens, past, hq, hkv, d), f"lens {lens}", runs=1)


def test_cut_sequences_in_place_in_a_replayed_graph(pkv):
    """Every replay goes on from the state that the last one left."""
    b = Batch(240, [900, 700, 800], [3, 3, 3], 8, 8, 128, packed=False)
    dev = [dev_tensor(x) for x in (b.g, b.qsl, b.slots, b.ctx)]
    ws = torch.empty(pkv.linear_prefill_workspace_size(3, 2400, 8, 8, 128), dtype=torch.uint8, device="cuda")
    out = torch.zeros((2400, 8, 128), device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pkv.linear_prefill_attention(b.states, dev[0], b.q, b.k, b.v, dev[1], dev[2], dev[3], b.scale, out=out,
                                     workspace=ws, query_start_loc_host=b.qsl)
    states = dev_tensor(b.S0)
    for _ in range(3):
        graph.replay()
        new = dev_tensor(b.new)
        want, states = run(pkv, b, new, states)  # to spare slots, then back
        states[dev[2].long()] = states[new.long()]
        torch.cuda.synchronize()
        assert pkv.get_error() == (0, 0)
        assert torch.equal(out, want)
        assert torch.equal(b.states[dev[2].long()], states[dev[2].long()])


# Batches whose plan deals the q heads of a state to several blocks, with
# sequences that lie whole in a range.
DEALT = [
    ([80], 8, 1, 64),
    ([40], 8, 1, 128),
    ([64] * 6, 8, 2, 128),
    ([100] * 40, 32, 8, 64),
    ([90, 64, 3, 200, 1, 70, 65], 16, 2, 64),
    ([30, 1, 64, 2, 100], 32, 4, 128),
]


@pytest.mark.parametrize("lens,hq,hkv,d", DEALT)
def test_dealt_heads_in_place(pkv, lens, hq, hkv, d):
    b = Batch(250 + len(lens), lens, [4 + s % 3 for s in range(len(lens))], hq, hkv, d)
    assert_in_place_equals_separate(pkv, b, "dealt")


def test_dealt_heads_in_place_against_the_oracle(pkv):
    b = Batch(260, [64, 40, 100, 1, 128], [3, 0, 4, 5, 6], 8, 2, 64, separate=False)
    b.check(b.prefill(pkv), "in place")
    assert pkv.get_error() == (0, 0)


def test_in_place_while_another_stream_holds_multiprocessors(pkv):
    """The blocks of a call then start at different times."""
    other = Batch(261, [6000], [0], 16, 16, 128, packed=False)
    batches = [Batch(262, [100] * 40, [4] * 40, 32, 8, 64), Batch(263, [64] * 12, [4] * 12, 16, 4, 128),
               Batch(264, [1283, 1092, 453, 1107], [4] * 4, 16, 16, 128)]
    wants = [run(pkv, b, dev_tensor(b.new), dev_tensor(b.S0)) for b in batches]
    want_other = other.prefill(pkv)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        outs = []
        with torch.cuda.stream(side):
            others = [other.prefill(pkv) for _ in range(8)]
        for b in batches:
            outs.append(run(pkv, b, None, dev_tensor(b.S0)))
        torch.cuda.synchronize()
        assert pkv.get_error() == (0, 0)
        for b, (want, after), (out, states) in zip(batches, wants, outs):
            assert torch.equal(out, want)
            assert torch.equal(states[dev_tensor(b.slots).long()], after[dev_tensor(b.new).long()])
        for x in others:
            assert torch.equal(x, want_other)


@pytest.mark.parametrize("lens,hq,hkv,d", [([100] * 40, 32, 8, 64), ([90, 64, 3, 200, 1, 70, 65], 16, 2, 64),
                                           ([500, 300, 640], 16, 8, 128)])
def test_counters_and_copies_stay_in_a_workspace_that_needs_no_clearing(pkv, lens, hq, hkv, d):
    """Dealt heads alone, both, and a cut alone, in a workspace of the size
    asked for, full of ones before each call."""
    b = Batch(270 + len(lens), lens, [4] * len(lens), hq, hkv, d)
    want, after = run(pkv, b, dev_tensor(b.new), dev_tensor(b.S0))
    need = pkv.linear_prefill_workspace_size(len(lens), b.T, hq, hkv, d)
    ws = torch.empty(need + 4096, dtype=torch.uint8, device="cuda")
    for fill in (0xFF, 0x11, 0):
        ws.fill_(fill)
        out, states = run(pkv, b, None, dev_tensor(b.S0), workspace=ws[:need])
        assert pkv.get_error() == (0, 0)
        assert torch.all(ws[need:] == fill)
        assert torch.equal(out, want)
        assert torch.equal(states[dev_tensor(b.slots).long()], after[dev_tensor(b.new).long()])
