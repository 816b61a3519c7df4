"""Deltas into lists of about 17 million values, where the apply with replica
changes its steps and its way: snapshots and replica bit for bit against the
reference in 64 bits, with and without counting bad entries, through a plan and
in a graph."""
import functools

import pytest
import torch

import mx_reference
import sparse_bf16_delta_amd as sbd
from mx_rules import apply_way
from sparse_bf16_delta_amd import DeltaError

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
LISTS = {
    "one": [(4096, 4096)],
    "one ragged": [(4001, 4099)],
    # hundreds of tensors to a step between large ones, ragged and not
    "many": [(1024, 4096), (700, 4097)] + [(3, 45), (1, 1), (2, 64)] * 250 + [(0, 32), (7, 0)]
            + [(2048, 2048), (1, 100001), (700, 4097), (1024, 4096)],
}
DENSITY = {"256": 0.02, "1024": 0.08, "dense": 0.25}
WAYS = [(name, way) for name in LISTS for way in DENSITY]


def elems(name):
    return sum(torch.Size(s).numel() for s in LISTS[name])


@functools.lru_cache(maxsize=None)
def case(name, way):
    """Snapshots, a delta that takes `way`, and the snapshots after it."""
    g = torch.Generator(device="cuda").manual_seed(17)
    snaps = [torch.randn(s, generator=g, device="cuda").to(BF16) for s in LISTS[name]]
    idx, val, counts, after = [], [], [], []
    for s in snaps:
        i = (torch.rand(s.numel(), generator=g, device="cuda") < DENSITY[way]).nonzero().view(-1)
        # values of other sizes than the old ones, so that scales change
        v = (torch.randn(i.numel(), generator=g, device="cuda") * 5).to(BF16)
        new = s.clone().view(-1)
        new[i] = v
        after.append(new.view(s.shape))
        idx.append(i.int())
        val.append(v)
        counts.append(i.numel())
    off = torch.tensor([0] + counts, device="cuda").cumsum(0)
    assert apply_way(elems(name), int(off[-1])) == way
    return snaps, torch.cat(idx), torch.cat(val), off, after


def copies(snaps):
    return [s.clone() for s in snaps]


def check(got, quants, want):
    for s, q, w in zip(got, quants, want):
        assert torch.equal(s.view(torch.int16), w.view(torch.int16))
        if w.numel():
            codes, scales = mx_reference.quantize(w.view(-1, w.shape[-1]))
            assert torch.equal(q.codes.view(codes.shape), codes)
            assert torch.equal(q.scales.view(scales.shape), scales)


@pytest.mark.parametrize("counted", [False, True])
@pytest.mark.parametrize("name,way", WAYS)
def test_one_shot(name, way, counted):
    snaps, idx, val, off, after = case(name, way)
    snaps = copies(snaps)
    quants = sbd.mxfp4_quantize_many(snaps)
    sbd.mxfp4_apply_many_(snaps, quants, idx, val, off, check_indices=counted)
    check(snaps, quants, after)


@pytest.mark.parametrize("counted", [False, True])
@pytest.mark.parametrize("name,way", WAYS)
def test_plan(name, way, counted):
    """The delta in a buffer larger than it is, its count given."""
    snaps, idx, val, off, after = case(name, way)
    snaps = copies(snaps)
    plan = sbd.Mxfp4Plan(snaps)
    plan.quantize()
    room = torch.cat([idx, torch.zeros(5000, dtype=torch.int32, device="cuda")])
    vroom = torch.cat([val, torch.zeros(5000, dtype=BF16, device="cuda")])
    bad = torch.full((1,), 77, dtype=torch.int64, device="cuda") if counted else None
    plan.apply(room, vroom, off, max_nnz=idx.numel(), violations=bad)
    check(snaps, plan.quants, after)
    assert bad is None or int(bad) == 0


@pytest.mark.parametrize("name,way", WAYS)
def test_bad_entries_are_counted_and_left_out(name, way):
    """In every large tensor of the list the last entries' positions lie behind
    the end, still ascending; everything else is as if they were not there."""
    snaps, idx, val, off, _ = case(name, way)
    snaps, idx = copies(snaps), idx.clone()
    bounds, count = off.tolist(), 0
    want = copies(snaps)
    for s, w, a, b in zip(snaps, want, bounds, bounds[1:]):
        drop = 3 if b - a > 1000 else 0
        idx[b - drop:b] = s.numel() + torch.arange(drop, device="cuda", dtype=torch.int32)
        w.view(-1)[idx[a:b - drop].long()] = val[a:b - drop]
        count += drop
    quants = sbd.mxfp4_quantize_many(snaps)
    with pytest.raises(DeltaError, match=f"^(.*[^0-9])?{count} delta entries"):
        sbd.mxfp4_apply_many_(snaps, quants, idx, val, off, check_indices=True)
    check(snaps, quants, want)


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("name", list(LISTS))
def test_captured_and_replayed(name, planned):
    """A delta of each way in one graph, one after another, with and without
    counting; the values change between the replays."""
    snaps = copies(case(name, "dense")[0])
    deltas = [tuple(t.clone() for t in case(name, way)[1:4]) for way in DENSITY]
    expect = copies(snaps)
    plan = sbd.Mxfp4Plan(snaps)
    plan.quantize()
    bad = torch.full((1,), 5, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for idx, val, off in deltas:
            if planned:
                plan.apply(idx, val, off)
                plan.apply(idx, val, off, violations=bad)
            else:
                sbd.mxfp4_apply_many_(snaps, plan.quants, idx, val, off)
    for _ in range(3):
        for _, val, _ in deltas:
            val.mul_(-1.3)
        for idx, val, off in deltas:
            sbd.apply_many_(expect, idx, val, off)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(snaps, plan.quants, expect)
        assert int(bad) == (0 if planned else 5)


def test_dense_deltas_in_a_row_through_one_plan():
    """Sparse, dense and sparse again, on two streams."""
    snaps = copies(case("many", "dense")[0])
    expect = copies(snaps)
    plan = sbd.Mxfp4Plan(snaps)
    plan.quantize()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for step, way in enumerate(("1024", "dense", "256", "dense")):
        idx, val, off = case("many", way)[1:4]
        val = val * (step + 1)
        sbd.apply_many_(expect, idx, val, off)
        torch.cuda.synchronize()
        with torch.cuda.stream(side if step % 2 else torch.cuda.current_stream()):
            plan.apply(idx, val, off)
        torch.cuda.synchronize()
        check(snaps, plan.quants, expect)
