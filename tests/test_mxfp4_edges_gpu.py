"""Calls of the MXFP4 operators at the edge of what the documentation allows:
deltas out of order, empty ones, lists without values, and products of several
launches in graphs."""
import pytest
import torch

import mx_reference
import mx_rules
import sparse_bf16_delta_amd as sbd
from sparse_bf16_delta_amd.plan import ApplyPlan

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def normal(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(BF16)


@pytest.mark.parametrize("counted", [False, True])
@pytest.mark.parametrize("shapes", [[(700, 96)], [(700, 96), (3, 45), (64, 33), (1, 1), (900, 64)]],
                         ids=["one", "list"])
def test_out_of_order_touches_only_what_it_names(shapes, counted):
    """Positions shuffled, some of them many times over and some outside: what
    the entries' blocks hold is unspecified, their other values and everything
    else are as before, and the bad entries are counted as the apply does."""
    # the snapshots and replicas lie between guards
    room = torch.full((1 << 18,), 7.0, dtype=BF16, device="cuda")
    bytes_ = torch.full((1 << 18,), 0xA5, dtype=torch.uint8, device="cuda")
    snaps, quants, at, bt = [], [], 64, 64
    for t, s in enumerate(shapes):
        v = normal(s, t)
        part = room[at:at + v.numel()].view(s)
        part.copy_(v)
        snaps.append(part)
        at += -(-v.numel() // 8) * 8 + 64
        e = sbd.mxfp4_empty(s, "cuda")
        views = []
        for b in (e.codes, e.scales):
            views.append(bytes_[bt:bt + b.numel()].view(b.shape))
            bt += -(-b.numel() // 16) * 16 + 64
        quants.append(sbd.Mxfp4(*views, s))
    sbd.mxfp4_quantize_many(snaps, quants)
    before, bytes_before = room.clone(), bytes_.clone()
    g = torch.Generator(device="cuda").manual_seed(9)
    idx, counts = [], []
    for s in snaps:
        n = s.numel()
        i = torch.randint(0, n, (max(1, n // 50),), generator=g, device="cuda")
        i = torch.cat([i, i[:1].repeat(300), torch.tensor([-5, n, n + 9], device="cuda"), i.flip(0)])
        i = i[torch.randperm(i.numel(), generator=g, device="cuda")]
        idx.append(i.int())
        counts.append(i.numel())
    off = torch.tensor([0] + counts, device="cuda").cumsum(0)
    flat = torch.cat(idx)
    val = normal((flat.numel(),), 77)
    copies = [s.clone() for s in snaps]
    want_bad = torch.zeros(1, dtype=torch.int64, device="cuda")
    ApplyPlan(copies).run(flat, val, off, violations=want_bad)
    bad = torch.zeros(1, dtype=torch.int64, device="cuda") if counted else None
    plan = sbd.Mxfp4Plan(snaps, quants)
    plan.apply(flat, val, off, violations=bad)
    torch.cuda.synchronize()
    assert int(want_bad) > 0 and (bad is None or int(bad) == int(want_bad))
    seen = torch.zeros(room.shape, dtype=torch.bool, device="cuda")
    named = torch.zeros(bytes_.shape, dtype=torch.bool, device="cuda")
    for s, q, i in zip(snaps, quants, idx):
        i = i[(i >= 0) & (i < s.numel())].long()
        start = (s.data_ptr() - room.data_ptr()) // 2
        seen[start + i] = True
        blocks = ((i // q.cols) * (-(-q.cols // 32)) + i % q.cols // 32).unique()
        sc = q.scales.data_ptr() - bytes_.data_ptr()
        cd = q.codes.data_ptr() - bytes_.data_ptr()
        named[sc + blocks] = True
        named[(cd + 16 * blocks[:, None] + torch.arange(16, device="cuda")).view(-1)] = True
    assert torch.equal(room[~seen].view(torch.int16), before[~seen].view(torch.int16))
    assert torch.equal(bytes_[~named], bytes_before[~named])


def test_empty_deltas_and_lists_without_values():
    snaps = [normal((50, 64), 1), normal((3, 33), 2)]
    before = [s.clone() for s in snaps]
    plan = sbd.Mxfp4Plan(snaps)
    plan.quantize()
    bad = torch.full((1,), 9, dtype=torch.int64, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    zero = torch.zeros(3, dtype=torch.int64, device="cuda")
    plan.apply(none, none.to(BF16), zero, violations=bad)
    assert int(bad) == 0
    room = torch.zeros(5000, dtype=torch.int32, device="cuda")  # a buffer without an entry
    bad.fill_(9)
    plan.apply(room, room.to(BF16), zero, violations=bad)
    plan.apply(room, room.to(BF16), zero)
    assert int(bad) == 0
    for s, b, q in zip(snaps, before, plan.quants):
        assert torch.equal(s, b)
        codes, scales = mx_reference.quantize(b)
        assert torch.equal(q.codes, codes) and torch.equal(q.scales, scales)
    # entries of tensors that have no values: all of them are outside
    hollow = [torch.empty(0, 5, dtype=BF16, device="cuda"), torch.empty(4, 0, dtype=BF16, device="cuda")]
    plan = sbd.Mxfp4Plan(hollow)
    plan.quantize()
    plan.apply(room[:3], room[:3].to(BF16), torch.tensor([0, 1, 3], device="cuda"), violations=bad)
    assert int(bad) >= 3 and all(v.numel() == 0 for v in plan.dequantize())


def test_products_of_several_launches_in_two_graphs():
    """Shares of k and a last round of their own, captured twice over, replayed
    in turn with eager products in between: every replay has the eager bits."""
    shapes = [(62, 7023, 8625), (117, 33, 12158), (2885, 7755, 1523), (3213, 16123, 381)]
    for s in shapes:
        cut = mx_rules.cut_of(*s)
        assert cut[1] > 1 or cut[2] > 0
    ws = [sbd.mxfp4_quantize(normal((n, k), 3)) for _, n, k in shapes]
    xs = [normal((m, k), 4) for m, _, k in shapes]
    outs = [[torch.empty(m, n, device="cuda", dtype=BF16) for m, n, _ in shapes] for _ in range(2)]
    sbd.mxfp4_matmul(xs[0], ws[0])
    torch.cuda.synchronize()
    graphs = []
    for o in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for x, w, y in zip(xs, ws, o):
                sbd.mxfp4_matmul(x, w, out=y)
    for _ in range(3):
        for x in xs:
            x.mul_(-1.25)
        want = [sbd.mxfp4_matmul(x, w) for x, w in zip(xs, ws)]
        for graph, o in zip(graphs, outs):
            for y in o:
                y.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            again = sbd.mxfp4_matmul(xs[0], ws[0])
            torch.cuda.synchronize()
            assert torch.equal(again, want[0])
            for y, w in zip(o, want):
                assert torch.equal(y, w)
