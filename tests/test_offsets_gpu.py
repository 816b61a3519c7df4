"""A delta whose offsets do not start at 0, as they may come over a wire: every
way of applying, encoding and decoding it stays inside its buffers, and the
entries in front of offsets[0] count as parameter 0's."""
import ctypes

import pytest
import torch

import mx_reference
import sparse_bf16_delta_amd as sbd
from sparse_bf16_delta_amd import DeltaError, _abi

pytestmark = pytest.mark.gpu

LISTS = {
    "one": [(100, 96)],
    "two": [(40, 33), (64, 64)],
    "many": [(3, 33)] * 150,  # the search's first step is longer than one entry
}


def delta(snaps, density, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx = [(torch.rand(s.numel(), generator=g, device="cuda") < density).nonzero().view(-1).int()
           for s in snaps]
    val = torch.randn(sum(i.numel() for i in idx), generator=g, device="cuda").to(torch.bfloat16)
    off = torch.tensor([0] + [i.numel() for i in idx], device="cuda").cumsum(0)
    return torch.cat(idx), val, off


def started_at(off, first):
    off = off.clone()
    off[0] = first
    return off


def make(name):
    g = torch.Generator(device="cuda").manual_seed(1)
    return [torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in LISTS[name]]


@pytest.mark.parametrize("first", [-3, 1, 7])
@pytest.mark.parametrize("counted", [False, True])
@pytest.mark.parametrize("name", list(LISTS))
def test_apply_and_replica(name, counted, first):
    snaps = make(name)
    idx, val, off = delta(snaps, 0.3, 2)
    assert int(off[1]) > 7
    want = [s.clone() for s in snaps]
    sbd.apply_many_(want, idx, val, off)
    got = [s.clone() for s in snaps]
    sbd.apply_many_(got, idx, val, started_at(off, first), check_indices=counted)
    both = [s.clone() for s in snaps]
    quants = sbd.mxfp4_quantize_many(both)
    sbd.mxfp4_apply_many_(both, quants, idx, val, started_at(off, first), check_indices=counted)
    for w, a, b, q in zip(want, got, both, quants):
        assert torch.equal(w.view(torch.int16), a.view(torch.int16))
        assert torch.equal(w.view(torch.int16), b.view(torch.int16))
        codes, scales = mx_reference.quantize(w)
        assert torch.equal(q.codes, codes) and torch.equal(q.scales, scales)


@pytest.mark.parametrize("first", [-3, 7])
def test_dense_apply_with_replica(first):
    snaps = [torch.randn(1024, 1024, device="cuda").to(torch.bfloat16) for _ in range(2)]
    idx, val, off = delta(snaps, 0.9, 3)
    want = [s.clone() for s in snaps]
    sbd.apply_many_(want, idx, val, off)
    quants = sbd.mxfp4_quantize_many(snaps)
    sbd.mxfp4_apply_many_(snaps, quants, idx, val, started_at(off, first))
    for w, s, q in zip(want, snaps, quants):
        assert torch.equal(w.view(torch.int16), s.view(torch.int16))
        codes, scales = mx_reference.quantize(w)
        assert torch.equal(q.codes, codes) and torch.equal(q.scales, scales)


@pytest.mark.parametrize("name", list(LISTS))
def test_encode_stays_inside_its_block(name):
    snaps = make(name)
    numels = [s.numel() for s in snaps]
    idx, _, off = delta(snaps, 0.3, 4)
    pos, _ = sbd.wire_encode(idx, off, numels)
    k = len(snaps)
    room = torch.full((256 + pos.numel() + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    block = room[256:256 + pos.numel()]
    po = torch.empty(k + 1, dtype=torch.int64, device="cuda")
    ws = torch.empty(_abi.load().delta_workspace_size(0, k), dtype=torch.uint8, device="cuda")
    P = ctypes.c_void_p
    moved = started_at(off, 7)
    status = _abi.load().delta_wire_encode(
        k, (ctypes.c_int64 * k)(*numels), P(idx.data_ptr()), P(moved.data_ptr()), idx.numel(),
        P(block.data_ptr()), block.numel(), P(po.data_ptr()), P(ws.data_ptr()), ws.numel(),
        P(torch.cuda.current_stream().cuda_stream))
    assert status == _abi.DELTA_OK
    width = 2  # every parameter has at most 65536 elements
    assert torch.equal(block[:-7 * width], pos[7 * width:])
    assert bool((room[:256] == 0xA5).all()) and bool((room[-256 - 7 * width:] == 0xA5).all())


@pytest.mark.parametrize("name", list(LISTS))
def test_decode_reports_what_has_no_place(name):
    snaps = make(name)
    numels = [s.numel() for s in snaps]
    idx, _, off = delta(snaps, 0.3, 5)
    pos, po = sbd.wire_encode(idx, off, numels)
    with pytest.raises(DeltaError, match="malformed"):
        sbd.wire_decode(pos, po, started_at(off, 7), numels)
    blocked = sbd.wire_encode_blocked(idx, off, numels)
    # 16-bit places within the parameter's first block: nothing here is lost
    assert torch.equal(sbd.wire_decode_blocked(blocked, started_at(off, 7), numels), idx)


@pytest.mark.parametrize("first", [-(1 << 62) + 1, -(1 << 61) + 1, -(1 << 63)])
def test_decode_of_places_at_the_end_of_int64(first):
    """An entry's byte from such an offset lies just below 2^63, where the
    position's own bytes pass it."""
    numels = [70000, 300]  # 4 bytes and 2 bytes a position
    snaps = [torch.zeros(n, device="cuda", dtype=torch.bfloat16) for n in numels]
    idx, _, off = delta(snaps, 0.1, 6)
    pos, po = sbd.wire_encode(idx, off, numels)
    blocked = sbd.wire_encode_blocked(idx, off, numels)
    bad = started_at(off, first)
    for sizes in (numels, numels[::-1]):  # the first parameter's width is 4, then 2
        with pytest.raises(DeltaError, match="malformed"):
            sbd.wire_decode(pos, po, bad, sizes)
    # the blocked form takes nothing but the entries' order from offsets
    with pytest.raises(DeltaError, match="malformed"):
        sbd.wire_decode_blocked(blocked, bad, numels)
