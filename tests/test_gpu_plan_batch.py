"""plan_batch (block table, positions and slots of a step) against a sequential plan: whole numbers, equal."""
import numpy as np
import pytest
import torch

import operators_ref as R

pytestmark = pytest.mark.gpu


def _batch(B, page, cached_hi, new_hi, seed, zero_new=False):
    g = np.random.default_rng(seed)
    cached = g.integers(0, cached_hi + 1, B)
    new = g.integers(0 if zero_new else 1, new_hi + 1, B)
    have = -(-cached // page)
    need = -(-(cached + new) // page)
    M = int(need.max(initial=1)) + 2
    total, fresh = int(have.sum()), int((need - have).sum())
    ids = g.permutation(total + fresh + 5)
    table = np.full((B, M), -7, np.int64)
    k = 0
    for b in range(B):
        table[b, :have[b]] = ids[k:k + have[b]]
        k += have[b]
    return cached, new, table, ids[total:]


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", torch.int32)


def _run(cached, new, table, free, page, T, out=None):
    import gated_mla_b200 as gmla
    tab = _dev(table)
    p = gmla.plan_batch(_dev(cached), _dev(new), tab, _dev(free), page, T, out=out)
    return p, tab


def _same(p, tab, ref):
    assert np.array_equal(tab.cpu().numpy(), ref["table"])
    for k in ("seq_lens", "cu_seqlens", "positions", "seq_ids", "slots"):
        assert np.array_equal(getattr(p, k).cpu().numpy(), ref[k]), k
    assert int(p.pages_used) == ref["pages_used"]


@pytest.mark.parametrize("B,page,cached_hi,new_hi,pad,zero", [
    (1, 64, 0, 1, 0, False), (1, 8, 63, 1, 3, False), (3, 16, 40, 5, 0, True), (64, 64, 32767, 1, 0, False),
    (257, 16, 300, 70, 129, True), (1000, 128, 2000, 33, 1, True), (31, 7, 100, 1000, 2, False),
    (4096, 64, 500, 2, 0, True), (4097, 64, 500, 2, 5, True), (9001, 32, 90, 3, 7, True)])
def test_plan_matches_the_sequential_plan(B, page, cached_hi, new_hi, pad, zero):
    import gated_mla_b200 as gmla
    cached, new, table, free = _batch(B, page, cached_hi, new_hi, seed=B + page, zero_new=zero)
    T = int(new.sum()) + pad
    p, tab = _run(cached, new, table, free, page, T)
    _same(p, tab, R.plan(cached, new, table, free, page, T))
    gmla.sync_status()


def test_empty_batch_and_no_tokens():
    import gated_mla_b200 as gmla
    p, _ = _run(np.zeros(0, int), np.zeros(0, int), np.zeros((0, 4), int), np.zeros(0, int), 16, 6)
    assert p.positions.tolist() == [-1] * 6 and p.cu_seqlens.tolist() == [0] and int(p.pages_used) == 0
    p, tab = _run(np.array([5, 0]), np.array([0, 0]), np.array([[3, -7], [-7, -7]]), np.zeros(0, int), 16, 0)
    assert p.seq_lens.tolist() == [5, 0] and p.cu_seqlens.tolist() == [0, 0, 0] and tab.tolist() == [[3, -7], [-7, -7]]
    gmla.sync_status()


def test_pages_past_32_bits_of_slots():
    page = 128
    big = 2 ** 31 // page + 11
    p, _ = _run(np.array([130]), np.array([2]), np.array([[big, big + 1, -1]]), np.array([4]), page, 2)
    assert p.slots.tolist() == [(big + 1) * page + 2, (big + 1) * page + 3]


def test_length_near_the_largest():
    page = 1 << 20
    M = 2047
    cached, new = np.array([page * M - 3]), np.array([3])
    table = np.arange(M)[None, :] + 10
    p, _ = _run(cached, new, table, np.zeros(0, int), page, 4)
    assert p.positions.tolist() == [page * M - 3, page * M - 2, page * M - 1, -1]
    assert p.seq_lens.tolist() == [page * M]


@pytest.mark.parametrize("what", ["tokens", "pages", "negative", "too long", "negative new", "many"])
def test_a_batch_that_cannot_be_is_planned_as_empty(what):
    import gated_mla_b200 as gmla
    B = 5000 if what == "many" else 6
    cached, new, table, free = _batch(B, 16, 50, 20, seed=3)
    T = int(new.sum())
    if what == "tokens":
        T -= 1
    elif what == "pages":
        free = free[:int((-(-(cached + new) // 16) - -(-cached // 16)).sum()) - 1]
    elif what == "negative":
        cached[2] = -1
    elif what == "negative new":
        new[3] = -4
    else:
        cached[B - 1] = 16 * table.shape[1]
    gmla.sync_status()
    p, tab = _run(cached, new, table, free, 16, T)
    assert np.array_equal(tab.cpu().numpy(), table)
    assert not p.seq_lens.any() and not p.cu_seqlens.any() and int(p.pages_used) == 0
    assert (p.positions == -1).all() and (p.seq_ids == -1).all() and (p.slots == -1).all()
    with pytest.raises(gmla._lib.GmlaError) as e:
        gmla.sync_status()
    assert e.value.status == gmla._lib.GMLA_ERR_DEVICE_RANGE
    from gated_mla_b200 import api
    for ws in api._scratch._held.values():      # the fault has been seen: later tests start clean
        ws[:4].zero_()


def test_captured_plan_replays_on_new_lengths():
    import gated_mla_b200 as gmla
    page, B = 16, 9
    cached, new, table, free = _batch(B, page, 40, 6, seed=11)
    T = 9 * 6
    dc, dn, dt, df = _dev(cached), _dev(new), _dev(table), _dev(free)
    p = gmla.plan_batch(dc, dn, dt, df, page, T)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gmla.plan_batch(dc, dn, dt, df, page, T, out=p)
    cached2, new2, table2, free2 = _batch(B, page, 40, 6, seed=12)
    M = min(table.shape[1], table2.shape[1])
    keep = (-(-(cached2 + new2) // page) <= M)
    cached2, new2 = np.where(keep, cached2, 0), np.where(keep, new2, 1)
    t2 = np.full_like(table, -7)
    t2[:, :M] = table2[:, :M]
    f2 = np.arange(100, 100 + len(free))
    used = int((-(-(cached2 + new2) // page) - -(-cached2 // page)).sum())
    if used > len(f2):
        new2 = np.zeros_like(new2)
    dc.copy_(_dev(cached2)), dn.copy_(_dev(new2)), dt.copy_(_dev(t2)), df.copy_(_dev(f2))
    graph.replay()
    torch.cuda.synchronize()
    _same(p, dt, R.plan(cached2, new2, t2, f2, page, T))
