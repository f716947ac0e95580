"""Slots of state pools copied, cleared and compacted: every pool of a call against indexing on the CPU."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attention_recurrence_forward_b200 as kda
from linear_attention_recurrence_forward_b200 import STATUS
import serving_refs as ref

OK, INVALID, UNSUPPORTED, MISALIGNED = (STATUS[n] for n in
                                        ("KDA_OK", "KDA_ERR_INVALID_ARG", "KDA_ERR_UNSUPPORTED",
                                         "KDA_ERR_MISALIGNED"))
BASE, SZ = 0x7F0000000000, 1 << 32

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from linear_attention_recurrence_forward_b200 import build
    build.build()
    return kda.lib()


# ---------------------------------------------------------------------- refusals (CPU)

def desc(*pools):
    """kda_pool array from (base, slot_stride, pieces, piece_stride, piece_bytes) tuples."""
    flat = [v for p in pools for v in p]
    return (ctypes.c_longlong * len(flat))(*flat)


A0 = (BASE, 1024, 1, 0, 1024)
B0 = (BASE + SZ, 1024, 1, 0, 1024)
IX = BASE + 8 * SZ


def copy(L, dst, src, n_pools=1, n_dst=8, n_src=8, si=IX, di=IX + 64, n=4):
    return L.kda_pool_copy(dst, src, n_pools, n_dst, n_src, si, di, n, None)


def test_copy_refusals(L):
    a, b = desc(A0), desc(B0)
    assert copy(L, None, b) == INVALID and copy(L, a, None) == INVALID
    for k in (dict(n_pools=0), dict(n_pools=513), dict(n_dst=0), dict(n_src=0), dict(n=-1), dict(si=None), dict(di=None)):
        assert copy(L, a, b, **k) == INVALID, k
    assert copy(L, a, b, si=IX + 2) == MISALIGNED
    assert copy(L, a, b, di=BASE + 64) == INVALID                       # the indices inside a written pool
    assert copy(L, a, b, n=0) == OK                                     # nothing to do
    assert copy(L, a, desc((BASE + 4096, 1024, 1, 0, 1024))) == INVALID  # partly overlapping pools
    assert copy(L, a, desc((BASE, 2048, 1, 0, 1024))) == INVALID        # one base, other slots
    assert copy(L, a, desc(A0), n_src=9) == INVALID                     # one base, another number of slots
    assert copy(L, a, desc((BASE + SZ, 1024, 1, 0, 512))) == INVALID    # slots of another size
    assert copy(L, desc(A0, A0), desc(B0, B0), n_pools=2) == INVALID    # one pool written twice
    assert copy(L, desc(A0, B0), desc(B0, A0), n_pools=2) == INVALID    # a pool read by another pair of pools
    assert copy(L, desc((BASE + 8, 1024, 1, 0, 1024)), b) == MISALIGNED
    assert copy(L, desc((BASE, 1032, 1, 0, 1024)), b) == MISALIGNED
    assert copy(L, desc((BASE, 1024, 1, 0, 1000)), desc((BASE + SZ, 1024, 1, 0, 1000))) == MISALIGNED
    assert copy(L, desc((BASE, 512, 1, 0, 1024)), b) == INVALID         # overlapping slots
    two = (BASE, 1024, 2, 4096, 1024)                                   # 8 slots of 1 KB inside runs 4 KB apart
    assert copy(L, desc(two), desc((BASE + SZ,) + two[1:])) == INVALID
    assert copy(L, desc((None or 0,) + A0[1:]), b) == INVALID


def test_clear_and_compact_refusals(L):
    a = desc(A0)
    clear = lambda p=a, k=1, s=8, i=IX, n=4: L.kda_pool_clear(p, k, s, i, n, None)  # noqa: E731
    assert clear(p=None) == INVALID and clear(k=0) == INVALID and clear(s=0) == INVALID and clear(n=-1) == INVALID
    assert clear(i=None) == INVALID and clear(i=BASE) == INVALID and clear(i=IX + 1) == MISALIGNED
    assert clear(n=0) == OK
    def comp(p=a, k=1, s=8, sl=IX, done=IX + SZ, out=IX + 2 * SZ, B=4, ws=IX + 3 * SZ):
        return L.kda_pool_compact(p, k, s, sl, done, out, B, ws, None)
    assert comp(p=None) == INVALID and comp(k=0) == INVALID and comp(s=0) == INVALID and comp(B=0) == INVALID
    assert comp(sl=None) == INVALID and comp(out=None) == INVALID and comp(ws=None) == INVALID
    assert comp(s=65537) == UNSUPPORTED
    assert comp(ws=IX) == INVALID and comp(out=IX + 3 * SZ) == INVALID and comp(out=IX + 4) == INVALID
    assert comp(done=IX + 2 * SZ) == INVALID and comp(done=BASE) == INVALID and comp(out=BASE) == INVALID


def test_binding_refuses_bad_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_pool_copy([], i, i)
    with pytest.raises(ValueError):
        kda.kda_pool_copy([torch.zeros(4, 16)], i, i)                               # not on a GPU
    with pytest.raises(ValueError):
        kda.kda_pool_copy([torch.zeros(4, 16), torch.zeros(5, 16)], i, i)           # other slot counts
    with pytest.raises(ValueError):
        kda.kda_pool_copy([torch.zeros(4, 16)], i.long(), i)
    with pytest.raises(ValueError):
        kda.kda_pool_copy([torch.zeros(4, 8, 4, 4).transpose(2, 3)[..., :2]], i, i)  # runs that are not contiguous
    with pytest.raises(ValueError):
        kda.kda_pool_copy([torch.zeros(4, 16)], i, i, src_pools=[torch.zeros(4, 8)])


# ---------------------------------------------------------------------- GPU

def ids(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def make(n_slots, seed=0):
    """Pools of several dtypes and slot sizes, one smaller and one larger than a 32 KB part."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    shapes = [((n_slots, 3, 128, 128), torch.float32), ((n_slots, 3, 1096), torch.bfloat16), ((n_slots, 16), torch.uint8),
              ((n_slots, 1, 2064), torch.float32)]
    return [(torch.randn(s, generator=g, device="cuda") * 50).to(d) for s, d in shapes]


@gpu
@pytest.mark.parametrize("n_slots,src,dst", [
    (9, [3], [5]), (9, [3, 3, 3, 3], [0, 8, 2, 5]), (64, list(range(0, 30)), list(range(30, 60))),
    (9, [1, -1, 4, 2], [0, 7, -3, 5]), (9, [4], [4]), (300, [7] * 280, [i for i in range(300) if i not in range(7, 27)]),
    (1, [0], [0])])
def test_copy(n_slots, src, dst):
    pools = make(n_slots)
    want = [p.clone() for p in pools]
    kda.kda_pool_copy(pools, ids(src), ids(dst))
    for p, w in zip(pools, want):
        old = w.clone()
        for s, d in zip(src, dst):
            if s >= 0 and d >= 0:
                w[d] = old[s]
        assert torch.equal(p, w)
    assert kda.kda_get_device_status() == 0


@gpu
@pytest.mark.parametrize("src,dst,left", [
    ([0, 1, 2], [5, 5, 6], {6: 2}),             # one destination twice: neither is written
    ([0, 5, 2], [5, 7, 6], {7: 5, 6: 2}),       # slot 5 is read by the second pair: the first is left out
    ([0, 12], [5, 6], {5: 0}),                  # a source past the pool
    ([0, 1], [12, 6], {6: 1}),                  # a destination past the pool
    ([3, 4], [4, 3], {})])                      # a swap
def test_conflicting_pairs_are_left_out_and_reported(src, dst, left):
    pools = make(12)
    want = [p.clone() for p in pools]
    for w in want:
        old = w.clone()
        for d, s in left.items():
            w[d] = old[s]
    kda.kda_pool_copy(pools, ids(src), ids(dst))
    assert kda.kda_get_device_status() == INVALID
    assert all(torch.equal(p, w) for p, w in zip(pools, want))


@gpu
def test_boundary_states_restored_into_a_pool():
    """States after every 64 tokens (kda_forward_chunked_states) into slots of a pool, and a decode from one."""
    from linear_attention_recurrence_forward_b200.inputs import make_prefill_inputs
    H, n_slots = 3, 6
    q, k, v, g, beta, _ = make_prefill_inputs(2, 256, H, 128, 64, "bf16", seed=1, device="cuda")
    _, _, mid = kda.kda_forward_chunked_states(q, k, v, g, beta, interval=64)
    pool = torch.full((n_slots, H, 128, 64), 9.0, device="cuda")
    kda.kda_pool_copy([pool], ids([1, 3, 1]), ids([4, 0, 5]), src_pools=[mid[1].transpose(0, 1)])
    assert torch.equal(pool[4], mid[1, :, 1]) and torch.equal(pool[5], mid[1, :, 1]) and torch.equal(pool[0], mid[1, :, 3])
    assert bool((pool[1:4] == 9).all()) and kda.kda_get_device_status() == 0
    kda.kda_decode_step_paged(*(t[1:, 128].contiguous() for t in (q, k, v, g, beta)), pool, ids([4]))
    again = mid[1:, :, 1].contiguous()
    kda.kda_decode_step(*(t[1:, 128].contiguous() for t in (q, k, v, g, beta)), again)
    assert torch.equal(pool[4], again[0])
    # and back: a state into the boundary array, whose slots are runs apart
    kda.kda_pool_copy([mid[0].transpose(0, 1)], ids([5]), ids([2]), src_pools=[pool])
    assert torch.equal(mid[0, :, 2], pool[5])


@gpu
def test_many_pools():
    """More pools than one launch carries."""
    pools = [torch.full((5, 64), float(i), device="cuda") + torch.arange(5, device="cuda")[:, None] for i in range(97)]
    kda.kda_pool_copy(pools, ids([1]), ids([4]))
    assert all(float(p[4, 0]) == i + 1 and float(p[3, 5]) == i + 3 for i, p in enumerate(pools))
    kda.kda_pool_clear(pools, ids([0, 4]))
    assert all(bool((p[[0, 4]] == 0).all()) and float(p[1, 63]) == i + 1 for i, p in enumerate(pools))


@gpu
def test_clear():
    pools = make(10)
    want = [p.clone() for p in pools]
    kda.kda_pool_clear(pools, ids([2, -1, 9, 2]))
    for p, w in zip(pools, want):
        w[[2, 9]] = 0
        assert torch.equal(p, w)
    assert kda.kda_get_device_status() == 0
    kda.kda_pool_clear(pools, ids([10, 3]))
    assert kda.kda_get_device_status() == INVALID
    for p, w in zip(pools, want):
        w[3] = 0
        assert torch.equal(p, w)


@gpu
@pytest.mark.parametrize("n_slots,B,ended", [(1, 1, 0.0), (8, 8, 0.0), (8, 8, 0.5), (33, 20, 0.3), (64, 64, 1.0),
                                             (300, 150, 0.4), (5000, 3000, 0.5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(n_slots, B, ended, in_place):
    rng = np.random.RandomState(n_slots + B)
    slots = rng.permutation(n_slots)[:B]
    slots[rng.rand(B) < 0.1] = -1
    done = rng.rand(B) < ended
    pools = make(n_slots) if n_slots <= 300 else [torch.randn(n_slots, 64, device="cuda")]
    want = [p.clone() for p in pools]
    table, flags = ids(slots), torch.tensor(done, device="cuda")
    new = kda.kda_pool_compact(pools, table, flags, out=table if in_place else None)
    expect, moves = ref.compact(slots.tolist(), done.tolist(), n_slots)
    assert new.tolist() == expect
    if not in_place:
        assert table.tolist() == slots.tolist()
    for p, w in zip(pools, want):
        old = w.clone()
        for s, d in moves.items():
            w[d] = old[s]
        assert torch.equal(p, w)
    assert kda.kda_get_device_status() == 0


@gpu
@pytest.mark.parametrize("slots", [[3, 5, 3], [3, 9, 1]])
def test_compact_reports_a_bad_table(slots):
    pools = make(8)
    want = [p.clone() for p in pools]
    new = kda.kda_pool_compact(pools, ids(slots))
    assert kda.kda_get_device_status() == INVALID and new.tolist() == slots
    assert all(torch.equal(p, w) for p, w in zip(pools, want))
    done = torch.tensor([0, 0, 1], dtype=torch.uint8, device="cuda")
    if slots[0] == slots[2]:       # the same slot twice is fine when one of the two ended
        assert kda.kda_pool_compact(pools, ids(slots), done).tolist() == [0, 1, -1]
        assert kda.kda_get_device_status() == 0


@gpu
def test_in_a_graph():
    pools = make(16)
    ref_pools = [p.clone() for p in pools]
    src, dst, table = ids([1, 1]), ids([7, 12]), ids([9, 12, 7, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_pool_copy(pools, src, dst)
        new = kda.kda_pool_compact(pools, table)
    assert all(torch.equal(p, r) for p, r in zip(pools, ref_pools))     # captured, not run
    graph.replay()
    kda.kda_pool_copy(ref_pools, src, dst)
    want = kda.kda_pool_compact(ref_pools, table)
    assert torch.equal(new, want) and all(torch.equal(p, r) for p, r in zip(pools, ref_pools))


# ---------------------------------------------------------------------- pools with slots apart

def pairs_of_layouts(device):
    """Pools of six slots [3, 8, 16], one element type, in the layouts the binding takes: (name, tensor)."""
    z = lambda *s: torch.zeros(*s, device=device)  # noqa: E731
    return [("contiguous", z(6, 3, 8, 16)),
            ("slots of one layer of several", z(6, 2, 3, 8, 16)[:, 1]),
            ("every other slot", z(12, 3, 8, 16)[::2]),
            ("runs apart", z(3, 9, 8, 16).transpose(0, 1)[:6])]


@pytest.mark.parametrize("a", range(4))
@pytest.mark.parametrize("b", range(4))
def test_layouts_of_a_pool_and_its_source_agree(L, a, b):
    """Any two layouts of the same slots are described by the same runs, in both directions, and only split into
    runs where one of the two needs it."""
    (name, to), (_, frm) = pairs_of_layouts("cpu")[a], pairs_of_layouts("cpu")[b]
    d, n_dst, dev = kda._pools([to], "pools", beside=[frm])
    s, n_src, _ = kda._pools([frm], "src_pools", dev, beside=[to])
    assert L.kda_pool_copy(d, s, 1, n_dst, n_src, IX, IX + 64, 0, None) == OK, name
    one_run = 3 not in (a, b)
    for t, bytes_ in ((to, d), (frm, s)):
        base, slot, pieces, apart, run = np.frombuffer(bytes_, np.int64).tolist()
        assert (base, slot) == (t.data_ptr(), t.stride(0) * 4)
        assert (pieces, run) == ((1, 3 * 8 * 16 * 4) if one_run else (3, 8 * 16 * 4))
        assert one_run or apart == t.stride(1) * 4


@gpu
@pytest.mark.parametrize("a", range(4))
@pytest.mark.parametrize("b", range(4))
def test_copy_between_layouts(a, b):
    to, frm = pairs_of_layouts("cuda")[a][1], pairs_of_layouts("cuda")[b][1]
    whole = to._base if to._base is not None else to
    whole.fill_(7.0)
    frm.copy_(torch.randn(frm.shape, device="cuda"))
    want = whole.clone()
    view = want.as_strided(to.shape, to.stride(), to.storage_offset())
    view[4], view[0] = frm[1], frm[5]
    kda.kda_pool_copy([to], ids([1, 5, -1]), ids([4, 0, 2]), src_pools=[frm])
    assert kda.kda_get_device_status() == 0
    assert torch.equal(whole, want)                  # what lies between the slots too


# ---------------------------------------------------------------------- many pairs

@gpu
@pytest.mark.parametrize("n", [1023, 1024, 1025, 5000, 40000])
@pytest.mark.parametrize("within", [True, False])
def test_many_pairs_with_conflicts(n, within):
    """Lists of more than 1024 pairs: destinations that come twice, are read, or lie past the pool, far apart in the
    list, are left out; all others are copied."""
    rng = np.random.RandomState(n)
    n_slots = 3 * n
    order = rng.permutation(n_slots)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    for _ in range(8):
        a, b = rng.choice(n, 2, replace=False)
        dst[a] = dst[b]                                    # one destination twice
        a, b = rng.choice(n, 2, replace=False)
        src[a] = dst[b]                                    # a destination that another pair reads
        dst[rng.randint(n)] = n_slots + rng.randint(100)   # past the pool
        src[rng.randint(n)] = n_slots + rng.randint(100)
        dst[rng.randint(n)] = -1
        a = rng.randint(n)
        src[a] = dst[a]                                    # a slot with itself
    pools = [torch.arange(n_slots * k, dtype=torch.int32, device="cuda").reshape(n_slots, k) for k in (4, 12)]
    source = None if within else [p + 1000000 for p in pools]
    frm = [p.clone() for p in (pools if within else source)]
    want = [p.clone() for p in pools]
    kda.kda_pool_copy(pools, ids(src), ids(dst), src_pools=source)
    used = (src >= 0) & (dst >= 0)
    times = np.bincount(dst[used], minlength=n_slots + 100)
    read = np.zeros(n_slots + 100, bool)
    read[src[used]] = True
    fine = used & (src < n_slots) & (dst < n_slots) & (times[np.maximum(dst, 0)] == 1)
    if within:
        fine &= (src == dst) | ~read[np.maximum(dst, 0)]
    s, d = (torch.tensor(t[fine], device="cuda") for t in (src, dst))
    for p, f, w in zip(pools, frm, want):
        w[d] = f[s]
        assert torch.equal(p, w)
    assert kda.kda_get_device_status() == INVALID          # some were left out


@gpu
def test_the_check_of_many_pairs_is_short():
    """65536 pairs in 16 pools of small slots: the check does not compare every pair with every other for each pool
    (100 ms when it did)."""
    n = 65536
    pools = [torch.zeros(2 * n, 64, device="cuda") for _ in range(16)]
    order = torch.randperm(2 * n, device="cuda").to(torch.int32)
    src, dst = order[:n].contiguous(), order[n:].contiguous()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    kda.kda_pool_copy(pools, src, dst)
    start.record()
    kda.kda_pool_copy(pools, src, dst)
    end.record()
    end.synchronize()
    assert kda.kda_get_device_status() == 0
    assert start.elapsed_time(end) < 20


# ---------------------------------------------------------------------- pools beyond any memory

def test_sizes_that_overflow_are_refused(L):
    """A pool whose size does not fit 64 bits would pass for a small one: its slots and the indices, or another pool,
    would seem apart."""
    stride = 1 << 40
    far = desc((BASE, stride, 1, 0, 1024))
    n = (1 << 24) + 1                                                   # the last slot wraps around to the first
    assert L.kda_pool_clear(far, 1, n, BASE + stride, 4, None) == INVALID
    assert L.kda_pool_copy(far, desc((BASE + stride, 1024, 1, 0, 1024)), 1, n, 8, IX, IX + 64, 4, None) == INVALID
    assert L.kda_pool_clear(far, 1, 2 ** 31 - 1, IX, 0, None) == INVALID
    assert L.kda_pool_clear(desc((BASE, stride, 1 << 20, 1 << 26, 1 << 26)), 1, 1, IX, 0, None) == INVALID
    assert L.kda_pool_clear(desc((BASE, 1 << 38, 1, 0, 1 << 38)), 1, 16, IX + (1 << 44), 0, None) == OK
