"""Fork, compact and truncate: packed rows move byte for byte, the tail holds the newest
tokens (raw, or the cached value rounded once when it had left the tail), shared pages
are copied before they are written, and the pool gets back what nobody holds."""
import ctypes

import numpy as np
import pytest
import torch

from quantized_kv_cache_15_b200 import kvq
from tests.seqkit import VARIANTS, Kit

gpu = pytest.mark.gpu


def same_packed(a, b, rows_a=None, rows_b=None):
    assert a.keys() == b.keys()
    for key in a:
        x = a[key] if rows_a is None else a[key][rows_a]
        y = b[key] if rows_b is None else b[key][rows_b]
        np.testing.assert_array_equal(x, y, err_msg=str(key))


def expected_after(kit, values, packed, keep):
    """What the sequence holds when only the positions `keep` of it are kept."""
    n, m = values[0].shape[1], len(keep)
    keep = np.asarray(keep, np.int64)
    old, cut = max(0, n - kit.T), max(0, m - kit.T)
    idx = torch.from_numpy(keep).cuda()
    vals = []
    for x in values:
        y = x[:, idx]
        back = torch.from_numpy((np.arange(m) >= cut) & (keep < old)).cuda()
        vals.append(torch.where(back[None, :, None, None], y.to(kit.dt).float(), y))
    return vals, {k: p[keep[:cut]] for k, p in packed.items()}


def check(kit, seq, vals, packed):
    got = kit.values(seq)
    for kv in range(2):
        assert torch.equal(got[kv], vals[kv])
    same_packed(kit.packed(seq), packed)


@gpu
@pytest.mark.parametrize("name", list(VARIANTS))
@pytest.mark.parametrize("n", [1, 63, 64, 65, 200, 333])
def test_fork_then_append_matches_separate_sequences(name, n):
    """Two forks and their source continue differently; each holds exactly what a sequence
    that was appended to alone holds."""
    a = Kit(seed=3, **VARIANTS[name])
    ref = Kit(seed=3, **VARIANTS[name])
    prompt = a.fill(0, n)
    ref.rows(n)
    a.plan.fork(0, [2, 1])
    more = {s: a.rows(c) for s, c in ((0, 1), (1, 130), (2, 7))}
    for s in (1, 0, 2):
        a.append(s, more[s])
    for s in range(3):
        ref.append(s, prompt)
        ref.append(s, more[s])
        assert a.length(s) == ref.length(s)
        same_packed(a.packed(s), ref.packed(s))
        for x, y in zip(a.values(s), ref.values(s)):
            assert torch.equal(x, y)
    q = a.queries(3)
    assert torch.equal(a.decode(0, [0, 1, 2], q), ref.decode(0, [0, 1, 2], q))


@gpu
def test_pages_are_counted_once_and_come_back():
    kit = Kit(layers=1, seqs=4, max_tokens=640, max_pages=11)
    kit.fill(0, 200)                                     # 4 pages, the last one partly filled
    one = kit.plan.bytes_in_use()
    kit.plan.fork(0, [1, 2, 3])
    assert kit.plan.bytes_in_use() == one
    before = kit.values(0)
    kit.append(1, kit.rows(1))                           # its own copy of the last page
    assert kit.plan.bytes_in_use() == one * 5 // 4
    kit.plan.seq_reset(0)
    assert kit.plan.bytes_in_use() == one * 5 // 4
    for x, y in zip(before, kit.values(2)):
        assert torch.equal(x, y)
    kit.append(2, kit.rows(1))
    kit.append(3, kit.rows(1))                           # the last holder writes in place
    assert kit.plan.bytes_in_use() == one * 6 // 4
    for s in (1, 2, 3):
        kit.plan.seq_reset(s)
    assert kit.plan.bytes_in_use() == 0
    kit.fill(0, 640)
    assert kit.plan.bytes_in_use() == one * 10 // 4


@gpu
def test_append_to_a_shared_page_needs_a_free_page():
    kit = Kit(layers=1, seqs=3, max_tokens=128, max_pages=2)
    kit.fill(0, 100)
    kit.plan.fork(0, [1, 2])
    before = kit.values(0)
    with pytest.raises(kvq.KVQError) as e:
        kit.append(1, kit.rows(1))
    assert e.value.status == 3 and kit.length(1) == 100
    for x, y in zip(before, kit.values(1)):
        assert torch.equal(x, y)
    kit.plan.seq_reset(0)
    kit.plan.seq_reset(2)
    kit.append(1, kit.rows(1))                           # alone again: nothing to copy
    assert kit.length(1) == 101


@gpu
def test_two_forks_in_one_append_share_the_last_copy():
    """Both holders of a page append in one call: one copies, the other keeps the page."""
    kit = Kit(layers=1, seqs=2, max_tokens=128, max_pages=3)
    kit.fill(0, 100)
    kit.plan.fork(0, [1])
    r = kit.rows(2)
    before = kit.values(0)
    kit.plan.append(0, [0, 1], [1, 1], r[0][0].contiguous(), r[1][0].contiguous())
    ref = Kit(layers=1, seqs=2, max_tokens=128)
    ref.plan.append(0, [0, 1], [1, 1], r[0][0].contiguous(), r[1][0].contiguous())
    for s in range(2):
        got, one = kit.values(s), ref.values(s)
        for kv in range(2):
            assert torch.equal(got[kv][:, :100], before[kv]) and torch.equal(got[kv][:, 100:], one[kv])


@gpu
def test_fork_between_two_layers_of_a_step():
    """Layers of different lengths: a page that is full in one layer and open in another."""
    a, ref = Kit(seed=5), Kit(seed=5)
    r = a.rows(64)
    ref.rows(64)
    a.append(0, r, layers=[0])
    a.append(0, [x[:, :40] for x in r], layers=[1])
    a.plan.fork(0, [1])
    a.append(1, [x[:, 40:] for x in r], layers=[1])
    a.append(0, [x[:, 40:50] for x in r], layers=[1])
    ref.append(0, r)
    for x, y in zip(a.values(1), ref.values(0)):
        assert torch.equal(x, y)
    assert a.plan.seq_length(0, 1) == 50


KEEPS = {
    "all": lambda n, r: list(range(n)),
    "none": lambda n, r: [],
    "first": lambda n, r: [0],
    "last": lambda n, r: [n - 1],
    "drop_first": lambda n, r: list(range(1, n)),
    "even": lambda n, r: list(range(0, n, 2)),
    "random": lambda n, r: sorted(r.choice(n, (2 * n + 2) // 3, replace=False).tolist()),
    "few": lambda n, r: sorted(r.choice(n, max(1, n // 9), replace=False).tolist()),
}


@gpu
@pytest.mark.parametrize("name", list(VARIANTS))
@pytest.mark.parametrize("n", [1, 64, 97, 193, 450])
@pytest.mark.parametrize("which", list(KEEPS))
def test_compact_keeps_rows(name, n, which):
    kit = Kit(seed=7, **VARIANTS[name])
    kit.fill(0, n)
    kit.fill(1, 70)
    other = kit.values(1)
    keep = KEEPS[which](n, np.random.default_rng(n))
    vals, packed = expected_after(kit, kit.values(0), kit.packed(0), keep)
    kit.plan.compact([0], [0], [len(keep)], torch.tensor(keep, dtype=torch.int32, device="cuda"))
    assert [kit.plan.seq_length(0, l) for l in range(kit.L)] == [len(keep)] * kit.L
    check(kit, 0, vals, packed)
    for x, y in zip(other, kit.values(1)):
        assert torch.equal(x, y)
    # the sequence goes on
    more = kit.rows(75)
    kit.append(0, more)
    assert kit.length(0) == len(keep) + 75
    last = min(75, kit.T)
    if last:
        for x, y in zip(kit.values(0), more):
            assert torch.equal(x[:, -last:], y[:, -last:].float())


@gpu
@pytest.mark.parametrize("name", list(VARIANTS))
@pytest.mark.parametrize("n,m", [(1, 0), (65, 64), (200, 199), (200, 129), (333, 60), (450, 0), (100, 100), (450, 300)])
def test_truncate(name, n, m):
    kit = Kit(seed=9, **VARIANTS[name])
    kit.fill(0, n)
    vals, packed = expected_after(kit, kit.values(0), kit.packed(0), list(range(m)))
    kit.plan.truncate([0], [m])
    check(kit, 0, vals, packed)
    free = Kit(seed=9, **VARIANTS[name])
    free.fill(0, m)
    assert kit.plan.bytes_in_use() == free.plan.bytes_in_use()


@gpu
@pytest.mark.parametrize("tail", [0, 64])
def test_compact_batch_with_starts(tail):
    """Several sequences in one call, each with its own untouched front; one keeps nothing behind it."""
    kit = Kit(seed=11, tail=tail, seqs=5)
    rng = np.random.default_rng(1)
    sizes = [300, 128, 5, 450, 64]
    for s, n in enumerate(sizes):
        kit.fill(s, n)
    starts = [100, 128, 0, 449, 10]
    keeps = [sorted(rng.choice(np.arange(100, 300), 77, replace=False).tolist()), [], [1, 3], [449], [63]]
    want = [expected_after(kit, kit.values(s), kit.packed(s), list(range(starts[s])) + keeps[s]) for s in range(5)]
    order = [3, 0, 4, 1, 2]
    flat = sum((keeps[s] for s in order), [])
    kit.plan.compact(order, [starts[s] for s in order], [len(keeps[s]) for s in order],
                     torch.tensor(flat, dtype=torch.int32, device="cuda"))
    for s in range(5):
        check(kit, s, *want[s])


@gpu
@pytest.mark.parametrize("spare", [1, 2, 3])
def test_compact_with_few_free_pages(spare):
    """Pages are handed on during the call: one free page is enough."""
    n = 640
    roomy = Kit(seed=13, layers=1, seqs=2, max_tokens=n)
    tight = Kit(seed=13, layers=1, seqs=2, max_tokens=n, max_pages=10 + spare)
    keep = [i for i in range(n) if i % 7]
    k = torch.tensor(keep, dtype=torch.int32, device="cuda")
    for kit in (roomy, tight):
        kit.fill(0, n)
        kit.plan.compact([0], [0], [len(keep)], k)
    same_packed(tight.packed(0), roomy.packed(0))
    assert tight.plan.bytes_in_use() == roomy.plan.bytes_in_use()
    full = Kit(seed=13, layers=1, seqs=2, max_tokens=n, max_pages=10)
    full.fill(0, n)
    before = full.packed(0)
    with pytest.raises(kvq.KVQError) as e:
        full.plan.compact([0], [0], [len(keep)], k)
    assert e.value.status == 3 and full.length(0) == n
    same_packed(full.packed(0), before)


@gpu
@pytest.mark.parametrize("name", ["q4", "kvarn_tail"])
def test_compacting_a_fork_leaves_its_source(name):
    kit = Kit(seed=15, **VARIANTS[name])
    kit.fill(0, 400)
    vals, packed = kit.values(0), kit.packed(0)
    kit.plan.fork(0, [1])
    keep = list(range(5, 400, 3))
    want = expected_after(kit, vals, packed, keep)
    kit.plan.compact([1], [0], [len(keep)], torch.tensor(keep, dtype=torch.int32, device="cuda"))
    check(kit, 1, *want)
    check(kit, 0, vals, packed)
    kit.plan.truncate([0], [130])
    check(kit, 1, *want)
    kit.append(0, kit.rows(80))
    check(kit, 1, *want)


@gpu
def test_bad_keep_list_is_reported_and_contained():
    kit = Kit(seed=17, tail=64)
    kit.fill(0, 300)
    kit.fill(1, 300)
    other = kit.values(1)
    for bad in ([5, 4, 9], [0, 0, 1], [1, 2, 300], [-1, 3, 4], [2**31 - 1, 2, 3], [3, 2**31 - 1, 4]):
        kit.plan.fork(1, [2])
        kit.plan.compact([2], [0], [3], torch.tensor(bad, dtype=torch.int32, device="cuda"))
        with pytest.raises(kvq.KVQError) as e:
            kit.plan.check_device_error()
        assert e.value.status == 6
        kit.plan.seq_reset(2)
    for x, y in zip(other, kit.values(1)):
        assert torch.equal(x, y)


@gpu
def test_refusals_enqueue_nothing():
    kit = Kit(seed=19, tail=64)
    kit.fill(0, 100)
    kit.fill(1, 10)
    before = kit.values(0)
    L = kvq.lib()
    launches = kvq.launch_count()
    k = torch.zeros(4, dtype=torch.int32, device="cuda")

    def status(f, *args):
        try:
            f(*args)
        except kvq.KVQError as e:
            return e.status
        return 0

    p = kit.plan
    assert status(p.fork, 0, [1]) == 8                   # the destination holds tokens
    assert status(p.fork, 0, [0]) == 1
    assert status(p.fork, 0, [2, 2]) == 1
    assert status(p.fork, 0, [4]) == 1
    assert status(p.fork, -1, [2]) == 1
    assert status(p.fork, 0, [2] * 257) == 1
    assert status(p.compact, [0, 0], [0, 0], [1, 1], k) == 1
    assert status(p.compact, [0], [0], [101], torch.zeros(101, dtype=torch.int32, device="cuda")) == 1
    assert status(p.compact, [0], [101], [0], k) == 1
    assert status(p.compact, [0], [-1], [1], k) == 1
    assert status(p.compact, [0], [0], [-1], k) == 1
    assert status(p.compact, [0], [0], [1], None) == 1
    assert status(p.truncate, [0], [101]) == 1
    assert status(p.truncate, [0], [-1]) == 1
    assert status(p.truncate, [7], [0]) == 1
    ids = (ctypes.c_int * 1)(0)
    assert L.kvq_seq_compact(p.handle, 1, ids, (ctypes.c_int64 * 1)(0), None, None, None) == 1
    assert L.kvq_seq_compact(p.handle, 1, ids, None, (ctypes.c_int * 1)(1), k.data_ptr(), None) == 1
    assert L.kvq_seq_compact(p.handle, 1, ids, (ctypes.c_int64 * 1)(0), (ctypes.c_int * 1)(1), k.data_ptr() + 2, None) == 1
    assert L.kvq_seq_fork(p.handle, 0, 1, None, None) == 1
    for bad in (dict(start=[0, 0]), dict(n_keep=[1, 1]), dict(keep=k.long()), dict(keep=k[::2])):
        a = dict(start=[0], n_keep=[3], keep=k)
        a.update(bad)
        with pytest.raises(ValueError):
            p.compact([0], **a)
    p.fork(0, [])
    p.compact([], [], [], None)
    assert kvq.launch_count() == launches
    kit.append(1, kit.rows(1), layers=[0])               # the layers differ now
    launches = kvq.launch_count()
    assert status(p.truncate, [1], [5]) == 8
    assert kvq.launch_count() == launches
    unbound = kvq.Plan(1, 8, 2, max_seqs=2, max_tokens_per_seq=64, k_codec=[3, 3], v_codec=[3, 3])
    assert status(unbound.fork, 0, [1]) == 8 and status(unbound.truncate, [0], [0]) == 8
    for x, y in zip(before, kit.values(0)):
        assert torch.equal(x, y)


@gpu
@pytest.mark.parametrize("name", list(VARIANTS))
@pytest.mark.parametrize("n", [1, 63, 64, 65, 129, 300])
def test_saved_rows_load_into_another_plan(name, n):
    """Saved packed rows and raw tail rows come back byte for byte, and the sequence goes on."""
    a, b = Kit(seed=25, **VARIANTS[name]), Kit(seed=25, **VARIANTS[name])
    r = a.fill(0, n)
    b.rows(n)
    b.fill(3, 130)                                       # other pages in use
    nt = min(n, a.T)
    for l in range(a.L):
        tail = [x[l, n - nt:].contiguous() for x in r] if nt else [None, None]
        b.plan.load(l, 1, n - nt, a.read(0, l, 0), a.read(0, l, 1), *tail)
    assert b.length(1) == n
    same_packed(b.packed(1), a.packed(0))
    for x, y in zip(a.values(0), b.values(1)):
        assert torch.equal(x, y)
    more = a.rows(70)
    a.append(0, more)
    b.append(1, more)
    same_packed(b.packed(1), a.packed(0))
    for x, y in zip(a.values(0), b.values(1)):
        assert torch.equal(x, y)


@gpu
def test_load_refusals_and_shared_pages():
    kit = Kit(layers=2, seed=27, tail=64, max_tokens=300)
    kit.fill(0, 200)
    k, v = kit.read(0, 0, 0), kit.read(0, 0, 1)
    t = kit.rows(64)[0][0].contiguous()

    def status(*args, **kw):
        try:
            kit.plan.load(*args, **kw)
        except kvq.KVQError as e:
            return e.status
        return 0

    launches = kvq.launch_count()
    assert status(0, 0, 136, k, v, t, t) == 8            # holds tokens
    assert status(2, 1, 136, k, v, t, t) == 1 and status(0, 4, 136, k, v, t, t) == 1
    assert status(0, 1, 136, k, v) == 1                  # packed rows behind a tail that is not full
    assert status(0, 1, 136, k, v, t[:63].contiguous(), t[:63].contiguous()) == 1
    assert status(0, 1, 136, None, v, t, t) == 1 and status(0, 1, 136, (k[0], None), v, t, t) == 1
    assert status(0, 1, -1, k, v, t, t) == 1
    big = (torch.zeros(237 * 128, dtype=torch.uint8, device="cuda"), torch.zeros(237 * 16, dtype=torch.uint8, device="cuda"))
    assert status(0, 1, 237, big, big, t, t) == 3
    for bad in (dict(k=(k[0][:100], k[1])), dict(k=(k[0].int(), k[1])), dict(k_tail=t.float()), dict(v_tail=t[:5])):
        a = dict(layer=0, seq=1, n_rows=136, k=k, v=v, k_tail=t, v_tail=t)
        a.update(bad)
        with pytest.raises(ValueError):
            kit.plan.load(**a)
    assert status(0, 1, 0) == 0
    assert kvq.launch_count() == launches and kit.length(1) == 0
    # a fork of a sequence whose second layer is still empty: its pages are copied before they are written
    part = Kit(layers=2, seed=29, tail=0, max_tokens=300)
    r = part.rows(100)
    part.append(0, r, layers=[0])
    part.plan.fork(0, [1])
    one = Kit(layers=2, seed=29, tail=0, max_tokens=300)
    one.append(0, one.rows(100))
    part.plan.load(1, 1, 100, one.read(0, 1, 0), one.read(0, 1, 1))
    for x, y in zip(part.values(1), one.values(0)):
        assert torch.equal(x, y)
    part.append(0, [x.flip(1) for x in r], layers=[1])
    for x, y in zip(part.values(1), one.values(0)):
        assert torch.equal(x, y)


@gpu
def test_another_stream():
    """Everything on one side stream, with no synchronisation in between."""
    a, ref = Kit(seed=21, tail=64), Kit(seed=21, tail=64)
    r, more = a.rows(200), a.rows(20)
    keep = torch.tensor(list(range(0, 220, 2)), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a.append(0, r, stream=s)
    a.plan.fork(0, [1], stream=s)
    a.append(1, more, stream=s)
    a.plan.compact([1], [0], [110], keep, stream=s)
    s.synchronize()
    ref.append(0, r)
    ref.append(1, r)
    ref.append(1, more)
    want = expected_after(ref, ref.values(1), ref.packed(1), list(range(0, 220, 2)))
    check(a, 1, *want)
    for x, y in zip(a.values(0), ref.values(0)):
        assert torch.equal(x, y)


@gpu
def test_regrade_and_reset_with_shared_pages():
    kit, ref = Kit(seed=23, k=kvq.Q8_0, v=kvq.Q8_0), Kit(seed=23, k=kvq.Q8_0, v=kvq.Q8_0)
    r = kit.fill(0, 150)
    ref.append(0, r)
    kit.plan.fork(0, [1])
    for x in (kit, ref):
        s = torch.empty(x.plan.regrade_bytes(1, [3, 3], [5, 5]), dtype=torch.uint8, device="cuda")
        x.plan.regrade(1, [3, 3], [5, 5], s)
    same_packed(kit.packed(1), ref.packed(0))
    keep = torch.tensor([3, 77, 149], dtype=torch.int32, device="cuda")
    kit.plan.compact([1], [0], [3], keep)                # the every-layer tables follow the regrade
    same_packed(kit.packed(1), ref.packed(0), None, [3, 77, 149])


def test_null_plan_is_refused_without_a_gpu():
    L = kvq.lib()
    one = (ctypes.c_int * 1)(0)
    assert L.kvq_seq_fork(None, 0, 1, one, None) == 1
    assert L.kvq_seq_load(None, 0, 0, 0, None, None, None, None, 0, None, None, None) == 1
    assert L.kvq_seq_truncate(None, 1, one, (ctypes.c_int64 * 1)(0), None) == 1
    assert L.kvq_seq_compact(None, 1, one, (ctypes.c_int64 * 1)(0), one, None, None) == 1


@gpu
@pytest.mark.parametrize("tail", [0, 64, 128])
def test_bad_keep_list_reads_no_other_sequence(tail):
    """A list out of order whose first entry is a token of the raw tail, on an id that held more pages
    before: the stale ends of its block table name pages that another sequence owns by now."""
    kit = Kit(seed=33, layers=1, seqs=3, tail=tail)
    kit.fill(2, 640)
    kit.plan.seq_reset(2)
    kit.fill(1, 640)
    n = tail + 136
    kit.fill(2, n)
    other = {key: {bytes(r) for r in rows} for key, rows in kit.packed(1).items()}
    mine = {key: {bytes(r) for r in rows} for key, rows in kit.packed(2).items()}
    values = kit.values(1)
    bad = [n - 1] + list(range(5, 5 + tail + 80 - 1))
    kit.plan.compact([2], [0], [len(bad)], torch.tensor(bad, dtype=torch.int32, device="cuda"))
    with pytest.raises(kvq.KVQError) as e:
        kit.plan.check_device_error()
    assert e.value.status == 6
    for key, rows in kit.packed(2).items():
        for r in rows:
            assert bytes(r) not in other[key] - mine[key]
    for x, y in zip(values, kit.values(1)):
        assert torch.equal(x, y)
