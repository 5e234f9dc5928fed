"""Attention of several new tokens per sequence over the cache, against softmax attention
in 64 bits over the rows that kvq_dequantize returns.

Tolerance of one output channel c of a row (w: softmax weights, y: the rows in the stored
basis, v: the original one, mul: the variance multipliers), in the order of size:
  eps/2 |o|                 the output's rounding;
  2^-11 mul_c |sum_t w |y_t||_2      values enter the products rounded once to fp16 (bf16 rows
                            as they are): an error of 2^-11 |y| a channel, taken through an
                            orthogonal transform;
  4 ds sum_t w |v_t|        ds = 2^-19 |q s_k| max|k_t / s_k| scale: the query as two fp16
                            halves (2^-21 a product), fp32 sums, the SFU's 2^x; numerator and
                            denominator each move by 2 ds;
  2^-18 mul_c |sum_t w |y_t||_2      weights as two halves, fp32 sums, and the transforms' own
                            fp32 rounding on both sides.
"""
import ctypes

import numpy as np
import pytest
import torch

from quantized_kv_cache_15_b200 import kvq
from tests.seqkit import D, VARIANTS, Kit

gpu = pytest.mark.gpu


def hadamard():
    h = torch.ones((1, 1), dtype=torch.float64)
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return (h / np.sqrt(128.0)).cuda()


def visible(n, nq, bits):
    see = torch.ones((nq, n), dtype=torch.bool)
    for i in range(nq):
        for j in range(nq):
            see[i, n - nq + j] = (j <= i) if bits is None else bool((int(bits[i]) >> j) & 1)
    return see.cuda()


def reference(kit, layer, seq, q, bits=None, values=None):
    """(out, tolerance) in 64 bits, [nq][hq][128], of the sequence's last nq tokens."""
    nq = q.shape[0]
    k, v = [x[layer].double() for x in (kit.values(seq) if values is None else values)]
    see = visible(k.shape[0], nq, bits)
    G, R = kit.hq // kit.hkv, hadamard()
    one = torch.ones((kit.hkv, D), dtype=torch.float64, device="cuda")
    muls = [one, one] if kit.inv is None else [1.0 / torch.from_numpy(kit.inv[layer, :, i]).double().cuda() for i in (0, 1)]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    eps = torch.finfo(kit.dt).eps
    for h in range(kit.hkv):
        qh = q[:, h * G:(h + 1) * G].double()
        s = torch.einsum("igd,td->igt", qh, k[:, h]) / np.sqrt(128.0)
        s = s.masked_fill(~see[:, None], -np.inf)
        w = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
        o = torch.einsum("igt,td->igd", w, torch.nan_to_num(v[:, h], nan=0.0, posinf=0.0, neginf=0.0))
        mk, mv = muls[0][h], muls[1][h]
        y = (torch.nan_to_num(v[:, h], nan=0.0, posinf=0.0, neginf=0.0) / mv) @ R
        wide = torch.einsum("igt,td->igd", w, y.abs()).norm(dim=-1, keepdim=True) * mv
        raw = torch.einsum("igt,td->igd", w, torch.nan_to_num(v[:, h], nan=0.0, posinf=0.0, neginf=0.0).abs())
        ds = 2.0 ** -19 * (qh * mk).norm(dim=-1, keepdim=True) * (torch.nan_to_num(k[:, h]) / mk).norm(dim=-1).max() / np.sqrt(128.0)
        out[:, h * G:(h + 1) * G] = o
        tol[:, h * G:(h + 1) * G] = eps / 2 * o.abs() + (2.0 ** -11 + 2.0 ** -18) * wide + 4 * ds * raw + 2.0 ** -25
    return out, tol


def extend(kit, layer, seqs, nqs, q, mask=None, stream=None, ws=None):
    out = torch.full_like(q, 77.0)
    ws = kit.plan.new_extend_workspace(len(seqs), sum(nqs)).fill_(255) if ws is None else ws
    kit.plan.extend(layer, seqs, nqs, q, out, ws, tree_mask=mask, stream=stream)
    torch.cuda.synchronize()
    kit.plan.check_device_error()
    return out


def check(kit, layer, seqs, nqs, q, got, bits=None):
    i = 0
    for s, n in zip(seqs, nqs):
        if n == 0:
            continue
        ref, tol = reference(kit, layer, s, q[i:i + n], None if bits is None else bits[i:i + n])
        err = (got[i:i + n].double() - ref).abs()
        assert bool((err <= tol).all()), (s, n, float((err / tol).max()))
        i += n


def tree(rng, n):
    rows = []
    for i in range(n):
        par = int(rng.integers(max(-1, i - 3), i)) if i else -1
        rows.append((1 << i) | (rows[par] if par >= 0 else 0))
    return rows


def words(bits):
    return torch.tensor([b - (1 << 64) if b >= 1 << 63 else b for b in bits], dtype=torch.int64, device="cuda")


@gpu
@pytest.mark.parametrize("name", list(VARIANTS))
@pytest.mark.parametrize("masked", [False, True])
def test_ragged_batch(name, masked):
    kit = Kit(seed=31, seqs=7, **VARIANTS[name])
    rng = np.random.default_rng(5)
    sizes, nqs = [1, 64, 65, 127, 300, 513, 40], [1, 3, 0, 17, 2, 9, 40]
    for s, n in enumerate(sizes):
        kit.fill(s, n)
    order = [5, 0, 3, 2, 6, 1, 4]
    nq = [nqs[s] for s in order]
    q = kit.queries(sum(nq))
    bits = sum((tree(rng, n) for n in nq), []) if masked else None
    for layer in (0, 1):
        got = extend(kit, layer, order, nq, q, words(bits) if masked else None)
        check(kit, layer, order, nq, q, got, bits)


@gpu
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (6, 2), (8, 2), (5, 1), (12, 2), (7, 1), (16, 2), (96, 32)])
@pytest.mark.parametrize("nq", [1, 5, 64])
def test_head_groupings(hq, hkv, nq):
    kit = Kit(layers=1, hq=hq, hkv=hkv, seqs=2, seed=33, tail=64)
    kit.fill(0, 331)
    kit.fill(1, 64 + nq)
    q = kit.queries(2 * nq)
    check(kit, 0, [0, 1], [nq, nq], q, extend(kit, 0, [0, 1], [nq, nq], q))


@gpu
@pytest.mark.parametrize("name", list(VARIANTS))
@pytest.mark.parametrize("nq", [4, 8, 16, 33])
def test_wide_units(name, nq):
    """So much work that units take 16, 32 and 64 rows (33 queries: more than one block of them)."""
    kit = Kit(seed=37, seqs=16, **dict(VARIANTS[name], max_tokens=2800))
    rng = np.random.default_rng(nq)
    for s in range(16):
        kit.fill(s, int(rng.integers(2300, 2700)))
    nqs = [int(rng.integers(max(1, nq - 3), nq + 1)) for _ in range(16)]
    q = kit.queries(sum(nqs))
    bits = sum((tree(rng, n) for n in nqs), []) if nq == 16 else None
    check(kit, 1, list(range(16)), nqs, q, extend(kit, 1, list(range(16)), nqs, q, words(bits) if bits else None), bits)


ALL = [kvq.Q8_0, kvq.Q6_0, kvq.Q5_0, kvq.Q4_0, kvq.Q3_0, kvq.Q2_0, kvq.Q8_1, kvq.Q6_1, kvq.Q5_1, kvq.Q4_1, kvq.Q3_1,
       kvq.Q2_1, kvq.F16]


@gpu
@pytest.mark.parametrize("rot", [kvq.ROT_NONE, kvq.ROT_HADAMARD, kvq.ROT_VARNORM_HADAMARD])
@pytest.mark.parametrize("i", range(len(ALL)))
def test_every_codec(rot, i):
    """Each codec once for the keys and once for the values of some head."""
    kit = Kit(layers=1, hq=8, hkv=2, seqs=1, seed=35 + i, rot=rot, k=[ALL[i], ALL[(i + 5) % 13]],
              v=[ALL[(i + 8) % 13], ALL[i]])
    kit.fill(0, 403)
    q = kit.queries(6)
    check(kit, 0, [0], [6], q, extend(kit, 0, [0], [6], q))


@gpu
@pytest.mark.parametrize("n,nq", [(5, 5), (64, 64), (65, 65), (200, 200), (700, 333), (129, 1), (128, 2)])
@pytest.mark.parametrize("tail", [0, 64, 256])
def test_chunks_up_to_the_whole_sequence(n, nq, tail):
    kit = Kit(layers=1, seqs=1, seed=37, tail=tail)
    kit.fill(0, n)
    q = kit.queries(nq)
    check(kit, 0, [0], [nq], q, extend(kit, 0, [0], [nq], q))


@gpu
@pytest.mark.parametrize("tail", [0, 64])
@pytest.mark.parametrize("n", [3, 70, 64, 200])
def test_masks_that_leave_rows_empty(tail, n):
    """A token that sees none of the new tokens sees the prefix; with no prefix, nothing: zeros."""
    kit = Kit(layers=1, seqs=1, seed=39, tail=tail)
    kit.fill(0, n)
    nq = min(n, 64)
    rng = np.random.default_rng(n)
    bits = [int(x) & ((1 << nq) - 1) for x in rng.integers(0, 1 << 63, nq, dtype=np.int64)]
    bits[0] = 0
    bits[nq // 2] = 0
    bits[-1] |= 1 << (nq - 1)
    q = kit.queries(nq)
    got = extend(kit, 0, [0], [nq], q, words(bits))
    check(kit, 0, [0], [nq], q, got, bits)
    if n == nq:
        assert not got[0].any() and not got[nq // 2].any()


@gpu
@pytest.mark.parametrize("bf16", [False, True])
def test_bits_above_the_last_token_are_ignored(bf16):
    kit = Kit(layers=1, seqs=1, seed=41, tail=64, bf16=bf16)
    kit.fill(0, 150)
    q = kit.queries(5)
    bits = [0b1, 0b11, 0b101, 0b1001, 0b10111]
    a = extend(kit, 0, [0], [5], q, words(bits))
    b = extend(kit, 0, [0], [5], q, words([x | (0x7ffffff << 5) | (1 << 63) for x in bits]))
    assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["k", "v", "both"])
def test_non_finite_rows_reach_only_those_who_see_them(bf16, bad, where):
    """A drafted token whose raw rows hold NaN or infinity: rows that mask it are as if it were finite."""
    kit = Kit(layers=1, seqs=1, seed=43, tail=64, bf16=bf16)
    kit.fill(0, 90)
    r = kit.rows(6)
    if where in ("k", "both"):
        r[0][:, 2, :, 5] = bad
    if where in ("v", "both"):
        r[1][:, 2, :, 7] = bad
    kit.append(0, r)
    q = kit.queries(6)
    bits = [0b1, 0b11, 0b111, 0b1011, 0b10001, 0b111011]
    got = extend(kit, 0, [0], [6], q, words(bits))
    ref, tol = reference(kit, 0, 0, q, bits)
    for i in (0, 1, 3, 4, 5):
        assert bool(((got[i].double() - ref[i]).abs() <= tol[i]).all()), i
    if where == "v":                                     # whoever sees it does not get a finite channel 7
        assert not torch.isfinite(got[2, :, 7]).any()


@gpu
def test_a_non_finite_query_stays_in_its_row():
    kit = Kit(layers=1, seqs=2, seed=45, tail=64)
    kit.fill(0, 300)
    kit.fill(1, 200)
    q = kit.queries(6)
    want = extend(kit, 0, [0, 1], [3, 3], q)
    q2 = q.clone()
    q2[1, 3, 9] = float("nan")
    q2[4, 0, 100] = float("inf")
    got = extend(kit, 0, [0, 1], [3, 3], q2)
    hit = torch.zeros((6, kit.hq), dtype=torch.bool, device="cuda")
    hit[1, 3] = hit[4, 0] = True
    assert torch.equal(got[~hit], want[~hit])
    assert not torch.isfinite(got[1, 3]).any()


@gpu
@pytest.mark.parametrize("scale", [1e-4, 1.0, 100.0, 2000.0])
def test_large_and_small_values(scale):
    kit = Kit(layers=1, seqs=1, seed=47, tail=64, spread=5.0)
    rows = [(x.float() * scale).to(kit.dt) for x in kit.rows(200)]
    rows[0] = (rows[0].float() / max(1.0, scale)).to(kit.dt)
    kit.append(0, rows)
    q = kit.queries(4)
    got = extend(kit, 0, [0], [4], q)
    ref, tol = reference(kit, 0, 0, q)
    # below fp16's normal range a rounding is half of 2^-24, in the output and in each value
    assert bool(((got.double() - ref).abs() <= tol + 2.0 ** -25 * (1 + np.sqrt(128.0))).all())


@gpu
def test_rising_scores_rescale_the_sum():
    """Keys that grow along the sequence: the running maximum moves in every tile."""
    kit = Kit(layers=1, seqs=1, seed=49, max_tokens=2000, spread=1.0, tail=128)
    base = torch.randn((1, 1, 2, D), device="cuda")
    up = torch.linspace(0.02, 3.0, 1900, device="cuda").reshape(1, -1, 1, 1)
    k = (base * up).to(kit.dt)
    kit.append(0, [k, kit.rows(1900)[1]])
    q = base[0].reshape(1, 2, 1, D).expand(1, 2, 4, D).reshape(1, 8, D).to(kit.dt).contiguous()
    q = torch.cat([q, -q, 2 * q])
    check(kit, 0, [0], [3], q, extend(kit, 0, [0], [3], q))


@gpu
@pytest.mark.parametrize("name", ["q4", "kvarn_tail", "bf16_q41_tail", "rank_tail"])
@pytest.mark.parametrize("n,forks,nq", [(256, 2, 1), (300, 3, 1), (450, 5, 4), (600, 8, 2), (520, 20, 3)])
def test_forks_share_their_prompt(name, n, forks, nq):
    kit = Kit(seed=51, seqs=forks + 3, max_tokens=700, **VARIANTS[name])
    kit.fill(0, n)
    kit.plan.fork(0, list(range(1, forks)))
    kit.fill(forks, 280)                                 # a second family, and a sequence of its own
    kit.plan.fork(forks, [forks + 1])
    kit.fill(forks + 2, 100)
    rng = np.random.default_rng(n)
    for s in range(forks):
        kit.append(s, kit.rows(nq + int(rng.integers(0, 70))))
    kit.append(forks + 1, kit.rows(nq))
    seqs = [int(s) for s in rng.permutation(forks + 3)]
    nqs = [int(rng.integers(1, nq + 1)) for _ in seqs]
    q = kit.queries(sum(nqs))
    for layer in (0, 1):
        check(kit, layer, seqs, nqs, q, extend(kit, layer, seqs, nqs, q))


@gpu
@pytest.mark.parametrize("name", list(VARIANTS))
@pytest.mark.parametrize("n,forks,nq", [(1700, 2, 1), (2300, 5, 4), (2000, 20, 3), (1650, 16, 1)])
def test_forks_share_a_long_prompt(name, n, forks, nq):
    """Prompts long enough to be walked once for all forks, beside a second family and a sequence of its own."""
    kit = Kit(seed=71, seqs=forks + 4, **dict(VARIANTS[name], max_tokens=2500))
    kit.fill(0, n)
    kit.plan.fork(0, list(range(1, forks)))
    kit.fill(forks, 1800)
    kit.plan.fork(forks, [forks + 1, forks + 2])
    kit.fill(forks + 3, 1900)
    rng = np.random.default_rng(n)
    for s in range(forks):
        kit.append(s, kit.rows(nq + int(rng.integers(0, 70))))
    kit.append(forks + 1, kit.rows(nq))
    seqs = [int(s) for s in rng.permutation(forks + 4)]
    nqs = [int(rng.integers(1, nq + 1)) for _ in seqs]
    q = kit.queries(sum(nqs))
    check(kit, 1, seqs, nqs, q, extend(kit, 1, seqs, nqs, q))


@gpu
@pytest.mark.parametrize("kw", [dict(), dict(rot=kvq.ROT_VARNORM_HADAMARD, tail=256), dict(rot=kvq.ROT_PROJECTION, tail=64),
                                dict(bf16=True, k=kvq.Q4_1, v=kvq.Q5_0, tail=128), dict(k=kvq.Q8_0, v=kvq.Q3_0)])
@pytest.mark.parametrize("forks,nq", [(16, 1), (20, 3), (9, 4)])
def test_many_forks_of_a_long_prompt(kw, forks, nq):
    """The shared prompt and the forks' own tokens in two launches that overlap: right, inside the
    workspace, the same again, captured, and under memory traffic."""
    kit = Kit(layers=1, hq=32, hkv=8, seed=73, seqs=forks + 1, max_tokens=4000, **kw)
    kit.fill(0, 3300)
    kit.plan.fork(0, list(range(1, forks)))
    kit.fill(forks, 500)
    rng = np.random.default_rng(forks)
    for s in range(forks):
        kit.append(s, kit.rows(nq + int(rng.integers(0, 300))))
    seqs = [int(s) for s in rng.permutation(forks + 1)]
    nqs = [nq] * (forks + 1)
    q = kit.queries(sum(nqs))
    size = kit.plan.extend_workspace_bytes(len(seqs), sum(nqs))
    room = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    before = kvq.launch_count()
    got = extend(kit, 0, seqs, nqs, q, ws=room[:size])
    assert kvq.launch_count() - before == 3
    assert bool((room[size:] == 255).all())
    check(kit, 0, seqs, nqs, q, got)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kit.plan.extend(0, seqs, nqs, q, out, room[:size])
    a, b = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"), torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    busy = torch.cuda.Stream()
    for i in range(8):
        out.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(busy):
            for _ in range(4 * (i % 2)):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got)
    kit.plan.check_device_error()


@gpu
@pytest.mark.parametrize("tail", [0, 64])
@pytest.mark.parametrize("far", [0, 1600])
def test_forks_that_lost_part_of_the_prompt(tail, far):
    """Truncated and compacted forks share less; drafts inside a shared page keep it out of the group."""
    kit = Kit(layers=1, seed=53, seqs=5, tail=tail, max_tokens=700 + far)
    kit.fill(0, 600 + far)
    kit.plan.fork(0, [1, 2, 3, 4])
    kit.plan.truncate([1, 2], [400 + far, 290 + far])
    keep = torch.tensor(list(range(300 + far, 600 + far, 2)), dtype=torch.int32, device="cuda")
    kit.plan.compact([3], [290 + far], [150], keep)
    seqs, nqs = [4, 3, 2, 1, 0], [60, 3, 30, 64, 1]
    q = kit.queries(sum(nqs))
    check(kit, 0, seqs, nqs, q, extend(kit, 0, seqs, nqs, q))


@gpu
def test_one_sequence_several_times():
    kit = Kit(layers=1, seed=55, seqs=2, tail=64)
    kit.fill(0, 500)
    kit.fill(1, 90)
    q = kit.queries(10)
    seqs, nqs = [0, 1, 0, 0], [4, 1, 1, 4]
    got = extend(kit, 0, seqs, nqs, q)
    check(kit, 0, seqs, nqs, q, got)


@gpu
def test_one_new_token_agrees_with_decode():
    kit = Kit(layers=2, seed=57, seqs=4, tail=64, rot=kvq.ROT_VARNORM_HADAMARD)
    for s, n in enumerate((1, 64, 200, 650)):
        kit.fill(s, n)
    q = kit.queries(4)
    a, b = extend(kit, 1, [0, 1, 2, 3], [1] * 4, q).float(), kit.decode(1, [0, 1, 2, 3], q)
    # decode's bar is 2e-3 of a row's largest value; the output's rounding is 2^-11 of it
    assert bool(((a - b).abs() <= (2e-3 + 2.0 ** -11 + 2e-3) * b.abs().amax(-1, keepdim=True)).all())


@gpu
def test_a_long_sequence():
    kit = Kit(layers=1, hq=8, hkv=2, seed=59, seqs=1, max_tokens=140000, tail=256, k=kvq.Q8_0)
    kit.fill(0, 139999)
    q = kit.queries(8)
    check(kit, 0, [0], [8], q, extend(kit, 0, [0], [8], q))


@gpu
@pytest.mark.parametrize("name", ["q4_tail", "rank_tail"])
def test_nothing_outside_the_buffers_is_written_and_results_repeat(name):
    kit = Kit(seed=61, seqs=3, **VARIANTS[name])
    for s, n in enumerate((300, 77, 650)):
        kit.fill(s, n)
    seqs, nqs = [0, 1, 2], [7, 3, 20]
    q = kit.queries(30)
    need = kit.plan.extend_workspace_bytes(3, 30)
    big = torch.full((need + 8192,), 171, dtype=torch.uint8, device="cuda")
    off = 4096 + (-big.data_ptr()) % 16
    outs = torch.full((30 + 8, kit.hq, D), 5.0, dtype=kit.dt, device="cuda")
    got = []
    for _ in range(3):
        kit.plan.extend(0, seqs, nqs, q, outs[4:34], big[off:off + need])
        torch.cuda.synchronize()
        got.append(outs[4:34].clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    assert bool((outs[:4] == 5).all()) and bool((outs[34:] == 5).all())
    assert bool((big[:off] == 171).all()) and bool((big[off + need:] == 171).all())


@gpu
@pytest.mark.parametrize("k,nq", [(kvq.Q4_0, 4), (kvq.Q8_0, 8), (kvq.Q6_0, 3), (kvq.Q4_0, 16)])
def test_results_repeat_under_memory_traffic(k, nq):
    """Pages arrive late while another stream keeps the memory busy; the result stays the same bits."""
    kit = Kit(layers=1, seed=64, seqs=3, max_tokens=40000, tail=256, k=k)
    for s, n in enumerate((39000, 300, 9000)):
        kit.fill(s, n)
    q = kit.queries(3 * nq)
    ws = kit.plan.new_extend_workspace(3, 3 * nq)
    want = extend(kit, 0, [0, 1, 2], [nq] * 3, q, ws=ws)
    check(kit, 0, [0, 1, 2], [nq] * 3, q, want)
    busy, side = torch.empty(1 << 28, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    for _ in range(60):
        with torch.cuda.stream(side):
            busy.add_(1)
        ws.fill_(255)
        kit.plan.extend(0, [0, 1, 2], [nq] * 3, q, out, ws)
        assert torch.equal(out, want)
    kit.plan.check_device_error()


@gpu
def test_captured_and_on_another_stream():
    kit = Kit(layers=2, seed=63, seqs=2, tail=64)
    kit.fill(0, 400)
    kit.fill(1, 650)
    q = kit.queries(9)
    q2 = kit.queries(9)
    bits = words([1, 3, 7, 1, 3, 5, 9, 17, 63])
    want = [extend(kit, l, [0, 1], [3, 6], x, bits) for l, x in ((0, q), (1, q), (0, q2), (1, q2))]
    buf, out = q.clone(), [torch.empty_like(q) for _ in range(2)]
    ws = kit.plan.new_extend_workspace(2, 9)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        for l in range(2):
            kit.plan.extend(l, [0, 1], [3, 6], buf, out[l], ws, tree_mask=bits)
    for x, w in ((q, want[:2]), (q2, want[2:])):
        buf.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])
    torch.cuda.synchronize()
    got = torch.empty_like(q)
    kit.plan.extend(0, [0, 1], [3, 6], q, got, ws, tree_mask=bits, stream=s)
    s.synchronize()
    assert torch.equal(got, want[0])


@gpu
def test_a_speculative_step():
    """Fork, append a tree of drafts, attend, keep the accepted path, go on: as if only the
    accepted tokens had been appended (their rows are still in the raw tail)."""
    kit, ref = Kit(seed=65, tail=64, seqs=3), Kit(seed=65, tail=64, seqs=3)
    prompt = kit.fill(0, 300)
    ref.rows(300)
    ref.append(0, prompt)
    draft = kit.rows(12)
    ref.rows(12)
    kit.plan.fork(0, [1])
    kit.append(1, draft)
    rng = np.random.default_rng(3)
    bits = tree(rng, 12)
    q = kit.queries(12)
    for l in range(2):
        got = extend(kit, l, [1], [12], q, words(bits))
        check(kit, l, [1], [12], q, got, bits)
    path = [i for i in range(12) if (bits[11] >> i) & 1]
    kit.plan.compact([1], [300], [len(path)], torch.tensor([300 + i for i in path], dtype=torch.int32, device="cuda"))
    ref.append(0, [x[:, path].contiguous() for x in draft])
    n = 300 + len(path)
    assert kit.length(1) == n == ref.length(0)
    back = 12 - len(path)                                # the oldest rows of the new tail came back from the pages
    for a, b in zip(kit.values(1), ref.values(0)):
        same = torch.cat([torch.arange(0, n - 64), torch.arange(n - 64 + back, n)]).cuda()
        assert torch.equal(a[:, same], b[:, same])
    kit.plan.seq_reset(0)
    more = kit.rows(3)
    kit.append(1, more)
    q = kit.queries(3)
    check(kit, 1, [1], [3], q, extend(kit, 1, [1], [3], q))


@gpu
def test_refusals_enqueue_nothing():
    kit = Kit(layers=1, seed=67, seqs=2, tail=64)
    kit.fill(0, 100)
    p, L = kit.plan, kvq.lib()
    q = kit.queries(4)
    out = torch.full_like(q, 3.0)
    ws = p.new_extend_workspace(2, 4)
    mask = torch.zeros(4, dtype=torch.int64, device="cuda")
    launches = kvq.launch_count()

    def status(layer=0, n=1, ids=(0,), nq=(4,), m=None, qp=None, op=None, wp=None, wb=None):
        return L.kvq_extend_attention(p.handle, layer, n, (ctypes.c_int * len(ids))(*ids) if ids else None,
                                      (ctypes.c_int * len(nq))(*nq) if nq else None, m,
                                      q.data_ptr() if qp is None else qp, out.data_ptr() if op is None else op,
                                      ws.data_ptr() if wp is None else wp, ws.numel() if wb is None else wb, None)

    assert status(layer=1) == 1 and status(layer=-1) == 1
    assert status(ids=(2,)) == 1 and status(ids=(-1,)) == 1
    assert status(ids=()) == 1 and status(nq=()) == 1
    assert status(nq=(101,)) == 1 and status(nq=(-1,)) == 1
    assert status(n=257) == 1 and status(n=-1) == 1
    assert status(nq=(65,), m=mask.data_ptr()) == 2
    assert status(m=mask.data_ptr() + 4) == 1
    assert status(qp=0) == 1 and status(op=0) == 1 and status(wp=0) == 1
    assert status(qp=q.data_ptr() + 2) == 1 and status(op=out.data_ptr() + 8) == 1 and status(wp=ws.data_ptr() + 4) == 1
    assert status(wb=64) == 1
    assert status(n=0) == 0 and status(nq=(0,)) == 0
    assert kvq.launch_count() == launches and bool((out == 3).all())
    b = ctypes.c_size_t()
    assert L.kvq_plan_extend_workspace_bytes(p.handle, -1, 1, ctypes.byref(b)) == 1
    assert L.kvq_plan_extend_workspace_bytes(p.handle, 1, -1, ctypes.byref(b)) == 1
    assert L.kvq_plan_extend_workspace_bytes(p.handle, 1, 1 << 40, ctypes.byref(b)) == 1
    for bad in (dict(q=q.float()), dict(q=q[:3]), dict(out=out.bfloat16()), dict(tree_mask=mask.int()), dict(tree_mask=mask[:3]),
                dict(n_q=[2, 2])):
        a = dict(layer=0, seq_ids=[0], n_q=[4], q=q, out=out, workspace=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            p.extend(**a)


def test_null_plan_is_refused_without_a_gpu():
    L = kvq.lib()
    one = (ctypes.c_int * 1)(1)
    b = ctypes.c_size_t()
    assert L.kvq_extend_attention(None, 0, 1, one, one, None, None, None, None, 0, None) == 1
    assert L.kvq_plan_extend_workspace_bytes(None, 1, 1, ctypes.byref(b)) == 1


@gpu
@pytest.mark.parametrize("hq,hkv", [(4, 2), (8, 2), (32, 8)])
def test_workspace_sizes_beyond_any_call_are_refused(hq, hkv):
    """Products of the count with the query heads must not wrap: 2^62 * 4 does to 0."""
    kit = Kit(layers=1, hq=hq, hkv=hkv, seqs=1, seed=69)
    L, b = kvq.lib(), ctypes.c_size_t(7)
    for total in (1 << 61, 1 << 62, (1 << 62) + 1, (1 << 63) - 1, (1 << 31) // hq, -(1 << 63)):
        assert L.kvq_plan_extend_workspace_bytes(kit.plan.handle, 1, total, ctypes.byref(b)) == 1
        assert b.value == 7
    assert L.kvq_plan_extend_workspace_bytes(kit.plan.handle, 1, ((1 << 31) - 1) // hq, ctypes.byref(b)) == 0


@gpu
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("new", [False, True])
@pytest.mark.parametrize("case", ["v_nan", "v_inf", "k_nan", "k_up", "k_down"])
def test_what_rows_that_see_a_non_finite_row_get(bf16, new, case):
    """NaN or infinities in a value row: the channels that hold them, or all where the token is a new
    one.  A NaN or +infinite score: NaN throughout.  A score of -infinity weighs nothing."""
    kit = Kit(layers=1, seqs=1, seed=75, tail=128, bf16=bf16)
    n, nq = 200, 4
    r = kit.rows(n)
    at = n - nq if new else n - 40
    (r[0] if case[0] == "k" else r[1])[:, at, :, 5] = float({"v_nan": "nan", "v_inf": "inf", "k_nan": "nan", "k_up": "inf",
                                                             "k_down": "-inf"}[case])
    kit.append(0, r)
    q = kit.queries(nq)
    q[..., 5] = 1.0
    got = extend(kit, 0, [0], [nq], q)
    if case in ("k_nan", "k_up"):
        assert bool(torch.isnan(got).all())
        return
    values = kit.values(0)
    if case == "k_down":
        rows = [i for i in range(n) if i != at]
        if new:                                          # the first of the new tokens: the others as if it were not there
            ref, tol = reference(kit, 0, 0, q[1:], values=[x[:, rows] for x in values])
            assert bool(((got[1:].double() - ref).abs() <= tol).all())
            ref, tol = reference(kit, 0, 0, q[:1], values=[x[:, :at] for x in values])
            assert bool(((got[:1].double() - ref).abs() <= tol).all())
        else:
            ref, tol = reference(kit, 0, 0, q, values=[x[:, rows] for x in values])
            assert bool(((got.double() - ref).abs() <= tol).all())
        return
    if new:
        assert bool(torch.isnan(got).all())
        return
    assert not torch.isfinite(got[..., 5]).any()
    ref, tol = reference(kit, 0, 0, q)
    rest = [c for c in range(D) if c != 5]
    assert bool(((got.double() - ref).abs() <= tol)[..., rest].all())
