"""Value rows whose stored form leaves the range of fp16: a rotation grows one channel of a
row up to sqrt(128) times, and bf16 rows are larger than any fp16.  Attention of several new
tokens gives what the cached rows give in 64 bits, as decode does."""
import numpy as np
import pytest
import torch

from quantized_kv_cache_15_b200 import kvq
from tests.seqkit import D, Kit
from tests.test_gpu_extend import extend, reference, tree, words

gpu = pytest.mark.gpu

PLANS = {
    "q4": dict(),
    "q8": dict(k=kvq.Q8_0, v=kvq.Q8_0),
    "q8_q4": dict(k=kvq.Q8_0, v=kvq.Q4_0),
    "q41": dict(k=kvq.Q4_1, v=kvq.Q4_1),
    "mixed": dict(k=[kvq.Q6_1, kvq.Q5_0], v=[kvq.Q2_0, kvq.Q8_1]),
    "three": dict(v=[kvq.Q3_1, kvq.Q6_0]),
    "kvarn_tail": dict(rot=kvq.ROT_VARNORM_HADAMARD, tail=128),
    "rank": dict(rot=kvq.ROT_PROJECTION),
}


def check(kit, seqs, nqs, q, got, bits=None):
    """As test_gpu_extend.check.  Values near fp16's end, quantized in few bits, can add up to more than
    fp16 holds: the rounding of 65520 and above is infinity, so that output is off by what is missing to 65520."""
    i = 0
    for s, n in zip(seqs, nqs):
        ref, tol = reference(kit, 0, s, q[i:i + n], None if bits is None else bits[i:i + n])
        out = got[i:i + n].double()
        err = torch.where(torch.isinf(out), (65520.0 - ref * out.sign()).clamp(min=0.0), (out - ref).abs())
        assert bool((err <= tol).all()), (s, n, float((err / tol).max()))
        i += n


def large_rows(kit, n, level, every):
    """Rows of ordinary size, every `every`-th with all channels near `level`: one stored value of sqrt(128) level."""
    k, v = kit.rows(n)
    big = torch.arange(0, n, every, device="cuda")
    v[:, big] = (level * (1.0 + 0.01 * v[:, big].float())).to(kit.dt)
    return [k, v]


@gpu
@pytest.mark.parametrize("name", list(PLANS))
@pytest.mark.parametrize("level", [2500.0, 5700.0, 5900.0, 50000.0])     # sqrt(128) 5790 is fp16's largest value
@pytest.mark.parametrize("every,nq", [(1, 3), (7, 3), (100, 1), (7, 16)])
def test_stored_values_above_fp16(name, level, every, nq):
    kit = Kit(layers=1, seqs=1, seed=91, spread=3.0, **PLANS[name])
    kit.append(0, large_rows(kit, 500, level, every))
    q = kit.queries(nq)
    check(kit, [0], [nq], q, extend(kit, 0, [0], [nq], q))


@gpu
@pytest.mark.parametrize("k,v", [(kvq.Q4_0, kvq.Q4_0), (kvq.Q8_0, kvq.Q8_0), (kvq.Q4_1, kvq.Q8_1)])
@pytest.mark.parametrize("level", [9000.0, 300000.0])
def test_large_bf16_rows(k, v, level):
    kit = Kit(layers=1, seqs=1, seed=93, spread=3.0, k=k, v=v, bf16=True, tail=64)
    kit.append(0, large_rows(kit, 500, level, 5))
    q = kit.queries(4)
    check(kit, [0], [4], q, extend(kit, 0, [0], [4], q))


@gpu
def test_large_rows_behind_a_mask_and_in_wide_units():
    """Rows that mask a large token do not see it; units of 64 rows; the tokens before stay exact."""
    kit = Kit(layers=1, hq=32, hkv=8, seqs=16, seed=95, spread=3.0, max_tokens=2500)
    rng = np.random.default_rng(7)
    for s in range(16):
        kit.append(s, large_rows(kit, int(rng.integers(2000, 2400)), 30000.0, 50 + s))
        kit.append(s, large_rows(kit, 16, 30000.0, 3))
    bits = sum((tree(rng, 16) for _ in range(16)), [])
    q = kit.queries(256)
    check(kit, list(range(16)), [16] * 16, q, extend(kit, 0, list(range(16)), [16] * 16, q, words(bits)), bits)


@gpu
def test_large_tokens_agree_with_decode():
    kit = Kit(layers=1, seqs=1, seed=97, spread=3.0, k=kvq.Q8_0, v=kvq.Q8_0)
    kit.append(0, large_rows(kit, 500, 20000.0, 11))
    q = kit.queries(1)
    a, b = extend(kit, 0, [0], [1], q).float(), kit.decode(0, [0], q)
    # decode's bar is 2e-3 of a row's largest value; the output's rounding is 2^-11 of it
    assert bool(((a - b).abs() <= (2e-3 + 2.0 ** -11 + 2e-3) * b.abs().amax(-1, keepdim=True)).all())


@gpu
@pytest.mark.parametrize("kw", [dict(), dict(k=kvq.Q8_0, v=kvq.Q4_1, tail=64), dict(rot=kvq.ROT_PROJECTION, tail=64),
                                dict(k=kvq.F16, v=kvq.Q8_0)])
@pytest.mark.parametrize("forks,nq", [(3, 2), (16, 1)])
def test_large_rows_in_a_shared_prompt(kw, forks, nq):
    """Pages that a group of forks reads once (for 16 forks in a launch of their own), and the forks' own."""
    kit = Kit(layers=1, hq=32, hkv=8, seqs=forks + 1, seed=99, spread=3.0, max_tokens=3500, **kw)
    kit.append(0, large_rows(kit, 3300, 20000.0, 700))
    kit.plan.fork(0, list(range(1, forks)))
    kit.append(forks, large_rows(kit, 300, 20000.0, 50))
    for s in range(forks):
        kit.append(s, large_rows(kit, nq + 10 * s, 20000.0, 20))
    seqs, nqs = list(range(forks + 1)), [nq] * (forks + 1)
    q = kit.queries(sum(nqs))
    got = extend(kit, 0, seqs, nqs, q)
    check(kit, seqs, nqs, q, got)
    assert torch.equal(got, extend(kit, 0, seqs, nqs, q))
