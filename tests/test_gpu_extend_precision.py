"""Attention of several new tokens where one token has nearly all of the weight: the others'
weights keep their bits however small they are.

One sink key scores `gap` log2 units above all other keys, which are zero, and its value row
is zero, so the output is made of weights 2^-gap of the largest.  The other value rows are
all alike, so their weights' roundings do not average out.  The tolerance is the one of
test_gpu_extend, relative to what these rows add up to."""
import numpy as np
import pytest
import torch

from quantized_kv_cache_15_b200 import kvq
from tests.seqkit import D, Kit
from tests.test_gpu_extend import check, extend

gpu = pytest.mark.gpu


def sink_rows(kit, n, gap, value):
    """[K, V] of n tokens and the query row: token 0 is the sink."""
    u = torch.from_numpy(np.where(kit.rng.random(D) < 0.5, -1.0, 1.0).astype(np.float32)).cuda()
    k = torch.zeros((kit.L, n, kit.hkv, D), device="cuda")
    k[:, 0] = u * (gap * np.log(2.0) / np.sqrt(128.0))
    v = (torch.from_numpy(kit.rng.standard_normal(D).astype(np.float32)).cuda() * value).expand(kit.L, n, kit.hkv, D).clone()
    v[:, 0] = 0.0
    return [k.to(kit.dt), v.to(kit.dt)], u.to(kit.dt)


SINKS = {
    "q4": dict(),
    "q8_plain": dict(rot=kvq.ROT_NONE, k=kvq.Q8_0, v=kvq.Q8_0),
    "q41": dict(k=kvq.Q4_1, v=kvq.Q4_1),
    "f16_pages": dict(k=kvq.F16, v=kvq.F16),
    "raw_tail": dict(tail=2048),
    "bf16_tail": dict(tail=2048, bf16=True),
    "rank": dict(rot=kvq.ROT_PROJECTION),
}


@gpu
@pytest.mark.parametrize("name", list(SINKS))
@pytest.mark.parametrize("gap", [15.3, 20.6, 22.3, 26.4, 30.5])
@pytest.mark.parametrize("nq", [1, 12])
def test_weights_far_below_the_largest_keep_their_bits(name, gap, nq):
    kit = Kit(layers=1, seqs=1, seed=81, max_tokens=2100, **SINKS[name])
    rows, u = sink_rows(kit, 2000, gap, 100.0)
    kit.append(0, rows)
    q = u.expand(nq, kit.hq, D).contiguous()
    check(kit, 0, [0], [nq], q, extend(kit, 0, [0], [nq], q))


@gpu
@pytest.mark.parametrize("gap", [20.6, 26.4])
def test_forks_of_a_prompt_with_a_sink(gap):
    """The same in the shared pages of a group and in the merge with the forks' own tokens."""
    kit = Kit(layers=1, hq=32, hkv=8, seqs=16, seed=83, max_tokens=3500)
    rows, u = sink_rows(kit, 3300, gap, 100.0)
    kit.append(0, rows)
    kit.plan.fork(0, list(range(1, 16)))
    for s in range(16):
        kit.append(s, [x[:, 1:2 + s].contiguous() for x in rows])
    q = u.expand(16, kit.hq, D).contiguous()
    check(kit, 0, list(range(16)), [1] * 16, q, extend(kit, 0, list(range(16)), [1] * 16, q))
