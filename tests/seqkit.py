"""Small plans with plain torch data for the tests of the sequence operations and of
the multi-token attention."""
from __future__ import annotations

import numpy as np
import torch

from quantized_kv_cache_15_b200 import kvq

D = 128


class Kit:
    """A plan, the raw rows appended to each of its sequences, and reads of its state."""

    def __init__(self, layers=2, hq=8, hkv=2, seqs=4, max_tokens=700, k=kvq.Q4_0, v=kvq.Q4_0, rot=kvq.ROT_HADAMARD,
                 tail=0, bf16=False, max_pages=0, seed=0, spread=20.0, f16_heads=()):
        self.L, self.hq, self.hkv, self.T = layers, hq, hkv, tail
        self.dt = torch.bfloat16 if bf16 else torch.float16
        self.rng = np.random.default_rng(seed)
        self.rot = rot
        n = layers * hkv
        self.kc = [k] * n if np.isscalar(k) else list(k)
        self.vc = [v] * n if np.isscalar(v) else list(v)
        kw = {}
        if rot == kvq.ROT_VARNORM_HADAMARD:
            kw["inv_rms"] = self.rng.uniform(0.05, 2.0, (layers, hkv, 2, D)).astype(np.float32)
        if rot == kvq.ROT_PROJECTION:
            rank = [(16, 32, 64, 96, 128)[i % 5] for i in range(n)]
            kw.update(rank=rank, k_bits=[1 + i % 4 for i in range(n)], v_bits=[1 + (i + 1) % 4 for i in range(n)],
                      proj_basis=[np.linalg.qr(self.rng.standard_normal((D, r)))[0] for r in rank])
            self.kc = self.vc = [kvq.F16 if i in f16_heads else kvq.RANK for i in range(n)]
        self.spread = np.ones(D, np.float32)
        self.spread[self.rng.choice(D, 4, replace=False)] = spread
        self.plan = kvq.Plan(layers, hq, hkv, max_seqs=seqs, max_tokens_per_seq=max_tokens, k_codec=self.kc,
                             v_codec=self.vc, rot=rot, tail_tokens=tail, max_pages=max_pages,
                             kv_dtype=kvq.KV_BF16 if bf16 else kvq.KV_F16, **kw)
        self.plan.allocate_cache()
        self.inv = kw.get("inv_rms")

    def rows(self, n):
        """n new tokens: [K, V], each [L][n][hkv][128]."""
        k = self.rng.standard_normal((self.L, n, self.hkv, D)).astype(np.float32) * self.spread
        v = self.rng.standard_normal((self.L, n, self.hkv, D)).astype(np.float32)
        return [torch.from_numpy(x).to("cuda").to(self.dt) for x in (k, v)]

    def append(self, seq, rows, layers=None, stream=None):
        for l in range(self.L) if layers is None else layers:
            if rows[0].shape[1]:
                self.plan.append(l, [seq], [rows[0].shape[1]], rows[0][l].contiguous(), rows[1][l].contiguous(),
                                 stream=stream)

    def fill(self, seq, n):
        r = self.rows(n)
        self.append(seq, r)
        return r

    def length(self, seq):
        return self.plan.seq_length(seq, 0)

    def values(self, seq):
        """Every cached row in the original basis: [K, V], each fp32 [L][n][hkv][128]."""
        n = self.length(seq)
        out = [torch.zeros((self.L, n, self.hkv, D), dtype=torch.float32, device="cuda") for _ in range(2)]
        for l in range(self.L):
            self.plan.dequantize(l, seq, 0, n, out[0][l], out[1][l])
        torch.cuda.synchronize()
        self.plan.check_device_error()
        return out

    def read(self, seq, layer, kv):
        """The packed rows below the tail, as kvq_read_rows lays them out: (codes, scales)."""
        nq = max(0, self.length(seq) - self.T)
        size = [self.plan.row_bytes(layer, h, kv) for h in range(self.hkv)]
        codes = torch.zeros(max(16, nq * sum(s[0] for s in size)), dtype=torch.uint8, device="cuda")
        scales = torch.zeros(max(16, nq * sum(s[1] for s in size)), dtype=torch.uint8, device="cuda")
        self.plan.read_rows(layer, seq, 0, nq, kv, codes, scales)
        torch.cuda.synchronize()
        return codes, scales

    def packed(self, seq):
        """Every packed row below the tail: {(layer, kv, head): bytes [rows][codes + scales]}."""
        nq = max(0, self.length(seq) - self.T)
        got = {}
        for l in range(self.L):
            for kv in range(2):
                size = [self.plan.row_bytes(l, h, kv) for h in range(self.hkv)]
                codes, scales = self.read(seq, l, kv)
                c, s, ci, si = codes.cpu().numpy(), scales.cpu().numpy(), 0, 0
                for h, (cb, sb) in enumerate(size):
                    got[l, kv, h] = np.concatenate([c[ci:ci + nq * cb].reshape(nq, cb), s[si:si + nq * sb].reshape(nq, sb)], 1)
                    ci += nq * cb
                    si += nq * sb
        return got

    def queries(self, n):
        return torch.from_numpy(self.rng.standard_normal((n, self.hq, D)).astype(np.float32)).to("cuda").to(self.dt)

    def decode(self, layer, seqs, q):
        out = torch.empty((len(seqs), self.hq, D), dtype=torch.float32, device="cuda")
        self.plan.decode(layer, seqs, q, out, self.plan.new_workspace(len(seqs)))
        torch.cuda.synchronize()
        self.plan.check_device_error()
        return out


#: (name, arguments of Kit): every rotation, codec family, raw type and tail the operations meet
VARIANTS = {
    "q4": dict(),
    "q4_tail": dict(tail=64),
    "kvarn_tail": dict(rot=kvq.ROT_VARNORM_HADAMARD, tail=128),
    "bf16_q41_tail": dict(k=kvq.Q4_1, v=kvq.Q4_1, tail=64, bf16=True, hq=6),
    "plain_mixed": dict(rot=kvq.ROT_NONE, k=[kvq.Q8_0, kvq.Q6_1, kvq.Q5_0, kvq.F16], v=[kvq.Q3_0, kvq.F16, kvq.Q2_1, kvq.Q8_1]),
    "mixed_tail": dict(k=[kvq.Q8_1, kvq.Q5_1, kvq.Q3_1, kvq.Q2_0], v=[kvq.Q4_0, kvq.Q6_0, kvq.F16, kvq.Q3_0], tail=64),
    "rank_tail": dict(rot=kvq.ROT_PROJECTION, tail=64, hq=4),
    "rank": dict(rot=kvq.ROT_PROJECTION, layers=3),
    "rank_f16_tail": dict(rot=kvq.ROT_PROJECTION, tail=64, f16_heads=(1, 2)),
}
