"""Cases of the serving operators around the quantized KV cache: attention of several
new tokens per sequence over the cache in one call (draft verification, mixed batches,
sequences that share a prompt), forking a sequence, compacting it to a list of kept
positions and rolling it back.

`run` with `own` false computes a case in elementary torch operations on the cache's
codes, scales and raw tail rows; with `own` true it makes the framework's calls.
"""
import random

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"
BITS = {"q8_0": 8, "q6_0": 6, "q5_0": 5, "q4_0": 4, "q3_0": 3, "q2_0": 2,
        "q8_1": 8, "q6_1": 6, "q5_1": 5, "q4_1": 4, "q3_1": 3, "q2_1": 2}
CODEC_ID = {"q8_0": 1, "q6_0": 2, "q4_0": 3, "q3_0": 4, "q2_0": 5, "q8_1": 6, "q6_1": 7, "q4_1": 8, "q3_1": 9,
            "q2_1": 10, "q5_0": 12, "q5_1": 13}
SCALE = float(np.float32(1.0 / np.sqrt(128.0)))


# ----------------------------------------------------------------------------- cases
def _case(name, kind, **kw):
    c = {"name": name, "kind": kind, "layers": 1, "hq": 32, "hkv": 8, "dtype": "f16", "k": "q4_0", "v": "q4_0",
         "varnorm": False, "tail": 0, "batch": 1, "tmin": 1024, "tmax": 1024, "nq": 1, "tree": False, "forks": 0,
         "keep": 0}
    c.update(kw)
    return c


def listed():
    return [
        # one short conversation, four drafted tokens to check: latency is all that counts
        _case("verify_short", "extend", hq=8, hkv=2, tmin=1024, tmax=1024, nq=4),
        # a small batch under the batched configuration's cache (variance-normalised 4 bits, raw tail), a tree of drafts
        _case("verify_tree", "extend", varnorm=True, tail=256, batch=8, tmin=500, tmax=4096, nq=16, tree=True),
        # a full batch of ragged sequences, four drafted tokens each: the ordinary load of a server that speculates
        _case("verify_batch", "extend", varnorm=True, tail=256, batch=64, tmin=1024, tmax=16384, nq=4),
        # one long document, eight drafted tokens, keys in 8 bits and values in 4
        _case("verify_long", "extend", k="q8_0", tmin=131072, tmax=131072, nq=8),
        # bf16 rows, a long raw tail, scale-and-minimum 4-bit codes, six query heads per kv head, an odd draft length
        _case("verify_bf16", "extend", hq=24, hkv=4, dtype="bf16", k="q4_1", v="q4_1", tail=1024, batch=16, tmin=1100,
              tmax=8191, nq=5),
        # four samples of one short prompt: fork, one new token each, attention over the shared pages
        _case("sample_short", "sample", hq=8, hkv=2, tmin=2000, tmax=2000, forks=4),
        # sixteen samples of one long prompt
        _case("sample_long", "sample", varnorm=True, tail=256, tmin=32768, tmax=32768, forks=16),
        # a speculative step: fork, append a tree of drafts, attend, keep the accepted path
        _case("accept", "spec", layers=2, varnorm=True, tail=256, tmin=4096, tmax=4096, nq=16, tree=True, keep=5),
        # a short cache pruned to half
        _case("prune_short", "prune", hq=8, hkv=2, tmin=1024, tmax=1024, keep=512),
        # a long cache pruned to its first, most used and newest tokens
        _case("prune_long", "prune", layers=2, varnorm=True, tail=256, tmin=32768, tmax=32768, keep=8192),
        # an edited conversation rolled back to an earlier token: raw rows come back from the pages
        _case("rollback", "rollback", hq=24, hkv=4, dtype="bf16", k="q8_0", v="q4_0", tail=1024, tmin=16384,
              tmax=16384, keep=12001),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["extend", "extend", "extend", "sample", "spec", "prune", "rollback"])
    hq, hkv = rng.choice([(8, 2), (32, 8), (24, 4), (16, 2), (6, 6)])
    c = {"kind": kind, "layers": 1, "hq": hq, "hkv": hkv, "dtype": rng.choice(["f16", "bf16"]),
         "k": rng.choice(["q4_0", "q4_0", "q4_1", "q8_0"]), "v": rng.choice(["q4_0", "q4_0", "q4_1", "q8_0"]),
         "varnorm": rng.random() < 0.5, "tail": rng.choice([0, 64, 256, 1024]), "batch": 1, "nq": 1, "tree": False,
         "forks": 0, "keep": 0}
    if kind == "extend":
        c["batch"] = _log(rng, 1, 64)
        c["nq"] = _log(rng, 1, 48)
        c["tree"] = rng.random() < 0.5
        tokens = min(250000, int(6.5e7 / (hq * c["nq"])))            # over the batch: no more work than the largest listed
        c["tmax"] = _log(rng, 300, max(400, min(131072, tokens // c["batch"])))
        c["tmin"] = max(c["nq"], c["tmax"] // rng.choice([1, 2, 8]))
        c["tmax"] = max(c["tmax"], c["tmin"])
    elif kind == "sample":
        c["tmin"] = c["tmax"] = _log(rng, 500, 32768)
        c["forks"] = rng.randint(2, 16)
    elif kind == "spec":
        c["layers"] = rng.randint(1, 2)
        c["tmin"] = c["tmax"] = _log(rng, 300, 16384)
        c["nq"] = rng.randint(2, 40)
        c["tree"] = rng.random() < 0.5
        c["keep"] = rng.randint(0, c["nq"])
    else:
        c["layers"] = rng.randint(1, 2)
        c["tmin"] = c["tmax"] = _log(rng, 300, 24000)
        c["keep"] = max(1, int(c["tmax"] * (0.1 + 0.8 * rng.random())))
    return c


def _lengths(case):
    r = random.Random(repr(("len", case["batch"], case["tmin"], case["tmax"], case["nq"])))
    n = [r.randint(case["tmin"], case["tmax"]) for _ in range(case["batch"])]
    n[r.randrange(len(n))] = case["tmax"]
    return n


# ----------------------------------------------------------------------------- the cache's format, in torch
def _hadamard(dtype):
    h = torch.ones((1, 1), dtype=torch.float64, device=DEV)
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h.to(dtype)


def _staged_hadamard(x):
    """The rotation of the cache's rows in 32 bits: seven add/subtract stages, then the product with 1/sqrt(128)."""
    shape = x.shape
    for h in (1, 2, 4, 8, 16, 32, 64):
        y = x.reshape(-1, D // (2 * h), 2, h)
        a, b = y[:, :, 0], y[:, :, 1]
        x = torch.stack([a + b, a - b], 2)
    return x.reshape(shape) * SCALE


def _quantize(x, codec, inv):
    """Raw rows [..., 128] -> codes (int16, the offset-binary u) and scales (and minima) fp16 [..., 4]."""
    y = x.float()
    if inv is not None:
        y = y * inv
    y = _staged_hadamard(y).reshape(*x.shape[:-1], 4, 32)
    bits = BITS[codec]
    if codec.endswith("_0"):
        half = 1 << (bits - 1)
        d = (y.abs().amax(-1) / float(half - 1)).clamp(max=65504.0).half()
        s = d.float()
        u = torch.round(y * (1.0 / s).unsqueeze(-1)).clamp(-half, half - 1) + half
        u = torch.where((s == 0).unsqueeze(-1), torch.full_like(u, half), u)
        m = None
    else:
        top = (1 << bits) - 1
        low = y.amin(-1).clamp(-65504.0, 65504.0)
        m = low.half()
        down = torch.where(m > 0, m.view(torch.int16) - 1, m.view(torch.int16) + 1)
        down = torch.where(m == 0, torch.full_like(down, -32767), down).view(torch.float16)
        m = torch.where(m.float() > low, down, m)
        d = ((y.amax(-1) - m.float()) / float(top)).clamp(max=65504.0).half()
        s = d.float()
        u = torch.round((y - m.float().unsqueeze(-1)) * (1.0 / s).unsqueeze(-1)).clamp(0, top)
        u = torch.where((s == 0).unsqueeze(-1), torch.zeros_like(u), u)
    return {"u": u.reshape(x.shape).to(torch.uint8), "d": d, "m": m}


def _stored(c, codec, dtype=torch.float32):
    """Codes and scales -> values in the rotated basis."""
    u = c["u"].to(dtype).reshape(*c["u"].shape[:-1], 4, 32)
    d = c["d"].to(dtype).unsqueeze(-1)
    if c["m"] is None:
        v = (u - float(1 << (BITS[codec] - 1))) * d
    else:
        v = u * d + c["m"].to(dtype).unsqueeze(-1)
    return v.reshape(c["u"].shape)


def _at(c, f):
    return {k: (None if t is None else f(t)) for k, t in c.items()}


def _rows(shape, kind, seed_gen, dtype, channels):
    x = torch.randn(shape, generator=seed_gen, device=DEV, dtype=torch.float16)
    if kind == "K":                            # a few channels of every kv head are 20 times as large
        x = x * channels
    return x.to(dtype)


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt = torch.float16 if case["dtype"] == "f16" else torch.bfloat16
    L, B, H, T = case["layers"], case["batch"], case["hkv"], case["tail"]
    lens, tmax = _lengths(case), case["tmax"]
    pick = torch.rand((L, 1, 1, H, D), generator=g, device=DEV).topk(4, dim=-1).indices
    channels = torch.ones((L, 1, 1, H, D), dtype=torch.float16, device=DEV).scatter_(-1, pick, 20.0)
    inv = None
    if case["varnorm"]:                        # per-channel inverse RMS of a calibration prefix of 512 tokens
        inv = []
        for kind in "KV":
            x = _rows((L, 1, 512, H, D), kind, g, dt, channels).double()
            inv.append((1.0 / x.square().mean(2).sqrt()).float())              # [L, 1, H, D]
    raw = [_rows((L, B, tmax, H, D), kind, g, dt, channels) for kind in "KV"]
    new = None
    n_new = case["nq"] if case["kind"] == "spec" else case["forks"]
    if n_new:
        new = [_rows((L, 1, n_new, H, D), kind, g, dt, channels)[:, 0].contiguous() for kind in "KV"]
    nq, total_q = case["nq"], (case["forks"] or B * case["nq"])
    q = torch.randn((L, total_q, case["hq"], D), generator=g, device=DEV, dtype=torch.float16).to(dt)
    r = random.Random(int(seed) * 7919 + 11)
    mask, parents = None, []
    if case["tree"]:                           # every draft hangs below an earlier one or below the last cached token
        bits = []
        for _ in range(B):
            par = [r.randint(max(-1, i - 4), i - 1) for i in range(nq)]
            row = []
            for i in range(nq):
                row.append((1 << i) | (row[par[i]] if par[i] >= 0 else 0))
            bits += [b - (1 << 64) if b >= 1 << 63 else b for b in row]
            parents.append(par)
        mask = torch.tensor(bits, dtype=torch.int64, device=DEV)
    keep = None
    if case["kind"] == "prune":                # the first 4, the newest quarter of the budget, the rest anywhere between
        n, k = tmax, case["keep"]
        first = min(4, k)
        last = min((k - first) // 4, n - first)
        mid = sorted(r.sample(range(first, n - last), k - first - last))
        keep = torch.tensor(list(range(first)) + mid + list(range(n - last, n)), dtype=torch.int32, device=DEV)
    elif case["kind"] == "spec":               # accepted drafts: positions behind the cached tokens
        chosen = sorted(r.sample(range(nq), case["keep"]))
        keep = torch.tensor([tmax + c for c in chosen], dtype=torch.int32, device=DEV)
    st = {"case": case, "lens": lens, "q": q, "mask": mask, "keep": keep, "new": new, "inv": inv, "dt": dt}
    if own:
        from quantized_kv_cache_15_b200 import kvq

        kinv = None
        if inv is not None:
            kinv = torch.stack([inv[0][:, 0], inv[1][:, 0]], 2).cpu().numpy()  # [L, H, 2, D]
        extra = max(case["forks"], 1)
        seqs = B if case["kind"] == "extend" else 1 + extra
        plan = kvq.Plan(L, case["hq"], H, max_seqs=seqs, max_tokens_per_seq=tmax + max(n_new, 1),
                        k_codec=[CODEC_ID[case["k"]]] * (L * H), v_codec=[CODEC_ID[case["v"]]] * (L * H),
                        rot=kvq.ROT_VARNORM_HADAMARD if inv is not None else kvq.ROT_HADAMARD, tail_tokens=T,
                        inv_rms=kinv, kv_dtype=kvq.KV_F16 if dt == torch.float16 else kvq.KV_BF16)
        plan.allocate_cache()
        _load(plan, case, lens, raw, inv)
        st["plan"] = plan
        entries = case["forks"] or B
        st["n_q"] = [1] * entries if case["forks"] else [nq] * B
        st["ws"] = plan.new_extend_workspace(entries, total_q)
        st["out"] = torch.empty_like(q)
        if case["kind"] in ("spec", "prune", "rollback"):
            n = tmax + case["keep"] if case["kind"] == "spec" else case["keep"]
            st["k"] = torch.empty((L, n, H, D), dtype=torch.float32, device=DEV)
            st["v"] = torch.empty((L, n, H, D), dtype=torch.float32, device=DEV)
        torch.cuda.synchronize()
        return st
    # the cache as the framework stores it: quantized rows below the tail, raw rows in it
    n_old = [max(0, n - T) for n in lens]
    nmax = max(n_old)
    cache = []
    for kv in range(2):
        codec = case["kv"[kv]]
        i5 = None if inv is None else inv[kv].unsqueeze(1)
        codes = [_quantize(raw[kv][:, b:b + 1, :nmax], codec, i5) for b in range(B)]
        codes = {k: (None if codes[0][k] is None else torch.cat([c[k] for c in codes], 1)) for k in ("u", "d", "m")}
        w = min(T, tmax)
        at = torch.tensor(n_old, device=DEV).unsqueeze(1) + torch.arange(w, device=DEV)
        at = at.clamp(max=tmax - 1).reshape(1, B, w, 1, 1).expand(L, B, w, H, D)
        cache.append({"codes": codes, "tail": torch.gather(raw[kv], 2, at)})
    st["cache"] = cache
    return st


# ----------------------------------------------------------------------------- plain forms
def _values(codes, codec, mul):
    """Rows of the cache in the original basis, 32 bits."""
    x = _staged_hadamard(_stored(codes, codec))
    return x if mul is None else x * mul


def _muls(st):
    if st["inv"] is None:
        return [None, None]
    return [(1.0 / i.double()).float() for i in st["inv"]]                     # [L, 1, H, D]


def _attend(q, k, v, seen):
    """q [N, n, Hq, D], k and v [N, T, H, D] in 32 bits, seen [N or 1, n, T]: softmax(q k^T / sqrt(D)) v."""
    N, n, hq, _ = q.shape
    H = k.shape[2]
    qh = q.float().reshape(N, n, H, hq // H, D).permute(0, 2, 3, 1, 4).reshape(N, H, -1, D)
    s = torch.matmul(qh, k.permute(0, 2, 3, 1)) * SCALE
    s = s.reshape(N, H, hq // H, n, -1).masked_fill(~seen[:, None, None], float("-inf"))
    e = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul((e / e.sum(-1, keepdim=True)).reshape(N, H, (hq // H) * n, -1), v.permute(0, 2, 1, 3))
    return o.reshape(N, H, hq // H, n, D).permute(0, 3, 1, 2, 4).reshape(N, n, hq, D)


def _seen(lens, nq, mask, total):
    """[N, nq, total]: what each of the last nq tokens of a sequence sees."""
    n = torch.tensor(lens, device=DEV).reshape(-1, 1, 1)
    t = torch.arange(total, device=DEV).reshape(1, 1, -1)
    base = n - nq
    j = t - base
    if mask is None:
        return j <= torch.arange(nq, device=DEV).reshape(1, -1, 1)
    bit = (mask.reshape(len(lens), nq, 1) >> j.clamp(0, 63)) & 1
    return (j < 0) | ((j < nq) & (bit == 1))


def _plain_extend(st):
    case, lens = st["case"], st["lens"]
    T, tmax, mul = case["tail"], case["tmax"], _muls(st)
    h = _hadamard(torch.float32) * SCALE
    full = []
    for kv in range(2):
        c = st["cache"][kv]
        x = torch.matmul(_stored(_at(c["codes"], lambda t: t[0]), case["kv"[kv]]), h)
        if mul[kv] is not None:
            x = x * mul[kv]
        if T:
            B, w = len(lens), c["tail"].shape[2]
            old = torch.tensor([max(0, n - T) for n in lens], device=DEV).unsqueeze(1)
            at = old + torch.arange(w, device=DEV)
            y = torch.zeros((B, tmax + 1, *x.shape[2:]), device=DEV)
            y[:, :x.shape[1]] = x
            at = torch.where(at < torch.tensor(lens, device=DEV).unsqueeze(1), at, torch.full_like(at, tmax))
            y.scatter_(1, at.reshape(B, w, 1, 1).expand(B, w, *x.shape[2:]), c["tail"][0].float())
            x = y[:, :tmax]
        full.append(x)
    nq = case["nq"]
    q = st["q"][0].reshape(len(lens), nq, case["hq"], D)
    o = _attend(q, full[0], full[1], _seen(lens, nq, st["mask"], tmax))
    return {"out": o.reshape(st["q"].shape).to(st["dt"])}


def _sequence(st):
    """The one cached sequence: per K|V its codes [L, n, H, ...] and its raw tail rows [L, w, H, D]."""
    return [{"codes": _at(c["codes"], lambda t: t[:, 0]), "tail": c["tail"][:, 0]} for c in st["cache"]]


def _append(st, seq, new, T):
    """Rows that leave the raw tail are quantized into the cache."""
    out = []
    for kv in range(2):
        tail = torch.cat([seq[kv]["tail"], new[kv]], 1)
        gone = max(0, tail.shape[1] - T)
        codes = _quantize(tail[:, :gone], st["case"]["kv"[kv]], None if st["inv"] is None else st["inv"][kv])
        codes = {k: (None if t is None else torch.cat([seq[kv]["codes"][k], t], 1)) for k, t in codes.items()}
        out.append({"codes": codes, "tail": tail[:, gone:]})
    return out


def _read(st, seq):
    mul = _muls(st)
    return [torch.cat([_values(c["codes"], st["case"]["kv"[kv]], mul[kv]), c["tail"].float()], 1)
            for kv, c in enumerate(seq)]


def _select(st, seq, keep, T):
    """Only the positions `keep` (ascending) stay; rows that re-enter the raw tail are the cached values, rounded."""
    mul, out = _muls(st), []
    n = keep.shape[0]
    cut = max(0, n - T)
    for kv in range(2):
        c, old = seq[kv], seq[kv]["codes"]["u"].shape[1]
        back = keep[cut:]
        rows = _at(c["codes"], lambda t: t[:, back.clamp(max=max(old - 1, 0))] if old else t[:, :0])
        tail = c["tail"][:, (back - old).clamp(min=0, max=max(c["tail"].shape[1] - 1, 0))] if T else c["tail"]
        if old and T:
            deq = _values(rows, st["case"]["kv"[kv]], mul[kv]).to(st["dt"])
            tail = torch.where((back < old).reshape(1, -1, 1, 1), deq, tail)
        out.append({"codes": _at(c["codes"], lambda t: t[:, keep[:cut]]), "tail": tail})
    return out


def _plain_sequence(st):
    case = st["case"]
    T, n = case["tail"], case["tmax"]
    seq = _sequence(st)
    if case["kind"] == "sample":
        # every fork: the prompt and its own new token
        F = case["forks"]
        mul = _muls(st)
        shared = [_values(_at(c["codes"], lambda t: t[0]), case["kv"[kv]], None if mul[kv] is None else mul[kv][0])
                  for kv, c in enumerate(seq)]
        full = []
        for kv in range(2):
            w = seq[kv]["tail"].shape[1]
            own_rows = torch.cat([seq[kv]["tail"][0].unsqueeze(0).expand(F, -1, -1, -1), st["new"][kv][0].unsqueeze(1)], 1)
            gone = max(0, w + 1 - T)
            q = _quantize(own_rows[:, :gone], case["kv"[kv]], None if st["inv"] is None else st["inv"][kv])
            back = _values(q, case["kv"[kv]], None if mul[kv] is None else mul[kv])
            full.append(torch.cat([shared[kv].unsqueeze(0).expand(F, -1, -1, -1), back, own_rows[:, gone:].float()], 1))
        seen = torch.ones((1, 1, n + 1), dtype=torch.bool, device=DEV)
        o = _attend(st["q"][0].unsqueeze(1), full[0], full[1], seen)
        return {"out": o.reshape(st["q"].shape).to(st["dt"])}
    if case["kind"] == "spec":
        seq = _append(st, seq, st["new"], T)
        k, v = _read(st, seq)
        nq = case["nq"]
        o = _attend(st["q"], k, v, _seen([n + nq], nq, st["mask"], n + nq))
        keep = torch.cat([torch.arange(n, device=DEV), st["keep"].long()])
        k, v = _read(st, _select(st, seq, keep, T))
        return {"out": o.to(st["dt"]), "k": k, "v": v}
    keep = st["keep"].long() if case["kind"] == "prune" else torch.arange(case["keep"], device=DEV)
    k, v = _read(st, _select(st, seq, keep, T))
    return {"k": k, "v": v}


# ----------------------------------------------------------------------------- the framework's calls
def _load(plan, case, lens, raw, inv):
    """The cache that the plain form reads, brought into the plan as saved rows."""
    for l in range(case["layers"]):
        for b, n in enumerate(lens):
            old = max(0, n - case["tail"])
            packed = [None, None]
            for kv in range(2):
                if not old:
                    continue
                codec = case["kv"[kv]]
                c = _quantize(raw[kv][l, b, :old], codec, None if inv is None else inv[kv][l])
                u = c["u"] if BITS[codec] == 8 else c["u"][..., 0::2] | (c["u"][..., 1::2] << 4)
                d = c["d"] if c["m"] is None else torch.stack([c["d"], c["m"]], -1)
                packed[kv] = (u.transpose(0, 1).contiguous(), d.transpose(0, 1).contiguous().view(torch.uint8))
            tail = [raw[kv][l, b, old:n].contiguous() if n > old else None for kv in range(2)]
            plan.load(l, b, old, packed[0], packed[1], tail[0], tail[1])


def _own_extend(st):
    st["plan"].extend(0, range(len(st["lens"])), st["n_q"], st["q"][0], st["out"][0], st["ws"], tree_mask=st["mask"])
    return {"out": st["out"]}


def _own_sequence(st):
    case, plan, n = st["case"], st["plan"], st["case"]["tmax"]
    if case["kind"] == "sample":
        forks = list(range(1, 1 + case["forks"]))
        plan.fork(0, forks)
        plan.append(0, forks, st["n_q"], st["new"][0][0], st["new"][1][0])
        plan.extend(0, forks, st["n_q"], st["q"][0], st["out"][0], st["ws"])
        for s in forks:
            plan.seq_reset(s)
        return {"out": st["out"]}
    plan.fork(0, [1])
    if case["kind"] == "spec":
        for l in range(case["layers"]):
            plan.append(l, [1], st["n_q"], st["new"][0][l], st["new"][1][l])
            plan.extend(l, [1], st["n_q"], st["q"][l], st["out"][l], st["ws"], tree_mask=st["mask"])
        plan.compact([1], [n], [case["keep"]], st["keep"])
    elif case["kind"] == "prune":
        plan.compact([1], [0], [case["keep"]], st["keep"])
    else:
        plan.truncate([1], [case["keep"]])
    for l in range(case["layers"]):
        plan.dequantize(l, 1, 0, st["k"].shape[1], st["k"][l], st["v"][l])
    plan.seq_reset(1)
    if case["kind"] == "spec":
        return {"out": st["out"], "k": st["k"], "v": st["v"]}
    return {"k": st["k"], "v": st["v"]}


def run(state):
    if own:
        return _own_extend(state) if state["case"]["kind"] == "extend" else _own_sequence(state)
    return _plain_extend(state) if state["case"]["kind"] == "extend" else _plain_sequence(state)


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    H, T, L, lens = case["hkv"], case["tail"], case["layers"], _lengths(case)
    row = sum(16 * BITS[c] + (16 if c.endswith("_1") else 8) for c in (case["k"], case["v"]))
    raw = 2 * 2 * D

    def cached(n):
        return L * H * (max(0, n - T) * row + min(n, T) * raw)

    qo = 2 * 2 * D * case["hq"]
    if case["kind"] == "extend":
        nq = case["nq"]
        return {"bytes": sum(cached(n) for n in lens) + len(lens) * nq * qo,
                "flops": sum(4.0 * D * case["hq"] * nq * n for n in lens)}
    n = lens[0]
    if case["kind"] == "sample":
        return {"bytes": cached(n) + case["forks"] * (qo + H * raw), "flops": 4.0 * D * case["hq"] * case["forks"] * (n + 1)}
    if case["kind"] == "spec":
        nq, m = case["nq"], n + case["keep"]
        return {"bytes": cached(n) + L * nq * (qo + H * raw) + 2 * 4 * D * H * L * m,
                "flops": L * (4.0 * D * case["hq"] * nq * n + 2 * 7.0 * D * H * m)}
    m = case["keep"]
    moved = cached(m) if case["kind"] == "prune" else 0
    return {"bytes": cached(m) + moved + 2 * 4 * D * H * L * m, "flops": 2 * 7.0 * D * H * L * m}


# ----------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """From the cached codes, scales and raw rows: values in 64 bits through the Hadamard matrix, attention one
    (sequence, kv head) at a time."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    H, G, T, dt = case["hkv"], case["hq"] // case["hkv"], case["tail"], torch.float64
    R = _hadamard(dt) / np.sqrt(128.0)
    lens, L = st["lens"], case["layers"]

    def original(codes, kv, l):                # codes [n, H, 128] of layer l -> values
        x = _stored(codes, case["kv"[kv]], dt) @ R
        return x if st["inv"] is None else x / st["inv"][kv][l, 0].double()

    def sequence(l, b):
        n = lens[b]
        rows = []
        for kv in range(2):
            c = st["cache"][kv]
            a = original(_at(c["codes"], lambda t: t[l, b, :max(0, n - T)]), kv, l)
            rows.append(torch.cat([a, c["tail"][l, b, :n - a.shape[0]].to(dt)]))
        return rows

    def requantized(x, kv, l):                 # raw rows that left the tail
        return original(_quantize(x, case["kv"[kv]], None if st["inv"] is None else st["inv"][kv][l]), kv, l)

    def attention(q, k, v, visible):           # q [n, Hq, D], k and v [t, H, D], visible [n, t]
        o = torch.empty(q.shape, dtype=dt, device=DEV)
        for h in range(H):
            s = torch.einsum("igd,td->igt", q[:, h * G:(h + 1) * G].to(dt), k[:, h]) * SCALE
            s = torch.where(visible[:, None], s, torch.full_like(s, -np.inf))
            o[:, h * G:(h + 1) * G] = torch.einsum("igt,td->igd", torch.softmax(s, -1), v[:, h])
        return o

    def visible(n, nq, bits):
        a = torch.ones((nq, n), dtype=torch.bool, device=DEV)
        for i in range(nq):
            a[i, n - nq:] = torch.tensor([(j <= i) if bits is None else bool((bits[i] >> j) & 1) for j in range(nq)],
                                         device=DEV)
        return a

    if case["kind"] == "extend":
        nq, outs = case["nq"], []
        bits = None if st["mask"] is None else st["mask"].tolist()
        for b in range(case["batch"]):
            k, v = sequence(0, b)
            mine = None if bits is None else bits[b * nq:(b + 1) * nq]
            outs.append(attention(st["q"][0, b * nq:(b + 1) * nq], k, v, visible(lens[b], nq, mine)))
        return {"out": torch.cat(outs).unsqueeze(0)}
    n = lens[0]
    base = [sequence(l, 0) for l in range(L)]
    if case["kind"] == "sample":
        outs = []
        for f in range(case["forks"]):
            rows = []
            for kv in range(2):
                raw = torch.cat([st["cache"][kv]["tail"][0, 0], st["new"][kv][0, f:f + 1]])
                gone = max(0, raw.shape[0] - T)
                rows.append(torch.cat([base[0][kv][:max(0, n - T)], requantized(raw[:gone], kv, 0), raw[gone:].to(dt)]))
            outs.append(attention(st["q"][0, f:f + 1], rows[0], rows[1],
                                  torch.ones((1, n + 1), dtype=torch.bool, device=DEV)))
        return {"out": torch.cat(outs).unsqueeze(0)}
    if case["kind"] == "spec":
        nq = case["nq"]
        bits = None if st["mask"] is None else st["mask"].tolist()
        keep = list(range(n)) + st["keep"].tolist()
    else:
        keep = st["keep"].tolist() if case["kind"] == "prune" else list(range(case["keep"]))
    outs, got = [], [[], []]
    for l in range(L):
        rows = base[l]
        total = n
        if case["kind"] == "spec":
            rows, total = [], n + nq
            for kv in range(2):
                raw = torch.cat([st["cache"][kv]["tail"][l, 0], st["new"][kv][l]])
                gone = max(0, raw.shape[0] - T)
                rows.append(torch.cat([base[l][kv][:max(0, n - T)], requantized(raw[:gone], kv, l), raw[gone:].to(dt)]))
            outs.append(attention(st["q"][l], rows[0], rows[1], visible(total, nq, bits)))
        index = torch.tensor(keep, device=DEV)
        cut, old = max(0, len(keep) - T), max(0, total - T)
        for kv in range(2):
            x = rows[kv][index]
            back = (torch.arange(len(keep), device=DEV) >= cut) & (index < old)   # rows that come back as raw rows
            got[kv].append(torch.where(back[:, None, None], x.float().to(st["dt"]).to(dt), x))
    r = {"k": torch.stack(got[0]), "v": torch.stack(got[1])}
    if outs:
        r["out"] = torch.stack(outs)
    return r
