"""What the cache operators are measured on.

Four operators that read or shrink the key/value cache of one attention layer
(head dimension 128, grouped-query heads, bf16 or fp32):

* ``window``: attention with a sliding window and a few first tokens that stay
  visible, for whole prompts, appended chunks and single tokens;
* ``scored``: attention over the cache that adds every key's softmax weight to
  its accumulated score;
* ``evict``: the cache compacted to its first, its most recent and its highest
  scored keys;
* ``prefix``: attention of a batch whose sequences share a long prefix.

``run`` computes them in plain torch operations, or through the framework's
entry points when ``own`` is set. Sequence lengths are spread evenly over
their range and dealt to the sequences by the seed, so the work of a case does
not depend on the seed.
"""
import math

import numpy as np
import torch

own = False

D = 128


def _case(name, op, dtype="bf16", batch=1, h_q=32, h_kv=8, n_q=1, n_k=1, min_len=None, window=0, sinks=0,
          n_prefix=0, budget=0, recent=0, n_new=0):
    c = dict(op=op, dtype=dtype, batch=batch, h_q=h_q, h_kv=h_kv, n_q=n_q, n_k=n_k,
             min_len=n_k if min_len is None else min_len, window=window, sinks=sinks, n_prefix=n_prefix,
             budget=budget, recent=recent, n_new=n_new)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # a whole 32K prompt of a 32Q/8KV layer through a 4096-key window: the largest compute
        _case("window prompt 32K", "window", n_q=32768, n_k=32768, window=4096, sinks=128),
        # a left-padded batch of odd prompts, 7 query heads per key head: rows before a prompt's start are empty
        _case("window ragged prompts", "window", batch=3, h_q=28, h_kv=4, n_q=1537, n_k=1537, min_len=701,
              window=257, sinks=5),
        # one token for each of 32 sequences, young and old, through the window
        _case("window decode", "window", batch=32, n_k=8192, min_len=1, window=1024, sinks=4),
        # the fp32 layer: one head, 4096 tokens
        _case("window prompt fp32", "window", dtype="fp32", h_q=1, h_kv=1, n_q=4096, n_k=4096, window=512, sinks=128),
        # one token on a young cache: the smallest call, launch latency counts
        _case("scored decode 512", "scored", n_k=512),
        # one token on a 512K-token cache: all of its keys and values are read
        _case("scored decode 512K", "scored", n_k=524288),
        # three tokens (a checked draft) for a ragged batch, one of its sequences still empty
        _case("scored draft ragged", "scored", batch=24, h_q=28, h_kv=4, n_q=3, n_k=6001, min_len=0),
        # one token in fp32, every head with its own keys
        _case("scored decode fp32", "scored", dtype="fp32", batch=2, h_q=8, h_kv=8, n_k=8191, min_len=4096),
        # a 128K-token cache cut to an eighth
        _case("evict 128K to 16K", "evict", n_q=0, n_k=131072, sinks=128, recent=1024, budget=16384, n_new=18432),
        # a ragged batch of short caches, some of which fit the budget as they are
        _case("evict ragged", "evict", batch=16, h_q=28, h_kv=4, n_q=0, n_k=2111, min_len=100, sinks=4, recent=64,
              budget=513, n_new=600),
        # a few requests over one system prompt
        _case("prefix 777 x 3", "prefix", batch=3, n_k=40, min_len=1, n_prefix=777),
        # 64 requests over one 128K-token document, answers of up to 512 tokens
        _case("prefix 128K x 64", "prefix", batch=64, n_k=512, min_len=1, n_prefix=131072),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    h_kv, group = rng.choice([(8, 4), (4, 7), (1, 1), (2, 16), (8, 1), (4, 2), (5, 3)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    op = rng.choice(["window", "window", "scored", "evict", "prefix"])
    kw = dict(dtype=dtype, h_q=h_kv * group, h_kv=h_kv)
    size = (4 if dtype == "fp32" else 2) * 2 * D
    if op == "window":
        if rng.random() < 0.4:          # single tokens and short drafts
            batch, n_q = _log(rng, 1, 64), rng.choice([1, 1, 2, 5, 16])
            n_k = _log(rng, max(n_q, 2), 32768)
        else:                           # prompts and appended chunks
            batch, n_q = rng.choice([1, 1, 2, 3]), _log(rng, 17, 8192 if dtype == "bf16" else 1024)
            n_k = n_q + rng.choice([0, 0, _log(rng, 1, 8192)])
        window = _log(rng, 1, 4096)
        while batch * h_kv * n_k * size > 1 << 30:
            n_k = max(n_q, n_k // 2)
            batch = max(1, batch // 2)
        return _case(None, op, batch=batch, n_q=n_q, n_k=n_k, window=window, sinks=rng.choice([0, 1, 4, 128]),
                     min_len=rng.choice([n_k, n_k // 2, 0]), **kw)
    if op == "scored":
        batch, n_q = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 16])
        n_k = _log(rng, max(n_q, 2), 131072)
        while batch * h_kv * n_k * size > 1 << 30 or batch * n_q * h_kv * group * n_k > 1 << 27:
            n_k = max(n_q, n_k // 2)
            batch = max(1, batch // 2)
        return _case(None, op, batch=batch, n_q=n_q, n_k=n_k, min_len=rng.choice([n_k, n_k // 3, 0]), **kw)
    if op == "evict":
        batch, n_k = _log(rng, 1, 64), _log(rng, 16, 131072)
        while batch * h_kv * n_k * size > 1 << 30:
            n_k = max(16, n_k // 2)
            batch = max(1, batch // 2)
        budget = max(2, int(n_k * rng.uniform(0.05, 0.9)))
        sinks = min(rng.choice([0, 1, 4, 128]), budget // 2)
        recent = min(rng.choice([0, 1, 32, 1024]), budget - sinks)
        return _case(None, op, batch=batch, n_q=0, n_k=n_k, min_len=rng.choice([n_k, n_k // 2, 0]), sinks=sinks,
                     recent=recent, budget=budget, n_new=budget + rng.choice([0, 1, 128]), **kw)
    batch, n_q = _log(rng, 1, 96), rng.choice([1, 1, 2, 4])
    n_prefix, n_k = _log(rng, 1, 65536), _log(rng, n_q, 2048)
    while h_kv * n_prefix * size > 1 << 29 or batch * n_q * h_kv * group * n_prefix > 1 << 27:
        n_prefix = max(1, n_prefix // 2)
    while batch * h_kv * n_k * size > 1 << 29:
        n_k = max(n_q, n_k // 2)
    return _case(None, op, batch=batch, n_q=n_q, n_k=n_k, min_len=rng.choice([n_k, n_q, 0]), n_prefix=n_prefix, **kw)


def _lengths(c):
    """The lengths of the sequences, smallest first: evenly from min_len to n_k (a lone sequence is full)."""
    b = c["batch"]
    return [c["n_k"] if b == 1 else c["min_len"] + (c["n_k"] - c["min_len"]) * i // (b - 1) for i in range(b)]


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)
    dt = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    b, hq, hkv, nq, nk = c["batch"], c["h_q"], c["h_kv"], c["n_q"], c["n_k"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dt)

    lens = torch.tensor(_lengths(c), dtype=torch.int32, device=dev)
    lens = lens[torch.randperm(b, generator=gen, device=dev)].contiguous()
    s = {"case": c, "kv_len": lens, "k": normal(b, hkv, nk, D), "v": normal(b, hkv, nk, D), "kept": {}}
    if c["op"] != "evict":
        # a first token that draws a large share of the attention, as in trained models: every query of a
        # key head leans towards one direction, and the sequence's first key lies far along it
        u = torch.randn(hkv, D, generator=gen, device=dev)
        u = u / u.norm(dim=-1, keepdim=True) * D ** 0.25
        q = normal(b, hkv, hq // hkv, nq, D) + u[None, :, None, None]
        s["q"] = q.reshape(b, hq, nq, D).to(dt)
        s["out"] = torch.zeros_like(s["q"])
        first = s["k"]
        if c["op"] == "prefix":
            s["k_prefix"], s["v_prefix"] = normal(hkv, c["n_prefix"], D), normal(hkv, c["n_prefix"], D)
            first = s["k_prefix"][None]
        first[:, :, :1] += (math.log(first.shape[2]) * u[None, :, None]).to(dt)
    if c["op"] in ("scored", "evict"):
        # the weights that ten earlier tokens left: heavy-tailed; some keys, as the newest, have none yet
        s["score"] = 10 * hq / hkv / nk * torch.exp(2 * torch.randn(b, hkv, nk, generator=gen, device=dev) - 2)
        s["score"] *= (torch.rand(b, hkv, nk, generator=gen, device=dev) > 0.05).float()
    if c["op"] == "evict":
        s["k_new"] = torch.zeros(b, hkv, c["n_new"], D, dtype=dt, device=dev)
        s["v_new"] = torch.zeros_like(s["k_new"])
        s["score_new"] = torch.zeros(b, hkv, c["n_new"], device=dev)
        s["kept_idx"] = torch.zeros(b, hkv, c["budget"], dtype=torch.int32, device=dev)
        s["new_len"] = torch.zeros(b, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------- plain forms

def _masked_softmax(x, seen):
    """Softmax over the last axis of x where `seen`; rows that see nothing are zero."""
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-38)


def _plain_window(s):
    """Blocks of up to 256 queries, each with the first keys and the keys of its windows gathered."""
    c = s["case"]
    b, hq, hkv, nq, nk = c["batch"], c["h_q"], c["h_kv"], c["n_q"], c["n_k"]
    g, w, sinks = hq // hkv, c["window"], min(c["sinks"], nk)
    step = min(nq, 256)
    blocks = -(-nq // step)
    q = torch.nn.functional.pad(s["q"].float(), (0, 0, 0, blocks * step - nq)).view(b, hkv, g, blocks, step, D)
    q = q.transpose(2, 3).reshape(b, hkv, blocks, g * step, D)
    dev = q.device
    pos = (s["kv_len"].long()[:, None] - nq + torch.arange(blocks * step, device=dev)).view(b, blocks, step)
    j = torch.cat([torch.arange(sinks, device=dev).expand(b, blocks, sinks),
                   pos[:, :, :1] - w + 1 + torch.arange(w + step - 1, device=dev)], -1)
    late = torch.arange(j.shape[-1], device=dev) >= sinks          # the window's part of the gathered keys
    behind = pos[..., None] - j[:, :, None]                        # [b, blocks, step, keys]
    seen = (j[:, :, None] >= 0) & (behind >= 0) & torch.where(late, behind < w, behind >= w)
    at = j.clamp(0, nk - 1)[:, None].expand(b, hkv, blocks, j.shape[-1])
    bi, hi = torch.arange(b, device=dev)[:, None, None, None], torch.arange(hkv, device=dev)[:, None, None]
    x = q @ s["k"][bi, hi, at].float().transpose(-1, -2) / math.sqrt(D)
    p = _masked_softmax(x.view(b, hkv, blocks, g, step, -1), seen[:, None, :, None])
    o = p.view(b, hkv, blocks, g * step, -1) @ s["v"][bi, hi, at].float()
    o = o.view(b, hkv, blocks, g, step, D).transpose(2, 3).reshape(b, hq, blocks * step, D)[:, :, :nq]
    s["out"].copy_(o)
    return s["out"]


def _causal(s, n_q, n_k):
    """[b, n_q, n_k]: the key is at or before the query's place."""
    place = s["kv_len"].long()[:, None] - n_q + torch.arange(n_q, device=s["q"].device)
    return torch.arange(n_k, device=s["q"].device) <= place[..., None]


def _plain_scored(s):
    c = s["case"]
    b, hq, hkv, nq, nk = c["batch"], c["h_q"], c["h_kv"], c["n_q"], c["n_k"]
    g = hq // hkv
    x = s["q"].float().view(b, hkv, g * nq, D) @ s["k"].float().transpose(-1, -2) / math.sqrt(D)
    p = _masked_softmax(x.view(b, hkv, g, nq, nk), _causal(s, nq, nk)[:, None, None])
    s["out"].copy_((p.view(b, hkv, g * nq, nk) @ s["v"].float()).view(b, hq, nq, D))
    s["score"] += p.sum((2, 3))
    return s["out"], s["score"]


def _plain_prefix(s):
    c = s["case"]
    b, hq, hkv, nq, nk, npre = c["batch"], c["h_q"], c["h_kv"], c["n_q"], c["n_k"], c["n_prefix"]
    g = hq // hkv
    q = s["q"].float().view(b, hkv, g * nq, D)
    every = q.transpose(0, 1).reshape(hkv, b * g * nq, D)
    x0 = (every @ s["k_prefix"].float().transpose(-1, -2)).view(hkv, b, g, nq, npre).transpose(0, 1)
    x1 = (q @ s["k"].float().transpose(-1, -2)).view(b, hkv, g, nq, nk)
    seen = _causal(s, nq, nk)[:, None, None].expand(b, hkv, g, nq, nk)
    p = _masked_softmax(torch.cat([x0, x1], -1) / math.sqrt(D), torch.cat([torch.ones_like(x0, dtype=torch.bool), seen], -1))
    p0 = p[..., :npre].transpose(0, 1).reshape(hkv, b * g * nq, npre)
    o = (p0 @ s["v_prefix"].float()).view(hkv, b, g * nq, D).transpose(0, 1)
    o = o + p[..., npre:].reshape(b, hkv, g * nq, nk) @ s["v"].float()
    s["out"].copy_(o.reshape(b, hq, nq, D))
    return s["out"]


def _plain_evict(s):
    c = s["case"]
    b, hkv, nk, m = c["batch"], c["h_kv"], c["n_k"], c["budget"]
    lens = s["kv_len"].long()[:, None, None]
    j = torch.arange(nk, device=s["k"].device)
    worth = torch.where((j < c["sinks"]) | (j >= lens - c["recent"]), torch.full_like(s["score"], math.inf), s["score"])
    worth = torch.where(j < lens, worth, torch.full_like(worth, -math.inf))
    best = torch.sort(worth, dim=-1, descending=True, stable=True).indices[..., :m]
    new_len = lens.clamp_max(m)
    kept = torch.where(torch.arange(best.shape[-1], device=j.device) < new_len, best, torch.full_like(best, nk))
    kept = torch.nn.functional.pad(torch.sort(kept, dim=-1).values, (0, m - best.shape[-1]), value=nk)
    have = kept < nk
    at = kept.clamp_max(nk - 1)
    rows = at[..., None].expand(b, hkv, m, D)
    for_k, for_v = torch.gather(s["k"], 2, rows), torch.gather(s["v"], 2, rows)
    s["k_new"][:, :, :m] = torch.where(have[..., None], for_k, s["k_new"][:, :, :m])
    s["v_new"][:, :, :m] = torch.where(have[..., None], for_v, s["v_new"][:, :, :m])
    s["score_new"].zero_()
    s["score_new"][:, :, :m] = torch.where(have, torch.gather(s["score"], 2, at), torch.zeros_like(at, dtype=torch.float32))
    s["kept_idx"].copy_(torch.where(have, kept, torch.full_like(kept, -1)))
    s["new_len"].copy_(new_len.view(b))
    return s["k_new"], s["v_new"], s["score_new"], s["kept_idx"], s["new_len"]


_PLAIN = {"window": _plain_window, "scored": _plain_scored, "prefix": _plain_prefix, "evict": _plain_evict}


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import long_context_prefill_last_b200 as crisp
    c = s["case"]
    cfg = s["kept"].get("cfg")
    if cfg is None:      # a program's own configuration and workspace, kept from call to call
        cfg = crisp.CacheConfig(batch=c["batch"], n_q=max(1, c["n_q"]), n_k=c["n_k"], h_q=c["h_q"], h_kv=c["h_kv"],
                                dtype=crisp.FP32 if c["dtype"] == "fp32" else crisp.BF16, window=c["window"],
                                sinks=c["sinks"], n_prefix=c["n_prefix"], budget=c["budget"], recent=c["recent"],
                                n_new=c["n_new"])
        cfg.allocate_workspace({"window": crisp.CACHE_WINDOW, "scored": crisp.CACHE_SCORED,
                                "prefix": crisp.CACHE_PREFIX, "evict": crisp.CACHE_EVICT}[c["op"]])
        s["kept"]["cfg"] = cfg
    if c["op"] == "window":
        crisp.window_attention(s["q"], s["k"], s["v"], s["out"], cfg, kv_len=s["kv_len"])
        return s["out"]
    if c["op"] == "scored":
        crisp.scored_attention(s["q"], s["k"], s["v"], s["out"], s["score"], cfg, kv_len=s["kv_len"])
        return s["out"], s["score"]
    if c["op"] == "prefix":
        crisp.shared_prefix_attention(s["q"], s["k_prefix"], s["v_prefix"], s["k"], s["v"], s["out"], cfg,
                                      kv_len=s["kv_len"])
        return s["out"]
    crisp.evict(s["k"], s["v"], s["score"], s["k_new"], s["v_new"], s["score_new"], s["kept_idx"], s["new_len"], cfg,
                kv_len=s["kv_len"])
    return s["k_new"], s["v_new"], s["score_new"], s["kept_idx"], s["new_len"]


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def _visible(c, n):
    """(keys that some query of a sequence of n tokens sees, pairs of one query head)."""
    w, sinks, nq = c["window"] or c["n_k"] + 1, c["sinks"], c["n_q"]
    p = np.arange(max(0, n - nq), n)
    if not len(p):
        return 0, 0
    low = np.maximum(p - w + 1, 0)
    pairs = (p - low + 1 + np.minimum(low, sinks)).sum()
    return int(n - low[0] + min(low[0], sinks)), int(pairs)


def work(case):
    c = case
    e = 4 if c["dtype"] == "fp32" else 2
    row, lens = D * e, _lengths(c)
    if c["op"] == "evict":
        kept = sum(min(n, c["budget"]) for n in lens)
        rows = c["batch"] * c["h_kv"]
        return {"bytes": c["h_kv"] * (kept * 4 * row + kept * 4 + sum(lens) * 4) + rows * (c["budget"] + c["n_new"]) * 4,
                "flops": 0}
    see = [_visible(c, n) for n in lens]
    keys, pairs = sum(k for k, _ in see), sum(p for _, p in see)
    queries = c["batch"] * c["h_q"] * c["n_q"]
    got = {"bytes": 2 * queries * row + c["h_kv"] * keys * 2 * row, "flops": 4 * D * c["h_q"] * pairs}
    if c["op"] == "scored":
        got["bytes"] += c["h_kv"] * keys * 8
    if c["op"] == "prefix":
        got["bytes"] += c["h_kv"] * c["n_prefix"] * 2 * row
        got["flops"] += 4 * D * queries * c["n_prefix"]
    return got


# ---------------------------------------------------------------- the definition in 64 bits

def _attend64(q, k, v, mask):
    """One key head: q [rows, D], k and v [keys, D], mask [rows, keys] -> outputs and weights in float64."""
    x = (q.double() @ k.double().T) * (1.0 / math.sqrt(D))
    x = x.masked_fill(~mask, -math.inf)
    z = torch.logsumexp(x, -1, keepdim=True)
    p = torch.exp(x - z).nan_to_num(0.0)
    return p @ v.double(), p


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    lens = s["kv_len"].tolist()
    hkv, nq = c["h_kv"], c["n_q"]
    g = c["h_q"] // hkv
    if c["op"] == "evict":
        return _exact_evict(c, s, lens)
    out = torch.zeros(c["batch"], hkv, g, nq, D, dtype=torch.float64, device="cuda")
    score = s["score"].double() if c["op"] == "scored" else None
    q = s["q"].view(c["batch"], hkv, g, nq, D)
    for b, n in enumerate(lens):
        for h in range(hkv):
            for i0 in range(0, nq, 512):
                i1 = min(nq, i0 + 512)
                p = torch.arange(n - nq + i0, n - nq + i1, device="cuda")[:, None]
                # only keys that one of these queries can see are taken up
                low = max(0, n - nq + i0 - c["window"] + 1) if c["window"] else 0
                high = max(0, n - nq + i1)
                j = torch.cat([torch.arange(min(c["sinks"], low, high), device="cuda"),
                               torch.arange(min(low, high), high, device="cuda")])
                mask = j <= p
                if c["window"]:
                    mask &= (j < c["sinks"]) | (j > p - c["window"])
                kk, vv = s["k"][b, h][j], s["v"][b, h][j]
                if c["op"] == "prefix":
                    kk, vv = torch.cat([s["k_prefix"][h], kk]), torch.cat([s["v_prefix"][h], vv])
                    mask = torch.cat([torch.ones(i1 - i0, c["n_prefix"], dtype=torch.bool, device="cuda"), mask], 1)
                if kk.shape[0] == 0:
                    continue
                rows = q[b, h, :, i0:i1].reshape(-1, D)
                o, weight = _attend64(rows, kk, vv, mask.repeat(g, 1))
                out[b, h, :, i0:i1] = o.view(g, i1 - i0, D)
                if score is not None:
                    score[b, h, j] += weight.sum(0)
    out = out.view(c["batch"], c["h_q"], nq, D)
    return out if score is None else (out, score)


def _exact_evict(c, s, lens):
    score = s["score"].double().cpu().numpy()
    shape = score.shape[:2]
    kept = np.full(shape + (c["budget"],), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for h in range(shape[1]):
            idx = np.arange(n)
            if n > c["budget"]:
                forced = (idx < c["sinks"]) | (idx >= n - c["recent"])
                free = idx[~forced]
                order = free[np.lexsort((free, -score[b, h, free]))]
                idx = np.sort(np.concatenate([idx[forced], order[:c["budget"] - forced.sum()]]))
            kept[b, h, :len(idx)] = idx
    at = torch.from_numpy(kept.astype(np.int64)).cuda()
    new = {}
    for name in ("k", "v", "score"):
        src, dst = s[name].double(), torch.zeros_like(s[name + "_new"], dtype=torch.float64)
        for b, n in enumerate(lens):
            m = min(n, c["budget"])
            for h in range(shape[1]):
                dst[b, h, :m] = src[b, h, at[b, h, :m]]
        new[name] = dst
    lengths = torch.tensor([min(n, c["budget"]) for n in lens], dtype=torch.int32)
    return new["k"], new["v"], new["score"], at.to(torch.int32), lengths
