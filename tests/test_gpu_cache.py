"""The cache operators on the GPU against their definitions in 64 bits
(tests/cache_plain.py, where the tolerances are derived)."""
import math

import pytest

import cache_plain as plain

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import long_context_prefill_last_b200 as crisp  # noqa: E402

DT = {"bf16": (torch.bfloat16, crisp.BF16), "fp32": (torch.float32, crisp.FP32)}
D = 128


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_prefill_last_b200 import build
    build.build()
    crisp.lib()


def randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def make(dtype, b, hq, hkv, nq, nk, lens, seed=0, sharp=1.0, **kw):
    """Inputs; slots that no query may see hold NaN."""
    gen = torch.Generator("cuda").manual_seed(seed)
    t = DT[dtype][0]
    q, k, v = randn(gen, b, hq, nq, D, dtype=t) * sharp, randn(gen, b, hkv, nk, D, dtype=t), randn(gen, b, hkv, nk, D, dtype=t)
    window, sinks = kw.get("window", 0), kw.get("sinks", 0)
    for s in range(b):
        dead = ~plain.seen_mask(nq, nk, lens[s], window, sinks, "cuda").any(0)
        k[s, :, dead] = math.nan
        v[s, :, dead] = math.nan
        v[s, :, dead.nonzero()[::2, 0]] = math.inf
    cfg = crisp.CacheConfig(batch=b, n_q=nq, n_k=nk, h_q=hq, h_kv=hkv, dtype=DT[dtype][1], **kw)
    return q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), cfg


def guarded(*shape, dtype, fill=7.0):
    """A tensor between two guard zones of its own allocation, and a check that they are untouched."""
    n = math.prod(shape)
    pad = 1024
    buf = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    t = buf[pad:pad + n].view(*shape)

    def check():
        assert (buf[:pad] == fill).all() and (buf[pad + n:] == fill).all()
    return t, check


def close(got, want, tol):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside their bound; worst "
                           f"{float((err / tol.clamp_min(1e-30)).nan_to_num(1e9).max()):.3g} times it at "
                           f"{bad.nonzero()[0].tolist()}")


def run_window(q, k, v, lens, cfg, use_len=True):
    out, check = guarded(*q.shape, dtype=q.dtype)
    cfg.allocate_workspace(crisp.CACHE_WINDOW)
    crisp.window_attention(q, k, v, out, cfg, kv_len=lens if use_len else None)
    assert crisp.cache_device_status(cfg) == 0
    check()
    return out


# (b, hq, hkv, nq, nk, lens, window, sinks)
WINDOW = [
    (1, 1, 1, 1, 1, [1], 0, 0),                                   # one key
    (1, 4, 1, 1, 1, [0], 5, 1),                                   # nothing to see
    (2, 8, 2, 1, 65, [65, 64], 0, 0),
    (3, 28, 4, 1, 777, [777, 0, 130], 64, 4),
    (2, 32, 8, 1, 2050, [2050, 1], 1, 0),                         # a window of one: its own value
    (2, 16, 1, 1, 515, [515, 300], 100, 128),                     # 16 heads on one key head
    (5, 6, 6, 3, 100, [100, 2, 3, 0, 50], 7, 2),
    (2, 16, 1, 16, 333, [333, 20], 40, 3),                        # 256 rows of drafts
    (1, 20, 4, 5, 4099, [4099], 0, 0),
    (1, 32, 2, 13, 600, [599], 128, 600),                         # sinks cover everything
    (1, 4, 4, 17, 17, [17], 0, 0),
    (1, 4, 2, 128, 128, [128], 0, 0),
    (1, 4, 2, 129, 129, [129], 1, 0),
    (2, 8, 2, 100, 700, [700, 60], 0, 0),                         # appended chunk; a padded row block
    (2, 14, 2, 301, 301, [301, 77], 33, 5),
    (1, 7, 1, 500, 1000, [1000], 256, 128),
    (1, 4, 1, 700, 700, [700], 128, 128),
    (1, 8, 8, 257, 513, [400], 129, 1),
    (3, 3, 3, 40, 64, [64, 0, 39], 16, 64),
    (1, 16, 1, 1024, 1024, [1024], 200, 127),
    (1, 32, 8, 1000, 2000, [1999], 1000, 130),                    # sinks run into the first windows
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", WINDOW, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_window(case, dtype):
    b, hq, hkv, nq, nk, lens, window, sinks = case
    q, k, v, kv_len, cfg = make(dtype, b, hq, hkv, nq, nk, lens, window=window, sinks=sinks)
    out = run_window(q, k, v, kv_len, cfg)
    want, tol, _, _ = plain.attention(q, k, v, lens, window, sinks)
    close(out, want, tol)
    for s in range(b):      # rows that see nothing are zero, not merely small
        empty = max(0, min(nq, nq - lens[s]))
        assert (out[s, :, :empty] == 0).all()
    if all(n == nk for n in lens):
        again = run_window(q, k, v, kv_len, cfg, use_len=False)
        assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("nq", [1, 50])
def test_sharp_logits_and_scale(dtype, nq):
    """Logits of some hundreds: one key takes nearly all the weight; and a scale of the caller's."""
    q, k, v, kv_len, cfg = make(dtype, 2, 8, 2, nq, 400, [400, 399], seed=3, sharp=30.0)
    close(run_window(q, k, v, kv_len, cfg), *plain.attention(q, k, v, [400, 399])[:2])
    cfg.sm_scale = 0.013
    close(run_window(q, k, v, kv_len, cfg), *plain.attention(q, k, v, [400, 399], scale=0.013)[:2])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("nq", [2, 90])
def test_token_major_and_sliced_layouts(dtype, nq):
    """[batch, token, head, d] tensors, a slice of a longer cache, keys and values packed side by side."""
    gen = torch.Generator("cuda").manual_seed(5)
    t = DT[dtype][0]
    b, hq, hkv, nk = 2, 8, 2, 333
    q = randn(gen, b, nq, hq, D, dtype=t).transpose(1, 2)
    kv = randn(gen, b, nk + 50, hkv, 2 * D, dtype=t)[:, 10:10 + nk].transpose(1, 2)
    k, v = kv[..., :D], kv[..., D:]
    out = torch.full((b, nq, hq, D), 7.0, dtype=t, device="cuda").transpose(1, 2)
    cfg = crisp.CacheConfig(batch=b, n_q=nq, n_k=nk, h_q=hq, h_kv=hkv, dtype=DT[dtype][1], window=100, sinks=3)
    cfg.allocate_workspace(crisp.CACHE_WINDOW)
    crisp.window_attention(q, k, v, out, cfg)
    want, tol, _, _ = plain.attention(q, k, v, [nk] * b, 100, 3)
    close(out, want, tol)


SCORED = [
    (1, 1, 1, 1, 1, [1], 0, 0),
    (2, 8, 2, 1, 300, [300, 0], 0, 0),
    (3, 28, 4, 3, 1000, [1000, 2, 517], 0, 0),
    (2, 16, 1, 16, 200, [200, 9], 0, 0),
    (1, 32, 8, 1, 5000, [4990], 0, 0),
    (2, 8, 4, 2, 900, [900, 30], 50, 4),
    (1, 32, 8, 1, 512, [512], 0, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", SCORED, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_scored(case, dtype):
    b, hq, hkv, nq, nk, lens, window, sinks = case
    q, k, v, kv_len, cfg = make(dtype, b, hq, hkv, nq, nk, lens, seed=1, window=window, sinks=sinks)
    gen = torch.Generator("cuda").manual_seed(2)
    score, check = guarded(b, hkv, nk, dtype=torch.float32)
    score.copy_(torch.rand(score.shape, generator=gen, device="cuda"))
    before = score.clone()
    out, check_out = guarded(*q.shape, dtype=q.dtype)
    cfg.allocate_workspace(crisp.CACHE_SCORED)
    crisp.scored_attention(q, k, v, out, score, cfg, kv_len=kv_len)
    assert crisp.cache_device_status(cfg) == 0
    check(), check_out()
    want, tol, add, add_tol = plain.attention(q, k, v, lens, window, sinks)
    close(out, want, tol)
    close(score, before.double() + add, add_tol + plain.U * (before.double() + add))
    for s in range(b):
        dead = ~plain.seen_mask(nq, nk, lens[s], window, sinks, "cuda").any(0)
        assert torch.equal(score[s][:, dead], before[s][:, dead])
    # the added weights of a row sum to one
    rows = sum(max(0, min(nq, n)) for n in lens) * hq
    assert abs(float((score.double() - before.double()).sum()) - rows) <= 1e-4 * max(1, rows)


PREFIX = [
    (1, 1, 1, 1, 1, 1, [1]),
    (1, 4, 1, 1, 300, 20, [0]),            # only the prefix
    (3, 32, 8, 1, 777, 40, [40, 1, 17]),
    (2, 28, 4, 2, 129, 64, [64, 1]),
    (5, 16, 1, 4, 1000, 200, [200, 0, 4, 3, 150]),
    (40, 8, 2, 1, 2000, 33, list(range(0, 33)) + [33] * 7),
    (20, 14, 2, 3, 515, 70, [70] * 20),
    (33, 16, 1, 16, 260, 100, [100] * 30 + [0, 5, 16]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", PREFIX, ids=lambda c: "-".join(map(str, c[:6])))
def test_shared_prefix(case, dtype):
    b, hq, hkv, nq, npre, nk, lens = case
    q, k, v, kv_len, cfg = make(dtype, b, hq, hkv, nq, nk, lens, seed=4, n_prefix=npre)
    gen = torch.Generator("cuda").manual_seed(6)
    kp, vp = randn(gen, hkv, npre, D, dtype=q.dtype), randn(gen, npre, hkv, D, dtype=q.dtype).transpose(0, 1)
    out, check = guarded(*q.shape, dtype=q.dtype)
    cfg.allocate_workspace(crisp.CACHE_PREFIX)
    crisp.shared_prefix_attention(q, kp, vp, k, v, out, cfg, kv_len=kv_len)
    assert crisp.cache_device_status(cfg) == 0
    check()
    want, tol, _, _ = plain.attention(q, k, v, lens, k_prefix=kp, v_prefix=vp)
    close(out, want, tol)


def run_evict(k, v, score, lens, cfg):
    b, hkv = score.shape[:2]
    kn, c1 = guarded(b, hkv, cfg.n_new, D, dtype=k.dtype)
    vn, c2 = guarded(b, hkv, cfg.n_new, D, dtype=k.dtype)
    sn, c3 = guarded(b, hkv, cfg.n_new, dtype=torch.float32)
    kept, c4 = guarded(b, hkv, cfg.budget, dtype=torch.int32, fill=77)
    nl, c5 = guarded(b, dtype=torch.int32, fill=77)
    cfg.allocate_workspace(crisp.CACHE_EVICT)
    crisp.evict(k, v, score, kn, vn, sn, kept, nl, cfg, kv_len=lens)
    assert crisp.cache_device_status(cfg) == 0
    for c in (c1, c2, c3, c4, c5):
        c()
    return kn, vn, sn, kept, nl


def check_evict(k, v, score, lens, cfg, got):
    kn, vn, sn, kept, nl = got
    want = plain.evict(score, lens, cfg.sinks, cfg.recent, cfg.budget)
    assert nl.tolist() == [min(n, cfg.budget) for n in lens]
    for s in range(score.shape[0]):
        for h in range(score.shape[1]):
            w = want[s][h]
            m = len(w)
            assert kept[s, h].tolist() == w + [-1] * (cfg.budget - m), (s, h)
            at = torch.tensor(w, dtype=torch.long, device="cuda")
            # bit patterns: NaN scores and payloads move as they are
            for new, old in ((kn, k), (vn, v), (sn, score)):
                kind = torch.int16 if new.dtype == torch.bfloat16 else torch.int32
                assert torch.equal(new[s, h, :m].contiguous().view(kind), old[s, h][at].contiguous().view(kind))
            assert (kn[s, h, m:] == 7).all() and (vn[s, h, m:] == 7).all() and (sn[s, h, m:] == 0).all()


# (b, hkv, nk, lens, sinks, recent, budget, n_new)
EVICT = [
    (1, 1, 1, [1], 0, 0, 1, 1),
    (1, 1, 2, [2], 0, 0, 1, 3),
    (2, 3, 100, [100, 0], 4, 8, 50, 64),
    (3, 2, 1000, [1000, 300, 301], 0, 0, 300, 300),
    (2, 1, 5000, [4999, 5000], 128, 1024, 1152, 1200),        # no room beside the first and the last
    (1, 4, 3000, [2999], 1, 1, 2998, 3010),                   # one goes
    (2, 2, 70000, [70000, 65537], 4, 32, 4096, 4096),
    (1, 1, 40, [40], 0, 0, 100, 120),                         # a budget above the cache
    (1, 8, 20000, [20000], 0, 16384, 17000, 17000),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["normal", "ties", "odd"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_evict(case, kind, dtype):
    b, hkv, nk, lens, sinks, recent, budget, n_new = case
    gen = torch.Generator("cuda").manual_seed(9)
    k, v = randn(gen, b, hkv, nk, D, dtype=DT[dtype][0]), randn(gen, b, hkv, nk, D, dtype=DT[dtype][0])
    score = torch.exp(2 * randn(gen, b, hkv, nk))
    if kind == "ties":
        score = torch.floor(score)                # many equal, many zero
        score[:, 0] = 3.0                         # a head with one value only
        score *= torch.where(randn(gen, b, hkv, nk) > 0, 1.0, -0.0)     # zeros of both signs
    elif kind == "odd":
        pick = torch.randint(0, 8, score.shape, generator=gen, device="cuda")
        for i, x in enumerate((math.nan, math.inf, -math.inf, -1.0, 0.0, 1e-42)):
            score = torch.where(pick == i, torch.full_like(score, x), score)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cfg = crisp.CacheConfig(batch=b, n_q=1, n_k=nk, h_q=hkv, h_kv=hkv, dtype=DT[dtype][1], sinks=sinks, recent=recent,
                            budget=budget, n_new=n_new)
    check_evict(k, v, score, lens, cfg, run_evict(k, v, score, lens_t, cfg))
    if lens == [nk] * b:
        check_evict(k, v, score, lens, cfg, run_evict(k, v, score, None, cfg))


def test_evict_strided_caches():
    gen = torch.Generator("cuda").manual_seed(10)
    b, hkv, nk, n_new = 2, 3, 400, 200
    kv = randn(gen, b, nk, hkv, 2 * D, dtype=torch.bfloat16).transpose(1, 2)
    new = torch.full((b, n_new, 2, hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kn, vn = new[:, :, 0].transpose(1, 2), new[:, :, 1].transpose(1, 2)
    score = torch.rand(b, hkv, nk, generator=gen, device="cuda")
    cfg = crisp.CacheConfig(batch=b, n_q=1, n_k=nk, h_q=hkv, h_kv=hkv, sinks=2, recent=5, budget=150, n_new=n_new)
    cfg.allocate_workspace(crisp.CACHE_EVICT)
    sn = torch.empty(b, hkv, n_new, device="cuda")
    kept = torch.empty(b, hkv, 150, dtype=torch.int32, device="cuda")
    nl = torch.empty(b, dtype=torch.int32, device="cuda")
    crisp.evict(kv[..., :D], kv[..., D:], score, kn, vn, sn, kept, nl, cfg)
    check_evict(kv[..., :D], kv[..., D:], score, [nk, nk], cfg, (kn, vn, sn, kept, nl))


def test_lengths_outside_the_cache_are_clamped_and_reported():
    q, k, v, _, cfg = make("bf16", 2, 4, 2, 1, 64, [64, 64])
    cfg.allocate_workspace(crisp.CACHE_SCORED)
    lens = torch.tensor([65, -1], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    score = torch.zeros(2, 2, 64, device="cuda")
    crisp.scored_attention(q, k, v, out, score, cfg, kv_len=lens)
    assert crisp.cache_device_status(cfg) == 1
    assert crisp.cache_device_status(cfg) == 0
    want, tol, _, _ = plain.attention(q, k, v, [64, 0])
    close(out, want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("nq", [1, 64])
def test_repeated_and_captured_calls_agree_bit_for_bit(dtype, nq):
    q, k, v, lens, cfg = make(dtype, 3, 8, 2, nq, 900, [900, 100, 64], seed=8, window=300, sinks=4)
    cfg.allocate_workspace(crisp.CACHE_WINDOW)
    first, out = torch.empty_like(q), torch.empty_like(q)
    crisp.window_attention(q, k, v, first, cfg, kv_len=lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        crisp.window_attention(q, k, v, out, cfg, kv_len=lens)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        crisp.window_attention(q, k, v, out, cfg, kv_len=lens)
    for n in ([900, 100, 64], [64, 899, 0]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        k.nan_to_num_(0.5), v.nan_to_num_(0.5, 0.5, 0.5)
        out.fill_(7.0)
        graph.replay()
        crisp.window_attention(q, k, v, first, cfg, kv_len=lens)
        assert torch.equal(first, out)
        close(out, *plain.attention(q, k, v, n, 300, 4)[:2])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_captured_decode_loop_with_scores(dtype):
    """Score, then evict, captured as one graph and replayed on new inputs."""
    q, k, v, lens, cfg = make(dtype, 2, 8, 2, 1, 500, [500, 420], seed=12, sinks=4, recent=16, budget=200, n_new=256)
    k.nan_to_num_(0.5), v.nan_to_num_(0.5, 0.5, 0.5)
    cfg.sinks = 0
    cfg.allocate_workspace(crisp.CACHE_SCORED)
    score = torch.zeros(2, 2, 500, device="cuda")
    out = torch.empty_like(q)
    new = [torch.zeros(2, 2, 256, D, dtype=k.dtype, device="cuda") for _ in range(2)]
    sn, kept = torch.zeros(2, 2, 256, device="cuda"), torch.zeros(2, 2, 200, dtype=torch.int32, device="cuda")
    nl = torch.zeros(2, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            crisp.scored_attention(q, k, v, out, score, cfg, kv_len=lens)
        crisp.evict(k, v, score, *new, sn, kept, nl, cfg, kv_len=lens)
    for seed in (1, 2):
        gen = torch.Generator("cuda").manual_seed(seed)
        q.copy_(randn(gen, *q.shape))
        score.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, tol, add, add_tol = plain.attention(q, k, v, [500, 420])
        close(out, want, tol)
        close(score, 3 * add, 3 * add_tol + 9 * plain.U * add)
        assert kept.tolist() == plain.evict(score, [500, 420], 0, 16, 200)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_serving_run(dtype):
    """A prompt through the layer's dense prefill, drafts that score the cache, eviction, decoding on what stays,
    and a batch that shares the kept cache as its prefix."""
    gen = torch.Generator("cuda").manual_seed(20)
    t, code = DT[dtype]
    hq, hkv, n, slots = 8, 2, 512, 640
    q, k, v = randn(gen, 1, hq, n, D, dtype=t), randn(gen, 1, hkv, slots, D, dtype=t), randn(gen, 1, hkv, slots, D, dtype=t)
    # the prompt: dense prefill and the window operator without a window agree
    pre = crisp.Config(n=n, h_q=hq, h_kv=hkv, dtype=code)
    pre.allocate_workspace()
    dense = torch.empty_like(q[0])
    crisp.dense_attention(q[0], k[0, :, :n].contiguous(), v[0, :, :n].contiguous(), dense, pre)
    cfg = crisp.CacheConfig(batch=1, n_q=n, n_k=slots, h_q=hq, h_kv=hkv, dtype=code)
    cfg.allocate_workspace(crisp.CACHE_WINDOW)
    out = torch.empty_like(q)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    crisp.window_attention(q, k, v, out, cfg, kv_len=lens)
    want, tol, _, _ = plain.attention(q, k, v, [n])
    close(out, want, tol)
    assert float((out[0].double() - dense.double()).norm() / dense.double().norm()) < (1e-2 if dtype == "bf16" else 1e-5)
    # drafts of 1, 4 and 16 tokens score the cache
    score = torch.zeros(1, hkv, slots, device="cuda")
    total = torch.zeros(1, hkv, slots, dtype=torch.float64, device="cuda")
    bound = total.clone()
    for step in (1, 4, 16):
        lens += step
        c = crisp.CacheConfig(batch=1, n_q=step, n_k=slots, h_q=hq, h_kv=hkv, dtype=code)
        c.allocate_workspace(crisp.CACHE_SCORED)
        qd = randn(gen, 1, hq, step, D, dtype=t)
        o = torch.empty_like(qd)
        crisp.scored_attention(qd, k, v, o, score, c, kv_len=lens)
        want, tol, add, add_tol = plain.attention(qd, k, v, lens.tolist())
        close(o, want, tol)
        total += add
        bound += add_tol + plain.U * total
    close(score, total, bound)
    # eviction to 200 keys in a cache of 256 slots, then a decode through a window on it
    ev = crisp.CacheConfig(batch=1, n_q=1, n_k=slots, h_q=hq, h_kv=hkv, dtype=code, sinks=4, recent=32, budget=200,
                           n_new=256)
    got = run_evict(k, v, score, lens, ev)
    check_evict(k, v, score, lens.tolist(), ev, got)
    kn, vn, _, _, nl = got
    c = crisp.CacheConfig(batch=1, n_q=1, n_k=256, h_q=hq, h_kv=hkv, dtype=code, window=50, sinks=4)
    qd = randn(gen, 1, hq, 1, D, dtype=t)
    close(run_window(qd, kn, vn, nl, c), *plain.attention(qd, kn, vn, [200], 50, 4)[:2])
    # six requests on the kept keys as their shared prefix
    b = 6
    c = crisp.CacheConfig(batch=b, n_q=1, n_k=64, h_q=hq, h_kv=hkv, dtype=code, n_prefix=200)
    c.allocate_workspace(crisp.CACHE_PREFIX)
    ks, vs, qd = (randn(gen, b, h, m, D, dtype=t) for h, m in ((hkv, 64), (hkv, 64), (hq, 1)))
    sl = torch.tensor([0, 1, 7, 30, 63, 64], dtype=torch.int32, device="cuda")
    o = torch.empty_like(qd)
    crisp.shared_prefix_attention(qd, kn[0, :, :200], vn[0, :, :200], ks, vs, o, c, kv_len=sl)
    close(o, *plain.attention(qd, ks, vs, sl.tolist(), k_prefix=kn[0, :, :200], v_prefix=vn[0, :, :200])[:2])


@pytest.mark.parametrize("kind", ["normal", "ties"])
@pytest.mark.parametrize("n", [300000, 350000])
def test_evict_long(n, kind):
    """Stretches of more than one round of words, and more than shared memory holds."""
    gen = torch.Generator("cuda").manual_seed(13)
    k, v = randn(gen, 1, 1, n, D, dtype=torch.bfloat16), randn(gen, 1, 1, n, D, dtype=torch.bfloat16)
    score = torch.exp(2 * randn(gen, 1, 1, n))
    if kind == "ties":
        score = torch.floor(score / 4)
    cfg = crisp.CacheConfig(batch=1, n_q=1, n_k=n, h_q=1, h_kv=1, sinks=5, recent=77, budget=150001, n_new=150016)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    check_evict(k, v, score, [n], cfg, run_evict(k, v, score, lens, cfg))


def test_offsets_past_32_bits():
    """The last sequence of a cache whose elements number more than 2^31, in every operator."""
    gen = torch.Generator("cuda").manual_seed(14)
    b, hq, hkv, nk = 3, 16, 8, 1 << 20
    k = torch.zeros(b, hkv, nk, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    n = 3000
    for t in (k, v):
        t[:, :, :n] = randn(gen, b, hkv, n, D, dtype=torch.bfloat16)
    lens = [1, 0, n]
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    small = (k[:, :, :n], v[:, :, :n])
    for nq in (1, 40):
        cfg = crisp.CacheConfig(batch=b, n_q=nq, n_k=nk, h_q=hq, h_kv=hkv, window=700, sinks=3)
        q = randn(gen, b, hq, nq, D, dtype=torch.bfloat16)
        close(run_window(q, k, v, kv_len, cfg), *plain.attention(q, *small, lens, 700, 3)[:2])
    score = torch.zeros(b, hkv, nk, device="cuda")
    cfg = crisp.CacheConfig(batch=b, n_q=1, n_k=nk, h_q=hq, h_kv=hkv)
    cfg.allocate_workspace(crisp.CACHE_SCORED)
    q = randn(gen, b, hq, 1, D, dtype=torch.bfloat16)
    out = torch.empty_like(q)
    crisp.scored_attention(q, k, v, out, score, cfg, kv_len=kv_len)
    want, tol, add, add_tol = plain.attention(q, *small, lens)
    close(out, want, tol)
    close(score[:, :, :n], add, add_tol + plain.U * add)
    assert (score[:, :, n:] == 0).all()
    cfg = crisp.CacheConfig(batch=b, n_q=1, n_k=nk, h_q=hq, h_kv=hkv, sinks=3, recent=50, budget=500, n_new=512)
    check_evict(k, v, score, lens, cfg, run_evict(k, v, score, kv_len, cfg))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_short_sequences(dtype):
    """The largest batch, of caches of 0 to 40 tokens."""
    b = 1024
    lens = [(i * 7) % 41 for i in range(b)]
    q, k, v, kv_len, cfg = make(dtype, b, 4, 2, 1, 40, lens, seed=15, n_prefix=33, sinks=0, recent=3, budget=20, n_new=21)
    cfg.allocate_workspace(crisp.CACHE_SCORED)
    score, out = torch.zeros(b, 2, 40, device="cuda"), torch.empty_like(q)
    crisp.scored_attention(q, k, v, out, score, cfg, kv_len=kv_len)
    want, tol, add, add_tol = plain.attention(q, k, v, lens)
    close(out, want, tol)
    close(score, add, add_tol + plain.U * add)
    check_evict(k, v, score, lens, cfg, run_evict(k, v, score, kv_len, cfg))
    gen = torch.Generator("cuda").manual_seed(16)
    kp, vp = (randn(gen, 2, 33, D, dtype=q.dtype) for _ in range(2))
    cfg.allocate_workspace(crisp.CACHE_PREFIX)
    crisp.shared_prefix_attention(q, kp, vp, k, v, out, cfg, kv_len=kv_len)
    close(out, *plain.attention(q, k, v, lens, k_prefix=kp, v_prefix=vp)[:2])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_calls_in_a_chain(dtype):
    """Each call's output is the next one's query, and the scores run on: no kernel may start on what the one before
    has not finished. With a wait after every call the results are the same to the bit."""
    gen = torch.Generator("cuda").manual_seed(17)
    t, code = DT[dtype]
    b, hq, hkv, nk = 3, 8, 2, 700
    k, v = randn(gen, b, hkv, nk, D, dtype=t), randn(gen, b, hkv, nk, D, dtype=t)
    kp, vp = randn(gen, hkv, 900, D, dtype=t), randn(gen, hkv, 900, D, dtype=t)
    q0 = randn(gen, b, hq, 2, D, dtype=t)
    lens = torch.tensor([700, 3, 350], dtype=torch.int32, device="cuda")
    cfg = crisp.CacheConfig(batch=b, n_q=2, n_k=nk, h_q=hq, h_kv=hkv, dtype=code)
    pre = crisp.CacheConfig(batch=b, n_q=2, n_k=nk, h_q=hq, h_kv=hkv, dtype=code, n_prefix=900)
    cfg.workspace = pre.workspace = torch.empty(max(crisp.cache_workspace_size(cfg, crisp.CACHE_SCORED),
                                                    crisp.cache_workspace_size(pre, crisp.CACHE_PREFIX)),
                                                dtype=torch.uint8, device="cuda")

    def run(wait):
        a, c = q0.clone(), torch.empty_like(q0)
        score = torch.zeros(b, hkv, nk, device="cuda")
        for _ in range(20):
            crisp.scored_attention(a, k, v, c, score, cfg, kv_len=lens)
            wait()
            c.mul_(8)
            crisp.shared_prefix_attention(c, kp, vp, k, v, a, pre, kv_len=lens)
            wait()
            crisp.window_attention(a, k, v, c, cfg, kv_len=lens)
            wait()
            a.copy_(c).mul_(8)
        torch.cuda.synchronize()
        return a, c, score

    for x, y in zip(run(lambda: None), run(torch.cuda.synchronize)):
        assert torch.equal(x, y)
        assert torch.isfinite(x).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("b", [2, 40])
def test_shared_prefix_captured_and_on_another_stream(dtype, b):
    gen = torch.Generator("cuda").manual_seed(18)
    t, code = DT[dtype]
    hq, hkv, nk, npre = 8, 2, 60, 700
    q, k, v, kp, vp = (randn(gen, *s, D, dtype=t) for s in ((b, hq, 1), (b, hkv, nk), (b, hkv, nk), (hkv, npre), (hkv, npre)))
    lens = torch.full((b,), nk, dtype=torch.int32, device="cuda")
    cfg = crisp.CacheConfig(batch=b, n_q=1, n_k=nk, h_q=hq, h_kv=hkv, dtype=code, n_prefix=npre)
    cfg.allocate_workspace(crisp.CACHE_PREFIX)
    out, other = torch.empty_like(q), torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        crisp.shared_prefix_attention(q, kp, vp, k, v, out, cfg, kv_len=lens)
    side = torch.cuda.Stream()
    for n in (nk, 13):
        lens.fill_(n)
        q.copy_(randn(gen, *q.shape))
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        crisp.shared_prefix_attention(q, kp, vp, k, v, other, cfg, kv_len=lens, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, other)
        close(out, *plain.attention(q, k, v, [n] * b, k_prefix=kp, v_prefix=vp)[:2])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("nq", [40, 5])
def test_lengths_outside_the_cache_in_every_kernel(dtype, nq):
    """Prompt and flat-list kernels, and eviction: clamped to [0, n_k], reported once."""
    nk, lens = 4200, [1 << 30, -5, 100]
    q, k, v, _, cfg = make(dtype, 3, 16, 1, nq, nk, [nk, nk, nk], seed=21, window=300, sinks=2, recent=4, budget=70, n_new=70)
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k.nan_to_num_(0.5), v.nan_to_num_(0.5, 0.5, 0.5)
    out, check = guarded(*q.shape, dtype=q.dtype)
    cfg.allocate_workspace(crisp.CACHE_WINDOW)
    crisp.window_attention(q, k, v, out, cfg, kv_len=kv_len)
    assert crisp.cache_device_status(cfg) == 1 and crisp.cache_device_status(cfg) == 0
    check()
    real = [nk, 0, 100]
    close(out, *plain.attention(q, k, v, real, 300, 2)[:2])
    score = torch.rand(3, 1, nk, device="cuda")
    cfg.allocate_workspace(crisp.CACHE_EVICT)
    got = [torch.full((3, 1, 70, D), 7.0, dtype=k.dtype, device="cuda") for _ in range(2)]
    got += [torch.zeros(3, 1, 70, device="cuda"), torch.zeros(3, 1, 70, dtype=torch.int32, device="cuda"),
            torch.zeros(3, dtype=torch.int32, device="cuda")]
    crisp.evict(k, v, score, *got, cfg, kv_len=kv_len)
    assert crisp.cache_device_status(cfg) == 1
    check_evict(k, v, score, real, cfg, got)
