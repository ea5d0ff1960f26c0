"""Paths of the cache operators that single out a kernel form, on the GPU
against the definitions in 64 bits (tests/cache_plain.py derives the
tolerances; tests/test_cache_plans.py checks that the shapes take the path)."""
import math

import pytest

import cache_plain as plain
import cache_shapes as shapes

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import long_context_prefill_last_b200 as crisp  # noqa: E402
from test_gpu_cache import D, built, close, guarded, make, randn, run_window  # noqa: E402, F401


@pytest.mark.parametrize("case", [c for c, _ in shapes.TWO_TILES], ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_window_with_two_row_tiles(case):
    b, hq, hkv, nq, nk, lens, window, sinks = case
    q, k, v, kv_len, cfg = make("bf16", b, hq, hkv, nq, nk, lens, seed=30, window=window, sinks=sinks)
    out = run_window(q, k, v, kv_len, cfg)
    want, tol, _, _ = plain.attention(q, k, v, lens, window, sinks)
    close(out, want, tol)
    for s in range(b):
        empty = max(0, min(nq, nq - lens[s]))
        assert (out[s, :, :empty] == 0).all()
    assert torch.equal(out, run_window(q, k, v, kv_len, cfg))


def test_token_major_layout_with_two_row_tiles():
    gen = torch.Generator("cuda").manual_seed(31)
    b, hq, hkv, nq, nk = 2, 14, 2, 1900, 2300
    q = randn(gen, b, nq, hq, D, dtype=torch.bfloat16).transpose(1, 2)
    kv = randn(gen, b, nk + 7, hkv, 2 * D, dtype=torch.bfloat16)[:, 7:].transpose(1, 2)
    k, v = kv[..., :D], kv[..., D:]
    buf, check = guarded(b, nq, hq, D, dtype=torch.bfloat16)
    out = buf.transpose(1, 2)
    cfg = crisp.CacheConfig(batch=b, n_q=nq, n_k=nk, h_q=hq, h_kv=hkv, window=1850, sinks=33)
    cfg.allocate_workspace(crisp.CACHE_WINDOW)
    crisp.window_attention(q, k, v, out, cfg)
    assert crisp.cache_device_status(cfg) == 0
    check()
    close(out, *plain.attention(q, k, v, [nk] * b, 1850, 33)[:2])


@pytest.mark.parametrize("case", shapes.SKEWED, ids=lambda c: "-".join(map(str, c)))
def test_one_long_sequence_among_short_ones(case):
    b, hq, hkv, nq, nk = case
    lens = [(7 * s) % 60 for s in range(b)]
    lens[b // 2] = nk
    q, k, v, kv_len, cfg = make("bf16", b, hq, hkv, nq, nk, lens, seed=32)
    out = run_window(q, k, v, kv_len, cfg)
    want, tol, add, add_tol = plain.attention(q, k, v, lens)
    close(out, want, tol)
    cfg.allocate_workspace(crisp.CACHE_SCORED)
    score = torch.zeros(b, hkv, nk, device="cuda")
    crisp.scored_attention(q, k, v, out, score, cfg, kv_len=kv_len)
    assert crisp.cache_device_status(cfg) == 0
    close(out, want, tol)
    close(score, add, add_tol + plain.U * add)


def test_device_status_works_on_its_stream():
    """Reading and clearing the status waits for its own stream only, so that what follows there comes after it."""
    q, k, v, _, cfg = make("bf16", 1, 4, 2, 1, 64, [64])
    cfg.allocate_workspace(crisp.CACHE_WINDOW)
    lens = torch.tensor([65], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):      # the first call loads the kernels
        crisp.window_attention(q, k, v, out, cfg, kv_len=lens, stream=side)
        assert crisp.cache_device_status(cfg, side) == 1
    crisp.window_attention(q, k, v, out, cfg, kv_len=lens, stream=side)
    torch.cuda._sleep(1_000_000_000)        # half a second on the current stream
    busy = torch.cuda.Event()
    busy.record()
    assert crisp.cache_device_status(cfg, side) == 1
    assert crisp.cache_device_status(cfg, side) == 0
    assert not busy.query()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", shapes.WIDE_DRAFTS, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_drafts_of_many_rows(case, dtype):
    """Through a window, with scores, and behind a shared prefix."""
    b, hq, hkv, nq, nk, lens, window, sinks = case
    q, k, v, kv_len, cfg = make(dtype, b, hq, hkv, nq, nk, lens, seed=33, window=window, sinks=sinks)
    out = run_window(q, k, v, kv_len, cfg)
    want, tol, add, add_tol = plain.attention(q, k, v, lens, window, sinks)
    close(out, want, tol)
    score, check = guarded(b, hkv, nk, dtype=torch.float32, fill=0.0)
    cfg.allocate_workspace(crisp.CACHE_SCORED)
    crisp.scored_attention(q, k, v, out, score, cfg, kv_len=kv_len)
    assert crisp.cache_device_status(cfg) == 0
    check()
    close(out, want, tol)
    close(score, add, add_tol + plain.U * add)
    gen = torch.Generator("cuda").manual_seed(34)
    for npre in (1, 500, 2500):
        q, k, v, kv_len, cfg = make(dtype, b, hq, hkv, nq, nk, lens, seed=35, n_prefix=npre)
        kp, vp = (randn(gen, hkv, npre, D, dtype=q.dtype) for _ in range(2))
        out, check = guarded(*q.shape, dtype=q.dtype)
        cfg.allocate_workspace(crisp.CACHE_PREFIX)
        crisp.shared_prefix_attention(q, kp, vp, k, v, out, cfg, kv_len=kv_len)
        assert crisp.cache_device_status(cfg) == 0
        check()
        close(out, *plain.attention(q, k, v, lens, k_prefix=kp, v_prefix=vp)[:2])


@pytest.mark.parametrize("path,delta,held", [("decode", 1.2, 0), ("tile", 1.7, 64)])
def test_long_fp32_sums_of_like_weights(path, delta, held):
    """Keys that all weigh 2^-delta of a few first ones: a CTA's sums run over thousands of equal tiles, where the
    roundings of a plain running sum fall to one side (off by 4e-5 and 3e-5 here).

    Bounds, from u = 2^-24 and the arithmetic alone. q and k have one dimension that is not zero, so a logit is one
    product (u), scaled (u, and 2 u for the scale itself), subtracted (u) and of a key rounded to fp32 (u): off by 6 u of
    the larger logit in base 2, which a weight's relative error stays below. An exponential is off by 2^-21 at most.
    The denominator: 8 additions inside a tile, then a compensated sum (2 u) or `held` tiles at a time (held + tiles /
    held), then 4 pieces. A score: two exponentials' errors, the denominator's, up to 36 rows added. An output: every
    value is the same, so the weights' errors cancel; a chain of 64 inside a tile and over tiles as before, twice."""
    (b, hq, hkv, nq, nk), tiles = shapes.LONG_RUNS_DECODE if path == "decode" else shapes.LONG_RUNS_TILE
    first = 200
    # sequence s, head h: the same keys from token s + h on, with 50 heavy keys or more in front
    gen = torch.Generator("cuda").manual_seed(36)
    keys = torch.zeros(nk + first, D, device="cuda")
    x = 2.5
    keys[:first, 5] = x
    keys[first:, 5] = x - delta
    values = torch.randn(D, generator=gen, device="cuda").expand(nk + first, D).contiguous()
    step = 128
    k, v = (t.as_strided((b, hkv, nk, D), (step, step, D, 1)) for t in (keys, values))
    q = torch.zeros(b, hq, nq, D, device="cuda")
    q[..., 5] = 1.0
    cfg = crisp.CacheConfig(batch=b, n_q=nq, n_k=nk, h_q=hq, h_kv=hkv, dtype=crisp.FP32, sm_scale=math.log(2))
    cfg.allocate_workspace(crisp.CACHE_SCORED)
    out, score = torch.empty_like(q), torch.zeros(b, hkv, nk, device="cuda")
    crisp.scored_attention(q, k, v, out, score, cfg)
    assert crisp.cache_device_status(cfg) == 0
    u = plain.U
    over = (held + tiles / held if held else 2) + 4
    rel_score = 2 * (6 * u * x + 2.0 ** -21) + (8 + over + 36) * u
    rel_out = (8 + 64 + 2 * over) * u
    for s, h in ((0, 0), (b - 1, hkv - 1), (b // 2, 0)):
        heavy = first - s - h
        w = torch.full((nk,), 2.0 ** -delta, dtype=torch.float64, device="cuda")
        w[:heavy] = 1.0
        place = nk - nq + torch.arange(nq, device="cuda")[:, None]
        p = torch.where(torch.arange(nk, device="cuda") <= place, w, torch.zeros_like(w))
        p = p / p.sum(1, keepdim=True)
        want = p.sum(0) * (hq // hkv)
        close(score[s, h], want, want * rel_score)
        want = values[0].double().expand(hq // hkv, nq, D)
        close(out[s, h * (hq // hkv):(h + 1) * (hq // hkv)], want, want.abs() * rel_out)


@pytest.mark.parametrize("case", [(1, 2, 2, 5000, 5000, [5000], 0, 0), (2, 4, 4, 2500, 14000, [14000, 9000], 0, 3),
                                  (2, 48, 16, 3, 9000, [9000, 8998], 0, 0)],
                         ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_fp32_prompts_of_more_tiles_than_registers_hold(case):
    b, hq, hkv, nq, nk, lens, window, sinks = case
    q, k, v, kv_len, cfg = make("fp32", b, hq, hkv, nq, nk, lens, seed=37, sharp=2.0, window=window, sinks=sinks)
    want, tol, _, _ = plain.attention(q, k, v, lens, window, sinks)
    out = run_window(q, k, v, kv_len, cfg)
    close(out, want, tol)
    assert torch.equal(out, run_window(q, k, v, kv_len, cfg))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", [(3, 28, 4, 1, 500), (2, 8, 2, 16, 6000), (2, 28, 4, 16, 600), (1, 4, 2, 4500, 4500),
                                  (1, 16, 1, 60, 5000), (37, 32, 8, 1, 2500)], ids=lambda c: "-".join(map(str, c)))
def test_outputs_in_place_of_the_queries(case, dtype):
    b, hq, hkv, nq, nk = case
    q, k, v, lens, cfg = make(dtype, b, hq, hkv, nq, nk, [nk - 3 * s for s in range(b)], seed=38, n_prefix=900)
    out, same = run_window(q, k, v, lens, cfg), q.clone()
    crisp.window_attention(same, k, v, same, cfg, kv_len=lens)
    assert torch.equal(out, same)
    if nq > 16:
        return
    cfg.allocate_workspace(crisp.CACHE_SCORED)
    scores = [torch.zeros(b, hkv, nk, device="cuda") for _ in range(2)]
    same = q.clone()
    crisp.scored_attention(q, k, v, out, scores[0], cfg, kv_len=lens)
    crisp.scored_attention(same, k, v, same, scores[1], cfg, kv_len=lens)
    assert torch.equal(out, same) and torch.equal(*scores)
    gen = torch.Generator("cuda").manual_seed(39)
    kp, vp = (randn(gen, hkv, 900, D, dtype=q.dtype) for _ in range(2))
    cfg.allocate_workspace(crisp.CACHE_PREFIX)
    same = q.clone()
    crisp.shared_prefix_attention(q, kp, vp, k, v, out, cfg, kv_len=lens)
    crisp.shared_prefix_attention(same, kp, vp, k, v, same, cfg, kv_len=lens)
    assert torch.equal(out, same)
