"""The plans of the cache operators: which kernel, row tiles, pieces and
clusters a shape takes (host code only, no GPU needed)."""
import ctypes
import os
import subprocess

import pytest

import cache_shapes as shapes
import long_context_prefill_last_b200 as crisp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIMT_TILE, DECODE_MMA, TILE_TC, DECODE_SIMT = range(4)

PROGRAM = r"""
#include <stdio.h>
#include "cache.h"
int main() {
  int op, batch, n_q, n_k, h_q, h_kv, fp32, window, sinks, n_prefix;
  while (scanf("%d %d %d %d %d %d %d %d %d %d", &op, &batch, &n_q, &n_k, &h_q, &h_kv, &fp32, &window, &sinks,
               &n_prefix) == 10) {
    crisp::CacheShape s{};
    s.batch = batch, s.n_q = n_q, s.n_k = n_k, s.h_q = h_q, s.h_kv = h_kv, s.group = h_q / h_kv;
    s.window = window == 0 ? crisp::kNoWindow : window;
    s.sinks = sinks < n_k ? sinks : n_k;
    s.n_prefix = n_prefix, s.fp32 = fp32 != 0;
    const crisp::CachePlan p = crisp::plan_cache(s, op);
    const crisp::AttnPlan& a = p.main;
    printf("%d %d %d %d %d %d %d %zu\n", a.kernel, a.block, a.blocks, a.splits, a.row_tiles, a.cluster, a.ctas, p.total);
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from long_context_prefill_last_b200 import build
    lib = build.build()
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cc").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I" + build.INCLUDE, "-I" + build.CSRC, "-I/usr/local/cuda/include",
                    str(at / "plan.cc"), lib, "-o", str(at / "plan")], check=True)

    def of(op, batch, hq, hkv, nq, nk, window=0, sinks=0, n_prefix=0, fp32=0):
        line = " ".join(str(x) for x in (op, batch, nq, nk, hq, hkv, fp32, window, sinks, n_prefix))
        out = subprocess.run([str(at / "plan")], input=line, capture_output=True, text=True, check=True,
                             env={**os.environ, "LD_LIBRARY_PATH": os.path.dirname(lib)}).stdout.split()
        names = ("kernel", "block", "blocks", "splits", "row_tiles", "cluster", "ctas", "total")
        got = dict(zip(names, map(int, out)))
        cfg = crisp.CacheConfig(batch=batch, n_q=nq, n_k=nk, h_q=hq, h_kv=hkv, dtype=crisp.FP32 if fp32 else crisp.BF16,
                                window=window, sinks=sinks, n_prefix=n_prefix)
        size = ctypes.c_size_t(0)
        assert crisp.lib().crisp_cache_workspace_size(ctypes.byref(cfg._c()), op, ctypes.byref(size)) == 0
        assert size.value == got["total"]      # the plan that the library itself makes
        return got

    return of


@pytest.mark.parametrize("case,split", shapes.TWO_TILES, ids=lambda c: "-".join(map(str, c)).replace(" ", "")
                         if isinstance(c, tuple) else "")
def test_long_key_lists_take_two_row_tiles(plan, case, split):
    b, hq, hkv, nq, nk, _, window, sinks = case
    p = plan(crisp.CACHE_WINDOW, b, hq, hkv, nq, nk, window, sinks)
    assert (p["kernel"], p["block"]) == (TILE_TC, 256)
    assert (p["splits"] > 1) == split


def test_two_row_tile_shapes_include_a_cta_without_a_second_one(plan):
    odd = [plan(crisp.CACHE_WINDOW, *c[:5], c[6], c[7])["row_tiles"] % 2 for c, _ in shapes.TWO_TILES]
    assert 0 in odd and 1 in odd


@pytest.mark.parametrize("op", [crisp.CACHE_WINDOW, crisp.CACHE_SCORED])
def test_a_cluster_never_walks_a_long_list_alone(plan, op):
    """Lengths are unknown to the plan: in a batch of one full sequence and many short ones a cluster's CTAs walk the
    full one alone, so their share has to stay small whatever the flat list's share of a full batch would be."""
    took = 0
    for b, hq, hkv, nq in ((1, 32, 8, 1), (8, 32, 8, 1), (36, 32, 8, 1), (37, 32, 8, 1), (74, 28, 4, 3), (148, 32, 2, 1),
                           (296, 8, 1, 2), (37, 32, 8, 7)):
        for nk in (512, 1024, 2048, 4096, 9472, 131072):
            p = plan(op, b, hq, hkv, nq, nk)
            if p["cluster"] == 0:
                continue
            took += 1
            share = -(-(-(-nk // 64)) // p["cluster"]) * (p["block"] // 16)
            assert share <= (12 if op == crisp.CACHE_SCORED else 20), (b, hq, hkv, nq, nk, p)
    assert took > 8
    for case in shapes.SKEWED:
        assert plan(op, *case)["cluster"] == 0
    # short caches and windows keep their one launch
    assert plan(op, 1, 32, 8, 1, 512)["cluster"] == 8
    assert plan(op, 37, 32, 8, 1, 512)["cluster"] == 1
    if op == crisp.CACHE_WINDOW:
        assert plan(op, 32, 32, 8, 1, 8192, 1024, 4)["cluster"] == 1


def test_drafts_that_one_job_cannot_hold_read_their_keys_once(plan):
    """Above 64 rows the decode kernel would read every key once per 64 rows; only scores need it."""
    for c in shapes.WIDE_DRAFTS:
        b, hq, hkv, nq, nk, _, window, sinks = c
        assert nq * hq // hkv > 64
        assert plan(crisp.CACHE_WINDOW, b, hq, hkv, nq, nk, window, sinks)["kernel"] == TILE_TC
        assert plan(crisp.CACHE_PREFIX, b, hq, hkv, nq, nk, n_prefix=500)["kernel"] == TILE_TC
        assert plan(crisp.CACHE_SCORED, b, hq, hkv, nq, nk, window, sinks)["kernel"] == DECODE_MMA
    for op in (crisp.CACHE_WINDOW, crisp.CACHE_PREFIX):
        assert plan(op, 2, 28, 4, 9, 5000, n_prefix=500)["kernel"] == DECODE_MMA     # 63 rows
        assert plan(op, 2, 32, 8, 16, 5000, n_prefix=500)["kernel"] == DECODE_MMA    # 64
        assert plan(op, 2, 28, 4, 10, 5000, n_prefix=500)["kernel"] == TILE_TC       # 70
    assert plan(crisp.CACHE_WINDOW, 2, 4, 4, 17, 5000)["kernel"] == TILE_TC           # a prompt
    assert plan(crisp.CACHE_WINDOW, 2, 4, 4, 17, 5000, fp32=1)["kernel"] == DECODE_SIMT
    assert plan(crisp.CACHE_SCORED, 2, 28, 4, 16, 5000, fp32=1)["kernel"] == SIMT_TILE


def test_fp32_long_runs(plan):
    (b, hq, hkv, nq, nk), tiles = shapes.LONG_RUNS_DECODE
    p = plan(crisp.CACHE_SCORED, b, hq, hkv, nq, nk, fp32=1)
    assert p["kernel"] == DECODE_SIMT and b * hkv * p["blocks"] * (nk // 32) == tiles * p["ctas"]
    (b, hq, hkv, nq, nk), tiles = shapes.LONG_RUNS_TILE
    p = plan(crisp.CACHE_SCORED, b, hq, hkv, nq, nk, fp32=1)
    assert p["kernel"] == SIMT_TILE and p["splits"] == 1 and nk // 64 == tiles
