"""The cache operators' host side: struct layout, workspace sizes, and the
refusal of bad arguments before anything is launched (no GPU needed)."""
import ctypes
import os
import subprocess
import tempfile

import pytest

import long_context_prefill_last_b200 as crisp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20     # an aligned address that is never read: every call below is refused


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_prefill_last_b200 import build
    build.build()


def make(**kw):
    d = dict(batch=2, n_q=1, n_k=1000, h_q=32, h_kv=8, n_prefix=100, budget=64, n_new=64)
    d.update(kw)
    cfg = crisp.CacheConfig(**d)
    c = cfg._c()
    c.workspace, c.workspace_bytes = 1 << 30, 1 << 40
    return c


def call(op, c, **kw):
    """The entry point of operator op on stand-in pointers."""
    L = crisp.lib()
    r = ctypes.byref(c) if c is not None else None
    a = dict(q=P, k=2 * P, v=3 * P, out=4 * P, kv_len=5 * P, score=6 * P, kp=7 * P, vp=8 * P, kn=1 << 40, vn=1 << 41,
             sn=9 * P, kept=10 * P, new_len=11 * P)
    a.update(kw)
    if op == crisp.CACHE_WINDOW:
        return L.crisp_window_attention(a["q"], a["k"], a["v"], a["out"], a["kv_len"], r, None)
    if op == crisp.CACHE_SCORED:
        return L.crisp_scored_attention(a["q"], a["k"], a["v"], a["out"], a["score"], a["kv_len"], r, None)
    if op == crisp.CACHE_PREFIX:
        return L.crisp_shared_prefix_attention(a["q"], a["kp"], a["vp"], a["k"], a["v"], a["out"], a["kv_len"], r, None)
    return L.crisp_evict(a["k"], a["v"], a["score"], a["kv_len"], a["kn"], a["vn"], a["sn"], a["kept"], a["new_len"], r,
                         None)


OPS = [crisp.CACHE_WINDOW, crisp.CACHE_SCORED, crisp.CACHE_PREFIX, crisp.CACHE_EVICT]
ATTEND = OPS[:3]


def test_struct_layout_matches_header():
    src = r"""
    #include <stdio.h>
    #include <stddef.h>
    #include "crisp.h"
    int main(void) {
      printf("%zu %zu %zu %zu %zu\n", sizeof(crisp_cache_cfg), offsetof(crisp_cache_cfg, sm_scale),
             offsetof(crisp_cache_cfg, q), offsetof(crisp_cache_cfg, v_new), offsetof(crisp_cache_cfg, workspace_bytes));
      return 0;
    }"""
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(c, "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        vals = [int(x) for x in subprocess.run([exe], capture_output=True, text=True).stdout.split()]
    C = crisp._CacheCfg
    assert vals == [ctypes.sizeof(C), C.sm_scale.offset, C.q.offset, C.v_new.offset, C.workspace_bytes.offset]


def test_cfg_init_matches_python_config():
    c = crisp._CacheCfg()
    assert crisp.lib().crisp_cache_cfg_init(ctypes.byref(c), 3, 2, 500, 28, 4, 128, crisp.BF16) == 0
    assert bytes(c) == bytes(crisp.CacheConfig(batch=3, n_q=2, n_k=500, h_q=28, h_kv=4)._c())
    assert crisp.lib().crisp_cache_cfg_init(None, 3, 2, 500, 28, 4, 128, crisp.BF16) == 1


def test_changed_config_makes_a_new_struct():
    cfg = crisp.CacheConfig(batch=1, n_q=1, n_k=64, h_q=8, h_kv=8)
    torch = pytest.importorskip("torch")
    names, t = ("k",), [torch.zeros(1, 8, 64, 128)]
    ref = cfg._ref(names, t)
    assert cfg._ref(names, t) is ref
    cfg.window = 7
    assert cfg._ref(names, t)._obj.window == 7
    assert cfg._ref(names, [torch.zeros(1, 64, 8, 128).transpose(1, 2)])._obj.k.head == 128


@pytest.mark.parametrize("op", OPS)
def test_workspace_sizes(op):
    cfg = crisp.CacheConfig(batch=4, n_q=1, n_k=4096, h_q=32, h_kv=8, n_prefix=1000, budget=100, n_new=100)
    n = crisp.cache_workspace_size(cfg, op)
    assert n >= 256 and n % 256 == 0
    assert n < 1 << 28
    out = ctypes.c_size_t(0)
    assert crisp.lib().crisp_cache_workspace_size(ctypes.byref(cfg._c()), 4, ctypes.byref(out)) == 1
    assert crisp.lib().crisp_cache_workspace_size(ctypes.byref(cfg._c()), op, None) == 1


BAD = [
    (OPS, dict(reserved=1), 1), (OPS, dict(dtype=2), 3), (OPS, dict(d=64), 2), (OPS, dict(batch=0), 2),
    (OPS, dict(batch=1025, h_q=8), 2), (OPS, dict(batch=65, h_q=1024, h_kv=1024), 2), (OPS, dict(n_k=0), 2),
    (OPS, dict(n_k=(1 << 24) + 1), 2), (OPS, dict(h_q=30), 2), (OPS, dict(h_q=34, h_kv=2), 2), (OPS, dict(h_kv=0), 2),
    (OPS, dict(sm_scale=float("nan")), 1), (OPS, dict(sm_scale=float("inf")), 1), (OPS, dict(window=-1), 1),
    (OPS, dict(sinks=-1), 1),
    (ATTEND, dict(n_q=0), 2), (ATTEND, dict(n_q=1001), 2),
    (ATTEND[1:], dict(n_q=17), 2),
    ([crisp.CACHE_PREFIX], dict(n_prefix=0), 2), ([crisp.CACHE_PREFIX], dict(n_prefix=(1 << 24) + 1), 2),
    ([crisp.CACHE_PREFIX], dict(window=5), 6), ([crisp.CACHE_PREFIX], dict(sinks=5), 6),
    ([crisp.CACHE_EVICT], dict(budget=0), 1), ([crisp.CACHE_EVICT], dict(recent=-1), 1),
    ([crisp.CACHE_EVICT], dict(sinks=33, recent=32), 1), ([crisp.CACHE_EVICT], dict(sinks=2**31 - 1, recent=2**31 - 1), 1),
    ([crisp.CACHE_EVICT], dict(n_new=63), 2), ([crisp.CACHE_EVICT], dict(n_new=(1 << 24) + 1), 2),
]


@pytest.mark.parametrize("ops,kw,code", BAD)
def test_bad_configurations_are_refused(ops, kw, code):
    for op in ops:
        assert call(op, make(**kw)) == code, (op, kw)


@pytest.mark.parametrize("op", OPS)
def test_bad_pointers_and_workspaces_are_refused(op):
    assert call(op, None) == 1
    used = {crisp.CACHE_WINDOW: ["q", "k", "v", "out"], crisp.CACHE_SCORED: ["q", "k", "v", "out"],
            crisp.CACHE_PREFIX: ["q", "kp", "vp", "k", "v", "out"], crisp.CACHE_EVICT: ["k", "v", "kn", "vn"]}[op]
    for name in used:
        assert call(op, make(), **{name: 0}) == 1, name
        assert call(op, make(), **{name: P + 8}) == 4, name
    words = {crisp.CACHE_SCORED: ["score"], crisp.CACHE_EVICT: ["score", "sn", "kept", "new_len"]}.get(op, [])
    for name in words:
        assert call(op, make(), **{name: 0}) == 1, name
    for name in words + ["kv_len"]:
        assert call(op, make(), **{name: P + 2}) == 4, name
    c = make()
    c.workspace = None
    assert call(op, c) == 5
    c = make()
    c.workspace = (1 << 30) + 128
    assert call(op, c) == 4
    c = make()
    need = ctypes.c_size_t(0)
    assert crisp.lib().crisp_cache_workspace_size(ctypes.byref(c), op, ctypes.byref(need)) == 0
    c.workspace_bytes = need.value - 1
    assert call(op, c) == 5


@pytest.mark.parametrize("op", OPS)
def test_bad_strides_are_refused(op):
    used = {crisp.CACHE_WINDOW: ["k", "v"], crisp.CACHE_SCORED: ["k", "v"], crisp.CACHE_PREFIX: ["k", "k_prefix"],
            crisp.CACHE_EVICT: ["k", "v", "k_new", "v_new"]}[op]
    for name in used:
        for st, code in (((1 << 20, 1 << 17, 0), 2), ((1 << 20, 1 << 17, -128), 2), ((1 << 20, 1 << 17, 64), 2),
                         ((1 << 20, 1 << 17, 132), 4), ((1 << 20, 0, 128), 2), ((1 << 20, 1 << 37, 128), 2)):
            c = make()
            setattr(c, name, crisp._Strides(*st))
            assert call(op, c) == code, (name, st)


def test_an_evicted_cache_must_not_overlap_the_old_one():
    size = 2 * 8 * 1000 * 128 * 2
    new = 2 * 8 * 64 * 128 * 2
    ev = crisp.CACHE_EVICT
    far = dict(k=1 << 32, v=1 << 33)
    assert call(ev, make(), **far, kn=(1 << 32) + size - 16) == 1
    assert call(ev, make(), **far, kn=(1 << 32) - new + 16) == 1
    assert call(ev, make(), **far, vn=(1 << 33) + 16) == 1
    assert call(ev, make(), **far, kn=1 << 33) == 1
    assert call(ev, make(), **far, score=9 * P + 4) == 1
    assert call(ev, make(), **far, new_len=5 * P) == 1


def test_device_status_arguments():
    st = ctypes.c_int32(0)
    c = make()
    L = crisp.lib()
    assert L.crisp_cache_device_status(None, None, ctypes.byref(st)) == 1
    assert L.crisp_cache_device_status(ctypes.byref(c), None, None) == 1
    c.workspace = None
    assert L.crisp_cache_device_status(ctypes.byref(c), None, ctypes.byref(st)) == 5


def test_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    cfg = crisp.CacheConfig(batch=1, n_q=1, n_k=16, h_q=2, h_kv=1)
    q, k = torch.zeros(1, 2, 1, 128, dtype=torch.bfloat16), torch.zeros(1, 1, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        crisp.window_attention(q, k, k, torch.zeros_like(q), cfg)

    class Fake:          # a tensor's face on a device that is not there
        def __init__(self, t, device="cuda:0"):
            self.t, self.device = t, torch.device(device)

        def get_device(self):
            return self.device.index

        def __getattr__(self, name):
            return getattr(self.t, name)

    f = Fake
    with pytest.raises(ValueError, match="k: expected"):
        crisp.window_attention(f(q), f(k.float()), f(k), f(q), cfg)
    with pytest.raises(ValueError, match="v: expected"):
        crisp.window_attention(f(q), f(k), f(k[:, :, :15]), f(q), cfg)
    with pytest.raises(ValueError, match="out: expected"):
        crisp.window_attention(f(q), f(k), f(k), f(q, "cuda:1"), cfg)
    with pytest.raises(ValueError, match="kv_len: expected"):
        crisp.window_attention(f(q), f(k), f(k), f(q), cfg, kv_len=f(torch.zeros(1)))
    with pytest.raises(ValueError, match="score: expected"):
        crisp.scored_attention(f(q), f(k), f(k), f(q), f(torch.zeros(1, 1, 32)[:, :, ::2]), cfg)
    cfg.workspace = f(torch.zeros(256, dtype=torch.uint8), "cuda:1")
    with pytest.raises(ValueError, match="workspace is on"):
        crisp.window_attention(f(q), f(k), f(k), f(q), cfg)
    with pytest.raises(ValueError, match="broadcast"):
        cfg._c(k=torch.zeros(1, 1, 1, 128).expand(1, 1, 16, 128))
    with pytest.raises(ValueError, match="contiguous"):
        cfg._c(k=torch.zeros(1, 1, 128, 16).transpose(2, 3))
