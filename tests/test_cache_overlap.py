"""Eviction refuses outputs that overlap an input or one another (host checks
on stand-in addresses; nothing is launched)."""
import pytest

import long_context_prefill_last_b200 as crisp
from test_cache_host import built, call, make  # noqa: F401

G = 1 << 32      # every array far from every other
AT = dict(k=G, v=2 * G, score=3 * G, kv_len=4 * G, kn=5 * G, vn=6 * G, sn=7 * G, kept=8 * G, new_len=9 * G)
WORDS = dict(score=2 * 8 * 1000 * 4, kv_len=2 * 4, sn=2 * 8 * 64 * 4, kept=2 * 8 * 64 * 4, new_len=2 * 4)
SIZE = dict(k=2 * 8 * 1000 * 256, v=2 * 8 * 1000 * 256, kn=2 * 8 * 64 * 256, vn=2 * 8 * 64 * 256, **WORDS)
INPUTS, OUTPUTS = ("k", "v", "score", "kv_len"), ("kn", "vn", "sn", "kept", "new_len")
PAIRS = ([(o, x) for o in OUTPUTS for x in INPUTS] + [(o, x) for o in OUTPUTS[2:] for x in OUTPUTS if o != x])


@pytest.mark.parametrize("out,other", PAIRS)
def test_overlap_is_refused(out, other):
    step = 4 if out in WORDS else 16
    for at in (AT[other], AT[other] + SIZE[other] - step, AT[other] - SIZE[out] + step):
        if at % step == 0:
            assert call(crisp.CACHE_EVICT, make(), **{**AT, out: at}) == 1, (out, other, at - AT[other])


def test_one_buffer_for_keys_and_values_is_refused():
    assert call(crisp.CACHE_EVICT, make(), **{**AT, "vn": AT["kn"]}) == 1
