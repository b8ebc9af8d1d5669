"""Host side of the calls around the recall: what a context's workspace keeps for them."""
import ctypes

import pytest

import serve_ref as ref
from paged_kv_cache_meank_gb300 import _abi, config_for
from test_serve_host import lib   # noqa: F401


@pytest.mark.parametrize("act,kv", [("f32", "f32"), ("f32", "bf16"), ("f32", "e4m3"), ("bf16", "f32"),
                                    ("bf16", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_scratch_goes_by_types_and_width(lib, act, kv, d):
    """Two parts a CTA, d + 2 float32 a row: of 16 rows for up to 608 CTAs where attention
    runs in float32, of 256 for up to 160 where it runs on the tensor cores."""
    wl = ref.workload(L=1, G=1, H=1, d=d, kv=kv, act=act, n_blocks=1)
    got = lib.kvm_workspace_bytes(ctypes.byref(config_for(wl, max_positions=32)))
    small = 608 * 2 * 16 * (d + 2) * 4
    large = 160 * 2 * 256 * (d + 2) * 4
    want = large if act == "bf16" and kv != "f32" else small
    # what else a context of one block keeps is the same for all of them, below 3 MB
    assert want <= got < want + 3_000_000, got
