"""lora_cache_append and lora_attention where earlier tests do not reach: scores far
apart on tiles without hidden keys.  Against the float64 form."""
import numpy as np
import pytest
import torch

import attn_ref as R
from test_gpu_14_attention import Dev, check, dev, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import segmented_gather_rank_amd as lib
    return lib


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [0.0, 3000.0])
def test_large_scores_of_full_tiles(L, D, cache, cap):
    """Scores hundreds apart, most of each in the last dimensions, on a prompt and on
    decode tokens whose tiles of keys are seen by every row."""
    b = R.Batch([200, 1, 1], [900, 1500, 200], 2, 1, D, 16, cache, seed=D)
    if cache == "e4m3":
        b.k_scale = torch.ones(1)
    k, _ = b.views()
    k[..., D - 16:] = (k[..., D - 16:].float() * 8).to(k.dtype)
    b.q[..., D - 16:] *= 4
    o, lse, _, _ = run(L, b, scale=1.0, cap=cap)
    out, rl, out_tol, lse_tol = b.reference(scale=1.0, cap=cap)
    assert np.ptp(rl) > 100
    # weights that fp32 cannot hold are zeros: each is off by less than its smallest
    # normal number, times a value
    out_tol = out_tol + max(b.kv_len) * np.finfo(np.float32).tiny * float(b.v_store.float().abs().max())
    check(b, o, lse, (out, rl, out_tol, lse_tol))
