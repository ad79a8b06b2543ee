"""Values the serving calls have to keep: weights next to the largest number."""
import numpy as np
import pytest
import torch

import hybrid_attention_ssm_hymba_b200 as H
from gpu_util import requires_cuda
from serve_util import DTYPE, TINY, TORCH

pytestmark = [pytest.mark.gpu, requires_cuda]


# --------------------------------------------------------------------------- 4-bit weights

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 128])
def test_quantise_w4_of_the_largest_weights(dtype, group):
    """Groups whose largest weight is next to the type's largest number, and on both sides of a
    seventh of it, where 7 w leaves fp32's range."""
    top = torch.finfo(TORCH[dtype]).max
    r = np.random.default_rng(group)
    most = np.array([top, top / 2, top / 6.9, top / 7.0, top / 7.1, 1e37, 1e36])
    w = r.uniform(-1, 1, (len(most), 2 * group)) * most[:, None]
    w[:, 3] = most * np.where(np.arange(len(most)) % 2, -1, 1)
    w[:, group + 5] = most
    t = torch.from_numpy(w).clamp(-top, top).to(TORCH[dtype]).cuda()
    assert torch.isfinite(t).all()
    n, k = t.shape
    q4 = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    sc = torch.empty(n, k // group, device="cuda")
    H.check(H.hymba_quantize_w4(t, q4, sc, n, k, group, DTYPE[dtype]), "quantize")
    x = t.double().cpu().numpy().reshape(n, -1, group)
    amax = np.abs(x).max(-1)
    q = np.rint(7 * x / amax[..., None]).reshape(n, k)
    scale = np.maximum(amax.astype(np.float32) / np.float32(7), TINY)
    got = q4.cpu().numpy()
    assert np.array_equal((got & 15) - 8.0, q[:, 0::2]) and np.array_equal((got >> 4) - 8.0, q[:, 1::2])
    assert np.array_equal(sc.cpu().numpy(), scale)
