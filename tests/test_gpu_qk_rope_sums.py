"""The sums over tokens and heads of the head norm's gradient."""
import numpy as np
import pytest
import torch

from tests import _attn as A
from tests import _ffn as H

pytestmark = pytest.mark.gpu

import fp4_spectral_split_amd as M


# tokens, query heads, key heads, head size, turned elements; the most heads that a workgroup adds up
SHAPES = [((6000, 4, 0, 64, 0), 128), ((3000, 4, 4, 64, 4), 48), ((900, 9, 3, 128, 64), 58), ((500, 5, 2, 512, 6), 16), ((1, 1, 1, 64, 8), 1)]


@pytest.mark.parametrize("shape,heads", SHAPES)
def test_weight_gradients_are_joined_without_loss(shape, heads):
    """Heads of ones have xh = 1 exactly (eps = 0), and an angle of zero leaves dy, so
    dw is the sum of dy over tokens and heads. With integers below 2^18 a workgroup
    of up to 64 heads has a sum below 2^24, exact in fp32, and what is left is the
    rounding of the whole: dw is within half a step of the exact sum. A workgroup of
    128 heads has one below 2^25, where fp32 holds the even integers: off by 1 for
    each of the 512 workgroups."""
    T, hq, hk, D, rot = shape
    g = H.rng(251)
    rope = torch.cat([torch.ones(1, rot // 2), torch.zeros(1, rot // 2)], 1).cuda() if rot else None
    pos = torch.zeros(T, dtype=torch.int32, device="cuda") if rot else None
    dy = [g.integers(1 << 16, 1 << 18, (T, h, D)) for h in (hq, hk)]
    x = [torch.ones(T, h * D, device="cuda") for h in (hq, hk)]
    w = torch.ones(D, device="cuda")
    d = [A.dev(a.reshape(T, -1).astype(np.float32)) for a in dy]
    print("case sums", shape, flush=True)
    out = M.metis_qk_norm_rope_bwd(d[0], d[1] if hk else None, x[0], x[1] if hk else None, pos, rope, D, w, w if hk else None, eps=0.0)
    torch.cuda.synchronize()
    for got, a, there in ((out[2], dy[0], True), (out[3], dy[1], hk > 0)):
        if there:
            want = a.sum((0, 1))
            off = np.abs(H.np64(got) - want) - np.spacing(want.astype(np.float32)) / 2
            assert off.max() <= (512 if heads > 64 else 0), off.max()
