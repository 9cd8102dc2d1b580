"""Angles of the rotation over the whole range of positions and frequencies.  Where a sine or cosine is near 0, bf16
shows the angle's error far below its own rounding of values near 1."""
import numpy as np
import pytest
import torch

import io_aware_exact_tcgen05_gb300 as fa
from oracle import scored as so
from tests.parity import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
FREQS = [2.0 ** 24 - 1, -(2.0 ** 24 - 1), 7654321.0, -3.3e6, 1.0e5, 12345.678, 1.0e3, 100.0, 63.7, 8.0, 7.5, 1.0, 0.3, 1e-3,
         2.0 ** -30, 3e-38]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("back", [False, True])
def test_angles_over_the_whole_range(interleaved, back):
    S, d, rot = 4096, 64, 2 * len(FREQS)
    rng = np.random.RandomState(1)
    pos = rng.randint(-2 ** 31, 2 ** 31, S, dtype=np.int64)
    pos[:4] = 2 ** 31 - 1, -2 ** 31, 0, -1
    f = np.array(FREQS, np.float32)
    ang = so.angles(pos[None, None], f, None)[0, :, 0]
    one = torch.zeros(1, S, 1, d, dtype=torch.bfloat16, device=DEV)
    one[..., 0:rot:2 if interleaved else 1][..., :rot // 2] = 1.0  # the first of each pair
    how = dict(positions=torch.tensor(pos[None], dtype=torch.int32, device=DEV), inv_freq=torch.tensor(f, device=DEV),
               interleaved=interleaved)
    if back:
        g = one.transpose(1, 2).contiguous()
        got = to_np(fa.fa_qk_norm_rope_bwd(None, None, g, g, **how)[0])[0, :, 0]
    else:
        got = to_np(fa.fa_qk_norm_rope(one, one, **how)[0])[0, 0]
    a, b = (got[:, 0:rot:2], got[:, 1:rot:2]) if interleaved else (got[:, :rot // 2], got[:, rot // 2:rot])
    for x, want in ((a, np.cos(ang)), (b, -np.sin(ang) if back else np.sin(ang))):
        # one rounding to bf16, half a step; 2^-19 for the angle and the sine
        over = np.abs(x - want) - (2.0 ** -8 * np.abs(want) + 2.0 ** -19)
        assert over.max() <= 0, (FREQS[int(over.max(0).argmax())], over.max())
