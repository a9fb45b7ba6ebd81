"""Scores with options at the ends of their ranges: caps, scales, weights and values."""
import numpy as np
import pytest
import torch

import test_gpu_score_opts as S
from oracle import serving_oracle as SO
from test_gpu_score_opts import H  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


def attend(H, q, k, v, opts, out_dtype):  # noqa: F811
    """One prompt: (out, lse) of the library, and its inputs in 64 bits."""
    out, lse = S.prefill(H, q, k, v, [q.shape[0]], opts, out_dtype)
    return out, lse, *(x.double().cpu().numpy() for x in (q, k, v))


@TYPES
@pytest.mark.parametrize("cap,scale", [(25, 37), (26, 38), (30, 42), (47, 59), (48, 60), (60, 60), (-44, -59), (-48, -60), (-60, -60)])
def test_large_and_small_caps_beside_their_scales(H, cap, scale, out_dtype):  # noqa: F811
    """Caps and scales of 2^cap and 2^scale, where the powers of their ratio leave float32's range: ordinary scores, and
    queries of zeros, whose scores are 0 (large caps); scores beyond a cap that weighs nothing (small ones)."""
    g = torch.Generator(device="cuda").manual_seed(71)
    n, Hq, d = 300, 2, 64
    cap, scale = 2.0 ** cap, 2.0 ** scale
    q, k, v = S.rand(g, n, Hq, d) / max(scale, cap), S.rand(g, n, 1, d), S.rand(g, n, 1, d)
    q[::7] = 0
    out, lse, qh, kh, vh = attend(H, q, k, v, S.Opts(cap=cap, scale=scale), out_dtype)
    for h in range(Hq):
        want, wl, tol, tol_lse, mag = SO.attention(qh[:, h], kh[:, 0], vh[:, 0], cap=cap, scale=scale)
        if cap > 1:  # scores far below the cap: they take no share of its error, but 2^-20 of their own size
            plain = SO.attention(qh[:, h], kh[:, 0], vh[:, 0], scale=scale)
            z = (np.abs(qh[:, h]) @ np.abs(kh[:, 0]).T).max(1) * scale
            tol, tol_lse = plain[2] + 2.0 ** -19 * z[:, None] * plain[4], plain[3] + 2.0 ** -20 * z
        S.check_rows(out[:, h], lse[:, h], (want, wl, tol, tol_lse, mag), f"head {h}")
