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


@TYPES
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("cap", [30.0, 50.0, 57.0, 60.0, 62.0, 66.0, 70.0, 100.0])
def test_small_values_beside_a_saturated_cap(H, cap, sign, out_dtype):  # noqa: F811
    """All of a row's scores saturate at -cap (or +cap), so all weights are equal: values of 2^-40 to 2^0 in turn along
    the dims keep their precision.

    out is a mean: weights, equal but for 2^-20 cap + 2^-22 (score and exponential, relative), and sums of n
    terms of 2^-23 each; a bf16 result as in check_rows."""
    g = torch.Generator(device="cuda").manual_seed(72)
    n, d = 300, 128
    q, k = S.rand(g, n, 1, d).abs() + 1, torch.full((n, 1, d), sign * 500.0, device="cuda").bfloat16()
    v = (torch.rand(n, 1, d, generator=g, device="cuda") + 1) * 2.0 ** -(torch.arange(d, device="cuda") % 41).float()
    v = (v * torch.where(torch.rand(n, 1, d, generator=g, device="cuda") < 0.3, -1.0, 1.0)).bfloat16()
    out, lse, _, _, vh = attend(H, q, k, v, S.Opts(cap=cap), out_dtype)
    count = np.arange(1, n + 1)[:, None]
    want, mag = np.cumsum(vh[:, 0], 0) / count, np.cumsum(np.abs(vh[:, 0]), 0) / count
    E = 2.0 ** -20 * cap + 2.0 ** -23 * (n + 16) + 2.0 ** -22
    wl = sign * cap + np.log(count[:, 0])
    S.check_rows(out[:, 0], lse[:, 0], (want, wl, 2 * E * mag, np.full(n, E + 2.0 ** -22 * (1 + 3 * cap)), mag), f"cap {cap}")
    if out_dtype == torch.float32:  # the weights' common error cancels in the mean
        off = np.abs(out[:, 0].double().cpu().numpy() - want) / mag
        assert off.max() <= 2.0 ** -23 * (n + 16), off.max()


@TYPES
@pytest.mark.parametrize("cap", [57.0, 60.0, 62.0, 66.0, 70.0, 200.0])
def test_weights_over_the_whole_range_of_larger_caps(H, cap, out_dtype):  # noqa: F811
    """Scores from -cap to +cap in either order, with values up to 2^19."""
    g = torch.Generator(device="cuda").manual_seed(73)
    n, d = 400, 128
    q, v = S.rand(g, n, 1, d).abs() + 1, (torch.rand(n, 1, d, generator=g, device="cuda") * 2.0 ** 19).bfloat16()
    k = torch.full((n, 1, d), 500.0, device="cuda").bfloat16()
    k[:200] = -500.0
    for keys in (k, k.flip(0)):
        out, lse, qh, kh, vh = attend(H, q, keys, v, S.Opts(cap=cap), out_dtype)
        want, wl, _, _, mag = SO.attention(qh[:, 0], kh[:, 0], vh[:, 0], cap=cap)
        E = 2.0 ** -20 * cap + 2.0 ** -23 * (n + 16) + 2.0 ** -19
        S.check_rows(out[:, 0], lse[:, 0], (want, wl, 2 * E * mag, np.full(n, E + 2.0 ** -22 * (1 + 3 * cap)), mag), f"cap {cap}")


@TYPES
@pytest.mark.parametrize("slope", [0.0, 0.01])
def test_large_values_under_a_bias(H, slope, out_dtype):  # noqa: F811
    """Values up to 2^56 (what slopes without a cap allow); the last keys give the reference, and all others weigh almost
    2^40 times as much, which does not move it."""
    g = torch.Generator(device="cuda").manual_seed(74)
    n, Hq, d = 700, 2, 64
    q, k = torch.zeros(n, Hq, d, device="cuda"), torch.zeros(n, 1, d, device="cuda")
    q[..., 0] = 1.0
    k[:300, 0, 0] = 27.5
    v = (torch.rand(n, 1, d, generator=g, device="cuda") * 2.0 ** 56).bfloat16()
    out, lse, qh, kh, vh = attend(H, q.bfloat16(), k.bfloat16(), v, S.Opts(scale=1.0, slopes=[slope, -slope / 4]), out_dtype)
    for h, s in enumerate([slope, -slope / 4]):
        ref = SO.attention(qh[:, h], kh[:, 0], vh[:, 0], scale=1.0, slope=float(np.float32(s)))
        S.check_rows(out[:, h], lse[:, h], ref, f"head {h}")


# relative error of the tanh's polynomials (csrc/hashattn_api.cu) up to half the cap, and up to the cap
FITS = {torch.bfloat16: (5.4e-7, 5.9e-7), torch.float32: (1.3e-8, 5.0e-8)}


@TYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("upto", [0.5, 1.0, 4.0])
@pytest.mark.parametrize("bias", [False, True], ids=["cap", "cap-bias"])
@pytest.mark.parametrize("whole", [True, False], ids=["tile", "part"])
def test_the_cap_itself(H, whole, bias, upto, d, out_dtype):  # noqa: F811
    """All keys of a row score x, a number of bf16: lse - log(keys) is the capped x, read off to the polynomial's own error
    (that of bf16 weights would not do for float32 results). One tile of keys or less; slopes of 0 take the biased kernel.

    Relative to the score: the fit; its roundings, 2.5 of 2^-24 up to half the cap (the first coefficient, the last sum
    and a twelfth of what comes before) and 4.5 up to the cap (the ratio to the cap and the product with it, a
    quarter of what comes before); 2.5 of lse (the sum with the logarithm, log 2 and the product with it). Absolute: the exponential
    2^-22, the sum of the weights 2^-24 an addition (13 in a row for float32 results, 70 else), the logarithm 2^-21.
    Beyond the cap 2^-22 cap."""
    g = torch.Generator(device="cuda").manual_seed(75)
    n, Hq, cap, keys = 60, 4, 50.0, (64 if out_dtype == torch.float32 else 128) - (0 if whole else 9)
    x = ((torch.rand(n, Hq, generator=g, device="cuda") * 0.4 + 0.6) * upto * cap).bfloat16()
    x[::2] *= -1
    K, V, table = S.pages(g, [1] * n, [keys] * n, 128, 1, d, "token", S.Opts())
    q = torch.zeros(n, Hq, d, dtype=torch.bfloat16, device="cuda")
    q[..., 3] = x
    K.zero_()
    K[..., 3] = 1.0
    _, lse = S.chunk(H, q, K, V, table, [1] * n, [keys] * n, 1, S.Opts(cap=cap, scale=1.0, slopes=[0.0] * Hq if bias else None), out_dtype)
    z = x.double().cpu().numpy()
    want = cap * np.tanh(z / cap)
    got = lse.double().cpu().numpy() - np.log(keys)
    adds = 13 if out_dtype == torch.float32 else 70
    tol = np.abs(want) * (FITS[out_dtype][upto > 0.5] + (5 if upto == 0.5 else 7) * 2.0 ** -24) + 2.0 ** -22 + adds * 2.0 ** -24 + 2.0 ** -21
    if upto > 1:
        tol = tol + 2.0 ** -22 * cap
    off = np.abs(got - want) / tol
    assert off.max() <= 1, off.max()
