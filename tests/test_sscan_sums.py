"""The selective scan's sums over channels, dB and dC (GPU): an fp32 sum rounded to bf16 once, against 64 bits.

Tolerances. A correct rounding to bf16's 8 significant bits is off by at most 2^-8 of the value, so by at most 2^-8 / sqrt(3) rms
where the errors fill that range evenly. What precedes it is fp32: the recurrences' own errors are allowed 1e-4 of the values, far
above what they have, and far below the 2^-11 of operands held in 11 bits.
* The signed error, summed with the values' signs, averages out over the roundings: six standard deviations and 2^-16 are allowed.
* The whole error is at most sqrt(1 + 0.1^2) of the rounding's alone, as long as all else is under a tenth of it.
* A value is rounded to the other side only when it lies within its error of a tie: for an error of 1e-5 of the value that is
  2e-5 of a range of 2^-8 or more, 0.5%; 1% is allowed for values near 0, whose terms cancel.
* Where the channels cancel to 2^-7 of their terms, 2^-20 of a term is 2^-13 of the result: bf16's rounding with a tenth more."""
import numpy as np
import pytest
import torch

from _util import f64, rel_l2
from oracle import block

pytestmark = pytest.mark.gpu


def bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


def gradients(T, D, N, G, z, opposed=False):
    """dB and dC of the library and of the definition. ``opposed``: neighbouring channels are alike but for dy, whose second is
    minus the first one's next bf16 value."""
    import chunked_gated_delta_05_gb300 as m
    g = torch.Generator().manual_seed(D + N)

    def rn(*shape, dtype=torch.bfloat16, std=1.0):
        t = torch.randn(*shape, generator=g) * std
        return t.to(dtype).cuda()

    def chan(t, dim):
        return t.index_select(dim, torch.arange(D, device="cuda") // 2 * 2) if opposed else t

    u, delta, dy = chan(rn(1, T, D), 2), chan(rn(1, T, D, std=0.5), 2), chan(rn(1, T, D), 2)
    if opposed:
        bits = dy.view(torch.int16)
        bits[..., 1::2] = (bits[..., 1::2] + 1) ^ -32768
    A, bias = chan(-torch.exp(rn(D, N, dtype=torch.float32, std=0.5)) * 4, 0), chan(rn(D, dtype=torch.float32, std=0.5) - 3, 0)
    Bm, Cm, zt = rn(1, T, G, N), rn(1, T, G, N), chan(rn(1, T, D), 2) if z else None
    out = m.selective_scan_bwd(u, delta, A, Bm, Cm, dy, z=zt, delta_bias=bias)
    want = block.scan_bwd(f64(u)[0], f64(delta)[0], f64(A), f64(Bm)[0], f64(Cm)[0], f64(dy)[0], z=None if zt is None else f64(zt)[0], delta_bias=f64(bias))
    return [(name, f64(x)[0], want[name]) for name, x in (("dB", out[3]), ("dC", out[4]))]


@pytest.mark.parametrize("T,D,N,G,z", [(1024, 256, 16, 1, True), (1030, 129, 13, 1, False), (1024, 192, 8, 2, True), (2048, 64, 4, 1, True)])
def test_sums_are_an_fp32_sum_rounded_once(T, D, N, G, z):
    for name, x, ref in gradients(T, D, N, G, z):
        assert np.isfinite(x).all()
        bias = ((x - ref) * np.sign(ref)).sum() / np.abs(ref).sum()
        spread = 2.0 ** -8 / np.sqrt(3) * np.sqrt((ref * ref).sum()) / np.abs(ref).sum()
        assert abs(bias) <= 6 * spread + 2.0 ** -16, f"{name}: shifted by {bias:.2e}"
        once = bf16(ref)
        assert rel_l2(x, ref) <= np.sqrt(1.01) * rel_l2(once, ref), name
        assert (x != once).mean() <= 0.01, f"{name}: {(x != once).mean():.2%} rounded to the other side"


@pytest.mark.parametrize("N", [16, 8])
def test_channels_that_cancel(N):
    for name, x, ref in gradients(256, 128, N, 1, True, opposed=True):
        assert np.isfinite(x).all()
        assert rel_l2(x, ref) <= 1.1 * 2.0 ** -8 / np.sqrt(3), name


def test_nan_reaches_only_the_sums_that_hold_it():
    """A NaN input makes the states after it NaN, and with them dC there; dB is a sum over what comes back from later tokens."""
    import chunked_gated_delta_05_gb300 as m
    g = torch.Generator().manual_seed(1)
    T, D, N, at = 300, 80, 16, 150
    u, delta, dy, Bm, Cm = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda() for s in ((1, T, D), (1, T, D), (1, T, D), (1, T, 1, N), (1, T, 1, N)))
    A = -torch.exp(torch.randn(D, N, generator=g)).cuda()
    clean = m.selective_scan_bwd(u, delta, A, Bm, Cm, dy)
    u[0, at, 7] = float("nan")
    out = m.selective_scan_bwd(u, delta, A, Bm, Cm, dy)
    others = [t for t in range(T) if t != at]
    assert torch.equal(out[3][0, others], clean[3][0, others]) and out[3][0, at].isnan().all()
    assert torch.equal(out[4][0, :at], clean[4][0, :at]) and out[4][0, at:].isnan().all()
