"""Single-token steps of batches that are larger than the grid: a block walks several rows in turn (GPU).

The scan step of 4096 channels covers a row by 64 blocks of 912 resident ones, so 14 blocks share the rows: two, or three and two, or
nine and eight each. The convolution step of 6144 channels has 12 blocks a row of 1216: 101 share 250 rows. Padding rows and indices
outside the pool fall on first, middle and last turns of a walk. Tolerances as in the steps' other tests: a bf16 rounding (2^-8) of
values within 1e-5 of the largest; states within 1e-5 rel-L2, the convolution's equal."""
import numpy as np
import pytest
import torch

from _util import f64, rel_l2
from oracle import block

pytestmark = pytest.mark.gpu


def lib():
    import chunked_gated_delta_05_gb300 as m
    return m


def generator(seed):
    g = torch.Generator().manual_seed(seed)
    return g, lambda *s, dtype=torch.bfloat16, std=1.0: (torch.randn(*s, generator=g) * std).to(dtype).cuda()


def indices(B, slots, g, turns):
    """Each row's slot, none twice. Rows are padding or outside the pool at every turn of a block's walk (``turns`` rows apart)."""
    idx = torch.randperm(slots, generator=g)[:B].to(torch.int32)
    for turn in range((B + turns - 1) // turns):
        at = [turn * turns + i for i in range(turns) if turn * turns + i < B]
        if at:
            idx[at[turn % len(at)]] = -1
            idx[at[(turn + 3) % len(at)]] = slots + turn
    idx[-1] = -1 if B % 2 else idx[-1]
    return idx.cuda()


def close_bf16(x, ref):
    x = f64(x)
    assert np.isfinite(x).all()
    bad = np.abs(x - ref) - (2.0 ** -8 * np.abs(ref) + 1e-5 * np.abs(ref).max())
    assert bad.max() <= 0, f"off by {bad.max():.3e} more than allowed"


def check_pool(call, state, idx, step):
    """``call(state, idx, status)`` against ``step(states of the live rows, live rows) -> (outputs, new states)``."""
    slots = state.shape[0]
    before, status = state.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    y = call(state, idx, status)
    rows = None if idx is None else idx.cpu().numpy()
    B = y.shape[0]
    live = list(range(B)) if rows is None else [b for b in range(B) if 0 <= rows[b] < slots]
    places = live if rows is None else [int(rows[b]) for b in live]
    want, states = step(f64(before[places]), live)
    close_bf16(y[live], want)
    dead = [b for b in range(B) if b not in set(live)]
    assert (y[dead] == 0).all()
    others = sorted(set(range(slots)) - set(places))
    assert torch.equal(state[others], before[others])
    assert status.item() == (5 if rows is not None and (rows >= slots).any() else 0)
    return state[places], states


@pytest.mark.parametrize("B", [28, 31, 120])
@pytest.mark.parametrize("N,strided,indexed", [(16, False, True), (16, True, True), (13, False, True), (8, False, True), (8, True, False), (16, False, False)])
def test_scan_step_rows(B, N, strided, indexed):
    """N = 13, and B and C at odd places of wider rows, take the element path; the others the vector path."""
    D = 4096
    g, rn = generator(B * 100 + N)
    slots = B + 9 if indexed else B
    state, A = rn(slots, D, N, dtype=torch.float32), -torch.exp(rn(D, N, dtype=torch.float32))
    Ds, db = rn(D, dtype=torch.float32), rn(D, dtype=torch.float32) - 2

    def row(*shape):
        w = int(np.prod(shape))
        return rn(B, w + 7)[:, 7:].view(B, *shape) if strided else rn(B, *shape)

    u, delta, z, Bm, Cm = row(D), row(D), row(D), row(1, N), row(1, N)
    idx = indices(B, slots, g, 14) if indexed else None

    def step(states, live):
        y, final, _ = block.scan(*(f64(t)[live] if t.shape[0] == B and t is not A else f64(t) for t in (u, delta, A, Bm, Cm)), f64(Ds), f64(z)[live], f64(db), True,
                                 states, list(range(len(live) + 1)))
        return y, final

    got, want = check_pool(lambda s, i, st: lib().selective_scan_step(s, u, delta, A, Bm, Cm, D=Ds, z=z, delta_bias=db, state_indices=i, status=st), state, idx, step)
    assert rel_l2(f64(got), want) <= 1e-5


@pytest.mark.parametrize("B", [202, 250])
@pytest.mark.parametrize("dil,W,indexed", [(1, 4, True), (2, 4, True), (1, 4, False), (3, 3, True), (1, 1, True)])
def test_conv_step_rows(B, dil, W, indexed):
    C, HW = 6144, (W - 1) * dil
    g, rn = generator(B + dil)
    slots = B + 30 if indexed else B
    state, x, w, b = rn(slots, HW, C), rn(B, C + 8)[:, 8:], rn(C, W, dtype=torch.float32, std=0.5), rn(C, dtype=torch.float32)
    idx = indices(B, slots, g, 101) if indexed else None

    def step(states, live):
        return block.conv_step(states, f64(x)[live], f64(w), f64(b), dil)

    got, want = check_pool(lambda s, i, st: lib().causal_conv1d_step(s, x, w, b, dilation=dil, state_indices=i, status=st), state, idx, step)
    assert np.array_equal(f64(got), want)


def test_all_rows_padding():
    """A batch of padding rows only, many to a block, touches nothing."""
    _, rn = generator(3)
    B, D, N = 100, 4096, 16
    u, Bm, A, state = rn(B, D), rn(B, 1, N), -torch.exp(rn(D, N, dtype=torch.float32)), rn(4, D, N, dtype=torch.float32)
    before = state.clone()
    u.fill_(float("nan"))
    y = lib().selective_scan_step(state, u, u, A, Bm, Bm, state_indices=torch.full((B,), -1, dtype=torch.int32, device="cuda"))
    assert (y == 0).all() and torch.equal(state, before)
