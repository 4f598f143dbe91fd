"""A token's attention over a paged cache against its fp64 definition (GPU). Tolerance: weights rounded once to bf16 (half a step, 2^-8
relative), the output once more, scores fp32 sums of D terms (``D 2^-22`` of their magnitudes' sum, twice for the sum of weights)."""
import numpy as np
import pytest
import torch

from _util import f64
from oracle import attention as A

pytestmark = pytest.mark.gpu
I32 = torch.int32


def lib():
    import chunked_gated_delta_05_gb300 as m
    return m


def case(lengths, H, Hk, D, page, width=None, seed=0, std=1.0, extra=3):
    g = torch.Generator().manual_seed(seed + 31 * len(lengths) + page)
    need = [-(-max(n, 0) // page) for n in lengths]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=g).to(I32)
    table = torch.full((len(lengths), width or max(1, max(need))), -7, dtype=I32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at: at + n]
        at += n
    rn = lambda *s: (torch.randn(*s, generator=g) * std).to(torch.bfloat16)  # noqa: E731
    q, kc, vc = rn(len(lengths), H, D), rn(pages, page, Hk, D), rn(pages, page, Hk, D)
    return q, kc, vc, table, torch.tensor(lengths, dtype=I32)


def check(q, kc, vc, table, lengths, scale=None, out=None):
    status = torch.zeros(1, dtype=I32, device="cuda")
    o = lib().attention_step(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lengths.cuda(), scale=scale, status=status) if out is None else out
    assert int(status.item()) == 0
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    Q, K, V, n = f64(q), f64(kc), f64(vc), lengths.tolist()
    want = A.attention_step(Q, K, V, table.numpy(), n, scale)
    size = A.attention_step(Q, K, np.abs(V), table.numpy(), n, scale)
    ds = D * 2.0 ** -22 * scale * np.abs(Q).sum(-1).max() * np.abs(K[np.isfinite(K)]).max() + 2.0 ** -20
    over = np.abs(f64(o) - want) - (2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * ds) * size)
    assert np.isfinite(f64(o)).all() and over.max() <= 0, f"off by {over.max():.3e} more than allowed"
    return o


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 7, 16, 64, 100])
def test_lengths_and_pages(page, D):
    check(*case([1, 2, 15, 16, 17, 63, 64, 65, 100, 0, 129, -3, 300], 4, 2, D, page))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 1), (7, 1), (8, 8), (9, 1), (16, 1), (24, 2), (17, 1), (40, 1), (32, 2)])
def test_heads(H, Hk, D):
    check(*case([70, 0, 300], H, Hk, D, 16))


@pytest.mark.parametrize("B,n", [(1, 1), (1, 5000), (1, 40000), (3, 9000), (200, 600)])
def test_batches(B, n):
    g = np.random.default_rng(B)
    check(*case([n] + [int(x) for x in g.integers(0, n + 1, B - 1)], 4, 2, 128, 64))


def test_one_page_a_sequence():
    """A cache of one slot a sequence."""
    check(*case([33, 100, 7], 4, 4, 128, 100))


def test_peaked_scores():
    check(*case([1000, 37], 4, 2, 128, 16, std=3.0))


def test_strided_queries():
    q, kc, vc, table, lengths = case([50, 60, 70], 4, 2, 128, 16)
    wide = torch.zeros(3, 4 * 128 + 64, dtype=torch.bfloat16)
    wide[:, 32: 32 + 512] = q.view(3, 512)
    view = wide.cuda()[:, 32: 32 + 512].view(3, 4, 128)
    a = lib().attention_step(view, kc.cuda(), vc.cuda(), table.cuda(), lengths.cuda())
    assert torch.equal(a, check(q, kc, vc, table, lengths))


def test_what_lies_behind_a_sequence_is_not_read():
    """NaN in the rest of a page, in other pages and in the unused part of the table changes nothing."""
    q, kc, vc, table, lengths = case([5, 64, 90], 4, 2, 128, 64)
    a = check(q, kc, vc, table, lengths)
    for c in (kc, vc):
        keep = torch.full_like(c, float("nan"))
        for b, n in enumerate(lengths.tolist()):
            for t in range(n):
                keep[table[b, t // 64], t % 64] = c[table[b, t // 64], t % 64]
        c.copy_(keep)
    o = lib().attention_step(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lengths.cuda())
    assert torch.equal(a, o)


def test_bad_pages_and_lengths_are_reported():
    from chunked_gated_delta_05_gb300 import GDN_ERANGE
    q, kc, vc, table, lengths = case([40, 40, 40, 40], 4, 2, 128, 16)
    run = lambda table, lengths, st: lib().attention_step(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lengths.cuda(), status=st)  # noqa: E731
    st = torch.zeros(1, dtype=I32, device="cuda")
    good = run(table, lengths, st)
    assert int(st.item()) == 0
    for page in (-1, kc.shape[0]):
        bad, st = table.clone(), torch.zeros(1, dtype=I32, device="cuda")
        bad[1, 1] = page
        o = run(bad, lengths, st)
        assert int(st.item()) == GDN_ERANGE
        assert torch.equal(o[[0, 2, 3]], good[[0, 2, 3]])
        # the row's other keys remain
        K, V = (f64(c[table[1].long()[[0, 2]]]).reshape(-1, 2, 128)[:24] for c in (kc, vc))
        for h in range(4):
            P, _ = A.weights(f64(q)[1, h][None], K[:, h // 2], 128 ** -0.5, False)
            assert np.abs(f64(o)[1, h] - (P @ V[:, h // 2])[0]).max() <= 2.0 ** -7 * (P @ np.abs(V[:, h // 2])).max()
    long, st = lengths.clone(), torch.zeros(1, dtype=I32, device="cuda")
    long[2] = 16 * table.shape[1] + 1
    o = run(table, long, st)
    assert int(st.item()) == GDN_ERANGE and not o[2].any() and torch.equal(o[[0, 1, 3]], good[[0, 1, 3]])


def test_far_into_a_large_cache():
    """Pages whose elements lie past 2^31."""
    pages, page, Hk, D = 66000, 64, 4, 128
    kc = torch.empty(pages, page, Hk, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    q, k1, v1, _, lengths = case([150], 8, Hk, D, 64)
    table = torch.tensor([[65999, 1, 65535]], dtype=I32)
    for i, p in enumerate(table[0].tolist()):
        kc[p], vc[p] = k1[i].cuda(), v1[i].cuda()
    o = lib().attention_step(q.cuda(), kc, vc, table.cuda(), lengths.cuda())
    small = torch.tensor([[0, 1, 2]], dtype=I32)
    check(q, k1, v1, small, lengths, out=o)
