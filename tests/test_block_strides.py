"""Row strides of strided inputs (CPU): what is accepted lies where the kernels read it, all else is refused."""
import itertools

import pytest
import torch

from chunked_gated_delta_05_gb300.block_ops import _rows_of

BF16 = torch.bfloat16


def rows_of(t, inner):
    width = 1
    for n in t.shape[t.dim() - inner:]:
        width *= n
    return _rows_of("x", t, BF16, t.shape, -1, inner, width)


@pytest.mark.parametrize("t,inner", [
    (torch.zeros(1, 16, dtype=BF16).expand(5, 16), 1),                      # one row for a whole batch
    (torch.zeros(1, 2, 8, dtype=BF16).expand(5, 2, 8), 2),
    (torch.zeros(1, 1, 1, 16, dtype=BF16).expand(1, 50, 1, 16), 2),         # one token's vector for a sequence
    (torch.zeros(3, 1, 1, 16, dtype=BF16).expand(3, 50, 1, 16), 2),         # one for each of several sequences
    (torch.zeros(1, 1, 16, dtype=BF16).expand(1, 50, 16), 1),
    (torch.zeros(3, 1, 16, dtype=BF16).expand(3, 50, 16), 1),
    (torch.zeros(1, 50, 16, dtype=BF16).expand(3, 50, 16), 1),              # one sequence for all
    (torch.zeros(1, 50, 1, 16, dtype=BF16).expand(3, 50, 1, 16), 2),
    (torch.zeros(40, dtype=BF16).as_strided((4, 16), (8, 1)), 1),           # rows that overlap
    (torch.zeros(1, dtype=BF16).expand(5, 1), 1),                           # rows of one element
])
def test_rows_in_the_same_place_are_refused(t, inner):
    with pytest.raises(ValueError):
        rows_of(t, inner)


@pytest.mark.parametrize("t,inner,row", [
    (torch.zeros(1, 16, dtype=BF16).expand(1, 16), 1, 16),
    (torch.zeros(5, 24, dtype=BF16)[:, 8:], 1, 24),
    (torch.zeros(1, 24, dtype=BF16)[:, 8:], 1, 16),
    (torch.zeros(3, 1, 24, dtype=BF16)[..., 8:], 1, 24),
    (torch.zeros(1, 7, 24, dtype=BF16)[..., 8:], 1, 24),
    (torch.zeros(3, 7, 24, dtype=BF16)[..., 8:], 1, 24),
    (torch.zeros(3, 7, 24, dtype=BF16)[..., 8:].view(3, 7, 2, 8), 2, 24),
    (torch.zeros(3, 7, 24, dtype=BF16)[:, ::2, 8:], 1, None),               # sequences do not follow each other at 4 of these rows
    (torch.zeros(3, 8, 24, dtype=BF16)[:, ::2, 8:], 1, 48),
])
def test_slices(t, inner, row):
    if row is None:
        with pytest.raises(ValueError):
            rows_of(t, inner)
    else:
        assert rows_of(t, inner) == row


def test_every_small_layout():
    """Of all small shapes and strides: a stride is given only where row i starts i strides on and no two rows share an element."""
    store = torch.zeros(4096, dtype=BF16)
    accepted = 0
    for lead in (1, 2):
        for inner in (1, 2):
            for shape in itertools.product((1, 2, 3), repeat=lead + inner):
                for strides in itertools.product((0, 1, 2, 3, 6, 9), repeat=lead + inner):
                    t = store.as_strided(shape, strides)
                    try:
                        row = rows_of(t, inner)
                    except ValueError:
                        continue
                    accepted += 1
                    width, seen = 1, set()
                    for n in shape[lead:]:
                        width *= n
                    for i, at in enumerate(itertools.product(*map(range, shape))):
                        place = sum(a * s for a, s in zip(at, strides))
                        assert place == i // width * row + i % width, (shape, strides)
                        seen.add(place)
                    assert len(seen) == t.numel(), (shape, strides)
    assert accepted > 500
