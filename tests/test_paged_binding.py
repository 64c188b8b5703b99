"""Host-side parts of the paged cache's binding (CPU only)."""
import itertools

from precision_quantization_block_amd import pqb


def test_rows_that_meet_a_block():
    """Against the sets of bytes, for blocks before, inside, between and behind the rows."""
    for size, gap, count in itertools.product((1, 4, 7), (0, 1, 5, 30), (1, 2, 3, 5)):
        step, base = size + gap, 200
        rows = {base + t * step + i for t in range(count) for i in range(size)}
        for other in range(base - count * size - 3, base + count * step + 3):
            want = not rows.isdisjoint(range(other, other + count * size))
            assert pqb._rows_meet(base, step, size, count, other) == want, (size, gap, count, other)
