"""Scratch of matrices that are far smaller than a large tile does not jump with
their number, nor with a large matrix beside them."""

import pytest

KINDS = [1, 0]  # bf16, float32


def need(shapes, kind):
    from hash_table_cache_amd import training as T

    return T._polar_workspace_bytes(tuple(shapes), bytes([kind]) * len(shapes))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(70, 70), (128, 128), (129, 140), (192, 1000), (300, 300)])
def test_many_small(shape, kind):
    tiles = -(-shape[0] // 256) * -(-shape[1] // 256)
    for count in (64, 255, 256, 600):
        few = max(1, 200 // tiles)
        assert need([shape] * count, kind) <= 1.02 * count / few * need([shape] * few, kind), count


@pytest.mark.parametrize("kind", KINDS)
def test_beside_a_large_one(kind):
    small = [(70, 70)] * 100
    alone, large = need(small, kind), need([(4096, 4096)], kind)
    # groups follow each other in the same memory
    assert need(small + [(4096, 4096)], kind) <= max(alone, large)


@pytest.mark.parametrize("kind", KINDS)
def test_as_the_header_says(kind):
    element, square = (10, 4) if kind == 1 else (12, 8)

    def padded(rows, cols, tile):
        p, q = (-(-side // tile) * tile for side in sorted((rows, cols)))
        return element * p * q + square * p * p

    # sums of A's shared tiles, norms and diagonals come to less than 16 MiB
    for shape, tile in (((65, 65), 64), ((1000, 700), 128), ((4096, 4096), 256), ((70, 1 << 20), 128),
                        ((1, 1 << 24), 64), ((1 << 20, 16), 64), ((1 << 15, 1 << 17), 256)):
        assert need([shape], kind) <= padded(*shape, tile) + (16 << 20), shape
    for shape in ((1, 1 << 16), (64, 1 << 16), (1 << 16, 33), (10, 257)):
        assert need([shape], kind) <= 340 * max(shape) + (1 << 17), shape
    assert need([(4096, 4096)] * 300, kind) <= 4 << 30
