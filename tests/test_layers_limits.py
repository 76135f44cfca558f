"""What the layers' size queries and checks answer at and past the sizes where a limit begins (no GPU: every
call here is refused)."""
import os

import pytest

F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    pytest.importorskip("torch")
    from nearest_centroid_assignment_amd import layers

    return layers.lib()


@pytest.mark.parametrize("dtype,size", [(F32, 4), (BF16, 2)])
@pytest.mark.parametrize("width", [16, 64])
def test_pieces_of_dz(lib, dtype, size, width):
    """A piece's dz takes the larger of 512 MiB and 256 classes of all rows. Beside it lie dx's
    float32 sums between the pieces (rows x width) and the parts of products of few tiles, at
    most 1024 of 256 x 256 float32 (256 MiB)."""
    query = lib.layers_cross_entropy_backward_workspace_bytes
    for rows in (8192, 1 << 19, 1 << 20, (1 << 20) + 1, 1 << 21, 5000000):
        for classes in (256, 257, 1000, 2000):
            most = max(1 << 29, 256 * rows * size)
            assert 0 < query(rows, classes, width, dtype, 0) <= most + 4 * rows * width + (1 << 28) + 4096
    # Past 2^20 16-bit rows (2^19 of float32) a piece is 256 classes, and dz grows with the rows.
    for rows in (1 << 21, 1 << 22):
        assert query(rows, 2000, width, dtype, 0) >= 256 * rows * size
    # Between pieces only the rows count: more classes take no more.
    assert query(1 << 22, 65536, 16, BF16, 0) == query(1 << 22, 1024, 16, BF16, 0)


def test_most_rows(lib):
    """Rows past 2^28, whose sums are joined in several launches, up to a dispatch's tiles."""
    fwd, bwd = lib.layers_cross_entropy_workspace_bytes, lib.layers_cross_entropy_backward_workspace_bytes
    for rows in (2 ** 28, 2 ** 28 + 16, 2 ** 29 - 1024):
        assert fwd(rows, 64, 2, BF16, 0) >= 12 * rows and bwd(rows, 64, 2, BF16, 0) >= 128 * rows
    assert fwd(2 ** 29 + 1024, 64, 2, BF16, 0) == 0 and fwd(2 ** 31 - 1, 64, 2, BF16, 0) == 0


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="fake-pointer validation tests run only without a GPU")
def test_route_refuses_counts_that_overflow(lib):
    gib, shape = 1 << 30, -2
    for tokens in (2 ** 26, 2 ** 31, 2 ** 57, 2 ** 58, 2 ** 62, 2 ** 63 - 1):
        assert lib.layers_route(gib, 8, F32, tokens, 8, 2, 0, None, 1, 1, 1, 1, 1.0, 64 * gib, 128 * gib, None) == shape
        assert lib.layers_route_backward(gib, 32 * gib, 8, 64 * gib, F32, tokens, 8, 2, 0, 1, 1.0, 128 * gib, 8, None) == shape
        assert lib.layers_embed(gib, tokens, 32 * gib, F32, 8, 8, 1.0, 64 * gib, 8, None) == shape
