"""CPU: the sizes of the GPU tests take the ways of cutting a product that
they are there for (the rule goes by sizes alone)."""
import pytest

from integer_only_nn_amd import ops
from test_gpu_dfp8_paths import SIZES


@pytest.mark.parametrize("size", list(SIZES))
def test_sizes_take_their_ways(size):
    assert tuple(ops.dfp8_linear_path(p, *size) for p in ("fwd", "dX", "G")) == SIZES[size]


def test_every_way_is_taken_by_some_size():
    for i, ways in enumerate(({"rows", "tiles 256", "tiles 128", "tiles", "narrow"}, *[{"tiles 256", "tiles 128", "tiles", "narrow"}] * 2)):
        assert {v[i] for v in SIZES.values()} == ways
    # reductions cut into ranges, whose sums take a workspace
    assert ops.dfp8_linear_fwd_workspace_bytes(300, 9001, 600) > 0


def test_refuses_sizes_out_of_range():
    for size in ((-1, 4, 4), (4, (1 << 30) + 1, 4)):
        with pytest.raises(ValueError):
            ops.dfp8_linear_path("fwd", *size)
    with pytest.raises(ValueError):
        ops.dfp8_linear_path("dW", 4, 4, 4)
