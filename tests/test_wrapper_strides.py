"""Strides that the C calls cannot describe are refused by the torch wrappers: rows
(or columns) that start less than a row's length apart, as in expanded tensors, which
the kernels would read as others and behind the tensor's end."""
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc

BF, I32 = torch.bfloat16, torch.int32


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


OFFSETS = torch.zeros(3, dtype=I32)
# 8 x 5 matrices: one row for all, one column for all, one number for all, rows and columns that overlap
VIEWS = {
    "rows": lambda: z(1, 5).expand(8, 5),
    "columns": lambda: z(8, 1).expand(8, 5),
    "number": lambda: z(1, 1).expand(8, 5),
    "overlapping rows": lambda: z(32).as_strided((8, 5), (2, 1)),
    "overlapping columns": lambda: z(48).as_strided((8, 5), (1, 7)),
    "hankel": lambda: z(32).as_strided((8, 5), (1, 1)),
    "no unit stride": lambda: z(16, 10)[::2, ::2],
}


@pytest.mark.parametrize("view", sorted(VIEWS))
def test_weights(view):
    b = VIEWS[view]()
    grouped = b.as_strided((2, 8, 5), (0, *b.stride()))
    with pytest.raises(ValueError, match="row- or column-major"):
        ttc.gemm_grouped(z(4, 8), grouped, OFFSETS)


@pytest.mark.parametrize("view", [lambda: z(2, 1, 5).expand(2, 8, 5), lambda: z(2, 8, 1).expand(2, 8, 5),
                                  lambda: z(64).as_strided((2, 8, 5), (20, 2, 1))])
def test_weights_of_groups(view):
    with pytest.raises(ValueError, match="row- or column-major"):
        ttc.gemm_grouped(z(4, 8), view(), OFFSETS)


@pytest.mark.parametrize("view", sorted(VIEWS))
def test_gemm_operands(view):
    m = VIEWS[view]()
    with pytest.raises(ValueError, match="row- or column-major"):
        ttc.gemm(z(4, 8), m)
    with pytest.raises(ValueError, match="row- or column-major"):
        ttc.gemm(m, z(5, 3))


@pytest.mark.parametrize("cols", [1, 5])
def test_vectors_that_repeat_a_number(cols):
    with pytest.raises(ValueError, match="row- or column-major"):
        ttc.gemm(z(4, 8), z(1, 1).expand(8, 1) if cols == 1 else z(8, 1).expand(8, cols))
    with pytest.raises(ValueError, match="row- or column-major"):
        ttc.gemm(z(1, 1).expand(1, 8), z(8, 3))


@pytest.mark.parametrize("bad", [lambda: z(1, 5).expand(4, 5), lambda: z(5, 4).T, lambda: z(32).as_strided((4, 5), (2, 1)),
                                 lambda: z(1, 5), lambda: z(4, 4)])
def test_gemm_sum_and_result(bad):
    with pytest.raises(ValueError):
        ttc.gemm(z(4, 8), z(8, 5), out=bad())
    with pytest.raises(ValueError):
        ttc.gemm(z(4, 8), z(8, 5), c=bad(), out=z(4, 5), beta=1.0)


@pytest.mark.gpu
def test_a_sum_that_is_not_read_may_have_any_strides():
    a, b = torch.randn(4, 8, device="cuda").to(BF), torch.randn(8, 5, device="cuda").to(BF)
    c = torch.full((1, 5), float("nan"), dtype=BF, device="cuda").expand(4, 5)
    assert torch.equal(ttc.gemm(a, b, c=c), ttc.gemm(a, b))


R, C = ttc.ROW_MAJOR, ttc.COL_MAJOR


@pytest.mark.parametrize("t,rows,cols,want", [
    (lambda: z(8, 5), 8, 5, (R, 5)), (lambda: z(5, 8).T, 8, 5, (C, 8)), (lambda: z(8, 9)[:, :5], 8, 5, (R, 9)),
    (lambda: z(5, 11)[:, :8].T, 8, 5, (C, 11)), (lambda: z(8, 1), 8, 1, (C, 8)), (lambda: z(8, 3)[:, :1], 8, 1, (R, 3)),
    (lambda: z(1, 5), 1, 5, (R, 5)), (lambda: z(5, 3)[:, :1].T, 1, 5, (C, 3)), (lambda: z(1, 1), 1, 1, (C, 1)),
    (lambda: z(1, 1).expand(1, 1), 1, 1, (C, 1)), (lambda: z(1, 5).as_strided((1, 5), (0, 1)), 1, 5, (R, 5)),
    (lambda: z(8, 1).as_strided((8, 1), (1, 0)), 8, 1, (C, 8)), (lambda: z(0, 5), 0, 5, (R, 5)), (lambda: z(8, 0), 8, 0, (R, 1)),
])
def test_layouts_as_before(t, rows, cols, want):
    assert ttc._matrix_layout(t(), rows, cols) == want
