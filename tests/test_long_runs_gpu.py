"""The training operators where each thread does the same thing many times: rows
enough for a group of lanes to go round its ring of stages twice and more, grids
in several waves, sorts of more partitions and digits.  Against the 64-bit forms,
with the checks and tolerances of the operators' own tests."""
import pytest

import test_embed_gpu
import test_norm_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gaussian_splatting_differentiable_gb300 as m
    return m


# (n, D, type, parameters' type, padding, offset): 8 rows at least to a group of
# lanes, of which at most 4 lie in the ring; the widths take 1 to 4 vectors a lane
# in part of a warp, several warps, and rows that start everywhere between the
# 16-byte boundaries.  2,000,003 rows are past 48 turns of the device, where the
# grid is eight times what fits.
ROWS = [(300000, 48, "f32", "f32", 0, 0), (400000, 7, "bf16", "bf16", 2, 0), (250000, 35, "f16", "f32", 0, 1),
        (330000, 16, "bf16", "f32", 0, 0), (200000, 50, "f32", "f32", 1, 3), (120000, 128, "f16", "f16", 0, 0),
        (16000, 1000, "bf16", "f32", 0, 0), (16000, 1001, "f16", "f16", 0, 0), (9000, 1030, "f32", "f32", 0, 0),
        (4500, 4096, "bf16", "f32", 0, 0), (3500, 5001, "f32", "f32", 0, 0), (2000003, 3, "f32", "f32", 0, 0)]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(map(str, c)))
def test_norm(ss, case):
    test_norm_gpu.fwd_case(ss, *case)                # in place as well


@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(map(str, c)))
def test_norm_gradient(ss, case):
    test_norm_gpu.bwd_case(ss, *case)


@pytest.mark.parametrize("inplace", ["dy", "x"])
@pytest.mark.parametrize("case", [ROWS[0], ROWS[2], ROWS[7], ROWS[9]], ids=lambda c: "-".join(map(str, c)))
def test_norm_gradient_in_place(ss, case, inplace):
    test_norm_gpu.bwd_case(ss, *case, inplace=inplace)


@pytest.mark.parametrize("D", [61, 1030, 5001])
def test_every_row_of_many_is_far_from_its_spread(ss, D):
    """The correction of the mean, for every row of a ring that goes round."""
    n = {61: 200000, 1030: 9000, 5001: 3500}[D]
    test_norm_gpu.fwd_case(ss, n, D, "f32", "f32", 0, 0, shift=500.0)


# The widest rows that lie in registers, whatever their start, and the next.
@pytest.mark.parametrize("D,t", [(8195, "f32"), (8196, "f32"), (8199, "bf16"), (8200, "f16")])
@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1)])
def test_norm_where_registers_end(ss, D, t, pad, off):
    test_norm_gpu.fwd_case(ss, 5, D, t, "f32", pad, off)
    test_norm_gpu.bwd_case(ss, 5, D, t, "f32", pad, off)


# (n, V, D, type, gradient's type, ids' type, spread, padding, offset): more than
# the 1024 partitions that one turn of the scan takes; four digits of the key.
IDS = [(2200000, 1000, 1, "f32", "f32", "int32", "uniform", 0, 0),
       (2300001, 70000, 2, "bf16", "f32", "int64", "log", 0, 0),
       (2200000, 3, 1, "f16", "f16", "int32", "absent", 0, 0),
       (5000, (1 << 24) + 5, 1, "f32", "f32", "int64", "uniform", 0, 0),
       (70000, (1 << 24) + 5, 1, "bf16", "bf16", "int32", "log", 0, 0)]


@pytest.mark.parametrize("case", IDS, ids=lambda c: "-".join(map(str, c)))
def test_table_gradient(ss, case):
    test_embed_gpu.bwd_case(ss, *case)
