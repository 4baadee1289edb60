"""CPU tests that an F8Weight is not made of planes that the calls would read past:
each plane has the bytes of its sizes, and the transposed ones come together."""
import pytest
import torch

from decode_gemv_tensor_amd import binade as B

ROWS, COLS, COUNT = 300, 416, 2
BYTES = {"values": COUNT * 300 * 512, "scales": COUNT * 3 * 4, "values_t": COUNT * 416 * 384, "scales_t": COUNT * 4 * 4}


def planes(**kw):
    p = {name: torch.zeros(n, dtype=torch.uint8) for name, n in BYTES.items()}
    p.update(kw)
    return p


def test_planes_of_their_sizes():
    w = B.F8Weight(ROWS, COLS, COUNT, B.E8M0, **planes())
    assert w.desc().rows == ROWS and w.desc().count == COUNT
    B.F8Weight(ROWS, COLS, COUNT, B.E8M0, **planes(values_t=None, scales_t=None))
    B.F8Weight(ROWS, COLS, COUNT, B.F32, **planes(scales=torch.zeros(4 * BYTES["scales"], dtype=torch.uint8),
                                                  scales_t=torch.zeros(4 * BYTES["scales_t"], dtype=torch.uint8)))


@pytest.mark.parametrize("name", list(BYTES))
def test_planes_of_other_sizes(name):
    n = BYTES[name]
    for t in (torch.zeros(n - 1, dtype=torch.uint8), torch.zeros(n + 16, dtype=torch.uint8),
              torch.zeros(n, dtype=torch.int32), torch.zeros(2 * n, dtype=torch.uint8)[::2],
              torch.zeros(n, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match=name if t.device.type != "meta" else "is on"):
            B.F8Weight(ROWS, COLS, COUNT, B.E8M0, **planes(**{name: t}))


def test_sizes_that_no_weight_has():
    for rows, cols, count, dtype in ((0, 32, 1, B.E8M0), (1, 33, 1, B.E8M0), (1, 32, 0, B.E8M0), (1, 32, 1, B.BF16),
                                     (1, 32, 65536, B.E8M0)):
        with pytest.raises(B.BinadeError):
            B.F8Weight(rows, cols, count, dtype, **planes())
    for kw in ({"values_t": None}, {"scales_t": None}):
        with pytest.raises(ValueError, match="both"):
            B.F8Weight(ROWS, COLS, COUNT, B.E8M0, **planes(**kw))
