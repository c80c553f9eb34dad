"""More rows in 8 bits than one launch takes (2^34 values)."""
import pytest
import torch

from helpers import say
from test_gpu_kept import rows_of

pytestmark = pytest.mark.gpu


def test_more_than_one_launch(gpu_lib):
    """Rows on both sides of the border between launches, and the last ones, are as alone."""
    width, first = 32736, (1 << 34) // 32736  # rows of one launch, a group short of 2^15
    rows = first + 9
    say(f"keep {rows} x {width}")
    few = {0: 3, first - 4: 8, rows - 3: 3}
    assert rows * width > 1 << 34
    x = torch.zeros((rows, width), dtype=torch.bfloat16, device="cuda")
    alone = {}
    for n, (at, count) in enumerate(few.items()):
        part = rows_of(51 + n, count, width).cuda()
        x[at:at + count] = part
        alone[at] = gpu_lib.keep(part)
    kept = gpu_lib.keep(x)
    out = gpu_lib.restore(kept, out=x.fill_(3.0))
    for at, count in few.items():
        part = slice(at, at + count)
        assert torch.equal(kept.codes[part], alone[at].codes)
        assert torch.equal(kept.exponents[part], alone[at].exponents)
        assert torch.equal(out[part], gpu_lib.restore(alone[at]))
        kept.exponents[part] = 0
        out[part] = 0
    assert not bool(kept.exponents.any())
    for at in range(0, rows, 65536):  # in steps: the check's own memory
        assert not bool(out[at:at + 65536].any())
