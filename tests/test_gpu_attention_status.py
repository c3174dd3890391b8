"""Status words of spec_verify_attention for sequences that have no rows to compute."""
import numpy as np
import pytest

from tests.test_gpu_attention import SENT, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("root", [True, False])
@pytest.mark.parametrize("B", [7, 700])
def test_counts_out_of_range_are_reported_without_rows(B, root):
    num = np.resize([3, -2, 0, 4, -1, 2 ** 31 - 1, -2 ** 31], B)
    lens = np.resize([20, 30, 5, -1, -7, -1, 0], B)
    c = Case(60, list(lens), 3, 4, 2, 64, 16, root=root, num=num)
    out, st = c.run()
    assert st == [4 if not 0 <= n <= 3 else 0 for n in num]
    c.check(out, range(0, B, max(1, B // 20)))
    c.num[:] = -1                                       # nobody has rows
    c.lens[:] = -1
    out, st = c.run()
    assert st == [4] * B and (out == SENT).all()
