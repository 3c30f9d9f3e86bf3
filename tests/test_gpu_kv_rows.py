"""Every row of the cached contexts is read once and weighed by itself (tests/kv_rows.py): long contexts over all
shares, joins, windows, sinks, pages that end inside a tile."""
import pytest

from kv_rows import check_each_row, check_whole_numbers, whole_numbers
from plain_kv import KvCase
from test_gpu_kv_cache import attend

pytestmark = pytest.mark.gpu

CASES = [
    # lens, new, heads, kv_heads, page_size, window, sinks
    ([33000], [1], 1, 1, 8, 0, 0),
    ([20000], [1], 8, 2, 16, 0, 0),
    ([9000], [200], 8, 1, 3, 0, 0),
    ([7000], [130], 4, 2, 1, 0, 0),
    ([6000], [100], 6, 1, 24, 5000, 100),
    ([9000, 300], [3, 1], 4, 2, 16, 4097, 65),
    ([5000, 0, 40, 4000, 9], [1, 0, 0, 3, 0], 8, 4, 16, 0, 0),
    (list(range(0, 1400, 20)), [1] * 70, 8, 2, 16, 0, 0),
    ([3000] * 33 + [0] * 33, [1] * 33 + [0, 2] * 16 + [1], 4, 1, 16, 0, 0),
    ([10, 700, 64, 0], [128, 129, 256, 257], 1, 1, 16, 0, 0),
    ([700, 10], [1, 3], 160, 1, 16, 0, 0),
    ([63, 64, 127, 128, 129], [70, 1, 64, 65, 130], 4, 1, 16, 63, 65),
    ([63, 64, 65, 1000], [2, 1, 1, 300], 4, 2, 100, 64, 64),
    ([400, 1000], [65, 300], 2, 1, 8, 128, 1),
    ([2000, 1], [520, 700], 4, 2, 16, 0, 0),
]


@pytest.mark.parametrize("D, dtype", [(64, "bf16"), (128, "bf16"), (64, "e4m3"), (128, "e4m3"), (80, "e4m3"), (80, "bf16"),
                                      (128, "f32"), (256, "f32")])
@pytest.mark.parametrize("lens, new, H, KH, page_size, window, sinks", CASES)
def test_each_row_counts_once(lens, new, H, KH, page_size, window, sinks, D, dtype):
    case = KvCase(50, lens, new, H, KH, D, page_size=page_size, dtype=dtype, window=window, sinks=sinks)
    check_each_row(case, lambda c: attend(c, guard=False))
    if max(lens) <= 9000:
        whole_numbers(case)
        check_whole_numbers(case, attend(case)[1])
