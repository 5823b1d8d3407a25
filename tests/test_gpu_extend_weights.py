"""How exactly the softmax's weights enter the product with the values, bf16: a step that is given shared
prefixes is as good as one that reads every sequence apart.

`out` is rounded to bf16, which puts ||bf16(ref) - ref|| between it and the definition. Weights of two
bf16 numbers are off by 2^-16 of themselves, and by a score's error, below 2^-12 at the worst and 2^-15 on
average: beside the rounding, 0.0017 of the result, they do not count, and the distance is ||bf16(ref) - ref|| but for
the numbers that lie next to a border: 1.1 times that leaves room for an error of 0.0007. Weights of one
bf16 number are off like the result, 0.0017 on average, and the distance would be 1.4 times that.
"""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from _shared_prefix import BF16, Prefixed
from test_gpu_extend_groups import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


CASES = [
    # hq, hkv, dh, page, sequences of no group, groups, own keys, news
    (32, 8, 128, 64, 0, [(24, 4000)], [1 + i % 9 for i in range(24)], None),
    (8, 8, 64, 16, 2, [(40, 2000), (33, 1500)], [1 + i % 70 for i in range(75)], None),
    (16, 1, 64, 64, 0, [(33, 1000)], [1 + i % 3 for i in range(33)], None),     # 528 rows: three blocks
    (48, 1, 128, 64, 0, [(6, 1700)], [1, 2, 3, 4, 5, 600], None),               # own keys on the tensor cores too
    (130, 1, 64, 64, 0, [(4, 1700)], [1, 2, 3, 4], None),                        # (a tile's rows are too few to share)
    (12, 1, 64, 64, 0, [(3, 100000)], [3, 1, 40], None),
    (16, 4, 128, 16, 0, [(20, 3000)], [4 + i % 5 for i in range(20)], [1 + i % 4 for i in range(20)]),  # drafts
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}_dh{c[2]}_n{len(c[6])}_{'some' if c[7] else 'one'}")
def test_sharing_costs_no_precision(case):
    hq, hkv, dh, page, lead, groups, own, news = case
    b = Prefixed(7, BF16, hq, hkv, dh, page, groups, own, news, lead, hide=hq <= 64 * hkv)
    ref = b.reference()
    got = b.run()
    check(b, got, ref)
    least = (ref[0].bfloat16().double() - ref[0]).norm()
    off = ((got[0].double() - ref[0]).norm() / least).item()
    assert off <= 1.1, f"{off:.3f} of the result's own rounding"


def test_a_member_with_many_rows_takes_nothing_from_the_others():
    """Drafts beside a part of a prompt, behind one prefix, most rows being drafts': these are as good as alone."""
    news = [2, 1, 3, 2] * 5 + [30] + [2, 1, 3, 2] * 4
    b = Prefixed(8, BF16, 16, 4, 64, 64, [(37, 9000)], [5 + n for n in news], news)
    ref, got = b.reference(), b.run()
    check(b, got, ref)
    rows = torch.cat([torch.arange(b.cu[i], b.cu[i + 1]) for i in range(37) if i != 20]).cuda()
    want = ref[0][rows]
    off = ((got[0][rows].double() - want).norm() / (want.bfloat16().double() - want).norm()).item()
    assert off <= 1.1, f"{off:.3f} of the result's own rounding"
