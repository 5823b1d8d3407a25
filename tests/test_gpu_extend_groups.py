"""Which sequences share a prefix: offsets of groups that do not go together, groups behind sequences of
no group, idle first members, prefixes longer than the table. Against float64.

Tolerance of `out`, relative in the L2 norm, a sequence at a time: bf16 rounds the result and the weights, by
2^-8 of each number at most, and the weights' errors are as independent as the values that they
multiply: 2^-7. float32: a score is a sum of dh <= 128 products, off by at most dh 2^-24 sum |q k| scale < 2^-13,
and so is its weight; sums add less: 2^-12. lse is off by a score's error: 2^-12, and its rounding. A key tile
that is missing or another's is sqrt(64 / keys) or more: 0.02 of 131072 keys.
"""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from _shared_prefix import BF16, F32, Prefixed, ints
from context_blockwise_attention_step_gb300 import _abi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def check(b, got, ref, what="", status=_abi.RA_OK):
    assert ra.check_device_status() == status, f"{what} {ra.last_error()}"
    (out, lse), (want, want_lse) = got, ref
    for i, m in enumerate(b.lens):
        rows = slice(int(b.cu[i]), int(b.cu[i + 1]))
        if m == 0:
            assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all(), f"{what} sequence {i} is idle"
        elif b.news[i]:
            off = ((out[rows].double() - want[rows]).norm() / want[rows].norm()).item()
            assert off <= (2.0 ** -7 if b.dtype == BF16 else 2.0 ** -12), f"{what} out of sequence {i}: {off:.2e}"
            off = (lse[rows] - want_lse[rows]).abs() - 2.0 ** -22 * want_lse[rows].abs()
            assert off.max() <= 2.0 ** -12, f"{what} lse of sequence {i}: {off.max():.2e}"


@pytest.mark.parametrize("dtype,dh", [(BF16, 64), (F32, 40)], ids=str)
@pytest.mark.parametrize("news", [None, [1, 2, 1, 3, 1, 1]], ids=["one", "several"])
def test_offsets_that_do_not_go_together_share_nothing(dtype, dh, news):
    """Groups that would overlap, or leave the batch: recorded, and every sequence reads its own keys."""
    b = Prefixed(1, dtype, 8, 2, dh, 16, [(6, 4000)], [3, 5, 1, 20, 7, 2], news, hide=False)
    ref = b.reference()
    check(b, b.run(), ref, "in order")
    for cu in ([0, 5, 2, 6], [0, 6, 0, 6], [-1, 6, 6, 6], [0, 3, 6, 7], [4, 2, 1, 0], [0, 2147483647, 6, 6], [-2147483648, 2, 4, 6]):
        shared = ra.SharedPrefix(ints(cu), ints([4000] * 3))
        check(b, b.run(shared=shared), ref, str(cu), _abi.RA_ERR_CACHE_INDEX)
        assert ra.check_device_status() == _abi.RA_OK
        first = b.run(shared=shared)
        assert all(torch.equal(x, y) for x, y in zip(first, b.run(shared=shared)))
        ra.check_device_status()
    for cu in ([0, 0, 6, 6], [6, 6, 6, 6], [0, 3, 3, 6]):  # in order: groups may be empty, and need not be all
        check(b, b.run(shared=ra.SharedPrefix(ints(cu), ints([4000] * 3))), ref, str(cu))


@pytest.mark.parametrize("dtype,dh,news", [(BF16, 64, None), (BF16, 64, [1, 3, 0, 2]), (F32, 8, [2, 1, 0, 1])], ids=str)
def test_more_segments_than_the_plan_has_threads(dtype, dh, news):
    """1500 sequences, 700 groups among them, of which every 50th has a prefix long enough to be shared: the
    plan takes them in several rounds. Every 13th sequence is idle, or has no new token."""
    tile = 128 if dtype == BF16 else 64
    n, m = 1500, 700
    groups = [(2, 14 * tile + 5 if i % 50 == 0 else tile + i % 40) for i in range(m)]
    own = [0 if i % 13 == 5 and news is None else 5 + i % 7 for i in range(n)]
    new = None if news is None else [0 if i % 13 == 5 else news[i % 4] for i in range(n)]
    b = Prefixed(2, dtype, 4, 1, dh, 16, groups, own, new, lead=n - 2 * m, hide=False)
    ref = b.reference()
    got = b.run()
    check(b, got, ref)
    assert all(torch.equal(x, y) for x, y in zip(got, b.run()))
    check(b, b.run(shared=None), ref, "apart")
    one = ra.SharedPrefix(ints([0, 0] + [n] * 3), ints([7, 0, 0, 0]))  # groups of all, and of none
    check(b, b.run(shared=one), ref, "one group")


@pytest.mark.parametrize("dtype,dh", [(BF16, 128), (F32, 64)], ids=str)
def test_no_new_tokens_at_all(dtype, dh):
    """Offsets that give no sequence a row: nothing is written, and it is no error."""
    b = Prefixed(3, dtype, 8, 2, dh, 16, [(3, 4000)], [5, 7, 9], [1, 2, 1])
    out, lse = torch.full_like(b.q, 7.0), torch.full(b.q.shape[:2], 7.0, device="cuda")
    for at in (0, 2, 4):
        b.run(cu_new=ints([at] * 4), out=out, lse=lse)
    assert ra.check_device_status() == _abi.RA_OK, ra.last_error()
    assert (out == 7).all() and (lse == 7).all()
