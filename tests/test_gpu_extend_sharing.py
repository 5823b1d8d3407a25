"""Prefixes that are shared in fact. Only a group's first member has the shared pages in its row of the
block table (tests/_shared_prefix.py): a call that read a member's own row there would record an index outside the
cache, so a case that is not shared, for whatever rule, fails here. Tolerances as in test_gpu_extend_groups.py,
where they are derived; repeats of a call give the same bits.
"""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra
from _shared_prefix import BF16, F32, HIDDEN, Prefixed, ints
from context_blockwise_attention_step_gb300 import _abi
from test_gpu_extend_groups import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


CASES = [
    # dtype, hq, hkv, dh, page, sequences of no group, groups, own keys (0: idle), news, pages
    (BF16, 16, 4, 64, 16, 0, [(3, 2005), (3, 1100), (1, 0)], [5, 1, 30, 5, 1, 7, 40], None, "pshd"),
    (BF16, 32, 8, 128, 64, 1, [(8, 4000)], [9, 0, 1, 64, 130, 2, 3, 5, 128], None, "pshd"),   # an idle first member
    (BF16, 8, 2, 128, 48, 2, [(4, 1500), (9, 900)], [3, 700] + [1, 2, 3, 4] + [0, 0, 1, 2, 3, 4, 0, 5, 6], None, "phsd"),
    (BF16, 8, 4, 64, 16, 0, [(3, 2048)], [4, 18, 1], None, "wide"),
    (BF16, 8, 8, 64, 7, 0, [(5, 1000)], [1, 1, 2, 1, 9], None, "pshd"),                       # pages end inside a tile
    (BF16, 4, 1, 128, 64, 0, [(70, 2100)], [1 + i % 5 for i in range(70)], None, "pshd"),     # blocks of two tiles of rows
    (BF16, 48, 1, 64, 32, 0, [(6, 1700)], [1, 2, 3, 4, 5, 6], None, "pshd"),                  # more heads than few rows
    (BF16, 12, 1, 64, 64, 0, [(3, 100000)], [3, 1, 40], None, "pshd"),                        # a row's parts on every CTA
    (BF16, 6, 6, 128, 64, 0, [(2, 30000)], [1, 2], None, "pshd"),                             # two rows behind the prefix
    (BF16, 8, 2, 128, 64, 0, [(5, 6500)], [100, 13, 190, 1, 70], [100, 3, 190, 1, 70], "pshd"),
    (BF16, 8, 1, 128, 64, 0, [(3, 20011)], [70, 5, 60], [30, 5, 29], "pshd"),
    (BF16, 12, 4, 64, 32, 2, [(3, 1700), (4, 2600)], [40, 9] + [10, 30, 2, 9, 9, 9, 100], [4, 9] + [10, 1, 2, 0, 9, 4, 90], "phsd"),
    (BF16, 16, 4, 64, 16, 0, [(9, 3000)], [7, 2, 3, 4, 12, 4, 3, 2, 5], [4, 2, 3, 4, 4, 4, 3, 2, 1], "wide"),  # drafts
    (F32, 8, 2, 64, 16, 1, [(5, 2005), (3, 1333)], [20] + [0, 40, 3, 7, 9, 5, 1, 1], None, "pshd"),
    (F32, 6, 1, 40, 7, 0, [(6, 2000)], [12, 20, 3, 9, 5, 1], [12, 3, 1, 2, 5, 1], "pshd"),
    (F32, 8, 1, 64, 64, 0, [(4, 20000)], [3, 1, 40, 2], None, "phsd"),
    (F32, 4, 2, 128, 16, 0, [(5, 2000)], [50, 20, 3, 9, 1], [33, 12, 3, 1, 1], "wide"),
]


def made(case, hide=True, seed=3):
    dt, hq, hkv, dh, page, lead, groups, own, news, order = case
    return Prefixed(seed, dt, hq, hkv, dh, page, groups, own, news, lead, order, hide, scale=1.5)


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}_{c[1]}x{c[2]}_dh{c[3]}_n{len(c[7])}_{'some' if c[8] else 'one'}")
def test_one_table_row_is_read_for_the_group(case):
    b = made(case)
    ref = b.reference()
    got = b.run()
    check(b, got, ref)
    assert same(got, b.run())
    every = made(case, hide=False)
    assert same(got, every.run())
    check(b, every.run(shared=None), ref, "apart")
    if b.cu_new is None:
        assert same(got, ra.paged_attn_decode(b.q, b.cache, b.seq_lens, shared=b.shared))
        if all(b.lens):
            check(b, b.run(cu_new=ints(b.cu)), ref, "one token each, by offsets")
    assert ra.check_device_status() == _abi.RA_OK, ra.last_error()


def two():
    """One token each behind two prefixes, with an idle first member and a sequence of no group; and several tokens."""
    return (made((BF16, 16, 4, 64, 16, 1, [(4, 2005), (3, 1100), (1, 0)], [70, 0, 5, 1, 30, 5, 1, 7, 40], None, "pshd")),
            made((BF16, 8, 2, 128, 64, 0, [(5, 6500)], [100, 13, 190, 1, 70], [100, 3, 190, 1, 70], "pshd"), seed=4))


def test_streams_graphs_and_workspaces():
    for b in two():
        ref = b.reference()
        want = b.run()
        check(b, want, ref)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = b.run(stream=s)
        s.synchronize()
        assert same(got, want)
        n = ra.paged_extend_workspace_bytes(b.cache, b.q.shape[0], b.hq, b.shared)
        ws = torch.full((n,), 0xFF, device="cuda", dtype=torch.uint8)
        out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        graphs = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()  # that share the workspace
        for graph in graphs:
            with torch.cuda.graph(graph):
                b.run(workspace=ws, out=out, lse=lse)
        for fill in (0xFF, 0x00, 0x7F):
            ws.fill_(fill)
            for graph in graphs:
                out.zero_()
                graph.replay()
                assert same((out, lse), want)
        assert ra.check_device_status() == _abi.RA_OK, ra.last_error()
        # lengths and prefixes are read when the graph runs: a shorter prefix, then none
        keep = b.shared.prefix_lens.clone()
        b.table.copy_(made_table(b))
        for part in (keep // 2, torch.zeros_like(keep)):
            b.shared.prefix_lens.copy_(part)
            graphs[0].replay()
            check(b, (out, lse), ref, str(part.tolist()))
        b.shared.prefix_lens.copy_(keep)
        graphs[1].replay()
        assert same((out, lse), want)


def made_table(b):
    """b's block table with every member's pages."""
    t = b.table.clone()
    cu = b.shared.cu_groups.tolist()
    for lo, hi in zip(cu, cu[1:]):
        live = [i for i in range(lo, hi) if b.lens[i] and b.news[i]]
        for i in live[1:]:
            hidden = t[i] == HIDDEN
            hidden[-(-b.lens[i] // b.pages[0].shape[1]):] = False
            t[i][hidden] = t[live[0]][hidden]
    return t


def test_two_calls_at_once():
    """On two streams, with workspaces of their own, many times over: the same bits."""
    one, many = two()
    want = one.run(), many.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = [(one.run(stream=s1), many.run(stream=s2)) for _ in range(10)]
    torch.cuda.synchronize()
    for a, b in got:
        assert same(a, want[0]) and same(b, want[1])
    assert ra.check_device_status() == _abi.RA_OK, ra.last_error()


def test_prefixes_that_not_every_member_has():
    """Longer than the table or than a member, the new token in it, negative: that group shares nothing, another
    one does; and rows before and behind the sequences are left as they are."""
    b = made((BF16, 8, 2, 64, 16, 1, [(4, 1600), (3, 2000)], [5, 0, 7, 2, 200, 4, 1, 60], None, "pshd"), hide=False)
    ref = b.reference()
    for prefix in ([1 << 30, 2000], [2147483647, 5], [1603, 2000], [-3, 2000], [1602, 1999], [-2147483648, 0]):
        shared = ra.SharedPrefix(b.shared.cu_groups, ints(prefix))
        check(b, b.run(shared=shared), ref, str(prefix))
    b = made((BF16, 8, 2, 64, 16, 0, [(4, 6500)], [5, 70, 2, 200], [5, 66, 2, 90], "pshd"))
    want = b.run()
    pad = 5
    q = torch.cat([torch.full_like(b.q[:pad], float("nan")), b.q, torch.full_like(b.q[:pad], float("nan"))])
    out, lse = torch.full_like(q, 7.0), torch.full((q.shape[0], 8), 7.0, device="cuda")
    b.run(q=q, cu_new=b.cu_new + pad, out=out, lse=lse)
    check(b, want, b.reference())
    assert same((out[pad:-pad], lse[pad:-pad]), want)
    for t in (out, lse):
        assert (t[:pad] == 7).all() and (t[-pad:] == 7).all()
