"""Rotations of part of a head: what is not rotated passes through bit for bit, infinities as well."""
import pytest
import torch

import context_blockwise_attention_step_gb300 as ra

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _build():
    ra.build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")


# dtype, dh, rotary, interleaved: the 16-byte kernels, and (22, 20, odd sizes) the others
CASES = [(BF16, 128, 64, False), (BF16, 64, 16, False), (BF16, 64, 22, True), (BF16, 128, 4, True), (BF16, 64, 22, False),
         (F32, 128, 24, False), (F32, 64, 6, True), (F32, 48, 16, False), (F32, 24, 10, True), (F32, 96, 20, False),
         (F32, 33, 2, False), (F32, 7, 4, True)]
IDS = [f"{str(c[0])[6:]}_dh{c[1]}_r{c[2]}{'_i' if c[3] else ''}" for c in CASES]


def data(dt, dh, rd, seed):
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn(2, 12, h, dh, generator=g).to(dt).cuda() for h in (6, 3)]
    y = [t.clone() for t in x]
    for t in y:
        t[:, 1::2, :, rd] = float("inf")
        t[:, ::2, 1, -1] = -float("inf")
        t[0, 3, 0, rd:] = float("inf")
    return x, y


@pytest.mark.parametrize("dt,dh,rd,inter", CASES, ids=IDS)
def test_infinities_beside_the_rotation_pass(dt, dh, rd, inter):
    (q, k), (qi, ki) = data(dt, dh, rd, 3)
    prob = ra.problem_for(q, k, D=2, layout="zigzag")
    rope = ra.make_rope(rd, interleaved=inter)
    plain = ra.qk_norm_rope_fwd(q, k, prob, rope=rope)
    got = ra.qk_norm_rope_fwd(qi, ki, prob, rope=rope)
    for a, b, x in zip(got, plain, (qi, ki)):
        assert torch.equal(a[..., :rd], b[..., :rd])
        assert torch.equal(a[..., rd:], x[..., rd:])
    plain = ra.qk_norm_rope_bwd(q, k, q, k, prob, rope=rope)
    got = ra.qk_norm_rope_bwd(qi, ki, q, k, prob, rope=rope)
    for a, b, x in zip(got[:2], plain[:2], (qi, ki)):
        assert torch.equal(a[..., :rd], b[..., :rd])
        assert torch.equal(a[..., rd:], x[..., rd:])


@pytest.mark.parametrize("dt,dh,rd,inter", CASES, ids=IDS)
def test_infinities_beside_the_rotation_pass_into_the_cache(dt, dh, rd, inter):
    (q, k), (qi, ki) = data(dt, dh, rd, 4)
    q, k, qi, ki = (t[:, 3].contiguous() for t in (q, k, qi, ki))
    rope = ra.make_rope(rd, interleaved=inter)
    lens = torch.tensor([6, 2], dtype=torch.int32).cuda()
    out = []
    for a, b in ((q, k), (qi, ki)):
        pages = torch.zeros(2, 2, 8, 3, dh, dtype=dt, device="cuda")
        cache = ra.make_cache(pages[0], pages[1], torch.tensor([[0], [1]], dtype=torch.int32).cuda())
        out.append((a, ra.kv_cache_append(a, b, b, cache, lens, rope=rope), torch.stack([pages[0, 0, 5], pages[0, 1, 1]])))
    (_, q0, k0), (x, q1, k1) = out
    assert torch.equal(q1[..., :rd], q0[..., :rd]) and torch.equal(q1[..., rd:], x[..., rd:])
    assert torch.equal(k1[..., :rd], k0[..., :rd]) and torch.equal(k1[..., rd:], ki[..., rd:])
