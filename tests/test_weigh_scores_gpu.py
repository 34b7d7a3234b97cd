"""What weights and log-sum-exps are off by through their scores, which the tensor
cores cut off and both calls raise alike: nothing on average for ordinary data,
what they are raised by where a score's products sum without loss, and nothing
in the sum of a row's weights with the lse of mla_verify_attn_chunk."""
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb
from tests import chunk_util as C

pytestmark = pytest.mark.gpu

U = 2.0 ** -24       # half a step of fp32
RAISED = 2 * 3.8     # what scores are raised by, in U
ORDINARY = 4e-7      # of a score, on average: below the 4.5e-7 that it is raised by and the 4e-7 to 6e-7 that it loses


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def requests(B, n, page):
    """Tables of B requests of n rows each, one new token of one head each, in order in the cache."""
    entries = -(-n // page)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = -(-B * entries * page // 64) * 64
    return slots, dict(kv_indices=torch.arange(B * entries, dtype=torch.int32, device="cuda"),
                       kv_indptr=i32([entries * b for b in range(B + 1)]), kv_lens=i32([n] * B), q_indptr=i32(list(range(B + 1))),
                       H=1, page=page)


def weigh(plan, d, lse, scale):
    w = torch.zeros(d["kv_lens"].numel(), plan.max_kv_len, device="cuda")
    mb.weigh_kv(plan, d["q"], d["cache"], d["kv_indices"], d["kv_indptr"], d["kv_lens"], d["q_indptr"], lse, scale, w)
    torch.cuda.synchronize()
    assert plan.get_error() == 0
    return w.double()


@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("score", [64.0, 1000.0, 4096.0])
@pytest.mark.parametrize("scaled", [60.0, -60.0])
def test_scores_that_sum_without_loss(score, scaled, page):
    """Four products of few bits in a row of zeros: the score is exact in fp32
    and in every partial sum, and off by what it is raised by.  Beside that there
    are the roundings of the exponent: scale / ln 2, 1 / ln 2 and lse / ln 2 (U each
    of the scaled score, of which lse is the like), their difference (U of next to
    nothing), exp2 (2^-22) and the sum of one weight and 299 of zero."""
    B, n = 8, 300
    slots, d = requests(B, n, page)
    g = torch.Generator().manual_seed(int(score))
    d["q"], d["cache"] = torch.zeros(B, 1, 576), torch.zeros(slots, 576)
    at = torch.randint(0, n, (B,), generator=g)
    stride = -(-n // page) * page
    for b in range(B):
        dims = torch.randperm(576, generator=g)[:4]
        d["q"][b, 0, dims] = score / 64
        d["cache"][stride * b + at[b], dims] = 16
    d["q"], d["cache"] = d["q"].bfloat16().cuda(), d["cache"].bfloat16().cuda()
    scale = float(torch.tensor(scaled / score, dtype=torch.float32))
    value = float(d["q"][0, 0].double().sum()) * 16
    lse = torch.full((B, 1), scale * value, device="cuda")
    with C.plan_for(d) as plan:
        got = weigh(plan, d, lse, scale)[torch.arange(B), at.cuda()]
    want = scale * value - lse[0, 0].double()
    assert ((got.log() - want).abs() <= (RAISED + 3) * abs(scaled) * U + 2.0 ** -22).all()


def seekers(B, n, page, size, seed):
    """Requests whose row looks for one of its keys, to a score of size * 576 or so."""
    slots, d = requests(B, n, page)
    g = torch.Generator().manual_seed(seed)
    q, cache = torch.randn(B, 1, 576, generator=g), torch.randn(slots, 576, generator=g)
    at = torch.arange(B) * (-(-n // page) * page) + 7
    cache[at] += size * q[:, 0]
    for x in (q, cache):
        x[x.abs() < 2.0 ** -10] = 0      # (values that fp16 has, too)
    d["q"], d["cache"] = q.bfloat16().cuda(), cache.bfloat16().cuda()
    score = (d["q"][:, 0].double() * d["cache"][at].double()).sum(1)
    return d, score


@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("size", [0.3, 1.0])
def test_weights_of_a_row_add_up_to_one(size, page):
    """With the lse of mla_verify_attn_chunk.  Its scores are sums of the same
    products in the same order, lose the same and are raised alike; lse is off by
    the roundings of the maximum and of its sum with the logarithm, of ln 2 and of
    the product, the exponent by those of 1 / ln 2 and of the product: 6 U of
    lse.  Two exp2 and the logarithm, 2^-22 each, and some 16 additions one
    behind another on a side, U each."""
    d, _ = seekers(40, 300, page, size, int(10 * size))
    with C.plan_for(d) as plan:
        lse = C.attn(plan, d)[1]
        total = weigh(plan, d, lse, C.SCALE).sum(1)
    bound = (6 * lse[:, 0].double().abs() + 12 + 32) * U
    assert ((total - 1).abs() <= bound).all(), ((total - 1).abs() / bound).max()


@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("size", [0.3, 1.0])
def test_scores_of_ordinary_data(size, page):
    """The mean of a score's error, in weights with the lse of 64 bits and in the
    attention's lse, relative to the scores: neither without the raise nor with
    twice as much would it be within the bound."""
    d, score = seekers(64, 300, page, size, 100 + int(10 * size))
    keys = d["cache"].double()
    starts = torch.arange(64) * (-(-300 // page) * page)
    all_scores = torch.stack([keys[s:s + 300] @ q for s, q in zip(starts.tolist(), d["q"][:, 0].double())]) * C.SCALE
    exact = torch.logsumexp(all_scores, 1)
    with C.plan_for(d) as plan:
        lse = C.attn(plan, d)[1][:, 0].double()
        given = exact.float()
        got = weigh(plan, d, given[:, None].contiguous(), C.SCALE)[:, 7]
    off = got.log() - (score * C.SCALE - given.double())
    assert (off / (score * C.SCALE)).mean().abs() <= ORDINARY
    # (lse moves by the mean of its scores' errors, by their weights)
    weighed = (torch.softmax(all_scores, 1) * all_scores).sum(1)
    assert ((lse - exact) / weighed).mean().abs() <= ORDINARY
