"""GPU tests of the log probabilities of given tokens with entropy and
alternatives (sft_logprob), and of their gradient (sft_logprob_grad), against
their formulas in fp64."""
import math

import pytest
import torch

from sparse_full_weight_amd import _lib
from tests.rowwise import BF16, F32, MARK, U, Placed, close, gen, normal

pytestmark = pytest.mark.gpu

INF = math.inf
# around a group of 8, the steps of one wave, of 256 and of 1024 threads, and long ones
VOCABS = [1, 2, 3, 7, 8, 9, 63, 100, 511, 513, 2047, 2048, 2049, 8191, 8192, 8200, 16383, 16384, 32000, 50001]


def logits(N, V, seed, dtype=F32, std=2.5, masked=0.0):
    z = normal((N, V), std, seed)
    if masked:
        z[torch.rand((N, V), generator=gen(seed + 1)) < masked] = -INF
        z[:, seed % V] = 1.0
    return z.to(dtype)


def exact(z, target, scale, K):
    """M, L, logp, entropy, alternatives of rows of logits (fp64), and bounds for M, L, logp, entropy, any logp."""
    N, V = z.shape
    M = z.amax(1)
    d = (z - M[:, None]) * scale
    p = d.exp()
    total = p.sum(1)
    L = total.log()
    lp = d - L[:, None]
    p = p / total[:, None]
    plp = torch.where(p > 0, p * lp, 0.0)
    pd = torch.where(p > 0, p * d, 0.0).sum(1).abs()
    entropy = -plp.sum(1)
    # of a sum's term: two roundings of the exponent and one of scale * log2(e), relative to it; the power 2 U.  Of the sum:
    # one addition a logit of a thread (64 threads up to 2048 logits, else at least 256), one product a step, 6 steps and
    # 16 waves, the join
    terms = V / (64 if V <= 2048 else 256) * 1.125 + 40
    e_sum = (terms + 4) * U + 3 * U * pd
    e_L = e_sum + 4 * U * (L.abs() + scale * M.abs() * 2 ** -20) + 2 * U
    e_lp = e_L[:, None] + 3 * U * d.abs() + U * lp.abs()
    e_entropy = e_sum + (pd + 1) * (terms + 8) * U + 3 * U * (d * p).abs().nan_to_num().sum(1) + 4 * U * (L + pd) + 2 * U
    given = (target >= 0) & (target < V)
    at = target.clamp(0, V - 1).long()[:, None]
    logp = torch.where(given, lp.gather(1, at)[:, 0], 0.0)
    e_logp = torch.where(given, e_lp.gather(1, at)[:, 0], 0.0)
    value, index = torch.sort(z, dim=1, descending=True, stable=True)
    value, index = (torch.nn.functional.pad(x[:, :K], (0, max(0, K - V))) for x in (value, index))
    real = (torch.arange(K) < V) & (value > -INF)
    index_or_none = torch.where(real, index, -1).int()
    top = torch.where(real, lp.gather(1, index), -INF)
    e_top = torch.where(real, e_lp.gather(1, index), 0.0)
    return dict(M=M, L=L, logp=logp, entropy=entropy, index=index_or_none, top=top, lp=lp, p=p), dict(
        L=1.01 * e_L, logp=1.01 * e_logp, entropy=1.01 * e_entropy, top=1.01 * e_top)


def call(z, target, scale=1.0, K=0, entropy=True, pad=0, shift=0):
    N, V = z.shape
    on = Placed(z, pad, shift)
    out = dict(logp=torch.full((N + 1,), MARK, device="cuda"), stats=torch.full((N + 1, 2), MARK, device="cuda"),
               entropy=torch.full((N + 1,), MARK, device="cuda") if entropy else None,
               top_logp=torch.full((N + 1, K), MARK, device="cuda") if K else None,
               top_index=torch.full((N + 1, K), 77, dtype=torch.int32, device="cuda") if K else None)
    first = {k: None if x is None else x[:N] for k, x in out.items()}
    logp = first.pop("logp")
    _lib.sft_logprob(on.view, None if target is None else target.int().cuda(), None if target is None else logp,
                     scale=scale, **first)
    assert on.untouched() and torch.equal(on.view.cpu().nan_to_num(9.0), z.nan_to_num(9.0))
    for k, x in out.items():
        assert x is None or (x[N:] == (77 if k == "top_index" else MARK)).all(), k
    return {"logp": logp, **first}


def check(z, target, scale=1.0, K=0, entropy=True, **kw):
    got = call(z, target, scale, K, entropy, **kw)
    scale64 = float(torch.tensor(scale, dtype=F32))
    want, bound = exact(z.double(), target, scale64, K)
    what = f"{tuple(z.shape)}, {K} alternatives: "
    stats = got["stats"].cpu()
    assert torch.equal(stats[:, 0].double(), want["M"]), what + "M"
    close(stats[:, 1], want["L"], bound["L"], what + "L")
    close(got["logp"], want["logp"], bound["logp"], what + "logp")
    if entropy:
        close(got["entropy"], want["entropy"], bound["entropy"], what + "entropy")
    if K:
        assert torch.equal(got["top_index"].cpu(), want["index"]), what + "places of the alternatives"
        close(got["top_logp"], want["top"], bound["top"], what + "logp of the alternatives")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K", [0, 1, 5, 64])
def test_vocabularies(gpu_lib, dtype, K):
    for i, V in enumerate(VOCABS):
        N = [1, 2, 9][i % 3]
        z = logits(N, V, 10 * i, dtype, masked=[0.0, 0.5, 0.9][i % 3] if V > 4 else 0.0)
        # any given token; an allowed one, else its logp is -infinity, which is another test's
        target = z.float().argsort(1, descending=True)[:, [0, V // 50][i % 2]]
        check(z, target, [1.0, 0.7, 1.3][i % 3], K, i % 4 != 1, pad=[0, 0, 3, 8][i % 4], shift=[0, 1, 8][i % 3])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_rows_of_long_vocabularies(gpu_lib, dtype):
    # enough rows that a row is not given to 1024 threads
    z = logits(530, 20011, 5, dtype)
    check(z, torch.randint(0, 20011, (530,), generator=gen(3)), 1.0, 7)


@pytest.mark.parametrize("K", [32, 33, 51, 64])
@pytest.mark.parametrize("N,V", [(270, 9001), (3, 20000), (3, 40000)])
def test_many_alternatives(gpu_lib, N, V, K):
    # bf16: many logits are equal, the K-th among them
    z = logits(N, V, K, BF16)
    z[1] = 0.0
    z[1, 17::V // 40] = 1.0            # (40 or 41 of one value above all the others of another)
    check(z, torch.randint(0, V, (N,), generator=gen(K)), 1.0, K)


def test_rows_of_several_rounds_a_block(gpu_lib):
    # 256 threads a row, nine rounds of 32 logits a thread in eight blocks
    N, V, K = 520, 70001, 11
    z = torch.randn(N, V, device="cuda", generator=torch.Generator("cuda").manual_seed(4)) * 2.5
    target = torch.arange(N, device="cuda") * 130
    logp, index = torch.zeros(N, device="cuda"), torch.zeros(N, K, dtype=torch.int32, device="cuda")
    top = torch.zeros(N, K, device="cuda")
    _lib.sft_logprob(z, target.int(), logp, top_logp=top, top_index=index)
    lp = torch.log_softmax(z.double(), 1)
    want = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :K]
    assert torch.equal(index.long(), want)
    # as in exact(): the sum's additions, and roundings relative to differences from the largest logit (25 at most)
    bound = (V / 256 * 1.125 + 48 + 3 * 12 + 5 * 25) * U
    assert (logp.double() - lp.gather(1, target[:, None])[:, 0]).abs().max() <= bound
    assert (top.double() - lp.gather(1, want)).abs().max() <= bound


def test_targets_that_are_none_or_not_allowed(gpu_lib):
    z = logits(6, 1000, 4)
    z[2, 17] = -INF
    target = torch.tensor([-1, 1000, 17, 999, 2 ** 31 - 1, -2 ** 31])
    got = call(z, target)
    assert (got["logp"].cpu()[[0, 1, 4, 5]] == 0.0).all() and got["logp"][2] == -INF
    check(z[[0, 3]], target[[0, 3]])
    none = call(z, None, K=3)         # neither a target nor logp
    assert torch.equal(none["stats"], got["stats"]) and torch.equal(none["entropy"], got["entropy"])


@pytest.mark.parametrize("V", [5, 100, 2049, 40000])
def test_rows_with_few_allowed_tokens(gpu_lib, V):
    z = torch.full((5, V), -INF)
    z[1, V - 1] = -3.0
    z[2, 0], z[2, V // 2] = 1.0, 1.0
    z[3] = float(torch.finfo(F32).min)           # the type's lowest value everywhere: all alike
    z[4] = float(torch.finfo(F32).min)           # the same as a mask
    z[4, V // 3], z[4, 1] = 0.5, 2.0
    target = torch.tensor([0, V - 1, V // 2, 3, V // 3])
    got = call(z, target, 1.7, 3)
    host = {k: v.cpu() for k, v in got.items()}
    assert host["stats"][0].tolist() == [-INF, -INF] and host["logp"][0] == -INF and host["entropy"][0] == 0.0
    assert host["top_index"][0].tolist() == [-1] * 3 and host["top_logp"][0].tolist() == [-INF] * 3
    # a single term 2^off, off what M * log2(e) was rounded by (2 U for the power, 1 U each for the logarithm, for the
    # quotient and product with ln(2), and for off itself); its logarithm less ln(2) * off, limited to 0 and above
    assert -5 * U <= host["logp"][1] <= 0.0 and 0.0 <= host["entropy"][1] <= 5 * U
    assert host["top_index"][1].tolist() == [V - 1, -1, -1]
    assert host["top_index"][2].tolist() == [0, V // 2, -1] and abs(host["logp"][2] + math.log(2)) <= 4 * U
    assert abs(host["entropy"][2] - math.log(2)) <= 4 * U
    terms = V / 64 + 60
    for k in ("logp", "entropy"):
        want = -math.log(V) if k == "logp" else math.log(V)
        assert abs(host[k][3] - want) <= (terms + 4 * abs(want)) * U
    assert host["top_index"][3].tolist() == [0, 1, 2]
    assert host["top_index"][4].tolist() == torch.sort(z[4], descending=True, stable=True)[1][:3].tolist()
    z[4] = torch.where(z[4] < -1e30, -INF, z[4])         # the same as if they were not allowed
    assert torch.equal(call(z, target, 1.7)["logp"][4], got["logp"][4])


@pytest.mark.parametrize("V", [100, 5000, 40000])
def test_rows_that_are_not_finite(gpu_lib, V):
    z = logits(7, V, V)
    z[1, V // 2] = INF
    z[2, 0] = float("nan")
    z[3] = float("nan")
    z[4] = z[0]
    z[4, V - 1] = float("nan")
    z[5, :] = -INF
    z[5, 3] = float("nan")
    bad = [1, 2, 3, 4, 5]
    # a bf16 pattern that is a signalling NaN
    for dtype in (F32, BF16):
        x = z.to(dtype)
        if dtype == BF16:
            x.view(torch.int16)[2, 0] = 0x7f81
        got = {k: v.cpu() for k, v in call(x, torch.arange(7) + 1, 1.0, 4).items()}
        for k in ("logp", "entropy", "stats"):
            assert got[k][bad].isnan().all(), k
            assert not got[k][[0, 6]].isnan().any(), k
        assert got["top_index"][1, 0] == V // 2 and got["top_index"][3].tolist() == [-1] * 4
        rank = x.float().nan_to_num(-INF, posinf=INF, neginf=-INF)
        for row in (1, 2, 4):
            want = torch.sort(rank[row], descending=True, stable=True)[1][:4]
            assert got["top_index"][row].tolist() == want.tolist()
        assert got["top_logp"][[1, 2, 4]].isnan().all()
        stats = torch.zeros(7, 2)
        stats[:] = got["stats"]
        dz = torch.zeros(7, V, device="cuda", dtype=dtype)
        _lib.sft_logprob_grad(x.cuda(), (torch.arange(7) + 1).int().cuda(), stats.cuda(), torch.ones(7, device="cuda"), dz)
        assert dz[bad].isnan().all() and not dz[[0, 6]].isnan().any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,N", [(300, 3), (700, 2), (5000, 3), (20000, 2), (40000, 2), (300000, 2), (20000, 520)])
def test_alternatives_of_equal_logits(gpu_lib, dtype, V, N):
    # rows of few different values; of one value; ascending, descending; the two zeros; all large ones with few threads
    z = torch.round(normal((N, V), 1.2, V))
    z[0] = 0.25
    z[1, : V // 2] = torch.where(z[1, : V // 2] == 0, -0.0, z[1, : V // 2])
    check(z.to(dtype), torch.zeros(N, dtype=torch.int64), 1.0, 20)
    line = torch.arange(V).float() / V * 10
    z[0], z[1] = line, line.flip(0)
    check(z.to(dtype), torch.zeros(N, dtype=torch.int64), 1.0, 33)
    at = torch.arange(V)
    z[0] = torch.where(at % 2048 < 512, 3.0 + line, -line)
    z[1] = torch.where(at % 8192 < 512, 3.0 + normal((V,), 0.1, 5), -line)
    check(z.to(dtype), torch.zeros(N, dtype=torch.int64), 1.0, 64)


def test_far_logits(gpu_lib):
    # a shift of all logits changes nothing but M; huge spreads; a large scale
    z = logits(4, 3000, 9)
    z[1] += 1000.0
    z[2] *= 1e4
    z[3] = z[3] * 1e30 + 1e38
    check(z, torch.tensor([5, 6, 7, 8]), 1.0, 4)
    check(z[:3], torch.tensor([5, 6, 7]), 50.0, 4)


def test_no_rows_and_more_rows_than_workgroups(gpu_lib):
    none = torch.empty(0, device="cuda")
    _lib.sft_logprob(torch.empty(0, 10, device="cuda"), none.int(), none)
    _lib.sft_logprob_grad(torch.empty(0, 10, device="cuda"), none.int(), torch.empty(0, 2, device="cuda"), none,
                          torch.empty(0, 10, device="cuda"))
    N = (1 << 21) + 5
    z = torch.randn(N, 3, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    target = torch.arange(N, device="cuda").remainder(3).int()
    logp, top = torch.zeros(N, device="cuda"), torch.zeros(N, 1, dtype=torch.int32, device="cuda")
    _lib.sft_logprob(z, target, logp, top_index=top)
    want = torch.log_softmax(z.double(), 1).gather(1, target.long()[:, None])[:, 0]
    # three terms: exponents, powers, two additions, the logarithm, differences of up to 10
    assert ((logp.double() - want).abs() <= 60 * U).all()
    assert torch.equal(top[:, 0].long(), z.argmax(1))


def test_offsets_past_32_bits(gpu_lib):
    N, V, ld = 5, 777, 300_000_001       # rows 1.2 GB apart
    z = logits(N, V, 6)
    big, out = (torch.empty(N * ld, device="cuda").view(N, ld)[:, :V] for _ in range(2))
    big.copy_(z)
    target = torch.arange(N)
    logp, stats = torch.zeros(N, device="cuda"), torch.zeros(N, 2, device="cuda")
    _lib.sft_logprob(big, target.int().cuda(), logp, stats=stats)
    want, bound = exact(z.double(), target, 1.0, 0)
    close(logp, want["logp"], bound["logp"], "logp")
    _lib.sft_logprob_grad(big, target.int().cuda(), stats, torch.ones(N, device="cuda"), out)
    wantd, boundd = gradient(z.double(), target, stats.cpu().double(), torch.ones(N), None, None, 1.0)
    close(out, wantd, boundd, "dZ")


# ------------------------------------------------------------------ gradient
def gradient(z, target, stats, dlogp, entropy, dentropy, scale):
    """dZ in fp64 from the statistics as they are, and a bound."""
    N, V = z.shape
    d = (z - stats[:, :1]) * scale
    lp = d - stats[:, 1:]
    p = lp.exp()
    given = (target >= 0) & (target < V)
    own = (dlogp.double() * given if dlogp is not None else torch.zeros(N, dtype=torch.float64))[:, None]
    de = torch.zeros(N, 1, dtype=torch.float64) if dentropy is None else dentropy.double()[:, None]
    H = torch.zeros(N, 1, dtype=torch.float64) if entropy is None else entropy.double()[:, None]
    # p = 0 counts as 0
    finite = lp.clamp_min(-1e4)
    weight = own + de * (finite + H)
    dz = -p * weight
    # the exponent's difference, product and sum (and scale * log2(e), L * log2(e)), the power; the weight's parts
    e_p = 4 * U * (finite.abs() + stats[:, 1:].abs()) + 3 * U
    e_w = 4 * U * (own.abs() + (de * H).abs() + 2 * (de * finite).abs() + (de * stats[:, 1:]).abs())
    bound = p * (weight.abs() * e_p + e_w) + 3 * U * dz.abs()
    at = target.clamp(0, V - 1).long()[:, None]
    dz.scatter_add_(1, at, own)
    dz, bound = dz * scale, bound * scale
    return dz, 1.01 * bound + 2 * U * dz.abs() + 3 * U * scale * own.abs() * (dz != 0) * (torch.arange(V) == at) + 1e-37


def check_gradient(N, V, dtype, out_type, scale=1.0, with_logp=True, with_entropy=False, masked=0.0, pad=0, shift=0,
                   inplace=False, seed=0):
    z = logits(N, V, seed, dtype, masked=masked)
    target = z.float().argsort(1, descending=True)[:, V // 50]
    target[::4] = -1
    target = target.int()
    scale = float(torch.tensor(scale, dtype=F32))
    want, _ = exact(z.double(), target, scale, 0)
    stats = torch.stack([want["M"], want["L"]], 1).float()
    H = want["entropy"].float() if with_entropy else None
    dlogp = normal((N,), 1.0, seed + 3) if with_logp else None
    dH = normal((N,), 1.0, seed + 4) if with_entropy else None
    on = Placed(z, pad, shift)
    out = on if inplace else Placed(torch.full((N, V), 3.0, dtype=out_type), 2 * pad, shift)

    def up(x):
        return None if x is None else x.cuda()

    _lib.sft_logprob_grad(on.view, up(target) if with_logp else None, stats.cuda(), up(dlogp), out.view, scale=scale,
                          entropy=up(H), dentropy=up(dH))
    dz, bound = gradient(z.double(), target, stats.double(), dlogp, H, dH, scale)
    close(out.view, dz, bound, f"dZ of {N} x {V}")
    assert on.untouched() and out.untouched()
    assert inplace or torch.equal(on.view.cpu(), z)
    if with_logp and not with_entropy:
        assert (out.view.cpu()[::4] == 0).all()


@pytest.mark.parametrize("dtype,out_type", [(F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("parts", ["logp", "entropy", "both"])
def test_gradient(gpu_lib, parts, dtype, out_type):
    for i, V in enumerate(VOCABS):
        check_gradient([1, 2, 9][i % 3], V, dtype, out_type, [1.0, 0.7, 1.3][i % 3], parts != "entropy", parts != "logp",
                       masked=0.4 if i % 2 and V > 4 else 0.0, pad=[0, 0, 3, 8][i % 4], shift=[0, 1, 8][i % 3],
                       inplace=dtype == out_type and i % 3 == 1, seed=i)


def test_gradient_of_rows_that_count_nothing(gpu_lib):
    # zero derivatives, no given token, no allowed token: zeros, whatever the logits are
    z = logits(4, 9000, 3)
    z[0, 5], z[1, 5], z[2] = float("nan"), INF, -INF
    stats = torch.tensor([[1.0, 2.0], [1.0, 2.0], [-INF, -INF], [z[3].max(), 3.0]])
    dz = torch.full((4, 9000), MARK, device="cuda")
    dlogp = torch.tensor([0.0, 1.0, 1.0, 0.0])
    _lib.sft_logprob_grad(z.cuda(), torch.tensor([3, -1, 4, 4]).int().cuda(), stats.cuda(), dlogp.cuda(), dz)
    assert (dz == 0).all()


def test_gradient_is_the_derivative(gpu_lib):
    # central differences of the fp64 loss along random directions; a loss of both parts with ignored rows and a mask
    N, V, scale = 5, 400, 1.25
    z = logits(N, V, 8, masked=0.3)
    target = z.argsort(1, descending=True)[:, 3]
    target[1] = -1
    dlogp, dH = normal((N,), 1.0, 1), normal((N,), 1.0, 2)
    stats, H, logp = torch.empty(N, 2, device="cuda"), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    on, dz = z.cuda(), torch.empty(N, V, device="cuda")
    _lib.sft_logprob(on, target.int().cuda(), logp, scale=scale, stats=stats, entropy=H)
    _lib.sft_logprob_grad(on, target.int().cuda(), stats, dlogp.cuda(), dz, scale=scale, entropy=H, dentropy=dH.cuda())

    def loss(x):
        got, _ = exact(x, target, scale, 0)
        return float((got["logp"] * dlogp).sum() + (got["entropy"] * dH).sum())

    for seed in range(4):
        v = torch.where(z > -INF, normal((N, V), 1.0, 20 + seed), 0.0).double()
        slope = (loss(z.double() + 1e-5 * v) - loss(z.double() - 1e-5 * v)) / 2e-5
        got = float((dz.cpu().double() * v).sum())
        size = float((dz.cpu().double() * v).abs().sum())
        # the difference's own error is about 1e-9; statistics in fp32 count some ten U
        assert abs(got - slope) <= 1e-5 * size + 1e-7


def test_the_same_results_every_time(gpu_lib):
    z = logits(600, 30000, 1, BF16).cuda()
    target = torch.arange(600, device="cuda").int()
    first = None
    for _ in range(3):
        out = [torch.empty(600, device="cuda"), torch.empty(600, 2, device="cuda"), torch.empty(600, device="cuda"),
               torch.empty(600, 20, device="cuda"), torch.empty(600, 20, dtype=torch.int32, device="cuda")]
        _lib.sft_logprob(z, target, out[0], stats=out[1], entropy=out[2], top_logp=out[3], top_index=out[4])
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [300, 700, 5000, 20000, 40000])
def test_masks_of_large_finite_values(gpu_lib, V, dtype):
    # a padded vocabulary's end, all but three tokens, half of them at random, and a whole row masked by a finite value
    target = torch.tensor([5, V // 2, V // 3, 7])
    for i, mask in enumerate([-1e5, -3e7, -2e9, -1e10, -3e10, -7e12, -1e18, -1e21, -5e24, -1e30, -3e30, -7e33, -1e37]):
        z = logits(4, V, V + i)
        z[0, V - V // 3:] = mask
        z[1] = mask
        z[1, V // 2], z[1, 0], z[1, V - 1] = 0.5, -2.0, 3.25
        z[2, (torch.rand(V, generator=gen(i)) < 0.5) & (torch.arange(V) != V // 3)] = mask
        z[3] = mask
        z = z.to(dtype)
        check(z, target, [1.0, 0.7, 1.9][i % 3], 3)
        got = call(z, target, [1.0, 0.7, 1.9][i % 3])
        # the row of one value: V terms of 1, their sum as in exact(), the logarithm, a difference of 0
        L, H, logp = (float(x) for x in (got["stats"][3, 1], got["entropy"][3], got["logp"][3]))
        e = (V / (64 if V <= 2048 else 256) * 1.125 + 46 + 4 * math.log(V)) * U
        assert abs(L - math.log(V)) <= e and abs(H - math.log(V)) <= e and abs(logp + math.log(V)) <= e
        # and what is masked gets no gradient, what is given its own
        dz = torch.full(z.shape, MARK, device="cuda")
        _lib.sft_logprob_grad(z.float().cuda(), target.int().cuda(), got["stats"], torch.ones(4, device="cuda"), dz)
        dz = dz.cpu()
        assert (dz[:3][z[:3].float() < -5e4] == 0.0).all()
        own = (z[torch.arange(4), target].double() - z.amax(1).double() - got["stats"][:, 1].double().cpu()).exp()
        assert ((dz[torch.arange(4), target].double() - (1.0 - own)).abs() <= 80 * U).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logits_far_from_zero(gpu_lib, dtype):
    # all of a row around a large value: as exact as differences of such logits are, with products with the scale near
    # and far past what fp32 holds to a unit
    for V in (300, 5000, 20000):
        for i, far in enumerate([3e6, 1e8, -4e9, 2e12, -1e17, 6e25, -1e36]):
            z = normal((3, V), abs(far) * 2.0 ** -20, V + i) + far
            z = z.to(dtype)
            d = z.double() - z.double().amax(1, keepdim=True)
            for bits in (18, 25, 40):
                scale = float(torch.tensor(2.0 ** bits / abs(far), dtype=F32))
                got = call(z, torch.tensor([0, 1, V - 1]), scale)
                lp = d * scale
                p, L = lp.exp(), lp.exp().sum(1).log()
                pd = (torch.where(p > 0, p * lp, 0.0).sum(1) / p.sum(1)).abs()
                logp = lp[torch.arange(3), torch.tensor([0, 1, V - 1])] - L
                # additions as in exact(), three roundings of an exponent, the logarithm and what is taken off it
                e = (V / (64 if V <= 2048 else 256) * 1.125 + 46 + 3 * pd + 4 * L) * U
                assert ((got["stats"][:, 1].double().cpu() - L).abs() <= e).all(), (far, bits)
                assert ((got["logp"].double().cpu() - logp).abs() <= e + 4 * U * logp.abs()).all(), (far, bits)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [300, 500, 1001, 2048, 2049, 5000, 16383, 16384, 20000, 33001, 50001, 70001])
def test_a_row_is_the_same_in_any_batch_and_at_any_address(gpu_lib, V, dtype):
    # one row alone, as the last of more rows than the device has CUs, at other addresses, with and without the optional
    # outputs; around a value far from zero, too
    z = torch.empty(600, V, dtype=dtype, device="cuda")
    z.copy_(torch.randn(600, V, device="cuda", generator=torch.Generator("cuda").manual_seed(V)) * 2.5)
    for far in (0.0, -3e7):
        row = normal((1, V), 2.5, V, dtype).cuda()
        if far:
            row = (row.float() * 3e3 + far).to(dtype)
        z[599] = z[7] = row[0]
        target = torch.arange(600, device="cuda").int()
        target[599] = target[7] = V // 3
        want = None
        for at in (None, 0, 1, 3, 8, 16, 31, 57):
            if at is None:
                rows, given = z, target
            else:
                room = torch.zeros(V + 64, dtype=dtype, device="cuda")
                rows, given = room[at:at + V].view(1, V), target[7:8].contiguous()
                rows.copy_(row)
            for K in (0, 5):
                N = rows.shape[0]
                logp, H = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
                stats = torch.empty(N, 2, device="cuda")
                top, index = torch.empty(N, 5, device="cuda"), torch.empty(N, 5, dtype=torch.int32, device="cuda")
                more = dict(top_logp=top, top_index=index) if K else {}
                _lib.sft_logprob(rows, given, logp, stats=stats, entropy=H, **more)
                only = torch.empty(N, device="cuda")
                _lib.sft_logprob(rows, given, only)
                assert torch.equal(only, logp)
                dz = torch.empty_like(rows) if at is None else torch.empty(V + 64, dtype=dtype,
                                                                           device="cuda")[at:at + V].view(1, V)
                _lib.sft_logprob_grad(rows, given, stats, torch.ones(N, device="cuda"), dz, entropy=H,
                                      dentropy=torch.ones(N, device="cuda"))
                for i in ((7, 599) if at is None else (0,)):
                    got = [x[i].clone() for x in (logp, stats, H, dz)]
                    want = want or got
                    assert all(torch.equal(a, b) for a, b in zip(want, got)), (far, at, K, i)
                    if K:
                        best = [x[i].clone() for x in (top, index)]
                        want = want + best if len(want) == 4 else want
                        assert all(torch.equal(a, b) for a, b in zip(want[4:], best)), (far, at, K, i)


@pytest.mark.parametrize("N,V", [(8300, 300), (16500, 77), (8300, 700)])
def test_more_short_rows_than_waves(gpu_lib, N, V):
    # a wave a row, past the rows that the device holds at a time
    z = logits(N, V, V, BF16)
    check(z, torch.randint(0, V, (N,), generator=gen(N)), 1.0, 5)
    for dtype, out_type in ((F32, F32), (BF16, BF16), (F32, BF16)):
        check_gradient(N, V, dtype, out_type, with_entropy=dtype == F32, seed=V)


@pytest.mark.parametrize("N,dtype", [(1, F32), (300, BF16)])
def test_very_long_rows(gpu_lib, N, dtype):
    # 2^28 logits and some in one row by 1024 threads; 2^22 and some in each of more rows than CUs
    V, K = ((1 << 28) + 13, 9) if N == 1 else ((1 << 22) + 5, 9)
    z = torch.empty(N, V, dtype=dtype, device="cuda")
    for i in range(N):
        z[i] = torch.randn(V, device="cuda", generator=torch.Generator("cuda").manual_seed(i)) * 2.0
    best = torch.randperm(V, device="cuda", generator=torch.Generator("cuda").manual_seed(77))[:K]
    best[0], best[1] = V - 1, 0                     # the tail, and the first logit
    z[:, best] = torch.arange(30, 30 - K, -1, device="cuda").to(dtype)
    z[:, best[3]] = z[0, best[2]]                   # two alike
    target = torch.full((N,), V // 2 + 1, dtype=torch.int32, device="cuda")
    logp, H, stats = torch.empty(N, device="cuda"), torch.empty(N, device="cuda"), torch.empty(N, 2, device="cuda")
    top, index = torch.empty(N, K, device="cuda"), torch.empty(N, K, dtype=torch.int32, device="cuda")
    _lib.sft_logprob(z, target, logp, stats=stats, entropy=H, top_logp=top, top_index=index)
    order = best.clone()
    order[2:4] = best[2:4].sort().values
    assert (index.long() == order).all()
    for i in range(0, N, 60):
        total = along = 0.0
        for part in z[i].split(1 << 25):
            d = part.double() - 30.0
            total, along = total + d.exp().sum(), along + (d.exp() * d).sum()
        L = total.log()
        # additions as in exact(), differences of at most 45 from the largest logit
        e = (V / 256 * 1.125 + 50) * U + 3 * U * 45
        assert abs(stats[i, 0] - 30.0) == 0 and abs(stats[i, 1].double() - L) <= e
        assert abs(H[i].double() - (L - along / total)) <= 2 * e * (1 + abs(along / total))
        lp = z[i, V // 2 + 1].double() - 30.0 - L
        assert abs(logp[i].double() - lp) <= e + 4 * U * abs(lp)
        assert ((top[i].double() - (z[i, order].double() - 30.0 - L)).abs() <= e + 4 * U * 45).all()
