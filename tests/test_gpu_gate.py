"""GPU parity of the expert routing (the same experts as a choice in 64 bits,
weights within their rounding) and of its gradient, against oracle.routing.

Tolerances, with u = 2^-24 and D the spread of the finite logits that a row's
weights are made of: exp is within 2u of its argument's, whose subtraction
adds D u; a sum over E terms adds at most (ceil(E / 32) + 5) u; quotient and
scale one u each.  Numerator and denominator then give (2D + E/32 + 13) u, and
the sigmoid's own quotient 4u more.  A gradient's terms carry that error twice
(the share and the mean's shares) and 12u of their own sums and products, all
relative to the sum of their magnitudes; a BF16 result half a step more.
"""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_05_b200 import binding as dg
from oracle import routing

pytestmark = pytest.mark.gpu
INF = float("inf")
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dg.get_device_error()


def _f64(t):
    return t.double().cpu().numpy()


def _slack(l, score):
    """Relative error of a weight per row, in units of U (see above)."""
    finite = np.where(np.isfinite(l), l, np.nan)
    with np.errstate(all="ignore"):
        import warnings
        with warnings.catch_warnings():
            warnings.simplefilter("ignore")
            spread = np.nan_to_num(np.nanmax(finite, axis=1) - np.nanmin(finite, axis=1))
    # terms further than 110 below the largest are zero in both
    return 2 * np.minimum(spread, 110.0) + -(-l.shape[1] // 32) + 17


def check_gate(logits, topk, bias=None, **kw):
    logits = logits.cuda()
    bias = None if bias is None else bias.float().cuda()
    ids, w = dg.moe_gate(logits, topk, bias, **kw)
    torch.cuda.synchronize()
    l = _f64(logits)
    ref_ids, ref_w, bad = routing.moe_gate(l, topk, None if bias is None else _f64(bias), **kw)
    assert dg.get_device_error() == (dg.DG_DEVERR_BAD_LOGIT if bad.any() else 0)
    got = ids.cpu().numpy()
    assert np.array_equal(got, ref_ids), np.argwhere(got != ref_ids)[:4]
    tol = U * _slack(l, kw.get("score", "softmax"))[:, None] * np.abs(ref_w) + 2.0 ** -126
    err = np.abs(_f64(w) - ref_w)
    assert (err <= tol).all(), (err / np.maximum(np.abs(ref_w), 1e-300)).max() / U
    return ids, w


def _rand(T, E, seed, dtype=torch.float32, sigma=1.5):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(sigma * rng.standard_normal((T, E))).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (129, 32, 8), (64, 33, 4), (70, 60, 6),
                                      (33, 64, 1), (40, 100, 32), (200, 256, 8), (9, 257, 5), (17, 512, 16),
                                      (6, 1000, 7), (12, 1024, 32)])
def test_plain_choice(T, E, topk, score, dtype):
    l = _rand(T, E, T * 1000 + E, dtype)
    check_gate(l, topk, score=score)
    check_gate(l, topk, score=score, renormalize=True, scale=2.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,topk", [(1, 8, 2), (300, 64, 6), (50, 130, 9), (400, 256, 8), (20, 1024, 32)])
def test_biased_choice(T, E, topk, score, dtype):
    l = _rand(T, E, T + E, dtype)
    b = 0.05 * _rand(1, E, 5)[0]
    check_gate(l, topk, b, score=score, renormalize=True)
    check_gate(l, topk, torch.zeros(E), score=score)      # equal logits tie exactly: the lowest index


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,topk,n_group,topk_group", [
    (300, 256, 8, 8, 4), (40, 64, 4, 4, 2), (100, 160, 6, 8, 3), (50, 60, 4, 6, 2), (30, 256, 8, 32, 3),
    (20, 1024, 16, 16, 5), (25, 66, 3, 3, 1), (30, 16, 2, 8, 8), (10, 96, 8, 2, 1), (64, 512, 8, 4, 2),
    (21, 1020, 12, 17, 4), (15, 1000, 8, 8, 3), (33, 384, 8, 8, 2), (40, 100, 8, 5, 2), (9, 1024, 32, 32, 3),
    (13, 93, 7, 31, 9), (11, 992, 8, 31, 6), (50, 36, 12, 6, 3), (8, 1024, 8, 2, 1)])
def test_groups(T, E, topk, n_group, topk_group, score, biased, group_top):
    """Groups whose experts are whole runs of a lane, groups that fill their lanes
    in part, and (17 and 31 groups of many) groups that share lanes."""
    b = 0.05 * _rand(1, E, 9)[0] if biased else None
    check_gate(_rand(T, E, T + 7 * E), topk, b, score=score, n_group=n_group, topk_group=topk_group,
               group_top=group_top, renormalize=True, scale=2.5)
    check_gate(_rand(T, E, T + 8 * E, torch.bfloat16), topk, b, score=score, n_group=n_group, topk_group=topk_group,
               group_top=group_top)


@pytest.mark.parametrize("n_group", [2, 3, 4, 5, 7, 8, 12, 16, 17, 24, 32])
def test_groups_of_every_size(n_group):
    """Every group size up to 34 and those around the lanes' runs beyond it: groups that
    fill their lanes, that leave the last lane in part, and that leave lanes empty."""
    sizes = [g for g in [*range(1, 35), 42, 52, 56, 60, 112, 120, 127, 128, 224, 240, 496] if g * n_group <= 1024]
    for gsize in sizes:
        E, topk_group = gsize * n_group, (n_group + 1) // 2
        b = 0.05 * _rand(1, E, gsize)[0]
        few, many = min(4, topk_group * gsize), min(32, topk_group * gsize)
        check_gate(_rand(4, E, E), few, b, score="sigmoid", n_group=n_group, topk_group=topk_group,
                   group_top=min(2, gsize))
        check_gate(_rand(4, E, E + 1, torch.bfloat16), many, n_group=n_group, topk_group=topk_group)


def test_large_batch_and_ragged_tail():
    check_gate(_rand(20001, 64, 3, torch.bfloat16), 6, score="softmax", renormalize=True)
    check_gate(_rand(4099, 256, 4), 8, 0.05 * _rand(1, 256, 6)[0], score="sigmoid", n_group=8, topk_group=4,
               group_top=2, renormalize=True, scale=2.5)


def test_scores_that_32_bits_cannot_tell_apart():
    """Biases that bring every expert's score to nearly the same value: the
    order is decided by differences of about 2^-26, far below what the scores'
    32-bit values resolve, and the kernel still chooses as in 64 bits."""
    T, E = 64, 256
    for score in ("sigmoid", "softmax"):
        l = _rand(1, E, 21).repeat(T, 1)
        s = routing.scores(_f64(l[:1]), score)[0]
        b = torch.from_numpy((1.0 - s).astype(np.float32))
        check_gate(l, 8, b, score=score, renormalize=True)
        check_gate(l, 8, b, score=score, n_group=8, topk_group=4, group_top=2)
        check_gate(l, 8, b, score=score, n_group=4, topk_group=1, group_top=1)
    # a saturated sigmoid: every score is 1 in 32 bits
    l = 20.0 + _rand(50, 96, 22).abs() / 64
    check_gate(l, 8, torch.zeros(96), score="sigmoid")


@pytest.mark.parametrize("E,n_group,topk_group,topk", [(64, 4, 2, 4), (64, 1, 1, 6), (32, 4, 2, 8), (128, 1, 1, 8),
                                                       (128, 8, 4, 4), (60, 6, 2, 3), (100, 5, 2, 8), (256, 8, 4, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_neighbouring_tokens_that_take_different_ways(E, n_group, topk_group, topk, score):
    """Tokens that need 64 bits, tokens that do not, equal logits, padding and
    rows that are not numbers side by side: two tokens may share a warp."""
    T = 301
    l = _rand(1, E, 23).repeat(T, 1)
    s = routing.scores(_f64(l[:1]), score)[0]
    b = torch.from_numpy((1.0 - s).astype(np.float32))
    rng = np.random.default_rng(E)
    kind = torch.from_numpy(rng.integers(0, 6, T))
    other = _rand(T, E, 24)
    l[kind == 1] = other[kind == 1]
    l[kind == 2] = -INF
    l[kind == 3] = 0.25
    l[kind == 4, ::2] = -INF
    l[(kind == 5).nonzero()[:3, 0], E - 1] = float("nan")
    for group_top in (1, 2):
        for bias in (b, None, torch.zeros(E)):
            check_gate(l, topk, bias, score=score, renormalize=True, n_group=n_group, topk_group=topk_group,
                       group_top=group_top)


def test_masks_and_padding():
    T, E, topk = 40, 64, 6
    l = _rand(T, E, 31)
    l[torch.rand(T, E, generator=torch.Generator().manual_seed(1)) < 0.9] = -INF   # fewer experts than slots
    l[3] = -INF                                                                  # a padded token
    l[4, 1:] = -INF                                                              # one expert left
    l[5] = torch.finfo(torch.float32).min                                        # the lowest finite value: not masked
    l[6, ::2] = torch.finfo(torch.float32).min
    l[7] = -0.0
    l[7, ::3] = 0.0                                                              # -0 and 0 tie
    b = torch.zeros(E)
    b[10] = -INF
    for kw in (dict(score="softmax"), dict(score="sigmoid"), dict(score="softmax", renormalize=True),
               dict(score="sigmoid", renormalize=True), dict(score="sigmoid", renormalize=True, n_group=8, topk_group=2),
               dict(score="softmax", n_group=8, topk_group=3, group_top=2)):
        ids, w = check_gate(l, topk, **kw)
        assert (ids[3] == -1).all() and (w[3] == 0).all()
        ids, _ = check_gate(l, topk, b, **kw)
        assert not (ids == 10).any()
    ids, w = dg.moe_gate(torch.full((3, E), -INF, device="cuda"), topk, score="sigmoid", renormalize=True)
    assert (ids == -1).all() and (w == 0).all()


@pytest.mark.parametrize("T,E,topk,n_group,topk_group", [
    (5, 20, 6, 1, 1), (7, 24, 10, 4, 2), (9, 33, 20, 3, 2), (6, 60, 6, 6, 2), (12, 64, 8, 1, 1), (8, 256, 8, 8, 4),
    (5, 160, 6, 8, 3), (4, 1000, 16, 8, 3), (4, 1020, 12, 17, 4), (6, 32, 32, 1, 1), (11, 100, 32, 5, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_of_any_size(T, E, topk, n_group, topk_group, score):
    """Biases that push experts out of the choice without masking them (the type's lowest
    value, -1e9, -1e4), for fewer and for more experts than leave the slots filled, and
    biases in whose last place every score is lost."""
    lowest = torch.finfo(torch.float32).min
    rng = np.random.default_rng(E)
    l = _rand(T, E, E + 3)
    l[1, ::3] = -INF
    kw = dict(score=score, n_group=n_group, topk_group=topk_group)
    for value in (lowest, -1e9, -1e4, -2.0 ** 24, lowest / 2, 2.0 ** 23, 3e38):
        for share in (0.1, 0.5, 0.9, 1.0):
            b = 0.05 * _rand(1, E, 5)[0]
            b[torch.from_numpy(rng.random(E) < share)] = value
            for group_top in {1, min(2, E // n_group)}:
                check_gate(l, topk, b, group_top=group_top, **kw)
    b = torch.tensor([lowest, -lowest, 0.0, -INF])[torch.from_numpy(rng.integers(0, 4, E))]
    check_gate(l, topk, b, group_top=min(2, E // n_group), **kw)


@pytest.mark.parametrize("value", [torch.finfo(torch.float32).min, -1e9, -300.0, 1e9, torch.finfo(torch.float32).max, -INF])
@pytest.mark.parametrize("E,n_group,topk_group,topk", [(256, 8, 4, 8), (64, 8, 3, 6), (60, 6, 2, 4), (8, 8, 4, 2),
                                                       (1020, 17, 5, 12)])
def test_whole_groups_with_the_same_large_bias(E, n_group, topk_group, topk, value):
    """Groups that a bias pushes out (or in) as a whole, all but for one expert, or with one
    term of each sign: for a few groups, so that enough others are left, and for all but one."""
    gsize = E // n_group
    l = _rand(60, E, E + 5)
    l[50:] = l[:1]                                       # (and rows next to one another in value)
    l[52:, ::2] += 2.0 ** -20
    for score in ("softmax", "sigmoid"):
        for pushed in (1, n_group - topk_group, n_group - 1):
            for keep in (0, 1, 2):
                b = 0.05 * _rand(1, E, 9)[0]
                for g in range(pushed):
                    b[g * gsize + keep:(g + 1) * gsize] = value
                    if keep == 2 and gsize > 2 and abs(value) < 1e30:
                        b[g * gsize] = -value
                for group_top in {1, min(2, gsize)}:
                    check_gate(l, topk, b, score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)


@pytest.mark.parametrize("what", [float("nan"), INF])
def test_rows_that_are_not_numbers_are_not_routed(what):
    l = _rand(10, 60, 41)
    l[4, 59] = what
    l[9, 0] = what
    for score in ("softmax", "sigmoid"):
        ids, w = check_gate(l, 4, score=score, renormalize=True)
        assert (ids[4] == -1).all() and (w[9] == 0).all() and (ids[5] >= 0).all()
    b = torch.zeros(60)
    b[7] = what
    ids, _ = check_gate(_rand(10, 60, 42), 4, b, score="sigmoid")
    assert (ids == -1).all()


def test_extreme_logits():
    E = 48
    l = torch.linspace(-3e38, 3e38, 32 * E).reshape(32, E)
    check_gate(l, 8, score="softmax", renormalize=True)
    check_gate(l, 8, score="sigmoid", renormalize=True)
    l = -200.0 - _rand(32, E, 51).abs()           # every sigmoid is zero in 32 bits
    check_gate(l, 8, score="sigmoid", renormalize=True, scale=2.5)
    check_gate(200.0 + _rand(32, E, 52), 8, score="sigmoid", renormalize=True)
    check_gate(l, 8, torch.zeros(E), score="sigmoid")


@pytest.mark.parametrize("best", [-0.5, -30.0, -59.0, -61.0, 0.0, 3.0])
def test_sigmoid_shares_far_below_the_best(best):
    """Chosen logits down to 85 (and, where the share is still a normal number, 120) below
    the best: their shares are e^-36 and less, and not zero."""
    rng = np.random.default_rng(int(best * 2) + 200)
    T, E = 40, 24
    l = torch.full((T, E), best)
    l[:, 1:] = torch.from_numpy(best - rng.uniform(30, 84, (T, E - 1)))
    l[::2, 1:8] = torch.from_numpy(rng.uniform(-120, -85, (T // 2, 7)))
    for topk in (2, 8, 24):
        for scale in (1.0, 2.5):
            _, w = check_gate(l, topk, score="sigmoid", renormalize=True, scale=scale)
            assert (w[1::2] > 0).all()
    l = torch.tensor([[-59.0, -95.0]])
    _, w = check_gate(l, 2, score="sigmoid", renormalize=True)
    assert 2.3e-16 < float(w[0, 1]) < 2.4e-16


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,n_group", [(60, 1), (60, 6), (33, 1), (66, 3), (100, 5), (34, 2), (260, 1), (1020, 17), (7, 1)])
def test_a_batch_that_starts_at_any_row(E, n_group, dtype):
    """Slices of a larger batch: rows of 120 bytes start at multiples of 8, rows of 66 at multiples of 2."""
    T, topk = 21, 3
    whole = _rand(T + 8, E, E, dtype).cuda()
    d_whole = torch.full_like(whole, 7.0)
    bias = torch.zeros(3, E, device="cuda")
    bias[1] = 0.05 * _rand(1, E, 9)[0].cuda()
    kw = dict(score="sigmoid", renormalize=True)
    for first in (1, 2, 3, 4, 8):
        l = whole[first:first + T]
        for b in (None, bias[1]):
            ids, w = check_gate(l, topk, b, n_group=n_group, topk_group=(n_group + 1) // 2, **kw)
            again, _ = dg.moe_gate(l.clone(), topk, b, n_group=n_group, topk_group=(n_group + 1) // 2, **kw)
            assert torch.equal(ids, again)
        g = _rand(T, topk, 5).cuda()
        for score in ("sigmoid", "softmax"):
            d = dg.moe_gate_backward(l, ids, g, score=score, d_logits=d_whole[first:first + T])
            assert torch.equal(d, dg.moe_gate_backward(l.clone(), ids, g, score=score))
        assert (d_whole[:first] == 7).all() and (d_whole[first + T:] == 7).all()
        d_whole.fill_(7.0)


def test_outputs_beyond_the_rows_stay_and_no_tokens_is_nothing():
    ids = torch.full((12, 3), 77, dtype=torch.int32, device="cuda")
    w = torch.full((12, 3), 77.0, device="cuda")
    dg.moe_gate(_rand(5, 9, 61).cuda(), 3, ids=ids[:5], weights=w[:5])
    torch.cuda.synchronize()
    assert (ids[5:] == 77).all() and (w[5:] == 77).all() and (ids[:5] < 9).all()
    i0, w0 = dg.moe_gate(torch.empty((0, 9), device="cuda"), 3)
    assert i0.shape == (0, 3) and w0.shape == (0, 3)
    assert dg.moe_gate_backward(torch.empty((0, 9), device="cuda"), i0, w0).shape == (0, 9)


# ------------------------------------------------------------------ gradient


def check_backward(logits, ids, g, flag=0, **kw):
    logits, ids, g = logits.cuda(), ids.to(torch.int32).cuda(), g.float().cuda()
    out = torch.full_like(logits, 7.0)
    dg.moe_gate_backward(logits, ids, g, d_logits=out, **kw)
    torch.cuda.synchronize()
    assert dg.get_device_error() == flag
    l = _f64(logits)
    ref, size = routing.moe_gate_backward(l, ids.cpu().numpy(), _f64(g), **kw)
    tol = (2 * _slack(l, kw.get("score")) + 18)[:, None] * U * size + 2.0 ** -126
    if logits.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(_f64(out) - ref)
    assert (err <= tol).all(), np.argwhere(err > tol)[:4]
    again = dg.moe_gate_backward(logits, ids, g, **kw)
    assert torch.equal(again, out)
    return out


def _ids(T, E, topk, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, topk)) < drop] = -1
    return torch.from_numpy(ids)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (129, 32, 8), (64, 33, 4), (77, 60, 4),
                                      (40, 100, 32), (200, 256, 8), (9, 257, 5), (17, 512, 16), (12, 1024, 32)])
def test_gradient(T, E, topk, score, renormalize, dtype):
    check_backward(_rand(T, E, T + E, dtype), _ids(T, E, topk, T, 0.1), _rand(T, topk, E), score=score,
                   renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_edges(score, renormalize):
    T, E, topk = 12, 40, 4
    l, ids, g = _rand(T, E, 71), _ids(T, E, topk, 72), _rand(T, topk, 73)
    l[0] = -INF
    ids[0] = -1                               # a padded token
    ids[1] = -1
    l[1, 0] = float("nan")                    # not routed: zeros whatever its logits are
    l[2, 20:] = -INF
    ids[2] = torch.tensor([0, 3, 19, -1])     # masked experts, one slot left over
    ids[3] = torch.tensor([5, 5, 7, 5])       # one expert in three slots
    l[4] = -200.0 - l[4].abs()                # scores that are zero in 32 bits
    l[5] = 60.0
    g[6] = 0.0
    out = check_backward(l[2:], ids[2:], g[2:], score=score, renormalize=renormalize, scale=1.0)
    assert (out[4] == 0).all()
    out = dg.moe_gate_backward(l.cuda(), ids.int().cuda(), g.cuda(), score=score, renormalize=renormalize)
    assert (out[:2] == 0).all() and dg.get_device_error() == 0


def test_gradient_flags_ids_out_of_range():
    l, g = _rand(3, 8, 81), _rand(3, 2, 82)
    bad = torch.tensor([[0, 8], [1, -2], [3, 4]])
    out = check_backward(l, bad, g, flag=dg.DG_DEVERR_BAD_EXPERT, score="sigmoid", renormalize=True)
    assert out[0, 1:].eq(0).all()


def test_gradient_of_the_weights_by_differences():
    """The whole path against central differences of the forward kernel's own
    weights, in directions that leave the choice as it is."""
    T, E, topk = 50, 24, 4
    l = _rand(T, E, 91).cuda()
    g = _rand(T, topk, 92).cuda()
    v = _rand(T, E, 93).cuda()
    h = 2.0 ** -7
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            kw = dict(score=score, renormalize=renormalize, scale=2.5)
            ids, _ = dg.moe_gate(l, topk, **kw)
            d = dg.moe_gate_backward(l, ids, g, **kw)
            iu, wu = dg.moe_gate(l + h * v, topk, **kw)
            il, wl = dg.moe_gate(l - h * v, topk, **kw)
            same = ((iu == ids) & (il == ids)).all(dim=1)
            assert same.sum() > T // 2
            by_difference = ((wu - wl).double() * g).sum(1) / (2 * h)
            by_gradient = (d.double() * v).sum(1)
            # third derivatives along v: at most 2.5 * |g|_1 * |v|_max^3 * 1 each, times h^2 / 6; rounding
            # of the weights (at most 2.5 * 2^-20 each) over h
            bound = g.abs().sum(1).double() * (2.5 * v.abs().amax(1).double() ** 3 * h * h + 2.5 * 2.0 ** -19 / h)
            assert ((by_difference - by_gradient).abs()[same] <= bound[same]).all()


# ------------------------------------------------------------------ streams and graphs


def test_two_streams_and_a_captured_graph():
    T, E, topk = 300, 256, 8
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, renormalize=True, scale=2.5)
    b = (0.05 * _rand(1, E, 3)[0]).cuda()
    one, two = _rand(T, E, 1).cuda(), _rand(T, E, 2).cuda()
    want = [dg.moe_gate(x, topk, b, **kw) for x in (one, two)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for s, x in ((s1, one), (s2, two)):
        with torch.cuda.stream(s):
            got.append(dg.moe_gate(x, topk, b, **kw))
    torch.cuda.synchronize()
    for (i, w), (gi, gw) in zip(want, got):
        assert torch.equal(i, gi) and torch.equal(w, gw)
    # forward and gradient captured once, replayed on new inputs
    x, g = one.clone(), _rand(T, topk, 4).cuda()
    ids = torch.empty((T, topk), dtype=torch.int32, device="cuda")
    w, d = torch.empty((T, topk), device="cuda"), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.moe_gate(x, topk, b, ids=ids, weights=w, **kw)
        dg.moe_gate_backward(x, ids, g, score="sigmoid", renormalize=True, scale=2.5, d_logits=d)
    for src, (i, ww) in zip((one, two), want):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, i) and torch.equal(w, ww)
        assert torch.equal(d, dg.moe_gate_backward(src, i, g, score="sigmoid", renormalize=True, scale=2.5))
    assert dg.get_device_error() == 0
