"""GPU parity of the int8 products (exact int32 sums), of the per-token
quantisation (bit exact) and of its scattering form, against oracle.routing,
and the MoE chains that the routing opens.

Tolerances: the integer sum is exact; its conversion to FP32 and the two
products with the scales are off by half a step (2^-24) each, so
3.01 * 2^-24 relative, and a BF16 result by 2^-8 more.
"""
import numpy as np
import pytest
import torch

import oracle
from moe_grouped_gemm_05_b200 import binding as dg
from moe_grouped_gemm_05_b200 import synth
from oracle import routing

from helpers import bits, check_close, packed, to_device

pytestmark = pytest.mark.gpu
CONFIGS = [(64, 1, 1), (128, 1, 1), (256, 1, 1), (128, 2, 1), (256, 2, 1), (64, 1, 2), (128, 1, 2)]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dg.set_config(0)
    dg.get_device_error()
    yield
    dg.set_config(0)


def _codes(rng, *shape):
    q = rng.integers(-128, 128, shape, dtype=np.int8)
    return q, (rng.random(shape[:-1]) * 0.02 + 1e-4).astype(np.float32)


def _cuda(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in arrays]


def _check(got, ref):
    x = got.double().cpu().numpy()
    tol = 3.01 * 2.0 ** -24 * np.abs(ref) + 2.0 ** -149
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -134
    err = np.abs(x - ref)
    assert (err <= tol).all(), (np.argwhere(~(err <= tol))[:3], err.max())


# ------------------------------------------------------------------ dense


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 16, 128), (2, 32, 144), (64, 512, 2048), (65, 48, 272),
                                   (127, 240, 1008), (128, 256, 256), (129, 272, 2064), (257, 1040, 640),
                                   (300, 4112, 512)])
def test_dense(M, N, K, dtype):
    rng = np.random.default_rng(M + N + K)
    (a, sa), (b, sb) = _codes(rng, M, K), _codes(rng, N, K)
    d = dg.int8_gemm_nt(*_cuda(a, sa, b, sb), out_dtype=dtype)
    _check(d, routing.int8_gemm(a, sa, b, sb))
    assert dg.get_device_error() == 0


@pytest.mark.parametrize("cfg", CONFIGS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dense_every_configuration(cfg, dtype):
    """Ragged rows and columns, a K tail, several tiles a CTA (few SMs), and no write behind the rows."""
    rng = np.random.default_rng(7)
    M, N, K = 700, 1424, 1040
    (a, sa), (b, sb) = _codes(rng, M, K), _codes(rng, N, K)
    ref = routing.int8_gemm(a, sa, b, sb)
    dg.set_config(*cfg)
    prev = dg.set_num_sms(8)
    try:
        d = torch.full((M + 4, N), 7.0, dtype=dtype, device="cuda")
        dg.int8_gemm_nt(*_cuda(a, sa, b, sb), d=d[:M])
        _check(d[:M], ref)
        assert (d[M:] == 7).all()
    finally:
        dg.set_num_sms(prev)
    assert dg.get_device_error() == 0


def test_sums_at_the_edge_of_int32():
    """The largest K with every product at its extreme: 131056 * 2^14 < 2^31."""
    K = 131056
    a = np.full((3, K), -128, np.int8)
    b = np.full((16, K), -128, np.int8)
    b[1] = 127
    b[2, ::2] = 127
    one = np.ones(16, np.float32)
    d = dg.int8_gemm_nt(*_cuda(a, one[:3], b, one), out_dtype=torch.float32)
    _check(d, routing.int8_gemm(a, one[:3], b, one))


def test_scales_of_every_size():
    """Scales near the ends of FP32's range, a NaN scale, zero scales."""
    rng = np.random.default_rng(3)
    M, N, K = 40, 64, 256
    (a, _), (b, _) = _codes(rng, M, K), _codes(rng, N, K)
    sa = np.exp2(rng.integers(-60, 60, M)).astype(np.float32)
    sb = np.exp2(rng.integers(-60, 30, N)).astype(np.float32)
    sa[5], sb[9] = 0.0, 0.0
    d = dg.int8_gemm_nt(*_cuda(a, sa, b, sb), out_dtype=torch.float32)
    _check(d, routing.int8_gemm(a, sa, b, sb))
    sa[7] = np.nan
    d = dg.int8_gemm_nt(*_cuda(a, sa, b, sb))
    assert torch.isnan(d[7]).all() and torch.isfinite(d[8]).all()


# ------------------------------------------------------------------ grouped


def _contiguous(rng, counts, N, K, extra=0):
    G = len(counts)
    idx = synth.contiguous_indices(np.asarray(counts))
    idx = np.concatenate([idx, np.full(128 * extra, -1, np.int32)]).astype(np.int32)
    (a, sa), (b, sb) = _codes(rng, len(idx), K), _codes(rng, G, N, K)
    sa[idx < 0] = np.nan       # padding rows hold anything
    return a, sa, b, sb, idx


def _check_contiguous(d, before, a, sa, b, sb, idx):
    for g in range(len(b)):
        rows = np.nonzero(idx == g)[0]
        if len(rows):
            _check(d[torch.from_numpy(rows).cuda()], routing.int8_gemm(a[rows], sa[rows], b[g], sb[g]))
    pad = torch.from_numpy(np.nonzero(idx < 0)[0]).cuda()
    assert torch.equal(d[pad], before[pad])


@pytest.mark.parametrize("cfg", [None, *CONFIGS])
@pytest.mark.parametrize("counts,N,K", [([100, 0, 150, 1, 300], 272, 400), ([128, 256, 384], 512, 128),
                                        ([0, 0, 7], 16, 16), ([1000], 1040, 256)])
def test_contiguous(counts, N, K, cfg):
    rng = np.random.default_rng(sum(counts) + N)
    a, sa, b, sb, idx = _contiguous(rng, counts, N, K, extra=2)
    if cfg:
        dg.set_config(*cfg)
    before = torch.full((len(idx), N), 7.0, dtype=torch.bfloat16, device="cuda")
    d = before.clone()
    prev = dg.set_num_sms(6)
    try:
        dg.m_grouped_int8_gemm_nt_contiguous(*_cuda(a, sa, b, sb, idx), d=d)
        torch.cuda.synchronize()
    finally:
        dg.set_num_sms(prev)
    _check_contiguous(d, before, a, sa, b, sb, idx)
    assert dg.get_device_error() == 0


@pytest.mark.parametrize("cfg", [(128, 1, 1), (256, 2, 1)])
def test_contiguous_flags_bad_rows(cfg):
    rng = np.random.default_rng(5)
    a, sa, b, sb, idx = _contiguous(rng, [128, 128, 128, 128], 64, 128)
    idx[130] = 0           # a second expert in expert 1's tile
    idx[256:384] = 4       # no such expert
    dg.set_config(*cfg)
    before = torch.full((len(idx), 64), 7.0, dtype=torch.bfloat16, device="cuda")
    d = before.clone()
    dg.m_grouped_int8_gemm_nt_contiguous(*_cuda(a, sa, b, sb, idx), d=d)
    torch.cuda.synchronize()
    assert dg.get_device_error() == dg.DG_DEVERR_BAD_EXPERT | dg.DG_DEVERR_MIXED_TILE
    sa = np.where(np.isnan(sa), 1, sa)
    ref = {g: routing.int8_gemm(a, sa, b[g], sb[g]) for g in range(4)}
    _check(d[:128], ref[0][:128])
    keep = np.r_[128:130, 131:256]
    _check(d[torch.from_numpy(keep).cuda()], ref[1][keep])
    _check(d[384:], ref[3][384:])
    assert (d[130] == 7).all() and (d[256:384] == 7).all()


@pytest.mark.parametrize("cfg", [None, *CONFIGS])
@pytest.mark.parametrize("M_max,N,K,counts", [(256, 272, 400, [0, 1, 255, 256, 37]), (96, 512, 144, [96, 0, 50]),
                                              (1, 16, 16, [1, 0]), (300, 128, 256, [300] * 9)])
def test_masked(M_max, N, K, counts, cfg):
    rng = np.random.default_rng(M_max + N)
    G = len(counts)
    (a, sa), (b, sb) = _codes(rng, G, M_max, K), _codes(rng, G, N, K)
    if cfg:
        dg.set_config(*cfg)
    d = torch.full((G, M_max, N), 7.0, dtype=torch.bfloat16, device="cuda")
    prev = dg.set_num_sms(6)
    try:
        dg.m_grouped_int8_gemm_nt_masked(*_cuda(a, sa, b, sb, np.array(counts, np.int32)), d=d)
        torch.cuda.synchronize()
    finally:
        dg.set_num_sms(prev)
    for g, n in enumerate(counts):
        if n:
            _check(d[g, :n], routing.int8_gemm(a[g, :n], sa[g, :n], b[g], sb[g]))
        assert (d[g, n:] == 7).all()
    assert dg.get_device_error() == 0


def test_masked_clamps_and_flags_bad_counts():
    rng = np.random.default_rng(8)
    (a, sa), (b, sb) = _codes(rng, 3, 64, 128), _codes(rng, 3, 32, 128)
    d = torch.full((3, 64, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    dg.m_grouped_int8_gemm_nt_masked(*_cuda(a, sa, b, sb, np.array([-5, 1000, 2], np.int32)), d=d)
    torch.cuda.synchronize()
    assert dg.get_device_error() == dg.DG_DEVERR_BAD_MASKED_M
    assert (d[0] == 7).all()
    _check(d[1], routing.int8_gemm(a[1], sa[1], b[1], sb[1]))
    assert (d[2, 2:] == 7).all()


def test_no_rows_is_nothing():
    b, sb = torch.zeros((32, 64), dtype=torch.int8, device="cuda"), torch.ones(32, device="cuda")
    e8, ef = torch.empty((0, 64), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    assert dg.int8_gemm_nt(e8, ef, b, sb).shape == (0, 32)
    idx = torch.empty(0, dtype=torch.int32, device="cuda")
    assert dg.m_grouped_int8_gemm_nt_contiguous(e8, ef, b[None], sb[None], idx).shape == (0, 32)
    q, s = dg.quantize_int8_per_token(torch.empty((0, 64), device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,)


@pytest.mark.parametrize("cfg", [(128, 1, 1), (64, 1, 2)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(cfg):
    rng = np.random.default_rng(9)
    M, N, K = 128, 512, 32768
    (a, sa), (b, sb) = _codes(rng, M, K), _codes(rng, N, K)
    t = _cuda(a, sa, b, sb)
    dg.set_config(*cfg)
    prev = dg.set_wait_limit_ns(0)
    try:
        dg.int8_gemm_nt(*t)
        torch.cuda.synchronize()
    finally:
        dg.set_wait_limit_ns(prev)
    assert dg.get_device_error() & dg.DG_DEVERR_TIMEOUT
    _check(dg.int8_gemm_nt(*t), routing.int8_gemm(a, sa, b, sb))
    assert dg.get_device_error() == 0


def test_one_sm():
    """Products that take CTA pairs on more SMs, on one (which holds no pair)."""
    rng = np.random.default_rng(15)
    (a, sa), (b, sb) = _codes(rng, 300, 272), _codes(rng, 528, 272)
    idx = np.repeat(np.arange(3, dtype=np.int32), 128)
    (x, sx), (w, sw) = _codes(rng, 384, 272), _codes(rng, 3, 528, 272)
    want = dg.int8_gemm_nt(*_cuda(a, sa, b, sb))
    grouped = dg.m_grouped_int8_gemm_nt_contiguous(*_cuda(x, sx, w, sw, idx))
    t = _cuda(x.reshape(3, 128, 272), sx.reshape(3, 128), w, sw, np.full(3, 128, np.int32))
    prev = dg.set_num_sms(1)
    try:
        for cfg in ((0, 0, 0), (256, 2, 1)):
            dg.set_config(*cfg)
            assert torch.equal(dg.int8_gemm_nt(*_cuda(a, sa, b, sb)), want)
            assert torch.equal(dg.m_grouped_int8_gemm_nt_contiguous(*_cuda(x, sx, w, sw, idx)), grouped)
            assert torch.equal(dg.m_grouped_int8_gemm_nt_masked(*t).reshape(384, 528), grouped)
        p = synth.dense_problem(300, 528, 256, seed=3)
        qa, qb = packed(p)
        f = to_device(p, qa, qb)
        d = dg.fp8_gemm_nt(f["a"], f["sfa"], f["b"], f["sfb"])
        check_close(bits(d), oracle.fp8_gemm_nt(p.a, qa, p.b, qb, 300, 528, 256), "one SM")
    finally:
        dg.set_num_sms(prev)
    _check(want, routing.int8_gemm(a, sa, b, sb))
    assert dg.get_device_error() == 0


@pytest.mark.parametrize("cfg", [(128, 2, 1), (256, 2, 1)])
def test_pairs_whose_second_cta_has_no_rows(cfg):
    """The second CTA of a pair hands its accumulators back and is done before the
    first: from one to five tiles a pair (both accumulators used never, once and
    again), one K block and more than the ring holds, in runs of dependent launches."""
    rng = np.random.default_rng(12)
    dg.set_config(*cfg)
    prev = dg.set_num_sms(2)
    try:
        for tiles in range(1, 6):
            for K in (16, 128, 1040, 2064):
                M, N = 100, cfg[0] * tiles - 16
                (a, sa), (b, sb) = _codes(rng, M, K), _codes(rng, N, K)
                t = _cuda(a, sa, b, sb)
                d = [dg.int8_gemm_nt(*t) for _ in range(20)]
                _check(d[0], routing.int8_gemm(a, sa, b, sb))
                assert all(torch.equal(x, d[0]) for x in d)
                # masked: pairs with rows of the first CTA only, of both, of none
                counts, G = [128, 256, 0, 1, 129], 5
                (a, sa), (b, sb) = _codes(rng, G, 256, K), _codes(rng, G, N, K)
                t = _cuda(a, sa, b, sb, np.array(counts, np.int32))
                d = [torch.full((G, 256, N), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(5)]
                for x in d:
                    dg.m_grouped_int8_gemm_nt_masked(*t, d=x)
                for g, n in enumerate(counts):
                    if n:
                        _check(d[0][g, :n], routing.int8_gemm(a[g, :n], sa[g, :n], b[g], sb[g]))
                    assert (d[0][g, n:] == 7).all()
                assert all(torch.equal(x, d[0]) for x in d)
        # contiguous: runs of one and of three blocks, each ending in a half-empty pair
        a, sa, b, sb, idx = _contiguous(rng, [100, 300, 128], 272, 400)
        t = _cuda(a, sa, b, sb, idx)
        before = torch.full((len(idx), 272), 7.0, dtype=torch.bfloat16, device="cuda")
        d = [before.clone() for _ in range(20)]
        for x in d:
            dg.m_grouped_int8_gemm_nt_contiguous(*t, d=x)
        _check_contiguous(d[0], before, a, sa, b, sb, idx)
        assert all(torch.equal(x, d[0]) for x in d)
    finally:
        dg.set_num_sms(prev)
    assert dg.get_device_error() == 0


@pytest.mark.parametrize("cfg", [(128, 2, 1), (256, 2, 1)])
def test_a_pair_whose_wait_runs_out_is_reported_and_the_next_call_is_right(cfg):
    rng = np.random.default_rng(14)
    M, N, K = 256, 512, 32768
    (a, sa), (b, sb) = _codes(rng, M, K), _codes(rng, N, K)
    t = _cuda(a, sa, b, sb)
    dg.set_config(*cfg)
    prev = dg.set_wait_limit_ns(0)
    try:
        dg.int8_gemm_nt(*t)
        torch.cuda.synchronize()
    finally:
        dg.set_wait_limit_ns(prev)
    assert dg.get_device_error() & dg.DG_DEVERR_TIMEOUT
    _check(dg.int8_gemm_nt(*t), routing.int8_gemm(a, sa, b, sb))
    assert dg.get_device_error() == 0


@pytest.mark.parametrize("cfg", [None, (128, 2, 1)])
def test_row_and_column_counts_next_to_2_to_the_31(cfg):
    """The largest row counts of every layout and the largest column count, every element:
    sums of 16 products are exact in FP32, so torch's product takes the same roundings."""
    most, K = 2 ** 31 - 1, 16
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 140 << 30:
        pytest.skip("140 GiB of device memory needed")
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.empty((most, K), dtype=torch.int8, device="cuda").random_(-128, 128, generator=g)
    sa = torch.empty(most, device="cuda").uniform_(0.5, 1.5, generator=g)
    b, sb = a[:K].clone(), sa[:K].clone()
    d = torch.empty((most, K), dtype=torch.bfloat16, device="cuda")

    def check(rows):
        for i in range(0, most, 2 ** 25):
            p = slice(i, min(most, i + 2 ** 25))
            want = ((a[p].float() @ b.float().t()) * sa[p, None] * sb).to(torch.bfloat16)
            if p.stop > rows:
                want[max(0, rows - i):] = 7
            assert torch.equal(d[p], want), i
        d.fill_(7)

    if cfg:
        dg.set_config(*cfg)
    d.fill_(7)
    dg.int8_gemm_nt(a, sa, b, sb, d=d)
    check(most)
    counts = torch.tensor([most], dtype=torch.int32, device="cuda")
    dg.m_grouped_int8_gemm_nt_masked(a[None], sa[None], b[None], sb[None], counts, d=d[None])
    check(most)
    whole = most // 128 * 128
    idx = torch.zeros(whole, dtype=torch.int32, device="cuda")
    dg.m_grouped_int8_gemm_nt_contiguous(a[:whole], sa[:whole], b[None], sb[None], idx, d=d[:whole])
    check(whole)
    del idx, d
    # one row against 2^31 - 16 columns
    N = most - 15
    d = dg.int8_gemm_nt(b[:1], sb[:1], a[:N], sa[:N])
    for i in range(0, N, 2 ** 25):
        p = slice(i, min(N, i + 2 ** 25))
        assert torch.equal(d[:, p], ((b[:1].float() @ a[p].float().t()) * sb[:1, None] * sa[p]).to(torch.bfloat16)), i
    assert dg.get_device_error() == 0
    del a, sa, d
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ quantisation


def _activations(M, K, seed, dtype):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp(rng.uniform(-12, 12, size=(M, 1)))
    x = torch.from_numpy(x).to(dtype)
    if M > 4:
        x[0] = 0.0
        x[1] *= 1e-35 / x[1].abs().max()          # scale below 2^-126 but for the clamp, or next to it
        x[2] = torch.linspace(-127, 127, K).to(dtype)
        x[3, 0] = torch.finfo(dtype).max
        x[4] = 2.0 ** -133                          # subnormal
    return x


def _same(got_q, got_s, x):
    q, s = routing.quantize_int8_per_token(x.float().numpy())
    assert np.array_equal(got_q.cpu().numpy(), q)
    assert np.array_equal(got_s.cpu().numpy().view(np.uint32), s.view(np.uint32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 16), (7, 16), (33, 144), (5, 512), (130, 528), (64, 1040), (37, 7168), (6, 8208),
                                 (5, 16400), (5, 32784), (6, 65536), (6, 131056)])
def test_quantize_bit_exact(M, K, dtype):
    x = _activations(M, K, M + K, dtype)
    q = torch.full((M + 2, K), 77, dtype=torch.int8, device="cuda")
    s = torch.full((M + 2,), 77.0, device="cuda")
    dg.quantize_int8_per_token(x.cuda(), q=q[:M], scale=s[:M])
    _same(q[:M], s[:M], x)
    assert (q[M:] == 77).all() and (s[M:] == 77).all()


def test_quantize_leading_dimensions_and_ties():
    x = _activations(60, 256, 4, torch.float32).reshape(3, 20, 256)
    q, s = dg.quantize_int8_per_token(x.cuda())
    assert q.shape == (3, 20, 256) and s.shape == (3, 20)
    _same(q.reshape(60, 256), s.reshape(60), x.reshape(60, 256))
    t = torch.arange(-127, 128).float().mul(0.5)
    x = torch.cat([torch.tensor([127.0]), t]).reshape(1, 256)         # amax 127: halves tie to even
    q, _ = dg.quantize_int8_per_token(x.cuda())
    assert np.array_equal(q.cpu().numpy()[0, 1:], np.rint(t.numpy()))


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_finite(what):
    for dtype in (torch.bfloat16, torch.float32):
        for K in (64, 7168, 131056):
            x = _activations(7, K, 5, dtype)
            x[5, K - 1] = what
            q, s = dg.quantize_int8_per_token(x.cuda())
            assert torch.isnan(s[5]) and (q[5] == 0).all()
            keep = [0, 1, 2, 3, 4, 6]
            _same(q[keep], s[keep], x[keep])


def _routing(T, topk, G, seed, drop=0.1):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(G)[:topk] for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, topk)) < drop] = -1
    return ids


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,topk,G,K", [(300, 2, 6, 512), (1, 1, 1, 16), (1, 1, 3, 144), (700, 8, 32, 640),
                                        (64, 4, 256, 8208), (50, 40, 50, 272), (20, 2, 4, 131056), (256, 8, 64, 2064),
                                        (1, 64, 1024, 512), (255, 8, 1024, 16400), (1100, 2, 9, 7168)])
def test_quantize_permute_bit_exact(T, topk, G, K, dtype):
    """Into buffers that hold something else first: all that is defined is
    written, and the codes of padding rows are not."""
    ids = _routing(T, topk, G, T + G)
    x = _activations(T, K, T + K, dtype)
    cap = dg.load().dg_moe_permute_capacity(T, topk, G)
    out = {"a": torch.full((cap, K), 77, dtype=torch.int8, device="cuda"),
           "sa": torch.full((cap,), 7.0, device="cuda"),
           "m_indices": torch.full((cap,), 77, dtype=torch.int32, device="cuda"),
           "src_of": torch.full((cap,), 77, dtype=torch.int32, device="cuda"),
           "row_of": torch.full((T, topk), 77, dtype=torch.int32, device="cuda")}
    dg.moe_quantize_permute_int8(torch.from_numpy(ids).cuda(), G, x.cuda(), out=out)
    torch.cuda.synchronize()
    assert dg.get_device_error() == 0
    m, row_of, src, Mt, _ = oracle.fp8_gemm.moe_permute(ids, G)
    got = {k: v.cpu().numpy() for k, v in out.items()}
    assert np.array_equal(got["m_indices"][:Mt], m) and (got["m_indices"][Mt:] == -1).all()
    assert np.array_equal(got["src_of"][:Mt], src) and (got["src_of"][Mt:] == -1).all()
    assert np.array_equal(got["row_of"], row_of)
    q, s = routing.quantize_int8_per_token(x.float().numpy())
    valid = np.nonzero(m >= 0)[0]
    pad = np.setdiff1d(np.arange(cap), valid)
    assert np.array_equal(got["a"][valid], q[src[valid]]) and (got["a"][pad] == 77).all()
    assert np.array_equal(got["sa"][valid], s[src[valid]]) and (got["sa"][pad] == 0).all()


def test_quantize_permute_no_tokens_and_bad_ids():
    x = torch.ones((2, 128), device="cuda")
    out = dg.moe_quantize_permute_int8(torch.tensor([[0, 5], [1, -3]], dtype=torch.int32, device="cuda"), 2, x)
    assert dg.get_device_error() & dg.DG_DEVERR_BAD_EXPERT
    assert out["row_of"].tolist() == [[0, -1], [128, -1]]
    out = dg.moe_quantize_permute_int8(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4, x[:0])
    torch.cuda.synchronize()
    assert (out["m_indices"] == -1).all() and (out["sa"] == 0).all() and dg.get_device_error() == 0


# ------------------------------------------------------------------ together


class Layer:
    """gate -> quantise and permute -> grouped int8 product -> combine, on fixed buffers."""

    T, E, TOPK, K, N = 700, 32, 4, 640, 272
    KW = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, renormalize=True, scale=2.5)

    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        self.w, self.sw = _codes(rng, self.E, self.N, self.K)
        self.bias = (0.05 * rng.standard_normal(self.E)).astype(np.float32)
        self.b, self.sb, self.g_bias = _cuda(self.w, self.sw, self.bias)
        T, E, topk, K, N = self.T, self.E, self.TOPK, self.K, self.N
        cap = dg.load().dg_moe_permute_capacity(T, topk, E)
        empty = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")
        self.logits, self.x = empty(T, E), empty(T, K, t=torch.bfloat16)
        self.ids, self.weights = empty(T, topk, t=torch.int32), empty(T, topk)
        self.per = {"a": empty(cap, K, t=torch.int8), "sa": empty(cap), "m_indices": empty(cap, t=torch.int32),
                    "src_of": empty(cap, t=torch.int32), "row_of": empty(T, topk, t=torch.int32)}
        self.d, self.out = empty(cap, N, t=torch.bfloat16), empty(T, N, t=torch.bfloat16)

    def inputs(self, seed):
        rng = np.random.default_rng(seed)
        l = torch.from_numpy(rng.standard_normal((self.T, self.E)).astype(np.float32))
        l[rng.random(self.T) < 0.05] = -float("inf")     # padded tokens
        x = torch.from_numpy(rng.standard_normal((self.T, self.K))).to(torch.bfloat16)
        return l, x

    def run(self):
        dg.moe_gate(self.logits, self.TOPK, self.g_bias, ids=self.ids, weights=self.weights, **self.KW)
        dg.moe_quantize_permute_int8(self.ids, self.E, self.x, out=self.per)
        dg.m_grouped_int8_gemm_nt_contiguous(self.per["a"], self.per["sa"], self.b, self.sb, self.per["m_indices"],
                                             d=self.d)
        dg.moe_unpermute_combine(self.d, self.per["row_of"], self.weights, out=self.out)

    def expected(self, l, x):
        ids, w, _ = routing.moe_gate(l.numpy(), self.TOPK, self.bias, **self.KW)
        q, s = routing.quantize_int8_per_token(x.float().numpy())
        out = np.zeros((self.T, self.N))
        size = np.zeros((self.T, self.N))
        for e in range(self.E):
            t, j = np.nonzero(ids == e)
            if len(t):
                part = w[t, j][:, None] * routing.int8_gemm(q[t], s[t], self.w[e], self.sw[e])
                out[t] += part
                size[t] += np.abs(part)
        return ids, out, size


def _check_layer(layer, l, x):
    ids, ref, size = layer.expected(l, x)
    assert np.array_equal(layer.ids.cpu().numpy(), ids)
    # each expert's row is rounded to BF16 (2^-8), weights and sums add a few 2^-24, the result is rounded to BF16
    tol = (2.0 ** -8 + 64 * 2.0 ** -24) * size
    tol += 2.0 ** -8 * (np.abs(ref) + tol)
    assert (np.abs(layer.out.double().cpu().numpy() - ref) <= tol).all()
    assert (layer.out[(ids < 0).all(axis=1)] == 0).all()
    assert dg.get_device_error() == 0


def test_layer_from_logits_to_outputs():
    layer = Layer(1)
    l, x = layer.inputs(2)
    layer.logits.copy_(l)
    layer.x.copy_(x)
    layer.run()
    torch.cuda.synchronize()
    _check_layer(layer, l, x)
    first = layer.out.clone()
    prev = dg.set_pdl(False)
    try:
        layer.out.fill_(7)
        layer.run()
        torch.cuda.synchronize()
    finally:
        dg.set_pdl(prev)
    assert torch.equal(layer.out, first)


def test_two_captured_layers_replayed():
    """Two layers' graphs, replayed on two streams at once on new inputs; each keeps to its own buffers."""
    layers, graphs, streams = [Layer(3), Layer(4)], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for layer in layers:
        l, x = layer.inputs(5)
        layer.logits.copy_(l)
        layer.x.copy_(x)
        layer.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.run()
        graphs.append(g)
    for seed in (6, 7):
        given = []
        for layer, off in zip(layers, (0, 100)):
            l, x = layer.inputs(seed + off)
            layer.logits.copy_(l)
            layer.x.copy_(x)
            given.append((l, x))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for layer, (l, x) in zip(layers, given):
            _check_layer(layer, l, x)


def test_decode_layer_in_the_masked_layout():
    """A captured decode step: quantise a slab of tokens per expert, product over the valid rows."""
    rng = np.random.default_rng(11)
    G, M, N, K = 4, 64, 272, 528
    (w, sw) = _codes(rng, G, N, K)
    b, sb = _cuda(w, sw)
    x = torch.empty((G, M, K), dtype=torch.bfloat16, device="cuda")
    counts = torch.zeros(G, dtype=torch.int32, device="cuda")
    q, s = torch.empty((G, M, K), dtype=torch.int8, device="cuda"), torch.empty((G, M), device="cuda")
    d = torch.full((G, M, N), 7.0, dtype=torch.bfloat16, device="cuda")

    def step():
        dg.quantize_int8_per_token(x, q=q, scale=s)
        dg.m_grouped_int8_gemm_nt_masked(q, s, b, sb, counts, d=d)

    x.zero_()
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed, n in ((1, [0, 1, 64, 13]), (2, [5, 0, 0, 33])):
        xs = torch.from_numpy(np.random.default_rng(seed).standard_normal((G, M, K))).to(torch.bfloat16)
        x.copy_(xs)
        counts.copy_(torch.tensor(n, dtype=torch.int32))
        d.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        cq, cs = routing.quantize_int8_per_token(xs.float().numpy())
        for e in range(G):
            if n[e]:
                _check(d[e, :n[e]], routing.int8_gemm(cq[e, :n[e]], cs[e, :n[e]], w[e], sw[e]))
            assert (d[e, n[e]:] == 7).all()
    assert dg.get_device_error() == 0


def test_gate_feeds_the_fp8_chain():
    """The routing's ids and weights through the FP8 permutation, product and combine."""
    T, E, topk, K, N = 300, 8, 2, 512, 256
    rng = np.random.default_rng(13)
    l = rng.standard_normal((T, E)).astype(np.float32)
    x = torch.from_numpy(rng.standard_normal((T, K))).to(torch.bfloat16)
    w = synth.contiguous_problem(E, N, K, rows=0, seed=6, counts=[1] * E)
    sb, _ = oracle.pack_sf_ue8m0(w.sfb)
    ids, gate = dg.moe_gate(torch.from_numpy(l).cuda(), topk, score="softmax", renormalize=True)
    q, sfa = dg.quantize_fp8_1x128(x.cuda())
    per = dg.moe_permute(ids, E, q, sfa)
    d = dg.m_grouped_fp8_gemm_nt_contiguous(per["a"], per["sfa"], torch.from_numpy(w.b).cuda().view(torch.float8_e4m3fn),
                                            torch.from_numpy(sb).cuda(), per["m_indices"])
    out = dg.moe_unpermute_combine(d, per["row_of"], gate)
    torch.cuda.synchronize()
    ref_ids, ref_w, _ = routing.moe_gate(l, topk, renormalize=True)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    _, row_of, _, _, _ = oracle.fp8_gemm.moe_permute(ref_ids, E)
    assert np.array_equal(per["row_of"].cpu().numpy(), row_of)
    check_close(bits(out), oracle.fp8_gemm.moe_unpermute_combine(bits(d), row_of, ref_w.astype(np.float32)), "combine")
    assert dg.get_device_error() == 0


def test_wrong_operands_are_refused_before_a_launch():
    x = torch.zeros((4, 64), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    a, s = torch.zeros((4, 64), dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    with pytest.raises(ValueError, match="topk_ids"):
        dg.moe_quantize_permute_int8(ids[:3], 4, x)
    with pytest.raises(TypeError, match="topk_ids"):
        dg.moe_quantize_permute_int8(ids.long(), 4, x)
    with pytest.raises(dg.DGError):
        dg.moe_quantize_permute_int8(ids, 0, x)
    with pytest.raises(dg.DGError):
        dg.moe_quantize_permute_int8(ids, 2000, x)
    with pytest.raises(ValueError, match="sa"):
        dg.int8_gemm_nt(a, s[:3], a, s)
    with pytest.raises(ValueError, match="b must"):
        dg.int8_gemm_nt(a, s, torch.zeros((16, 32), dtype=torch.int8, device="cuda"), torch.ones(16, device="cuda"))
    with pytest.raises(dg.DGError, match="multiple of 16"):
        dg.int8_gemm_nt(a, s, a, s)                       # N = 4
    with pytest.raises(ValueError, match="contiguous"):
        dg.quantize_int8_per_token(x.t())
    with pytest.raises(dg.DGError, match="aligned"):
        dg.quantize_int8_per_token(torch.zeros(4 * 64 + 1, device="cuda")[1:].reshape(4, 64))
    with pytest.raises(dg.DGError, match="topk"):
        dg.moe_gate(x, 65)
    assert dg.get_device_error() == 0
