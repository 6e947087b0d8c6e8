"""Refusals of the routing and int8 entry points, on the host (no GPU)."""
import ctypes

import pytest
import torch

from moe_grouped_gemm_05_b200 import binding as dg
from moe_grouped_gemm_05_b200 import build

P = ctypes.c_void_p
GOOD, NULL, ODD8, ODD2 = P(0x10000), P(0), P(0x10008), P(0x10002)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dg.load()


def test_int8_gemm_refusals(lib):
    def dense(a=GOOD, sa=GOOD, b=GOOD, sb=GOOD, d=GOOD, M=64, N=256, K=256, f32=0):
        return lib.dg_int8_gemm_nt(a, sa, b, sb, d, M, N, K, f32, None)

    for name in ("a", "sa", "b", "sb", "d"):
        assert dense(**{name: NULL}) == dg.DG_ERR_NULL, name
        assert dense(**{name: ODD8}) == dg.DG_ERR_ALIGN, name
    assert dense(K=0) == dense(K=24) == dense(K=-16) == dg.DG_ERR_SHAPE
    assert dense(K=131072) == dg.DG_ERR_SHAPE                # 128 * 128 * K leaves int32
    assert b"131056" in lib.dg_get_last_error()
    assert dense(N=0) == dense(N=24) == dg.DG_ERR_SHAPE
    assert dense(M=-1) == dg.DG_ERR_SHAPE
    assert dense(f32=2) == dg.DG_ERR_UNSUPPORTED
    assert dense(a=NULL, d=NULL, M=0) == 0                   # no rows: nothing to do

    def contiguous(idx=GOOD, M=256, G=4, **kw):
        return lib.dg_m_grouped_int8_gemm_nt_contiguous(kw.get("a", GOOD), GOOD, GOOD, GOOD, GOOD, idx, M,
                                                        kw.get("N", 256), kw.get("K", 256), G, None)

    assert contiguous(idx=NULL) == dg.DG_ERR_NULL and contiguous(a=ODD8) == dg.DG_ERR_ALIGN
    assert contiguous(M=200) == contiguous(G=0) == contiguous(K=20) == contiguous(M=-128) == dg.DG_ERR_SHAPE
    assert contiguous(M=0) == 0

    def masked(cnt=GOOD, M=256, G=4, K=256):
        return lib.dg_m_grouped_int8_gemm_nt_masked(GOOD, GOOD, GOOD, GOOD, GOOD, cnt, G, M, 256, K, None)

    assert masked(cnt=NULL) == dg.DG_ERR_NULL
    assert masked(G=0) == masked(G=513) == masked(M=-1) == masked(K=8) == dg.DG_ERR_SHAPE
    assert masked(M=0) == 0


def test_quantize_refusals(lib):
    def quantize(x=GOOD, t=0, q=GOOD, s=GOOD, M=8, K=256):
        return lib.dg_quantize_int8_per_token(x, t, q, s, M, K, None)

    assert quantize(x=NULL) == quantize(q=NULL) == quantize(s=NULL) == dg.DG_ERR_NULL
    assert quantize(x=ODD8) == quantize(q=ODD8) == quantize(s=ODD2) == dg.DG_ERR_ALIGN
    assert quantize(t=2) == dg.DG_ERR_UNSUPPORTED
    assert quantize(K=8) == quantize(K=0) == quantize(M=-1) == dg.DG_ERR_SHAPE
    assert quantize(x=NULL, M=0) == 0

    def permute(ids=GOOD, T=100, topk=2, G=4, x=GOOD, t=0, K=256, a=GOOD, sa=GOOD, row_of=GOOD, cap=None):
        c = lib.dg_moe_permute_capacity(100, 2, 4) if cap is None else cap
        return lib.dg_moe_quantize_permute_int8(ids, T, topk, G, x, t, K, a, sa, GOOD, row_of, GOOD, c, None)

    assert permute(ids=NULL) == permute(x=NULL) == permute(a=NULL) == permute(row_of=NULL) == dg.DG_ERR_NULL
    assert permute(x=ODD8) == permute(a=ODD8) == permute(sa=ODD8) == dg.DG_ERR_ALIGN
    assert permute(t=7) == dg.DG_ERR_UNSUPPORTED
    assert permute(K=100) == permute(G=1025) == permute(topk=0) == permute(T=-1) == dg.DG_ERR_SHAPE
    assert permute(cap=lib.dg_moe_permute_capacity(100, 2, 4) - 128) == dg.DG_ERR_SHAPE
    assert permute(cap=lib.dg_moe_permute_capacity(100, 2, 4) + 64) == dg.DG_ERR_SHAPE


def test_gate_refusals(lib):
    def gate(l=GOOD, t=1, bias=GOOD, T=10, E=64, k=4, score=1, ng=8, kg=4, gt=2, renorm=1, scale=1.0, ids=GOOD, w=GOOD):
        return lib.dg_moe_gate(l, t, bias, T, E, k, score, ng, kg, gt, renorm, scale, ids, w, None)

    assert gate(l=NULL) == gate(ids=NULL) == gate(w=NULL) == dg.DG_ERR_NULL
    assert gate(l=ODD8) == gate(bias=ODD8) == gate(ids=ODD2) == gate(w=ODD2) == dg.DG_ERR_ALIGN
    assert gate(t=2) == gate(score=2) == gate(renorm=2) == dg.DG_ERR_UNSUPPORTED
    assert gate(E=0) == gate(E=1025) == gate(T=-1) == dg.DG_ERR_SHAPE
    assert gate(k=0) == gate(k=33) == gate(E=3, k=4, ng=1, kg=1, gt=1) == dg.DG_ERR_SHAPE
    assert gate(ng=0) == gate(ng=7) == gate(ng=64, kg=1, gt=1, k=1) == dg.DG_ERR_SHAPE
    assert gate(kg=0) == gate(kg=9) == gate(kg=1, k=9) == dg.DG_ERR_SHAPE
    assert gate(gt=0) == gate(gt=3) == gate(E=8, ng=8, k=4, gt=2) == dg.DG_ERR_SHAPE
    assert gate(scale=float("inf")) == gate(scale=float("nan")) == dg.DG_ERR_SHAPE
    assert gate(T=0, l=NULL, ids=NULL, w=NULL) == 0

    def backward(l=GOOD, t=1, ids=GOOD, g=GOOD, T=10, E=64, k=4, score=1, renorm=1, scale=1.0, d=P(0x20000)):
        return lib.dg_moe_gate_backward(l, t, ids, g, T, E, k, score, renorm, scale, d, None)

    assert backward(l=NULL) == backward(ids=NULL) == backward(g=NULL) == backward(d=NULL) == dg.DG_ERR_NULL
    assert backward(l=ODD8) == backward(d=ODD8) == backward(g=ODD2) == dg.DG_ERR_ALIGN
    assert backward(t=3) == backward(score=-1) == backward(renorm=-1) == dg.DG_ERR_UNSUPPORTED
    assert backward(d=GOOD) == dg.DG_ERR_UNSUPPORTED            # in place
    assert backward(k=65) == backward(E=2000) == backward(T=-3) == dg.DG_ERR_SHAPE
    assert backward(scale=float("-inf")) == dg.DG_ERR_SHAPE
    assert backward(T=0, l=NULL, d=NULL) == 0


def test_gate_alignment_goes_by_the_rows_length(lib):
    """Rows of 120 bytes start at multiples of 8, rows of 66 at multiples of 2, rows of 256 at multiples of 16."""
    def gate(l, E, t, bias=NULL):
        return lib.dg_moe_gate(l, t, bias, 10, E, 2, 1, 1, 1, 1, 0, 1.0, GOOD, GOOD, None)

    def backward(l, d, E, t):
        return lib.dg_moe_gate_backward(l, t, GOOD, GOOD, 10, E, 2, 1, 0, 1.0, d, None)

    odd4, odd1 = P(0x10004), P(0x10001)
    for E, t, bad in ((64, 1, ODD8), (64, 0, ODD8), (60, 1, ODD8), (60, 0, odd4), (33, 1, ODD2), (33, 0, odd1),
                      (34, 0, ODD2), (100, 0, odd4)):
        assert gate(bad, E, t) == dg.DG_ERR_ALIGN, (E, t)
        assert backward(bad, GOOD, E, t) == backward(GOOD, bad, E, t) == dg.DG_ERR_ALIGN, (E, t)
    assert gate(GOOD, 64, 0, bias=ODD8) == gate(GOOD, 33, 0, bias=ODD2) == dg.DG_ERR_ALIGN


def test_binding_refuses_before_the_library_is_called():
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        dg.moe_gate(x, 2)
    with pytest.raises(TypeError, match="bfloat16"):
        dg.moe_gate(x.half(), 2)
    with pytest.raises(ValueError, match="score"):
        dg.moe_gate(x, 2, score="tanh")
    with pytest.raises(ValueError, match="CUDA"):
        dg.quantize_int8_per_token(x)
    with pytest.raises(TypeError, match="int8"):
        dg.int8_gemm_nt(x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        dg.moe_quantize_permute_int8(x, 4, x)
    cpu = -1      # the device number of CPU tensors
    assert dg._operand(x, (torch.float32,), (4, 16), "x", cpu) == x.data_ptr()
    with pytest.raises(TypeError):
        dg._operand(x, (torch.int8,), (4, 16), "x", cpu)
    with pytest.raises(ValueError):
        dg._operand(x, (torch.float32,), (16, 4), "x", cpu)
    with pytest.raises(ValueError):
        dg._operand(x.t(), (torch.float32,), (16, 4), "x", cpu)
    with pytest.raises(ValueError):
        dg._operand(x, (torch.float32,), (4, 16), "x", 0)


def test_sizes_beyond_32_bits_are_refused(monkeypatch):
    """The library takes C ints: 2^32 + 5 tokens must not become 5."""
    monkeypatch.setattr(dg, "_cuda_matrix", lambda t, *args: (t.shape, 0))
    many = torch.empty((2 ** 32 + 5, 1), device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        dg.moe_gate(many, 1)
    with pytest.raises(ValueError, match="32 bits"):
        dg.moe_gate_backward(many, many.to(torch.int32), many)
    for name in ("n_group", "topk_group", "group_top"):
        with pytest.raises(ValueError, match="32 bits"):
            dg.moe_gate(torch.zeros(4, 16), 2, **{name: 2 ** 32 + 1})


BIG = 2 ** 32 + 16        # 16 modulo 2^32, which every entry point takes


def _meta(*shape, t=torch.int8):
    return torch.empty(shape, dtype=t, device="meta")


def _beyond():
    """(name, call) for every size that the wrappers of the routing and int8 entry points pass on."""
    f32, i32 = torch.float32, torch.int32
    yield "gate E", lambda: dg.moe_gate(_meta(1, BIG, t=f32), 2)
    yield "gate topk", lambda: dg.moe_gate(_meta(4, 16, t=f32), 2 ** 32 + 2)
    yield "gate topk below", lambda: dg.moe_gate(_meta(4, 16, t=f32), -2 ** 32 + 2)
    yield "gate n_group below", lambda: dg.moe_gate(_meta(4, 16, t=f32), 2, n_group=-2 ** 32 + 1)
    yield "gradient E", lambda: dg.moe_gate_backward(_meta(1, BIG, t=f32), _meta(1, 2, t=i32), _meta(1, 2, t=f32))
    yield "gradient topk", lambda: dg.moe_gate_backward(_meta(1, 16, t=f32), _meta(1, 2 ** 32 + 2, t=i32),
                                                        _meta(1, 2 ** 32 + 2, t=f32))
    yield "quantize K", lambda: dg.quantize_int8_per_token(_meta(1, BIG, t=f32))
    yield "quantize M", lambda: dg.quantize_int8_per_token(_meta(2 ** 16, 2 ** 16 + 1, 16, t=f32))
    yield "permute T", lambda: dg.moe_quantize_permute_int8(_meta(BIG, 2, t=i32), 4, _meta(BIG, 16, t=f32))
    yield "permute K", lambda: dg.moe_quantize_permute_int8(_meta(4, 2, t=i32), 4, _meta(4, BIG, t=f32))
    yield "permute topk", lambda: dg.moe_quantize_permute_int8(_meta(4, BIG, t=i32), 4, _meta(4, 16, t=f32))
    yield "permute experts", lambda: dg.moe_quantize_permute_int8(_meta(4, 2, t=i32), 2 ** 32 + 4, _meta(4, 16, t=f32))
    for name, (M, N, K) in (("M", (BIG, 16, 16)), ("N", (16, BIG, 16)), ("K", (16, 16, BIG))):
        a, b, sa, sb = _meta(M, K), _meta(N, K), _meta(M, t=f32), _meta(N, t=f32)
        yield f"dense {name}", lambda a=a, b=b, sa=sa, sb=sb: dg.int8_gemm_nt(a, sa, b, sb)
        yield f"contiguous {name}", lambda a=a, b=b, sa=sa, sb=sb: dg.m_grouped_int8_gemm_nt_contiguous(
            a, sa, b[None], sb[None], _meta(a.shape[0], t=i32))
        yield f"masked {name}", lambda a=a, b=b, sa=sa, sb=sb: dg.m_grouped_int8_gemm_nt_masked(
            a[None], sa[None], b[None], sb[None], _meta(1, t=i32))
    yield "contiguous G", lambda: dg.m_grouped_int8_gemm_nt_contiguous(
        _meta(128, 16), _meta(128, t=f32), _meta(BIG, 16, 16), _meta(BIG, 16, t=f32), _meta(128, t=i32))
    yield "masked G", lambda: dg.m_grouped_int8_gemm_nt_masked(
        _meta(BIG, 1, 16), _meta(BIG, 1, t=f32), _meta(BIG, 16, 16), _meta(BIG, 16, t=f32), _meta(BIG, t=i32))


@pytest.mark.parametrize("name,call", [pytest.param(n, c, id=n) for n, c in _beyond()])
def test_no_size_is_taken_modulo_2_to_the_32(name, call, monkeypatch):
    """A size of 2^32 + 16 must not reach the library, which would see 16."""
    reached = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: reached.append((name, args)) or 0

    monkeypatch.setattr(dg, "_cuda_matrix", lambda t, *args: (t.shape, 0))
    monkeypatch.setattr(dg, "_operand", lambda t, *args: 0x10000)
    monkeypatch.setattr(dg, "_launch_stream", lambda dev: 0)
    monkeypatch.setattr(dg, "load", lambda: Library())
    with pytest.raises(ValueError, match="32 bits"):
        call()
    assert not reached


def test_fp8_sizes_beyond_32_bits_are_refused(monkeypatch):
    for name in ("_fp8", "_i32", "_sfa_kind", "_packed_numel"):
        monkeypatch.setattr(dg, name, lambda *args: False)
    i32 = torch.int32
    for M, N, K in ((BIG, 16, 128), (16, BIG, 128), (16, 16, 2 ** 32 + 128)):
        a, b, s = _meta(M, K), _meta(N, K), _meta(1, 4, t=i32)
        for call in (lambda: dg.fp8_gemm_nt(a, s, b, s), lambda: dg.fp8_gemm_nt_ex(a, s, b, s),
                     lambda: dg.fp8_gemm("nn", a, s, _meta(K, N), s),
                     lambda: dg.m_grouped_fp8_gemm_nt_contiguous(a, s, b[None], s, _meta(M, t=i32)),
                     lambda: dg.m_grouped_fp8_gemm_nt_masked(a[None], s, b[None], s, _meta(1, t=i32))):
            with pytest.raises(ValueError, match="32 bits"):
                call()
    with pytest.raises(ValueError, match="32 bits"):
        dg.moe_permute(_meta(4, 2, t=i32), 2 ** 32 + 4, _meta(4, 128), s)
    with pytest.raises(ValueError, match="32 bits"):
        dg.describe_config("dense", 2 ** 32 + 64, 256, 256)
    for call in (lambda: dg.set_num_sms(2 ** 32 + 8), lambda: dg.set_tc_util(2 ** 32 + 50),
                 lambda: dg.set_config(2 ** 32 + 128)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_operands_of_another_device_than_the_current_one_are_refused(monkeypatch):
    monkeypatch.setattr(dg, "_current_device", lambda: 1)
    monkeypatch.setattr(dg, "_current_stream", lambda dev: 7 + dev)
    assert dg._launch_stream(1) == 8
    with pytest.raises(ValueError, match="cuda:0 but the current device is cuda:1"):
        dg._launch_stream(0)


def test_tiles_are_counted_at_the_ends_of_int(lib):
    """2^31 - 1 rows or 2^31 - 16 columns are millions of tiles: the grid must be as
    full as for a million rows (a sum beyond int had left none of them)."""
    most = 2 ** 31 - 1
    for ctas in (1, 2):
        assert lib.dg_set_config(128, ctas, 1) == 0
        try:
            for kind in ("int8_dense", "int8_contiguous", "int8_masked", "dense", "masked"):
                want = dg.describe_config(kind, 2 ** 20, 16, 128, 1)
                assert want.split("/")[1] == "148"
                assert dg.describe_config(kind, most, 16, 128, 1) == dg.describe_config(kind, 2 ** 24, 16, 128, 1)
                assert dg.describe_config(kind, 1, most - 15, 128, 1).split("/")[1] == "148"
        finally:
            assert lib.dg_set_config(0, 0, 0) == 0
    for kind in ("int8_dense", "int8_contiguous", "int8_masked"):
        assert dg.describe_config(kind, most, 7168, 2048, 4).split("/")[1] == "148"
        assert dg.describe_config(kind, 64, most - 15, 2048, 4).split("/")[1] == "148"


@pytest.mark.parametrize("sms", [1, 2, 3])
def test_few_sms_still_get_a_grid(lib, sms):
    """A CTA pair needs two SMs: with one, neither the heuristic nor a forced tile
    takes pairs (their grid would be empty), whatever the layout."""
    kinds = ["dense", "contiguous", "masked", "int8_dense", "int8_contiguous", "int8_masked"]
    prev = dg.set_num_sms(sms)
    try:
        for forced in [(0, 0, 0), (128, 2, 1), (256, 2, 1), (224, 2, 2), (256, 2, 0)]:
            assert lib.dg_set_config(*forced) == 0
            for kind in kinds:
                for M, N, K in ((128, 256, 256), (4096, 7168, 2048), (32768, 4096, 7168)):
                    tile, grid = dg.describe_config(kind, M, N, K, 8).split("/")
                    assert 1 <= int(grid) <= sms and (sms > 1 or "(2cta)" not in tile), (kind, M, forced)
    finally:
        assert lib.dg_set_config(0, 0, 0) == 0
        dg.set_num_sms(prev)


def test_int8_tile_choice(lib):
    """The heuristic is host logic (148 SMs assumed without a device): narrow
    1-CTA tiles for a few rows, pairs of CTAs for many, no pairs beyond the
    contiguous layout's table; a forced tile holds where it is built."""
    assert dg.describe_config("int8_dense", 64, 7168, 2048) == "128x64x8(2pipe)(splitk)/112"
    assert "(splitk)" not in dg.describe_config("int8_dense", 64, 7168, 128)      # one K block
    assert dg.describe_config("int8_dense", 4096, 7168, 2048).startswith("256x256x6(2cta)")
    assert dg.describe_config("int8_contiguous", 4096, 4096, 7168, 8).startswith("256x256x6(2cta)")
    assert dg.describe_config("int8_contiguous", 32768, 4096, 7168, 8) == "256x256x6(2cta)/148"
    assert "(2cta)" not in dg.describe_config("int8_contiguous", 1024 * 128 + 128, 4096, 7168, 8)
    assert dg.describe_config("int8_masked", 256, 7168, 2048, 16).startswith("128x256")
    assert lib.dg_set_config(128, 2, 1) == 0
    try:
        assert dg.describe_config("int8_dense", 64, 7168, 2048).startswith("256x128x8(2cta)")
        assert lib.dg_set_config(64, 1, 2) == 0
        assert "(splitk)" not in dg.describe_config("int8_dense", 64, 7168, 128)
        assert lib.dg_set_config(224, 2, 2) == 0          # not built for int8: the choice stands
        assert dg.describe_config("int8_dense", 64, 7168, 2048) == "128x64x8(2pipe)(splitk)/112"
    finally:
        assert lib.dg_set_config(0, 0, 0) == 0
