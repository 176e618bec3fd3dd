"""Argument checks, plans and generated code of the int8 products and of what
stands around an expert layer's products, on the CPU: every refusal comes before
any device call (pointers are made up and never followed), and a call that passes
the checks here stops at the missing device."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

from dense_gemm_08_amd import binding, build
from tests import test_codegen as codegen
from tests import test_layer_cpu as layer_cpu
from tests.test_layer_cpu import E, Gr, S, SIZE, accepted

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "dense_gemm_08_amd", "csrc")
F16, BF16, F32 = 0, 1, 2


def lib():
    return binding.load_library()


def i8(fmt=BF16, M=64, N=48, K=32, A=256, lda=None, SA=256, B=256, ldb=None, SB=256, sb_stride=0, D=256,
       ldd=None, epi=None, groups=None, ws=None, nbytes=0):
    return S(lib().dense_gemm_i8(fmt, M, N, K, A, K if lda is None else lda, SA, B, K if ldb is None else ldb,
                                 SB, sb_stride, D, N if ldd is None else ldd, epi, groups, ws, nbytes, None))


def i8_bytes(M, N, K, A=256, lda=None, B=256, ldb=None, groups=None, cus=256):
    out = SIZE(7)
    st = lib().dense_gemm_i8_workspace_size(M, N, K, A, K if lda is None else lda, B, K if ldb is None else ldb,
                                            groups, cus, ctypes.byref(out))
    assert S(st) == S.OK, S(st)
    return out.value


def quantize(fmt=BF16, R=8, K=32, X=256, ldx=None, x_rows=8, rows=None, Q=256, ldq=None, Sc=256):
    return S(lib().dense_gemm_quantize_i8(fmt, R, K, X, K if ldx is None else ldx, x_rows, rows, Q,
                                          K if ldq is None else ldq, Sc, None))


def routing(bias=None, score=0, renorm=1, scale=1.0, groups=1, top_groups=1, group_top=1):
    return binding.Routing(bias, score, renorm, scale, groups, top_groups, group_top)


def route(fmt=F32, T=8, E=16, k=2, logits=256, ldl=None, r=None, weights=256, experts=256, places=256,
          ends=256, tokens=256, ws=None, nbytes=0, **kw):
    r = routing(**kw) if r is None else r
    return S(lib().dense_gemm_route(fmt, T, E, k, logits, E if ldl is None else ldl, r, weights, experts, places,
                                    ends, tokens, ws, nbytes, None))


def route_grad(fmt=F32, T=8, E=16, k=2, logits=256, ldl=None, r=None, experts=256, dweights=256, dlogits=256,
               ldd=None, **kw):
    r = routing(**kw) if r is None else r
    return S(lib().dense_gemm_route_grad(fmt, T, E, k, logits, E if ldl is None else ldl, r, experts, dweights,
                                         dlogits, E if ldd is None else ldd, None))


def combine(fmt=BF16, T=8, N=32, k=2, H=256, ldh=None, h_rows=16, places=256, weights=256, residual=None,
            ldr=0, Y=256, ldy=None):
    return S(lib().dense_gemm_combine(fmt, T, N, k, H, N if ldh is None else ldh, h_rows, places, weights,
                                      residual, ldr, Y, N if ldy is None else ldy, None))


def combine_grad(fmt=BF16, T=8, N=32, k=2, DY=256, lddy=None, H=256, ldh=None, h_rows=16, places=256,
                 weights=256, DH=256, lddh=None, dweights=256):
    return S(lib().dense_gemm_combine_grad(fmt, T, N, k, DY, N if lddy is None else lddy, H,
                                           N if ldh is None else ldh, h_rows, places, weights, DH,
                                           N if lddh is None else lddh, dweights, None))


@accepted
def test_accepted_calls_reach_the_device():
    for fmt in (F16, BF16):
        assert i8(fmt) == S.NO_DEVICE
        assert i8(fmt, A=257, B=259, lda=33, ldb=35) == S.NO_DEVICE      # any address
        assert i8(fmt, K=0, A=None, B=None) == S.NO_DEVICE
        assert i8(fmt, K=131071, lda=131072, ldb=131072) == S.NO_DEVICE
        assert i8(fmt, epi=E(bias=256, act=4, residual=256, ldr=48, preact=256, ldz=50)) == S.NO_DEVICE
        assert i8(fmt, groups=Gr(), sb_stride=48) == S.NO_DEVICE
        assert quantize(fmt) == S.NO_DEVICE
        assert quantize(fmt, rows=256, R=9, Q=257, ldq=33, X=258, ldx=33) == S.NO_DEVICE
        assert quantize(fmt, K=0, X=None, Q=None) == S.NO_DEVICE         # the scales are still written
        assert quantize(fmt, rows=256, x_rows=0, X=None) == S.NO_DEVICE
        assert combine(fmt) == S.NO_DEVICE
        assert combine(fmt, weights=None, residual=256, ldr=32, h_rows=0, H=None) == S.NO_DEVICE
        assert combine_grad(fmt) == S.NO_DEVICE
        assert combine_grad(fmt, dweights=None, H=None) == S.NO_DEVICE
        assert combine_grad(fmt, DH=None, weights=None) == S.NO_DEVICE
    for fmt in (F16, BF16, F32):
        assert route(fmt) == S.NO_DEVICE
        assert route(fmt, T=0, logits=None, weights=None, experts=None, places=None, tokens=None) == S.NO_DEVICE
        assert route(fmt, E=1024, k=64, groups=64, top_groups=4, group_top=2, bias=256) == S.NO_DEVICE
        assert route_grad(fmt, score=1, renorm=0) == S.NO_DEVICE


def test_calls_with_nothing_to_do():
    assert i8(M=0, A=None, D=None, SA=None) == S.OK
    assert i8(N=0, D=None) == S.OK
    assert i8(groups=Gr(ends=None, count=0), A=None, B=None, SA=None, SB=None) == S.OK
    assert quantize(R=0, X=None, Q=None, Sc=None) == S.OK
    assert combine(T=0, H=None, places=None, Y=None) == S.OK
    assert combine(N=0, H=None, places=None, Y=None) == S.OK
    assert combine_grad(T=0, DY=None, places=None) == S.OK
    assert combine_grad(N=0, dweights=None, DY=None) == S.OK
    assert route_grad(T=0, logits=None, experts=None, dweights=None, dlogits=None) == S.OK


def test_i8_refusals():
    assert i8(fmt=2) == S.BAD_ARG and i8(fmt=-1) == S.BAD_ARG
    assert i8(M=-1) == S.INVALID_DIM and i8(N=-1) == S.INVALID_DIM and i8(K=-1) == S.INVALID_DIM
    for p in ("A", "B", "D", "SA", "SB"):
        assert i8(**{p: None}) == S.NULL_PTR
    assert i8(lda=31) == S.BAD_LD and i8(ldb=31) == S.BAD_LD and i8(ldd=47) == S.BAD_LD
    assert i8(D=257) == S.MISALIGNED and i8(SA=258) == S.MISALIGNED and i8(SB=257) == S.MISALIGNED
    assert i8(K=131072) == S.TOO_LARGE                      # a sum could pass 32 bits
    assert i8(lda=1 << 31) == S.TOO_LARGE and i8(ldb=1 << 24) == S.TOO_LARGE  # 255 rows span 2^31
    assert i8(M=1 << 31) == S.TOO_LARGE
    assert i8(epi=E(act=5)) == S.BAD_ARG
    assert i8(epi=E(act=1, grad=1, preact=256, ldz=48)) == S.BAD_ARG    # no gradient form
    assert i8(epi=E(bias=257)) == S.MISALIGNED
    assert i8(epi=E(residual=256, ldr=47)) == S.BAD_LD
    assert i8(epi=E(preact=256, ldz=1 << 31)) == S.TOO_LARGE
    assert i8(groups=Gr(), sb_stride=-1) == S.BAD_ARG
    assert i8(groups=Gr(stride=-1)) == S.BAD_ARG
    assert i8(groups=Gr(ends=None)) == S.NULL_PTR
    assert i8(groups=Gr(ends=258)) == S.MISALIGNED
    assert i8(groups=Gr(count=-1)) == S.INVALID_DIM
    assert i8(groups=Gr(count=(1 << 20) + 1)) == S.TOO_LARGE


def test_i8_workspace():
    # aligned rows of whole words are read in place: only split products need memory
    assert i8_bytes(4096, 4096, 4096) == 0
    assert i8_bytes(16, 4096, 4096) == 0
    # small outputs take any K, rows off 4 bytes are copied (16 bytes a piece, 256 a copy)
    assert i8_bytes(16, 4096, 4093, lda=4096, ldb=4096) == 0
    assert i8_bytes(16, 4096, 4096, A=257) == 16 * 4096
    assert i8_bytes(16, 4096, 100, lda=101) == 7 * 256      # 16 rows of 112 bytes
    # the tiled kernels copy both operands off whole words
    assert i8_bytes(4096, 4096, 4095) == 2 * 4096 * 4096
    assert i8_bytes(4096, 4096, 4096, lda=4098) == 4096 * 4096
    g = binding.Groups(256, 8, 4096 * 1002)
    assert i8_bytes(4096, 4096, 1000, groups=g) == 0
    g = binding.Groups(256, 8, 4096 * 1000 + 2)
    assert i8_bytes(4096, 4096, 1000, groups=g) == 8 * 4096 * 1008
    # one matrix for all groups is copied once
    assert i8_bytes(4096, 4096, 1001, groups=binding.Groups(256, 8, 0)) == 2 * 4096 * 1008
    out = SIZE()
    f = lib().dense_gemm_i8_workspace_size
    assert S(f(8, 8, 8, 256, 8, 256, 8, None, 256, None)) == S.BAD_ARG
    assert S(f(8, 8, 8, 256, 8, 256, 8, None, -1, ctypes.byref(out))) == S.BAD_ARG
    assert S(f(8, 8, 8, 256, 7, 256, 8, None, 256, ctypes.byref(out))) == S.BAD_LD
    if not layer_cpu.has_gpu():
        assert S(f(8, 8, 8, 256, 8, 256, 8, None, 0, ctypes.byref(out))) == S.NO_DEVICE


def test_quantize_refusals():
    assert quantize(fmt=2) == S.BAD_ARG and quantize(fmt=-1) == S.BAD_ARG
    assert quantize(R=-1) == S.INVALID_DIM and quantize(K=-1) == S.INVALID_DIM
    assert quantize(x_rows=-1) == S.INVALID_DIM
    assert quantize(R=9) == S.BAD_ARG                       # more rows than X has, without an index
    for p in ("X", "Q", "Sc"):
        assert quantize(**{p: None}) == S.NULL_PTR
    assert quantize(ldx=31) == S.BAD_LD and quantize(ldq=31) == S.BAD_LD
    assert quantize(X=257) == S.MISALIGNED and quantize(Sc=258) == S.MISALIGNED
    assert quantize(rows=257) == S.MISALIGNED
    assert quantize(R=1 << 31, x_rows=1 << 31) == S.TOO_LARGE
    assert quantize(K=1 << 31) == S.TOO_LARGE and quantize(ldq=1 << 31) == S.TOO_LARGE


def test_route_refusals():
    assert route(fmt=3) == S.BAD_ARG and route(fmt=-1) == S.BAD_ARG
    assert S(lib().dense_gemm_route(F32, 8, 16, 2, 256, 16, None, 256, 256, 256, 256, 256, None, 0,
                                    None)) == S.BAD_ARG
    assert route(T=-1) == S.INVALID_DIM and route(E=-1) == S.INVALID_DIM and route(k=-1) == S.INVALID_DIM
    assert route(E=0) == S.BAD_ARG and route(k=0) == S.BAD_ARG and route(k=17) == S.BAD_ARG
    assert route(E=1025) == S.TOO_LARGE and route(E=128, k=65) == S.TOO_LARGE
    # T k stays 2^20 below 2^31
    assert route(T=(1 << 31) - (1 << 20) + 1, k=1) == S.TOO_LARGE and route(T=1 << 30) == S.TOO_LARGE
    assert route(score=2) == S.BAD_ARG and route(renorm=2) == S.BAD_ARG
    for kw in (dict(groups=0), dict(groups=3), dict(groups=4, top_groups=0), dict(groups=4, top_groups=5),
               dict(groups=4, top_groups=2, group_top=0), dict(groups=4, top_groups=2, group_top=3),
               dict(groups=128, top_groups=128, E=128), dict(groups=8, top_groups=1, k=3)):
        assert route(**kw) == S.BAD_ARG, kw
    for p in ("logits", "weights", "experts", "places", "ends", "tokens"):
        assert route(**{p: None}) == S.NULL_PTR
        assert route(**{p: 258}) == S.MISALIGNED
    assert route(fmt=BF16, logits=257) == S.MISALIGNED
    assert route(bias=258) == S.MISALIGNED
    assert route(ldl=15) == S.BAD_LD and route(ldl=1 << 31) == S.TOO_LARGE
    assert route_grad(fmt=3) == S.BAD_ARG and route_grad(k=17) == S.BAD_ARG
    assert route_grad(score=-1) == S.BAD_ARG
    for p in ("logits", "experts", "dweights", "dlogits"):
        assert route_grad(**{p: None}) == S.NULL_PTR
        assert route_grad(**{p: 258}) == S.MISALIGNED
    assert route_grad(ldd=15) == S.BAD_LD and route_grad(ldl=15) == S.BAD_LD


def route_bytes(T, E, k):
    out = SIZE(7)
    assert S(lib().dense_gemm_route_workspace_size(T, E, k, ctypes.byref(out))) == S.OK
    return out.value


def test_route_workspace():
    assert route_bytes(0, 64, 2) == 0 and route_bytes(128, 1024, 64) == 0
    assert route_bytes(129, 64, 2) == 512                   # 3 blocks of 64 tokens, 32 words each
    assert route_bytes(16384, 256, 8) == 256 * 256 * 2
    assert route_bytes(40000, 7, 2) == 313 * 4 * 4 // 256 * 256 + 256   # 2 chunks a block
    assert lib().dense_gemm_route_workspace_size(8, 8, 2, None) == S.BAD_ARG
    assert lib().dense_gemm_route_workspace_size(8, 0, 2, ctypes.byref(SIZE())) == S.BAD_ARG


def test_combine_refusals():
    for call in (combine, combine_grad):
        assert call(fmt=2) == S.BAD_ARG
        assert call(T=-1) == S.INVALID_DIM and call(N=-1) == S.INVALID_DIM
        assert call(k=-1) == S.INVALID_DIM and call(h_rows=-1) == S.INVALID_DIM
        assert call(k=0) == S.BAD_ARG and call(k=65) == S.TOO_LARGE
        assert call(T=1 << 30, k=2) == S.TOO_LARGE and call(N=1 << 31) == S.TOO_LARGE
        assert call(h_rows=1 << 31) == S.TOO_LARGE
        assert call(places=None) == S.NULL_PTR and call(places=258) == S.MISALIGNED
        assert call(weights=257) == S.MISALIGNED
        assert call(H=None) == S.NULL_PTR and call(H=257) == S.MISALIGNED and call(ldh=31) == S.BAD_LD
    assert combine(Y=None) == S.NULL_PTR and combine(Y=257) == S.MISALIGNED and combine(ldy=31) == S.BAD_LD
    assert combine(residual=257, ldr=32) == S.MISALIGNED and combine(residual=256, ldr=31) == S.BAD_LD
    assert combine(ldy=1 << 31) == S.TOO_LARGE
    assert combine_grad(DY=None) == S.NULL_PTR and combine_grad(lddy=31) == S.BAD_LD
    assert combine_grad(DH=257) == S.MISALIGNED and combine_grad(lddh=31) == S.BAD_LD
    assert combine_grad(dweights=258) == S.MISALIGNED
    assert combine_grad(DH=None, dweights=None) == S.BAD_ARG
    assert combine_grad(N=0) == S.BAD_ARG                   # dweights of nothing


def test_python_entry_points_refuse_host_tensors():
    import torch
    import dense_gemm_08_amd as dg
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    q, s, i = torch.zeros((4, 8), dtype=torch.int8), torch.zeros(4), torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: dg.gemm_nt_i8(q, s, q, s), lambda: dg.quantize_rows(x), lambda: dg.route(x, 2),
                 lambda: dg.gemm_nt_i8_grouped(q, s, q[None], s[None], i[:1, 0]),
                 lambda: dg.route_grad(x, i, torch.zeros(4, 2)), lambda: dg.combine_rows(x, i),
                 lambda: dg.combine_rows_grad(x, x, i)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dg.gemm_nt_i8(x, s, x, s), lambda: dg.quantize_rows(q), lambda: dg.route(q, 2),
                 lambda: dg.combine_rows(q, i)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_planning_under_sanitizers(tmp_path):
    exe = str(tmp_path / "experts_fuzz")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-g", "-O1", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(HERE, "experts_fuzz.cpp"), os.path.join(CSRC, "plan.cpp"),
                    os.path.join(CSRC, "plan_layer.cpp"), os.path.join(CSRC, "plan_experts.cpp"), "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.startswith("planned"), r.stdout + r.stderr[-4000:]


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not available")
def test_generated_code_of_the_int8_kernels(tmp_path):
    # MFMA operands kept apart, no compiler waits in the rings, no scratch memory
    layer_cpu.test_generated_code_of_the_layer_kernels("i8.hip", tmp_path)


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not available")
def test_row_kernels_use_no_scratch_memory(tmp_path):
    asm = codegen.compile_asm("rows.hip", str(tmp_path / "rows.s"))
    sizes = re.findall(r"^; ScratchSize: (\d+)", asm, re.M)
    assert len(sizes) >= 18 and set(sizes) == {"0"}, sizes
