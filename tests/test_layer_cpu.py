"""Argument checks, plans and workspace sizes of the layer products, on the
CPU: every refusal comes before any device call (pointers are made up and
never followed), and a call that passes the checks here stops at the missing
device.  Also the generated code of their kernels: MFMA hazards, compiler
waits in the rings, scratch memory."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

from dense_gemm_08_amd import binding, build
from tests import test_codegen as codegen

S = binding.Status
NT_F16, NN_BF16, NT_BF16, NN_F16 = range(4)
SIZE = ctypes.c_size_t


def has_gpu():
    import torch
    return torch.cuda.is_available()


# on a machine with a GPU a call with made-up pointers must not get past its
# checks
accepted = pytest.mark.skipif(has_gpu(), reason="made-up pointers")


def layer(op=NT_BF16, M=64, N=48, K=32, A=256, lda=None, B=256, ldb=None, D=256, ldd=None, epi=None,
          groups=None, ws=None, nbytes=0):
    lib = binding.load_library()
    lda = K if lda is None else lda
    ldb = (K if op in (NT_F16, NT_BF16) else N) if ldb is None else ldb
    ldd = N if ldd is None else ldd
    return S(lib.dense_gemm_layer(op, M, N, K, A, lda, B, ldb, D, ldd, epi, groups, ws, nbytes, None))


def tn(fmt=1, M=64, N=48, K=32, A=256, lda=None, B=256, ldb=None, D=256, ldd=None, colsum=None,
       groups=None, ws=None, nbytes=0):
    lib = binding.load_library()
    return S(lib.dense_gemm_tn(fmt, M, N, K, A, M if lda is None else lda, B,
                               N if ldb is None else ldb, D, N if ldd is None else ldd, colsum,
                               groups, ws, nbytes, None))


def E(bias=None, bias_stride=0, residual=None, ldr=0, preact=None, ldz=0, act=0, grad=0):
    return binding.Epilogue(bias, bias_stride, residual, ldr, preact, ldz, act, grad)


def Gr(ends=256, count=4, stride=1 << 20):
    return binding.Groups(ends, count, stride)


@accepted
def test_accepted_calls_reach_the_device():
    for op in range(4):
        assert layer(op) == S.NO_DEVICE
        assert layer(op, epi=E(bias=256, act=4, residual=256, ldr=48, preact=256, ldz=50)) == S.NO_DEVICE
        assert layer(op, epi=E(preact=256, ldz=48, act=2, grad=1)) == S.NO_DEVICE
        assert layer(op, groups=Gr()) == S.NO_DEVICE
        assert layer(op, groups=Gr(stride=0)) == S.NO_DEVICE
        assert layer(op, K=0, A=None, B=None, lda=0, ldb=48) == S.NO_DEVICE
    for fmt in (0, 1):
        assert tn(fmt) == S.NO_DEVICE
        assert tn(fmt, colsum=256, groups=Gr()) == S.NO_DEVICE
        assert tn(fmt, K=0, A=None, B=None) == S.NO_DEVICE


def test_calls_with_nothing_to_do():
    assert layer(M=0, A=None, D=None) == S.OK
    assert layer(N=0, D=None) == S.OK
    assert layer(groups=Gr(ends=None, count=0)) == S.OK
    assert layer(M=0, groups=Gr(ends=None)) == S.OK
    assert tn(M=0, D=None) == S.OK
    assert tn(N=0, D=None) == S.OK
    assert tn(groups=Gr(ends=None, count=0)) == S.OK


def test_layer_refusals():
    assert layer(op=4) == S.BAD_ARG and layer(op=-1) == S.BAD_ARG
    assert layer(M=-1) == S.INVALID_DIM and layer(K=-1) == S.INVALID_DIM
    assert layer(A=None) == S.NULL_PTR and layer(B=None) == S.NULL_PTR and layer(D=None) == S.NULL_PTR
    assert layer(lda=31) == S.BAD_LD and layer(ldb=31) == S.BAD_LD and layer(ldd=47) == S.BAD_LD
    assert layer(A=255) == S.MISALIGNED and layer(D=257) == S.MISALIGNED
    assert layer(epi=E(act=5)) == S.BAD_ARG and layer(epi=E(act=-1)) == S.BAD_ARG
    assert layer(epi=E(act=1, grad=2, preact=256, ldz=48)) == S.BAD_ARG
    assert layer(epi=E(grad=1, preact=256, ldz=48)) == S.BAD_ARG          # no activation
    assert layer(epi=E(grad=1, act=1, preact=256, ldz=48, bias=256)) == S.BAD_ARG
    assert layer(epi=E(grad=1, act=1, preact=256, ldz=48, residual=256, ldr=48)) == S.BAD_ARG
    assert layer(epi=E(grad=1, act=1)) == S.NULL_PTR
    assert layer(epi=E(bias=257)) == S.MISALIGNED
    assert layer(epi=E(bias=256, bias_stride=-1)) == S.BAD_ARG
    assert layer(epi=E(residual=256, ldr=47)) == S.BAD_LD
    assert layer(epi=E(residual=257, ldr=48)) == S.MISALIGNED
    assert layer(epi=E(residual=256, ldr=1 << 31)) == S.TOO_LARGE
    assert layer(epi=E(preact=256, ldz=47)) == S.BAD_LD
    assert layer(epi=E(preact=256, ldz=1 << 40)) == S.TOO_LARGE


def test_group_refusals():
    for call in (layer, tn):
        assert call(groups=Gr(ends=None)) == S.NULL_PTR
        assert call(groups=Gr(ends=258)) == S.MISALIGNED
        assert call(groups=Gr(count=-1)) == S.INVALID_DIM
        assert call(groups=Gr(count=1 << 31)) == S.TOO_LARGE
        assert call(groups=Gr(stride=-8)) == S.BAD_ARG
        assert call(groups=Gr(count=1 << 20, stride=1 << 45)) == S.TOO_LARGE
        # sizes and tile numbers stay this far from 2^31: the kernels look past
        # the end in 32 bits
        dims = dict(M=1, N=1, K=1, lda=1 << 20, ldb=1 << 20, ldd=1 << 20)
        for d in "MNK":
            big = dict(dims, **{d: (1 << 31) - 1023}, groups=Gr(count=1))
            for ld in {"M": ["lda"] if call is tn else [], "N": ["ldb", "ldd"] if call is tn else ["ldd"],
                       "K": [] if call is tn else ["lda", "ldb"]}[d]:
                big[ld] = (1 << 31) - 1
            assert call(**big) == S.TOO_LARGE
    assert layer(groups=Gr(count=(1 << 20) + 1)) == S.TOO_LARGE
    assert tn(M=1, N=1, groups=Gr(count=(1 << 31) - (1 << 20) + 1, stride=1)) == S.TOO_LARGE
    # output tiles past 32-bit numbers
    big = (1 << 31) - 8
    assert layer(M=big, N=1024, ldd=1024, groups=Gr(count=big)) == S.TOO_LARGE
    assert tn(M=1 << 16, N=1 << 16, groups=Gr(count=1 << 16, stride=1 << 32)) == S.TOO_LARGE


def test_tn_refusals():
    assert tn(fmt=2) == S.BAD_ARG and tn(fmt=-1) == S.BAD_ARG
    assert tn(M=-1) == S.INVALID_DIM and tn(N=-2) == S.INVALID_DIM and tn(K=-1) == S.INVALID_DIM
    assert tn(N=0, colsum=256) == S.BAD_ARG
    assert tn(A=None) == S.NULL_PTR and tn(B=None) == S.NULL_PTR and tn(D=None) == S.NULL_PTR
    assert tn(lda=63) == S.BAD_LD and tn(ldb=47) == S.BAD_LD and tn(ldd=47) == S.BAD_LD
    assert tn(A=257) == S.MISALIGNED and tn(B=257) == S.MISALIGNED and tn(D=257) == S.MISALIGNED
    assert tn(colsum=257) == S.MISALIGNED
    assert tn(M=1 << 31, lda=1 << 31) == S.TOO_LARGE and tn(lda=1 << 31) == S.TOO_LARGE
    assert tn(lda=1 << 25) == S.TOO_LARGE  # the rows of one K step span 2^31 bytes
    assert tn(ldd=1 << 31) == S.TOO_LARGE
    # the groups' outputs would overlap
    assert tn(groups=Gr(stride=63 * 48 + 47)) == S.BAD_LD


def layer_bytes(op, M, N, K, A=256, lda=None, B=256, ldb=None, groups=None, cus=256):
    out = SIZE()
    lda = K if lda is None else lda
    ldb = (K if op in (NT_F16, NT_BF16) else N) if ldb is None else ldb
    st = binding.load_library().dense_gemm_layer_workspace_size(op, M, N, K, A, lda, B, ldb, groups,
                                                                cus, ctypes.byref(out))
    assert S(st) == S.OK
    return out.value


def tn_bytes(M, N, K, A=256, lda=None, B=256, ldb=None, groups=None, cus=256, colsum=0):
    out = SIZE()
    st = binding.load_library().dense_gemm_tn_workspace_size(
        M, N, K, A, M if lda is None else lda, B, N if ldb is None else ldb, colsum, groups,
        cus, ctypes.byref(out))
    assert S(st) == S.OK
    return out.value


def up256(n):
    return (n + 255) // 256 * 256


def test_layer_workspace():
    for op in range(4):
        # the small-output kernel, and whole tiles of either size
        assert layer_bytes(op, 1, 4096, 4096) == 0
        assert layer_bytes(op, 2048, 2048, 2048) == 0
        assert layer_bytes(op, 4096, 4096, 4096) == 0
        # few tiles, long K: 128 x 128 partial tiles, at most one per CU
        n = layer_bytes(op, 256, 128, 8192)
        assert n % (128 * 128 * 4) == 0 and 4 <= n // (128 * 128 * 4) <= 256
        # a last wave of 256 x 256 tiles in parts, as in the plain product
        layout, fmt = {v: k for k, v in binding.OPS.items()}[op]
        assert layer_bytes(op, 4096, 4352, 4096) == binding.workspace_size(
            layout, fmt, 4096, 4352, 4096, 256, 4096, 256, 4096 if layout == "nt" else 4352,
            num_cus=256) > 0
        # rows of whole words at 4 bytes are read in place
        assert layer_bytes(op, 300, 304, 80, A=260, lda=82, B=268, ldb=306) == 0
        assert layer_bytes(op, 300, 304, 82) == 0
        # (by the small-output kernel with K a multiple of 8)
        assert layer_bytes(op, 8, 304, 82) == up256(8 * 88 * 2) + (
            up256(304 * 88 * 2) if op in (NT_F16, NT_BF16) else 0)
        # operands off 4 bytes, copied
        assert layer_bytes(op, 300, 304, 80, A=258) == up256(300 * 80 * 2)
        assert layer_bytes(op, 300, 304, 80, B=258) == up256(304 * 80 * 2)


def test_grouped_workspace_holds_the_repacked_operands():
    assert layer_bytes(NT_BF16, 500, 64, 128, groups=Gr(count=7, stride=64 * 128)) == 0
    # K off 8: both operands
    assert layer_bytes(NT_BF16, 500, 64, 129, groups=Gr(count=7, stride=64 * 129)) == \
        up256(500 * 136 * 2) + up256(7 * 64 * 136 * 2)
    # a distance between the matrices off 8 elements: B alone
    assert layer_bytes(NT_BF16, 500, 64, 128, groups=Gr(count=7, stride=64 * 128 + 1)) == \
        up256(7 * 64 * 128 * 2)
    assert layer_bytes(NT_BF16, 500, 64, 128, groups=Gr(count=7, stride=64 * 128 + 2)) == 0
    assert layer_bytes(NN_F16, 500, 66, 128, groups=Gr(count=7, stride=128 * 66)) == 0
    # A @ B with an odd N: B alone
    assert layer_bytes(NN_F16, 500, 65, 128, groups=Gr(count=7, stride=128 * 65)) == \
        up256(7 * 128 * 72 * 2)


def test_tn_workspace():
    assert tn_bytes(4096, 4096, 4096) == 0
    assert tn_bytes(4096, 4096, 4096, A=258) == 4096 * 4096 * 2
    assert tn_bytes(4098, 4094, 64, A=260) == 0
    assert tn_bytes(4097, 4096, 64) == up256(64 * 4104 * 2)
    # few tiles, long K: 128 x 128 partial tiles, at most one per CU
    n = tn_bytes(256, 512, 65536)
    per = 128 * 128 * 4
    assert n % per == 0 and 8 < n // per <= 256
    # groups, split for their average length
    n = tn_bytes(256, 256, 65536, groups=Gr(count=4))
    assert n % per == 0 and 16 < n // per <= 256
    assert tn_bytes(256, 256, 512, groups=Gr(count=300)) == 0
    # a last wave of 256 x 256 tiles (16 of 272) in parts
    n = tn_bytes(4096, 4352, 4096)
    parts = n // (256 * 256 * 4)
    assert n % (256 * 256 * 4) == 0 and 16 < parts <= 256
    # column sums: two rows of a tile's columns per task (256 whole tiles and
    # those parts)
    assert tn_bytes(4096, 4352, 4096, colsum=1) == n + (256 + parts) * 2 * 256 * 4
    # sizes near the limits plan without overflow on any device
    for cus in (1, 256, 1 << 30):
        tn_bytes((1 << 22) - 8, (1 << 22) - 8, (1 << 31) - 1024, cus=cus)


def test_size_queries_refuse_bad_arguments():
    lib = binding.load_library()
    out = SIZE()
    assert lib.dense_gemm_layer_workspace_size(0, 8, 8, 8, 256, 8, 256, 8, None, 256, None) == S.BAD_ARG
    assert lib.dense_gemm_layer_workspace_size(9, 8, 8, 8, 256, 8, 256, 8, None, 256,
                                               ctypes.byref(out)) == S.BAD_ARG
    assert lib.dense_gemm_layer_workspace_size(0, 8, 8, 8, 256, 8, 256, 8, None, -1,
                                               ctypes.byref(out)) == S.BAD_ARG
    assert lib.dense_gemm_layer_workspace_size(0, 8, 8, 8, 256, 8, 256, 8, Gr(count=-1), 256,
                                               ctypes.byref(out)) == S.INVALID_DIM
    assert lib.dense_gemm_tn_workspace_size(8, 8, 8, 256, 7, 256, 8, 0, None, 256,
                                            ctypes.byref(out)) == S.BAD_LD
    assert lib.dense_gemm_tn_workspace_size(8, 8, 8, 256, 8, 256, 8, 0, None, 256, None) == S.BAD_ARG


def test_python_entry_points_refuse_host_tensors():
    import torch
    import dense_gemm_08_amd as dg
    A = torch.zeros((4, 8), dtype=torch.bfloat16)
    for call in (lambda: dg.gemm_nt_fused(A, A), lambda: dg.gemm_tn(A, A),
                 lambda: dg.gemm_nn_dact(A, A, A, "silu"),
                 lambda: dg.gemm_nt_grouped(A, A[None], torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        dg.gemm_tn(A.float(), A.float())


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_planning_under_sanitizers(tmp_path):
    here = os.path.dirname(os.path.abspath(__file__))
    csrc = os.path.join(os.path.dirname(here), "dense_gemm_08_amd", "csrc")
    exe = str(tmp_path / "layer_fuzz")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-g", "-O1",
                    "-I", os.path.join(os.path.dirname(here), "include"), "-I", csrc,
                    os.path.join(here, "layer_fuzz.cpp"), os.path.join(csrc, "plan.cpp"),
                    os.path.join(csrc, "plan_layer.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.startswith("planned"), r.stdout + r.stderr[-4000:]


# ---- generated code -------------------------------------------------------------

@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src", ["layer.hip", "grouped.hip", "tn.hip"])
def test_generated_code_of_the_layer_kernels(src, tmp_path):
    asm = codegen.compile_asm(src, str(tmp_path / (src + ".s")))
    bad = codegen.check(asm)
    assert not bad, "\n".join(bad[:20])
    # no kernel spills to scratch memory
    sizes = re.findall(r"^; ScratchSize: (\d+)", asm, re.M)
    assert sizes and set(sizes) == {"0"}, sizes
    # the ring loops (a block of MFMAs that reaches itself through at most two
    # others) hold no memory wait of the compiler's
    found = 0
    for name, items in codegen.gemm_functions(asm).items():
        blocks, succ, _ = codegen.cfg([(label, ins) for label, ins, _ in items])
        flags = iter([a for label, _, a in items if label is None])
        own = [[next(flags) for _ in ins] for ins in blocks]

        def ring(b):
            """The blocks of the shortest cycle through block b, if it has at
            most three."""
            paths = [[s] for s in succ[b]]
            for _ in range(3):
                for p in paths:
                    if p[-1] == b:
                        return p
                paths = [p + [s] for p in paths for s in succ[p[-1]]]
            return []

        for b, ins in enumerate(blocks):
            if not any(codegen.is_mfma(i) for i in ins):
                continue
            cycle = ring(b)
            found += bool(cycle)
            for c in cycle:
                for i, a in zip(blocks[c], own[c]):
                    assert a or not (i.startswith("s_waitcnt") and "vmcnt" in i), (name, i)
    assert found > 0
