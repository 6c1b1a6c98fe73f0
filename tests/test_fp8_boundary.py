"""The 8-bit products and the mixture of experts without a GPU: the library
exports what include/fp8_ops.h declares, the Python structures have the header's
layout, bad arguments are refused with the documented status codes before any
HIP call, and the workspace queries answer."""
import ctypes
import os
import re
import shutil
import struct
import subprocess

import pytest
import torch

import dense_gemm_elementwise_amd as ge
from dense_gemm_elementwise_amd import binding, fp8, operators

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TEXT = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8_ops.h")).read(), flags=re.S)

P = 0x7F0000001000  # a fake device address: never dereferenced by the checks under test
F16, BF16, F32 = 0, 1, 2
SHAPE, NULL_IN, NULL_OUT, KIND, ALIGN, WORKSPACE, DTYPE = 1, 2, 3, 4, 5, 7, 8


def fields(name):
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", TEXT).group(1)
    names = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        for n in re.sub(r"^(const )?(int64_t|void|float) ?\*?", "", decl).split(","):
            names.append(n.strip().lstrip("*"))
    return names


class Call:
    def __init__(self, name, **defaults):
        self.name, self.defaults, self.names = name, defaults, fields(name + "_args")

    def pack(self, **kw):
        v = {n: 0 for n in self.names}
        v.update(self.defaults)
        for k, x in kw.items():
            assert k in v, k
            v[k] = x
        return struct.pack(f"@{len(self.names)}q", *(v[n] for n in self.names))

    def run(self, **kw):
        return fp8._functions()[self.name](self.pack(**kw))

    def workspace(self, **kw):
        return fp8.workspace_bytes(self.name, self.pack(**kw))


QUANT = Call("ge_quantize_fp8", R=300, C=200, X=P, ldx=200, Q=P, ldq=208, S=P, lds=4, QT=P, ldqt=304, ST=P, ldst=4,
             block=0, format=0, dtype=F32)
LINEAR = Call("ge_linear_fp8", M=300, N=96, K=200, X=P, ldx=208, XS=P, ldxs=4, W=P, ldw=208, WS=P, ldws=4, bias=P,
              residual=P, ldr=96, D=P, ldd=96, Z=P, ldz=96, act=2, dtype=BF16, format=0)
LINEAR_B = Call("ge_linear_fp8_backward", M=300, N=96, K=200, dD=P, lddd=96, XT=P, ldxt=304, XTS=P, ldxts=4, WT=P,
                ldwt=96, WTS=P, ldwts=4, Z=P, ldz=96, dX=P, lddx=200, dW=P, lddw=200, dbias=P, act=2, dtype=F16,
                format=1)
MOE = Call("ge_moe", T=5, hidden=200, experts=6, inner=72, top_k=2, X=P, ldx=200, Wr=P, ldwr=200, Up=P, ldu=200,
           up_stride=144 * 200, Down=P, lddn=72, down_stride=200 * 72, residual=P, ldr=200, D=P, ldd=200, act=3,
           gated=1, renormalize=1, dtype=BF16)
MOE8 = dict(US=P, ldus=2, us_stride=4, DS=P, ldds=1, ds_stride=2)
CALLS = (QUANT, LINEAR, LINEAR_B, MOE)


def test_library_exports_every_declared_function():
    names = set(re.findall(r"\bint (ge_[a-z_0-9]+)\(", TEXT))
    assert names == set(fp8.FP8_EXPORTS) | set(fp8._WORKSPACE.values())
    raw = ctypes.CDLL(binding.LIB_PATH)
    for n in names:
        assert hasattr(raw, n), n


def test_python_structures_match_the_header():
    heads = {"ge_quantize_fp8": fp8._QUANTIZE, "ge_linear_fp8": fp8._LINEAR8,
             "ge_linear_fp8_backward": fp8._LINEAR8_GRAD, "ge_moe": fp8._MOE}
    for name, head in heads.items():
        tail = operators._STREAM if name == "ge_quantize_fp8" else operators._TAIL
        assert head.size + tail.size == 8 * len(fields(name + "_args")), name


def test_enums_match_the_header():
    for name, val in fp8.FORMATS.items():
        assert re.search(rf"GE_FP8_{name.upper()} = {val}\b", TEXT)
    for name, val in fp8.BLOCKS.items():
        assert re.search(rf"GE_BLOCK_{name.upper()} = {val}\b", TEXT)


def test_header_is_plain_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    checks = "\n".join(f"typedef char size_{c.name}[sizeof({c.name}_args) == 8 * {len(c.names)} ? 1 : -1];"
                       for c in CALLS)
    src = tmp_path / "header.c"
    src.write_text(f'#include "fp8_ops.h"\n{checks}\nint main(void) {{ return 0; }}\n')
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                    os.path.join(ROOT, "include"), str(src)], check=True)


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.name)
def test_null_structures_and_types(call):
    assert fp8._functions()[call.name](None) == NULL_IN
    for bad in (-1, 3) + ((2,) if call is not QUANT else ()):
        assert call.run(dtype=bad) == DTYPE
    if "format" in call.names:
        for bad in (-1, 2):
            assert call.run(format=bad) == DTYPE
    if "act" in call.names:
        for bad in (-1, 4):
            assert call.run(act=bad) == KIND


def test_quantize_refusals():
    for f in ("R", "C"):
        assert QUANT.run(**{f: -1}) == SHAPE and QUANT.run(**{f: 2097001}) == SHAPE
    assert QUANT.run(C=0) == SHAPE
    assert QUANT.run(block=2) == KIND and QUANT.run(block=-1) == KIND
    for f in ("ldx", "ldq", "lds", "ldqt", "ldst"):
        assert QUANT.run(**{f: {"ldx": 199, "ldq": 199, "lds": 1, "ldqt": 299, "ldst": 2}[f]}) == SHAPE, f
    assert QUANT.run(X=0) == NULL_IN and QUANT.run(Q=0) == NULL_OUT and QUANT.run(S=0) == NULL_OUT
    assert QUANT.run(QT=0) == NULL_OUT and QUANT.run(ST=0) == NULL_OUT  # both or none
    assert QUANT.run(X=P + 2) == ALIGN and QUANT.run(X=P + 1, dtype=F16) == ALIGN
    assert QUANT.run(R=0, X=0, Q=0, S=0, QT=0, ST=0) == 0


def test_linear_refusals():
    for f in ("M", "N", "K"):
        assert LINEAR.run(**{f: -1}) == SHAPE and LINEAR.run(**{f: 2 ** 31}) == SHAPE
    assert LINEAR.run(N=0) == SHAPE and LINEAR.run(K=0) == SHAPE and LINEAR.run(K=2097001) == SHAPE
    for f, v in (("ldx", 199), ("ldxs", 1), ("ldw", 199), ("ldws", 1), ("ldr", 95), ("ldd", 95), ("ldz", 95)):
        assert LINEAR.run(**{f: v}) == SHAPE, f
    assert LINEAR.run(X=0) == NULL_IN and LINEAR.run(W=0) == NULL_IN and LINEAR.run(WS=0) == NULL_IN
    assert LINEAR.run(D=0) == NULL_OUT
    for f in ("bias", "residual", "D", "Z"):
        assert LINEAR.run(**{f: P + 1}) == ALIGN, f
    assert LINEAR.run(XS=0, X=P + 1) == ALIGN  # 16-bit x
    assert LINEAR.run(M=0, X=0, XS=0, D=0, residual=0, Z=0) == 0


def test_linear_backward_refusals():
    assert LINEAR_B.run(dX=0, dW=0, dbias=0) == NULL_OUT
    assert LINEAR_B.run(dD=0) == NULL_IN and LINEAR_B.run(Z=0) == NULL_IN
    assert LINEAR_B.workspace(Z=0, act=0)[0] == 0
    for f in ("XT", "XTS", "WT", "WTS"):
        assert LINEAR_B.run(**{f: 0}) == NULL_IN, f
    assert LINEAR_B.workspace(XT=0, XTS=0, dW=0)[0] == 0  # only dW reads X, only dX reads W
    assert LINEAR_B.workspace(WT=0, WTS=0, dX=0)[0] == 0
    for f, v in (("ldxt", 299), ("ldxts", 2), ("ldwt", 95), ("ldwts", 0), ("lddx", 199), ("lddw", 199), ("lddd", 95)):
        assert LINEAR_B.run(**{f: v}) == SHAPE, f
    assert LINEAR_B.run(M=2097001, ldxt=2097008) == SHAPE  # a row of X^T
    assert LINEAR_B.run(dbias=P + 2) == ALIGN and LINEAR_B.run(dX=P + 1) == ALIGN and LINEAR_B.run(dW=P + 1) == ALIGN
    assert LINEAR_B.run(M=0, dX=0, dW=0, dbias=0) == 0


def test_moe_refusals():
    for f, bad in (("T", (-1, 2 ** 31)), ("hidden", (0, 2097001)), ("inner", (0, 1048501)), ("experts", (0, 1025)),
                   ("top_k", (0, 7, 33)), ("ldx", (199,)), ("ldwr", (199,)), ("ldu", (199,)), ("lddn", (71,)),
                   ("up_stride", (143 * 200 + 199,)), ("down_stride", (199 * 72 + 71,)), ("ldr", (199,)),
                   ("ldd", (199,))):
        for v in bad:
            assert MOE.run(**{f: v}) == SHAPE, (f, v)
    assert MOE.run(experts=64, top_k=33, up_stride=10 ** 6, down_stride=10 ** 6) == SHAPE
    for f, v in (("ldus", 1), ("us_stride", 3), ("ldds", 0), ("ds_stride", 1)):
        assert MOE.run(**{**MOE8, f: v}) == SHAPE, f
    for f in ("X", "Wr", "Up", "Down"):
        assert MOE.run(**{f: 0}) == NULL_IN, f
        assert MOE.run(**{f: P + 1}) == ALIGN, f
    assert MOE.workspace(**MOE8, Up=P + 1, Down=P + 3)[0] == 0  # 8-bit weights lie anywhere
    assert MOE.run(US=P) == NULL_IN and MOE.run(DS=P) == NULL_IN
    assert MOE.run(D=0) == NULL_OUT and MOE.run(residual=P + 1) == ALIGN
    assert MOE.run(gated=2) == KIND and MOE.run(renormalize=-1) == KIND
    assert MOE.run(T=0, X=0, D=0, residual=0) == 0


@pytest.mark.parametrize("call", [LINEAR_B, MOE, LINEAR], ids=lambda c: c.name)
def test_workspace_is_checked(call):
    more = {"XS": 0, "ldx": 200} if call is LINEAR else {}  # x in 16 bits
    rc, need = call.workspace(**more)
    assert rc == 0 and need > 0
    assert call.run(**more) == WORKSPACE
    assert call.run(workspace=P, workspace_bytes=need - 1, **more) == WORKSPACE
    assert call.run(workspace=P + 8, workspace_bytes=need, **more) == ALIGN


def test_workspace_sizes():
    # operands on the 16-byte rule and scales on the 4-byte rule are read in place
    staged = LINEAR.workspace(M=4096, N=4096, K=4096, ldx=4104, ldw=4096, ldxs=32, ldws=32, ldr=4096, ldd=4096,
                              ldz=4096)[1]
    assert staged >= 4096 * 4096
    assert LINEAR.workspace(M=4096, N=4096, K=4096, ldx=4096, ldw=4096, ldxs=32, ldws=32, ldr=4096, ldd=4096,
                            ldz=4096)[1] < 4096
    # the layer's scratch does not grow past one chunk of tokens
    assert MOE.workspace(T=64)[1] == MOE.workspace(T=100000)[1]


def test_few_rows_need_no_copies():
    """Up to 16 rows read their operands in place at any alignment; x of 16 bits is quantised first past 4 rows."""
    odd = dict(X=P + 1, ldx=203, XS=P + 1, ldxs=3, W=P + 3, ldw=201, WS=P + 1, ldws=2)
    assert LINEAR.workspace(M=16, **odd) == (0, 0)
    assert LINEAR.workspace(M=17, **odd)[1] > 0
    half = dict(odd, XS=0, X=P + 2)
    assert LINEAR.workspace(M=4, **half) == (0, 0)
    rc, n = LINEAR.workspace(M=5, **half)
    assert rc == 0 and n >= 5 * 200


def test_a_single_row_has_no_pitch():
    """Where it begins alone decides whether it is read in place."""
    kw = dict(K=300, ldx=304, ldw=304, ldws=4, ldr=129, ldd=129, ldz=129)
    for n in (1, 96, 128):
        rc, least = LINEAR.workspace(N=n, **kw)
        assert rc == 0
        assert LINEAR.workspace(N=n, **{**kw, "ldws": 3}) == (0, least)
        assert LINEAR.workspace(N=n, WS=P + 2, **{**kw, "ldws": 3})[1] > least
    assert LINEAR.workspace(N=129, **{**kw, "ldws": 3})[1] > LINEAR.workspace(N=129, **kw)[1]  # two rows of scales
    least = LINEAR.workspace(N=1, **kw)[1]
    assert LINEAR.workspace(N=1, **{**kw, "ldw": 300}) == (0, least)
    assert LINEAR.workspace(N=1, W=P + 8, **{**kw, "ldw": 300})[1] > least
    kw = dict(K=1, lddx=1, lddw=1)
    rc, least = LINEAR_B.workspace(**kw)
    assert rc == 0 and LINEAR_B.workspace(**kw, ldxt=300, ldxts=3, ldwt=96, ldwts=1) == (0, least)


def test_quantised_matrices_have_fewer_than_2_23_blocks():
    assert QUANT.run(R=2000000, C=2000000, ldx=2000000, ldq=2000000, lds=20000, ldqt=2000000, ldst=20000) == SHAPE
    big = dict(K=1, ldx=1, ldw=16, N=1, XS=0)
    assert LINEAR.workspace(M=2 ** 30, **big)[0] == SHAPE
    assert LINEAR.workspace(M=9 * 10 ** 6, **big)[0] == 0
    assert LINEAR_B.workspace(M=2000000, N=2000000, lddd=2000000, ldxt=2000000, ldxts=16000, ldwt=2000000, ldwts=16000,
                              ldz=2000000, dW=0)[0] == SHAPE


def test_python_refusals():
    h, e = torch.float16, torch.float8_e4m3fn
    x, w = torch.zeros(4, 8, dtype=h), torch.zeros(6, 8, dtype=e)
    s = torch.zeros(1, 1, dtype=torch.float8_e8m0fnu)
    for call in (lambda: ge.quantize_fp8(x), lambda: ge.linear_fp8(x, w, s),
                 lambda: ge.linear_fp8_backward(x, w, s, w, s),
                 lambda: ge.moe(x, x, x[None], x[None], top_k=1)):
        with pytest.raises(ValueError, match="GPU device"):
            call()
    with pytest.raises(TypeError, match="must be one of"):
        ge.quantize_fp8(w)
    with pytest.raises(TypeError, match="must be one of"):
        ge.linear_fp8(x.float(), w, s)
    with pytest.raises(TypeError, match="torch.Tensor"):
        ge.moe(None, x, x[None], x[None], top_k=1)
