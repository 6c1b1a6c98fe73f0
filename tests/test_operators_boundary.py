"""The training and serving operators without a GPU: the library exports what
include/linear_ops.h declares, the Python structures have the header's layout,
bad arguments are refused with the documented status codes before any HIP call,
and the workspace queries answer."""
import ctypes
import os
import re

import pytest
import torch

import dense_gemm_elementwise_amd as ge
from dense_gemm_elementwise_amd import binding, operators

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TEXT = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "linear_ops.h")).read(), flags=re.S)

# fake device addresses: never dereferenced by the checks under test
P = 0x7F0000001000
P2 = P + 2
P1 = P + 1
F16, BF16, F32 = 0, 1, 2


def fields(name):
    """(field names, struct format characters) of an argument structure of the header."""
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", TEXT).group(1)
    names, kinds = [], ""
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        kind = "d" if decl.startswith("double") else "q"
        for n in re.sub(r"^(const )?(int64_t|double|void|float) ?\*?", "", decl).split(","):
            names.append(n.strip().lstrip("*"))
            kinds += kind
    return names, kinds


class Call:
    """A call of one entry point with named fields."""
    def __init__(self, name, **defaults):
        self.name, self.defaults = name, defaults
        self.names, self.kinds = fields(name + "_args")

    def pack(self, **kw):
        import struct
        v = {n: 0 for n in self.names}
        v.update(self.defaults)
        for k, x in kw.items():
            assert k in v, k
            v[k] = x
        return struct.pack("@" + self.kinds, *(v[n] for n in self.names))

    def run(self, **kw):
        return operators._functions()[self.name](self.pack(**kw))

    def workspace(self, **kw):
        return operators.workspace_bytes(self.name, self.pack(**kw))


LINEAR = Call("ge_linear", M=64, N=96, K=128, X=P, ldx=128, W=P, ldw=128, bias=P, residual=P, ldr=96, D=P, ldd=96,
              Z=P, ldz=96, act=2, dtype=BF16)
LINEAR_B = Call("ge_linear_backward", M=64, N=96, K=128, dD=P, lddd=96, X=P, ldx=128, W=P, ldw=128, Z=P, ldz=96,
                dX=P, lddx=128, dW=P, lddw=128, dbias=P, act=2, dtype=F16)
XENT = Call("ge_linear_xent", T=64, V=1000, K=128, X=P, ldx=128, W=P, ldw=128, target=P, ignore_index=-100, loss=P,
            lse=P, dtype=F16)
XENT_B = Call("ge_linear_xent_backward", T=64, V=1000, K=128, dloss=P, X=P, ldx=128, W=P, ldw=128, target=P, lse=P,
              ignore_index=-100, dX=P, lddx=128, dW=P, lddw=128, dtype=BF16)
NORM = Call("ge_norm_residual", T=8, hidden=96, G=2, H=P, ldh=96, Y=P, ldy=96, w_post=P, w_pre=P, gate=P, post=1,
            pre=2, scale=0.5, eps=1e-5, H_out=P, ldho=96, X=P, ldx=96, dtype=BF16, stream_dtype=F32)
NORM_B = Call("ge_norm_residual_backward", T=8, hidden=96, G=2, dX=P, lddx=96, dH_out=P, lddho=96, H_out=P, ldho=96,
              Y=P, ldy=96, w_post=P, w_pre=P, gate=P, post=1, pre=1, scale=0.5, eps=1e-5, dH=P, lddh=96, dY=P,
              lddy=96, dw_post=P, dw_pre=P, dgate=P, dtype=F16, stream_dtype=F16)
CALLS = (LINEAR, LINEAR_B, XENT, XENT_B, NORM, NORM_B)


def test_library_exports_every_declared_function():
    names = set(re.findall(r"\bint (ge_[a-z_]+)\(", TEXT))
    assert names == set(operators.OPERATOR_EXPORTS) | set(operators._WORKSPACE.values())
    raw = ctypes.CDLL(binding.LIB_PATH)
    for n in names:
        assert hasattr(raw, n), n


def test_python_structures_match_the_header():
    tails = {"ge_norm_residual": operators._STREAM}
    heads = {"ge_linear": operators._LINEAR, "ge_linear_backward": operators._LINEAR_GRAD,
             "ge_linear_xent": operators._XENT, "ge_linear_xent_backward": operators._XENT_GRAD,
             "ge_norm_residual": operators._NORM, "ge_norm_residual_backward": operators._NORM_GRAD}
    for name, head in heads.items():
        fmt = "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([qd])", head.format))
        tail = "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([qd])", tails.get(name, operators._TAIL).format))
        assert fmt + tail == fields(name + "_args")[1], name


def test_enums_match_the_header():
    for name, val in operators.ACTS.items():
        assert re.search(rf"GE_ACT_{name.upper()} = {val}\b", TEXT)
    for name, val in operators.NORMS.items():
        assert re.search(rf"GE_NORM_{name.upper()} = {val}\b", TEXT)


def test_null_structures():
    for c in CALLS:
        assert operators._functions()[c.name](None) == 2


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.name)
def test_element_types(call):
    for bad in (2, 3, -1):
        assert call.run(dtype=bad) == 8


@pytest.mark.parametrize("call, dims", [(LINEAR, "MNK"), (LINEAR_B, "MNK"), (XENT, "TVK"), (XENT_B, "TVK")],
                         ids=lambda v: v if isinstance(v, str) else v.name)
def test_product_shapes(call, dims):
    rows, outs, k = dims
    assert call.run(**{rows: -1}) == 1
    assert call.run(**{rows: 2 ** 31}) == 1
    assert call.run(**{outs: 0}) == 1
    assert call.run(**{outs: 2 ** 31}) == 1
    assert call.run(**{k: 0}) == 1
    assert call.run(**{k: 2097001}) == 1
    assert call.run(ldx=127) == 1      # rows overlap
    assert call.run(ldw=2097001) == 1  # past the row stride's limit
    assert call.run(X=P1) == 5
    assert call.run(W=P1) == 5
    assert call.run(X=0) == 2
    assert call.run(W=0) == 2


def test_linear_refusals():
    assert LINEAR.run(D=0) == 3
    assert LINEAR.run(act=4) == 4 and LINEAR.run(act=-1) == 4
    for f in ("bias", "residual", "D", "Z"):
        assert LINEAR.run(**{f: P1}) == 5, f
    for f in ("ldr", "ldd", "ldz"):
        assert LINEAR.run(**{f: 95}) == 1, f
    assert LINEAR.run(N=2097001, ldr=2097001, ldd=2097001, ldz=2097001) == 1
    assert LINEAR.workspace(act=9)[0] == 4


def test_linear_backward_refusals():
    assert LINEAR_B.run(dX=0, dW=0, dbias=0) == 3
    assert LINEAR_B.run(dD=0) == 2
    assert LINEAR_B.run(Z=0) == 2                   # an activation needs Z
    assert LINEAR_B.workspace(Z=0, act=0)[0] == 0   # the identity does not read it
    assert LINEAR_B.workspace(X=0, dW=0)[0] == 0    # only dW reads X, only dX reads W
    assert LINEAR_B.workspace(W=0, dX=0)[0] == 0
    assert LINEAR_B.run(dbias=P2) == 5
    assert LINEAR_B.run(dX=P1) == 5 and LINEAR_B.run(dW=P1) == 5
    assert LINEAR_B.run(lddx=127) == 1 and LINEAR_B.run(lddd=95) == 1


def test_xent_refusals():
    for c in (XENT, XENT_B):
        assert c.run(target=0) == 2
        assert c.run(target=P + 4) == 5
        assert c.run(lse=P2) == 5
    assert XENT.run(loss=0) == 3 and XENT.run(lse=0) == 3
    assert XENT_B.run(lse=0) == 2 and XENT_B.run(dloss=0) == 2
    assert XENT_B.run(dX=0, dW=0) == 3
    assert XENT_B.run(dloss=P2) == 5


@pytest.mark.parametrize("call", [NORM, NORM_B], ids=lambda c: c.name)
def test_norm_refusals(call):
    assert call.run(T=-2) == 1
    assert call.run(hidden=0) == 1
    assert call.run(hidden=16385 if call is NORM else 8193) == 1
    assert call.run(G=3) == 1              # does not divide the rows
    assert call.run(G=0) == 1
    assert call.run(gate=0) == 1           # no gate, but two gate rows
    assert call.run(post=3) == 4 and call.run(pre=0) == 4 and call.run(pre=3) == 4
    assert call.run(stream_dtype=1 - call.defaults["dtype"]) == 8
    assert call.run(eps=-1.0) == 1 and call.run(eps=float("nan")) == 1 and call.run(scale=float("nan")) == 1
    for f in ("w_post", "w_pre", "gate", "Y"):
        assert call.run(**{f: P1}) == 5, f
    assert call.run(Y=0) == 2
    assert call.run(ldy=95) == 1


def test_norm_outputs():
    assert NORM.run(H=0) == 2 and NORM.run(X=0) == 3 and NORM.run(H_out=0) == 3
    assert NORM.run(H=P2) == 5             # an fp32 stream is 4-byte aligned
    assert NORM_B.run(dX=0) == 2 and NORM_B.run(dH_out=0) == 2 and NORM_B.run(dH=0) == 3 and NORM_B.run(dY=0) == 3
    assert NORM_B.run(dgate=P2) == 5


@pytest.mark.parametrize("call", [c for c in CALLS if c is not NORM], ids=lambda c: c.name)
def test_workspace_is_checked(call):
    rows = "M" if "M" in call.names else "T"
    rc, need = call.workspace(**{rows: 512})
    if call is LINEAR:
        rc, need = call.workspace(M=512, ldx=129, K=128)   # rows off the 16-byte rule are staged
        assert rc == 0 and need >= 512 * 128 * 2
        big = {"M": 512, "ldx": 129}
    else:
        assert rc == 0 and need > 0
        big = {rows: 512}
    assert call.run(**big) == 7                                            # none given
    assert call.run(workspace=P, workspace_bytes=need - 1, **big) == 7     # too small
    assert call.run(workspace=P + 8, workspace_bytes=need, **big) == 5     # not 16-byte aligned


def test_workspace_sizes():
    assert LINEAR.workspace(M=1) == (0, 0)        # few rows read everything in place
    assert LINEAR.workspace(M=0) == (0, 0)
    rc, a = XENT_B.workspace(T=4096, V=100003, K=4096, ldx=4096, ldw=4096, lddx=4096, lddw=4096)
    assert rc == 0 and a < 4096 * 100003 * 2      # P is never whole
    rc, b = XENT_B.workspace(T=4096, V=1000003, K=4096, ldx=4096, ldw=4096, lddx=4096, lddw=4096)
    assert rc == 0 and b < 1.5 * a                # nor does the workspace grow with the vocabulary


@pytest.mark.parametrize("T", [1, 2, 16, 17, 31, 32, 33, 64])
@pytest.mark.parametrize("V", [2096897, 2097000, 2097001, 3000000, 2 ** 31 - 257])
def test_xent_gradient_takes_every_vocabulary_of_the_forward(T, V):
    """A small batch would fit more columns in one piece than a row may have."""
    assert XENT.workspace(T=T, V=V)[0] == 0
    rc, need = XENT_B.workspace(T=T, V=V)
    assert rc == 0
    # one piece of P, and no more than that grows with the vocabulary
    assert need < T * 2097000 * 2 + (256 << 20)


def test_empty_batch_needs_no_output_address():
    """An empty dX has no memory: with no rows, its address may be NULL and the only output."""
    assert LINEAR_B.run(M=0, dX=0, dW=0, dbias=0) == 0
    assert LINEAR_B.workspace(M=0, dX=0, dW=0, dbias=0) == (0, 0)
    assert XENT_B.run(T=0, dX=0, dW=0) == 0
    assert XENT_B.workspace(T=0, dX=0, dW=0) == (0, 0)
    assert LINEAR.run(M=0, X=0, D=0, residual=0, Z=0) == 0
    assert XENT.run(T=0, X=0, target=0, loss=0, lse=0) == 0


@pytest.mark.parametrize("T", [1, 3, 16, 17, 128, 129, 256, 257, 512])
def test_longest_vocabulary_is_taken(T):
    """Up to 2^24 tiles of 256 x 256, whichever tile would be the fastest."""
    V = 2 ** 31 - 257
    assert XENT.workspace(T=T, V=V, K=8, ldx=8, ldw=8)[0] == 0
    assert XENT.workspace(T=V, V=T, K=8, ldx=8, ldw=8)[0] == 0
    assert LINEAR_B.workspace(M=V, N=min(T, 256), K=8, ldx=8, ldw=8, lddd=1024, ldz=1024, lddx=8, lddw=8)[0] == 0


def test_products_past_a_launch_are_refused():
    assert XENT.workspace(T=513, V=2 ** 31 - 257, K=8, ldx=8, ldw=8)[0] == 1
    assert XENT.workspace(T=2 ** 20, V=2 ** 20 - 256, K=8, ldx=8, ldw=8)[0] == 0
    assert XENT.workspace(T=2 ** 20, V=2 ** 20, K=8, ldx=8, ldw=8)[0] == 1
    assert LINEAR.workspace(M=2 ** 31 - 257, N=1024, ldr=1024, ldd=1024, ldz=1024)[0] == 1


def test_python_refusals():
    x, w = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(6, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU device"):
        ge.linear(x, w)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        ge.linear(x.float(), w.float())
    with pytest.raises(TypeError, match="torch.Tensor"):
        ge.linear(None, w)
    with pytest.raises(ValueError, match="GPU device"):
        ge.linear_xent(x, w, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU device"):
        ge.norm_residual(x, x)
    with pytest.raises(AttributeError):
        ge.no_such_operator


def test_header_is_plain_c(tmp_path):
    """The header compiles as C99, and every structure is made of 8-byte fields only."""
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    checks = "\n".join(f"typedef char size_{c.name}[sizeof({c.name}_args) == 8 * {len(c.names)} ? 1 : -1];"
                       for c in CALLS)
    src = tmp_path / "header.c"
    src.write_text(f'#include "linear_ops.h"\n{checks}\nint main(void) {{ return 0; }}\n')
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                    os.path.join(ROOT, "include"), str(src)], check=True)


def test_forward_mode_tangents_are_refused():
    """A dual tensor's tangent would vanish: no call may take its address."""
    from torch.autograd import forward_ad
    x = torch.zeros(4, 8, dtype=torch.float16)
    calls = []
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for inputs in ((dual,), (x, None, dual)):
            with pytest.raises(ValueError, match="tangent"):
                operators._run(calls.append, inputs, torch.device("cuda:0"), None)
    assert not calls
