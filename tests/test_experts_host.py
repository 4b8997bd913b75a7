"""Host-side checks of the expert products (no GPU needed): bad arguments come
back as status codes before anything touches a device, and the binding refuses
tensors it cannot describe."""
import ctypes

import pytest

from tiled_newton_schulz_b200 import himuon as hm

torch = pytest.importorskip("torch")
INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -4
P = 0x100000


@pytest.fixture(scope="module")
def lib():
    from tiled_newton_schulz_b200 import build
    build.build()
    return hm.load()


def M(rows, cols, ld=None, dtype=hm.BF16, data=P):
    return hm.Mat(data, rows, cols, cols if ld is None else ld, dtype)


def arr(*ms):
    return (hm.Mat * len(ms))(*ms)


def addr(a):
    return ctypes.addressof(a)


def product(lib, X=None, W=None, Y=None, n=2, offsets=P, trans=0):
    X, Y = X or M(10, 64), Y or M(10, 32)
    W = W or arr(M(64, 32), M(64, 32))
    return lib.himuon_expert_product(X, addr(W), n, offsets, trans, Y, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), INVALID),
    (dict(offsets=None), INVALID),                                       # n = 2 needs offsets
    (dict(trans=2), INVALID),
    (dict(trans=1), INVALID),                                            # W is K x N here
    (dict(X=M(10, 64, data=0)), INVALID),
    (dict(X=M(10, 64, ld=56)), INVALID),
    (dict(X=M(10, 63, ld=64)), INVALID),
    (dict(X=M(10, 64, dtype=hm.FP16)), INVALID),                         # W is BF16
    (dict(Y=M(9, 32)), INVALID),
    (dict(Y=M(10, 40)), INVALID),
    (dict(W=arr(M(64, 32), M(64, 40))), INVALID),
    (dict(W=arr(M(64, 32), M(64, 32, ld=40))), INVALID),
    (dict(W=arr(M(64, 32), M(64, 32, data=0))), INVALID),
    (dict(X=M(10, 64, dtype=hm.FP32), W=arr(*[M(64, 32, dtype=hm.FP32)] * 2)), UNSUPPORTED),
    (dict(X=M(10, 64, dtype=hm.I8), W=arr(*[M(64, 32, dtype=hm.I8)] * 2)), UNSUPPORTED),
    (dict(Y=M(10, 32, dtype=hm.I8)), UNSUPPORTED),
    (dict(X=M(10, 64, dtype=7)), UNSUPPORTED),
    (dict(X=M((1 << 30) + 1, 64), Y=M((1 << 30) + 1, 32)), UNSUPPORTED),
    (dict(X=M((1 << 27) + 8, 64), Y=M((1 << 27) + 8, 32)), UNSUPPORTED),   # longer than the bounded waits allow
    (dict(n=65537), INVALID),
    (dict(X=M(10, 64, data=P + 8)), ALIGNMENT),
    (dict(Y=M(10, 32, ld=36)), ALIGNMENT),
    (dict(W=arr(M(64, 32, data=P + 2), M(64, 32))), ALIGNMENT),
])
def test_product_refusals(lib, kw, code):
    assert product(lib, **kw) == code


def test_product_null_pointers(lib):
    W = arr(M(64, 32))
    assert lib.himuon_expert_product(None, addr(W), 1, None, 0, M(10, 32), None) == INVALID
    assert lib.himuon_expert_product(M(10, 64), None, 1, None, 0, M(10, 32), None) == INVALID
    assert lib.himuon_expert_product(M(10, 64), addr(W), 1, None, 0, None, None) == INVALID


def gradient(lib, A=None, B=None, G=None, C=None, n=2, offsets=P, alpha=1.0, beta=0.0):
    A, B = A or M(10, 64), B or M(10, 32)
    G = G or arr(M(64, 32), M(64, 32, data=2 * P))
    return lib.himuon_expert_gradient(A, B, n, offsets, alpha, beta, addr(C) if C else None, addr(G), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), INVALID),
    (dict(offsets=None), INVALID),
    (dict(beta=1.0), INVALID),                                           # no C
    (dict(alpha=float("nan")), INVALID),
    (dict(beta=float("inf"), C=arr(*[M(64, 32)] * 2)), INVALID),
    (dict(B=M(11, 32)), INVALID),
    (dict(B=M(10, 32, dtype=hm.FP16)), INVALID),
    (dict(G=arr(M(64, 40), M(64, 40, data=2 * P))), INVALID),
    (dict(G=arr(M(64, 32), M(64, 32))), INVALID),                        # the same matrix twice
    (dict(C=arr(*[M(64, 40)] * 2), beta=1.0), INVALID),
    # C in the place of G, in another type or pitch
    (dict(C=arr(M(64, 32, dtype=hm.FP32), M(64, 32, dtype=hm.FP32, data=4 * P)), beta=1.0), INVALID),
    (dict(C=arr(M(64, 32, ld=64), M(64, 32, ld=64, data=4 * P)), beta=1.0), INVALID),
    (dict(A=M(10, 64, dtype=hm.FP32), B=M(10, 32, dtype=hm.FP32)), UNSUPPORTED),
    (dict(G=arr(M(64, 32, dtype=hm.I8), M(64, 32, dtype=hm.I8, data=2 * P))), UNSUPPORTED),
    (dict(C=arr(*[M(64, 32, dtype=hm.I8)] * 2), beta=1.0), UNSUPPORTED),
    (dict(A=M(10, 64, ld=68)), ALIGNMENT),
    (dict(G=arr(M(64, 32), M(64, 32, data=2 * P + 4))), ALIGNMENT),
])
def test_gradient_refusals(lib, kw, code):
    assert gradient(lib, **kw) == code


def product8(lib, X=None, xs=None, W=None, ws=None, Y=None, n=2, offsets=P):
    X, xs = X or M(10, 64, dtype=hm.I8), xs or M(1, 10, dtype=hm.FP32)
    W = W or arr(*[M(32, 64, dtype=hm.I8)] * 2)
    return lib.himuon_expert_product_i8(X, xs, addr(W), ws or M(2, 32, dtype=hm.FP32), n, offsets, Y or M(10, 32), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INVALID),
    (dict(offsets=None), INVALID),
    (dict(xs=M(1, 9, dtype=hm.FP32)), INVALID),
    (dict(ws=M(1, 32, dtype=hm.FP32)), INVALID),
    (dict(ws=M(2, 33, dtype=hm.FP32)), INVALID),
    (dict(W=arr(*[M(32, 80, dtype=hm.I8)] * 2)), INVALID),
    (dict(xs=M(1, 10)), UNSUPPORTED),                                    # scales are fp32
    (dict(X=M(10, 64)), UNSUPPORTED),
    (dict(W=arr(*[M(32, 64)] * 2)), UNSUPPORTED),
    (dict(X=M(10, 131072, dtype=hm.I8), W=arr(*[M(32, 131072, dtype=hm.I8)] * 2)), UNSUPPORTED),   # int32's range
    (dict(X=M(10, 64, ld=72, dtype=hm.I8)), ALIGNMENT),
    (dict(xs=M(1, 10, dtype=hm.FP32, data=P + 2)), ALIGNMENT),
])
def test_product_i8_refusals(lib, kw, code):
    assert product8(lib, **kw) == code


def quant(lib, i=None, q=None, s=None, n=1, dim=0):
    i, q, s = i or M(10, 64), q or M(10, 64, dtype=hm.I8), s or M(1, 10, dtype=hm.FP32)
    i, q, s = arr(i), arr(q), arr(s)
    return lib.himuon_quantize(addr(i), n, dim, addr(q), addr(s), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), INVALID),
    (dict(dim=2), INVALID),
    (dict(dim=1), INVALID),                                              # codes are not transposed
    (dict(q=M(10, 80, dtype=hm.I8)), INVALID),
    (dict(s=M(1, 64, dtype=hm.FP32)), INVALID),
    (dict(q=M(10, 64)), UNSUPPORTED),
    (dict(i=M(10, 64, dtype=hm.I8)), UNSUPPORTED),
    (dict(s=M(1, 10)), UNSUPPORTED),
    (dict(q=M(10, 64, ld=72, dtype=hm.I8)), ALIGNMENT),
    (dict(dim=1, i=M(0, 64), q=M(64, 0, dtype=hm.I8), s=M(1, 64, dtype=hm.FP32)), INVALID),
])
def test_quantize_refusals(lib, kw, code):
    assert quant(lib, **kw) == code


def test_other_entry_points_refuse_int8(lib):
    p = hm.params(128, (3.4445, -4.7750, 2.0315), steps=5)
    m = arr(M(16, 16, dtype=hm.I8))
    assert lib.himuon_ns_tiled(m, m, 1, None, ctypes.byref(p), None, 0, None) == UNSUPPORTED


def test_binding_refuses_what_it_cannot_describe(lib):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    w = torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                                      # not on a CUDA device
        hm.expert_product(x, w, x, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        hm.expert_gradient(x, x, w, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        hm.quantize([x], [x.to(torch.int8)], [torch.zeros(4)])
    with pytest.raises(ValueError):
        hm.quantize([x], [], [])
    with pytest.raises(ValueError):
        hm._stack(w.transpose(1, 2))
    with pytest.raises(ValueError):
        hm._stack(w[0])
    for bad in (torch.zeros(3, dtype=torch.int64), torch.zeros(4, dtype=torch.int32),
                torch.zeros(6, dtype=torch.int32)[::2], torch.zeros(3, 1, dtype=torch.int32)):
        with pytest.raises(ValueError):
            hm._offsets(bad, 2)


def test_stacked_matrices_are_described_as_the_list_is(lib):
    w = torch.zeros(5, 8, 24, dtype=torch.float16)[1:, :6, 8:]
    rec, a, n = hm._stack(w)
    arr_, b, m = hm._stack(list(w))
    assert n == m == 4
    got = (hm.Mat * n).from_address(a)
    for g, e in zip(got, arr_):
        assert (g.data, g.rows, g.cols, g.ld, g.dtype) == (e.data, e.rows, e.cols, e.ld, e.dtype)


def _blocks(text):
    """(opening brace, closing brace, what stands before the opening one on its line or, for an else, `if ... else`)
    of every block of a source text, comments and strings aside."""
    import re
    text = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), text)
    text = re.sub(r'"(?:[^"\\\n]|\\.)*"', lambda m: '"' + " " * (len(m.group()) - 2) + '"', text)
    out, stack = [], []
    for i, c in enumerate(text):
        if c == "{":
            stack.append(i)
        elif c == "}":
            a = stack.pop()
            out.append((a, i, text[text.rfind("\n", 0, a) + 1:a].strip()))
    assert not stack
    return out


def test_register_moves_are_one_instruction_per_warpgroup():
    """setmaxnreg is undefined unless all threads of a warpgroup run the same instruction, and an increase waits for
    the decreases: one of each per kernel, in the blocks that tell the warpgroups apart and outside every branch
    between the warps of one."""
    import re
    from tiled_newton_schulz_b200 import build
    found = 0
    for name in build.SOURCES + build.HEADERS:
        with open(f"{build.CSRC}/{name}") as f:
            text = f.read()
        where = {d: [m.start() for m in re.finditer(rf"setmaxnreg\.{d}", text)] for d in ("dec", "inc")}
        if not (where["dec"] or where["inc"]):
            continue
        found += 1
        assert len(where["dec"]) == len(where["inc"]) == 1, name
        blocks = _blocks(text)
        around = {d: sorted((b for b in blocks if b[0] < w[0] < b[1]), reverse=True) for d, w in where.items()}
        dec, inc = around["dec"][0], around["inc"][0]
        assert dec[2] == "if (warp < 4)" and inc[2] == "} else"
        assert text[dec[1]:inc[0] + 1] == "} else {"                      # the other warpgroups are the block's else
        assert around["dec"][1] == around["inc"][1]                      # both directly in the kernel's body
        assert around["dec"][1][2].startswith("expert_kernel(")
    assert found == 1
