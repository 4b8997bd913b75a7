"""Expert products against their definitions in 64 bits (needs a B200).

Tolerances.  An output y = round(s) to a type of unit roundoff u (half of
torch.finfo's eps) of an fp32 sum s of K products: the products of 16-bit
values are exact in fp32, and each of the K additions, in any order, is off by
at most 2^-23 of a partial sum, whose size is at most S = sum |a| |b| (2^-23
rather than 2^-24: the tensor cores truncate instead of rounding).  So
    |y - exact| <= (K + 16) 2^-23 S + u |exact| (1 + ...) + half the type's
smallest step, the 16 covering the epilogue's operations (alpha, beta, the
scales).  The 8-bit sum is exact, so there only the epilogue's part is left.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def hm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_newton_schulz_b200 import himuon
    himuon.load()
    return himuon


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def matrix(shape, dtype, g, scale=1.0, lead=8, margin=0, fill=float("nan")):
    """Normal values as a view into a larger buffer of `fill`: `margin` extra
    columns and a pitch that is a multiple of `lead`."""
    pitch = -(-(shape[-1] + margin) // lead) * lead
    buf = torch.full((*shape[:-1], pitch), fill, device=DEV, dtype=torch.float32).to(dtype)
    view = buf[..., :shape[-1]]
    view.copy_(torch.randn(*shape, generator=g, device=DEV) * scale)
    return view


def offsets(counts, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def groups(off):
    o = off.tolist()
    return list(zip(o, o[1:]))


def close(y, exact, size, k, dtype):
    f = torch.finfo(dtype)
    y = y.double()
    lim = (k + 16) * 2.0 ** -23 * size + f.eps / 2 * exact.abs() * (1 + 2 ** -8) + f.smallest_normal * f.eps / 2
    d = (y - exact).abs()
    assert torch.isfinite(y).all()
    bad = d > lim
    assert not bad.any(), f"{int(bad.sum())} off, worst {float((d / lim).max()):.3g} of the bound, {bad.nonzero()[:4].tolist()}"


def check_product(hm, dtype, out, K, N, counts, trans, start=0, behind=0, listed=False, seed=0, margin=0):
    g = gen(seed)
    n, off = len(counts), offsets(counts, start)
    rows = start + sum(counts) + behind
    X = matrix((rows, K), dtype, g, margin=margin)
    X[:start] = float("nan")                      # rows outside every group must not matter
    X[rows - behind:] = float("inf")
    W = matrix((n, N, K) if trans else (n, K, N), dtype, g, 0.5, margin=margin)
    Y = torch.full((rows, -(-(N + margin) // 8) * 8), -7.0, device=DEV).to(out)
    Yv = Y[:, :N]
    hm.expert_product(X, [w for w in W] if listed else W, Yv, off, w_trans=trans)
    assert hm.device_status() == 0
    for e, (a, b) in enumerate(groups(off)):
        x, w = X[a:b].double(), W[e].double()
        w = w.T if trans else w
        close(Yv[a:b], x @ w, x.abs() @ w.abs(), K, out)
    assert (Y[:start] == -7).all() and (Y[rows - behind:] == -7).all() and (Y[:, N:] == -7).all()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp16", "bf16")])
@pytest.mark.parametrize("K,N,counts", [
    (64, 128, [1]),
    (8, 8, [0, 1, 0, 2]),
    (1, 1, [3]),
    (200, 136, [5, 0, 33, 130, 1]),
    (129, 257, [31, 32, 33, 0]),
    (512, 384, [300, 257, 0, 256, 17]),
    (1100, 2050, [100, 7]),
])
def test_product(hm, dtype, out, K, N, counts, trans):
    check_product(hm, TYPES[dtype], TYPES[out], K, N, counts, trans, seed=K + N)


@pytest.mark.parametrize("trans", [False, True])
def test_product_views_rows_outside_groups_and_lists(hm, trans):
    check_product(hm, torch.bfloat16, torch.bfloat16, 320, 264, [40, 0, 90], trans, start=13, behind=70, listed=True,
                  margin=24)
    check_product(hm, torch.float16, torch.float32, 72, 40, [1, 1, 1], trans, start=1, behind=1, margin=8)


@pytest.mark.parametrize("n,listed", [(130, True), (300, False), (700, False)])
def test_product_many_experts(hm, n, listed):
    rng = np.random.default_rng(n)
    check_product(hm, torch.bfloat16, torch.bfloat16, 72, 136, rng.integers(0, 4, n).tolist(), False, listed=listed)
    counts = np.zeros(n, dtype=int)
    counts[n - 1], counts[n // 2] = 70, 1
    check_product(hm, torch.bfloat16, torch.float32, 64, 64, counts.tolist(), True, start=2, listed=listed)


@pytest.mark.parametrize("rows", [1, 8, 64, 700])
@pytest.mark.parametrize("K,N", [(4096, 1024), (1024, 4096), (2048, 256)])
@pytest.mark.parametrize("trans", [False, True])
def test_product_few_rows_long_sums(hm, rows, K, N, trans):
    rng = np.random.default_rng(rows)
    check_product(hm, torch.bfloat16, torch.bfloat16, K, N, rng.multinomial(rows, np.ones(6) / 6).tolist(), trans)


def test_product_one_group_without_offsets_and_empty_operands(hm):
    g = gen(3)
    X, W = matrix((77, 96), torch.bfloat16, g), matrix((1, 96, 48), torch.bfloat16, g)
    Y = torch.empty(77, 48, device=DEV, dtype=torch.float32)
    hm.expert_product(X, W, Y)
    x, w = X.double(), W[0].double()
    close(Y, x @ w, x.abs() @ w.abs(), 96, torch.float32)
    hm.expert_product(X[:0], W, Y[:0])
    hm.expert_product(X[:0], W, Y[:0], torch.zeros(2, dtype=torch.int32, device=DEV))
    # a single row of a width that is no multiple of 16 bytes
    X1, W1, Y1 = X[:1, :93].contiguous(), W[:, :93], torch.empty(1, 45, device=DEV, dtype=torch.bfloat16)
    hm.expert_product(X1, W1[:, :, :45], Y1)
    x, w = X1.double(), W1[0, :, :45].double()
    close(Y1, x @ w, x.abs() @ w.abs(), 93, torch.bfloat16)
    assert hm.device_status() == 0


@pytest.mark.parametrize("trans", [False, True])
def test_product_all_groups_empty_and_column_blocks(hm, trans):
    """No row in any group; and matrices that are column blocks of one fused matrix, as a list and as a 3-D view."""
    g = gen(21)
    n, K, N = 3, 64, 40
    X = matrix((50, K), torch.bfloat16, g)
    fused = matrix((N if trans else K, n * (K if trans else N)), torch.bfloat16, g)
    blocks = list(fused.split(K if trans else N, dim=1))
    W3 = fused.reshape(fused.shape[0], n, -1).transpose(0, 1)
    assert W3.data_ptr() == fused.data_ptr()
    Y = torch.full((50, N), -7.0, device=DEV)
    for off in (offsets([0, 0, 0]), offsets([0, 0, 0], start=50)):
        hm.expert_product(X, blocks, Y, off, w_trans=trans)
        assert (Y == -7).all()
    off = offsets([20, 0, 30])
    for W in (blocks, W3):
        Y.fill_(-7)
        hm.expert_product(X, W, Y, off, w_trans=trans)
        for e, (a, b) in enumerate(groups(off)):
            x, w = X[a:b].double(), (blocks[e].double().T if trans else blocks[e].double())
            close(Y[a:b], x @ w, x.abs() @ w.abs(), K, torch.float32)
    assert hm.device_status() == 0


def test_gradient_into_column_blocks(hm):
    g = gen(22)
    n, P, Q = 4, 72, 48
    A, B = matrix((90, P), torch.bfloat16, g), matrix((90, Q), torch.bfloat16, g)
    off = offsets([30, 0, 25, 35])
    for out in (torch.bfloat16, torch.float32):
        fused = torch.full((P, n * Q), 2.0, device=DEV).to(out)
        for G in (list(fused.split(Q, dim=1)), fused.reshape(P, n, Q).transpose(0, 1)):
            fused.fill_(2)
            hm.expert_gradient(A, B, G, off, beta=1.0, C=G)
            for e, (a, b) in enumerate(groups(off)):
                x, y = A[a:b].double(), B[a:b].double()
                close(G[e], 2 + x.T @ y, 2 + x.abs().T @ y.abs(), b - a, out)
    assert hm.device_status() == 0


def test_first_run_of_a_variant_inside_a_capture(hm):
    """After one call on the device, a call whose kernel has not run yet can be captured and replayed."""
    import subprocess
    import sys
    code = """
import torch
from tiled_newton_schulz_b200 import himuon as hm
x = torch.randn(40, 64, device="cuda").bfloat16()
w = torch.randn(1, 64, 48, device="cuda").bfloat16()
y = torch.zeros(40, 48, device="cuda", dtype=torch.bfloat16)
hm.expert_product(x, w, y)
a, b = torch.randn(3000, 64, device="cuda").bfloat16(), torch.randn(3000, 48, device="cuda").bfloat16()
G = torch.zeros(1, 64, 48, device="cuda")
q, s = torch.zeros(40, 64, device="cuda", dtype=torch.int8), torch.zeros(40, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    hm.expert_gradient(a, b, G)
    hm.quantize([x], [q], [s])
g.replay()
torch.cuda.synchronize()
ref = a.double().T @ b.double()
assert (G[0].double() - ref).norm() <= 1e-5 * ref.norm()
assert q.abs().amax(1).eq(127).all()
assert hm.device_status() == 0
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]


def test_product_shared_matrix_and_nonfinite_rows(hm):
    """One matrix for two groups; a row with an infinity or a NaN changes no other row."""
    g = gen(4)
    W1 = matrix((160, 96), torch.bfloat16, g)
    X = matrix((50, 160), torch.bfloat16, g)
    off = offsets([20, 30])
    Y = torch.empty(50, 96, device=DEV, dtype=torch.bfloat16)
    hm.expert_product(X, [W1, W1], Y, off)
    want = Y.clone()
    hm.expert_product(X, W1.expand(2, -1, -1), Y, off)
    assert torch.equal(Y, want)
    X[7, 3], X[20, 159] = float("nan"), float("inf")
    hm.expert_product(X, [W1, W1], Y, off)
    keep = [r for r in range(50) if r not in (7, 20)]
    assert torch.equal(Y[keep], want[keep])
    assert Y[7].isnan().all() and not torch.isfinite(Y[20]).any()


def check_gradient(hm, dtype, out, P, Q, counts, beta=0.0, alpha=1.0, cdtype=None, alias=False, start=0, behind=0,
                   listed=False, seed=0, margin=0):
    g = gen(seed)
    n, off = len(counts), offsets(counts, start)
    rows = start + sum(counts) + behind
    A = matrix((rows, P), dtype, g, margin=margin)
    B = matrix((rows, Q), dtype, g, margin=margin)
    for t, v in ((A, float("nan")), (B, float("inf"))):   # rows outside every group must not matter
        t[:start] = v
        t[rows - behind:] = v
    pitch = -(-(Q + margin) // 8) * 8
    G = torch.full((n, P, pitch), -7.0, device=DEV).to(out)
    Gv = G[:, :, :Q]
    C = None
    if beta != 0 or cdtype is not None:
        C = matrix((n, P, Q), cdtype or out, g, 3.0)
        if alias:
            Gv.copy_(C)
    c0 = C.double() if C is not None else None
    lst = (lambda t: [m for m in t]) if listed else (lambda t: t)
    hm.expert_gradient(A, B, lst(Gv), off, alpha=alpha, beta=beta, C=lst(Gv if alias else C) if C is not None else None)
    assert hm.device_status() == 0
    for e, (a, b) in enumerate(groups(off)):
        x, y = A[a:b].double(), B[a:b].double()
        exact, size = alpha * (x.T @ y), abs(alpha) * (x.abs().T @ y.abs())
        if beta != 0:
            exact, size = exact + beta * c0[e], size + abs(beta) * c0[e].abs()
        close(Gv[e], exact, size, b - a, out)
    assert (G[:, :, Q:] == -7).all()


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp16", "fp32")])
@pytest.mark.parametrize("beta", [0.0, 1.0])
@pytest.mark.parametrize("P,Q,counts", [
    (128, 128, [64]),
    (8, 8, [0, 1, 0, 2]),
    (1, 1, [3]),
    (136, 200, [5, 0, 33, 130, 1]),
    (257, 129, [31, 16, 17, 0]),
    (384, 512, [300, 257, 0, 15, 128]),
    (64, 2050, [63, 65]),
])
def test_gradient(hm, dtype, out, beta, P, Q, counts):
    check_gradient(hm, TYPES[dtype], TYPES[out], P, Q, counts, beta=beta, seed=P + Q)


def test_gradient_views_scales_types_and_alias(hm):
    bf, f32 = torch.bfloat16, torch.float32
    check_gradient(hm, bf, bf, 120, 264, [40, 0, 90], start=13, behind=70, listed=True, margin=24, alpha=-0.5)
    check_gradient(hm, bf, f32, 120, 264, [40, 0, 90], beta=1.0, alias=True, start=3, behind=5, listed=True)
    check_gradient(hm, bf, bf, 120, 264, [40, 0, 90], beta=0.95, alias=True, margin=40)
    check_gradient(hm, torch.float16, bf, 72, 40, [9, 9], beta=-2.0, alpha=0.25, cdtype=f32)
    check_gradient(hm, bf, f32, 72, 40, [9, 9], beta=1.0, cdtype=torch.float16)
    check_gradient(hm, bf, f32, 40, 72, [0, 0, 0], beta=1.0)
    check_gradient(hm, bf, f32, 40, 72, [0, 0, 0])


def test_gradient_leaves_c_unread_without_beta(hm):
    g = gen(8)
    A, B = matrix((20, 48), torch.bfloat16, g), matrix((20, 56), torch.bfloat16, g)
    G = torch.full((1, 48, 56), float("nan"), device=DEV)
    hm.expert_gradient(A, B, G, beta=0.0, C=G)
    x, y = A.double(), B.double()
    close(G[0], x.T @ y, x.abs().T @ y.abs(), 20, torch.float32)
    hm.expert_gradient(A[:0], B[:0], G)                       # no rows: zeros
    assert (G == 0).all()


@pytest.mark.parametrize("n,listed", [(130, True), (300, False)])
def test_gradient_many_experts(hm, n, listed):
    rng = np.random.default_rng(n)
    check_gradient(hm, torch.bfloat16, torch.bfloat16, 72, 136, rng.integers(0, 6, n).tolist(), listed=listed)


@pytest.mark.parametrize("counts", [[80, 37, 16, 100, 0, 192], [5, 144, 63, 64, 1000, 33], [17, 48, 300, 49, 2, 0, 31]])
def test_gradient_many_tiles_per_cta_pair(hm, counts):
    """Every pair runs several tiles, of groups whose last stretch of rows is whole, a multiple of 16 or neither."""
    check_gradient(hm, torch.bfloat16, torch.float32, 1032, 2050, counts)


@pytest.mark.parametrize("trans", [False, True])
def test_product_many_tiles_per_cta_pair(hm, trans):
    check_product(hm, torch.bfloat16, torch.bfloat16, 208, 4104, [257, 513, 1, 0, 700, 64, 31, 1025], trans)
    check_i8(hm, torch.float32, 400, 2056, [257, 513, 1, 0, 700, 64, 31, 1025])


@pytest.mark.parametrize("P,Q", [(520, 771), (264, 448), (768, 352), (72, 1000), (2048, 224)])
def test_gradient_tile_widths(hm, P, Q):
    """Sizes at which the tiles are narrower than 256 columns."""
    check_gradient(hm, torch.bfloat16, torch.bfloat16, P, Q, [140, 7, 0, 96, 33], beta=1.0, margin=16)
    check_gradient(hm, torch.float16, torch.float32, P, Q, [64, 7, 700])
    check_gradient(hm, torch.float16, torch.float16, P, Q, [65, 130], cdtype=torch.float32, beta=0.5)


@pytest.mark.parametrize("counts", [[300] * 5, [1531], [100, 180, 260, 20], [129], [193, 257], [90] * 9])
def test_product_tile_widths(hm, counts):
    """Row counts at which the tiles are narrower than 256 rows."""
    check_product(hm, torch.bfloat16, torch.bfloat16, 520, 2050, counts, False)
    check_product(hm, torch.bfloat16, torch.float32, 200, 1000, counts, True, start=7, behind=300)
    check_i8(hm, torch.float32, 600, 520, counts, start=1, behind=300)


@pytest.mark.parametrize("counts", [[1], [33], [200], [1, 2], [300, 0]])
@pytest.mark.parametrize("K,N", [(2048, 264), (4100, 136), (520, 520)])
def test_product_tiles_shared_by_pairs(hm, K, N, counts):
    """Few tiles: their sums are cut among the pairs of a cluster, every result type."""
    for trans in (False, True):
        for out in TYPES.values():
            check_product(hm, torch.bfloat16, out, K, N, counts, trans, start=2, behind=40, listed=trans)
    check_i8(hm, torch.bfloat16, K, N, counts, start=2, behind=40)
    check_i8(hm, torch.float32, 2 * K, N, counts, full=True)


@pytest.mark.parametrize("counts", [[5003], [4, 2000, 0], [65], [777, 1024]])
@pytest.mark.parametrize("P,Q", [(8, 8), (264, 136), (520, 771)])
def test_gradient_tiles_shared_by_pairs(hm, P, Q, counts):
    for out in TYPES.values():
        check_gradient(hm, torch.bfloat16, out, P, Q, counts, start=3, behind=70)
        check_gradient(hm, torch.float16, out, P, Q, counts, beta=1.0, cdtype=torch.float32, alpha=0.5, listed=True)
    check_gradient(hm, torch.bfloat16, torch.bfloat16, P, Q, counts, beta=-1.0, alias=True, margin=8)


def test_gradient_long_sum(hm):
    check_gradient(hm, torch.bfloat16, torch.float32, 200, 264, [5003, 1])
    check_gradient(hm, torch.bfloat16, torch.bfloat16, 64, 64, [9001])


def test_gradient_against_differences(hm):
    """The products are linear in W and in X, so differences along one entry are the gradients up to rounding."""
    g = gen(9)
    off = offsets([37, 0, 64])
    X, W = matrix((101, 80), torch.bfloat16, g), matrix((3, 80, 48), torch.bfloat16, g)
    dY = matrix((101, 48), torch.bfloat16, g)
    G = torch.empty(3, 80, 48, device=DEV)
    dX = torch.empty(101, 80, device=DEV)
    hm.expert_gradient(X, dY, G, off)
    hm.expert_product(dY, W, dX, off, w_trans=True)

    def loss(x, w):
        y = torch.empty(101, 48, device=DEV)
        hm.expert_product(x, w, y, off)
        return float((y.double() * dY.double()).sum())

    base = loss(X, W)
    # every fp32 output of a forward product is within (K + 16) 2^-23 sum |x| |w| of its sum; times |dY|, summed
    err = 2 * (80 + 16) * 2.0 ** -23 * float((X.double().abs().sum(1) * 6 * dY.double().abs().sum(1)).sum())
    for e, i, j in [(0, 0, 0), (0, 79, 47), (1, 3, 3), (2, 17, 40)]:
        w = W.clone()
        w[e, i, j] = W[e, i, j] + 4
        h = float(w[e, i, j].double() - W[e, i, j].double())
        x = X[slice(*groups(off)[e]), i].double() @ dY[slice(*groups(off)[e]), j].double()
        assert abs((loss(X, w) - base) / h - float(G[e, i, j])) <= err / abs(h) + 1e-4 * abs(float(x))
    for r, i in [(0, 0), (36, 79), (37, 5), (100, 33)]:
        x = X.clone()
        x[r, i] = X[r, i] + 4
        h = float(x[r, i].double() - X[r, i].double())
        assert abs((loss(x, W) - base) / h - float(dX[r, i])) <= err / abs(h) + 1e-4 * abs(float(dX[r, i]))


# ---------------------------------------------------------------- 8 bits
def exact_codes(x):
    x = x.double()
    top = x.abs().amax(1, keepdim=True)
    return torch.where(top > 0, 127 * x / top, torch.zeros_like(x)), top[:, 0]


@pytest.mark.parametrize("dim", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 8), (33, 257), (64, 4096), (1000, 72), (3, 11008)])
def test_quantize(hm, dim, dtype, rows, cols):
    x = matrix((rows, cols), TYPES[dtype], gen(rows + cols), 2.0, margin=16)
    x[rows // 2] = 0
    if rows > 1:
        x[0] = x[0].abs().amax() * torch.randint(-254, 255, (cols,), generator=gen(1), device=DEV).to(x.dtype) / 254
        x[0, 0] = x[0].abs().amax()
    xt = x.T if dim else x
    L, n = xt.shape
    q = torch.full((L, -(-n // 16) * 16 + 16), 99, dtype=torch.int8, device=DEV)
    s = torch.empty(L, device=DEV)
    hm.quantize([x], [q[:, :n]], [s], dim=dim)
    want, top = exact_codes(xt)
    assert torch.equal(s, (top / 127).float())
    if dtype == "fp32":   # 127 x and the quotient are each rounded: a code may fall to the other side of a near tie
        assert ((q[:, :n].double() - want).abs() <= 0.5 + 127 * 2.0 ** -22).all()
    else:                 # halves are met exactly (round's ties go to even, as the codes')
        assert torch.equal(q[:, :n].double(), want.round())
    assert (q[:, n:] == 99).all()
    assert hm.device_status() == 0


def test_quantize_lists_and_nonfinite(hm):
    g = gen(5)
    shapes = [(3, 40), (100, 8), (1, 300)] * 30
    xs = [matrix(s, [torch.bfloat16, torch.float32][i % 2], g) for i, s in enumerate(shapes)]
    xs[0][1, 7], xs[1][50, 3], xs[3][0, 0] = float("nan"), float("-inf"), float("inf")
    qs = [torch.full((r, -(-c // 16) * 16), 99, dtype=torch.int8, device=DEV)[:, :c] for r, c in shapes]
    ss = [torch.empty(r, device=DEV) for r, _ in shapes]
    hm.quantize(xs, qs, ss)
    for i, (x, q, s) in enumerate(zip(xs, qs, ss)):
        fine = torch.isfinite(x).all(1)
        want, top = exact_codes(x[fine])
        assert ((q[fine].double() - want).abs() <= 0.5 + 127 * 2.0 ** -22).all()
        assert torch.equal(s[fine], (top / 127).float())
        assert s[~fine].isnan().all() and (q[~fine] == 0).all()
    assert int(sum((~torch.isfinite(x).all(1)).sum() for x in xs)) == 3
    big = matrix((4, 264), torch.bfloat16, g, 1e37)       # 127 x is out of fp32's range
    big[1] *= 20
    for dim in (0, 1):
        q = torch.empty(4, 272, dtype=torch.int8, device=DEV)[:, :264] if dim == 0 else \
            torch.empty(264, 16, dtype=torch.int8, device=DEV)[:, :4]
        s = torch.empty(4 if dim == 0 else 264, device=DEV)
        hm.quantize([big], [q], [s], dim=dim)
        lines = big.T if dim else big                        # (row 1 overflows bf16 in places)
        fine = torch.isfinite(lines).all(1)
        want, top = exact_codes(lines[fine])
        assert torch.equal(q[fine].double(), want.round()) and torch.equal(s[fine], (top / 127).float())
        assert s[~fine].isnan().all() and (q[~fine] == 0).all()
    assert hm.device_status() == 0
    tiny = torch.tensor([[1e-40, -2e-40, 0, 0]] * 2, dtype=torch.bfloat16, device=DEV).repeat(1, 2).contiguous()
    q, s = torch.empty(2, 16, dtype=torch.int8, device=DEV)[:, :8], torch.empty(2, device=DEV)
    hm.quantize([tiny], [q], [s])
    assert torch.equal(q.double(), exact_codes(tiny)[0].round())
    hm.quantize([tiny[:0]], [q[:0]], [s[:0]])


@pytest.mark.parametrize("dim", [0, 1])
def test_quantize_stacked(hm, dim):
    """Stacked matrices, codes and scales give what the lists give."""
    x = matrix((5, 96, 136), torch.bfloat16, gen(41), margin=8)
    L, n = (136, 96) if dim else (96, 136)
    q, q2 = (torch.full((5, L, -(-n // 16) * 16 + 16), 99, dtype=torch.int8, device=DEV)[:, :, :n] for _ in range(2))
    s, s2 = (torch.zeros(5, L + 4, device=DEV)[:, :L] for _ in range(2))
    hm.quantize(x, q, s, dim=dim)
    hm.quantize(list(x), list(q2), list(s2), dim=dim)
    assert torch.equal(q, q2) and torch.equal(s, s2) and (s > 0).all()
    for e in range(5):
        want, top = exact_codes(x[e].T if dim else x[e])
        assert torch.equal(q[e].double(), want.round()) and torch.equal(s[e], (top / 127).float())


def check_i8(hm, out, K, N, counts, start=0, behind=0, listed=False, full=False, seed=0):
    g = gen(seed)
    n, off = len(counts), offsets(counts, start)
    rows = start + sum(counts) + behind
    pitch = -(-K // 16) * 16 + 16
    lo, hi = (127, 128) if full else (-128, 128)
    X = torch.randint(lo, hi, (rows, pitch), generator=g, device=DEV).to(torch.int8)[:, :K]
    W = torch.randint(lo, hi, (n, N, pitch), generator=g, device=DEV).to(torch.int8)[:, :, :K]
    xs = torch.rand(rows, generator=g, device=DEV) + 0.01
    ws = torch.rand(n, N + 3, generator=g, device=DEV)[:, :N] + 0.01
    xs[:start] = float("nan")
    Y = torch.full((rows, -(-N // 8) * 8 + 8), -7.0, device=DEV).to(out)
    hm.expert_product_i8(X, xs, [w for w in W] if listed else W, ws, Y[:, :N], off)
    assert hm.device_status() == 0
    for e, (a, b) in enumerate(groups(off)):
        exact = (X[a:b].double() @ W[e].double().T) * xs[a:b].double()[:, None] * ws[e].double()
        close(Y[a:b, :N], exact, exact.abs(), 0, out)
    assert (Y[:start] == -7).all() and (Y[rows - behind:] == -7).all() and (Y[:, N:] == -7).all()


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("K,N,counts", [
    (128, 128, [1]),
    (1, 1, [3, 0, 1]),
    (200, 136, [5, 0, 33, 130, 1]),
    (129, 257, [31, 32, 33, 0]),
    (1024, 384, [300, 257, 0, 256, 17]),
    (4096, 136, [2, 9, 1, 1]),
])
def test_product_i8(hm, out, K, N, counts):
    check_i8(hm, TYPES[out], K, N, counts, seed=K + N) if out != "fp16" else check_i8_small(hm, K, N, counts)


def check_i8_small(hm, K, N, counts):
    """fp16 results: scales that keep them in fp16's range."""
    g = gen(K)
    off, rows = offsets(counts), sum(counts)
    pitch = -(-K // 16) * 16
    X = torch.randint(-128, 128, (rows, pitch), generator=g, device=DEV).to(torch.int8)[:, :K]
    W = torch.randint(-128, 128, (len(counts), N, pitch), generator=g, device=DEV).to(torch.int8)[:, :, :K]
    xs, ws = torch.full((rows,), 1e-3, device=DEV), torch.full((len(counts), N), 2e-3, device=DEV)
    Y = torch.empty(rows, -(-N // 8) * 8, device=DEV, dtype=torch.float16)[:, :N]
    hm.expert_product_i8(X, xs, W, ws, Y, off)
    for e, (a, b) in enumerate(groups(off)):
        exact = (X[a:b].double() @ W[e].double().T) * xs[a:b].double()[:, None] * ws[e].double()
        close(Y[a:b], exact, exact.abs(), 0, torch.float16)


def test_product_i8_edges(hm):
    check_i8(hm, torch.float32, 300, 200, [40, 0, 20], start=5, behind=9, listed=True)
    check_i8(hm, torch.float32, 11008, 64, [3, 5], full=True)                    # sums beyond 2^24
    check_i8(hm, torch.bfloat16, 131071, 8, [2], full=True)                      # the longest sum
    check_i8(hm, torch.bfloat16, 64, 72, np.random.default_rng(1).integers(0, 3, 300).tolist())


# ---------------------------------------------------------------- how they are called
@pytest.mark.parametrize("op", ["product", "product_few_tiles", "gradient", "gradient_few_tiles"])
def test_device_timeout_is_reported_and_the_next_call_is_right(hm, op):
    """HIMUON_TEST_STALL=1 makes the first pair's MMA warp wait on a barrier that nothing arrives on: every other wait
    of its cluster then runs out too (two seconds), the kernel ends, and the status says so."""
    import os
    g = gen(31)
    few = op.endswith("few_tiles")
    K, N, rows = 1024, 256 if few else 8192, 300
    X, W, dY = (matrix(s, torch.bfloat16, g) for s in ((rows, K), (1, K, N), (rows, N)))
    Y, C = torch.zeros(rows, N, device=DEV), matrix((1, K, N), torch.float32, g)
    G = torch.zeros(1, K, N, device=DEV)
    run = (lambda: hm.expert_product(X, W, Y)) if op.startswith("product") else \
        (lambda: hm.expert_gradient(X, dY, G, beta=1.0, C=C))
    assert hm.device_status() == 0
    os.environ["HIMUON_TEST_STALL"] = "1"
    try:
        run()
        status = hm.device_status()
    finally:
        del os.environ["HIMUON_TEST_STALL"]
    assert status == -6                                                          # HIMUON_ERR_TIMEOUT
    assert hm.device_status() == 0
    run()
    x, w, dy = X.double(), W[0].double(), dY.double()
    if op.startswith("product"):
        close(Y, x @ w, x.abs() @ w.abs(), K, torch.float32)
    else:
        close(G[0], x.T @ dy + C[0].double(), x.abs().T @ dy.abs() + C[0].double().abs(), rows, torch.float32)
    assert hm.device_status() == 0


def test_bad_offsets_are_reported_and_stay_in_bounds(hm):
    g = gen(11)
    X, W = matrix((40, 64), torch.bfloat16, g), matrix((3, 64, 32), torch.bfloat16, g)
    Y = torch.full((60, 32), -7.0, device=DEV, dtype=torch.bfloat16)
    G = torch.empty(3, 64, 32, device=DEV)
    q, w8 = torch.ones(40, 64, dtype=torch.int8, device=DEV), torch.ones(3, 32, 64, dtype=torch.int8, device=DEV)
    s1, s2 = torch.ones(40, device=DEV), torch.ones(3, 32, device=DEV)
    for bad in ([0, 10, 5, 40], [-3, 10, 20, 40], [0, 10, 20, 55], [0, 50, 20, 40], [70, 80, 90, 100]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        hm.expert_product(X, W, Y[:40], off)
        assert hm.device_status() == -7                                          # HIMUON_ERR_DEVICE
        hm.expert_gradient(X, X[:, :32], G, off)
        assert hm.device_status() == -7
        hm.expert_product_i8(q, s1, w8, s2, Y[:40], off)
        assert hm.device_status() == -7
    assert (Y[40:] == -7).all()
    assert hm.device_status() == 0


def test_streams_and_graph_replay_with_new_offsets(hm):
    """Two streams at once; two captured graphs, replayed in turn with other
    offsets and inputs in the same buffers, beside eager calls."""
    g = gen(12)
    X, W = matrix((600, 256), torch.bfloat16, g), matrix((4, 256, 384), torch.bfloat16, g)
    dY = matrix((600, 384), torch.bfloat16, g)
    off = offsets([100, 200, 0, 300])
    other = offsets([256, 1, 343, 0])

    def eager(o):
        y, gr = torch.zeros(600, 384, device=DEV), torch.zeros(4, 256, 384, device=DEV)
        hm.expert_product(X, W, y, o)
        hm.expert_gradient(X, dY, gr, o)
        return y, gr

    want, want_other = eager(off), eager(other)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for s, o in ((s1, off), (s2, other), (s1, other), (s2, off)):
        y, gr = torch.zeros(600, 384, device=DEV), torch.zeros(4, 256, 384, device=DEV)
        torch.cuda.synchronize()
        got.append((y, gr, o, s))
    for y, gr, o, s in got:
        hm.expert_product(X, W, y, o, stream=s)
        with torch.cuda.stream(s):
            hm.expert_gradient(X, dY, gr, o)
    torch.cuda.synchronize()
    for y, gr, o, _ in got:
        w = want if o is off else want_other
        assert torch.equal(y, w[0]) and torch.equal(gr, w[1])

    cur = off.clone()
    outs = [(torch.zeros(600, 384, device=DEV), torch.zeros(4, 256, 384, device=DEV)) for _ in range(2)]
    graphs = []
    for y, gr in outs:
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            hm.expert_product(X, W, y, cur)
            hm.expert_gradient(X, dY, gr, cur)
        graphs.append(gph)
    for turn, (o, w) in enumerate(((off, want), (other, want_other), (off, want))):
        cur.copy_(o)
        for gph in graphs:
            gph.replay()
        y2, g2 = eager(o)
        torch.cuda.synchronize()
        for y, gr in (*outs, (y2, g2)):
            assert torch.equal(y, w[0]) and torch.equal(gr, w[1])
    assert hm.device_status() == 0


@pytest.mark.parametrize("captured", [False, True])
def test_launches_wait_for_work_of_other_streams_and_of_torch(hm, captured):
    """A launch may start under the end of the one before it, but not ahead of what its stream waits for: inputs that
    another stream, a torch kernel or a copy writes between two calls, and outputs that a torch kernel reads."""
    g = gen(43)
    src = [matrix((512, 512), torch.bfloat16, g, fill=0.0) for _ in range(4)]
    big = torch.randn(3000, 3000, generator=g, device=DEV)
    X, W = torch.zeros(512, 512, dtype=torch.bfloat16, device=DEV), matrix((2, 512, 256), torch.bfloat16, g)
    off = offsets([200, 312])
    Y = torch.zeros(512, 256, device=DEV)
    keep = [torch.zeros(512, 256, device=DEV) for _ in range(8)]
    slow = torch.zeros(3000, 3000, device=DEV)
    other = torch.cuda.Stream()

    def work():
        main = torch.cuda.current_stream()
        for i in range(8):
            other.wait_stream(main)
            with torch.cuda.stream(other):
                torch.mm(big, big, out=slow)          # long enough for a call that does not wait to be early
                if i % 2:
                    X.copy_(src[i % 4])
                else:
                    torch.add(src[i % 4], 0, out=X)
            hm.expert_product(src[0], W, Y, off)      # the launch before, with nothing to wait for
            main.wait_stream(other)
            hm.expert_product(X, W, Y, off)
            keep[i].copy_(Y)

    if captured:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            work()
        torch.cuda.synchronize()
        for k in keep:
            k.zero_()
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            work()
        gph.replay()
    else:
        work()
    torch.cuda.synchronize()
    for i in range(8):
        want = torch.zeros(512, 256, device=DEV)
        hm.expert_product(src[i % 4], W, want, off)
        assert torch.equal(keep[i], want), i
    assert hm.device_status() == 0


def test_calls_from_several_host_threads(hm):
    """Each thread on its own stream, calls of every kind at once."""
    import threading
    g = gen(42)
    X, W = matrix((700, 256), torch.bfloat16, g), matrix((6, 256, 320), torch.bfloat16, g)
    off = offsets([100, 0, 255, 45, 299, 1])
    want = torch.zeros(700, 320, device=DEV)
    hm.expert_product(X, W, want, off)
    want_g = torch.zeros(6, 256, 256, device=DEV)
    hm.expert_gradient(X, X, want_g, off)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            y, gr = torch.zeros(700, 320, device=DEV), torch.zeros(6, 256, 256, device=DEV)
            q, qs = torch.zeros(700, 256, dtype=torch.int8, device=DEV), torch.zeros(700, device=DEV)
            for _ in range(20):
                hm.expert_product(X, list(W), y, off)
                hm.expert_gradient(X, X, gr, off)
                hm.quantize([X], [q], [qs])
            s.synchronize()
            if not (torch.equal(y, want) and torch.equal(gr, want_g) and bool(q.abs().amax(1).eq(127).all())):
                bad.append(1)

    ts = [threading.Thread(target=work) for _ in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad and hm.device_status() == 0


def test_results_do_not_depend_on_other_groups_or_repeat(hm):
    """The same call twice gives the same bits; so does a group alone and among others of other sizes."""
    g = gen(13)
    X, W = matrix((900, 512), torch.bfloat16, g), matrix((5, 512, 256), torch.bfloat16, g)
    off = offsets([300, 0, 100, 477, 23])
    Y = torch.empty(900, 256, device=DEV)
    hm.expert_product(X, W, Y, off)
    Z = torch.empty_like(Y)
    hm.expert_product(X, W, Z, off)
    assert torch.equal(Y, Z)
    G, H = torch.empty(5, 512, 256, device=DEV), torch.empty(5, 512, 256, device=DEV)
    hm.expert_gradient(X, X[:, :256], G, off)
    hm.expert_gradient(X, X[:, :256], H, off)
    assert torch.equal(G, H)


def test_expert_layer_and_optimizer_step(hm):
    """An expert layer's pass as it is used: forward, both gradients, the Muon step on the weights, the stepped
    weights' 8-bit codes and the product with them."""
    import oracle
    from tiled_newton_schulz_b200 import inputs
    g = gen(14)
    n, K, N, rows = 3, 256, 384, 500
    off = offsets([200, 0, 300])
    W = matrix((n, K, N), torch.bfloat16, g, 0.05)
    M = matrix((n, K, N), torch.bfloat16, g, 0.01)
    X = matrix((rows, K), torch.bfloat16, g)
    Y, dX = torch.empty(rows, N, device=DEV, dtype=torch.bfloat16), torch.empty(rows, K, device=DEV, dtype=torch.bfloat16)
    G = torch.empty(n, K, N, device=DEV, dtype=torch.bfloat16)
    w0, m0 = W.double(), M.double()
    hm.expert_product(X, W, Y, off)
    dY = (Y.float() * 1e-3).to(torch.bfloat16)
    hm.expert_product(dY, W, dX, off, w_trans=True)
    hm.expert_gradient(X, dY, G, off)
    x, dy = X.double(), dY.double()
    for e, (a, b) in enumerate(groups(off)):
        close(Y[a:b], x[a:b] @ w0[e], x[a:b].abs() @ w0[e].abs(), K, torch.bfloat16)
        close(dX[a:b], dy[a:b] @ w0[e].T, dy[a:b].abs() @ w0[e].abs().T, N, torch.bfloat16)
        close(G[e], x[a:b].T @ dy[a:b], x[a:b].abs().T @ dy[a:b].abs(), b - a, torch.bfloat16)
    p = hm.params(128, inputs.QUINTIC, steps=5)
    hm.momentum_step(list(W), list(M), list(G), 0.95, 0.02, p)
    c32 = [tuple(float(np.float32(v)) for v in inputs.QUINTIC)] * 5
    for e in range(n):
        w1, _, o = oracle.momentum_step(w0[e].cpu().numpy(), m0[e].cpu().numpy(), G[e].double().cpu().numpy(), 0.95,
                                        0.02, 128, c32)
        got = (w0[e].cpu().numpy() - W[e].double().cpu().numpy()) / 0.02
        # the step's own bound (3e-2 of O) and the rounding of W to bf16, divided by lr
        lim = 3e-2 * np.linalg.norm(o) + 2.0 ** -8 * np.linalg.norm(w1) / 0.02
        assert np.linalg.norm(got - o) <= lim
    q = torch.empty(n, N, K, dtype=torch.int8, device=DEV)
    ws = torch.empty(n, N, device=DEV)
    hm.quantize(list(W), list(q), list(ws), dim=1)
    xq, xs = torch.empty(rows, K, dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
    hm.quantize([X], [xq], [xs])
    Y8 = torch.empty(rows, N, device=DEV)
    hm.expert_product_i8(xq, xs, q, ws, Y8, off)
    hm.expert_product(X, W, Y, off)
    for e, (a, b) in enumerate(groups(off)):
        # each code is off by at most half a step of its row's or channel's scale
        ex, ew = xs[a:b].double()[:, None] / 2, ws[e].double()[None, :] / 2
        lim = (x[a:b].abs().sum(1, keepdim=True) * ew + ex * W[e].double().abs().sum(0, keepdim=True) + K * ex * ew)
        d = (Y8[a:b].double() - x[a:b] @ W[e].double()).abs()
        assert (d <= lim * (1 + 2.0 ** -20)).all()
    assert hm.device_status() == 0


# ---------------------------------------------------------------- long sums
def long_sum_limit(length, dtype, equal=False):
    """The relative error of a sum of terms of one sign and of similar size, rounded to dtype.

    Per 16 products the tensor core cuts each product at a quarter of the last place of the sum so far and the sum at
    its last place: 5 places at most, 2.5 on average (equal terms may lose the most every time).  The last place of a
    sum that grows evenly is on average at most 0.89 2^-24 of what it ends as (the worst end is 3 2^k: (1 + 1/2 + 1/4
    + ..) 2^-22 2 / 9).  So a piece of c elements loses at most 2.25 (equal terms) or on average 1.12 (1.25 with a
    margin for the average) times c / 16 2^-23.  Pieces have 512 elements for fp32, 4096 for fp16, 32768 for bf16
    results and at least the root of twice the length beyond 2^20; every addition of a piece is off by 2^-24 of what
    has been added up."""
    f = torch.finfo(dtype)
    c = {torch.float32: 2 ** 9, torch.float16: 2 ** 12, torch.bfloat16: 2 ** 15}[dtype]
    while length > 2 ** 20 and c * c < 2 * length:
        c *= 2
    loss = (2.25 if equal else 1.25) * min(c, length) / 16 * 2.0 ** -23 + length / c * 2.0 ** -24
    return f.eps / 2 * (1 + 2 ** -8) + loss + 16 * 2.0 ** -23


def one_sign(shape, dtype, g, scale):
    """Values in [1, 2) x scale, a power of two."""
    t = torch.empty(shape, device=DEV, dtype=dtype)
    for part in t.flatten().split(1 << 26):
        part.copy_((torch.rand(part.shape, generator=g, device=DEV) + 1) * scale)
    return t


@pytest.mark.parametrize("length", [4096, 4097, 33000, 300000, 1 << 22])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_gradient_sums_of_one_sign(hm, dtype, length):
    """A long group among many, so that no pairs share its tile; results of every type."""
    g, n, P, Q = gen(51), 40, 64, 48
    scale = 2.0 ** -int(np.log2(length) / 2)      # results near 2
    A, B = one_sign((length + 6, P), TYPES[dtype], g, scale), one_sign((length + 6, Q), TYPES[dtype], g, scale)
    counts = [0] * n
    counts[3], counts[17], counts[39] = 2, length, 4
    exact = sum(x.double().T @ y.double() for x, y in zip(A[2:length + 2].split(1 << 18), B[2:length + 2].split(1 << 18)))
    for out in {TYPES[dtype], torch.float32}:
        G = torch.empty(n, P, Q, device=DEV, dtype=out)
        hm.expert_gradient(A, B, G, offsets(counts))
        assert hm.device_status() == 0
        off = float(((G[17].double() - exact) / exact).abs().max())
        assert off <= long_sum_limit(length, out), (out, off)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("length", [4096, 4104, 33000, 300000, 1 << 22])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_product_sums_of_one_sign(hm, dtype, length, trans):
    g, n, N, rows = gen(52), 64, 48, 64
    scale = 2.0 ** -int(np.log2(length) / 2)
    X = one_sign((rows, length), TYPES[dtype], g, scale)
    W = one_sign((N, length) if trans else (length, N), TYPES[dtype], g, scale)
    w = W.T if trans else W
    exact = sum(x.double() @ y.double() for x, y in zip(X.split(1 << 18, dim=1), w.split(1 << 18)))
    counts = [0] * n
    counts[5], counts[41] = 1, rows - 1
    for out in {TYPES[dtype], torch.float32}:
        Y = torch.empty(rows, N, device=DEV, dtype=out)
        hm.expert_product(X, W.expand(n, -1, -1), Y, offsets(counts), w_trans=trans)
        assert hm.device_status() == 0
        off = float(((Y.double() - exact) / exact).abs().max())
        assert off <= long_sum_limit(length, out), (out, off)


def test_gradient_longest_sums_of_equal_terms(hm):
    """Equal terms: every addition of a piece is off in the same direction."""
    rows, n = 1 << 25, 40
    A, B = torch.full((rows, 8), 1 / 3, device=DEV, dtype=torch.bfloat16), torch.full((rows, 8), 1.7, device=DEV).bfloat16()
    exact = float(A[0, 0].double() * B[0, 0].double())
    counts = [0] * n
    counts[20] = rows
    for many in (counts, [rows]):                  # a tile of its own, and one shared by pairs
        for out in (torch.float16, torch.bfloat16, torch.float32):
            G = torch.empty(len(many), 8, 8, device=DEV, dtype=out)
            hm.expert_gradient(A, B, G, offsets(many), alpha=1 / rows)
            off = float((G[len(many) // 2].double() / exact - 1).abs().max())
            assert off <= long_sum_limit(rows, out, equal=True), (len(many), out, off)
    assert hm.device_status() == 0


@pytest.mark.parametrize("P,Q", [(64, 64), (136, 267), (520, 1032)])
def test_gradient_16_bit_results_of_long_groups(hm, P, Q):
    """Groups long enough for their sums to run in pieces; the forms of C, views, lists."""
    f16, bf = torch.float16, torch.bfloat16
    counts = [0] * 37 + [5, 33000, 64]
    check_gradient(hm, f16, f16, P, Q, counts, alpha=2.0 ** -4)
    check_gradient(hm, f16, f16, P, Q, counts, alpha=2.0 ** -4, beta=0.5, alias=True, margin=8, start=3, behind=9)
    check_gradient(hm, bf, f16, P, Q, counts, alpha=2.0 ** -4, beta=-1.0, cdtype=torch.float32, listed=True)
    if P == 136:
        check_gradient(hm, bf, bf, P, Q, [0] * 37 + [70, 263000, 1], beta=1.0, cdtype=f16)


@pytest.mark.parametrize("trans", [False, True])
def test_product_16_bit_results_of_long_sums(hm, trans):
    f16, bf = torch.float16, torch.bfloat16
    check_product(hm, f16, f16, 32776, 264, [70, 0, 500, 3], trans, start=2, behind=5, margin=8)
    check_product(hm, bf, f16, 33001, 2050, [300, 513], trans, listed=True)
    check_product(hm, bf, bf, 262200, 72, [1] * 45, trans)


def test_gradient_host_work_does_not_grow_with_the_width(hm):
    """A call's work on the host is that of a few tile widths, whatever the columns (each time the quickest of several
    calls, with nothing queued before it)."""
    import time
    g = gen(61)

    def quickest(Q):
        A, B = matrix((2000, 8), torch.bfloat16, g), torch.ones(2000, Q, device=DEV, dtype=torch.bfloat16)
        G = torch.empty(1, 8, Q, device=DEV, dtype=torch.bfloat16)
        best = float("inf")
        for _ in range(20):
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            hm.expert_gradient(A, B, G)
            best = min(best, time.perf_counter() - t0)
        want = A.double().sum(0)[:, None].expand(-1, Q)
        close(G[0], want, A.double().abs().sum(0)[:, None], 2000, torch.bfloat16)
        return best

    narrow, wide = quickest(4096), quickest(113408)
    assert wide <= 3 * narrow, (narrow, wide)


@pytest.mark.parametrize("form", ["plain", "add", "views", "listed", "bf16", "none_long", "all_empty"])
def test_gradient_long_groups_in_a_launch_of_their_own(hm, form):
    """Large calls with 16-bit results: groups whose sums run in one piece and the others, in two launches."""
    f16, bf, n = torch.float16, torch.bfloat16, 64
    rng = np.random.default_rng(71)
    counts = rng.integers(0, 90, n)
    counts[[0, 7, 31, 32, 63]] = 4097, 4096, 9000, 0, 5001
    if form == "none_long":
        counts[[0, 31, 63]] = 4096, 4095, 1
    if form == "bf16":
        counts[[3, 9]] = 32769, 32768
    if form == "all_empty":
        counts[:] = 0
    kw = dict(plain=dict(), add=dict(beta=0.5, alias=True), views=dict(start=5, behind=77, margin=8, beta=1.0, cdtype=bf),
              listed=dict(listed=True, beta=-1.0, cdtype=torch.float32), bf16=dict(beta=1.0), none_long=dict(),
              all_empty=dict(beta=2.0, behind=5000))[form]
    dtype = bf if form == "bf16" else f16
    before = hm.launch_count()
    check_gradient(hm, dtype, dtype, 1032, 1027, counts.tolist(), alpha=2.0 ** -4, **kw)
    assert hm.launch_count() - before == 2


def test_gradient_long_groups_replayed_with_other_offsets(hm):
    """A captured call: groups that become longer or shorter than a piece go to the other launch."""
    g, n, rows, P, Q = gen(72), 80, 12000, 520, 1288
    A, B = matrix((rows, P), torch.float16, g, 0.1), matrix((rows, Q), torch.float16, g)
    first, second = [150] * n, [0] * n
    second[4], second[5], second[79] = 5000, 4096, 2904
    cur = offsets(first)
    G = torch.empty(n, P, Q, device=DEV, dtype=torch.float16)
    hm.expert_gradient(A, B, G, cur)
    torch.cuda.synchronize()
    before = hm.launch_count()
    gph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gph):
        hm.expert_gradient(A, B, G, cur)
    assert hm.launch_count() - before == 2
    for counts in (second, first, second):
        off = offsets(counts)
        cur.copy_(off)
        G.fill_(float("nan"))
        gph.replay()
        torch.cuda.synchronize()
        for e, (a, b) in enumerate(groups(off)):
            if b == a:
                assert (G[e] == 0).all()
                continue
            x, y = A[a:b].double(), B[a:b].double()
            close(G[e], x.T @ y, x.abs().T @ y.abs(), b - a, torch.float16)
    cur.copy_(torch.tensor([0, 40, 20] + [12000] * (n - 2), dtype=torch.int32))
    gph.replay()
    assert hm.device_status() == -7
    assert hm.device_status() == 0


@pytest.mark.parametrize("dim", [0, 1])
@pytest.mark.parametrize("scale,length", [(1.0, 0), (1.0, 13001), (1.0, 140003), (2.0 ** -75, 0), (2.0 ** 90, 5003),
                                          (2.0 ** -130, 0)])
def test_quantize_fp32_next_to_ties(hm, dim, scale, length):
    """fp32 values at, and a few units to either side of, the borders between codes, with maxima inside and outside
    the range of the short division and below the normal numbers.  127 x is exact in 64 bits and the quotient, if no
    tie, at least 2^-33 from one, so its rounding in 64 bits falls to the right side."""
    rows = 96
    rng = np.random.default_rng(81)
    top = (rng.random(rows) + 1).astype(np.float32)
    top[:8] = 127 * 2.0 ** -6, 254 * 2.0 ** -7, 127 * 3 * 2.0 ** -8, 127 * 5 * 2.0 ** -9, 1.5, 1.25, 1, 127 * 7 * 2.0 ** -9
    half = np.arange(-127, 127) + 0.5
    bits = (half * top[:, None].astype(np.float64) / 127).astype(np.float32).view(np.int32)
    x = np.concatenate([(bits + d).view(np.float32) for d in range(-4, 5)] + [top[:, None]], axis=1)
    x = torch.from_numpy((x.astype(np.float64) * scale).astype(np.float32))
    assert (x.abs().amax(1) == x[:, -1]).all()
    length = length or x.shape[1]
    x = x[:, torch.arange(length) % x.shape[1]]
    pad = torch.zeros(rows, -(-length // 4) * 4 - length)
    X = torch.cat([x, pad], 1).cuda()
    X = X.T.contiguous() if dim else X
    L, n = (X.shape[1], X.shape[0]) if dim else X.shape
    q, s = torch.empty(L, -(-n // 16) * 16, dtype=torch.int8, device=DEV)[:, :n], torch.empty(L, device=DEV)
    hm.quantize([X], [q], [s], dim=dim)
    lines = X.T if dim else X
    want, top = exact_codes(lines)
    assert torch.equal(q.double(), want.round())
    assert torch.equal(s, (top / 127).float())
    assert hm.device_status() == 0


# ---------------------------------------------------------------- fp32 results as a whole
# An uncut sum of 1100 terms of either sign is off by 1.1e-6 of itself (relative norms), 1.6e-8 per 16 terms.  Pieces
# of 512 make that 32 x 1.6e-8 = 5.1e-7 of each piece, whose errors are independent, so 5.1e-7 of the sum however
# many there are; rounding adds 0.3e-7.  The limit lies half way (in ratio) to the uncut sum's error at 1100 terms;
# 4096 uncut terms are off by 4e-6.
NORM = 7.5e-7


def norm_error(y, exact):
    return float((y.double() - exact).norm() / exact.norm())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("length", [1100, 4096])
def test_norm_of_errors_of_fp32_results(hm, dtype, length, few):
    """few: tiles that several pairs share."""
    g, t = gen(91), TYPES[dtype]
    n, rows, N = (1, 100, 264) if few else (40, 400, 2056)
    off = offsets([rows] if few else [rows // n] * n)
    X = matrix((rows, length), t, g)
    for trans in (False, True):
        W = matrix((n, N, length) if trans else (n, length, N), t, g)
        Y = torch.empty(rows, N, device=DEV)
        hm.expert_product(X, W, Y, off, w_trans=trans)
        exact = torch.cat([X[a:b].double() @ (w.double().T if trans else w.double()) for (a, b), w in zip(groups(off), W)])
        assert norm_error(Y, exact) <= NORM, trans
    P = 200 if few else 1032
    counts = [length] if few else [length, 0, length]
    A, B = matrix((sum(counts), P), t, g), matrix((sum(counts), N), t, g)
    G = torch.empty(len(counts), P, N, device=DEV)
    hm.expert_gradient(A, B, G, offsets(counts))
    for e in range(0, len(counts), 2):
        a = length * (e // 2)
        assert norm_error(G[e], A[a:a + length].double().T @ B[a:a + length].double()) <= NORM, e
    assert hm.device_status() == 0


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
def test_a_group_alone_and_among_others(hm, out):
    """The order of a group's sums may depend on the call's other groups (which tiles are shared), its values only
    within the rounding: fp32 norms within two errors, 16-bit values at most one step apart beyond two sums' errors."""
    g, t = gen(92), TYPES[out]
    n, K, N, rows = 24, 1100, 520, 2400
    counts = [100] * n
    counts[7], counts[8] = 190, 10
    off = offsets(counts)
    a, b = groups(off)[7]
    X, W, dY = matrix((rows, K), torch.bfloat16, g), matrix((n, K, N), torch.bfloat16, g, 0.1), matrix((rows, N), torch.bfloat16, g)
    Y, Y1 = torch.empty(rows, N, device=DEV, dtype=t), torch.empty(b - a, N, device=DEV, dtype=t)
    G, G1 = torch.empty(n, K, N, device=DEV, dtype=t), torch.empty(1, K, N, device=DEV, dtype=t)
    hm.expert_product(X, W, Y, off)
    hm.expert_product(X[a:b], W[7:8], Y1)
    hm.expert_gradient(X, dY, G, off)
    hm.expert_gradient(X[a:b], dY[a:b], G1)
    x, w, dy = X[a:b].double(), W[7].double(), dY[a:b].double()
    for many, one, size, k in ((Y[a:b], Y1, x.abs() @ w.abs(), K), (G[7], G1[0], x.abs().T @ dy.abs(), b - a)):
        if out == "fp32":
            assert norm_error(many, one.double()) <= 2 * NORM
            continue
        f = torch.finfo(t)
        lim = f.eps * torch.maximum(many.double().abs(), one.double().abs()) + 2 * (k + 16) * 2.0 ** -23 * size + f.smallest_normal * f.eps
        assert ((many.double() - one.double()).abs() <= lim).all()
    assert hm.device_status() == 0
