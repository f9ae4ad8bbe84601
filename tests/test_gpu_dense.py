"""The 16-bit products on the GPU against plain 64-bit forms: grouped by expert (plain and SwiGLU),
the dense product with its epilogue, the vocabulary cross entropy, and every gradient, at the sizes
where they can go wrong: one row, rows and columns that end inside a tile, experts without rows,
shares, strided and slot-ordered rows, ignored targets, NaN wherever nothing may be read."""
import sys

import pytest
import torch

import dense_ref as R
from dense_ref import CURVE, FEW, SLOPE, U32, check, d, half_step, mm

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
NAN = float("nan")


@pytest.fixture(scope="module")
def dense():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    from quantized_moe_routed_amd import dense as m
    return m


@pytest.fixture(autouse=True)
def _say(request):
    print(f"[gpu-dense] {request.node.name}", flush=True)
    sys.stdout.flush()


def randn(gen, shape, std, dt):
    return (torch.randn(shape, generator=gen) * std).to(dt)


def strided(t, pad, fill=NAN):
    """t on the device with `pad` more elements of `fill` after each row."""
    if not pad:
        return t.cuda()
    big = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    v = big[:, : t.shape[1]]
    v.copy_(t)
    return v


def blank(rows, cols, dt, pad=0, fill=7.0):
    big = torch.full((rows, cols + pad), fill, dtype=dt, device="cuda")
    return big[:, :cols], big


def groups(dense, r):
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    return dense.Groups(c(r.offsets), c(r.slots), r.T, r.k, g2l=c(r.g2l), E_local=r.E_local)


# T, k, E, N, K, x order, out order, out type (None: the input's), owned experts, empty experts, pad
GROUPED = [
    (1, 1, 1, 8, 8, 0, 0, None, None, (), 0),
    (1, 2, 4, 40, 72, 2, 1, torch.float32, None, (), 8),
    (3, 2, 5, 136, 264, 2, 0, None, (3, 0, 2), (0,), 0),
    (17, 1, 3, 64, 64, 1, 1, None, None, (1,), 8),
    (70, 4, 8, 200, 128, 2, 1, torch.float32, (7, 1, 4), (2, 4), 16),
    (333, 3, 6, 328, 200, 2, 0, None, None, (5,), 0),
    (600, 1, 2, 520, 136, 0, 1, None, None, (), 8),
    (130, 8, 130, 48, 520, 2, 1, torch.float32, None, tuple(range(60, 90)), 0),
]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "T%d_k%d_E%d_N%d_K%d" % c[:5])
def test_grouped_matmul(dense, case, dt):
    T, k, E, N, K, xo, yo, ydt, own, empty, pad = case
    g = torch.Generator().manual_seed(T * 31 + N)
    r = R.Routing(T, k, E, 5 + T, empty, own=own)
    x, w = randn(g, (r.rows(xo), K), 1.0, dt), randn(g, (r.E_local, N, K), 0.1, dt)
    out, whole = blank(T * k, N, ydt or dt, pad)
    before = whole.clone()
    got = dense.grouped_matmul(strided(x, pad), w.cuda(), groups(dense, r), x_rows=xo, out_rows=yo, out=out)
    assert got is out
    src, dst = r.index(xo), r.index(yo)
    touched = torch.zeros(T * k, dtype=torch.bool)
    for l, a, b in r.spans():
        if b > a:
            ref, bound = mm(d(x)[src[a:b]], d(w[l]))
            check(out.cpu()[dst[a:b]], ref, bound, f"expert {l}")
            touched[dst[a:b]] = True
    # rows of slots that are not owned and the bytes between the rows keep what they held
    keep = whole.cpu()
    assert torch.equal(keep[~touched], before.cpu()[~touched])
    assert torch.equal(keep[:, N:], before.cpu()[:, N:])


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "T%d_k%d_E%d_N%d_K%d" % c[:5])
def test_grouped_matmul_grad(dense, case, dt):
    T, k, E, N, K, xo, yo, ydt, own, empty, pad = case
    g = torch.Generator().manual_seed(T * 37 + N)
    r = R.Routing(T, k, E, 6 + T, empty, own=own)
    x, w = randn(g, (r.rows(xo), K), 1.0, dt), randn(g, (r.E_local, N, K), 0.1, dt)
    dyo = yo if pad else 2
    dy = randn(g, (r.rows(dyo), N), 0.3, dt)
    acc = T % 2 == 0
    dw0 = randn(g, (r.E_local, N, K), 1.0, ydt or dt)
    dw = dw0.cuda() if acc else torch.full((r.E_local, N, K), NAN, dtype=ydt or dt, device="cuda")
    dx, whole = blank(T * k, K, ydt or dt, pad)
    before = whole.clone()
    dense.grouped_matmul_grad(strided(dy, pad), strided(x, pad), w.cuda(), groups(dense, r), dy_rows=dyo, x_rows=xo,
                              dx_rows=yo, dx=dx, dw=dw, accumulate=acc)
    src, dst, up = r.index(xo), r.index(yo), r.index(dyo)
    touched = torch.zeros(T * k, dtype=torch.bool)
    for l, a, b in r.spans():
        xs, ds = d(x)[src[a:b]], d(dy)[up[a:b]]
        ref, bound = mm(ds.T, xs.T) if b > a else (torch.zeros(N, K).double(), torch.zeros(N, K).double())
        if acc:
            ref = ref + d(dw0[l])
            bound = bound + U32 * ref.abs()
        check(dw[l], ref, bound, f"dw of expert {l}")
        if b > a:
            ref, bound = mm(ds, d(w[l]).T)
            check(dx.cpu()[dst[a:b]], ref, bound, f"dx of expert {l}")
            touched[dst[a:b]] = True
    keep = whole.cpu()
    assert torch.equal(keep[~touched], before.cpu()[~touched])
    assert torch.equal(keep[:, K:], before.cpu()[:, K:])


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (FP, torch.float32)])
@pytest.mark.parametrize("T,k,E,N,K,lead", [(1, 1, 9, 8, 8, 8), (2, 2, 5, 16, 24, 24), (1, 2, 30, 136, 72, 40), (3, 4, 12, 200, 520, 8),
                                            (40, 2, 4, 1032, 1096, 56), (2, 2, 7, 520, 4168, 64)])
def test_weight_gradients_where_most_groups_have_no_rows(dense, T, k, E, N, K, lead, dt, wdt):
    """Zeros for every group without rows, at edges that are no whole lines, and nothing outside."""
    g = torch.Generator().manual_seed(N + K)
    r = R.Routing(T, k, E, 11 + T, tuple(range(1, E - k)) if E > k + 1 else ())
    x, dy = randn(g, (T * k, K), 1.0, dt), randn(g, (T * k, N), 0.3, dt)
    w = torch.zeros((E, N, K), dtype=dt, device="cuda")
    whole = torch.full((lead + E * N * K + 64,), NAN, dtype=wdt, device="cuda")
    whole[:lead] = 7.0
    whole[-64:] = 7.0
    dw = whole[lead:-64].view(E, N, K)
    dense.grouped_matmul_grad(dy.cuda(), x.cuda(), w, groups(dense, r), dw=dw, need_dx=False)
    assert any(a == b for _, a, b in r.spans())
    for l, a, b in r.spans():
        if b > a:
            ref, bound = mm(d(dy)[a:b].T, d(x)[a:b].T)
            check(dw[l], ref, bound, f"dw of expert {l}")
        else:
            assert torch.equal(dw[l], torch.zeros_like(dw[l])), f"expert {l}"
    assert bool((whole[:lead] == 7.0).all()) and bool((whole[-64:] == 7.0).all())


# sizes at which each tile of a product is taken, by the rule in dense.hip: (T, N, K) of dense
# products (forward; the gradient of the rows has K columns and contraction N)
TILES = [(1, 40, 136), (30, 520, 72), (200, 264, 200), (200, 520, 136), (400, 520, 72), (500, 2056, 72), (12, 16392, 72), (250, 2056, 72), (1000, 2056, 72),
         (1030, 4104, 72), (2050, 3976, 72), (4000, 4096, 72)]


@pytest.mark.parametrize("T,N,K", TILES)
@pytest.mark.parametrize("dt", [BF, FP])
def test_every_tile_of_the_dense_product(dense, T, N, K, dt):
    g = torch.Generator().manual_seed(T + N)
    x, w = randn(g, (T, K), 1.0, dt), randn(g, (N, K), 0.2, dt)
    res, bias = randn(g, (T, N), 1.0, dt), randn(g, (N,), 0.5, torch.float32)
    z, bz = mm(d(x), d(w))
    y = dense.linear(strided(x, 8), w.cuda(), bias=bias.cuda(), residual=strided(res, 8))
    r = z + d(bias)[None]
    check(y, r + d(res), bz + U32 * (z.abs() + r.abs() + (r + d(res)).abs()), "y")
    # the transposed storage: dx = dy w with dy [T, K'] of K' = K rows of a weight [K, N]
    wt = w.t().contiguous()
    dx, _, _ = dense.linear_grad(strided(x, 8), torch.empty((T, N), dtype=dt, device="cuda"), wt.cuda(), need_dw=False, need_dbias=False)
    check(dx, z, bz, "dx")
    # loss over N columns from the same product
    t = torch.randint(0, N, (T,), generator=g, dtype=torch.int32)
    _, _, lse, nll, b, _ = loss_ref(x, w, t)
    gn, gl = dense.cross_entropy(strided(x, 8), w.cuda(), t.cuda())
    check(gl, lse, b, "lse")
    check(gn, nll, 2 * b, "nll")


# tokens, experts, columns: 5, 30, 100 and 700 rows an expert, ragged, some experts without rows
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,k,E,N,K", [(40, 4, 32, 1032, 72), (120, 4, 16, 2056, 72), (300, 4, 12, 4104, 72), (1000, 4, 6, 4104, 72),
                                       (90, 4, 12, 2056, 136), (40, 2, 16, 520, 520)])
def test_every_tile_of_the_grouped_products(dense, T, k, E, N, K, dt):
    g = torch.Generator().manual_seed(T + N)
    r = R.Routing(T, k, E, 3, empty=(1,), skew=0.15)
    x, w, w2 = randn(g, (T, K), 1.0, dt), randn(g, (E, N, K), 0.2, dt), randn(g, (E, N, K), 0.2, dt)
    gr = groups(dense, r)
    src = r.index(2)
    xd, wd = strided(x, 8), w.cuda()
    y = dense.grouped_matmul(xd, wd, gr, x_rows=2)
    h = dense.grouped_swiglu(xd, wd, w2.cuda(), gr)
    wt = w.transpose(1, 2).contiguous().cuda()
    dx, _ = dense.grouped_matmul_grad(xd, torch.empty((T * k, N), dtype=dt, device="cuda"), wt, gr, dy_rows=2, need_dw=False)
    for l, a, b in r.spans():
        if b > a:
            ref, bound = mm(d(x)[src[a:b]], d(w[l]))
            check(y[a:b], ref, bound, f"y of expert {l}")
            check(dx[a:b], ref, bound, f"dx of expert {l}")
            _, _, _, _, rh, bh = swiglu_ref(d(x)[src[a:b]], d(w[l]), d(w2[l]))
            check(h[a:b], rh, bh, f"h of expert {l}")


def swiglu_ref(xs, gw, uw):
    g, bg = mm(xs, gw)
    u, bu = mm(xs, uw)
    h = g * R.sig(g) * u
    # silu(g) moves by at most SLOPE bg, and costs a few fp32 steps of itself
    return g, bg, u, bu, h, (SLOPE * bg) * (u.abs() + bu) + (g * R.sig(g)).abs() * bu + FEW * h.abs()


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "T%d_k%d_E%d_I%d_H%d" % c[:5])
def test_grouped_swiglu_and_its_gradients(dense, case, dt):
    T, k, E, I, H, xo, yo, _, own, empty, pad = case
    g = torch.Generator().manual_seed(T * 41 + I)
    r = R.Routing(T, k, E, 7 + T, empty, own=own)
    x = randn(g, (r.rows(xo), H), 1.0, dt)
    gw, uw = randn(g, (r.E_local, I, H), 0.1, dt), randn(g, (r.E_local, I, H), 0.1, dt)
    gr = groups(dense, r)
    h, whole = blank(T * k, I, dt, pad)
    kg, ku = blank(T * k, I, dt, pad)[0], blank(T * k, I, dt, 2 * pad)[0]
    xd, gd, ud = strided(x, pad), gw.cuda(), uw.cuda()
    dense.grouped_swiglu(xd, gd, ud, gr, x_rows=xo, out_rows=yo, out=h, keep_g=kg, keep_u=ku)
    src, dst = r.index(xo), r.index(yo)
    for l, a, b in r.spans():
        if b > a:
            rg, bg, ru, bu, rh, bh = swiglu_ref(d(x)[src[a:b]], d(gw[l]), d(uw[l]))
            check(h.cpu()[dst[a:b]], rh, bh, f"h of expert {l}")
            check(kg[a:b], rg, bg, f"g of expert {l}")
            check(ku[a:b], ru, bu, f"u of expert {l}")
    assert bool((whole[:, I:] == 7.0).all())
    assert bool((h.cpu()[r.index(yo)][~r.owned()] == 7.0).all())
    # without keeping g and u: the same h
    h2 = blank(T * k, I, dt, pad)[0]
    dense.grouped_swiglu(xd, gd, ud, gr, x_rows=xo, out_rows=yo, out=h2)
    assert torch.equal(h2, h)

    # gradients, from the g and u that were kept
    dho = yo if pad else 1
    dh = randn(g, (r.rows(dho), I), 0.3, dt)
    dx = blank(T * k, H, torch.float32, pad)[0]
    dgate, dup = (torch.full(gw.shape, NAN, dtype=torch.float32, device="cuda") for _ in range(2))
    dense.grouped_swiglu_grad(strided(dh, pad), xd, gd, ud, kg, ku, gr, dh_rows=dho, x_rows=xo, dx_rows=yo, dx=dx,
                              dgate=dgate, dup=dup)
    up = r.index(dho)
    e = half_step(dt)
    for l, a, b in r.spans():
        gg, uu, dd, xs = d(kg[a:b]), d(ku[a:b]), d(dh)[up[a:b]], d(x)[src[a:b]]
        dg, du = dd * uu * R.slope("silu", gg), dd * gg * R.sig(gg)
        # dg and du are rounded to the type after a few fp32 steps (relative to their factors, as the
        # slope passes zero)
        eg = e * dg.abs() + FEW * (dd * uu).abs() * (1 + gg.abs()) + R.tiny(dt)
        eu = e * du.abs() + FEW * du.abs() + R.tiny(dt)
        for got, v, ev, name in ((dgate, dg, eg, "dgate"), (dup, du, eu, "dup")):
            ref, bound = mm(v.T, xs.T) if b > a else (torch.zeros(I, H).double(), torch.zeros(I, H).double())
            if b > a:
                bound = bound * (1 + e) + ev.T @ xs.abs()
            check(got[l], ref, bound, f"{name} of expert {l}")
        if b > a:
            r1, b1 = mm(torch.cat([dg, du], 1), torch.cat([d(gw[l]), d(uw[l])], 0).T)
            b1 = b1 * (1 + e) + eg @ d(gw[l]).abs() + eu @ d(uw[l]).abs()
            check(dx.cpu()[dst[a:b]], r1, b1, f"dx of expert {l}")


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,k,E,I,H,empty,lead", [(2, 1, 5, 8, 8, (1, 3), 8), (3, 4, 12, 264, 136, tuple(range(1, 8)), 24), (40, 2, 4, 136, 520, (), 40),
                                                  (600, 1, 1, 1032, 1096, (), 8), (1300, 2, 3, 520, 4104, (1,), 64)])
def test_both_swiglu_weight_gradients(dense, T, k, E, I, H, empty, lead, dt):
    """In 16 bits, at tile edges of either, zeros for experts without rows, and nothing outside."""
    gen = torch.Generator().manual_seed(T + I)
    r = R.Routing(T, k, E, 13 + T, empty)
    x, dh, g, u = randn(gen, (T * k, H), 1.0, dt), randn(gen, (T * k, I), 0.3, dt), randn(gen, (T * k, I), 1.2, dt), randn(gen, (T * k, I), 1.2, dt)
    w = torch.zeros((E, I, H), dtype=dt, device="cuda")
    wholes = [torch.full((lead + E * I * H + 64,), NAN, dtype=dt, device="cuda") for _ in range(2)]
    for b in wholes:
        b[:lead] = 7.0
        b[-64:] = 7.0
    dgate, dup = (b[lead:-64].view(E, I, H) for b in wholes)
    dense.grouped_swiglu_grad(dh.cuda(), x.cuda(), w, w, g.cuda(), u.cuda(), groups(dense, r), x_rows=0, need_dx=False,
                              dgate=dgate, dup=dup)
    e = half_step(dt)
    for l, a, b in r.spans():
        if b == a:
            assert not bool(dgate[l].any()) and not bool(dup[l].any()), f"expert {l}"
            continue
        gg, uu, dd, xs = d(g[a:b]), d(u[a:b]), d(dh[a:b]), d(x[a:b])
        dg, du = dd * uu * R.slope("silu", gg), dd * gg * R.sig(gg)
        eg = e * dg.abs() + FEW * (dd * uu).abs() * (1 + gg.abs()) + R.tiny(dt)
        eu = e * du.abs() + FEW * du.abs() + R.tiny(dt)
        for got, v, ev, name in ((dgate, dg, eg, "dgate"), (dup, du, eu, "dup")):
            ref, bound = mm(v.T, xs.T)
            check(got[l], ref, bound * (1 + e) + ev.T @ xs.abs(), f"{name} of expert {l}")
    for b in wholes:
        assert bool((b[:lead] == 7.0).all()) and bool((b[-64:] == 7.0).all())


LINEAR = [(1, 8, 8, 0), (1, 264, 520, 8), (2, 64, 4096, 0), (5, 40, 72, 8), (16, 1000, 256, 0), (17, 72, 136, 8),
          (33, 512, 64, 0), (64, 136, 200, 0), (127, 264, 8, 8), (300, 328, 328, 0), (515, 136, 72, 16), (1030, 520, 264, 0)]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("T,N,K,pad", LINEAR)
def test_linear_and_its_gradients(dense, T, N, K, pad, act, dt):
    g = torch.Generator().manual_seed(T * 43 + N + K)
    x, w = randn(g, (T, K), 1.0, dt), randn(g, (N, K), K ** -0.5, dt)
    bias, res = randn(g, (N,), 0.5, torch.float32), randn(g, (T, N), 1.0, dt)
    z, bz = mm(d(x), d(w))
    xd, wd = strided(x, pad), w.cuda()
    # the bare product, fp32 out
    check(dense.linear(xd, wd, out_dtype=torch.float32), z, bz, "x w^T")
    zb = z + d(bias)
    bz = bz + U32 * (z.abs() + zb.abs())
    y = R.act(act, zb)
    by = SLOPE * bz + FEW * (y.abs() + zb.abs())
    out, whole = blank(T, N, dt, pad)
    pre = blank(T, N, dt, pad)[0]
    dense.linear(xd, wd, bias=bias.cuda(), act=act, residual=strided(res, pad), out=out, pre=pre)
    check(pre, zb, bz, "pre")
    check(out, y + d(res), by + U32 * (y.abs() + d(res).abs()), "out")
    assert bool((whole[:, N:] == 7.0).all())
    # in place over the residual, without bias and pre
    acc = strided(res, pad)
    dense.linear(xd, wd, act=act, residual=acc, out=acc)
    y0 = R.act(act, z)
    check(acc, y0 + d(res), SLOPE * bz + FEW * (y0.abs() + z.abs() + d(res).abs()), "in place")

    dy = randn(g, (T, N), 0.2, dt)
    dyd = strided(dy, pad)
    s = R.slope(act, d(pre))
    dz = d(dy) * s
    e = half_step(dt) if act != "none" else 0.0
    ez = e * dz.abs() + FEW * d(dy).abs() * (1 + d(pre).abs()) + (R.tiny(dt) if act != "none" else 0.0)
    dx, dw, db = dense.linear_grad(dyd, xd, wd, pre=pre, act=act, dw_dtype=torch.float32)
    ref, bound = mm(dz, d(w).T)
    check(dx, ref, bound * (1 + e) + ez @ d(w).abs(), "dx")
    ref, bound = mm(dz.T, d(x).T)
    check(dw, ref, bound * (1 + e) + ez.T @ d(x).abs(), "dw")
    ref = dz.sum(0)
    check(db, ref, T * U32 * dz.abs().sum(0) + (FEW * d(dy).abs() * (1 + d(pre).abs())).sum(0), "dbias")
    # accumulated on top: the fp32 sum of both
    dw2, db2 = dw.clone(), db.clone()
    r = dense.linear_grad(dyd, xd, wd, pre=pre, act=act, need_dx=False, dw=dw2, dbias=db2, accumulate=True)
    assert r[0] is None and torch.equal(dw2, dw + dw) and torch.equal(db2, db + db)
    # in 16 bits: the fp32 result rounded once
    _, dw16, none = dense.linear_grad(dyd, xd, wd, pre=pre, act=act, need_dx=False, need_dbias=False)
    assert none is None and torch.equal(dw16, dw.to(dt))


LOSS = [(1, 1, 8, 0), (1, 7, 72, 0), (1, 1000, 256, 8), (3, 129, 64, 0), (16, 777, 136, 0), (20, 257, 520, 8),
        (65, 1025, 128, 0), (130, 4099, 72, 8), (300, 513, 264, 0), (515, 130, 64, 0)]


def loss_ref(x, w, t):
    z, bz = mm(d(x), d(w))
    lse = torch.logsumexp(z, 1)
    top = bz.max(1).values           # lse moves by no more than the logits do
    counted = (t >= 0) & (t < w.shape[0])
    hit = z.gather(1, t.clamp(0, w.shape[0] - 1).long()[:, None])[:, 0]
    nll = torch.where(counted, lse - hit, torch.zeros_like(lse))
    spread = (z.max(1).values - z.min(1).values) + 1
    # exponentials of differences up to the spread: a few steps of the difference each; the sum of V
    # positive terms in any order
    b = top + U32 * (lse.abs() + 4 * spread + w.shape[0])
    return z, bz, lse, nll, b, counted


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("std", [0.3, 4.0])
@pytest.mark.parametrize("T,V,H,pad", LOSS)
def test_cross_entropy_and_its_gradients(dense, T, V, H, pad, std, dt):
    g = torch.Generator().manual_seed(T * 47 + V)
    x, w = randn(g, (T, H), 1.0, dt), randn(g, (V, H), std * H ** -0.5, dt)
    t = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    if T > 2:
        t[::3] = torch.tensor([-100, V, -1, 2 ** 31 - 1], dtype=torch.int32)[torch.arange(len(t[::3])) % 4]
    z, bz, lse, nll, b, counted = loss_ref(x, w, t)
    xd, wd, td = strided(x, pad), w.cuda(), t.cuda()
    gn, gl = dense.cross_entropy(xd, wd, td)
    check(gl, lse, b, "lse")
    check(gn, nll, torch.where(counted, 2 * b, torch.zeros_like(b)), "nll")

    dnll = torch.rand(T, generator=g) * 2 - 1
    dnll[~counted] = NAN                  # ignored tokens: nothing of theirs is read
    for i in (~counted).nonzero()[:, 0].tolist():
        x[i] = NAN
    xd = strided(x, pad)
    dx, dw = dense.cross_entropy_grad(xd, wd, td, gl, dnll.cuda(), dw_dtype=torch.float32)
    p = torch.exp(z - lse[:, None])
    one = torch.zeros_like(p)
    one[counted, t[counted].long()] = 1.0
    up = torch.where(counted, d(dnll), torch.zeros_like(lse))
    ds = (p - one) * up[:, None]
    # p is off by its exponent's error; the difference is rounded to the type
    ep = (bz + b[:, None] + U32 * (4 * (z - lse[:, None]).abs() + 4)) * p + U32
    eds = ep * up.abs()[:, None] + half_step(dt) * (ds.abs() + ep * up.abs()[:, None]) + 2.0 ** -38 * up.abs().max()
    eds[~counted] = 0.0
    x0 = torch.where(counted[:, None], d(x), torch.zeros(()).double())
    ref, bound = mm(ds, d(w).T)
    check(dx, ref, bound * 1.01 + eds @ d(w).abs(), "dx")
    assert not dx[~counted.cuda()].any()
    ref, bound = mm(ds.T, x0.T)
    check(dw, ref, bound * 1.01 + eds.T @ x0.abs(), "dw")
    dw2 = dw.clone()
    none, _ = dense.cross_entropy_grad(xd, wd, td, gl, dnll.cuda(), need_dx=False, dw=dw2, accumulate=True)
    assert none is None and torch.equal(dw2, dw + dw)


def test_cross_entropy_grad_in_pieces_of_the_vocabulary(dense):
    """So many tokens that the vocabulary is taken in three pieces, the last of 4 columns."""
    T, V, H, dt = 65537, 4100, 16, BF
    g = torch.Generator().manual_seed(3)
    x, w = randn(g, (T, H), 1.0, dt), randn(g, (V, H), 0.5, dt)
    t = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    t[5::7] = -1
    counted = (t >= 0).cuda()
    xd, wd, td = x.cuda(), w.cuda(), t.cuda()
    _, lse = dense.cross_entropy(xd, wd, td)
    dnll = (torch.rand(T, generator=g) / T).cuda()
    dx, dw = dense.cross_entropy_grad(xd, wd, td, lse, dnll)
    x64, w64 = xd.double(), wd.double()
    z = x64 @ w64.T
    ds = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    ds[torch.arange(T, device="cuda"), td.clamp(min=0).long()] -= 1.0
    ds *= torch.where(counted, dnll.double(), 0.0)[:, None]
    e = half_step(dt)
    # the exponent's error of H products, the type's rounding of ds, V or T fp32 additions
    rel = e + 2 * H * U32 * float((x64.abs() @ w64.abs().T).max()) + 64 * U32
    check(dx, (ds @ w64).cpu(), ((rel + V * U32) * (ds.abs() @ w64.abs()) + U32 * dnll[:, None].double() * w64.abs().sum(0)).cpu(), "dx")
    check(dw, (ds.T @ x64).cpu(), ((rel + T * U32) * (ds.T.abs() @ x64.abs()) + U32 * (dnll[:, None].double() * x64.abs()).sum(0)).cpu(), "dw")


def test_every_target_ignored_and_empty_batches(dense):
    x, w = torch.full((9, 64), NAN, dtype=BF, device="cuda"), torch.ones((50, 64), dtype=BF, device="cuda")
    t = torch.full((9,), -100, dtype=torch.int32, device="cuda")
    lse = torch.full((9,), NAN, device="cuda")
    dx, dw = dense.cross_entropy_grad(x, w, t, lse, lse)
    assert not dx.any() and not dw.any()
    e = x[:0]
    dx, dw = dense.cross_entropy_grad(e, w, t[:0], lse[:0], lse[:0])
    assert dx.shape == (0, 64) and not dw.any()
    nll, l0 = dense.cross_entropy(e, w, t[:0])
    assert nll.numel() == 0 and l0.numel() == 0
    dx, dw, db = dense.linear_grad(torch.empty((0, 50 - 2), dtype=BF, device="cuda"), e, w[:48].contiguous())
    assert dx.numel() == 0 and not dw.any() and not db.any()
    assert dense.linear(e, w[:48].contiguous()).shape == (0, 48)
    gr = dense.Groups(torch.zeros(4, dtype=torch.int32, device="cuda"), None, 0, 2)
    ew = torch.ones((3, 16, 64), dtype=BF, device="cuda")
    assert dense.grouped_matmul(e, ew, gr).shape == (0, 16)
    dw = torch.full((3, 16, 64), 5.0, dtype=BF, device="cuda")
    dense.grouped_matmul_grad(torch.empty((0, 16), dtype=BF, device="cuda"), e, ew, gr, dw=dw, accumulate=True)
    assert bool((dw == 5.0).all())
    dense.grouped_matmul_grad(torch.empty((0, 16), dtype=BF, device="cuda"), e, ew, gr, dw=dw)
    assert not dw.any()


def test_infinite_logits(dense):
    """A logit of +inf makes lse +inf, one of -inf leaves it alone; other rows are not touched."""
    x, w = torch.zeros((4, 8), dtype=BF), torch.zeros((300, 8), dtype=BF)
    w[:, 0] = 1.0
    w[200, 1] = 1.0
    x[1, 1] = float("inf")       # z[1, 200] = inf, 0 * inf elsewhere
    x[2, 0] = 2.0
    w64 = d(w)
    z = torch.stack([(d(x)[i][None] * w64).sum(1) for i in range(4)])
    nll, lse = dense.cross_entropy(x.cuda(), w.cuda(), torch.tensor([0, 200, 3, -1], dtype=torch.int32, device="cuda"))
    ref = torch.logsumexp(z, 1)
    assert torch.isnan(lse[1]) and torch.isnan(ref[1])
    keep = torch.tensor([0, 2, 3])
    check(lse.cpu()[keep], ref[keep], 400 * U32 * (1 + ref[keep].abs()), "lse")
    # +inf and -inf without a product of zero and infinity
    x = torch.tensor([[1.0] + [0.0] * 7] * 2, dtype=FP)
    w = torch.zeros((300, 8), dtype=FP)
    w[7, 0] = -float("inf")
    nll, lse = dense.cross_entropy(x.cuda()[:, :8], w.cuda(), torch.tensor([3, 7], dtype=torch.int32, device="cuda"))
    assert abs(float(lse[0]) - 5.700443573390687) < 400 * U32 * 7 and float(nll[1]) == float("inf")
    w[7, 0] = float("inf")
    _, lse = dense.cross_entropy(x.cuda(), w.cuda(), torch.tensor([3, 7], dtype=torch.int32, device="cuda"))
    assert float(lse[0]) == float("inf")
    # beside logits of 200 in other column tiles, for one row and for many; and rows of NaN
    w[8:, 0] = 200.0
    for T in (2, 40, 300):
        x = torch.zeros((T, 8), dtype=FP)
        x[:, 0] = 1.0
        x[1] = NAN
        nll, lse = dense.cross_entropy(x.cuda(), w.cuda(), torch.full((T,), 3, dtype=torch.int32, device="cuda"))
        assert bool((lse[[0, -1] if T > 2 else [0]] == float("inf")).all())
        assert torch.isnan(lse[1]) and torch.isnan(nll[1])


def test_nan_of_other_experts_and_rows_never_enters(dense):
    """Weights of experts without rows, rows of other tokens and values past K are never multiplied."""
    r = R.Routing(40, 2, 6, 9, empty=(1, 4))
    g = torch.Generator().manual_seed(1)
    x, w = randn(g, (40, 72), 1.0, BF), randn(g, (6, 40, 72), 0.1, BF)
    w[1], w[4] = NAN, NAN
    gr = groups(dense, r)
    wd = w.cuda()
    y = dense.grouped_matmul(strided(x, 8), wd, gr, x_rows=2)
    assert bool(torch.isfinite(y).all())
    dx, dw = dense.grouped_matmul_grad(y, strided(x, 8), wd, gr, x_rows=2)
    assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())
    # one token's NaN stays in its own slots
    x[11] = NAN
    y = dense.grouped_matmul(strided(x, 8), wd, gr, x_rows=2)
    hit = (r.slots // 2 == 11)
    assert bool(torch.isnan(y[hit.cuda()]).all()) and bool(torch.isfinite(y[(~hit).cuda()]).all())


@pytest.mark.parametrize("op", ["linear", "swiglu", "loss"])
def test_gradients_against_differences(dense, op):
    """The change of L = sum c * f over a step of a parameter, both ends computed by the kernels,
    against the gradient's prediction.  Steps are representable, the central difference's error is
    third order (step^3) and the values' own rounding is counted."""
    g = torch.Generator().manual_seed(8)
    dt = FP
    step = 2.0 ** -6
    if op == "linear":
        x, w = randn(g, (9, 64), 1.0, dt), (torch.randn((40, 64), generator=g) * 16).round().to(dt) / 128
        c = randn(g, (9, 40), 1.0, dt)
        dirn = (torch.randint(0, 2, w.shape, generator=g) * 2 - 1).to(dt)
        f = lambda s: dense.linear(x.cuda(), (w + s * dirn).cuda(), act="silu", out_dtype=torch.float32)  # noqa: E731
        pre = torch.empty((9, 40), dtype=dt, device="cuda")
        dense.linear(x.cuda(), w.cuda(), act="silu", pre=pre)
        _, dw, _ = dense.linear_grad(c.cuda(), x.cuda(), w.cuda(), pre=pre, act="silu", dw_dtype=torch.float32)
        pred = float((d(dw) * d(dirn)).sum()) * 2 * step
        got = float(((d(f(step)) - d(f(-step))) * d(c)).sum())
        dirz = d(x) @ d(dirn).T
        # third derivative of silu below 0.7; pre and dz are rounded to 11 bits
        err = float((d(c).abs() * (dirz.abs() * step) ** 3).sum()) * 0.7 / 3 \
            + 2 * step * float((d(c).abs() * dirz.abs() * (CURVE * d(pre).abs() + 1.13)).sum()) * half_step(dt) + 1e-4
    elif op == "swiglu":
        r = R.Routing(9, 2, 3, 4)
        gr = groups(dense, r)
        x = randn(g, (9, 64), 1.0, dt)
        gw, uw = ((torch.randn((3, 40, 64), generator=g) * 16).round().to(dt) / 128 for _ in range(2))
        c = randn(g, (18, 40), 1.0, dt)
        dirn = (torch.randint(0, 2, gw.shape, generator=g) * 2 - 1).to(dt)
        kg, ku = (torch.empty((18, 40), dtype=dt, device="cuda") for _ in range(2))
        f = lambda s: dense.grouped_swiglu(x.cuda(), (gw + s * dirn).cuda(), uw.cuda(), gr)  # noqa: E731
        h0 = dense.grouped_swiglu(x.cuda(), gw.cuda(), uw.cuda(), gr, keep_g=kg, keep_u=ku)
        _, dgate, _ = dense.grouped_swiglu_grad(c.cuda(), x.cuda(), gw.cuda(), uw.cuda(), kg, ku, gr, dw_dtype=torch.float32)
        pred = float((d(dgate) * d(dirn)).sum()) * 2 * step
        hi, lo = f(step), f(-step)
        got = float(((d(hi) - d(lo)) * d(c)).sum())
        src = r.index(2)
        dirz = torch.cat([d(x)[src[a:b]] @ d(dirn[l]).T for l, a, b in r.spans()])
        cu = (d(c) * d(ku)).abs()
        err = float((cu * (dirz.abs() * step) ** 3).sum()) * 0.7 / 3 \
            + 2 * step * float((cu * dirz.abs() * (CURVE * d(kg).abs() + 3)).sum()) * half_step(dt) \
            + float((d(c).abs() * (d(hi).abs() + d(lo).abs())).sum()) * half_step(dt) + 1e-4
        assert h0.shape == hi.shape
    else:
        x, w = randn(g, (9, 64), 1.0, dt), (torch.randn((300, 64), generator=g) * 16).round().to(dt) / 128
        t = torch.randint(0, 300, (9,), generator=g, dtype=torch.int32).cuda()
        c = torch.rand(9, generator=g)
        dirn = (torch.randint(0, 2, w.shape, generator=g) * 2 - 1).to(dt)
        f = lambda s: dense.cross_entropy(x.cuda(), (w + s * dirn).cuda(), t)[0]  # noqa: E731
        _, lse = dense.cross_entropy(x.cuda(), w.cuda(), t)
        _, dw = dense.cross_entropy_grad(x.cuda(), w.cuda(), t, lse, c.cuda(), dw_dtype=torch.float32)
        pred = float((d(dw) * d(dirn)).sum()) * 2 * step
        got = float(((d(f(step)) - d(f(-step))) * d(c)).sum())
        dirz = (d(x) @ d(dirn).T).abs().max(1).values
        # the third cumulant of a value within +-dirz is below 2 dirz^3; ds is rounded to 11 bits
        err = float((d(c) * 2 * (2 * dirz * step) ** 3).sum()) / 3 \
            + 2 * step * float((d(c) * 2 * dirz).sum()) * half_step(dt) + 1e-4
    assert abs(got - pred) <= err, (got, pred, err)
    assert abs(pred) > 3 * err or op != "linear", "the step says nothing"


def _calls(dense):
    """One call of every operator on fixed inputs, as a function of nothing."""
    g = torch.Generator().manual_seed(12)
    r = R.Routing(150, 3, 9, 2, empty=(3,))
    gr = groups(dense, r)
    x = randn(g, (150, 136), 1.0, BF).cuda()
    gw, uw = randn(g, (9, 72, 136), 0.1, BF).cuda(), randn(g, (9, 72, 136), 0.1, BF).cuda()
    dwn, vw = randn(g, (9, 136, 72), 0.1, BF).cuda(), randn(g, (1003, 136), 0.1, BF).cuda()
    pw, pb = randn(g, (136, 136), 0.1, BF).cuda(), randn(g, (136,), 0.1, torch.float32).cuda()
    t = torch.randint(0, 1003, (150,), generator=g, dtype=torch.int32)
    t[4::9] = -1
    t = t.cuda()
    up = torch.rand(150, generator=g).cuda()

    def run():
        kg, ku = torch.empty((450, 72), dtype=BF, device="cuda"), torch.empty((450, 72), dtype=BF, device="cuda")
        h = dense.grouped_swiglu(x, gw, uw, gr, keep_g=kg, keep_u=ku)
        y = dense.grouped_matmul(h, dwn, gr, out_rows=dense.ROWS_SLOT)
        dh, ddown = dense.grouped_matmul_grad(y, h, dwn, gr, dy_rows=dense.ROWS_SLOT)
        dx, dgate, dup = dense.grouped_swiglu_grad(dh, x, gw, uw, kg, ku, gr)
        pre = torch.empty((150, 136), dtype=BF, device="cuda")
        o = dense.linear(x, pw, bias=pb, act="gelu", residual=x, pre=pre)
        l1 = dense.linear(x[:1], pw, bias=pb, act="silu", residual=x[:1])
        gl = dense.linear_grad(o, x, pw, pre=pre, act="gelu")
        nll, lse = dense.cross_entropy(o, vw, t)
        gx, gv = dense.cross_entropy_grad(o, vw, t, lse, up)
        return [h, y, dh, ddown, dx, dgate, dup, o, l1, *gl, nll, lse, gx, gv]

    return run


def test_calls_repeat_bit_for_bit_and_run_on_another_stream(dense):
    run = _calls(dense)
    ref = run()
    torch.cuda.synchronize()
    for a, b in zip(ref, run()):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_stream_argument(dense):
    """Outputs and workspace of a call on a stream passed in belong to that stream."""
    g = torch.Generator().manual_seed(2)
    x, w = randn(g, (130, 64), 1.0, BF).cuda(), randn(g, (72, 64), 0.1, BF).cuda()
    dy = randn(g, (130, 72), 1.0, BF).cuda()
    ref = dense.linear(x, w), *dense.linear_grad(dy, x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for st in (s, s.cuda_stream):
        got = dense.linear(x, w, stream=st), *dense.linear_grad(dy, x, w, stream=st)
        s.synchronize()
        for a, b in zip(ref, got):
            assert torch.equal(a, b)


def test_captured_calls_replay_to_the_eager_results(dense):
    run = _calls(dense)
    ref = [t.clone() for t in run()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, out):
            assert torch.equal(a, b), f"replay {i}"
        eager = run()
        torch.cuda.synchronize()
        for a, b in zip(ref, eager):
            assert torch.equal(a, b), f"eager after replay {i}"
