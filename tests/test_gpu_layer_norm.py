"""Layer norm over token slabs vs a plain 64-bit implementation (GPU).

Bounds, per element, with u = 2^-24 (half a step of fp32) and half a step of the output's type
(bf16 2^-8, fp32 2^-24) for its one rounding.  A sum of n fp32 terms is off by at most n u times
the sum of their magnitudes; the kernels' chains are shorter than 64 + n / 256 terms plus the tree.
"""
import pytest
import torch

import tensor_transformer_layer_way_gb300 as ttl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
F8 = torch.float64


def _inputs(t, rows, h, dt, wt, seed, residual=False, pad=0):
    g = torch.Generator().manual_seed(seed)

    def slabs(std=1.0, mean=0.0):
        out = []
        for _ in range(t):
            wide = (torch.randn(rows, h + pad, generator=g) * std + mean).to(dt).cuda()
            out.append(wide[:, pad:] if pad else wide)
        return out

    d = {"X": slabs(2.0, 0.5), "R": slabs() if residual else None, "dY": slabs(0.5), "dS": slabs(0.5)}
    d["gamma"] = (torch.randn(h, generator=g) * 0.2 + 1).to(wt).cuda()
    d["beta"] = (torch.randn(h, generator=g) * 0.2).to(wt).cuda()
    return d


def _chain(n):
    return (64 + n / 256 + 16) * U


def _check_fwd(d, out, eps, beta=True):
    for i, x in enumerate(d["X"]):
        dt, h = x.dtype, x.shape[1]
        s = x.to(F8)
        if d["R"] is not None:
            s = (x.float() + d["R"][i].float()).to(dt)      # one fp32 addition, one rounding
            assert torch.equal(out["S"][i], s)
            s = s.to(F8)
        mean = s.mean(1, keepdim=True)
        rstd = ((s - mean).square().mean(1, keepdim=True) + eps) ** -0.5
        n = (s - mean) * rstd
        gamma = d["gamma"].to(F8)
        y = n * gamma + (d["beta"].to(F8) if beta else 0.0)
        c, mag = _chain(h), s.abs().mean(1, keepdim=True)
        assert ((out["mean"][i].to(F8) - mean[:, 0]).abs() <= c * mag[:, 0] + 1e-30).all()
        # the deviations are off by c mag + u (|s| + mag) each; relative to their rms that moves rstd
        rel = 2 * c + 4 * U + (c + 2 * U) * mag * rstd * 2
        assert ((out["rstd"][i].to(F8) - rstd[:, 0]).abs() <= (rel * rstd)[:, 0]).all()
        off = gamma.abs() * (rstd * ((c + 2 * U) * mag + 2 * U * s.abs()) + n.abs() * (rel + 4 * U)) + 4 * U * y.abs()
        assert ((out["Y"][i].to(F8) - y).abs() <= off + HALF[dt] * (y.abs() + off)).all(), f"slab {i}"


def _check_bwd(d, X, out, fwd, base=None, dS=True):
    gamma = d["gamma"].to(F8)
    total = sum(x.shape[0] for x in X)
    dg, db, dg_mag, db_mag = 0, 0, 0, 0
    for i, x in enumerate(X):
        dt, h = x.dtype, x.shape[1]
        s, dy = x.to(F8), d["dY"][i].to(F8)
        mean, rstd = fwd["mean"][i].to(F8)[:, None], fwd["rstd"][i].to(F8)[:, None]
        n = (s - mean) * rstd
        g = dy * gamma
        c1, c2 = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
        dx = rstd * (g - c1 - n * c2)
        if dS:
            dx = dx + d["dS"][i].to(F8)
        c = _chain(h)
        n_off = 4 * U * (s.abs() + mean.abs()) * rstd + 4 * U * n.abs()
        off = rstd * (4 * U * g.abs() + c * g.abs().mean(1, keepdim=True) + 4 * U * c1.abs() + n_off * c2.abs()
                      + n.abs() * (c * (g * n).abs().mean(1, keepdim=True) + (g.abs() * n_off).mean(1, keepdim=True)))
        off = off + 4 * U * (dx.abs() + (d["dS"][i].to(F8).abs() if dS else 0.0))
        assert ((out["dX"][i].to(F8) - dx).abs() <= off + HALF[dt] * (dx.abs() + off)).all(), f"dX[{i}]"
        dg, db = dg + (dy * n).sum(0), db + dy.sum(0)
        dg_mag, db_mag = dg_mag + (dy.abs() * (n.abs() + n_off / U / 64)).sum(0), db_mag + dy.abs().sum(0)
    k = (64 + total / 304 + 304 / 8 + 16) * U
    if base is not None:
        dg, db = dg + base[0].to(F8), db + base[1].to(F8)
        dg_mag, db_mag = dg_mag + base[0].to(F8).abs(), db_mag + base[1].to(F8).abs()
    assert ((out["dgamma"].to(F8) - dg).abs() <= k * dg_mag).all()
    if out["dbeta"] is not None:
        assert ((out["dbeta"].to(F8) - db).abs() <= k * db_mag).all()


SHAPES = [(1, 1, 1), (1, 1, 8), (2, 3, 24), (1, 5, 7), (2, 64, 256), (1, 33, 1001), (4, 9, 1024), (8, 16, 4096),
          (1, 7, 4104), (1, 5, 8192), (1, 3, 12288), (1, 2, 16384), (1, 2, 16392), (1, 2, 9001), (1, 2, 40000),
          (3, 700, 64)]


@pytest.mark.parametrize("t,rows,h", SHAPES)
@pytest.mark.parametrize("dt,wt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.float32)])
def test_forward_and_backward(t, rows, h, dt, wt):
    eps = 1e-5
    d = _inputs(t, rows, h, dt, wt, seed=rows + h)
    fwd = ttl.layer_norm_fwd(d["X"], d["gamma"], d["beta"], eps=eps)
    assert fwd["S"] is None
    _check_fwd(d, fwd, eps)
    bwd = ttl.layer_norm_bwd(d["X"], d["dY"], d["gamma"], fwd, dS=d["dS"])
    _check_bwd(d, d["X"], bwd, fwd)
    assert ttl.device_status() == 0


@pytest.mark.parametrize("t,rows,h,dt", [(2, 33, 256, torch.bfloat16), (8, 40, 4096, torch.bfloat16),
                                         (1, 17, 1001, torch.float32), (1, 9, 20000, torch.bfloat16)])
def test_residual_no_beta_and_accumulation(t, rows, h, dt):
    d = _inputs(t, rows, h, dt, dt, seed=h, residual=True)
    fwd = ttl.layer_norm_fwd(d["X"], d["gamma"], residual=d["R"], eps=1e-6)
    _check_fwd(d, fwd, 1e-6, beta=False)
    out = ttl.layer_norm_bwd_buffers(t, rows, h, dt)
    out["dgamma"].normal_()
    out["dbeta"].normal_()
    base = out["dgamma"].clone(), out["dbeta"].clone()
    ttl.layer_norm_bwd(fwd["S"], d["dY"], d["gamma"], fwd, accumulate=True, out=out)
    _check_bwd(d, fwd["S"], out, fwd, base=base, dS=False)
    out["dbeta"] = None
    ttl.layer_norm_bwd(fwd["S"], d["dY"], d["gamma"], fwd, out=out)
    _check_bwd(d, fwd["S"], out, fwd, dS=False)


@pytest.mark.parametrize("pad", [1, 8, 64])
@pytest.mark.parametrize("h", [256, 1000, 4096])
def test_row_strides(pad, h):
    """Slabs that are column ranges of wider matrices: the same bits as contiguous copies."""
    d = _inputs(2, 21, h, torch.bfloat16, torch.bfloat16, seed=pad, residual=True, pad=pad)
    flat = {k: [x.contiguous() for x in v] if isinstance(v, list) else v for k, v in d.items()}
    a = ttl.layer_norm_fwd(d["X"], d["gamma"], d["beta"], residual=d["R"])
    _check_fwd(d, a, 1e-5)
    b = ttl.layer_norm_bwd(d["X"], d["dY"], d["gamma"], a, dS=d["dS"])
    c = ttl.layer_norm_fwd(flat["X"], d["gamma"], d["beta"], residual=flat["R"])
    for x, y in zip(a["S"], c["S"]):
        assert torch.equal(x, y)
    _check_bwd(d, d["X"], b, a)


def test_same_inputs_same_bits():
    d = _inputs(8, 300, 1024, torch.bfloat16, torch.bfloat16, seed=5)
    fwd = ttl.layer_norm_fwd(d["X"], d["gamma"], d["beta"])
    first = ttl.layer_norm_bwd(d["X"], d["dY"], d["gamma"], fwd)
    for _ in range(5):
        again = ttl.layer_norm_bwd(d["X"], d["dY"], d["gamma"], fwd)
        assert torch.equal(first["dgamma"], again["dgamma"]) and torch.equal(first["dbeta"], again["dbeta"])


def test_constant_rows_and_large_means():
    """A row of one value has variance 0 (rstd = eps^-1/2); a mean 4096 times the spread loses no variance."""
    for h in (256, 1000, 4096):
        x = torch.full((3, h), 7.0, device="cuda")
        w = torch.ones(h, device="cuda")
        out = ttl.layer_norm_fwd([x], w, eps=1e-4)
        assert torch.count_nonzero(out["Y"][0]) == 0 and torch.allclose(out["rstd"][0], torch.full_like(out["rstd"][0], 100.0))
        d = {"X": [(torch.randn(5, h, generator=torch.Generator().manual_seed(h)) + 4096.0).cuda()], "R": None,
             "gamma": w, "beta": w}
        out = ttl.layer_norm_fwd(d["X"], w, w)
        _check_fwd(d, out, 1e-5)


def test_not_finite_stays_in_its_row():
    d = _inputs(1, 8, 512, torch.bfloat16, torch.bfloat16, seed=3)
    d["X"][0][3, 100] = float("inf")
    d["X"][0][5, 7] = float("nan")
    out = ttl.layer_norm_fwd(d["X"], d["gamma"], d["beta"])
    bad = torch.zeros(8, dtype=torch.bool, device="cuda")
    bad[[3, 5]] = True
    assert torch.isnan(out["Y"][0][bad]).all() and torch.isfinite(out["Y"][0][~bad]).all()


def test_gradient_against_differences():
    """<dx, v> + <dgamma, w> + <dbeta, z> against central differences of the 64-bit forward."""
    t, rows, h, eps, step = 2, 11, 333, 1e-5, 1e-5
    d = _inputs(t, rows, h, torch.float32, torch.float32, seed=8)
    fwd = ttl.layer_norm_fwd(d["X"], d["gamma"], d["beta"], eps=eps)
    out = ttl.layer_norm_bwd(d["X"], d["dY"], d["gamma"], fwd)
    x, dy = torch.cat(d["X"]).to(F8), torch.cat(d["dY"]).to(F8)
    g, b = d["gamma"].to(F8), d["beta"].to(F8)
    gen = torch.Generator("cuda").manual_seed(1)
    v, w, z = (torch.randn(s.shape, generator=gen, device="cuda", dtype=F8) for s in (x, g, b))

    def loss(e):
        s = x + e * v
        c = s - s.mean(1, keepdim=True)
        return (dy * (c * (c.square().mean(1, keepdim=True) + eps) ** -0.5 * (g + e * w) + b + e * z)).sum()

    want = (loss(step) - loss(-step)) / (2 * step)
    dx = torch.cat(out["dX"]).to(F8)
    terms = (dx * v).sum(), (out["dgamma"].to(F8) * w).sum(), (out["dbeta"].to(F8) * z).sum()
    size = dx.norm() * v.norm() + out["dgamma"].norm() * w.norm() + out["dbeta"].norm() * z.norm()
    # gradients are good to about 100 u of their norm; the differences to step^2 and 1e-16 / step
    assert (sum(terms) - want).abs() <= 200 * U * size + 1e-6 * want.abs()


def test_side_stream_and_graph_replay():
    d = _inputs(2, 64, 1024, torch.bfloat16, torch.bfloat16, seed=11, residual=True)
    fwd = ttl.layer_norm_fwd(d["X"], d["gamma"], d["beta"], residual=d["R"])
    bwd = ttl.layer_norm_bwd(fwd["S"], d["dY"], d["gamma"], fwd, dS=d["dS"])
    f2 = ttl.layer_norm_fwd_buffers(2, 64, 1024, residual=True)
    b2 = ttl.layer_norm_bwd_buffers(2, 64, 1024)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ttl.layer_norm_fwd(d["X"], d["gamma"], d["beta"], residual=d["R"], out=f2)
        ttl.layer_norm_bwd(f2["S"], d["dY"], d["gamma"], f2, dS=d["dS"], out=b2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(fwd["Y"]), torch.cat(f2["Y"])) and torch.equal(torch.cat(bwd["dX"]), torch.cat(b2["dX"]))
    assert torch.equal(bwd["dgamma"], b2["dgamma"])


# Rows beyond the ring (its widths, or the shared memory that its stages take): more rows than CTAs, sums of the
# weight gradients in shared memory and beyond it, whole words and single values.
@pytest.mark.parametrize("t,rows,h,dt", [(1, 700, 16400, torch.bfloat16), (2, 200, 16403, torch.bfloat16),
                                         (1, 400, 12288, torch.float32), (1, 330, 9401, torch.float32),
                                         (1, 170, 27504, torch.bfloat16), (1, 500, 27600, torch.float32)])
def test_rows_beyond_the_ring(t, rows, h, dt):
    test_residual_no_beta_and_accumulation(t, rows, h, dt)


# Short rows: around the widths at which the words, the warps of a row and the ring change.
@pytest.mark.parametrize("t,rows,h", [(3, 50, 77), (2, 41, 128), (2, 40, 150), (1, 90, 200), (1, 17, 255), (1, 9, 257),
                                      (2, 333, 301), (1, 20, 384), (4, 15, 511), (1, 2500, 129)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_short_rows(t, rows, h, dt):
    test_forward_and_backward(t, rows, h, dt, torch.float32)
    test_residual_no_beta_and_accumulation(t, rows, h, dt)


# Each way a row is taken: registers, the ring with 16-byte words and single values, with xhat kept and read again, and
# beyond the ring.
BWD_WIDTHS = [(h, dt) for h, dt in [(77, torch.float32), (256, torch.bfloat16), (256, torch.float32), (1000, torch.bfloat16),
                                    (1001, torch.float32), (1001, torch.bfloat16), (4001, torch.bfloat16), (4096, torch.bfloat16),
                                    (4096, torch.float32), (9001, torch.bfloat16), (12288, torch.bfloat16),
                                    (12288, torch.float32), (20000, torch.bfloat16)]]


@pytest.mark.parametrize("h,dt", BWD_WIDTHS)
def test_gradient_of_constant_rows(h, dt):
    """A row of one value has xhat = 0: it adds nothing to dgamma, and dx = rstd (g - mean(g))."""
    d = _inputs(1, 5, h, dt, dt, seed=h)
    d["X"] = [torch.full((5, h), 7.0, device="cuda", dtype=dt)]
    fwd = ttl.layer_norm_fwd(d["X"], d["gamma"], d["beta"])
    assert (fwd["mean"][0] == 7.0).all()
    out = ttl.layer_norm_bwd(d["X"], d["dY"], d["gamma"], fwd)
    assert torch.count_nonzero(out["dgamma"]) == 0
    g = d["dY"][0].to(F8) * d["gamma"].to(F8)
    rstd, c1 = fwd["rstd"][0].to(F8)[:, None], g.mean(1, keepdim=True)
    dx = rstd * (g - c1)
    off = rstd * (4 * U * g.abs() + _chain(h) * g.abs().mean(1, keepdim=True) + 4 * U * c1.abs()) + 4 * U * dx.abs()
    assert ((out["dX"][0].to(F8) - dx).abs() <= off + HALF[dt] * (dx.abs() + off)).all()


@pytest.mark.parametrize("h", sorted({h for h, dt in BWD_WIDTHS if dt == torch.float32} | {4099, 9401}))
def test_gradient_with_a_large_mean(h):
    """A mean 4096 times the spread.  x - mean is exact to u of itself and xhat to 3 u, so the sums are off by their
    chains' u of the terms' magnitudes and by no multiple of |mean| rstd."""
    rows = 9
    d = _inputs(1, rows, h, torch.float32, torch.float32, seed=h)
    x = (torch.randn(rows, h, generator=torch.Generator().manual_seed(h)) + 4096.0).cuda()
    fwd = ttl.layer_norm_fwd([x], d["gamma"], d["beta"])
    out = ttl.layer_norm_bwd([x], d["dY"], d["gamma"], fwd)
    mean, rstd = fwd["mean"][0].to(F8)[:, None], fwd["rstd"][0].to(F8)[:, None]
    n, dy = (x.to(F8) - mean) * rstd, d["dY"][0].to(F8)
    g = dy * d["gamma"].to(F8)
    c1, c2 = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
    dx = rstd * (g - c1 - n * c2)
    c, n_off = _chain(h), 4 * U * n.abs()
    off = rstd * (4 * U * g.abs() + c * g.abs().mean(1, keepdim=True) + 4 * U * c1.abs() + n_off * c2.abs()
                  + n.abs() * (c + 4 * U) * (g * n).abs().mean(1, keepdim=True)) + 4 * U * dx.abs()
    assert ((out["dX"][0].to(F8) - dx).abs() <= off + U * (dx.abs() + off)).all()
    mag = (dy * n).abs().sum(0)
    assert ((out["dgamma"].to(F8) - (dy * n).sum(0)).abs() <= (rows + 8) * U * mag).all()


# More rows to a group than its ring has places (and two more): every place is filled again, its barrier's phase turns,
# and with rows above 8192 values (read again, released a row late) too.  304 groups at most of rows of 4096.
@pytest.mark.parametrize("t,rows,h,dt", [(1, 20000, 1024, torch.bfloat16), (2, 2000, 4096, torch.bfloat16),
                                         (1, 2500, 4001, torch.bfloat16), (1, 1000, 12288, torch.bfloat16),
                                         (1, 1000, 9001, torch.bfloat16), (1, 8000, 1001, torch.float32),
                                         (4, 750, 4096, torch.float32), (1, 30000, 513, torch.bfloat16)])
def test_ring_places_are_filled_again(t, rows, h, dt):
    test_forward_and_backward(t, rows, h, dt, torch.float32)
    test_residual_no_beta_and_accumulation(t, rows, h, dt)


@pytest.mark.parametrize("pad", [8, 64])
@pytest.mark.parametrize("h", [256, 1000, 4096, 12288])
def test_strided_rows_of_whole_words_give_the_same_bits(pad, h):
    """Slabs that are column ranges of wider matrices, rows on 16 bytes: every output as from contiguous copies."""
    d = _inputs(2, 700, h, torch.bfloat16, torch.bfloat16, seed=pad, residual=True, pad=pad)
    flat = {k: [x.contiguous() for x in v] if isinstance(v, list) else v for k, v in d.items()}
    a = ttl.layer_norm_fwd(d["X"], d["gamma"], d["beta"], residual=d["R"])
    c = ttl.layer_norm_fwd(flat["X"], d["gamma"], d["beta"], residual=flat["R"])
    e = ttl.layer_norm_bwd(d["X"], d["dY"], d["gamma"], a, dS=d["dS"])
    f = ttl.layer_norm_bwd(flat["X"], flat["dY"], d["gamma"], a, dS=flat["dS"])
    for n in ("Y", "S", "mean", "rstd"):
        assert all(torch.equal(x, y) for x, y in zip(a[n], c[n])), n
    assert all(torch.equal(x, y) for x, y in zip(e["dX"], f["dX"]))
    assert torch.equal(e["dgamma"], f["dgamma"]) and torch.equal(e["dbeta"], f["dbeta"])
