"""GPU: the norms before and after a block (norm_fwd, norm_bwd) against the
formulas in FP64, element by element.

Tolerances, derived before any run: an output rounded once to the stored type
is off by its unit roundoff u (2^-8 BF16, 2^-11 FP16; FP16 also by half its
smallest subnormal) times its value; the FP32 work before it by c 2^-24 times
the sum S of the magnitudes of the terms it adds.  A row's sum of squares is at
most 16 adds in a thread, 6 across lanes and 15 across waves, each operation one
rounding, so c = 64 covers a forward output (two chained norms, half of each
sum's error through the square root) and c = 128 a backward one.  A column sum
over M rows adds at most M / 512 + 1 values in a register and 128 + 3 parts:
c = M / 512 + 256."""
import numpy as np
import pytest
import torch

from deterministic_gated_ffn_amd import binding as dgf

pytestmark = pytest.mark.gpu

BF, FH = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, FH: 2.0 ** -11}
TINY = {BF: 2.0 ** -134, FH: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests need an MI355X")
    dgf.load()


def rows(gen, shape, dt, scale=1.0, shift=0.0, pad=0):
    """A row-major view whose leading dimension is a multiple of 8 and whose padding is NaN."""
    ld = -(-shape[-1] // 8) * 8 + pad
    buf = torch.full((*shape[:-1], ld), float("nan"), dtype=dt)
    buf[..., :shape[-1]] = (torch.randn(shape, generator=gen) * scale + shift).to(dt)
    return buf.cuda()[..., :shape[-1]]


def f64(t):
    return t.detach().cpu().double()


def close(name, got, want, size, dt, c):
    """|got - want| <= u |want| + c 2^-24 size + half the smallest subnormal."""
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.isfinite(got).all(), name
    tol = U[dt] * want.abs() + c * 2.0 ** -24 * size + TINY[dt]
    off = (got - want).abs()
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3f} of the tolerance"


def forward64(res, y, w_post, gate, alpha, w_next, eps):
    H = res.shape[1]
    z = res if y is None else alpha * res
    size = z.abs()
    r_y = torch.ones(res.shape[0], 1, dtype=torch.float64)
    if y is not None:
        t = y
        if w_post is not None:
            r_y = 1.0 / torch.sqrt(y.square().sum(1, keepdim=True) / H + eps)
            t = y * r_y * w_post
        t = t if gate is None else t * gate
        z, size = z + t, size + t.abs()
    r_z = torch.ones_like(r_y)
    h = hs = None
    if w_next is not None:
        r_z = 1.0 / torch.sqrt(z.square().sum(1, keepdim=True) / H + eps)
        h = z * r_z * w_next
        # z's own error moves r_z too, by at most its mean share
        hs = (size + z.abs() * (size.square().mean(1, keepdim=True).sqrt() * r_z)) * r_z * w_next.abs()
    return z, size, h, hs, r_y, r_z


def backward64(dz, dh, z, y, w_post, gate, alpha, w_next, r_y, r_z):
    """The gradients and, with every term's magnitude in its place, their sizes."""
    H = z.shape[1]
    out, sizes = {}, {}
    G, Gs = (dz, dz.abs()) if dz is not None else (torch.zeros_like(z), torch.zeros_like(z))
    if dh is not None:
        dn = dh * w_next
        G = G + r_z * (dn - z * r_z ** 2 * (dn * z).sum(1, keepdim=True) / H)
        Gs = Gs + r_z * (dn.abs() + z.abs() * r_z ** 2 * (dn * z).abs().sum(1, keepdim=True) / H)
        out["dw_next"], sizes["dw_next"] = (dh * z * r_z).sum(0), (dh * z * r_z).abs().sum(0)
    out["dres"], sizes["dres"] = alpha * G, abs(alpha) * Gs
    if y is not None:
        g = torch.ones_like(z[:1]) if gate is None else gate
        t = y if w_post is None else y * r_y * w_post
        if gate is not None:
            a, b = G * t, Gs * t.abs()
            out["dgate"], sizes["dgate"] = (a.sum(0), b.sum(0)) if gate.dim() == 1 else (a, b)
        if w_post is None:
            out["dy"], sizes["dy"] = G * g, Gs * g.abs()
        else:
            dq, dqs = G * g * w_post, Gs * (g * w_post).abs()
            out["dy"] = r_y * (dq - y * r_y ** 2 * (dq * y).sum(1, keepdim=True) / H)
            sizes["dy"] = r_y * (dqs + y.abs() * r_y ** 2 * (dqs * y.abs()).sum(1, keepdim=True) / H)
            out["dw_post"] = (G * g * y * r_y).sum(0)
            sizes["dw_post"] = (Gs * (g * y).abs() * r_y).sum(0)
    return out, sizes


def make(M, H, dt, gate, post=True, seed=0, pad=0):
    gen = torch.Generator().manual_seed(seed)
    d = {"res": rows(gen, (M, H), dt, 1.5, pad=pad), "y": rows(gen, (M, H), dt, 0.5, pad=8 - pad),
         "w_post": rows(gen, (H,), dt, 0.1, 1.0) if post else None, "w_next": rows(gen, (H,), dt, 0.1, 1.0),
         "gate": {"none": None, "row": rows(gen, (H,), dt, 0.3, 0.5), "full": rows(gen, (M, H), dt, 0.3, 0.5)}[gate],
         "dz": rows(gen, (M, H), dt, 0.1, pad=pad), "dh": rows(gen, (M, H), dt, 0.1)}
    return d, {k: None if v is None else f64(v) for k, v in d.items()}


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 64), (1, 511), (33, 513), (4, 4096), (7, 5125), (2, 8192), (3, 8200), (2, 16383),
          (1, 16384), (700, 96), (2100, 40)]


@pytest.mark.parametrize("dt", [BF, FH])
@pytest.mark.parametrize("M,H", SHAPES)
@pytest.mark.parametrize("gate,post,alpha", [("none", True, 1.0), ("row", True, 0.5), ("full", True, -1.25),
                                             ("row", False, 1.0), ("none", False, 2.0)])
def test_norms_and_their_gradients(M, H, gate, post, alpha, dt):
    d, e = make(M, H, dt, gate, post, seed=M * 31 + H, pad=8 if H % 16 else 0)
    eps = 1e-5
    r = dgf.norm_fwd(d["res"], d["y"], d["w_post"], d["gate"], alpha, d["w_next"], eps, training=True)
    z, zs, h, hs, r_y, r_z = forward64(e["res"], e["y"], e["w_post"], e["gate"], alpha, e["w_next"], eps)
    close("z", r["z"], z, zs, dt, 64)
    close("h", r["h"], h, hs, dt, 64)
    rstd = f64(r["rstd"])
    scale = (zs.square().mean(1, keepdim=True).sqrt() * r_z).clamp(min=1.0)
    assert ((rstd[:, :1] - r_y).abs() <= 64 * 2.0 ** -24 * r_y).all()
    assert ((rstd[:, 1:] - r_z).abs() <= 64 * 2.0 ** -24 * r_z * scale).all()

    b = dgf.norm_bwd(d["dz"], d["dh"], r["z"], d["y"], d["w_post"], d["gate"], alpha, d["w_next"], r["rstd"])
    want, sizes = backward64(e["dz"], e["dh"], f64(r["z"]), e["y"], e["w_post"], e["gate"], alpha, e["w_next"],
                             rstd[:, :1], rstd[:, 1:])
    assert set(b) == set(want)
    for k in want:
        close(k, b[k], want[k], sizes[k], dt, 128 if want[k].dim() == 2 else M / 512 + 256)


@pytest.mark.parametrize("dt", [BF, FH])
def test_norm_before_a_block_alone(dt):
    d, e = make(9, 1000, dt, "none")
    r = dgf.norm_fwd(d["res"], w_next=d["w_next"], eps=1e-6, training=True)
    assert r["z"] is d["res"]
    z, zs, h, hs, _, r_z = forward64(e["res"], None, None, None, 1.0, e["w_next"], 1e-6)
    close("h", r["h"], h, hs, dt, 64)
    assert (f64(r["rstd"])[:, 0] == 1).all()
    for dz, dh in ((None, d["dh"]), (d["dz"], d["dh"])):
        b = dgf.norm_bwd(dz, dh, r["z"], w_next=d["w_next"], rstd=r["rstd"])
        want, sizes = backward64(None if dz is None else e["dz"], e["dh"], e["res"], None, None, None, 1.0,
                                 e["w_next"], None, f64(r["rstd"])[:, 1:])
        assert set(b) == {"dres", "dw_next"}
        close("dres", b["dres"], want["dres"], sizes["dres"], dt, 128)
        close("dw_next", b["dw_next"], want["dw_next"], sizes["dw_next"], dt, 257)


@pytest.mark.parametrize("dt", [BF, FH])
def test_norm_after_a_block_alone(dt):
    d, e = make(6, 777, dt, "full")
    r = dgf.norm_fwd(d["res"], d["y"], d["w_post"], d["gate"], 0.5, training=True)
    assert "h" not in r and (f64(r["rstd"])[:, 1] == 1).all()
    z, zs, *_, r_y, _ = forward64(e["res"], e["y"], e["w_post"], e["gate"], 0.5, None, 1e-6)
    close("z", r["z"], z, zs, dt, 64)
    b = dgf.norm_bwd(d["dz"], None, r["z"], d["y"], d["w_post"], d["gate"], 0.5, rstd=r["rstd"])
    want, sizes = backward64(e["dz"], None, f64(r["z"]), e["y"], e["w_post"], e["gate"], 0.5, None,
                             f64(r["rstd"])[:, :1], None)
    assert set(b) == set(want)
    for k in want:
        close(k, b[k], want[k], sizes[k], dt, 128 if want[k].dim() == 2 else 257)


def test_gradients_against_differences():
    """<gradient, v> against the central difference of the FP64 forward along v.
    The difference's own error is O(step^2) (2^-26 here); the gradients' roundings
    add up to at most u sum |g v|, and z, rounded before the backward reads it,
    moves them by its relative rounding again: 4 u sum |g v| covers both."""
    M, H, dt, alpha, eps = 5, 96, FH, 0.75, 1e-5
    d, e = make(M, H, dt, "row", seed=5)
    r = dgf.norm_fwd(d["res"], d["y"], d["w_post"], d["gate"], alpha, d["w_next"], eps, training=True)
    b = dgf.norm_bwd(d["dz"], d["dh"], r["z"], d["y"], d["w_post"], d["gate"], alpha, d["w_next"], r["rstd"])

    def loss(**change):
        a = {**e, **change}
        z, _, h, *_ = forward64(a["res"], a["y"], a["w_post"], a["gate"], alpha, a["w_next"], eps)
        return (z * e["dz"]).sum() + (h * e["dh"]).sum()

    gen = torch.Generator().manual_seed(11)
    step = 2.0 ** -13
    for name, key in (("res", "dres"), ("y", "dy"), ("w_post", "dw_post"), ("gate", "dgate"), ("w_next", "dw_next")):
        v = torch.randn(e[name].shape, generator=gen, dtype=torch.float64)
        diff = (loss(**{name: e[name] + step * v}) - loss(**{name: e[name] - step * v})) / (2 * step)
        g = f64(b[key])
        tol = 4 * U[dt] * (g * v).abs().sum() + 1e-6
        assert abs((g * v).sum() - diff) <= tol, (name, float((g * v).sum()), float(diff), float(tol))


@pytest.mark.parametrize("dt", [BF, FH])
def test_zero_rows_and_large_values(dt):
    # a row of zeros normalises to zeros (r = 1/sqrt(eps)); large finite rows stay finite
    M, H = 3, 200
    d, e = make(M, H, dt, "none")
    res, y = d["res"].clone(), d["y"].clone()
    res[0], y[0] = 0, 0
    res[1], y[1] = 30000.0, -20000.0
    r = dgf.norm_fwd(res, y, d["w_post"], None, 1.0, d["w_next"], 1e-6, training=True)
    assert (f64(r["z"])[0] == 0).all() and (f64(r["h"])[0] == 0).all()
    assert np.isclose(f64(r["rstd"])[0].numpy(), 1000.0, rtol=1e-6).all()
    z, zs, h, hs, *_ = forward64(f64(res), f64(y), e["w_post"], None, 1.0, e["w_next"], 1e-6)
    close("z", r["z"], z, zs, dt, 64)
    close("h", r["h"], h, hs, dt, 64)


@pytest.mark.parametrize("M", [64, 600])
def test_rows_do_not_depend_on_the_batch_and_runs_repeat(M):
    d, _ = make(M, 1024, BF, "full", seed=3)
    call = lambda n: dgf.norm_fwd(d["res"][:n], d["y"][:n], d["w_post"], d["gate"][:n], 1.0, d["w_next"],  # noqa: E731
                                  training=True)
    full, few = call(M), call(5)
    for k in full:
        assert torch.equal(full[k][:5], few[k]), k
    bwd = lambda n: dgf.norm_bwd(d["dz"][:n], d["dh"][:n], full["z"][:n], d["y"][:n], d["w_post"], d["gate"][:n],  # noqa: E731
                                 1.0, d["w_next"], full["rstd"][:n].contiguous())
    one, again, part = bwd(M), bwd(M), bwd(5)
    for k in one:
        assert torch.equal(one[k], again[k]), k
        if one[k].dim() == 2:
            assert torch.equal(one[k][:5], part[k]), k


def test_in_place_and_other_streams():
    d, _ = make(40, 2048, BF, "row")
    want = dgf.norm_fwd(d["res"], d["y"], d["w_post"], d["gate"], 1.0, d["w_next"], training=True)
    side = torch.cuda.Stream()
    res = d["res"].clone()
    torch.cuda.synchronize()
    got = dgf.norm_fwd(res, d["y"], d["w_post"], d["gate"], 1.0, d["w_next"], training=True, out=res, stream=side)
    side.synchronize()
    assert got["z"] is res
    for k in want:
        assert torch.equal(got[k], want[k]), k
    dz = d["dz"].clone()
    a = dgf.norm_bwd(d["dz"], d["dh"], want["z"], d["y"], d["w_post"], d["gate"], 1.0, d["w_next"], want["rstd"])
    b = dgf.norm_bwd(dz, d["dh"], want["z"], d["y"], d["w_post"], d["gate"], 1.0, d["w_next"], want["rstd"],
                     stream=side)
    side.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_no_rows():
    H = 100
    d, _ = make(1, H, BF, "row")
    e = {k: v[:0] for k, v in d.items() if k in ("res", "y", "dz", "dh")}
    r = dgf.norm_fwd(e["res"], e["y"], d["w_post"], d["gate"], 1.0, d["w_next"], training=True)
    assert r["z"].shape == (0, H) and r["h"].shape == (0, H) and r["rstd"].shape == (0, 2)
    b = dgf.norm_bwd(e["dz"], e["dh"], r["z"], e["y"], d["w_post"], d["gate"], 1.0, d["w_next"], r["rstd"])
    for k in ("dw_post", "dw_next", "dgate"):
        assert b[k].shape == (H,) and (b[k].cpu().view(torch.int16) == 0).all(), k


@pytest.mark.parametrize("M,H", [(513, 64), (515, 256), (769, 1024), (1031, 200)])
def test_an_infinite_gradient_in_the_last_row_stays_an_infinity(M, H):
    # a workgroup of several row slots has some without a row here
    gen = torch.Generator().manual_seed(M)
    z, y, dz, dh = (rows(gen, (M, H), BF) for _ in range(4))
    w = torch.ones(H, dtype=BF, device="cuda")
    z[M - 1, 5], dh[M - 1, 5] = 1.0, float("inf")
    rstd = dgf.norm_fwd(z, y, w_post=w, w_next=w, training=True)["rstd"]
    rstd[:, 1] = 1.0 / torch.sqrt(z.float().square().mean(1) + 1e-6)
    d = dgf.norm_bwd(dz, dh, z, y, w_post=w, w_next=w, rstd=rstd)
    dw = f64(d["dw_next"])
    assert dw[5] == float("inf") and torch.isfinite(dw[torch.arange(H) != 5]).all()


@pytest.mark.parametrize("given,gate", [(a, b) for a in ("all", "no dz", "post") for b in ("none", "row", "full")]
                         + [("next", "none"), ("last", "none")])  # without a block output there is no gate
@pytest.mark.parametrize("M,H,dt", [(1100, 200, BF), (1100, 203, FH), (1031, 1024, FH), (520, 6001, BF), (520, 8200, BF),
                                    (520, 9819, FH), (530, 12288, FH), (300, 12296, BF), (300, 16379, FH)])
def test_gradients_over_several_rows_a_workgroup(M, H, dt, gate, given):
    # every way of loading ahead, with the parts that may be missing
    d, e = make(M, H, dt, gate, True, seed=M + H)
    drop = {"all": (), "no dz": ("dz",), "next": ("y", "w_post"), "last": ("dz", "y", "w_post"),
            "post": ("dh", "w_next")}[given]
    for k in drop:
        d[k] = e[k] = None
    alpha = 1.0 if d["y"] is None else 0.75
    r = dgf.norm_fwd(d["res"], d["y"], d["w_post"], d["gate"], alpha, d["w_next"], 1e-5, training=True)
    rstd = f64(r["rstd"])
    b = dgf.norm_bwd(d["dz"], d["dh"], r["z"], d["y"], d["w_post"], d["gate"], alpha, d["w_next"], r["rstd"])
    want, sizes = backward64(e["dz"], e["dh"], f64(r["z"]), e["y"], e["w_post"], e["gate"], alpha, e["w_next"],
                             rstd[:, :1], rstd[:, 1:])
    assert set(b) == set(want)
    for k in want:
        close(k, b[k], want[k], sizes[k], dt, 128 if want[k].dim() == 2 else M / 512 + 256)
    again = dgf.norm_bwd(d["dz"], d["dh"], r["z"], d["y"], d["w_post"], d["gate"], alpha, d["w_next"], r["rstd"])
    assert all(torch.equal(b[k], again[k]) for k in b)


@pytest.mark.parametrize("dz", [False, True])
@pytest.mark.parametrize("M,H", [(4, 200), (4, 203), (5, 4096), (5, 9819), (4, 12288), (3, 16379)])
def test_gradients_of_rows_far_from_one(M, H, dz):
    """BF16 rows of root mean square 1e15 and 1e-13, and rows of zeros under an eps
    of 1e-30 (r = 1e15): the cube of their r lies outside FP32, every term of the
    formula within.  dh follows the normed row, so that the projection is no small
    part of the gradient."""
    gen = torch.Generator().manual_seed(H)
    unit = torch.randn((3, M, H), generator=gen)
    rms = torch.tensor([1e15, 1e-13, 1.0, 0.0, 1e15])[:M, None]
    z, y = rows(gen, (M, H), BF), rows(gen, (M, H), BF)
    z.copy_((unit[0] * rms).to(BF))
    y.copy_((unit[1] * rms.flip(0)).to(BF))
    dh = rows(gen, (M, H), BF)
    dh.copy_((unit[0] + 0.5 * unit[2]).to(BF))
    g = rows(gen, (M, H), BF, 0.1) if dz else None
    w, wn, gate = rows(gen, (H,), BF, 0.1, 1.0), rows(gen, (H,), BF, 0.1, 1.0), rows(gen, (H,), BF, 0.3, 0.5)
    rstd = torch.stack([(f64(t).square().mean(1) + 1e-30).rsqrt() for t in (y, z)], 1).float().cuda()
    r_y, r_z = f64(rstd)[:, :1], f64(rstd)[:, 1:]
    for yy, ww, gg in ((None, None, None), (y, w, None), (y, w, gate)):
        b = dgf.norm_bwd(g, dh, z, yy, ww, gg, w_next=wn, rstd=rstd)
        want, sizes = backward64(f64(g) if dz else None, f64(dh), f64(z), None if yy is None else f64(y),
                                 None if ww is None else f64(w), None if gg is None else f64(gate), 1.0, f64(wn), r_y, r_z)
        assert set(b) == set(want)
        for k in want:
            close(k, b[k], want[k], sizes[k], BF, 128 if want[k].dim() == 2 else 257)


@pytest.mark.parametrize("given,gate", [("all", "none"), ("all", "row"), ("all", "full"), ("next", "none"),
                                        ("post", "row"), ("plain", "row")])
@pytest.mark.parametrize("M,H,dt", [(1031, 203, BF), (1100, 200, FH), (700, 1024, BF), (520, 4096, BF), (520, 6001, FH),
                                    (520, 9819, BF), (530, 12288, BF), (300, 16379, FH), (300, 16384, BF)])
def test_dres_written_over_dz(M, H, dt, gate, given):
    # rows loaded ahead, rows repeated in slots without one, ragged ends: the same bits as apart
    d, _ = make(M, H, dt, gate, given != "plain", seed=M)
    if given == "next":
        d["y"] = d["w_post"] = None
    if given == "post":
        d["dh"] = d["w_next"] = None
    alpha = 1.0 if d["y"] is None else 0.75
    r = dgf.norm_fwd(d["res"], d["y"], d["w_post"], d["gate"], alpha, d["w_next"], 1e-5, training=True)
    want = dgf.norm_bwd(d["dz"], d["dh"], r["z"], d["y"], d["w_post"], d["gate"], alpha, d["w_next"], r["rstd"])
    L = dgf.load()
    out = {k: torch.empty_strided(v.shape, v.stride(), dtype=dt, device="cuda") for k, v in want.items() if k != "dres"}
    dz = d["dz"]
    nbytes = L.dgf_norm_bwd_workspace(M, H)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    ld = lambda t: 0 if t is None or t.dim() == 1 else t.stride(0)  # noqa: E731
    st = L.dgf_norm_bwd(ptr(dz), ld(dz), ptr(d["dh"]), ld(d["dh"]), ptr(r["z"]), ld(r["z"]), ptr(d["y"]), ld(d["y"]),
                        ptr(d["w_post"]), ptr(d["gate"]), ld(d["gate"]), alpha, ptr(d["w_next"]), ptr(r["rstd"]),
                        ptr(dz), ld(dz), ptr(out.get("dy")), ld(out.get("dy")), ptr(out.get("dw_post")),
                        ptr(out.get("dgate")), ld(out.get("dgate")), ptr(out.get("dw_next")), M, H, ptr(ws), nbytes,
                        dgf.DGF_BF16 if dt == BF else dgf.DGF_FP16, torch.cuda.current_stream().cuda_stream)
    assert st == 0, L.dgf_last_error()
    assert torch.equal(dz, want["dres"])
    for k in out:
        assert torch.equal(out[k], want[k]), k
