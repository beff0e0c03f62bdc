"""The block norms against the fp64 oracle.

Tolerances, per element (A: the sum of the magnitudes of an output's terms, which
the oracle gives): fp32 sums of a lane's up to 32 values and a tree over at most
512 lanes round at most 41 times, products and the root a few times more, so the
arithmetic is off by less than 128 2^-24 A = 2^-17 A; a bf16 store adds 2^-8 |v|, an
fp32 store 2^-24 |v|.  8-bit values add half a step: 2^-4 |v|, or 2^-10 of the
scale for subnormals.  Without any norm x' has three roundings: 2^-22 A.
"""
import numpy as np
import pytest
import torch

import activation_sparse_gemm_amd as lynx
import tests.gpu_util as gu
from oracle import block_oracle as bo
from oracle.lynx_oracle import decode_bf16
from tests.gpu_util import dev, host_f64, say
from tests.test_gpu_fp8 import product_arith
from workloads import bf16_bits_from_f32, make_activation

pytestmark = pytest.mark.gpu

FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def bf(a):
    """(device bf16 tensor, its exact values)"""
    b = bf16_bits_from_f32(np.asarray(a, dtype=np.float32))
    return dev(b), decode_bf16(b)


class Case:
    """Inputs of one call, as device tensors (d) and fp64 arrays (f)."""

    def __init__(self, M, C, B=1, f32=False, y=True, gate=True, post=None, post_affine=False, norm="rms",
                 affine=False, mod=True, rho=1.0, seed=0, offset=0.0):
        rng = np.random.default_rng(seed + M + C)
        self.M, self.C, self.f32, self.norm = M, C, f32, norm
        self.d, self.f = {}, {}
        x = decode_bf16(make_activation("heavy", M, C, seed)) + offset
        if f32:
            x = np.float32(x * (1 + 1e-3 * rng.random((M, C))))
            self.x, self.xf = torch.from_numpy(x).cuda(), x.astype(np.float64)
        else:
            self.x, self.xf = bf(x)
        if y:
            self.put("y", decode_bf16(make_activation("gelu", M, C, seed + 1)) - offset / 2)
            if gate:
                self.mod("gate", rng, B)
            if post_affine:
                self.put("post_weight", 1 + 0.2 * rng.standard_normal(C))
                self.put("post_bias", 0.2 * rng.standard_normal(C))
            for k, v in (("post_norm", post), ("residual_scale", rho), ("post_eps", 1e-5)):
                self.d[k] = self.f[k] = v
        if norm:
            if affine:
                self.put("weight", 1 + 0.2 * rng.standard_normal(C))
                self.put("bias", 0.2 * rng.standard_normal(C))
            if mod:
                self.mod("scale", rng, B)
                self.mod("shift", rng, B)
            self.d["eps"] = self.f["eps"] = 1e-6
        self.d["norm"] = self.f["norm"] = norm

    def put(self, name, a):
        self.d[name], self.f[name] = bf(a)

    def mod(self, name, rng, B):
        """Rows of a wider tensor, as a modulation projection's chunks are."""
        wide, vals = bf(0.3 * rng.standard_normal((B, 3, self.C)))
        self.d[name], self.f[name] = wide[:, 1], vals[:, 1]

    def ref(self):
        return bo.block_norm(self.xf, **self.f)


def close(got, ref, mag, store, label, arith=2.0 ** -17):
    off, tol = np.abs(got - ref), store * np.abs(ref) + arith * mag
    say(f"{label}: max error / tolerance {np.max(off / np.maximum(tol, 1e-300)):.3f}")
    assert np.isfinite(got).all() and (off <= tol).all(), label


def run(c, fp8=False, x_out=None):
    M, C = c.M, c.C
    out = None
    if c.norm:
        out = gu.nan_bf16((M, C)) if not fp8 else (
            torch.full((M, C), 0xFF, dtype=torch.uint8, device="cuda").view(FP8),
            torch.full(((C + 511) // 512, M, 4), 0xAA, dtype=torch.uint8, device="cuda").view(E8M0))
    if "y" not in c.d:
        return None, lynx.norm_modulate(c.x, fp8=fp8, out=out, **c.d)
    if x_out is None:
        x_out = torch.full_like(c.x, float("nan"))
    return lynx.residual_norm(c.x, fp8=fp8, x_out=x_out, out=out, **c.d)


def check(c, label, fp8=False):
    say(label)
    xo, h = run(c, fp8)
    torch.cuda.synchronize()
    u, umag, hr, hmag = c.ref()
    if xo is not None:
        # without a post-norm there is no sum in x'
        close(host_f64(xo), u, umag, 2.0 ** -24 if c.f32 else 2.0 ** -8, label + " x'",
              2.0 ** -17 if c.f["post_norm"] else 2.0 ** -22)
    if c.norm is None:
        assert h is None
    elif not fp8:
        close(host_f64(h), hr, hmag, 2.0 ** -8, label + " h")
    else:
        check_fp8(h, hr, hmag, label)


def check_fp8(h, hr, hmag, label):
    M, C = hr.shape
    codes, stored = h[0].view(torch.uint8).cpu().numpy(), h[1].view(torch.uint8).cpu().numpy()
    kb = -(-C // 128)
    byte = stored.transpose(1, 0, 2).reshape(M, -1)
    assert np.all(byte[:, kb:] == 127)
    byte = byte[:, :kb]
    want_codes, want = bo.quantize(hr)
    # a scale may differ only where the largest value is within the arithmetic's error of 448 2^e
    amax = np.stack([np.abs(hr[:, 128 * i:128 * i + 128]).max(1) for i in range(kb)], 1)
    slack = np.stack([hmag[:, 128 * i:128 * i + 128].max(1) for i in range(kb)], 1) * 2.0 ** -17
    for i, j in zip(*np.nonzero(byte != want)):
        edge = 448 * 2.0 ** (min(int(byte[i, j]), int(want[i, j])) - 127)
        assert abs(int(byte[i, j]) - int(want[i, j])) == 1 and abs(amax[i, j] - edge) <= slack[i, j]
    v = bo.values(codes, byte)
    sub = np.exp2(byte.astype(float) - 127 - 10).repeat(128, 1)[:, :C]
    tol = np.maximum(2.0 ** -4 * np.abs(hr), sub) + 2.0 ** -16 * hmag
    assert np.all(np.abs(v - hr) <= tol), label
    # the codes are the oracle's but for values next to a rounding border: a border is within 2^-17 A of
    # a value with a chance of about 2^-17 A / (2^-4 |v|), A / |v| being a few for most
    assert np.mean(codes != want_codes) <= 0.01 + 16.0 / codes.size, label


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("M,C,B,f32", [(1, 8, 1, False), (3, 64, 3, True), (5, 504, 5, False), (6, 512, 2, False),
                                       (7, 520, 1, True), (64, 3072, 2, False), (30, 1160, 3, False),
                                       (9, 4096, 1, True), (9, 4104, 3, False), (4, 16384, 2, True),
                                       (2050, 1536, 2, False), (4100, 2056, 1, True), (2049, 520, 1, False),
                                       (2304, 3072, 2, True), (2064, 4096, 2, False)])
def test_norm_modulate(norm, M, C, B, f32):
    check(Case(M, C, B, f32, y=False, norm=norm, affine=bool(M % 2)), f"norm_modulate {norm} {M}x{C} B={B} f32={f32}")


@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("norm", [None, "rms", "layer"])
@pytest.mark.parametrize("M,C,B,f32", [(2, 64, 2, False), (33, 1024, 3, True), (2052, 1152, 2, False),
                                       (12, 6144, 1, True)])
def test_residual_norm(post, norm, M, C, B, f32):
    check(Case(M, C, B, f32, post=post, post_affine=post == "rms", norm=norm, affine=norm == "layer",
               rho=0.5 if f32 else 1.0), f"residual_norm {post} {norm} {M}x{C} B={B} f32={f32}")


@pytest.mark.parametrize("M,C,B,f32,y", [(1, 64, 1, False, False), (10, 192, 2, True, True), (33, 576, 3, False, True),
                                         (64, 3072, 2, False, False), (2304, 3072, 2, False, True),
                                         (2050, 704, 2, True, True), (7, 9216, 1, True, False)])
def test_fp8_output(M, C, B, f32, y):
    check(Case(M, C, B, f32, y=y, norm="layer", post="rms" if f32 else None, affine=f32),
          f"fp8 norm {M}x{C} B={B} f32={f32} y={y}", fp8=True)


def test_no_parameters_and_broadcast_gate():
    c = Case(40, 256, 1, gate=False, mod=False, norm="rms")
    check(c, "no parameters")
    c.d["gate"], c.f["gate"] = c.d["y"][0].clone(), c.f["y"][:1]      # one row [C] for all
    c.d["scale"], c.f["scale"] = c.d["y"][:4].clone(), c.f["y"][:4]   # and a row per sample
    check(c, "broadcast gate")
    c.d["shift"], c.f["shift"] = c.d["y"].clone(), c.f["y"]           # samples disagree
    with pytest.raises(ValueError, match="shift"):
        run(c)
    c.d["scale"], c.f["scale"] = c.d["shift"], c.f["shift"]           # a row per token
    check(c, "a modulation per token")


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_large_common_offset(norm):
    """A mean far above the spread: the variance is taken around the mean."""
    c = Case(20, 1024, 1, True, y=False, norm=norm, mod=False, offset=4096.0)
    check(c, f"offset {norm}")


def test_constant_and_zero_rows():
    x = np.zeros((6, 256))
    x[1] = 3.0
    x[2, 5] = 1e-3
    X, xf = bf(x)
    for norm in ("rms", "layer"):
        say(f"constant rows {norm}")
        h = lynx.norm_modulate(X, norm=norm)
        _, _, ref, mag = bo.block_norm(xf, norm=norm)
        close(host_f64(h), ref, mag, 2.0 ** -8, f"constant rows {norm}")
        q, s = lynx.norm_modulate(X, norm=norm, fp8=True)
        assert np.all(q.view(torch.uint8)[0].cpu().numpy() & 0x7F == 0)
        assert np.all(s.view(torch.uint8)[:, 0].cpu().numpy() == 127)


@pytest.mark.parametrize("M", [8, 2100])
def test_non_finite_rows_stay_in_their_row(M):
    c = Case(M, 1024, 1, post="rms", norm="layer")
    c.x[3, 100] = float("nan")
    c.d["y"][5, 900] = float("inf")
    say(f"non-finite rows M={M}")
    xo, h = run(c)
    _, (q, s) = run(c, fp8=True)
    good = torch.ones(M, dtype=torch.bool, device="cuda")
    good[[3, 5]] = False
    assert bool(torch.isfinite(h.float()[good]).all()) and bool(torch.isfinite(xo.float()[good]).all())
    assert bool(torch.isnan(h.float()[[3, 5]]).all())
    sb = s.view(torch.uint8)
    assert bool((sb[:, [3, 5]] == 255).all()) and not bool((sb[:, good] == 255).any())


def test_in_place_residual_and_fused_halves():
    """x_out may be x; and a fused call gives the residual of the unfused one."""
    for M in (50, 2060):
        c = Case(M, 1152, 2, True, post="rms", norm="rms")
        say(f"in place M={M}")
        xo, h = run(c)
        halves = {k: v for k, v in c.d.items() if k not in ("norm", "scale", "shift", "eps")}
        x1, none = lynx.residual_norm(c.x, **halves)
        assert none is None and torch.equal(x1, xo)
        h1 = lynx.norm_modulate(x1, **{k: c.d[k] for k in ("norm", "scale", "shift", "eps")})
        assert torch.equal(h1, h)      # fp32 x': nothing is lost between the two calls
        xi, hi = run(c, x_out=c.x)
        assert xi is c.x and torch.equal(xi, xo) and torch.equal(hi, h)


def test_refusals_on_device_tensors():
    x = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    p = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    for call, err, text in [
        (lambda: lynx.norm_modulate(x.half()), TypeError, "x"),
        (lambda: lynx.norm_modulate(x, norm="batch"), ValueError, "norm"),
        (lambda: lynx.norm_modulate(x, weight=p), ValueError, "weight"),
        (lambda: lynx.norm_modulate(x, scale=p.float()), TypeError, "scale"),
        (lambda: lynx.norm_modulate(x, scale=p[:, :32]), ValueError, "scale"),
        (lambda: lynx.norm_modulate(x, scale=p.t().contiguous().t()), ValueError, "scale"),
        (lambda: lynx.residual_norm(x, x.float()), TypeError, "y"),
        (lambda: lynx.residual_norm(x, x, out=x), ValueError, "output"),
        (lambda: lynx.residual_norm(x, x, post_weight=p[0]), lynx.LynxError, "NULL"),
        (lambda: lynx.norm_modulate(x, scale=torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")),
         lynx.LynxError, "SHAPE"),
        (lambda: lynx.norm_modulate(torch.zeros((2, 72), dtype=torch.bfloat16, device="cuda"), fp8=True),
         lynx.LynxError, "SHAPE"),
        (lambda: lynx.norm_modulate(x, scale=torch.zeros((2, 68), dtype=torch.bfloat16, device="cuda")[:, :64]),
         lynx.LynxError, "SHAPE"),
    ]:
        with pytest.raises(err, match=text):
            call()
    assert lynx.norm_modulate(x[:0]).shape == (0, 64)


def test_a_block_of_layers_end_to_end():
    """norm -> 8-bit MLP-up -> 8-bit MLP-down -> gate + residual + next norm -> sparse layer,
    eager, then captured and replayed, against the oracle on the stages' own inputs."""
    from oracle import lynx_oracle as orc
    from workloads import make_layer
    M, C, H, B = 600, 512, 1536, 2
    c = Case(M, C, B, norm="layer", post="rms")
    rng = np.random.default_rng(4)
    w1, w1f = bf(rng.standard_normal((H, C)) * C ** -0.5)
    w2, w2f = bf(rng.standard_normal((C, H)) * H ** -0.5)
    up, down = lynx.quantize_fp8_weight(w1), lynx.quantize_fp8_weight(w2)
    L = make_layer(M, C, 640, "heavy", seed=3, R=16)
    W, LA, LB = dev(L.W), dev(L.LA), dev(L.LB)
    mod = {k: c.d[k] for k in ("norm", "scale", "shift", "eps")}

    def block():
        q, s = lynx.norm_modulate(c.x, fp8=True, **mod)
        hid = lynx.linear_fp8_packed(q, s, *up)
        branch = lynx.linear_fp8(hid, *down)
        x1, h = lynx.residual_norm(c.x, branch, gate=c.d["gate"], post_norm="rms", **mod)
        return q, s, hid, branch, x1, h, lynx.linear_sparse_lora(h, W, LA, LB)

    say("block eager")
    q, s, hid, branch, x1, h, y = eager = block()
    torch.cuda.synchronize()
    byte = s.view(torch.uint8).cpu().numpy().transpose(1, 0, 2).reshape(M, -1)
    qv = bo.values(q.view(torch.uint8).cpu().numpy(), byte)

    def product(Y, xv, w):
        wv = bo.values(*bo.quantize_weight(w), 128)
        ref, mag = bo.linear(xv, wv)
        close(host_f64(Y), ref, mag, 2.0 ** -8, "block product", product_arith(xv.shape[1]))
        assert gu.row_rel_err(host_f64(Y), ref).max() <= gu.ROW_REL_TOL

    product(hid, qv, w1f)
    product(branch, bo.values(*bo.quantize(host_f64(hid))), w2f)
    f = {k: c.f[k] for k in ("norm", "scale", "shift", "eps", "gate")}
    u, um, hr, hm = bo.block_norm(c.xf, host_f64(branch), post_norm="rms", **f)
    close(host_f64(x1), u, um, 2.0 ** -8, "block x'")
    close(host_f64(h), hr, hm, 2.0 ** -8, "block h")
    ref = orc.linear_sparse_lora(gu.host_bits(h), L.W, L.LA, L.LB)
    assert gu.row_rel_err(host_f64(y), ref).max() <= gu.ROW_REL_TOL

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        captured = block()
    for i in range(3):
        say(f"block graph replay {i}")
        for t in captured:
            t.view(torch.uint8).fill_(0xFF)
        block()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
