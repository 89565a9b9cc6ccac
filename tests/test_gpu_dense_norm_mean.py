"""The layer norm's mean, each row held to its own values: rows with a common
offset, constant ones among them, lose nothing to the offset, whatever the
rounding of the row's plain sum."""
import pytest

import dense_reference as ref
from test_gpu_dense_norm import forward, make, say, vjp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [5, 48, 64, 777, 2048, 4100, 20000])
def test_constant_rows_of_any_value(C, dtype):
    """The mean of a constant row is its value and y is beta. The correction of the mean is a sum of equal differences,
    chains of at most 128 terms: what it leaves is below (128 2^-24)^2 of the value (long rows 2^-34), times rstd =
    eps^-1/2 in y."""
    import torch
    say("norm constant rows", C, dtype)
    p = make(8, C, dtype, 2)
    values = (1000.1, -100.1, 3.3, 0.1, 1e6 / 3, -7e-5, 1e-20, 12345.678)
    for r, v in enumerate(values):
        p["x"][r] = v
    y, mean, rstd = forward(p, 8, C)
    x = ref.f64(p["x"])[:, 0]
    assert torch.equal(ref.f64(mean), x)
    lim = (p["gamma"].cpu().double().abs()[None] * (x.abs() * 1e-5 ** -0.5 * 2.0 ** -34)[:, None]
           + p["beta"].cpu().double().abs()[None] * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -23))
    assert ((ref.f64(y) - ref.f64(p["beta"])).abs() <= lim).all()
    assert ((ref.f64(rstd) * 1e-5 ** 0.5 - 1).abs() < 1e-4).all()
    gx, gg, gb = vjp(p, mean, rstd, 8, C)
    assert (gg == 0).all() and torch.isfinite(ref.f64(gx)).all()


@pytest.mark.parametrize("C", [48, 64, 777, 2048, 4100])
@pytest.mark.parametrize("offset", [0.0, 300.0, 4096.0, -1e5])
def test_a_common_offset_costs_nothing(C, offset):
    """Float rows of spread 2 around an offset, as stored: the differences from the mean are exact to a unit of the
    spread, their own sums (chains of at most 128 terms) err by 2^-17 of the spread; the mean itself by its rounding."""
    import torch
    say("norm offset", C, offset)
    p = make(50, C, "f32", C, offset=offset)
    y, mean, rstd = forward(p, 50, C)
    yr, mr, rr = ref.layer_norm(p["x"], p["gamma"], p["beta"])
    assert ((ref.f64(mean) - mr).abs() <= 2.0 ** -24 * mr.abs() + 2.0 ** -17 / rr).all()
    assert ((ref.f64(rstd) / rr - 1).abs() <= 2.0 ** -18).all()
    h = (ref.f64(p["x"]) - mr[:, None]) * rr[:, None]
    lim = 2.0 ** -17 * (1 + h.abs()) * ref.f64(p["gamma"]).abs() + 2.0 ** -22 * yr.abs()
    bad = (ref.f64(y) - yr).abs() > lim
    assert not bad.any(), float(((ref.f64(y) - yr).abs() / lim).max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_vjp_offsets_beyond_32_bits(dtype):
    """Rows past 2^31 elements with a gradient of their own: every output is written, in place, and right."""
    import torch
    from equivariant_interatomic_potentials_amd import dense
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    M, C, pitch = 66000, 64, 33000
    say("norm VJP offsets", dtype)
    big = torch.empty(M, pitch, dtype=dt, device="cuda")
    x, gy, gx = big[:, :C], big[:, 1000:1000 + C], big[:, 20000:20000 + C]
    g = torch.Generator(device="cuda").manual_seed(5)
    x.copy_(torch.randn(M, C, generator=g, device="cuda"))
    gy.copy_(torch.randn(M, C, generator=g, device="cuda"))
    gx.fill_(float("nan"))
    gamma = 1 + 0.3 * torch.randn(C, generator=g, device="cuda")
    y = torch.empty(M, C, dtype=dt, device="cuda")
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    gg, gb = torch.full((C,), float("nan"), device="cuda"), torch.full((C,), float("nan"), device="cuda")
    ws = torch.empty(dense.etp_layer_norm_vjp_workspace(M, C, dt), dtype=torch.uint8, device="cuda")
    dense.etp_layer_norm(x, y, None, None, 1e-5, mean, rstd)
    dense.etp_layer_norm_vjp(x, mean, rstd, gy, gamma, gx, gg, gb, ws)
    wx, wg, wb = ref.layer_norm_vjp(x, mean, rstd, gy, gamma)
    h = (ref.f64(x) - ref.f64(mean)[:, None]) * ref.f64(rstd)[:, None]
    terms = float((ref.f64(rstd)[:, None] * (ref.f64(gy) * ref.f64(gamma)).abs() * (1 + h * h)).max())
    ref.close(gx, wx, scale=terms)
    ref.close(gg, wg)
    ref.close(gb, wb)
    assert float(wx.abs().max()) > 1e-3 * terms  # (zeros would not do)
