"""residual_rmsnorm against the 64-bit form: widths from one vector to the widest, both types, e4m3 with row
and group scales, row strides, in place, zero and non-finite rows."""
import math

import pytest
import torch

import rope_block_sparse_b200 as h3a
import prompt_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

EPS = 1e-6
E4M3 = torch.float8_e4m3fn


def draw(rows, width, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, width), generator=g, device="cuda") * (1 + 20 * (torch.rand(width, generator=g, device="cuda") < 0.02))
    x = x * torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))
    return x.to(dtype), torch.randn((rows, width), generator=g, device="cuda").to(dtype), 1 + 0.2 * torch.randn(width, generator=g, device="cuda")


def check(x, f, gamma, scales, h, y, s, label=""):
    want_h, want = ref.rmsnorm(x, f, gamma, EPS)
    if f is None:
        assert h is None
    else:
        assert torch.equal(h, want_h), label
    rel = ref.RMSNORM_RELATIVE
    if scales is None:
        assert s is None
        ref.within(y, want, want.abs() * (ref.half_step(x.dtype) + 2 * rel) + ref.HALF_SUBNORMAL[x.dtype], label)
        return
    rows, width = x.shape
    step = width if scales == "row" else 128
    groups = -(-width // step)
    padded = torch.nn.functional.pad(want, (0, groups * step - width)).view(rows, groups, step)
    want_s = padded.abs().amax(2).clamp(min=2.0 ** -100) / 448
    assert y.dtype == E4M3 and s.dtype == torch.float32
    ref.within(s.view(rows, groups), want_s, 2 * rel * want_s, label + " scales")
    target = (padded / want_s[..., None]).view(rows, -1)[:, :width]
    # e4m3: half a step is 2^-4 relative, 2^-10 among the subnormals; y and the scale are fp32 before it
    ref.within(y.double(), target, target.abs() * (2.0 ** -4 + 4 * rel) + 2.0 ** -10, label + " e4m3")


SHAPES = [(1, 8), (5, 128), (3, 136), (8, 5376), (1023, 2000), (33, 1024), (7, 1032), (300, 4096), (4, 14336), (2, 16384), (2000, 96), (700, 5376),
          (9000, 64), (40000, 120), (9001, 256), (3000, 392), (5000, 768), (2500, 8192)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scales", [None, "row", "group"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rmsnorm_matches(shape, scales, dtype):
    x, f, gamma = draw(*shape, dtype=dtype, seed=shape[1])
    if dtype == torch.float16:
        x = x.clamp(-3e4, 3e4)
    check(x, f, gamma, scales, *h3a.residual_rmsnorm(x, f, gamma, EPS, scales=scales), "residual")
    check(x, None, gamma, scales, *h3a.residual_rmsnorm(x, None, gamma, EPS, scales=scales), "alone")


@pytest.mark.parametrize("scales", [None, "row", "group"])
def test_rmsnorm_strides_and_in_place(scales):
    """Rows of wider buffers; h written over x or f; the buffers' other columns and rows untouched."""
    x, f, gamma = draw(61, 1288, seed=3)
    want = h3a.residual_rmsnorm(x, f, gamma, EPS, scales=scales)
    wide = [torch.full((64, 1408), 5.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    xs, fs = wide[0][2:63, 64:64 + 1288], wide[1][1:62, :1288]
    for target in (xs, fs):
        xs.copy_(x), fs.copy_(f)
        y8 = torch.zeros(64, 1360, device="cuda", dtype=torch.uint8)
        y = y8[:61, 16:16 + 1288].view(E4M3) if scales else torch.zeros(61, 1296, device="cuda", dtype=x.dtype)[:, 8:]
        s = None if want[2] is None else torch.zeros_like(want[2])
        h3a.residual_rmsnorm(xs, fs, gamma, EPS, scales=scales, out=(target, y, s))
        assert torch.equal(target, want[0]) and torch.equal(y.float(), want[1].float())
        assert s is None or torch.equal(s, want[2])
        target.fill_(5.0), (fs if target is xs else xs).fill_(5.0)
        assert (wide[0] == 5.0).all() and (wide[1] == 5.0).all()
        if scales:
            y.view(torch.uint8).zero_()
            assert not y8.any()


@pytest.mark.parametrize("scales", [None, "row", "group"])
def test_rmsnorm_zero_and_nonfinite_rows(scales):
    x, _, gamma = draw(6, 1024, seed=4)
    x[1] = 0
    x[2, 300] = math.nan
    x[3, 5] = math.inf
    x[4, 128:256] = 0
    h, y, s = h3a.residual_rmsnorm(x, torch.zeros_like(x), gamma, EPS, scales=scales)
    rows = torch.tensor([0, 1, 4, 5], device="cuda")
    check(x[rows], torch.zeros_like(x[rows]), gamma, scales, h[rows], y.float()[rows].to(y.dtype), None if s is None else s[rows])
    assert y[2].float().isnan().all()
    if scales == "row":
        assert s[2].isnan() and s[3].isnan() and y[3].float().isnan().all()
        assert abs(float(s[1]) * 448 / 2.0 ** -100 - 1) < 1e-6 and not y[1].float().any()
    elif scales == "group":
        assert s[2].isnan().all() and s[3, 0].isnan() and s[3, 1:].isfinite().all() and not y[3, 128:].float().any()
    else:
        assert y[3, 5].isnan() and not y[3, 6:].any()


@pytest.mark.parametrize("width", [256, 1024, 4096])
@pytest.mark.parametrize("scales", [None, "row", "group"])
def test_rmsnorm_small_rows_without_eps(width, scales):
    """Rows of about 1e-12 and no eps: 1 / rms is 1e12, and the reciprocal of the least scale 448 * 2^100.  Channels
    that are zero (a group of them, or by gamma) stay zero."""
    x, _, gamma = draw(3, width, seed=9)
    x = (x.float() * 1e-12).to(x.dtype)
    x[1, 128:256] = 0
    _, want = ref.rmsnorm(x, None, gamma, 0.0)
    _, y, s = h3a.residual_rmsnorm(x, None, gamma, 0.0, scales=scales)
    got = y.double()
    if scales:
        got = got * (s[:, None] if scales == "row" else s.repeat_interleave(128, 1)).double()
    amax = want.abs().view(3, -1, width if scales == "row" else 128).amax(2, keepdim=True).expand(-1, -1, width if scales == "row" else 128)
    half = 2.0 ** -4 if scales else ref.half_step(x.dtype)
    # e4m3: half a step relative, and half a step of its subnormals, 2^-10 scales of amax / 448
    ref.within(got, want, want.abs() * (half + 8 * ref.RMSNORM_RELATIVE) + (amax.reshape(want.shape) / 448 * 2.0 ** -10 * 1.01 if scales else 0), "small")
    assert not y[1, 128:256].float().any()
    _, y, s = h3a.residual_rmsnorm(x, None, torch.zeros_like(gamma), 0.0, scales=scales)
    assert not y.float().any() and (s is None or torch.equal(s, torch.full_like(s, 2.0 ** -100 / 448)))


def test_rmsnorm_is_deterministic_and_row_wise():
    """A row's result does not depend on its place or on the rows around it."""
    x, f, gamma = draw(3000, 512, seed=6)
    _, y, s = h3a.residual_rmsnorm(x, f, gamma, EPS, scales="row")
    for r in (0, 1, 1777, 2999):
        _, y1, s1 = h3a.residual_rmsnorm(x[r:r + 1], f[r:r + 1], gamma, EPS, scales="row")
        assert torch.equal(y1.float(), y[r:r + 1].float()) and torch.equal(s1, s[r:r + 1])


def test_rmsnorm_empty_and_refusals():
    x, f, gamma = draw(4, 64)
    h, y, s = h3a.residual_rmsnorm(x[:0], f[:0], gamma, scales="group")
    assert h.shape == (0, 64) and y.shape == (0, 64) and s.shape == (0, 1)
    with pytest.raises(ValueError, match="scales"):
        h3a.residual_rmsnorm(x, f, gamma, scales="tensor")
    with pytest.raises(ValueError, match="f must match"):
        h3a.residual_rmsnorm(x, f[:2], gamma)
    with pytest.raises(ValueError, match="gamma"):
        h3a.residual_rmsnorm(x, f, gamma.half())
    z = torch.zeros(2, 16392, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(h3a.H3AError, match="UNSUPPORTED"):
        h3a.residual_rmsnorm(z, None, torch.ones(16392, device="cuda"))
    with pytest.raises(h3a.H3AError, match="INVALID_ARG"):
        h3a.residual_rmsnorm(x[:, :60].contiguous(), None, gamma[:60].contiguous())


def test_rmsnorm_refuses_widths_past_32_bits():
    x = torch.empty(1, 2 ** 31 + 8, device="cuda", dtype=torch.bfloat16)  # 4.3 GB, not touched
    with pytest.raises(ValueError, match="2\\^31"):
        h3a.residual_rmsnorm(x, None, torch.ones(8, device="cuda"))
