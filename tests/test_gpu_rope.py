"""gtq_rope against the formula in fp64: both pairings, part of the head, every scaling, the gradient, strides,
positions from a row, a table or a start, in place and beside."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import decode_attention_13_b200 as gtq  # noqa: E402

pytestmark = pytest.mark.gpu

# Per output: the angle in half turns is rounded to fp32 (2^-25, i.e. pi 2^-25 of angle), sincospif is within 2 ulp
# (2^-23), the magnitude, two products and a sum round once each (4 x 2^-24): under 2^-21 (|x0| + |x1|) |m| together.
# An fp16 result adds half a step, 2^-11 of itself (2^-25 among the subnormals).
ARITH = 2.0 ** -21


def frequencies(r, theta, scaling, factor, context, low, high):
    out = []
    for i in range(r // 2):
        f = theta ** (-2.0 * i / r)
        if scaling == gtq.ROPE_LINEAR:
            f /= factor
        elif scaling == gtq.ROPE_LLAMA3:
            s = min(1.0, max(0.0, (context * f / (2 * math.pi) - low) / (high - low)))
            f = (1 - s) * f / factor + s * f
        elif scaling == gtq.ROPE_YARN:
            c = [r * math.log(context / (2 * math.pi * n)) / (2 * math.log(theta)) for n in (high, low)]
            lo, hi = max(math.floor(c[0]), 0), min(math.ceil(c[1]), r - 1)
            s = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = s * f / factor + (1 - s) * f
        out.append(f)
    return np.array(out)


def reference(x, pos, freq, r, half, magnitude, backward):
    """(y, |x0| + |x1| per element) in fp64; x [B, H, T, d], pos [B, T]."""
    x = x.astype(np.float64)
    a = pos.astype(np.float64)[:, None, :, None] * freq
    c, s = np.cos(a) * magnitude, np.sin(a) * magnitude * (-1 if backward else 1)
    i = np.arange(r // 2)
    i0, i1 = (i, i + r // 2) if half else (2 * i, 2 * i + 1)
    y, size = x.copy(), np.zeros_like(x)
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    size[..., i0] = size[..., i1] = (np.abs(x[..., i0]) + np.abs(x[..., i1])) * abs(magnitude)
    return y, size


def check(got, ref, size, dtype):
    got = got.double().cpu().numpy()
    tol = ARITH * size + (2.0 ** -11 * np.abs(ref) + 2.0 ** -24 if dtype == torch.float16 else 0.0)
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) - tol)


CASES = [
    # B, Hq, Hkv, T, d, rot, half, fp16, scaling, theta, factor, context, magnitude, backward
    (1, 1, 1, 1, 128, 128, True, True, gtq.ROPE_PLAIN, 1e4, 1.0, 0.0, 1.0, False),
    (2, 8, 2, 37, 128, 128, True, True, gtq.ROPE_LLAMA3, 5e5, 8.0, 8192.0, 1.0, False),
    (3, 4, 1, 65, 128, 64, False, False, gtq.ROPE_YARN, 1e6, 4.0, 32768.0, 1.14, True),
    (1, 3, 3, 1100, 64, 32, True, False, gtq.ROPE_LINEAR, 1e4, 4.0, 0.0, 1.0, False),
    (2, 2, 1, 600, 96, 80, False, True, gtq.ROPE_YARN, 1e4, 16.0, 4096.0, 0.5, False),
    (1, 5, 2, 9, 6, 2, True, True, gtq.ROPE_PLAIN, 1e4, 1.0, 0.0, 1.0, True),
    (1, 2, 2, 7, 256, 256, False, False, gtq.ROPE_LLAMA3, 1e4, 2.0, 1024.0, 1.0, True),
    (1, 1, 1, 5, 2, 2, False, True, gtq.ROPE_PLAIN, 1e4, 1.0, 0.0, 1.0, False),
]


@pytest.mark.parametrize("case", CASES)
def test_against_the_formula(case):
    B, hq, hkv, T, d, r, half, fp16, scaling, theta, factor, context, magnitude, backward = case
    rng = np.random.default_rng(T + d)
    dt = torch.float16 if fp16 else torch.float32
    cfg = gtq.make_rope(d, theta, rotary_dim=r, rope_pairing=0 if half else 1, dtype=0 if fp16 else 1, scaling=scaling,
                        factor=factor, original_context=context, low_freq=1.0, high_freq=4.0, magnitude=magnitude,
                        backward=backward)
    freq = frequencies(r, theta, scaling, factor, context, 1.0, 4.0)
    pos = rng.integers(0, 600000, (B, T))
    x = {n: torch.from_numpy(rng.standard_normal((B, T, h, d)).astype(np.float32)).to(dt).cuda().transpose(1, 2)
         for n, h in (("q", hq), ("k", hkv))}
    y = {n: torch.full((B, t.shape[1], T, d), float("nan"), dtype=dt, device="cuda") for n, t in x.items()}
    gtq.gtq_rope(cfg, x["q"], y["q"], x["k"], y["k"], positions=torch.from_numpy(pos).cuda())
    for n in "qk":
        ref, size = reference(x[n].float().cpu().numpy(), pos, freq, r, half, magnitude, backward)
        check(y[n], ref, size, dt)
        if r < d:
            assert torch.equal(y[n][..., r:], x[n][..., r:])
    # k alone, in place, at a run of positions from a start: the same values
    k = x["k"].clone()
    ref, size = reference(k.float().cpu().numpy(), np.arange(T)[None, :] + 12345 + np.zeros((B, 1)), freq, r, half,
                          magnitude, backward)
    gtq.gtq_rope(cfg, k=k, pos0=12345)
    check(k, ref, size, dt)


@pytest.mark.parametrize("pos", [0, 1, 131071, 524287, 2 ** 31, 2 ** 40 + 7])
def test_far_positions_keep_their_angle(pos):
    # the angle is formed from pos f / (2 pi) in fp64; against exact arithmetic the oracle's own fp64 angle is off by
    # pos f 2^-53, the kernel's by as much again
    cfg = gtq.make_rope(128, 1e4, dtype=gtq.DTYPE_FP32)
    x = torch.randn((1, 2, 1, 128), generator=torch.Generator().manual_seed(3)).cuda()
    y = torch.empty_like(x)
    gtq.gtq_rope(cfg, x, y, pos0=pos)
    freq = frequencies(128, 1e4, gtq.ROPE_PLAIN, 1, 0, 1, 4)
    ref, size = reference(x.cpu().numpy(), np.array([[pos]]), freq, 128, True, 1.0, False)
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= (ARITH + 4 * pos * 2.0 ** -53) * size)


@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (0, 3), (3, 5), (4, 4)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_any_alignment_and_stride(offset, pad, dtype):
    B, H, T, d = 2, 3, 20, 128
    g = torch.Generator().manual_seed(offset * 10 + pad)
    flat = torch.randn((B * T * H * (d + pad) + offset,), generator=g).to(dtype).cuda()
    x = flat[offset:].view(B, T, H, d + pad)[..., :d].transpose(1, 2)
    out = torch.full_like(flat, 7.0)
    y = out[offset:].view(B, T, H, d + pad)[..., :d].transpose(1, 2)
    cfg = gtq.make_rope(d, 1e4, dtype=0 if dtype == torch.float16 else 1, rope_pairing=pad % 2)
    gtq.gtq_rope(cfg, x, y)
    pos = np.arange(T)[None, :] + np.zeros((B, 1))
    ref, size = reference(x.float().cpu().numpy(), pos, frequencies(d, 1e4, 0, 1, 0, 1, 4), d, pad % 2 == 0, 1.0, False)
    check(y, ref, size, dtype)
    if pad:  # what lies between the rows is left alone
        assert bool((out[offset:].view(B, T, H, d + pad)[..., d:] == 7.0).all())


def test_gradient_is_the_transposed_turn():
    # <R x, g> = <x, R^T g>, and R^T by differences: R is linear, so differences of R along unit vectors are exact
    d, r = 16, 12
    kw = dict(rotary_dim=r, rope_pairing=1, dtype=gtq.DTYPE_FP32, magnitude=1.25)
    fwd, bwd = gtq.make_rope(d, 1e4, **kw), gtq.make_rope(d, 1e4, backward=True, **kw)
    eye = torch.eye(d, device="cuda").view(1, d, 1, d).contiguous()
    R = torch.empty_like(eye)
    gtq.gtq_rope(fwd, eye, R, pos0=911)
    Rt = torch.empty_like(eye)
    gtq.gtq_rope(bwd, eye, Rt, pos0=911)
    # entries agree but for one rounding of each product: the same sine and cosine are used
    assert torch.allclose(R.view(d, d), Rt.view(d, d).T, rtol=2.0 ** -23, atol=0)


def test_one_row_of_positions_for_all_and_a_stride():
    x = torch.randn((3, 2, 5, 128), generator=torch.Generator().manual_seed(1)).cuda()
    cfg = gtq.make_rope(128, 1e4, dtype=gtq.DTYPE_FP32)
    row = torch.tensor([9, 1, 4, 4, 700], device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    gtq.gtq_rope(cfg, x, a, positions=row)
    gtq.gtq_rope(cfg, x, b, positions=row.expand(3, 5))
    assert torch.equal(a, b)
    wide = torch.zeros((3, 8), dtype=torch.int64, device="cuda")
    wide[:, :5] = row
    gtq.gtq_rope(cfg, x, b, positions=wide[:, :5])
    assert torch.equal(a, b)


def test_on_a_stream_and_in_a_graph():
    x = torch.randn((2, 4, 33, 128), generator=torch.Generator().manual_seed(2)).half().cuda()
    cfg = gtq.make_rope(128, 1e4)
    want = torch.empty_like(x)
    gtq.gtq_rope(cfg, x, want, pos0=50)
    torch.cuda.synchronize()
    pos = torch.arange(33, device="cuda") + 50
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = torch.empty_like(x)
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            gtq.gtq_rope(cfg, x, got, positions=pos, stream=s)
        g.replay()
    s.synchronize()
    assert torch.equal(got, want)
