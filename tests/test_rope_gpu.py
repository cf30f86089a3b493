"""Rotary positions against the fp64 rotation.

Tolerance: the angle is exact up to one fp32 rounding of a fraction of half a
turn (<= pi 2^-25 in the angle), sincospif is within 2 ulp, and a rotated
element is two products and a sum: |error| <= 8 * 2^-24 (|a| + |b|) amplitude,
plus half a step of the output's type."""
import math

import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def K():
    from eviction_kvc_score_gb300 import kvc
    return kvc


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def table_of(rot, theta=10000.0, **kw):
    t = torch.empty(rot // 2, dtype=torch.int64, device="cuda")
    K().kvc_rope_table(rot, theta, t, **kw)
    return t


def check(got, x, pos, freq, interleaved, inverse=False, amplitude=1.0):
    want = ref.rope(x, pos, freq, interleaved, inverse, amplitude)
    rot = 2 * freq.numel()
    pair = ref.rope(x.abs(), torch.zeros_like(pos), freq, interleaved)   # |x| laid out alike
    a, b = (pair[..., 0:rot:2], pair[..., 1:rot:2]) if interleaved else (pair[..., :rot // 2], pair[..., rot // 2:rot])
    s = a + b
    tol = torch.zeros_like(want)
    if interleaved:
        tol[..., 0:rot:2] = tol[..., 1:rot:2] = s
    else:
        tol[..., :rot // 2] = tol[..., rot // 2:rot] = s
    tol = tol * 8 * 2.0 ** -24 * abs(amplitude) + want.abs() * torch.finfo(x.dtype).eps / 2 * 1.001
    err = (got.double() - want).abs()
    assert (err <= tol).all(), (err - tol).max()
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk,dim,rot", [
    (1, 1, 1, 64, 64), (64, 32, 8, 128, 128), (3, 0, 2, 80, 40), (700, 5, 1, 256, 256), (5, 3, 3, 96, 2),
    (9, 2, 1, 34, 30), (33, 1, 0, 128, 64), (1300, 1, 1, 8, 6), (17, 4, 2, 2, 2)])
def test_matches_the_rotation(dtype, interleaved, n, hq, hk, dim, rot):
    kvc, g = K(), torch.Generator(device="cuda").manual_seed(n * 1000 + dim)
    q = torch.randn((n, hq, dim), generator=g, device="cuda").to(DT[dtype]) if hq else None
    k = torch.randn((n, hk, dim), generator=g, device="cuda").to(DT[dtype]) if hk else None
    pos = torch.randint(0, 131072, (n,), generator=g, device="cuda", dtype=torch.int32)
    outs = [None if x is None else torch.full_like(x, math.nan) for x in (q, k)]
    kvc.kvc_rope(table_of(rot), pos, q, k, *outs, rot, interleaved=interleaved)
    for x, y in zip((q, k), outs):
        if x is not None:
            check(y, x, pos, ref.rope_frequencies(rot, 10000.0), interleaved)


@pytest.mark.parametrize("kw", [dict(), dict(factor=8.0, alpha=1.0, beta=4.0, context=8192.0),
                                dict(factor=4.0, alpha=math.inf, beta=math.inf, context=4096.0),
                                dict(factor=2.5, alpha=3.0, beta=3.0, context=1000.0),
                                dict(factor=40.0, alpha=0.0, beta=32.0, context=4096.0)])
def test_frequencies(kw):
    for rot, theta in ((128, 500000.0), (2, 1.0), (256, 1e7), (50, 10000.0)):
        got = table_of(rot, theta, **kw).cpu()
        want = ref.rope_frequencies(rot, theta, **kw)
        turns = torch.tensor([int(x) % (1 << 64) / 2.0 ** 64 for x in got], dtype=torch.float64)
        # pow, a division and a product in fp64, and one rounding to 2^-64
        assert torch.allclose(turns * 2 * math.pi, want, rtol=2e-15, atol=2.0 ** -60)


def test_far_and_negative_positions_are_exact():
    """The angles of positions up to the int32 limits, against integers of any size."""
    kvc, rot = K(), 64
    table = table_of(rot)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 1 << 24, (1 << 24) + 1, -1, 0], dtype=torch.int32, device="cuda")
    x = torch.zeros((6, 1, rot), device="cuda")
    x[..., :rot // 2] = 1
    y = torch.empty_like(x)
    kvc.kvc_rope(table, pos, None, x, None, y, rot)
    for i, p in enumerate(pos.tolist()):
        for j, u in enumerate(table.tolist()):
            frac = (p * (u % (1 << 64))) % (1 << 64) / 2.0 ** 64
            want = (math.cos(2 * math.pi * frac), math.sin(2 * math.pi * frac))
            assert abs(y[i, 0, j].item() - want[0]) < 8 * 2.0 ** -24
            assert abs(y[i, 0, j + rot // 2].item() - want[1]) < 8 * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_inside_fused_rows(dtype):
    """Queries and keys of fused projection rows turned where they lie; the values beside them stay."""
    kvc = K()
    n, hq, hk, d = 37, 6, 2, 64
    x = torch.randn((n, (hq + 2 * hk) * d), device="cuda").to(DT[dtype])
    x0 = x.clone()
    q, k = x[:, :hq * d].view(n, hq, d), x[:, hq * d:(hq + hk) * d].view(n, hk, d)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 977
    kvc.kvc_rope(table_of(d), pos, q, k, q, k, d)
    f = ref.rope_frequencies(d, 10000.0)
    check(q, x0[:, :hq * d].view(n, hq, d), pos, f, False)
    check(k, x0[:, hq * d:(hq + hk) * d].view(n, hk, d), pos, f, False)
    assert torch.equal(x[:, (hq + hk) * d:], x0[:, (hq + hk) * d:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_unaligned_views_and_odd_strides(interleaved):
    """Rows that start off a 16-byte boundary take the one-element path."""
    kvc, n, h, d = K(), 21, 3, 32
    buf = torch.randn(n * (h * d + 3) + 1, device="cuda").to(torch.bfloat16)
    x = buf[1:].as_strided((n, h, d), (h * d + 3, d, 1))
    y = torch.empty((n, h, d), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    kvc.kvc_rope(table_of(d), pos, None, x, None, y, d, interleaved=interleaved)
    check(y, x.contiguous(), pos, ref.rope_frequencies(d, 10000.0), interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    """The inverse of a gradient equals autograd's through the fp64 formula and
    central differences of the kernel's own outputs; with an amplitude."""
    kvc, n, h, d, rot, amp = K(), 5, 2, 16, 12, 1.25
    table, freq = table_of(rot), ref.rope_frequencies(rot, 10000.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((n, h, d), generator=g, device="cuda")
    dy = torch.randn((n, h, d), generator=g, device="cuda")
    pos = torch.tensor([0, 1, 7, 1000, 123456], dtype=torch.int32, device="cuda")
    dx = torch.empty_like(x)
    kvc.kvc_rope(table, pos, None, dy, None, dx, rot, interleaved=interleaved, inverse=True, amplitude=amp)
    leaf = x.double().requires_grad_()
    y = leaf.clone()
    a = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    b = a + 1 if interleaved else a + rot // 2
    ang = pos.double()[:, None, None] * freq.cuda()
    u = amp * (leaf[..., a] * torch.cos(ang) - leaf[..., b] * torch.sin(ang))
    w = amp * (leaf[..., a] * torch.sin(ang) + leaf[..., b] * torch.cos(ang))
    (u * dy[..., a].double() + w * dy[..., b].double()).sum().backward()
    want = leaf.grad
    want[..., rot:] = dy[..., rot:].double()
    assert (dx.double() - want).abs().max() <= 8 * 2.0 ** -24 * 2 * dy.abs().max().item() * amp
    # differences: the map is linear, so a step of 1/2 has no truncation error
    # and each loss carries the rounding of its n h d products
    def loss(z):
        o = torch.empty_like(z)
        kvc.kvc_rope(table, pos, None, z, None, o, rot, interleaved=interleaved, amplitude=amp)
        return (o.double() * dy.double()).sum().item()
    for t, hh, e in ((0, 0, 0), (2, 1, 5), (3, 0, 11), (4, 1, 15)):
        z = x.clone()
        z[t, hh, e] += 0.5
        hi = loss(z)
        z[t, hh, e] -= 1.0
        bound = n * h * d * 16 * 2.0 ** -24 * (x.abs().max().item() + 1) * amp * dy.abs().max().item()
        assert abs(hi - loss(z) - want[t, hh, e].item()) <= bound


def test_no_tokens_and_captured_replay():
    kvc, d = K(), 64
    table = table_of(d)
    e = torch.empty((0, 2, d), device="cuda")
    kvc.kvc_rope(table, torch.empty(0, dtype=torch.int32, device="cuda"), None, e, None, e, d)
    x = torch.randn((6, 2, d), device="cuda")
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        kvc.kvc_rope(table, pos, None, x, None, y, d)
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    check(y, x, pos, ref.rope_frequencies(d, 10000.0), False)
