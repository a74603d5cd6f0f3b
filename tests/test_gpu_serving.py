"""The serving operators (residual RMS norm, 8-bit linear, rotary positions with the cache
write, paged attention) against their definitions in 64 bits.

Tolerances are bounds of the arithmetic, stated at each comparison: HALF[t] is the largest
relative error of one rounding to t (half a step), U one fp32 rounding, and sums of n fp32
terms are off by at most n U times the sum of the magnitudes.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0**-24
HALF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
TINY = {torch.float32: 2.0**-149, torch.bfloat16: 2.0**-133, torch.float16: 2.0**-25}
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def rb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rotated_bit_matmul_b200 import build_lib
    build_lib.build()
    import rotated_bit_matmul_b200 as rb
    return rb


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def close(got, want, tol):
    """Every element within tol (a tensor or a number) of want."""
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {(off - tol).nan_to_num(math.inf).max().item():.3e} beyond the bound"


def clean(rb):
    torch.cuda.synchronize()
    rb.harp_device_status()


# ------------------------------------------------------------------ norm
def norm64(x, w, r, eps):
    h = x.double() + (0 if r is None else r.double())
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    return h, y if w is None else y * w.double()


# h: one rounding; sum of squares: at most 32 + 10 additions on a path, halved by the root; the
# root, its product with h and the weight's: three more
NORM_REL = 32 * U

NORM_SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 127), (4, 128), (2, 129), (7, 1000), (2, 1001), (9, 4100), (2, 8192),
               (3, 11008), (2, 16384), (1, 32768), (2, 32767), (700, 64), (301, 200)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", NORM_SHAPES)
def test_rmsnorm(rb, rows, n, dtype):
    g = gen(rows * 100003 + n)
    x, r, w = randn(g, rows, n, dtype=dtype), randn(g, rows, n, dtype=dtype) * 3, randn(g, n, dtype=dtype)
    y = rb.harp_rmsnorm(x)
    close(y, norm64(x, None, None, 1e-5)[1], norm64(x, None, None, 1e-5)[1].abs() * (HALF[dtype] + NORM_REL) + TINY[dtype])
    y, h = rb.harp_rmsnorm(x, weight=w, residual=r, eps=1e-3, out_dtype=torch.float32)
    h64, y64 = norm64(x, w, r, 1e-3)
    close(h, h64, h64.abs() * (HALF[dtype] + U) + TINY[dtype])
    close(y, y64, y64.abs() * NORM_REL + 2.0**-149)
    clean(rb)


def e4m3_ok(q, scale, y, rel):
    """q is y / scale to half a step of e4m3 (2^-4 of the value, 2^-10 below 2^-6)."""
    rows, n = y.shape
    blocks = -(-n // 128)
    amax = torch.nn.functional.pad(y, (0, blocks * 128 - n)).view(rows, blocks, 128).abs().amax(-1)
    want = torch.where(amax == 0, torch.ones_like(amax), amax / 448)
    close(scale, want, want * (rel + 2 * U))
    v = y / want.repeat_interleave(128, 1)[:, :n]
    close(q.float(), v, torch.maximum(v.abs() * 2.0**-4, torch.tensor(2.0**-10, device="cuda")) + v.abs() * 2 * rel)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", NORM_SHAPES)
def test_rmsnorm_q8(rb, rows, n, dtype):
    g = gen(rows * 7 + n)
    x, r, w = randn(g, rows, n, dtype=dtype), randn(g, rows, n, dtype=dtype), randn(g, n, dtype=dtype)
    x[:, ::97] *= 30
    q, s, h = rb.harp_rmsnorm_q8(x, weight=w, residual=r)
    h64, y64 = norm64(x, w, r, 1e-5)
    close(h, h64, h64.abs() * (HALF[dtype] + U) + TINY[dtype])
    e4m3_ok(q, s, y64, NORM_REL)
    assert q.shape == x.shape and s.shape == (rows, -(-n // 128))
    q, s = rb.harp_quantize_q8(x)
    e4m3_ok(q, s, x.double(), 0)
    clean(rb)


def test_rmsnorm_views_and_in_place(rb):
    """Strided rows (wide and odd), a 3-D input, the residual updated in place, a weight of
    another type, and y over x."""
    g = gen(5)
    wide = randn(g, 6, 1040, dtype=torch.bfloat16)
    for x in (wide[:, :1000], wide[:, 8:1008], wide[:, 3:1003], wide[::2, :777]):
        close(rb.harp_rmsnorm(x), norm64(x, None, None, 1e-5)[1], norm64(x, None, None, 1e-5)[1].abs() * (HALF[x.dtype] + NORM_REL))
    x = randn(g, 2, 3, 512, dtype=torch.bfloat16)
    res = randn(g, 2, 3, 512)
    w = randn(g, 512, dtype=torch.float16)
    h64, y64 = norm64(x, w, res, 1e-5)
    q, s, h = rb.harp_rmsnorm_q8(x, w, res, residual_out=res)
    assert h is res and q.shape == x.shape and s.shape == (2, 3, 4)
    close(res, h64, h64.abs() * 2 * U)
    e4m3_ok(q.reshape(6, 512), s.reshape(6, 4), y64.view(6, 512), NORM_REL)
    y64 = norm64(x, None, None, 1e-5)[1]
    rb.harp_rmsnorm(x, out=x)
    close(x, y64, y64.abs() * (HALF[x.dtype] + NORM_REL))
    clean(rb)


def test_rmsnorm_special_values(rb):
    """A zero row (eps 0 gives NaN, as 0 / 0), infinities, NaN, and rows that stay apart."""
    x = torch.zeros(5, 256, device="cuda")
    x[1, 3] = math.inf
    x[2, 200] = math.nan
    x[3] = 1e-30
    x[4] = 1e18
    q, s = rb.harp_rmsnorm_q8(x)
    assert (q[0].float() == 0).all() and (s[0] == 1).all()
    deq = q.float() * s.repeat_interleave(128, 1)
    assert deq[1, :128].isnan().all() and deq[2].isnan().all()
    assert (deq[1, 128:] == 0).all()
    y64 = norm64(x[3:], None, None, 1e-5)[1]
    e4m3_ok(q[3:], s[3:], y64, NORM_REL)
    assert rb.harp_rmsnorm(x[:1], eps=0.0).isnan().all()
    qq, ss = rb.harp_quantize_q8(x)
    assert ss[1, 0].isinf() and (ss[1, 1] == 1) and ss[2, 1].isnan()
    clean(rb)


@pytest.mark.parametrize("n_out,n_in", [(1, 1), (128, 128), (129, 127), (300, 1000), (64, 4096)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_weights_q8(rb, n_out, n_in, dtype):
    W = randn(gen(n_out + n_in), n_out, n_in, dtype=dtype)
    q, s = rb.harp_quantize_weights_q8(W)
    nb, kb = -(-n_out // 128), -(-n_in // 128)
    tiles = torch.nn.functional.pad(W.double(), (0, kb * 128 - n_in, 0, nb * 128 - n_out)).view(nb, 128, kb, 128)
    want = tiles.abs().amax((1, 3)) / 448
    close(s, want, want * 2 * U)
    v = W.double() / want.repeat_interleave(128, 0)[:n_out].repeat_interleave(128, 1)[:, :n_in]
    close(q.float(), v, torch.maximum(v.abs() * 2.0**-4, torch.tensor(2.0**-10, device="cuda")) + v.abs() * 4 * U)
    clean(rb)


# ------------------------------------------------------------------ 8-bit linear
def linear64(x, sx, w, sw):
    rep = lambda s, n: s.double().repeat_interleave(128, 1)[:, :n]  # noqa: E731
    n_out, n_in = w.shape
    X = x.float().double() * rep(sx, n_in)
    W = w.float().double() * rep(sw.repeat_interleave(128, 0)[:n_out], n_in)
    return X @ W.t(), X.abs() @ W.abs().t()


def linear_case(rb, tokens, n_in, n_out, seed=0):
    g = gen(seed + tokens * 31 + n_in * 7 + n_out)
    w, sw = rb.harp_quantize_weights_q8(randn(g, n_out, n_in))
    x, sx = rb.harp_quantize_q8(randn(g, tokens, n_in) * torch.exp(randn(g, tokens, 1)))
    return x, sx, w, sw


def linear_tol(y, mag, n_in, dtype):
    # products of e4m3 are exact; 128 of them added on the tensor core (a step of fp32 each, not
    # half: it may truncate), their scaled sums and the two scale products in fp32
    return y.abs() * HALF[dtype] + TINY[dtype] + mag * (2 * 128 + -(-n_in // 128) + 3) * U


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,n_in,n_out", [
    (1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 130, 129), (3, 1000, 515), (15, 4096, 1000), (16, 8192, 256),
    (17, 4096, 640), (19, 11008, 4096), (33, 513, 777), (64, 2048, 128), (65, 640, 300), (100, 4096, 4096), (128, 384, 1000),
    (129, 1024, 512), (257, 1000, 2000), (700, 2048, 1537), (2049, 512, 4096)])
def test_linear8(rb, tokens, n_in, n_out, dtype):
    x, sx, w, sw = linear_case(rb, tokens, n_in, n_out)
    layer = rb.HarpLinear8(w, sw)
    y = layer(x, sx, out_dtype=dtype)
    want, mag = linear64(x, sx, w, sw)
    clean(rb)
    close(y, want, linear_tol(want, mag, n_in, dtype))
    again = layer(x, sx, out_dtype=dtype)
    assert torch.equal(y, again)
    layer.close()


def test_linear8_layouts(rb):
    """Unaligned rows, row-major scales, 3-D inputs, a strided output whose gaps stay."""
    x, sx, w, sw = linear_case(rb, 20, 1001, 260)
    want, mag = linear64(x, sx, w, sw)
    tol = linear_tol(want, mag, 1001, torch.float32)
    layer = rb.HarpLinear8(w, sw)
    tight = torch.empty(20, 1001, dtype=torch.uint8, device="cuda").copy_(x.view(torch.uint8)).view(torch.float8_e4m3fn)
    close(layer(tight, sx.contiguous(), out_dtype=torch.float32), want, tol)
    y = layer(tight.view(4, 5, 1001), sx.contiguous().view(4, 5, -1), out_dtype=torch.float32)
    close(y.view(20, 260), want, tol)
    wide = torch.full((20, 300), 7.0, device="cuda")
    layer(x, sx, out=wide[:, :260])
    close(wide[:, :260], want, tol)
    assert (wide[:, 260:] == 7).all()
    wt = torch.empty(260, 1001, dtype=torch.uint8, device="cuda").copy_(w.view(torch.uint8)).view(torch.float8_e4m3fn)
    close(rb.HarpLinear8(wt, sw)(x, sx, out_dtype=torch.float32), want, tol)
    assert layer(x[:0], sx[:0]).shape == (0, 260)
    # scales whose last block row ends with the storage
    ld = 20
    flat = torch.empty(8 * ld, device="cuda")
    view = flat.as_strided((20, 8), (1, ld))
    view.copy_(sx)
    close(layer(x, view, out_dtype=torch.float32), want, tol)
    clean(rb)


def test_linear8_nan_stays_in_its_row_and_column(rb):
    x, sx, w, sw = linear_case(rb, 40, 512, 384)
    x = x.clone()
    x.view(torch.uint8)[7, 100] = 0x7F
    w.view(torch.uint8)[200, 3] = 0x7F
    y = rb.HarpLinear8(w, sw)(x, sx, out_dtype=torch.float32)
    nan = y.isnan()
    assert nan[7].all() and nan[:, 200].all()
    nan[7] = False
    nan[:, 200] = False
    assert not nan.any()
    clean(rb)


# ------------------------------------------------------------------ rotary positions
def rope64(x, pos, freq, rot, interleaved, amplitude=1.0, inverse=False):
    a = pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda") * (-1 if inverse else 1)
    c, s = a.cos()[:, None] * amplitude, a.sin()[:, None] * amplitude
    y = x.double().clone()
    i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    p, q = x.double()[..., i0], x.double()[..., i1]
    y[..., i0], y[..., i1] = p * c - q * s, p * s + q * c
    mag = x.double().abs().clone()
    mag[..., i0] = mag[..., i1] = (p.abs() + q.abs()) * abs(amplitude)
    mag[..., rot:] = 0
    return y, mag


def rope_tol(y, mag, dtype):
    # cos and sin: the reduced angle rounded (pi 2^-24), sincospi within 2 units, times amplitude:
    # under 8 U together; two products and a sum: 3 U
    return y.abs() * HALF[dtype] + TINY[dtype] + mag * 12 * U


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hd,rot", [(128, 128), (128, 64), (64, 64), (96, 32), (256, 256), (80, 80), (20, 6), (2, 2), (130, 34)])
def test_rope_apply(rb, hd, rot, interleaved):
    g = gen(hd * 1000 + rot)
    pos = torch.tensor([0, 1, 5, 4095, 131071, 10**6 + 7, 2**31 - 1], dtype=torch.int32, device="cuda")
    rope = rb.HarpRope(hd, rot, interleaved=interleaved, amplitude=1.25)
    for dtype in DTYPES:
        x = randn(g, 7, 5, hd, dtype=dtype)
        y = rope(x, pos)
        want, mag = rope64(x, pos, rope.frequencies, rot, interleaved, 1.25)
        close(y, want, rope_tol(want, mag, dtype))
        back = rope(x, pos, inverse=True, out_dtype=torch.float32)
        want, mag = rope64(x, pos, rope.frequencies, rot, interleaved, 1.25, inverse=True)
        close(back, want, rope_tol(want, mag, torch.float32))
    clean(rb)


def test_rope_inverse_is_the_gradient(rb):
    """<rope(x), g> = <x, rope^T(g)> for every x, so the inverse call is the gradient; and a
    central difference agrees with it."""
    g = gen(11)
    rope = rb.HarpRope(64, 32)
    pos = torch.tensor([3, 100, 70000], dtype=torch.int32, device="cuda")
    x, gy = randn(g, 3, 4, 64), randn(g, 3, 4, 64)
    gx = rope(gy, pos, inverse=True)
    loss = lambda t: (rope(t, pos).double() * gy.double()).sum().item()  # noqa: E731
    # 768 products, each off by its rounding and the rotation's 12 U: under 16 U of the magnitudes
    lhs, rhs = loss(x), (x.double() * gx.double()).sum().item()
    mag = (x.double().norm() * gy.double().norm() * math.sqrt(2)).item()
    assert abs(lhs - rhs) <= 32 * U * mag * math.sqrt(768)
    for at in ((0, 0, 0), (1, 2, 17), (2, 3, 31), (2, 1, 50)):
        d = torch.zeros_like(x)
        d[at] = 0.5  # the call is linear: the difference has no truncation error
        diff = loss(x + d) - loss(x - d)
        assert abs(diff - gx[at].item()) <= 64 * U * mag


def test_rope_in_place_views_and_skipped_rows(rb):
    g = gen(13)
    rope = rb.HarpRope(128)
    pos = torch.tensor([4, -1, 9, -7], dtype=torch.int32, device="cuda")
    qkv = randn(g, 4, 12, 128, dtype=torch.bfloat16)
    before = qkv.clone()
    view = qkv[:, 2:10]
    want, mag = rope64(before[:, 2:10], pos, rope.frequencies, 128, False)
    rope(view, pos, out=view)
    live = [0, 2]
    close(qkv[live, 2:10], want[live], rope_tol(want, mag, torch.bfloat16)[live])
    assert torch.equal(qkv[[1, 3]], before[[1, 3]])
    assert torch.equal(qkv[:, :2], before[:, :2]) and torch.equal(qkv[:, 10:], before[:, 10:])
    odd = randn(g, 4, 3, 131, dtype=torch.bfloat16)[..., 1:129]  # rows at odd addresses
    want, mag = rope64(odd, pos.abs(), rope.frequencies, 128, False)
    close(rope(odd, pos.abs()), want, rope_tol(want, mag, torch.bfloat16))
    assert rope(qkv[:0], pos[:0]).shape == (0, 12, 128)
    clean(rb)


def make_cache(rb, n_pages, kv, page, hd, dtype, g, layout="heads"):
    if layout == "heads":
        k, v = randn(g, n_pages, kv, page, hd, dtype=dtype), randn(g, n_pages, kv, page, hd, dtype=dtype)
    else:  # [pages, rows, heads, dim] in memory
        k, v = (randn(g, n_pages, page, kv, hd, dtype=dtype).transpose(1, 2) for _ in range(2))
    return rb.HarpCache(k, v)


@pytest.mark.parametrize("dtype,cdtype", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16)])
@pytest.mark.parametrize("hd,rot,heads,kv,page,layout", [
    (128, 128, 64, 8, 16, "heads"), (64, 32, 4, 4, 1, "heads"), (96, 96, 6, 2, 32, "rows"), (32, 8, 3, 1, 8, "heads"),
    (40, 20, 2, 2, 4, "rows")])
def test_rope_append(rb, hd, rot, heads, kv, page, layout, dtype, cdtype):
    g = gen(hd + heads + page)
    cache = make_cache(rb, 40, kv, page, hd, cdtype, g, layout)
    k0, v0 = cache.k.clone(), cache.v.clone()
    rope = rb.HarpRope(hd, rot, interleaved=True, scaling="linear", factor=4.0)
    table = torch.randperm(40, generator=g, device="cuda")[:36].view(3, 12).to(torch.int32)
    # positions of three sequences, out of order, with skipped rows
    seq = torch.tensor([0, 2, 1, 1, 0, 2, 2], dtype=torch.int32, device="cuda")
    last = 12 * page - 1
    pos = torch.tensor([0, last, min(3, last), last // 2, -1, min(page, last - 1), last // 3], dtype=torch.int32, device="cuda")
    qkv = randn(g, 7, heads + 2 * kv, hd, dtype=dtype)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    out = torch.full((7, heads, hd), 9.0, dtype=cdtype, device="cuda")
    got = rope.append(cache, q, k, v, pos, table, seq_ids=seq, out=out)
    live = pos >= 0
    want, mag = rope64(q, pos, rope.frequencies, rot, True)
    close(got[live], want[live], rope_tol(want, mag, cdtype)[live])
    assert (got[~live] == 9).all()
    kw, kmag = rope64(k, pos, rope.frequencies, rot, True)
    tol = rope_tol(kw, kmag, cdtype)
    touched = torch.zeros(k0.shape[0], k0.shape[2], dtype=torch.bool, device="cuda")
    for t in range(7):
        if pos[t] < 0:
            continue
        p, r = table[seq[t], pos[t] // page].item(), (pos[t] % page).item()
        close(cache.k[p, :, r], kw[t], tol[t])
        assert torch.equal(cache.v[p, :, r], v[t].to(cdtype))
        touched[p, r] = True
    rest = ~touched[:, None, :, None].expand_as(k0)
    assert torch.equal(cache.k[rest], k0[rest]) and torch.equal(cache.v[rest], v0[rest])
    clean(rb)


def test_rope_append_reports_bad_places(rb):
    """Sequences and pages out of range write nothing and are reported; other rows are served."""
    g = gen(17)
    cache = make_cache(rb, 6, 2, 8, 64, torch.bfloat16, g)
    k0 = cache.k.clone()
    rope = rb.HarpRope(64)
    table = torch.tensor([[0, 6], [-3, 2]], dtype=torch.int32, device="cuda")
    q, k, v = (randn(g, 5, h, 64, dtype=torch.bfloat16) for h in (4, 2, 2))
    seq = torch.tensor([0, 0, 1, 2, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([1, 9, 0, 0, 16], dtype=torch.int32, device="cuda")  # good, page 6, page -3, sequence 2, past the table
    rope.append(cache, q, k, v, pos, table, seq_ids=seq)
    torch.cuda.synchronize()
    with pytest.raises(rb.HarpError) as e:
        rb.harp_device_status()
    assert e.value.status == 6
    rest = torch.ones_like(k0, dtype=torch.bool)
    rest[0, :, 1] = False
    assert torch.equal(cache.k[rest], k0[rest]) and not torch.equal(cache.k[0, :, 1], k0[0, :, 1])
    assert torch.equal(cache.v[0, :, 1], v[0])
    clean(rb)


def test_rope_frequencies(rb):
    """The scalings against their formulas, evaluated here pair by pair."""
    rot, base, f, orig, low, high = 64, 500.0, 8.0, 2048.0, 1.0, 4.0
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]

    def close_list(a, b):
        assert len(a) == len(b) and all(abs(x - y) <= 1e-13 * abs(y) for x, y in zip(a, b))

    close_list(rb.HarpRope(64, base=base).frequencies, plain)
    close_list(rb.HarpRope(64, base=base, scaling="linear", factor=f).frequencies, [x / f for x in plain])
    nb = base * f ** (rot / (rot - 2))
    close_list(rb.HarpRope(64, base=base, scaling="ntk", factor=f).frequencies, [nb ** (-2 * i / rot) for i in range(rot // 2)])
    bands = []
    for x in plain:
        wavelength = 2 * math.pi / x
        if wavelength < orig / high:
            bands.append(x)
        elif wavelength > orig / low:
            bands.append(x / f)
        else:
            s = (orig / wavelength - low) / (high - low)
            bands.append((1 - s) * x / f + s * x)
    got = rb.HarpRope(64, base=base, scaling="bands", factor=f, original=orig, low=low, high=high).frequencies
    assert all(abs(x - y) <= 1e-12 * y for x, y in zip(got, bands))
    index = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
    ramp = []
    for i, x in enumerate(plain):
        t = min(1.0, max(0.0, (i - lo) / (hi - lo)))
        ramp.append(x / f * t + x * (1 - t))
    got = rb.HarpRope(64, base=base, scaling="ramp", factor=f, original=orig, low=low, high=high).frequencies
    assert all(abs(x - y) <= 1e-12 * y for x, y in zip(got, ramp))


# ------------------------------------------------------------------ paged attention
def attention64(q, cache, table, lens, scale, window=0):
    """Definition, sequence by sequence; also the sums of p |v| and the largest |q| . |k| scale."""
    n, heads, hd = q.shape
    kv, page = cache.n_kv_heads, cache.page_size
    out, lse = torch.zeros(n, heads, hd, dtype=torch.float64, device="cuda"), torch.full((n, heads), -math.inf, dtype=torch.float64, device="cuda")
    mag, reach = torch.zeros_like(out), torch.zeros_like(lse)
    for s, length in enumerate(lens):
        length = min(length, table.shape[1] * page)
        if length <= 0:
            continue
        at = table[s, : -(-length // page)].long()
        first = max(0, length - window) if window else 0
        k, v = (t[at].transpose(0, 1).reshape(kv, -1, hd)[:, first:length].double().repeat_interleave(heads // kv, 0) for t in (cache.k, cache.v))
        sc = torch.einsum("hd,hnd->hn", q[s].double(), k) * scale
        p = torch.softmax(sc, -1)
        out[s], mag[s] = torch.einsum("hn,hnd->hd", p, v), torch.einsum("hn,hnd->hd", p, v.abs())
        lse[s] = torch.logsumexp(sc, -1)
        reach[s] = (torch.einsum("hd,hnd->hn", q[s].double().abs(), k.abs()) * abs(scale)).amax(-1)
    return out, lse, mag, reach


def attention_tol(out, lse, mag, reach, hd, dtype, longest):
    # a score is off by hd U of its magnitude (and the products with the scale and log2 e), a
    # probability by twice that, exp2 and its rescalings (8 U), and the split into two halves of the
    # cache's type: half a step squared of its value, and for f16 half of the smallest step
    # absolutely (2^-25); sums over the keys: one step per 16 keys of a share and one per join
    score = reach * (hd + 4) * U
    n = longest / 64 + 400
    p = 2 * score + (8 + n) * U + HALF[dtype] ** 2
    return (out.abs() * HALF[dtype] + TINY[dtype] + mag * p[..., None] + (2.0**-25 * longest if dtype == torch.float16 else 0) * mag.amax(),
            score + (8 + n) * U + lse.nan_to_num(0, 0, 0).abs() * 2 * U)


def attention_case(rb, lens, heads, kv, hd, page, dtype, layout="heads", seed=0, spare=3, poison=True):
    g = gen(seed + heads * 17 + hd + page + len(lens))
    per = max(1, max(-(-x // page) for x in lens)) if lens else 1
    total = len(lens) * per + spare
    cache = make_cache(rb, total, kv, page, hd, dtype, g, layout)
    table = torch.randperm(total, generator=g, device="cuda")[: len(lens) * per].view(len(lens), per).to(torch.int32)
    if poison:  # NaN in every row that no sequence owns: behind each sequence's end, and in unused pages
        owned = torch.zeros(total, page, dtype=torch.bool, device="cuda")
        for s, x in enumerate(lens):
            j = torch.arange(max(x, 0), device="cuda")
            owned[table[s, j // page].long(), j % page] = True
        dead = ~owned[:, None, :, None].expand_as(cache.k)
        cache.k[dead] = math.nan
        cache.v[dead] = math.nan
    q = randn(g, len(lens), heads, hd, dtype=dtype)
    return q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


CASES = [
    # lens, heads, kv, head_dim, page, layout, window
    ([1], 1, 1, 64, 16, "heads", 0),
    ([500], 32, 32, 128, 16, "heads", 0),
    ([0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0], 8, 2, 128, 16, "heads", 0),
    ([1000, 3, 0, 777, 64], 12, 4, 64, 32, "rows", 0),
    ([2049, 5], 40, 2, 96, 8, "heads", 0),           # 20 heads to a key head: two blocks
    ([300, 301, 302], 71, 1, 64, 1, "heads", 0),     # one key head, pages of one row
    ([257] * 5, 16, 16, 32, 64, "rows", 0),
    ([513, 100], 8, 4, 192, 16, "heads", 0),
    ([513, 100, 0], 34, 2, 256, 16, "heads", 0),
    ([20000, 1, 3000], 64, 8, 128, 64, "heads", 0),
    ([131072], 8, 1, 64, 256, "heads", 0),
    ([0, 0, 0], 4, 2, 64, 16, "heads", 0),
    ([1000, 100, 64, 65, 1], 8, 8, 128, 16, "heads", 64),
    ([5000, 129, 4097], 16, 2, 64, 32, "rows", 1),
    ([5000, 700, 0, 33], 6, 2, 128, 32, "heads", 333),
    (list(range(300)), 4, 2, 64, 16, "heads", 0),    # more sequences than threads of a CTA
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_paged_attention(rb, case, dtype):
    lens, heads, kv, hd, page, layout, window = CASES[case]
    q, cache, table, n = attention_case(rb, lens, heads, kv, hd, page, dtype, layout)
    for scale in (None, 0.3):
        out, lse = rb.harp_paged_attention(q, cache, table, n, scale=scale, window=window, return_lse=True)
        clean(rb)
        want, wlse, mag, reach = attention64(q, cache, table, lens, hd**-0.5 if scale is None else scale, window)
        tol, ltol = attention_tol(want, wlse, mag, reach, hd, dtype, max(lens))
        empty = torch.tensor([x == 0 for x in lens], device="cuda")
        assert (out[empty] == 0).all() and (lse[empty] == -math.inf).all()
        close(out, want, tol)
        close(lse[~empty], wlse[~empty], ltol[~empty])
        again, _ = rb.harp_paged_attention(q, cache, table, n, scale=scale, window=window, return_lse=True)
        assert torch.equal(out, again)  # joined in key order: repeatable


def test_paged_attention_negative_lengths_and_views(rb):
    """Rows of negative length stay as they were; q and out as strided views."""
    q, cache, table, n = attention_case(rb, [100, 50, 70], 4, 2, 64, 16, torch.bfloat16)
    wide = torch.zeros(3, 10, 64, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:7] = q
    n[1] = -1
    out = torch.full((3, 6, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    rb.harp_paged_attention(wide[:, 3:7], cache, table, n, out=out[:, 1:5])
    clean(rb)
    want, wlse, mag, reach = attention64(q, cache, table, [100, 0, 70], 64**-0.5)
    tol, _ = attention_tol(want, wlse, mag, reach, 64, torch.bfloat16, 100)
    live = [0, 2]
    close(out[live, 1:5], want[live], tol[live])
    assert (out[1] == 5).all() and (out[:, 0] == 5).all() and (out[:, 5] == 5).all()


def test_paged_attention_large_scores(rb):
    """Scores of thousands (a one-hot softmax), a live -inf key and a +inf score as the formula has them."""
    q, cache, table, n = attention_case(rb, [200, 90, 90, 90], 2, 2, 64, 16, torch.bfloat16)
    q[0] *= 100
    want, wlse, mag, reach = attention64(q, cache, table, [200, 90, 90, 90], 1.0)
    out = rb.harp_paged_attention(q, cache, table, n, scale=1.0)
    tol, _ = attention_tol(want, wlse, mag, reach, 64, torch.bfloat16, 200)
    close(out, want, tol)
    q[1:] = q[1:].abs()
    cache.k[table[1, 0].long(), :, 0] = -math.inf   # score -inf: weight 0
    cache.k[table[2, 0].long(), :, 0] = math.inf    # score inf: NaN
    want, wlse, mag, reach = attention64(q, cache, table, [200, 90, 90, 90], 1.0)
    out = rb.harp_paged_attention(q, cache, table, n, scale=1.0)
    assert out[2].isnan().all() and not out[[0, 1, 3]].isnan().any()
    off = (out[1].double() - want[1]).abs()
    assert (off <= want[1].abs() * HALF[torch.bfloat16] + mag[1] * 2.0**-10).all()
    clean(rb)


def test_paged_attention_reports_bad_pages_and_lengths(rb):
    q, cache, table, n = attention_case(rb, [40, 40], 4, 2, 64, 16, torch.bfloat16, poison=False)
    table[0, 1] = cache.n_pages
    out = rb.harp_paged_attention(q, cache, table, n)
    torch.cuda.synchronize()
    with pytest.raises(rb.HarpError) as e:
        rb.harp_device_status()
    assert e.value.status == 6
    want, wlse, mag, reach = attention64(q[1:], cache, table[1:], [40], 64**-0.5)
    tol, _ = attention_tol(want, wlse, mag, reach, 64, torch.bfloat16, 40)
    close(out[1:], want, tol)
    table[0, 1] = 0
    n[0] = 1000  # cut to the table's 48
    out = rb.harp_paged_attention(q, cache, table, n)
    torch.cuda.synchronize()
    with pytest.raises(rb.HarpError):
        rb.harp_device_status()
    want, wlse, mag, reach = attention64(q, cache, table, [48, 40], 64**-0.5)
    tol, _ = attention_tol(want, wlse, mag, reach, 64, torch.bfloat16, 48)
    close(out, want, tol)
    clean(rb)


def test_paged_attention_offsets_past_32_bits(rb):
    """Pages beyond 2^32 elements of the cache (k and v 9 GB each) hold and give what the first
    pages of a small cache do."""
    g = gen(23)
    hd, page, kv = 128, 64, 8
    n_pages = (2**32) // (kv * page * hd) + 8
    big = rb.HarpCache(*(torch.empty(n_pages, kv, page, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    small = rb.HarpCache(*(torch.empty(3, kv, page, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    far = torch.tensor([[n_pages - 1, 1, n_pages - 3]], dtype=torch.int32, device="cuda")
    near = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    rope = rb.HarpRope(hd)
    pos = torch.arange(150, dtype=torch.int32, device="cuda")
    ids = torch.zeros_like(pos)
    k, v = randn(g, 150, kv, hd, dtype=torch.bfloat16), randn(g, 150, kv, hd, dtype=torch.bfloat16)
    n = torch.tensor([150], dtype=torch.int32, device="cuda")
    out = []
    for cache, table in ((big, far), (small, near)):
        q = rope.append(cache, k, k, v, pos, table, seq_ids=ids)
        at = table[0].long()
        assert torch.equal(cache.v[at].transpose(1, 2).reshape(-1, kv, hd)[:150], v)
        out.append((rb.harp_paged_attention(q[149:], cache, table, n), cache.k[at].transpose(1, 2).reshape(-1, kv, hd)[:150]))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    clean(rb)


# ------------------------------------------------------------------ together
def test_graph_replay_follows_lengths_and_streams(rb):
    """rope.append, attention, norm and the 8-bit linear captured once: replays follow new
    positions, lengths and inputs, and equal eager calls bit for bit; two graphs and an eager
    call on another stream run side by side."""
    g = gen(29)
    hd, heads, kv, page = 64, 8, 2, 16
    cache = make_cache(rb, 40, kv, page, hd, torch.bfloat16, g)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    rope = rb.HarpRope(hd)
    w, sw = rb.harp_quantize_weights_q8(randn(g, 300, heads * hd))
    layer = rb.HarpLinear8(w, sw)
    qkv = randn(g, 2, heads + 2 * kv, hd, dtype=torch.bfloat16)
    pos = torch.tensor([100, 250], dtype=torch.int32, device="cuda")
    lens = pos + 1

    def step():
        q = rope.append(cache, qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:], pos, table)
        o = rb.harp_paged_attention(q, cache, table, lens)
        return layer(*rb.harp_rmsnorm_q8(o.view(2, heads * hd)), out_dtype=torch.float32)

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    side = torch.cuda.Stream()
    for i in range(3):
        qkv.copy_(randn(g, 2, heads + 2 * kv, hd, dtype=torch.bfloat16))
        pos += 5
        lens += 5
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = step()
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], want)
    with torch.cuda.stream(side):
        graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    clean(rb)


def test_back_to_back_calls_wait_for_each_other(rb):
    """Chains whose every call reads what the one before wrote, with kernels that start before
    their predecessors have ended: without a wait between the calls the results are those of the
    same chain with one."""
    g = gen(31)
    hd, heads, kv, page, seqs = 128, 8, 2, 16, 3
    width = heads * hd
    table = torch.arange(seqs * 8, dtype=torch.int32, device="cuda").view(seqs, 8)
    rope = rb.HarpRope(hd)
    layers = [rb.HarpLinear8(*rb.harp_quantize_weights_q8(randn(g, width, width) / 20)) for _ in range(2)]
    weight = 1 + 0.1 * randn(g, width, dtype=torch.bfloat16)
    start = randn(g, seqs, width, dtype=torch.bfloat16)
    kv_in = randn(g, seqs, 2 * kv, hd, dtype=torch.bfloat16)

    def chain(wait):
        cache = rb.HarpCache.empty(1, seqs * 8, kv, page, hd)
        x, res = start, torch.zeros_like(start)
        lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        out = []
        for t in range(60):
            pos = lens.clone()
            lens += 1
            q, s, res = rb.harp_rmsnorm_q8(x, weight, res)
            wait()
            y = layers[0](q, s)
            wait()
            q = rope.append(cache, y.view(seqs, heads, hd), kv_in[:, :kv], kv_in[:, kv:], pos, table)
            wait()
            o = rb.harp_paged_attention(q, cache, table, lens)
            wait()
            x = layers[1](*rb.harp_quantize_q8(o.view(seqs, width)))
            wait()
            out.append(x)
        return torch.stack(out)

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        got = chain(lambda: None)
        assert torch.equal(got, want)
    clean(rb)


def test_calls_on_two_streams_do_not_disturb_each_other(rb):
    g = gen(37)
    q, cache, table, n = attention_case(rb, [700, 31, 0, 2000], 16, 4, 128, 16, torch.bfloat16)
    x, sx, w, sw = linear_case(rb, 300, 1024, 2048)
    layer = rb.HarpLinear8(w, sw)
    a0, y0 = rb.harp_paged_attention(q, cache, table, n), layer(x, sx)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((rb.harp_paged_attention(q, cache, table, n), layer(x, sx)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, a0) and torch.equal(y, y0) for a, y in got)
    clean(rb)


def test_linear8_refuses_what_it_cannot_count(rb):
    codes = torch.zeros(128, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    layer = rb.HarpLinear8(codes, torch.ones(1, 1, device="cuda"))
    with pytest.raises(ValueError):
        layer(torch.zeros(2, 63, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), torch.ones(2, 1, device="cuda"))
    with pytest.raises(ValueError):
        layer(codes, torch.ones(127, 1, device="cuda"))
    with pytest.raises(ValueError):
        layer(codes, torch.ones(128, 1, device="cuda"), out=torch.empty(128, 127, device="cuda"))
    layer.close()
    with pytest.raises(rb.HarpError):
        layer(codes, torch.ones(128, 1, device="cuda"))


def stack_case(rb, hidden, ffn, nh, nkv, hd, blocks, wb):
    from harp_cases import device_layer, oracle_layer
    shapes = [(nh * hd, hidden), (nkv * hd, hidden), (nkv * hd, hidden), (hidden, nh * hd), (ffn, hidden), (ffn, hidden), (hidden, ffn)]
    width = lambda n: n if n & (n - 1) == 0 else wb  # noqa: E731
    cases = [oracle_layer(o, i, wb if i == ffn else width(i), wb if o == ffn else width(o), 4, workload=4, layer=l, linear=j)
             for l in range(blocks) for j, (o, i) in enumerate(shapes)]
    layers = [device_layer(c) for c in cases]
    return [c["lay"] for c in cases], layers, rb.HarpStack(layers, hidden, ffn, nh, nkv, hd)


@pytest.mark.parametrize("batch,nh,nkv", [(1, 4, 2), (3, 4, 4), (17, 8, 2)])
def test_stack_step_cached(rb, ora, batch, nh, nkv):
    """Steps of a two-block stack over an f16 cache against the same steps in fp64 (oracle
    linears): rel-L2 within the linears' own 2e-3 plus the roundings of q, k, v and the attention's
    output to f16 (2^-11 each)."""
    hidden, ffn, hd, page, steps = 256, 768, 64, 8, 5
    ol, layers, S = stack_case(rb, hidden, ffn, nh, nkv, hd, 2, 256)
    cache = rb.HarpCache.empty(2, 4 * batch, nkv, page, hd, torch.float16)
    rope = rb.HarpRope(hd, interleaved=False, base=100.0)
    table = torch.randperm(4 * batch, generator=gen(3), device="cuda").view(batch, 4).to(torch.int32)
    rng = np.random.default_rng(batch)
    keys = [[[] for _ in range(batch)] for _ in range(2)]
    f = np.array(rope.frequencies)

    def turned(x, pos):
        a, b = x[..., :hd // 2], x[..., hd // 2:]
        c, s = np.cos(pos * f), np.sin(pos * f)
        return np.concatenate([a * c - b * s, a * s + b * c], -1)

    rms = lambda u: u / np.sqrt((u * u).mean(-1, keepdims=True) + 1e-5)  # noqa: E731
    start = np.arange(batch) % 3
    for t in range(steps):
        x = rng.standard_normal((batch, hidden)).astype(np.float32)
        pos = start * 0 + t
        got = S.step_cached(torch.from_numpy(x).cuda(), rope, cache, torch.from_numpy(pos.astype(np.int32)).cuda(), table)
        h = x.astype(np.float64)
        for l in range(2):
            L = ol[7 * l:7 * l + 7]
            n1 = rms(h)
            q, k, v = (ora.linear_fwd(L[i], n1).reshape(batch, -1, hd) for i in range(3))
            att = np.zeros((batch, nh, hd))
            for b in range(batch):
                keys[l][b].append((turned(k[b], pos[b]), v[b]))
                K = np.repeat(np.stack([p[0] for p in keys[l][b]], 1), nh // nkv, 0)
                V = np.repeat(np.stack([p[1] for p in keys[l][b]], 1), nh // nkv, 0)
                sc = np.einsum("hd,hnd->hn", turned(q[b], pos[b]), K) / math.sqrt(hd)
                p = np.exp(sc - sc.max(-1, keepdims=True))
                att[b] = np.einsum("hn,hnd->hd", p / p.sum(-1, keepdims=True), V)
            h = h + ora.linear_fwd(L[3], att.reshape(batch, -1))
            n2 = rms(h)
            gate, up = ora.linear_fwd(L[4], n2), ora.linear_fwd(L[5], n2)
            h = h + ora.linear_fwd(L[6], gate / (1 + np.exp(-gate)) * up)
        err = np.linalg.norm(got.cpu().numpy() - h) / np.linalg.norm(h)
        assert err < 2e-3 + 4 * 2.0**-11, (t, err)
    clean(rb)
    S.close()


def test_stack_step_cached_first_token_and_padding(rb):
    """At position 0 the attention returns the value, so the step equals harp_stack_step up to the
    value's rounding to f16; a padded row touches no cache and leaves the others as they are."""
    ol, layers, S = stack_case(rb, 256, 768, 4, 2, 64, 2, 256)
    cache = rb.HarpCache.empty(2, 4, 2, 16, 64, torch.float16)
    rope = rb.HarpRope(64)
    x = randn(gen(1), 3, 256)
    pos = torch.tensor([0, -1, 0], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0], [1], [2]], dtype=torch.int32, device="cuda")
    got = S.step_cached(x, rope, cache, pos, table)
    want = S.step(x)
    live = [0, 2]
    assert (torch.linalg.norm(got[live] - want[live]) / torch.linalg.norm(want[live])).item() < 4 * 2.0**-11
    assert (cache.k[:, 1] == 0).all() and (cache.k[:, 3] == 0).all() and (cache.k[:, 0, :, 0] != 0).any()
    assert not got.isnan().any()
    with pytest.raises(ValueError):
        S.step_cached(x, rope, rb.HarpCache.empty(1, 4, 2, 16, 64, torch.float16), pos, table)
    with pytest.raises(rb.HarpError):
        S.step_cached(x, rope, rb.HarpCache.empty(2, 4, 1, 16, 64, torch.float16), pos, table)
    clean(rb)
    S.close()


@pytest.mark.parametrize("tokens,n_out,step", [(3, 256, 0), (3, 256, 3), (20, 4096, 1), (300, 8192, 2), (300, 8001, 9)])
def test_linear8_wait_that_runs_out(rb, tokens, n_out, step):
    """The testing hook leaves the copies out from a K step on, under a 1 ms limit: the call ends, the status
    word says so, and the next call on the device is right."""
    x, sx, w, sw = linear_case(rb, tokens, 2048, n_out)
    layer = rb.HarpLinear8(w, sw)
    want = layer(x, sx, out_dtype=torch.float32)
    clean(rb)
    rb.harp_test_set_faults(wait_limit_us=1000, gemv_skip_stage=step)
    try:
        layer(x, sx)
        torch.cuda.synchronize()
        with pytest.raises(rb.HarpError) as e:
            rb.harp_device_status()
    finally:
        rb.harp_test_set_faults()
    assert e.value.status == 5 and any(f"site {site}" in str(e.value) for site in range(100, 108)), e.value
    assert torch.equal(layer(x, sx, out_dtype=torch.float32), want)
    clean(rb)


def test_served_token_with_an_8_bit_head(rb):
    """A cached step of the stack, the last norm with its 8-bit output and the head, captured as one
    graph: logits within the codes' half steps of the same chain in fp64 from the step's output."""
    ol, layers, S = stack_case(rb, 256, 768, 4, 2, 64, 2, 256)
    g = gen(41)
    cache = rb.HarpCache.empty(2, 8, 2, 16, 64)
    rope = rb.HarpRope(64)
    weight = 1 + 0.1 * randn(g, 256)
    W = randn(g, 1000, 256) / 16
    head = rb.HarpLinear8(*rb.harp_quantize_weights_q8(W))
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = randn(g, 2, 256)
    ws = S.cached_workspace(2)

    def token():
        h = S.step_cached(x, rope, cache, pos, table, workspace=ws)
        return h, head(*rb.harp_rmsnorm_q8(h, weight=weight), out_dtype=torch.float32)

    token()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, logits = token()
    for t in range(20):
        x.copy_(randn(g, 2, 256))
        pos.fill_(t)
        graph.replay()
        eager_h, eager = token()  # writes the same cache rows again
        assert torch.equal(h, eager_h) and torch.equal(logits, eager)
        y = norm64(h, weight, None, 1e-5)[1]
        want = y @ W.double().t()
        # codes: half a step (2^-4) of a value each, or 2^-10 of the block's 448th; products of two
        # such errors, and their sum over the columns
        ey = y.abs() * 2.0**-4 + y.abs().amax(-1, keepdim=True) / 448 * 2.0**-10
        eW = W.double().abs() * 2.0**-4 + W.double().abs().amax() / 448 * 2.0**-10
        tol = ey @ W.double().abs().t() + y.abs() @ eW.t() + ey @ eW.t()
        close(logits, want, tol * (1 + 1e-3))
    clean(rb)
    S.close()


def test_paged_attention_windows_of_any_size(rb):
    q, cache, table, n = attention_case(rb, [100, 50], 4, 2, 64, 16, torch.bfloat16)
    full = rb.harp_paged_attention(q, cache, table, n)
    for window in (100, 2**31 - 1, 2**31, 2**40):
        assert torch.equal(rb.harp_paged_attention(q, cache, table, n, window=window), full)
    for window in (-1, -2**40):
        with pytest.raises(rb.HarpError):
            rb.harp_paged_attention(q, cache, table, n, window=window)
    clean(rb)


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_paged_attention_scales_of_any_sign(rb, scale):
    lens = [300, 17, 0, 64]
    q, cache, table, n = attention_case(rb, lens, 8, 2, 128, 16, torch.bfloat16)
    out, lse = rb.harp_paged_attention(q, cache, table, n, scale=scale, return_lse=True)
    want, wlse, mag, reach = attention64(q, cache, table, lens, scale)
    tol, ltol = attention_tol(want, wlse, mag, reach, 128, torch.bfloat16, max(lens))
    live = [0, 1, 3]
    close(out, want, tol)
    close(lse[live], wlse[live], ltol[live])
    clean(rb)


def test_outputs_that_cannot_hold_the_result_are_refused(rb):
    q, cache, table, n = attention_case(rb, [100, 50], 4, 2, 64, 16, torch.bfloat16)
    over = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda").expand(2, 4, 64)
    rope, pos = rb.HarpRope(64), torch.zeros(2, dtype=torch.int32, device="cuda")
    for call in (lambda: rb.harp_paged_attention(q, cache, table, n, out=over), lambda: rope(q, pos, out=over),
                 lambda: rope.append(cache, q, q[:, :2], q[:, :2], pos, table, out=over),
                 lambda: rb.harp_paged_attention(q, cache, table, n, out=torch.empty_like(q, dtype=torch.float32)),
                 lambda: rope(q, pos, out=q.new_empty(2, 64, 4).transpose(1, 2))):
        with pytest.raises(ValueError):
            call()
    ol, layers, S = stack_case(rb, 256, 768, 4, 2, 64, 2, 256)
    two = rb.HarpCache.empty(2, 8, 2, 16, 64)
    x = torch.zeros(2, 256, device="cuda")
    for out in (torch.empty(1, 256, device="cuda"), torch.empty(256, 2, device="cuda").t(), torch.empty(4, 128, device="cuda")):
        with pytest.raises(ValueError):
            S.step_cached(x, rope, two, pos, table[:, :4].contiguous(), out=out)
    clean(rb)
    S.close()
