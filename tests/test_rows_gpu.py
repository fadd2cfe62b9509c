"""ula_pack_rows and ula_rotate against their formulas in 64 bits.

Tolerances, from the arithmetic. With u = 2^-24:
  - a rotary angle in turns is one product of 64-bit values, its frequency off by
    a few 2^-53; here and in the reference: 8 x 2^-53 x |position| x frequency,
    in radians; its sine and cosine in 32 bits are off by 4 u (the reduced angle,
    the series' last steps); a turned value, two products and their sum, by
    (|a| + |b|)(angle + 4 u + 3 u) before it is rounded to its type once: half a step.
  - a scale is a 32-bit quotient: off by 2 u of itself (twice half a step, of amax
    and of it), plus what amax is off by;
  - a code is the nearest to the 32-bit quotient y of value and scale, which is
    off by u |y| (and by what value and scale are off by), so the distance of the
    code from the exact quotient is at most that of the nearest code, plus twice that.
"""

import numpy as np
import pytest

import rows_ref as ref

pytestmark = pytest.mark.gpu

u = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
LEAST = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -25, "fp32": 2.0 ** -149}


def torch_type(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def on_gpu(x, kind):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch_type(kind)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def assert_within(got, want, tol):
    over = np.abs(got - want) / tol
    worst = float(np.max(np.where(np.isnan(over), np.inf, over), initial=0.0))
    assert worst <= 1.0, f"off by {worst:.3g} of the tolerance"


def turned(x, pos, sections, theta, interleaved, inverse=False):
    """(exact turned x, bound of its error before the rounding to a type); x [tokens][..., dim]"""
    y = ref.turn(x, pos, sections, theta, interleaved, inverse)
    dim = x.shape[-1]
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = np.abs(pos[:, axis].astype(np.float64)) * theta ** (-2.0 * np.arange(dim // 2) / dim)
    angle = (angle * 8 * 2.0 ** -53 + 7 * u).reshape(len(pos), *([1] * (x.ndim - 2)), dim // 2)
    i0, i1 = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, dim // 2), slice(dim // 2, None))
    d = np.empty_like(y)
    d[..., i0] = d[..., i1] = (np.abs(x[..., i0]) + np.abs(x[..., i1])) * angle
    return y, d


def positions_of(rng, n, axes, far):
    pos = rng.integers(-2 ** 31, 2 ** 31, (n, axes)) if far else rng.integers(0, 4096, (n, axes))
    pos = pos.astype(np.int32)
    pos[0] = 0
    if far and n > 2:
        pos[1], pos[2] = -2 ** 31, 2 ** 31 - 1
    return pos


def check_codes(codes, scale, x, dx=0.0):
    """codes [..., m] and their fp32 scales [...] for values x off by dx, scale blocks along the last axis"""
    finite = np.isfinite(x)
    amax = np.where(finite, np.abs(x), 0).max(-1)
    da = np.max(np.broadcast_to(dx, x.shape), -1)
    want = np.maximum(amax / 448, 2.0 ** -126)
    ds = 2 * u * want + da / 448 + 2.0 ** -149
    assert_within(scale, want, ds)
    got = ref.E4M3[codes]
    assert np.array_equal(np.isnan(got), np.isnan(x))
    y = np.clip(np.where(np.isnan(x), 0, x) / scale[..., None], -1e6, 1e6)
    near = ref.E4M3[ref.e4m3_nearest(y)]
    slack = 2 * (u * 1.001 * np.abs(y) + dx / scale[..., None])
    y, near = np.clip(y, -448, 448), np.clip(near, -448, 448)
    far = np.where(np.isnan(x), 0, np.abs(np.where(np.isnan(x), 0, got) - y) - np.abs(near - y) - slack)
    assert far.max() <= 0, (far.max(), np.argwhere(far > 0)[:3])


def latent_parts(rows):
    rows = rows.cpu().numpy()
    scale = ref.f32_at(rows, 640, 4)
    codes = rows[..., :512].reshape(*rows.shape[:-1], 4, 128)
    rope = ref.bf16_values(np.ascontiguousarray(rows[..., 512:640]).view("<u2"))
    return codes, scale, rope


# entries, layers, type, axes (0: nothing turned), interleaved, far positions
LATENT = [(1, 1, "bf16", 0, False, False), (1, 3, "fp32", 1, True, True), (7, 1, "fp16", 1, False, False),
          (64, 3, "bf16", 1, True, False), (129, 2, "fp32", 2, False, True), (33, 5, "fp16", 3, True, True)]
SECTIONS = {1: (32,), 2: (20, 12), 3: (16, 0, 16)}


@pytest.mark.parametrize("n,layers,kind,axes,inter,far", LATENT)
def test_latent_rows(n, layers, kind, axes, inter, far):
    import torch
    from serving_pb_lru_amd import latent_rows, pack_rows
    rng = np.random.default_rng([n, layers, axes])
    lat = on_gpu(rng.standard_normal((n, layers, 512)) * 2.0 ** rng.uniform(-12, 12, (n, layers, 1)), kind)
    rope = on_gpu(rng.standard_normal((n, layers, 64)), kind)
    pos = positions_of(rng, n, axes, far) if axes else None
    dpos = torch.from_numpy(pos).cuda() if axes else None
    rows = pack_rows(latent_rows(), lat, rope, dpos, SECTIONS.get(axes), theta=5000.0, interleaved=inter)
    assert rows.shape == (n, layers, 656)
    codes, scale, got = latent_parts(rows)
    check_codes(codes, scale, f64(lat).reshape(n, layers, 4, 128))
    y, d = turned(f64(rope), pos, SECTIONS[axes], 5000.0, inter) if axes else (f64(rope), 0.0)
    assert_within(got, y, d + HALF["bf16"] * (np.abs(y) + d) + LEAST["bf16"])


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_latent_values_at_the_ends(kind):
    """Zeros, infinities, NaN, the largest and the least values of the type, ties between codes."""
    import torch
    from serving_pb_lru_amd import latent_rows, pack_rows
    info = torch.finfo(torch_type(kind))
    x = np.zeros((9, 1, 512))
    rng = np.random.default_rng(3)
    x[1] = rng.standard_normal(512)
    x[1, 0, 5], x[1, 0, 200], x[1, 0, 201], x[1, 0, 511] = np.inf, -np.inf, np.nan, np.nan
    x[2, 0, ::2], x[2, 0, 1::2] = info.max, info.min
    x[3, 0, :128] = info.tiny * np.arange(128)
    x[4] = np.nan
    x[5, 0, :128], x[5, 0, 128:] = np.inf, -np.inf
    x[6, 0, 3] = info.smallest_normal * 2.0 ** -3          # a subnormal alone
    x[7, 0] = 448.0 / 512 * np.arange(512)                 # scale 1 or less: exact ties and steps
    x[7, 0, 127::128] = 448.0
    x[8, 0, :] = np.repeat([2.0 ** -10, 2.0 ** -3, 1.0, 2.0 ** 4], 128)
    t = on_gpu(x, kind)
    rows = pack_rows(latent_rows(), t, torch.zeros((9, 1, 64), dtype=t.dtype, device="cuda"))
    codes, scale, rope = latent_parts(rows)
    v = f64(t).reshape(9, 1, 4, 128)
    check_codes(codes, scale, v)
    assert np.all(scale[0] == np.float32(2.0 ** -126)) and not codes[0].any() and not rope.any()
    at = ref.E4M3[codes]
    assert at[1, 0, 0, 5] == 448 and at[1, 0, 1, 72] == -448
    assert np.all(np.abs(at[5]) == 448) and np.all(np.isnan(at[4])) and np.all(scale[4:6] == np.float32(2.0 ** -126))


def test_latent_strides_and_alignment():
    """Views: every other entry, layers swapped, a misaligned first element; the result is that of packed copies."""
    import torch
    from serving_pb_lru_amd import latent_rows, pack_rows
    g = torch.Generator(device="cuda").manual_seed(5)
    whole = torch.randn((10, 3, 580), device="cuda", generator=g).to(torch.bfloat16)
    pos = torch.arange(10, dtype=torch.int32, device="cuda")
    for lat, rope, p in [(whole[::2, :, 1:513], whole[::2, :, 515:579], pos[::2].contiguous()),
                         (whole.transpose(0, 1)[:, :, 8:520], whole.transpose(0, 1)[:, :, 3:67], pos[:3].contiguous()),
                         (whole[:, 1:2].expand(10, 4, 580)[..., :512], whole[:, 1:2].expand(10, 4, 580)[..., 512:576], pos)]:
        a = pack_rows(latent_rows(), lat, rope, p)
        b = pack_rows(latent_rows(), lat.contiguous(), rope.contiguous(), p)
        assert torch.equal(a, b)
        out = torch.full((*a.shape[:2], 656), 7, dtype=torch.uint8, device="cuda")
        assert pack_rows(latent_rows(), lat, rope, p, out=out) is out and torch.equal(a, out)
    assert pack_rows(latent_rows(), whole[:0, :, :512], whole[:0, :, :64]).shape == (0, 3, 656)


# entries, layers, kv heads, dim, block, type, axes, interleaved, counts
HEADS = [(1, 1, 1, 64, 1, "bf16", 0, False, False), (5, 2, 8, 128, 1, "fp16", 1, False, False),
         (9, 1, 2, 64, 8, "bf16", 1, True, True), (3, 3, 1, 64, 16, "fp32", 2, False, True),
         (17, 1, 3, 128, 2, "bf16", 3, True, True), (2, 1, 1, 128, 8, "fp32", 1, False, True)]


@pytest.mark.parametrize("n,layers,kv,dim,block,kind,axes,inter,part", HEADS)
def test_heads_rows(n, layers, kv, dim, block, kind, axes, inter, part):
    import torch
    from serving_pb_lru_amd import head_rows, pack_rows
    rng = np.random.default_rng([n, kv, dim, block])
    shape = (n, layers, block, kv, dim)
    keys = on_gpu(rng.standard_normal(shape) * 2.0 ** rng.uniform(-5, 5, (n, layers, 1, kv, 1)), kind)
    vals = on_gpu(rng.standard_normal(shape), kind)
    fmt = head_rows(kv, dim, block)
    counts = rng.integers(-2, block + 3, n).astype(np.int32) if part else None
    if part:
        counts[0] = 0
    dcounts = torch.from_numpy(counts).cuda() if part else None
    half = dim // 2
    sections = {0: None, 1: (half,), 2: (half - 5, 5), 3: (0, half - 7, 7)}[axes]
    pos = positions_of(rng, n * block, axes, False) if axes else None
    dpos = torch.from_numpy(pos.reshape(n, block, axes)).cuda() if axes else None
    rows = pack_rows(fmt, keys, vals, dpos, sections, interleaved=inter, counts=dcounts).cpu().numpy()
    assert rows.shape == (n, layers, fmt.row_bytes)
    use = np.clip(counts, 0, block) if part else np.full(n, block)
    live = (np.arange(block)[None] < use[:, None])[:, None, :, None, None]
    size = kv * block * dim
    tail = rows[..., 2 * size:]
    assert np.array_equal(np.ascontiguousarray(tail[..., 8 * kv:8 * kv + 4]).view("<i4")[..., 0],
                          np.repeat(use[:, None], layers, 1))
    assert not tail[..., 8 * kv + 4:].any()
    for which, t in ((0, keys), (1, vals)):
        x, d = f64(t), np.zeros(shape)
        if axes and which == 0:
            flat = lambda z: z.transpose(0, 2, 1, 3, 4).reshape(n * block, layers, kv, dim)
            back = lambda z: z.reshape(n, block, layers, kv, dim).transpose(0, 2, 1, 3, 4)
            y, dy = turned(flat(x), pos, sections, 10000.0, inter)
            x, d = back(y), back(dy)
        x, d = np.where(live, x, 0), np.where(live, d, 0)
        per_head = lambda z: z.transpose(0, 1, 3, 2, 4).reshape(n, layers, kv, block * dim)
        codes = rows[..., which * size:(which + 1) * size].reshape(n, layers, kv, block * dim)
        check_codes(codes, ref.f32_at(rows, 2 * size + 4 * kv * which, kv), per_head(x), per_head(d))


@pytest.mark.parametrize("kv,dim,block", [(1, 64, 1), (8, 128, 1), (3, 64, 8), (1, 64, 16), (1, 128, 8), (2, 128, 4)])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_heads_values_at_the_ends(kv, dim, block, kind):
    """Infinities, NaN, zeros and subnormals in some scale blocks beside ordinary ones, of less and of
    more than a wave; strided sources give the same rows."""
    import torch
    from serving_pb_lru_amd import head_rows, pack_rows
    rng = np.random.default_rng([kv, dim, block])
    info = torch.finfo(torch_type(kind))
    n = 40
    x = rng.standard_normal((2, n, 1, block, kv, dim))
    x[0, 3, 0, :, 0] = 0.0
    x[0, 5, 0, 0, 0, 1], x[0, 7, 0, block - 1, kv - 1, dim - 1], x[1, 9, 0, 0, 0, 0] = np.inf, -np.inf, np.nan
    x[0, 11, 0, :, 0] = np.nan
    x[1, 13, 0, :, kv - 1] *= info.tiny
    x[0, 15] = info.max
    t = on_gpu(x, kind)
    fmt = head_rows(kv, dim, block)
    rows = pack_rows(fmt, t[0], t[1])
    part = kv * dim * block
    got = rows.cpu().numpy()
    for side in (0, 1):
        v = f64(t[side]).transpose(0, 1, 3, 2, 4).reshape(n, 1, kv, block * dim)
        codes = got[..., side * part:(side + 1) * part].reshape(n, 1, kv, block * dim)
        check_codes(codes, ref.f32_at(got, 2 * part + 4 * kv * side, kv), v)
    wide = torch.zeros((n, 1, block, kv, dim + 3), dtype=t.dtype, device="cuda")
    wide[..., 1:dim + 1] = t[0]
    swapped = t[1].transpose(2, 3).contiguous().transpose(2, 3)
    assert torch.equal(pack_rows(fmt, wide[..., 1:dim + 1], swapped), rows)


# tokens, heads, dim, type, axes, interleaved, inverse, far
ROTATE = [(1, 1, 2, "fp32", 1, True, False, False), (3, 5, 6, "bf16", 1, False, False, True),
          (16, 128, 64, "bf16", 1, True, False, False), (100, 3, 126, "fp16", 2, True, True, False),
          (257, 33, 128, "fp32", 3, False, True, True), (7, 9, 256, "fp16", 1, False, False, False),
          (165, 5, 256, "fp16", 3, False, False, True), (600, 1, 40, "bf16", 3, True, False, True), (2, 700, 256, "fp32", 2, False, False, False)]


@pytest.mark.parametrize("n,heads,dim,kind,axes,inter,inverse,far", ROTATE)
def test_rotate(n, heads, dim, kind, axes, inter, inverse, far):
    import torch
    from serving_pb_lru_amd import rotate
    rng = np.random.default_rng([n, heads, dim])
    x = on_gpu(rng.standard_normal((n, heads, dim)), kind)
    half = dim // 2
    sections = {1: (half,), 2: (half - half // 3, half // 3), 3: (half // 2, 0, half - half // 2)}[axes]
    pos = positions_of(rng, n, axes, far)
    dpos = torch.from_numpy(pos).cuda()
    y, d = turned(f64(x), pos, sections, 1e4, inter, inverse)
    tol = d + HALF[kind] * (np.abs(y) + d) + LEAST[kind]
    kept = x.clone()
    out = rotate(x, dpos, sections, interleaved=inter, inverse=inverse)
    assert torch.equal(x, kept)
    assert_within(f64(out), y, tol)
    # strided, misaligned, and in place: the same bits
    wide = torch.zeros((n, heads, dim + 3), dtype=x.dtype, device="cuda")
    view = wide[..., 1:dim + 1]
    view.copy_(x)
    assert torch.equal(rotate(view, dpos, sections, interleaved=inter, inverse=inverse), out)
    assert rotate(view, dpos, sections, interleaved=inter, inverse=inverse, out=view) is view
    assert torch.equal(view, out) and not wide[..., 0].any() and not wide[..., dim + 1:].any()
    swapped = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(rotate(swapped, dpos, sections, interleaved=inter, inverse=inverse, out=swapped), out)


def test_rotate_back_is_the_gradient():
    """The turn is linear, so its gradient is its transpose: <turn(x), g> = <x, back(g)>, and a
    difference turn(x + e) - turn(x) is turn(e); checked by component in 64 bits. Each result of
    32 bits is off by (|a| + |b|) 8 u at most, here summed over the vector."""
    import torch
    from serving_pb_lru_amd import rotate
    rng = np.random.default_rng(11)
    n, heads, dim = 5, 3, 64
    x, g, e = (on_gpu(rng.standard_normal((n, heads, dim)), "fp32") for _ in range(3))
    pos = torch.from_numpy(positions_of(rng, n, 2, False)).cuda()
    for inter in (False, True):
        turn = lambda t, back=False: f64(rotate(t, pos, (20, 12), interleaved=inter, inverse=back))
        bound = 2 * 8 * u * 2 * (np.abs(f64(x)).sum() * np.abs(f64(g)).max())
        assert abs((turn(x) * f64(g)).sum() - (f64(x) * turn(g, True)).sum()) <= bound
        big = np.abs(f64(x)).max() + np.abs(f64(e)).max()
        assert np.abs(turn(x + e) - turn(x) - turn(e)).max() <= 3 * 8 * u * 2 * big + 2 * u * big
        assert np.abs(turn(rotate(x, pos, (20, 12), interleaved=inter), True) - f64(x)).max() <= 2 * 8 * u * 2 * big


def test_rotate_empty_and_refusals():
    import torch
    from serving_pb_lru_amd import UlaError, latent_rows, pack_rows, rotate
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    assert rotate(x[:0], pos[:0]).shape == (0, 2, 64) and rotate(x[:, :0], pos).shape == (4, 0, 64)
    for bad in [dict(positions=pos[:3]), dict(positions=pos.long()), dict(positions=None),
                dict(positions=pos.expand(4, 2)), dict(sections=(16, 16)), dict(out=x[:3]),
                dict(out=torch.zeros_like(x, dtype=torch.float16)), dict(positions=pos.cpu())]:
        with pytest.raises(ValueError):
            rotate(**{"x": x, "positions": pos, **bad})
    for bad in [dict(sections=(31,)), dict(theta=0.0), dict(theta=float("nan"))]:
        with pytest.raises(UlaError):
            rotate(x, pos, **bad)
    with pytest.raises(ValueError):
        rotate(x.transpose(1, 2), pos)
    lat, rope = torch.zeros((4, 2, 512), device="cuda"), torch.zeros((4, 2, 64), device="cuda")
    for bad in [dict(a=lat[..., :511]), dict(b=rope[:3]), dict(b=rope.half()), dict(counts=pos[:, 0]),
                dict(positions=pos[:2]), dict(out=torch.zeros((4, 2, 655), dtype=torch.uint8, device="cuda")),
                dict(a=lat.transpose(1, 2))]:
        with pytest.raises(ValueError):
            pack_rows(**{"fmt": latent_rows(), "a": lat, "b": rope, **bad})


def test_graph_of_both_replays():
    """Row writer and turn captured into one graph: every replay sees the inputs of its time, with the
    program's own calls and synchronisations in between."""
    import torch
    from serving_pb_lru_amd import latent_rows, pack_rows, rotate
    gen = torch.Generator(device="cuda").manual_seed(2)
    lat = torch.randn((6, 2, 512), device="cuda", generator=gen).to(torch.bfloat16)
    rope = torch.randn((6, 2, 64), device="cuda", generator=gen).to(torch.bfloat16)
    q = torch.randn((6, 9, 64), device="cuda", generator=gen).to(torch.bfloat16)
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    rows = torch.zeros((6, 2, 656), dtype=torch.uint8, device="cuda")
    back = torch.zeros_like(q)
    pack_rows(latent_rows(), lat, rope, pos, out=rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pack_rows(latent_rows(), lat, rope, pos, out=rows)
        rotate(q, pos, out=back)
    for i in range(4):
        lat.normal_(generator=gen)
        rope.mul_(-1.25)
        q.normal_(generator=gen)
        pos.add_(1000 * i)
        want = pack_rows(latent_rows(), lat, rope, pos), rotate(q, pos)
        rows.zero_()
        back.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rows, want[0]) and torch.equal(back, want[1]), i


def test_tensors_past_32_bits():
    """Outputs and inputs of more than 2^32 bytes (rows) and elements (the turn): their ends equal calls
    of the ends alone."""
    import torch
    from serving_pb_lru_amd import latent_rows, pack_rows, rotate
    n = (1 << 32) // 656 + 1000
    lat = torch.zeros((n, 1, 512), dtype=torch.bfloat16, device="cuda")
    rope = torch.zeros((n, 1, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    lat[-700:].normal_()
    rope[-700:].normal_()
    rows = pack_rows(latent_rows(), lat, rope, pos)
    assert torch.equal(rows[-700:], pack_rows(latent_rows(), lat[-700:], rope[-700:], pos[-700:]))
    del lat, rope, rows
    n = (1 << 32) // (128 * 128) + 9
    x = torch.zeros((n, 128, 128), dtype=torch.bfloat16, device="cuda")
    x[-12:].normal_()
    want = rotate(x[-12:], pos[:n][-12:])
    rotate(x, pos[:n], out=x)
    assert torch.equal(x[-12:], want) and not bool(x[:100].any())


def test_two_streams():
    import torch
    from serving_pb_lru_amd import rotate
    x = torch.randn((2000, 16, 128), device="cuda")
    pos = torch.arange(2000, dtype=torch.int32, device="cuda")
    want = rotate(x, pos), rotate(x, pos, inverse=True)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(a):
            first = rotate(x, pos)
        second = rotate(x, pos, inverse=True, stream=b)
        torch.cuda.synchronize()
        assert torch.equal(first, want[0]) and torch.equal(second, want[1])


def test_tensors_dropped_while_another_stream_reads_them():
    """Inputs freed right after a call on a busy stream are not reused before it has read them, nor a
    result that the caller's stream still reads."""
    import torch
    from serving_pb_lru_amd import rotate
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    x = torch.randn((64, 16, 128), device="cuda")
    want = rotate(x, pos)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)               # about 0.1 s
    got = rotate(x, pos, stream=side)
    del x
    others = [torch.full((64, 16, 128), 7.0, device="cuda") for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    torch.cuda._sleep(200_000_000)
    copy = got.clone()
    del got
    with torch.cuda.stream(side):
        others += [torch.full((64, 16, 128), 9.0, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(others) == 8
