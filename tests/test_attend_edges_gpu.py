"""ula_attend where it can go wrong: layouts, selections other than the step's, rows out of use,
infinities and NaN, wide scales, other streams, errors. Tolerances are those of the formula's tests."""

import numpy as np
import pytest

from test_attend_gpu import (check, engine_of, f32_bytes, heads_rows_of, latent_rows_of, selection, torch_type)

pytestmark = pytest.mark.gpu


def formats():
    from serving_pb_lru_amd import head_rows, latent_rows
    return {"latent": latent_rows(), "heads": head_rows(2, 64, 2)}


def rows_for(name, rng, n, layers=1):
    return latent_rows_of(rng, n, layers) if name == "latent" else heads_rows_of(rng, n, layers, 2, 64, 2)


def width_of(fmt):
    return 576 if fmt.kind == 0 else fmt.head_dim


def queries(rng, fmt, sets, heads, kind="bf16"):
    import torch
    return torch.from_numpy(rng.standard_normal((sets, heads, width_of(fmt)))).to(torch_type(kind)).cuda()


class Opened:
    """An engine over `rows`, its one step done."""

    def __init__(self, fmt, rows, sel, **kw):
        import torch
        self.fmt, self.rows, self.sel = fmt, rows, sel
        self.eng = engine_of(rows, *sel.shape, **kw)
        self.dsel = torch.from_numpy(sel).cuda()
        self.eng.step(0, self.dsel)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.eng.close()

    def attend(self, q, sel=None, **kw):
        import torch
        return self.eng.attend(0, 0, self.dsel if sel is None else torch.from_numpy(sel).cuda(), q, self.fmt, **kw)

    def check(self, q, out, lse, sel=None, kind="bf16", scale=None):
        check(self.fmt, self.rows, 0, self.sel if sel is None else sel, q,
              width_of(self.fmt) ** -0.5 if scale is None else scale, out, lse, kind)


@pytest.mark.parametrize("name", ["latent", "heads"])
def test_strides_and_alignment(name):
    """q as a view of a wider, misaligned and transposed tensor, out the same: the bits of packed ones,
    and nothing beside them written."""
    import torch
    rng = np.random.default_rng(1)
    fmt = formats()[name]
    w, back = width_of(fmt), 512 if fmt.kind == 0 else 64
    with Opened(fmt, rows_for(name, rng, 200), selection(rng, 200, 3, 70, 2)) as o:
        q = queries(rng, fmt, 3, 6)
        out, lse = o.attend(q)
        o.check(q, out, lse)
        wide = torch.zeros((6, 3, w + 5), dtype=q.dtype, device="cuda")
        view = wide.transpose(0, 1)[..., 3:w + 3]
        view.copy_(q)
        target = torch.full((3, 8, back + 7), 3.0, dtype=q.dtype, device="cuda")
        got, glse = o.attend(view, out=target[:, 1:7, 5:back + 5], lse=torch.zeros_like(lse))
        assert torch.equal(got, out) and torch.equal(glse, lse)
        target[:, 1:7, 5:back + 5] = 3.0
        assert bool((target == 3.0).all())
        # one query for every head, read through a stride of 0
        same, _ = o.attend(q[:, :1].expand(3, 6, w))
        assert torch.equal(same[:, 0], same[:, 1]) if fmt.kind == 0 else torch.equal(same[:, 0], same[:, 2])
        o.eng.sync()


@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("k", [0, 1, 37])
def test_nothing_selected(name, k):
    """Sets of padding alone, sets of no entries, no sets."""
    import torch
    rng = np.random.default_rng(k)
    fmt = formats()[name]
    sel = selection(rng, 100, 3, k)
    if k:
        sel[1] = -1
    with Opened(fmt, rows_for(name, rng, 100), sel) as o:
        q = queries(rng, fmt, 3, 4)
        out, lse = o.attend(q)
        o.check(q, out, lse)
        assert not out[1].any() and bool(torch.isneginf(lse[1]).all())
        none, nlse = o.eng.attend(0, 0, o.dsel[:0], q[:0], fmt)
        assert none.shape[0] == 0 and nlse.shape == (0, 4)
        o.eng.sync()


@pytest.mark.parametrize("name", ["latent", "heads"])
def test_other_selections_than_the_steps(name):
    """Repeated addresses (counted as often), other orders and lengths, entries the step did not select."""
    rng = np.random.default_rng(4)
    fmt = formats()[name]
    with Opened(fmt, rows_for(name, rng, 300), selection(rng, 300, 2, 64)) as o:
        q = queries(rng, fmt, 2, 4)
        twice = o.sel.copy()
        twice[:, 32:] = twice[:, :32]
        twice[0, :8] = twice[0, 40]
        for sel in (o.sel[:, ::-1].copy(), twice, selection(rng, 300, 2, 61, 9), selection(rng, 300, 2, 1), o.sel[:, :33].copy()):
            out, lse = o.attend(q, sel)
            o.check(q, out, lse, sel)
        out, lse = o.attend(q[:1], o.sel[1:2].copy())
        o.check(q[:1], out, lse, o.sel[1:2])
        o.eng.sync()


@pytest.mark.parametrize("name", ["latent", "heads"])
def test_repeated_misses_and_evictions(name):
    """The step reads entries from the host pool and lists one of them twice in a set: attention of its selection."""
    import torch
    rng = np.random.default_rng(6)
    fmt = formats()[name]
    rows = rows_for(name, rng, 120)
    sel = selection(rng, 60, 2, 20)
    with Opened(fmt, rows, sel, gpu_slots=60, host_slots=80) as o:
        q = queries(rng, fmt, 2, 4)
        for t in range(4):
            new = rng.integers(60, 120, (2, 20)).astype(np.int32) if t % 2 == 0 else selection(rng, 120, 2, 20, 3)
            new[0, 3] = new[1, 7] = new[0, 9]
            o.eng.step(0, torch.from_numpy(new).cuda())
            out, lse = o.attend(q, new)
            o.check(q, out, lse, new)
        o.eng.sync()


@pytest.mark.parametrize("name", ["latent", "heads"])
def test_rows_out_of_use_may_hold_anything(name):
    """Every row that no set selects is all ones (NaN codes, scales and rotary channels)."""
    rng = np.random.default_rng(8)
    fmt = formats()[name]
    rows = rows_for(name, rng, 90)
    sel = selection(rng, 90, 2, 33, 5)
    rows[np.setdiff1d(np.arange(90), sel)] = 0xFF
    with Opened(fmt, rows, sel) as o:
        q = queries(rng, fmt, 2, 4, "fp16")
        out, lse = o.attend(q)
        o.check(q, out, lse, kind="fp16")


@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_infinities_and_nan(name, kind):
    """A NaN or an infinity in a query or a selected row makes the results that use it NaN (or, where the
    formula has a limit, that); the other heads and sets are untouched."""
    import torch
    rng = np.random.default_rng(9)
    fmt = formats()[name]
    rows = rows_for(name, rng, 120)
    sel = selection(rng, 100, 3, 40)
    sel[2, 5] = 110
    rows[110, 0, 3] = 0x7F                                     # one NaN code of a key, KV head 0
    with Opened(fmt, rows, sel) as o:
        q = queries(rng, fmt, 3, 4, kind)
        clean, _ = o.attend(q)
        bad = q.clone()
        bad[0, 1, 7] = float("nan")
        bad[1, 0, 9] = float("inf")
        out, lse = o.attend(bad)
        assert bool(out[0, 1].isnan().all()) and bool(lse[0, 1].isnan())
        assert bool(out[1, 0].isnan().all())
        for s, h in [(0, 0), (0, 2), (0, 3), (1, 1), (1, 2), (1, 3)]:
            assert torch.equal(out[s, h], clean[s, h]), (s, h)
        uses = slice(0, 4) if fmt.kind == 0 else slice(0, 2)   # the heads that read KV head 0
        assert bool(out[2, uses].isnan().all())
        if fmt.kind == 1:
            assert not bool(out[2, 2:].isnan().any())
        o.eng.sync()


@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("scale", [0.0, -0.04, 3.0, 1e-30])
def test_scales_of_the_logits(name, scale):
    rng = np.random.default_rng(10)
    fmt = formats()[name]
    with Opened(fmt, rows_for(name, rng, 150), selection(rng, 150, 2, 66, 1)) as o:
        q = queries(rng, fmt, 2, 4, "fp16")
        out, lse = o.attend(q, scale=scale)
        o.check(q, out, lse, kind="fp16", scale=scale)


@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("low,high", [(-40, -30), (20, 30), (-20, 0)])
def test_wide_value_scales(name, low, high):
    """Scales far from 1: the weights times them would leave fp16's range if their reference did not follow.
    (Key scales of latent rows are the same: q is scaled to keep the logits ordinary.)"""
    import torch
    rng = np.random.default_rng(12)
    fmt = formats()[name]
    rows = rows_for(name, rng, 150)
    if fmt.kind == 0:
        rows[..., 640:] = f32_bytes(2.0 ** rng.uniform(low, high, (150, 1, 4)) / 448)
        rows[..., 512:640] = 0
    else:
        size = 2 * 2 * 64 * 2
        rows[..., size + 8:size + 16] = f32_bytes(2.0 ** rng.uniform(low, high, (150, 1, 2)) / 448)
    with Opened(fmt, rows, selection(rng, 150, 2, 97, 1)) as o:
        q = queries(rng, fmt, 2, 4)
        if fmt.kind == 0:
            q = q * 2.0 ** -high
        out, lse = o.attend(q)
        o.check(q, out, lse)


@pytest.mark.parametrize("high", [-20, 0, 14])
def test_queries_of_any_magnitude(high):
    """Latent heads whose channels span many powers of two, and a head of zeros."""
    rng = np.random.default_rng(13)
    fmt = formats()["latent"]
    with Opened(fmt, rows_for("latent", rng, 150), selection(rng, 150, 2, 40)) as o:
        q = queries(rng, fmt, 2, 20, "fp16")
        import torch
        spread = torch.from_numpy(2.0 ** rng.uniform(high - 16, high, (2, 20, 576))).cuda()
        q = (q.double() * spread).clamp(-60000, 60000).to(q.dtype)
        q[1, 3] = 0
        scale = 2.0 ** -high / 24
        out, lse = o.attend(q, scale=scale)
        o.check(q, out, lse, kind="fp16", scale=scale)


@pytest.mark.parametrize("name", ["latent", "heads"])
def test_same_bits_again_and_on_two_streams(name):
    import torch
    rng = np.random.default_rng(14)
    fmt = formats()[name]
    with Opened(fmt, rows_for(name, rng, 500), selection(rng, 500, 9, 400, 3)) as o:
        q, r = queries(rng, fmt, 9, 40), queries(rng, fmt, 9, 40)
        want, other = o.attend(q), o.attend(r)
        torch.cuda.synchronize()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        for _ in range(3):
            with torch.cuda.stream(a):
                first = o.attend(q)
            second = o.attend(r, stream=b)
            torch.cuda.synchronize()
            for x, y in zip((*first, *second), (*want, *other)):
                assert torch.equal(x, y)
        o.check(q, *want)
        # the next step and the release of what these calls read wait for them
        o.eng.release(0, np.arange(250, dtype=np.int32))
        o.eng.sync()


def test_errors():
    import torch
    from serving_pb_lru_amd import UlaError, head_rows, latent_rows, ula
    rng = np.random.default_rng(15)
    fmt = latent_rows()
    rows = latent_rows_of(rng, 60, 2)
    eng = engine_of(rows, 2, 32, gpu_slots=40, host_slots=40)
    sel = torch.from_numpy(selection(rng, 30, 2, 32 - 8)).cuda()
    q = queries(rng, fmt, 2, 4)
    code = lambda **kw: pytest.raises(UlaError, eng.attend, **{**dict(group=0, layer=0, sel=sel, q=q, fmt=fmt), **kw}).value.name
    try:
        assert code() == "ENOTRESIDENT"                                   # no step yet
        eng.step(0, sel)
        assert code(group=1) == code(group=-1) == code(layer=2) == code(layer=-1) == "EINVAL"
        assert code(scale=float("nan")) == code(scale=float("inf")) == "EINVAL"
        assert code(sel=torch.zeros((3, 4), dtype=torch.int32, device="cuda"), q=queries(rng, fmt, 3, 4)) == "EINVAL"
        assert code(sel=torch.zeros((2, 33), dtype=torch.int32, device="cuda")) == "EINVAL"
        assert code(fmt=head_rows(2, 64), q=q[..., :64]) == "EINVAL"      # not the rows' size
        for bad in [dict(q=q[..., :575]), dict(q=q[:1]), dict(q=q.float()), dict(q=q.cpu()), dict(sel=sel.long()),
                    dict(q=q.transpose(1, 2)), dict(out=torch.zeros((2, 4, 511), dtype=q.dtype, device="cuda")),
                    dict(out=torch.zeros((2, 4, 512), dtype=torch.float16, device="cuda")),
                    dict(lse=torch.zeros(7, device="cuda")), dict(lse=torch.zeros(8, dtype=torch.float64, device="cuda")),
                    dict(q=q[0])]:
            with pytest.raises(ValueError):
                eng.attend(**{**dict(group=0, layer=0, sel=sel, q=q, fmt=fmt), **bad})
        args = ula.UlaAttendArgs()
        args.rows, args.type, args.heads, args.scale = fmt, ula.BF16, 4, 1.0
        args.q, args.out, args.q_set_stride, args.q_head_stride = q.data_ptr(), q.data_ptr(), 2304, 576
        many = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
        run = lambda n, k: ula.lib().ula_attend(eng.ctx, 0, 0, n, k, many.data_ptr(), ula.ctypes.byref(args), 0)
        assert run(3, 1) == run(1, 33) == run(-1, 1) == run(1, -1) == -1
        for strides in [(512, 0), (511, 512), (2048, 511), (0, 512)]:     # rows of out that share elements
            args.out_set_stride, args.out_head_stride = strides
            assert run(2 if strides[0] < 512 else 1, 1) == -1, strides
        args.out_set_stride, args.out_head_stride = 2048, 512
        args.q = q.data_ptr() + 1
        assert run(1, 1) == -1
        args.q, args.type = q.data_ptr(), ula.FP32
        assert run(1, 1) == -1
        args.type, args.heads = ula.BF16, 0
        assert run(1, 1) == -1
        # a capture would replay one step's state
        graph = torch.cuda.CUDAGraph()
        out, lse = eng.attend(0, 0, sel, q, fmt)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            err = pytest.raises(UlaError, eng.attend, 0, 0, sel, q, fmt, out=out, lse=lse).value.name
            q.add(1)
        assert err == "EINVAL"
        eng.sync()
        check(fmt, rows, 0, sel.cpu().numpy(), q, 1 / 24, out, lse, "bf16")
    finally:
        eng.close()


def test_rows_past_32_bits():
    """A pool of more than 2^32 bytes: attention, fork and release of entries at its end."""
    import torch
    from serving_pb_lru_amd import latent_rows
    fmt, chunk = latent_rows(), 65536
    n = (1 << 32) // 656 // chunk * chunk + 2 * chunk
    rng = np.random.default_rng(18)
    from serving_pb_lru_amd import Engine
    eng = Engine(num_groups=1, layers=1, row_bytes=656, ring=2, logical_capacity=n, gpu_slots=n, host_slots=0,
                 max_sets=2, max_k=64, max_append=chunk)
    try:
        filler = torch.zeros((chunk, 1, 656), dtype=torch.uint8, device="cuda")
        for at in range(0, n - chunk, chunk):
            eng.append(0, np.arange(at, at + chunk, dtype=np.int32), filler)
        last = n - chunk
        some = latent_rows_of(rng, 500, 1)
        eng.append(0, np.arange(last, last + 500, dtype=np.int32), some)
        eng.fork(0, last, last + 1000, 500)
        sel = rng.choice(500, (2, 64), replace=False).astype(np.int32)
        sel[1] += 1000
        d = torch.from_numpy(sel + last).cuda()
        assert last * 656 > 1 << 32
        eng.step(0, d)
        q = queries(rng, fmt, 2, 8)
        out, lse = eng.attend(0, 0, d, q, fmt)
        eng.sync()
        check(fmt, some, 0, sel - np.array([[0], [1000]], np.int32), q, 1 / 24, out, lse, "bf16")
        eng.release(0, np.arange(last - 5000, last + 500, dtype=np.int32))
        assert np.array_equal(eng.read_rows(0, np.arange(last + 1000, last + 1500, dtype=np.int32)), some)
        eng.sync()
    finally:
        eng.close()


def test_groups_and_layers():
    """Two groups of three layers with rows and steps of their own, read layer by layer."""
    import torch
    from serving_pb_lru_amd import Engine, latent_rows
    fmt = latent_rows()
    rng = np.random.default_rng(19)
    rows = [latent_rows_of(rng, 90, 3) for _ in range(2)]
    eng = Engine(num_groups=2, layers=3, row_bytes=656, ring=3, logical_capacity=90, gpu_slots=64, host_slots=64,
                 max_sets=3, max_k=20)
    try:
        for g in range(2):
            eng.append(g, rng.permutation(90).astype(np.int32)[:0], np.zeros((0, 3, 656), np.uint8))
            eng.append(g, np.arange(90, dtype=np.int32), rows[g])
        for t in range(3):
            sels = [selection(rng, 90, 3, 20, 2) for _ in range(2)]
            dev = [torch.from_numpy(x).cuda() for x in sels]
            for g in range(2):
                eng.step(g, dev[g])
            for layer in range(3):
                for g in (1, 0):
                    q = queries(rng, fmt, 3, 7)
                    out, lse = eng.attend(g, layer, dev[g], q, fmt)
                    check(fmt, rows[g], layer, sels[g], q, 1 / 24, out, lse, "bf16")
        eng.sync()
    finally:
        eng.close()


def test_a_stream_of_another_device_is_refused():
    import torch
    from serving_pb_lru_amd import rotate

    class Elsewhere:
        cuda_stream, device = 0, torch.device("cuda", 1)
    with pytest.raises(ValueError):
        rotate(torch.zeros((1, 1, 64), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), stream=Elsewhere())


@pytest.mark.parametrize("address,name", [(1 << 20, "ERANGE"), (-2, "ERANGE"), (59, "ENOTRESIDENT")])
def test_device_errors_are_latched(address, name):
    import torch
    from serving_pb_lru_amd import UlaError, latent_rows
    rng = np.random.default_rng(16)
    fmt = latent_rows()
    rows = latent_rows_of(rng, 60, 1)
    with Opened(fmt, rows, selection(rng, 30, 2, 24), gpu_slots=40, host_slots=40) as o:
        q = queries(rng, fmt, 2, 4)
        wrong, left = o.sel.copy(), o.sel.copy()
        wrong[0, 1], left[0, 1] = address, -1
        out, lse = o.attend(q, wrong)
        assert pytest.raises(UlaError, o.eng.sync).value.name == name
        o.check(q, out, lse, left)
        assert pytest.raises(UlaError, o.attend, q).value.name == "ESTATE"   # poisoned from here on
