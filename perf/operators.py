"""The operators that work on KV rows held in 8 bits, as measurable cases.

Five operators around the residency engine's rows: attention of each selection set
over the engine's rows in the latent format (512 e4m3 channels with a scale for
every 128, 64 bf16 rotary channels) and in the heads format (keys and values in
e4m3 with a scale for each block of tokens and head), the writer of such rows,
rotary positions with one to three axes, and the copying, renumbering and freeing
of entries. Each case is a dict of plain values; `run` computes it with the
engine's kernels (`own`) or in plain torch operations in 32 bits.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

LATENT, GROUP, ROPE, LATENT_ROW = 512, 128, 64, 656
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # a decode step of four short requests with few query heads: latency
        dict(name="latent_s4_k256_h16", op="latent", requests=4, drafts=0, k=256, heads=16, layers=1,
             context=4096, pad=0, type="bf16"),
        # 16 long requests, one of three layers that share the selection, all heads on this card
        dict(name="latent_s16_k2048_h128_l3", op="latent", requests=16, drafts=0, k=2048, heads=128, layers=3,
             context=16384, pad=0, type="bf16"),
        # a full batch: every request's 2048 selected positions, cold in the pool
        dict(name="latent_s256_k2048_h64", op="latent", requests=256, drafts=0, k=2048, heads=64, layers=1,
             context=4096, pad=0, type="bf16"),
        # speculative verify: a base and two draft sets per request that share nine tenths of their
        # positions, some entries of every set padding and one request's sets all padding
        dict(name="latent_s384_k2047_h128_pad", op="latent", requests=128, drafts=2, k=2047, heads=128, layers=1,
             context=8192, pad=61, type="fp16"),
        # grouped queries over per-token heads rows, 16 requests
        dict(name="heads_s16_k2048_g4_d128", op="heads", requests=16, k=2048, heads=32, kv_heads=8, head_dim=128,
             block=1, context=16384, pad=0, type="bf16"),
        # block-sparse selection: an entry is a block of 8 tokens with one scale per head, the last of them partly filled
        dict(name="heads_s64_k500_b8_d64", op="heads", requests=64, k=500, heads=24, kv_heads=2, head_dim=64,
             block=8, context=1500, pad=7, type="fp16"),
        # the rows that one decode step appends
        dict(name="pack_n64_l3", op="pack", n=64, layers=3, axes=1, interleaved=True, type="bf16"),
        # the rows of a prompt with images: three position axes
        dict(name="pack_n65536_axes3", op="pack", n=65536, layers=1, axes=3, interleaved=False, type="bf16"),
        # the rotary part of one decode step's queries
        dict(name="rotate_n16_h128", op="rotate", n=16, heads=128, dim=64, axes=1, interleaved=True,
             inverse=False, type="bf16"),
        # the queries of a prompt of video tokens, whole heads rotated, and their way back
        dict(name="rotate_n8191_h32_axes3", op="rotate", n=8191, heads=32, dim=128, axes=3, interleaved=False,
             inverse=True, type="fp32"),
        # a short prefix forked, moved down over a hole and freed again
        dict(name="cache_n257_l3", op="cache", n=257, layers=3, gap=129, context=4096),
        # a whole request's history
        dict(name="cache_n65536_l3", op="cache", n=65536, layers=3, gap=1000, context=131072),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["latent", "latent", "latent", "heads", "heads", "pack", "rotate", "cache"])
    if op == "latent":
        k, requests, heads = _log(rng, 1, 2048), _log(rng, 1, 256), _log(rng, 1, 128)
        return dict(op=op, requests=requests, drafts=rng.choice([0, 0, 2]) if requests <= 120 else 0, k=k, heads=heads,
                    layers=rng.choice([1, 1, 3]) if requests * k <= 1 << 17 else 1, context=2 * k + _log(rng, 1, 2048),
                    pad=rng.choice([0, 0, k // 7]), type=rng.choice(["bf16", "fp16"]))
    if op == "heads":
        dim, block, kv = rng.choice([64, 128]), rng.choice([1, 1, 2, 4, 8, 16]), rng.randint(1, 8)
        block = min(block, 1024 // dim)                            # a row holds at most 4096 bytes
        kv = max(1, min(kv, (4096 - 80) // (2 * dim * block)))
        k = max(1, _log(rng, 1, 2048) // block)
        return dict(op=op, requests=_log(rng, 1, 64), k=k, heads=kv * _log(rng, 1, 16), kv_heads=kv, head_dim=dim,
                    block=block, context=2 * k + _log(rng, 1, 1024), pad=rng.choice([0, 0, k // 7]),
                    type=rng.choice(["bf16", "fp16"]))
    if op == "pack":
        layers, kind = rng.choice([1, 1, 3]), rng.choice(["bf16", "fp16", "fp32"])
        return dict(op=op, n=_log(rng, 1, 65536 // (layers * (2 if kind == "fp32" else 1))), layers=layers,
                    axes=rng.choice([0, 1, 2, 3]), interleaved=rng.random() < 0.5, type=kind)
    if op == "rotate":
        n = _log(rng, 1, 8191)
        return dict(op=op, n=n, heads=min(_log(rng, 1, 128), 8191 * 32 // n), dim=rng.choice([64, 128]),
                    axes=rng.randint(1, 3), interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5,
                    type=rng.choice(["bf16", "fp16", "fp32"]))
    n = _log(rng, 1, 65536)
    return dict(op=op, n=n, layers=rng.randint(1, 3), gap=_log(rng, 1, 4096), context=n + _log(rng, 1, 8192))


# ---- inputs --------------------------------------------------------------------

def _sections(axes, pairs):
    """Frequency pairs of each axis: all for one, else a share for time and the rest for the picture's axes."""
    if axes == 1:
        return (pairs,)
    first = pairs // 4
    rest = pairs - first
    return (first, rest) if axes == 2 else (first, rest // 2, rest - rest // 2)


def _axis(sections):
    """The axis that each frequency pair turns by."""
    return torch.tensor([a for a, width in enumerate(sections) for _ in range(width)], device="cuda")


def _positions(n, axes, gen):
    """Positions along a sequence of up to 128K tokens: time anywhere, rows and columns of a picture."""
    cols = [torch.randint(0, 131072, (n,), device="cuda", generator=gen)]
    cols += [torch.randint(0, 4096, (n,), device="cuda", generator=gen) for _ in range(axes - 1)]
    return torch.stack(cols, 1).to(torch.int32)


def _magnitudes(shape, gen):
    """Activations' sizes differ from token to token and group to group by a few powers of two."""
    return torch.exp2(torch.randn(shape, device="cuda", generator=gen))


def _heads_row(case):
    used = 2 * case["kv_heads"] * case["block"] * case["head_dim"] + 8 * case["kv_heads"] + 4
    return (used + 15) // 16 * 16


def _latent_rows(n, gen):
    """n rows as bytes [n][656]: 512 e4m3 | 64 bf16 | 4 fp32 scales."""
    vals = torch.randn((n, LATENT), device="cuda", generator=gen).mul_(120).clamp_(-E4M3_MAX, E4M3_MAX)
    rope = torch.randn((n, ROPE), device="cuda", generator=gen).to(torch.bfloat16)
    scales = _magnitudes((n, LATENT // GROUP), gen) / 120
    return torch.cat([vals.to(torch.float8_e4m3fn).view(torch.uint8), rope.view(torch.uint8), scales.view(torch.uint8)], 1)


def _heads_rows(case, n, gen):
    """n rows as bytes: keys e4m3 [kv_heads][block][dim] | values the same | key scales fp32 [kv_heads] | value
    scales | tokens in the block int32 | zeros to a multiple of 16."""
    h, t, d = case["kv_heads"], case["block"], case["head_dim"]
    vals = torch.randn((n, 2 * h * t * d), device="cuda", generator=gen).mul_(120).clamp_(-E4M3_MAX, E4M3_MAX)
    scales = _magnitudes((n, 2 * h), gen) / 120
    count = torch.full((n, 1), t, dtype=torch.int32, device="cuda")
    if t > 1:
        count[::5] = torch.randint(1, t + 1, (len(count[::5]), 1), device="cuda", generator=gen, dtype=torch.int32)
    pad = torch.zeros((n, _heads_row(case) - 2 * h * t * d - 8 * h - 4), dtype=torch.uint8, device="cuda")
    return torch.cat([vals.to(torch.float8_e4m3fn).view(torch.uint8), scales.view(torch.uint8),
                      count.view(torch.uint8), pad], 1)


def _selection(case, gen):
    """int32 [sets][k]: each request's set picks distinct positions of its own context; a draft set replaces the
    last tenth of the base set's; -1 is padding, and with padding the last request has nothing but that."""
    r, k, c = case["requests"], case["k"], case["context"]
    drafts = case.get("drafts", 0)
    fresh = k // 10
    pick = torch.rand((r, c), device="cuda", generator=gen).topk(k + drafts * fresh, dim=1).indices
    sets = [pick[:, :k]] + [torch.cat([pick[:, :k - fresh], pick[:, k + i * fresh:k + (i + 1) * fresh]], 1)
                            for i in range(drafts)]
    sel = torch.stack(sets, 1) + (torch.arange(r, device="cuda") * c)[:, None, None]
    if case["pad"]:
        sel[:, :, (k - case["pad"]) // 2:(k + case["pad"]) // 2] = -1
        sel[-1] = -1
    return sel.reshape(r * (1 + drafts), k).to(torch.int32).contiguous()


def _engine(case, entries, layers, row_bytes, sets, k):
    from serving_pb_lru_amd import Engine
    return Engine(num_groups=1, layers=layers, row_bytes=row_bytes, ring=8, logical_capacity=entries,
                  gpu_slots=entries, host_slots=0, max_sets=sets, max_k=k, max_append=min(entries, 65536))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 17)
    s = dict(case)
    op = case["op"]
    if op in ("latent", "heads"):
        entries, layers = case["requests"] * case["context"], case.get("layers", 1)
        width = LATENT + ROPE if op == "latent" else case["head_dim"]
        s["sel"] = _selection(case, gen)
        q = torch.randn((len(s["sel"]), case["heads"], width), device="cuda", generator=gen)
        s["q"] = q.to(TYPES[case["type"]])
        s["scale"] = 1.0 / math.sqrt(width)
        part = 1 << 18
        rows = torch.cat([_latent_rows(min(part, entries * layers - i), gen) if op == "latent" else
                          _heads_rows(case, min(part, entries * layers - i), gen)
                          for i in range(0, entries * layers, part)]).view(entries, layers, -1)
        s["layer"] = layers - 1
        if own:
            from serving_pb_lru_amd import head_rows, latent_rows
            s["fmt"] = latent_rows() if op == "latent" else head_rows(case["kv_heads"], case["head_dim"], case["block"])
            s["engine"] = _engine(case, entries, layers, rows.shape[2], *s["sel"].shape)
            s["engine"].append(0, np.arange(entries, dtype=np.int32), rows)
            s["engine"].step(0, s["sel"])
            s["engine"].sync()
        else:
            s["rows"] = rows[:, layers - 1].contiguous()
    elif op == "pack":
        n, layers = case["n"], case["layers"]
        mags = _magnitudes((n, layers, LATENT // GROUP, 1), gen)
        latent = torch.randn((n, layers, LATENT // GROUP, GROUP), device="cuda", generator=gen) * mags
        s["latent"] = latent.reshape(n, layers, LATENT).to(TYPES[case["type"]])
        s["rope"] = torch.randn((n, layers, ROPE), device="cuda", generator=gen).to(TYPES[case["type"]])
        if case["axes"]:
            s["positions"] = _positions(n, case["axes"], gen)
            s["sections"] = _sections(case["axes"], ROPE // 2)
            s["axis"] = _axis(s["sections"])
        if own:
            from serving_pb_lru_amd import latent_rows
            s["fmt"] = latent_rows()
    elif op == "rotate":
        s["x"] = torch.randn((case["n"], case["heads"], case["dim"]), device="cuda", generator=gen).to(TYPES[case["type"]])
        s["positions"] = _positions(case["n"], case["axes"], gen)
        s["sections"] = _sections(case["axes"], case["dim"] // 2)
        s["axis"] = _axis(s["sections"])
    else:
        n, layers, context, gap = case["n"], case["layers"], case["context"], case["gap"]
        entries = context + gap + n
        rows = torch.randint(0, 256, (context, layers, LATENT_ROW), device="cuda", generator=gen, dtype=torch.uint8)
        s["src"], s["dst"], s["to"] = context - n, context + gap, context
        if own:
            s["sel"] = torch.arange(context, context + n, device="cuda", dtype=torch.int32).view(1, n)
            s["gone"] = np.arange(context, context + n, dtype=np.int32)
            s["engine"] = _engine(case, entries, layers, LATENT_ROW, 1, n)
            s["engine"].append(0, np.arange(context, dtype=np.int32), rows)
            s["engine"].step(0, torch.arange(min(n, context), device="cuda", dtype=torch.int32).view(1, -1))
            s["engine"].sync()
        else:
            s["pool"] = torch.zeros((entries, layers * LATENT_ROW), dtype=torch.uint8, device="cuda")
            s["pool"][:context] = rows.view(context, -1)
            s["map"] = torch.full((entries,), -1, dtype=torch.int64, device="cuda")
            s["map"][:context] = torch.arange(context, device="cuda")
            s["owner"] = s["map"].clone()
    return s


# ---- the plain forms -----------------------------------------------------------

def _plain_softmax(logits, values):
    """Rows of `logits` whose entries are all -inf give zeros and a log-sum of -inf."""
    top = logits.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    weights = torch.exp(logits - top)
    total = weights.sum(-1, keepdim=True)
    out = torch.matmul(weights, values) / torch.where(total > 0, total, torch.ones_like(total))
    return out, (top + torch.log(total)).squeeze(-1)


def _plain_latent(s):
    sel = s["sel"].long()
    rows = s["rows"][sel.clamp(min=0)]
    scales = rows[..., LATENT + 2 * ROPE:].contiguous().view(torch.float32)
    latent = rows[..., :LATENT].view(torch.float8_e4m3fn).float().view(*sel.shape, LATENT // GROUP, GROUP)
    latent = (latent * scales[..., None]).view(*sel.shape, LATENT)
    rope = rows[..., LATENT:LATENT + 2 * ROPE].contiguous().view(torch.bfloat16).float()
    logits = torch.matmul(s["q"].float(), torch.cat([latent, rope], -1).transpose(1, 2)) * s["scale"]
    logits = logits.masked_fill((sel < 0)[:, None, :], -math.inf)
    out, lse = _plain_softmax(logits, latent)
    return out.to(s["q"].dtype), lse


def _plain_heads(s):
    sel = s["sel"].long()
    sets, k = sel.shape
    h, t, d = s["kv_heads"], s["block"], s["head_dim"]
    rows = s["rows"][sel.clamp(min=0)]
    part = h * t * d
    scales = rows[..., 2 * part:2 * part + 8 * h].contiguous().view(torch.float32).view(sets, k, 2, h, 1, 1)
    count = rows[..., 2 * part + 8 * h:2 * part + 8 * h + 4].contiguous().view(torch.int32)
    kv = rows[..., :2 * part].view(torch.float8_e4m3fn).float().view(sets, k, 2, h, t, d) * scales
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, sets, h, k * t, d)
    q = s["q"].float().view(sets, h, -1, d)
    logits = torch.matmul(q, kv[0].transpose(-1, -2)) * s["scale"]
    empty = (sel < 0)[:, :, None] | (torch.arange(t, device="cuda") >= count)
    logits = logits.masked_fill(empty.view(sets, 1, 1, k * t), -math.inf)
    out, lse = _plain_softmax(logits, kv[1])
    return out.reshape(s["q"].shape).to(s["q"].dtype), lse.reshape(sets, -1)


def _plain_rotate(x, positions, axis, interleaved, inverse):
    """x [..., tokens in front, dim] with positions [tokens][axes]; angles in 64 bits, the product in 32."""
    dim = x.shape[-1]
    freq = 10000.0 ** (-2.0 * torch.arange(dim // 2, device="cuda", dtype=torch.float64) / dim)
    angle = positions.double()[:, axis] * freq
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if inverse:
        sin = -sin
    v = x.float()
    a, b = (v[..., 0::2], v[..., 1::2]) if interleaved else (v[..., :dim // 2], v[..., dim // 2:])
    lo, hi = a * cos - b * sin, a * sin + b * cos
    return torch.stack([lo, hi], -1).flatten(-2) if interleaved else torch.cat([lo, hi], -1)


def _plain_pack(s):
    x = s["latent"].float().view(s["n"], s["layers"], LATENT // GROUP, GROUP)
    scales = (x.abs().amax(-1) / E4M3_MAX).clamp(min=2.0 ** -126)
    vals = (x / scales[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    rope = _plain_rotate(s["rope"], s["positions"], s["axis"], s["interleaved"], False) if s["axes"] else s["rope"]
    return torch.cat([vals.view(torch.uint8).view(s["n"], s["layers"], LATENT),
                      rope.to(torch.bfloat16).view(torch.uint8), scales.view(torch.uint8)], -1)


def _plain_cache(s):
    n, src, dst, to = s["n"], s["src"], s["dst"], s["to"]
    slots = (s["owner"] < 0).nonzero()[:n, 0]                      # the lowest free slots
    s["pool"][slots] = s["pool"][s["map"][src:src + n]]             # fork
    s["map"][dst:dst + n] = slots
    s["owner"][slots] = torch.arange(dst, dst + n, device="cuda")
    moved = s["map"][dst:dst + n].clone()                           # rename
    s["map"][dst:dst + n] = -1
    s["map"][to:to + n] = moved
    s["owner"][moved] = torch.arange(to, to + n, device="cuda")
    rows = s["pool"][s["map"][to:to + n]]                           # read
    s["owner"][s["map"][to:to + n]] = -1                            # free
    s["map"][to:to + n] = -1
    return rows.view(1, n, s["layers"], LATENT_ROW).permute(2, 0, 1, 3).contiguous()


def _values_of(rows):
    """A packed row's contents as values: e4m3 channels, bf16 rotary channels, scales."""
    return (rows[..., :LATENT].view(torch.float8_e4m3fn), rows[..., LATENT:LATENT + 2 * ROPE].view(torch.bfloat16),
            rows[..., LATENT + 2 * ROPE:].view(torch.float32))


def run(state):
    s, op = state, state["op"]
    if op in ("latent", "heads"):
        if own:
            return s["engine"].attend(0, s["layer"], s["sel"], s["q"], s["fmt"], scale=s["scale"])
        return _plain_latent(s) if op == "latent" else _plain_heads(s)
    if op == "pack":
        if own:
            from serving_pb_lru_amd import pack_rows
            return _values_of(pack_rows(s["fmt"], s["latent"], s["rope"], positions=s.get("positions"),
                                        sections=s.get("sections"), interleaved=s["interleaved"]))
        return _values_of(_plain_pack(s))
    if op == "rotate":
        if own:
            from serving_pb_lru_amd import rotate
            return rotate(s["x"], s["positions"], s["sections"], interleaved=s["interleaved"], inverse=s["inverse"])
        return _plain_rotate(s["x"], s["positions"], s["axis"], s["interleaved"], s["inverse"]).to(s["x"].dtype)
    if own:
        eng = s["engine"]
        eng.fork(0, s["src"], s["dst"], s["n"])
        eng.rename(0, s["dst"], s["to"], s["n"])
        rows = eng.gather_layers(0, 0, s["layers"], s["sel"])
        eng.release(0, s["gone"])
        return rows
    return _plain_cache(s)


# ---- bytes and operations ------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("latent", "heads"):
        sets = case["requests"] * (1 + case.get("drafts", 0))
        full = case["requests"] - (1 if case["pad"] else 0)
        live = full * (case["k"] - case["pad"]) * (1 + case.get("drafts", 0))
        # the draft sets' rows that the base set has too are read once
        rows = full * (case["k"] - case["pad"] + case.get("drafts", 0) * (case["k"] // 10))
        width = LATENT + ROPE if op == "latent" else case["head_dim"]
        back = LATENT if op == "latent" else case["head_dim"]
        row = LATENT_ROW if op == "latent" else _heads_row(case)
        return dict(bytes=rows * row + sets * (4 * case["k"] + case["heads"] * (2 * width + 2 * back + 4)),
                    flops=2 * live * case.get("block", 1) * case["heads"] * (width + back))
    size = {"bf16": 2, "fp16": 2, "fp32": 4}.get(case.get("type"), 1)
    if op == "pack":
        rows = case["n"] * case["layers"]
        return dict(bytes=rows * (size * (LATENT + ROPE) + LATENT_ROW) + 4 * case["n"] * case["axes"], flops=4 * rows * LATENT)
    if op == "rotate":
        values = case["n"] * case["heads"] * case["dim"]
        return dict(bytes=2 * size * values + 4 * case["n"] * case["axes"], flops=3 * values)
    # the fork reads and writes the rows, the read back does so again; the map and owner words change
    return dict(bytes=4 * case["n"] * case["layers"] * LATENT_ROW + 24 * case["n"], flops=0)


# ---- 64 bits -------------------------------------------------------------------

def _exact_attention(q, keys, values, keep, scale):
    """q [sets][heads][width], keys and values [sets][heads][tokens][...], keep [sets][tokens]; all in 64 bits."""
    logits = (q[:, :, None, :] @ keys.transpose(2, 3))[:, :, 0] * scale
    logits = torch.where(keep[:, None], logits, torch.full_like(logits, -math.inf))
    lse = torch.logsumexp(logits, -1)
    share = torch.where(keep[:, None], torch.exp(logits - torch.nan_to_num(lse, neginf=0.0)[..., None]),
                        torch.zeros_like(logits))
    return (share[:, :, None, :] @ values)[:, :, 0], lse


def _e4m3_values(codes):
    """The values that e4m3 bytes stand for, from their fields."""
    c = codes.long()
    sign, exponent, fraction = 1 - 2 * (c >> 7), (c >> 3) & 15, (c & 7).double()
    normal = (1 + fraction / 8) * torch.exp2((exponent - 7).double())
    return sign * torch.where(exponent > 0, normal, fraction / 8 * 2.0 ** -6)


def _exact_rotate(x, positions, sections, interleaved, inverse):
    """Complex numbers turned by exp(i angle)."""
    dim = x.shape[-1]
    axis = [a for a, width in enumerate(sections) for _ in range(width)]
    freq = torch.exp(torch.arange(dim // 2, device="cuda", dtype=torch.float64) * (-2.0 * math.log(10000.0) / dim))
    angle = positions[:, axis].double() * freq * (-1.0 if inverse else 1.0)
    z = x.double()
    z = z.reshape(*x.shape[:-1], dim // 2, 2) if interleaved else z.reshape(*x.shape[:-1], 2, dim // 2).transpose(-1, -2)
    turned = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None]
    back = torch.view_as_real(turned)
    return (back if interleaved else back.transpose(-1, -2)).reshape(x.shape)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op == "cache":
        return None                      # bytes: the comparison of whole numbers says it all
    if op == "rotate":
        return _exact_rotate(s["x"], s["positions"], s["sections"], s["interleaved"], s["inverse"])
    if op == "pack":
        x = s["latent"].double().reshape(s["n"], s["layers"], LATENT // GROUP, GROUP)
        scales = torch.maximum(x.abs().amax(-1) / E4M3_MAX, torch.tensor(2.0 ** -126, device="cuda", dtype=torch.float64))
        rope = s["rope"].double()
        if s["axes"]:
            rope = _exact_rotate(rope, s["positions"], s["sections"], s["interleaved"], False)
        return ((x / scales[..., None]).reshape(s["n"], s["layers"], LATENT), rope, scales)
    outs = []
    sel = s["sel"].long()
    for i in range(len(sel)):            # one set at a time: 64 bits of a whole batch would not fit
        rows, keep = s["rows"][sel[i].clamp(min=0)], sel[i] >= 0
        q = s["q"][i].double()
        if op == "latent":
            parts = _e4m3_values(rows[:, :LATENT]).view(-1, LATENT // GROUP, GROUP)
            values = (parts * rows[:, LATENT + 2 * ROPE:].contiguous().view(torch.float32).double()[..., None]).view(-1, LATENT)
            keys = torch.cat([values, rows[:, LATENT:LATENT + 2 * ROPE].contiguous().view(torch.bfloat16).double()], 1)
            logits = q @ keys.t() * s["scale"]
            logits = torch.where(keep, logits, torch.full_like(logits, -math.inf))
            lse = torch.logsumexp(logits, -1)
            share = torch.where(keep, torch.exp(logits - torch.nan_to_num(lse, neginf=0.0)[:, None]), torch.zeros_like(logits))
            outs.append((share @ values, lse))
        else:
            h, t, d = s["kv_heads"], s["block"], s["head_dim"]
            codes = _e4m3_values(rows[:, :2 * h * t * d]).view(-1, 2, h, t, d)
            tail = rows[:, 2 * h * t * d:]
            scales = tail[:, :8 * h].contiguous().view(torch.float32).double().view(-1, 2, h, 1, 1)
            count = tail[:, 8 * h:8 * h + 4].contiguous().view(torch.int32)
            kv = (codes * scales).permute(1, 2, 0, 3, 4).reshape(2, h, -1, d)
            kv = kv.repeat_interleave(case["heads"] // h, dim=1)
            keep = (keep[:, None] & (torch.arange(t, device="cuda") < count)).reshape(1, -1)
            out, lse = _exact_attention(q[None], kv[0][None], kv[1][None], keep, s["scale"])
            outs.append((out[0], lse[0]))
    return tuple(torch.stack(o) for o in zip(*outs))
