"""The operators around speculative decoding and eviction by attention weight, as measurable cases.

Four operators beside those of perf/operators.py: norms of queries and keys with
the rotary turn in the same pass, attention of a tree of drafted tokens over the
selected rows of a request and over the drafted tokens' own rows, the softmax
weight that each selected entry got (summed over the queries and added to a score
for each address), and the entries of least score in ranges of addresses. Rows
are in the latent or the heads format of include/ula.h. Each case is a dict of
plain values; `run` computes it with the engine's kernels (`own`) or in plain
torch operations in 32 bits.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

LATENT, GROUP, ROPE, LATENT_ROW = 512, 128, 64, 656
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
SCORE_ONE = 2.0 ** 32                    # a weight of 1 in a score


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # the queries and keys of one decode step, 16 requests: latency
        dict(name="norm_n16_h32_kv8", op="norm", n=16, heads=32, kv_heads=8, dim=128, rotary=128, axes=1,
             interleaved=False, weights="same", type="bf16"),
        # a prompt with images, half of each head's channels turned, weights kept in 32 bits
        dict(name="norm_n8191_h32_kv4_half_axes3", op="norm", n=8191, heads=32, kv_heads=4, dim=128, rotary=64, axes=3,
             interleaved=True, weights="fp32", type="fp16"),
        # a few short requests verify a small tree with few query heads: latency
        dict(name="tree_latent_s4_t8_k256_h16", op="tree", rows="latent", requests=4, nodes=8, k=256, heads=16, layers=1,
             context=4096, pad=0, type="bf16"),
        # 16 long requests, chains and forks of eight drafted tokens, every head on this card, one of three layers
        dict(name="tree_latent_s16_t8_k2048_h128_l3", op="tree", rows="latent", requests=16, nodes=8, k=2048, heads=128,
             layers=3, context=8192, pad=0, type="bf16"),
        # a full batch with wide trees; some of every selection padding, one request without history
        dict(name="tree_latent_s61_t27_k1023_h64_pad", op="tree", rows="latent", requests=61, nodes=27, k=1023, heads=64,
             layers=1, context=4096, pad=61, type="fp16"),
        # grouped queries over per-token heads rows, trees of 16
        dict(name="tree_heads_s16_t16_k2048_g4_d128", op="tree", rows="heads", requests=16, nodes=16, k=2048, heads=32,
             kv_heads=8, head_dim=128, block=1, layers=1, context=16384, pad=0, type="bf16"),
        # block-sparse selection (entries of 8 tokens, the last partly filled), the largest trees
        dict(name="tree_heads_s32_t61_k500_b8_d64", op="tree", rows="heads", requests=32, nodes=61, k=500, heads=24,
             kv_heads=2, head_dim=64, block=8, layers=1, context=1500, pad=7, type="fp16"),
        # the weights of a small batch's decode step: latency
        dict(name="weigh_latent_s4_k256_h16", op="weigh", rows="latent", requests=4, k=256, heads=16, layers=1,
             context=4096, pad=0, type="bf16"),
        # the weights of a full batch's decode step
        dict(name="weigh_latent_s256_k2048_h64", op="weigh", rows="latent", requests=256, k=2048, heads=64, layers=1,
             context=4096, pad=61, type="bf16"),
        # grouped queries over per-token heads rows
        dict(name="weigh_heads_s16_k2048_g4_d128", op="weigh", rows="heads", requests=16, k=2048, heads=32, kv_heads=8,
             head_dim=128, block=1, layers=1, context=16384, pad=0, type="fp16"),
        # 16 requests give up 64 entries each of a short history
        dict(name="lightest_r16_l4096_n64", op="lightest", ranges=16, length=4096, n=64),
        # a few requests with a long history give up a thirtieth of it
        dict(name="lightest_r6_l131072_n4096", op="lightest", ranges=6, length=131072, n=4096),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _heads_sizes(rng):
    dim, block, kv = rng.choice([64, 128]), rng.choice([1, 1, 2, 4, 8, 16]), rng.randint(1, 8)
    block = min(block, 1024 // dim)                                # a row holds at most 4096 bytes
    kv = max(1, min(kv, (4096 - 80) // (2 * dim * block)))
    return dict(kv_heads=kv, head_dim=dim, block=block)


def draw(rng):
    op = rng.choice(["norm", "tree", "tree", "tree", "weigh", "weigh", "lightest"])
    if op == "norm":
        dim, kind = rng.choice([64, 96, 128, 192, 256]), rng.choice(["bf16", "fp16", "fp32"])
        n = _log(rng, 1, 8191)
        room = 8191 * 36 * 128 * 2 // (n * dim * (4 if kind == "fp32" else 2))
        heads = max(1, min(_log(rng, 1, 64), room))
        kv = rng.choice([0, max(1, heads // 4), heads])
        return dict(op=op, n=n, heads=heads, kv_heads=max(0, min(kv, room - heads)), dim=dim,
                    rotary=rng.choice([0, dim // 2, dim, dim]), axes=rng.randint(1, 3), interleaved=rng.random() < 0.5,
                    weights=rng.choice(["same", "fp32", "none"]), type=kind)
    if op in ("tree", "weigh"):
        kind = rng.choice(["latent", "latent", "heads"])
        c = dict(op=op, rows=kind, type=rng.choice(["bf16", "fp16"]))
        k, requests = _log(rng, 1, 2048), _log(rng, 1, 64 if op == "tree" else 256)
        if op == "tree":
            c["nodes"] = _log(rng, 1, 64)
        rows = c.get("nodes", 1)
        if kind == "latent":
            heads = _log(rng, 1, 128)
            most = 61 * 27 * 1023 * 64 if op == "tree" else 256 * 2048 * 64   # query rows x keys of the largest
            heads = max(1, min(heads, most // (requests * rows * k), 61 * 27 * 64 // (requests * rows)))
        else:
            c.update(_heads_sizes(rng))
            k = max(1, k // c["block"])
            heads = c["kv_heads"] * _log(rng, 1, 16)
            requests = min(requests, 64)
            most = 32 * 61 * 24 * 64                               # ... x head width
            while requests > 1 and requests * rows * heads * c["head_dim"] * max(4000, k * c["block"]) > 4000 * most:
                requests //= 2
        c.update(requests=requests, k=k, heads=heads, layers=rng.choice([1, 1, 3]) if requests * k <= 1 << 16 else 1,
                 context=2 * k + _log(rng, 1, 2048), pad=rng.choice([0, 0, k // 7]))
        return c
    length = _log(rng, 1, 131072)
    return dict(op=op, ranges=_log(rng, 1, min(512, 6 * 131072 // length)), length=length, n=_log(rng, 1, max(1, length // 4)))


# ---- inputs --------------------------------------------------------------------

def _sections(axes, pairs):
    """Frequency pairs of each axis: all for one, else a share for time and the rest for the picture's axes."""
    if axes == 1:
        return (pairs,)
    first = pairs // 4
    rest = pairs - first
    return (first, rest) if axes == 2 else (first, rest // 2, rest - rest // 2)


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


def _codes(shape, gen):
    vals = torch.randn(shape, device="cuda", generator=gen).mul_(120).clamp_(-E4M3_MAX, E4M3_MAX)
    return vals.to(torch.float8_e4m3fn).view(torch.uint8)


def _latent_rows(n, gen):
    """n rows as bytes [n][656]: 512 e4m3 | 64 bf16 | 4 fp32 scales."""
    rope = torch.randn((n, ROPE), device="cuda", generator=gen).to(torch.bfloat16)
    scales = _magnitudes((n, LATENT // GROUP), gen) / 120
    return torch.cat([_codes((n, LATENT), gen), rope.view(torch.uint8), scales.view(torch.uint8)], 1)


def _heads_rows(case, count, gen):
    """Rows as bytes: keys e4m3 [kv_heads][block][dim] | values the same | key scales fp32 [kv_heads] | value
    scales | tokens in the block int32 (`count`, [n]) | zeros to a multiple of 16."""
    h, t, d = case["kv_heads"], case["block"], case["head_dim"]
    n = len(count)
    scales = _magnitudes((n, 2 * h), gen) / 120
    pad = torch.zeros((n, _heads_row(case) - 2 * h * t * d - 8 * h - 4), dtype=torch.uint8, device="cuda")
    return torch.cat([_codes((n, 2 * h * t * d), gen), scales.view(torch.uint8),
                      count.to(torch.int32)[:, None].contiguous().view(torch.uint8), pad], 1)


def _rows(case, n, gen):
    """n entries' rows: every fifth block of tokens partly filled."""
    if case["rows"] == "latent":
        return _latent_rows(n, gen)
    t = case["block"]
    count = torch.full((n,), t, device="cuda")
    if t > 1:
        count[::5] = torch.randint(1, t + 1, (len(count[::5]),), device="cuda", generator=gen)
    return _heads_rows(case, count, gen)


def _selection(case, gen):
    """int32 [requests][k]: each request picks distinct positions of its own context; -1 is padding, and with
    padding the last request has nothing but that."""
    r, k, c = case["requests"], case["k"], case["context"]
    sel = torch.rand((r, c), device="cuda", generator=gen).topk(k, dim=1).indices
    sel = sel + (torch.arange(r, device="cuda") * c)[:, None]
    if case["pad"]:
        sel[:, (k - case["pad"]) // 2:(k + case["pad"]) // 2] = -1
        sel[-1] = -1
    return sel.to(torch.int32).contiguous()


def _trees(case, gen):
    """int64 [requests][nodes]: bit j of a node for each drafted token on its way to the root, itself too. With
    padding the last request's last node sees nothing."""
    r, t = case["requests"], case["nodes"]
    parent = (torch.rand((r, t), device="cuda", generator=gen) * torch.arange(t, device="cuda")).long()
    parent = torch.where(torch.rand((r, t), device="cuda", generator=gen) < 0.5, torch.arange(t, device="cuda") - 1, parent)
    seen = torch.zeros((r, t), dtype=torch.int64, device="cuda")
    for i in range(t):
        above = seen.gather(1, parent[:, i:i + 1].clamp(min=0))[:, 0] if i else torch.zeros_like(seen[:, 0])
        seen[:, i] = above | torch.tensor(1 << i if i < 63 else -(1 << 63), device="cuda")
    if case["pad"]:
        seen[-1, -1] = 0
    return seen


def _engine(case, rows, sel):
    from serving_pb_lru_amd import Engine
    entries, layers, row_bytes = rows.shape
    eng = Engine(num_groups=1, layers=layers, row_bytes=row_bytes, ring=8, logical_capacity=entries, gpu_slots=entries,
                 host_slots=0, max_sets=sel.shape[0], max_k=sel.shape[1], max_append=min(entries, 65536))
    eng.append(0, np.arange(entries, dtype=np.int32), rows)
    eng.step(0, sel)
    eng.sync()
    return eng


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 29)
    s = dict(case)
    op = case["op"]
    if op in ("tree", "weigh"):
        latent = case["rows"] == "latent"
        width = LATENT + ROPE if latent else case["head_dim"]
        entries, layers = case["requests"] * case["context"], case["layers"]
        s["sel"] = _selection(case, gen)
        nodes = (case["nodes"],) if op == "tree" else ()
        q = torch.randn((case["requests"], *nodes, case["heads"], width), device="cuda", generator=gen)
        s["q"] = q.to(TYPES[case["type"]])
        s["scale"], s["layer"] = 1.0 / math.sqrt(width), layers - 1
        part = 1 << 18
        rows = torch.cat([_rows(case, min(part, entries * layers - i), gen)
                          for i in range(0, entries * layers, part)]).view(entries, layers, -1)
        if op == "tree":
            s["visible"] = _trees(case, gen)
            t, b = case["nodes"], 1 if latent else case["block"]
            blocks = (t + b - 1) // b
            if latent:
                drafts = _latent_rows(case["requests"] * t * layers, gen)
            else:                                # the last block holds what is left of the tree
                count = (t - torch.arange(blocks, device="cuda") * b).clamp(max=b)
                drafts = _heads_rows(case, count[None, :, None].expand(case["requests"], blocks, layers).reshape(-1), gen)
            s["drafts"] = drafts.view(case["requests"] * blocks, layers, -1)
        else:
            chosen = rows[:, layers - 1][s["sel"].long().clamp(min=0)]
            s["lse"] = _plain_lse(s, chosen)
            # what earlier steps left: most entries have had little weight
            s["scores"] = (torch.exp(2 * torch.randn(entries, device="cuda", generator=gen)) * SCORE_ONE / 64).long()
        if own:
            from serving_pb_lru_amd import head_rows, latent_rows
            s["fmt"] = latent_rows() if latent else head_rows(case["kv_heads"], case["head_dim"], case["block"])
            s["engine"] = _engine(case, rows, s["sel"])
        else:
            s["cache"] = rows[:, layers - 1].contiguous()
            if op == "weigh":
                s["scores"] = s["scores"].double() / SCORE_ONE
    elif op == "norm":
        n, heads, kv, dim = case["n"], case["heads"], case["kv_heads"], case["dim"]
        # one projection's output: queries, keys and values of a token side by side
        x = torch.randn((n, heads + 2 * kv, dim), device="cuda", generator=gen) * _magnitudes((n, heads + 2 * kv, 1), gen)
        x = x.to(TYPES[case["type"]])
        s["q"], s["k"] = x[:, :heads], x[:, heads:heads + kv] if kv else None
        weights = 1 + 0.3 * torch.randn((2, dim), device="cuda", generator=gen)
        weights = weights if case["weights"] == "fp32" else weights.to(x.dtype)
        s["q_weight"], s["k_weight"] = (weights[0], weights[1] if kv else None) if case["weights"] != "none" else (None, None)
        s["positions"] = _positions(n, case["axes"], gen) if case["rotary"] else None
        s["sections"] = _sections(case["axes"], case["rotary"] // 2) if case["rotary"] else None
        if case["rotary"]:
            s["axis"] = torch.tensor([a for a, width in enumerate(s["sections"]) for _ in range(width)], device="cuda")
    else:
        ranges, length = case["ranges"], case["length"]
        score = torch.exp(2 * torch.randn(ranges * length, device="cuda", generator=gen)) * SCORE_ONE / 64
        luck = torch.rand(ranges * length, device="cuda", generator=gen)
        score = torch.where(luck < 0.1, torch.zeros_like(score), score).long()       # appended since, no weight yet
        s["scores"] = torch.where(luck > 0.95, torch.full_like(score, -1), score)    # given up before
        # all but a request's first four entries and a recent tail of its own length
        keep = np.random.default_rng(int(seed)).integers(0, max(1, length // 8), ranges)
        base = np.arange(ranges, dtype=np.int64) * length
        s["first"] = (base + min(4, length - 1)).astype(np.int32)
        s["last"] = (base + length - keep).astype(np.int32)
        s["last"] = np.maximum(s["first"], s["last"])
        s["count"] = np.full(ranges, case["n"], np.int32)
        s["count"][::3] = max(1, case["n"] // 2)
        if not own:
            s["ends"] = torch.from_numpy(np.stack([s["first"] - base, s["last"] - base, s["count"]], 1)).cuda()
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


def _latent_parts(rows):
    """Keys [..., 576] and values [..., 512] of latent rows."""
    lead = rows.shape[:-1]
    scales = rows[..., LATENT + 2 * ROPE:].contiguous().view(torch.float32)
    latent = rows[..., :LATENT].view(torch.float8_e4m3fn).float().view(*lead, LATENT // GROUP, GROUP)
    latent = (latent * scales[..., None]).view(*lead, LATENT)
    rope = rows[..., LATENT:LATENT + 2 * ROPE].contiguous().view(torch.bfloat16).float()
    return torch.cat([latent, rope], -1), latent


def _heads_parts(s, rows):
    """Keys and values [2][sets][kv_heads][tokens][dim] of heads rows [sets][k][bytes], tokens in use [sets][tokens]."""
    sets, k = rows.shape[:2]
    h, t, d = s["kv_heads"], s["block"], s["head_dim"]
    part = h * t * d
    scales = rows[..., 2 * part:2 * part + 8 * h].contiguous().view(torch.float32).view(sets, k, 2, h, 1, 1)
    count = rows[..., 2 * part + 8 * h:2 * part + 8 * h + 4].contiguous().view(torch.int32)
    kv = rows[..., :2 * part].view(torch.float8_e4m3fn).float().view(sets, k, 2, h, t, d) * scales
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, sets, h, k * t, d)
    return kv, (torch.arange(t, device="cuda") < count).view(sets, k * t)


def _plain_tree(s):
    sel = s["sel"].long()
    sets, k = sel.shape
    t = s["nodes"]
    drafts = s["drafts"][:, s["layer"]].view(sets, -1, s["drafts"].shape[-1])
    rows = torch.cat([s["cache"][sel.clamp(min=0)], drafts], 1)
    seen = (s["visible"][:, :, None] >> torch.arange(t, device="cuda")) & 1 > 0           # [sets][nodes][drafted]
    q = s["q"].float()
    if s["rows"] == "latent":
        keys, values = _latent_parts(rows)
        keep = torch.cat([(sel >= 0)[:, None].expand(-1, t, -1), seen], 2)[:, :, None]
        logits = torch.matmul(q.view(sets, t * s["heads"], -1), keys.transpose(1, 2)) * s["scale"]
        logits = logits.view(sets, t, s["heads"], -1).masked_fill(~keep, -math.inf)
        out, lse = _plain_softmax(logits.view(sets, t * s["heads"], -1), values)
        return out.view(sets, t, s["heads"], -1).to(s["q"].dtype), lse.view(sets, t, s["heads"])
    b, h = s["block"], s["kv_heads"]
    kv, used = _heads_parts(s, rows)
    history = (sel >= 0)[:, :, None].expand(-1, -1, b).reshape(sets, 1, k * b).expand(-1, t, -1)
    tail = torch.zeros((sets, t, kv.shape[3] - k * b - t), dtype=torch.bool, device="cuda")
    keep = torch.cat([history, seen, tail], 2) & used[:, None]                            # [sets][nodes][tokens]
    g = s["heads"] // h
    qh = q.view(sets, t, h, g, -1).transpose(1, 2).reshape(sets, h, t * g, -1)
    logits = (torch.matmul(qh, kv[0].transpose(-1, -2)) * s["scale"]).view(sets, h, t, g, -1)
    logits = logits.masked_fill(~keep[:, None, :, None], -math.inf)
    out, lse = _plain_softmax(logits.view(sets, h, t * g, -1), kv[1])
    out = out.view(sets, h, t, g, -1).transpose(1, 2).reshape(s["q"].shape)
    return out.to(s["q"].dtype), lse.view(sets, h, t, g).transpose(1, 2).reshape(sets, t, s["heads"])


def _plain_logits(s, rows):
    """[sets][heads][tokens], -inf for padding and tokens out of use; the tokens of an entry."""
    sel = s["sel"]
    sets, k = sel.shape
    q = s["q"].float()
    if s["rows"] == "latent":
        keys, _ = _latent_parts(rows)
        logits = torch.matmul(q, keys.transpose(1, 2)) * s["scale"]
        return logits.masked_fill((sel < 0)[:, None], -math.inf), 1
    kv, used = _heads_parts(s, rows)
    logits = torch.matmul(q.view(sets, s["kv_heads"], -1, q.shape[-1]), kv[0].transpose(-1, -2)) * s["scale"]
    keep = used & (sel >= 0)[:, :, None].expand(-1, -1, s["block"]).reshape(sets, -1)
    return logits.view(sets, s["heads"], -1).masked_fill(~keep[:, None], -math.inf), s["block"]


def _plain_lse(s, rows):
    logits, _ = _plain_logits(s, rows)
    return torch.logsumexp(logits, -1)


def _plain_weigh(s):
    logits, block = _plain_logits(s, s["cache"][s["sel"].long().clamp(min=0)])
    lse = s["lse"][..., None]
    shares = torch.exp(logits - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)).sum(1)
    shares = shares.view(*s["sel"].shape, block).sum(-1)
    s["scores"].index_add_(0, s["sel"].long().clamp(min=0).view(-1), shares.double().view(-1))    # padding adds 0
    return shares, s["scores"].float()


def _plain_norm(s, x, weight):
    v = x.float()
    v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    if weight is not None:
        v = v * weight.float()
    r = s["rotary"]
    if r:
        freq = 10000.0 ** (-2.0 * torch.arange(r // 2, device="cuda", dtype=torch.float64) / r)
        angle = s["positions"].double()[:, s["axis"]] * freq
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        turn = v[..., :r]
        a, b = (turn[..., 0::2], turn[..., 1::2]) if s["interleaved"] else (turn[..., :r // 2], turn[..., r // 2:])
        lo, hi = a * cos - b * sin, a * sin + b * cos
        turn = torch.stack([lo, hi], -1).flatten(-2) if s["interleaved"] else torch.cat([lo, hi], -1)
        v = torch.cat([turn, v[..., r:]], -1)
    return v.to(x.dtype)


def _plain_lightest(s):
    ranges, length, n = s["ranges"], s["length"], s["n"]
    at = torch.arange(length, device="cuda")
    first, last, count = s["ends"][:, 0:1], s["ends"][:, 1:2], s["ends"][:, 2:3]
    scores = s["scores"].view(ranges, length)
    out_of_it = (at < first) | (at >= last) | (scores < 0)
    order = torch.sort(scores.masked_fill(out_of_it, torch.iinfo(torch.int64).max), dim=1, stable=True).indices[:, :n]
    live = (~out_of_it).sum(1, keepdim=True)
    kept = torch.arange(order.shape[1], device="cuda") < torch.minimum(live, count)
    chosen = torch.where(kept, order, torch.full_like(order, length)).sort(1).values
    address = chosen + (torch.arange(ranges, device="cuda") * length)[:, None]
    picked = torch.full((ranges, n), -1, dtype=torch.int32, device="cuda")
    picked[:, :order.shape[1]] = torch.where(chosen < length, address, torch.full_like(address, -1)).to(torch.int32)
    return picked


def run(state):
    s, op = state, state["op"]
    if op == "tree":
        if own:
            return s["engine"].attend_tree(0, s["layer"], s["sel"], s["q"], s["fmt"], s["drafts"], s["visible"],
                                           scale=s["scale"])
        return _plain_tree(s)
    if op == "weigh":
        if own:
            shares = s["engine"].weigh(0, s["layer"], s["sel"], s["q"], s["lse"], s["fmt"], scores=s["scores"],
                                       scale=s["scale"])
            return shares, s["scores"] * (1 / SCORE_ONE)
        return _plain_weigh(s)
    if op == "norm":
        if own:
            from serving_pb_lru_amd import norm_rotate
            return norm_rotate(s["q"], s["k"], s["q_weight"], s["k_weight"], positions=s["positions"],
                               sections=s["sections"], interleaved=s["interleaved"], rotary=s["rotary"], eps=EPS)
        return _plain_norm(s, s["q"], s["q_weight"]), None if s["k"] is None else _plain_norm(s, s["k"], s["k_weight"])
    if own:
        from serving_pb_lru_amd import lightest
        return lightest(s["scores"], s["first"], s["last"], s["count"], most=s["n"])
    return _plain_lightest(s)


# ---- bytes and operations ------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("tree", "weigh"):
        latent = case["rows"] == "latent"
        width, back = (LATENT + ROPE, LATENT) if latent else (case["head_dim"],) * 2
        row, block = (LATENT_ROW, 1) if latent else (_heads_row(case), case["block"])
        live = (case["requests"] - (1 if case["pad"] else 0)) * (case["k"] - case["pad"])
        sel = 4 * case["requests"] * case["k"]
        if op == "tree":
            t = case["nodes"]
            queries = case["requests"] * t * case["heads"]
            drafts = case["requests"] * (t + block - 1) // block
            return dict(bytes=(live + drafts) * row + sel + queries * (2 * width + 2 * back + 4) + 8 * case["requests"] * t,
                        flops=2 * (live * block * t + case["requests"] * t * t) * case["heads"] * (width + back))
        used = row if latent else case["kv_heads"] * (block * width + 4) + 4     # heads rows: the keys alone
        # shares out, scores read and written where something is added
        return dict(bytes=live * used + 2 * sel + case["requests"] * case["heads"] * (2 * width + 4) + 16 * live,
                    flops=2 * live * block * case["heads"] * width)
    if op == "norm":
        size = 4 if case["type"] == "fp32" else 2
        values = case["n"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return dict(bytes=2 * size * values + 4 * case["n"] * case["axes"], flops=7 * values)
    return dict(bytes=8 * case["ranges"] * case["length"] + 4 * case["ranges"] * case["n"],
                flops=case["ranges"] * case["length"])


# ---- 64 bits -------------------------------------------------------------------

def _e4m3_values(codes):
    """The values that e4m3 bytes stand for, from their fields."""
    c = codes.long()
    sign, exponent, fraction = 1 - 2 * (c >> 7), (c >> 3) & 15, (c & 7).double()
    normal = (1 + fraction / 8) * torch.exp2((exponent - 7).double())
    return sign * torch.where(exponent > 0, normal, fraction / 8 * 2.0 ** -6)


def _exact_kv(case, rows):
    """[(heads, keys, values)] of rows [n][bytes] and the tokens in use, one part for each KV head."""
    if case["rows"] == "latent":
        parts = _e4m3_values(rows[:, :LATENT]).view(-1, LATENT // GROUP, GROUP)
        values = (parts * rows[:, LATENT + 2 * ROPE:].contiguous().view(torch.float32).double()[..., None]).view(-1, LATENT)
        keys = torch.cat([values, rows[:, LATENT:LATENT + 2 * ROPE].contiguous().view(torch.bfloat16).double()], 1)
        return [(slice(None), keys, values)], torch.ones(len(rows), dtype=torch.bool, device="cuda")
    h, t, d = case["kv_heads"], case["block"], case["head_dim"]
    codes = _e4m3_values(rows[:, :2 * h * t * d]).view(-1, 2, h, t, d)
    tail = rows[:, 2 * h * t * d:]
    scales = tail[:, :8 * h].contiguous().view(torch.float32).double().view(-1, 2, h, 1, 1)
    count = tail[:, 8 * h:8 * h + 4].contiguous().view(torch.int32)
    kv = codes * scales
    g = case["heads"] // h
    return ([(slice(i * g, (i + 1) * g), kv[:, 0, i].reshape(-1, d), kv[:, 1, i].reshape(-1, d)) for i in range(h)],
            (torch.arange(t, device="cuda") < count).reshape(-1))


def _exact_tree(case, s, i):
    sel, t = s["sel"][i].long(), case["nodes"]
    b = 1 if case["rows"] == "latent" else case["block"]
    own_rows = s["drafts"][:, s["layer"]].view(len(s["sel"]), -1, s["drafts"].shape[-1])[i]
    parts, used = _exact_kv(case, torch.cat([s["cache"][sel.clamp(min=0)], own_rows]))
    keep = torch.zeros((t, len(used)), dtype=torch.bool, device="cuda")
    keep[:, :len(sel) * b] = (sel >= 0).repeat_interleave(b)
    for j in range(t):
        keep[:, len(sel) * b + j] = (s["visible"][i] >> j) & 1 == 1
    keep &= used
    q = s["q"][i].double()
    out = torch.zeros((t, case["heads"], parts[0][2].shape[1]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((t, case["heads"]), dtype=torch.float64, device="cuda")
    for at, keys, values in parts:
        logits = torch.where(keep[:, None], q[:, at] @ keys.t() * s["scale"], -math.inf)
        lse[:, at] = torch.logsumexp(logits, -1)
        share = torch.exp(logits - torch.nan_to_num(lse[:, at], neginf=0.0)[..., None])
        out[:, at] = torch.where(keep[:, None], share, 0.0) @ values
    return out, lse


def _exact_weigh(case, s, i):
    sel = s["sel"][i].long()
    parts, used = _exact_kv(case, s["cache"][sel.clamp(min=0)])
    b = len(used) // len(sel)
    keep = used & (sel >= 0).repeat_interleave(b)
    total = torch.zeros(len(used), dtype=torch.float64, device="cuda")
    for at, keys, _ in parts:
        share = torch.exp(s["q"][i, at].double() @ keys.t() * s["scale"] - s["lse"][i, at].double()[:, None])
        total += torch.where(keep, share, 0.0).sum(0)
    return total.view(-1, b).sum(1)


def _exact_norm(case, s, x, weight):
    v = x.double()
    v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / case["dim"] + EPS)
    if weight is not None:
        v = v * weight.double()
    r = case["rotary"]
    if not r:
        return v
    axis = [a for a, width in enumerate(s["sections"]) for _ in range(width)]
    freq = torch.exp(torch.arange(r // 2, device="cuda", dtype=torch.float64) * (-2.0 * math.log(10000.0) / r))
    angle = s["positions"][:, axis].double() * freq
    z = v[..., :r]
    z = z.reshape(*z.shape[:-1], r // 2, 2) if case["interleaved"] else z.reshape(*z.shape[:-1], 2, r // 2).transpose(-1, -2)
    turned = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None]
    back = torch.view_as_real(turned)
    back = (back if case["interleaved"] else back.transpose(-1, -2)).reshape(*v.shape[:-1], r)
    return torch.cat([back, v[..., r:]], -1)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op == "lightest":
        return None                      # addresses: the comparison of whole numbers says it all
    if op == "norm":
        return (_exact_norm(case, s, s["q"], s["q_weight"]),
                None if s["k"] is None else _exact_norm(case, s, s["k"], s["k_weight"]))
    if op == "tree":                     # one request at a time: 64 bits of a whole batch would not fit
        return tuple(torch.stack(o) for o in zip(*(_exact_tree(case, s, i) for i in range(len(s["sel"])))))
    shares = torch.stack([_exact_weigh(case, s, i) for i in range(len(s["sel"]))])
    scores = s["scores"].clone()
    keep = s["sel"].view(-1) >= 0
    scores.index_add_(0, s["sel"].view(-1)[keep].long(), shares.view(-1)[keep])
    return shares, scores
