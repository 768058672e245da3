"""What stands around the attention of a decoder that reads a map, as cases to be measured:

- rotary: positions with several axes (rows and columns of a map, frames of a clip, a text's index)
  enter queries and keys as rotations of pairs of elements; and the gradients, also for fractional
  positions (a detector's reference points).
- join: what lies between two blocks of a layer in one pass: the norm after a block, its gate and
  residual scale, the residual sum and the norm before the next block; and the gradients.
- append: a batch's new keys and values go to their pages of a cache, rotated on the way, and the
  queries of the same tokens are rotated with them.
- paged: one new token of each sequence attends to its sequence's pages.

Sizes are those of this repository's feature maps (an 800 x 1344 image: c3 100x168, c4 50x84, c5
25x42; batches 1, 2 and 8; 256 and 512 channels) and decoder (8 heads of 32 and 64, 16 heads of 128
on 4), and odd ones.
"""

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    def rotary(name, direction, dtype, b, l, h, d, sections, layout, positions, packed):
        return {"name": name, "op": "rotary", "direction": direction, "dtype": dtype, "b": b, "l": l, "h": h, "d": d,
                "sections": sections, "layout": layout, "positions": positions, "packed": packed}

    def join(name, direction, dtype, b, p, c, after, before, gate, scale, affine):
        return {"name": name, "op": "join", "direction": direction, "dtype": dtype, "b": b, "p": p, "c": c,
                "after": after, "before": before, "gate": gate, "scale": scale, "affine": affine}

    def append(name, dtype, b, n, hq, hkv, d, page, past, ragged, sections, layout, positions):
        return {"name": name, "op": "append", "dtype": dtype, "b": b, "n": n, "hq": hq, "hkv": hkv, "d": d, "page": page,
                "past": past, "ragged": ragged, "sections": sections, "layout": layout, "positions": positions}

    def paged(name, dtype, b, length, hq, hkv, d, page, lengths, heads_first):
        return {"name": name, "op": "paged", "dtype": dtype, "b": b, "length": length, "hq": hq, "hkv": hkv, "d": d,
                "page": page, "lengths": lengths, "heads_first": heads_first}

    return [
        # keys of eight c3 maps, rotated by row and column out of a fused projection
        rotary("rotary_c3_batch8", "forward", "bf16", 8, 16800, 8, 32, "8,8", "blocks", "map", True),
        # a clip of eight c5 frames: time, row and column, a quarter of each head left as it is
        rotary("rotary_clip_c5", "forward", "bf16", 2, 8400, 8, 64, "8,8,8", "halves", "clip", False),
        # 900 reference points of two images in single precision: gradients of queries and of the points
        rotary("rotary_points_f32_grad", "backward", "f32", 2, 900, 8, 32, "8,8", "blocks", "points", False),
        # a decoder's 300 queries between two blocks (layer norm before the next): latency
        join("join_queries", "forward", "bf16", 2, 300, 256, "none", "layer", "none", False, True),
        # the positions of eight c3 maps: norms on both sides of the block, scale of its channels
        join("join_c3_batch8", "forward", "bf16", 8, 16800, 256, "layer", "layer", "none", True, True),
        # the training step's gradients over two c3 maps, gated by each image
        join("join_c3_grad", "backward", "bf16", 2, 16800, 256, "layer", "layer", "image", True, True),
        # wide rows that are no multiple of a vector, gated element by element, rms norms, single precision
        join("join_odd_f32_grad", "backward", "f32", 3, 517, 1030, "rms", "rms", "full", False, True),
        # one new token of each of eight sequences enters the cache: the smallest call
        append("append_tokens", "bf16", 8, 1, 16, 4, 128, 64, 4200, False, "64", "halves", "index"),
        # a prompt of ragged lengths with the positions of a c4 map, eight sequences
        append("append_c4_ragged", "bf16", 8, 4200, 16, 4, 128, 64, 333, True, "22,21,21", "halves", "clip"),
        # one sequence's token over 1050 cached positions: latency
        paged("token_1050", "bf16", 1, 1050, 8, 8, 64, 64, "full", False),
        # eight ragged sequences, shared key heads: a long cache
        paged("tokens_16800", "bf16", 8, 16800, 16, 4, 128, 64, "ragged", False),
        # odd pages and heads in single precision, an empty sequence and one longer than the others
        paged("tokens_odd_f32", "f32", 13, 2777, 6, 3, 40, 24, "uneven", True),
    ]


# ---------------------------------------------------------------- drawn cases

def _between(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 20)


def _split(rng, pairs, axes):
    """`pairs` in so many parts of one at least."""
    cuts = sorted(rng.sample(range(1, pairs), axes - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [pairs])]


def _rotated(rng, d, axes):
    """Sections for heads of d elements: all of them or a part, even parts or uneven ones."""
    pairs = d // 2 if rng.random() < 0.6 else max(axes, d // 2 - rng.randrange(0, d // 4 + 1))
    sections = [pairs // axes] * axes if rng.random() < 0.5 else _split(rng, pairs, axes)
    return ",".join(str(n) for n in sections)


def draw(rng):
    most = max(_cost(c) for c in listed())
    kind = rng.choice(["rotary", "rotary_grad", "join", "join_grad", "append", "paged", "paged"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([32, 64, 128, 32, 64, 128, rng.randrange(8, 129), 8 * rng.randrange(1, 17)])
    layout = rng.choice(["halves", "adjacent", "blocks"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    if kind.startswith("rotary"):
        positions = rng.choice(["index", "map", "clip", "points"])
        case = {"op": "rotary", "direction": "backward" if kind == "rotary_grad" else "forward", "dtype": dtype,
                "b": _between(rng, 1, 8), "l": _between(rng, 1, 16800), "h": rng.choice([1, 2, 3, 6, 8, 8, 16]), "d": d,
                "sections": _rotated(rng, d, {"index": 1, "clip": 3}.get(positions, 2)), "layout": layout,
                "positions": positions, "packed": rng.random() < 0.5}
        shrink = ("b", "l")
    elif kind.startswith("join"):
        after, before = rng.choice([("none", "layer"), ("none", "rms"), ("layer", "layer"), ("rms", "rms"),
                                    ("layer", "none"), ("rms", "layer")])
        case = {"op": "join", "direction": "backward" if kind == "join_grad" else "forward", "dtype": dtype,
                "b": _between(rng, 1, 8), "p": _between(rng, 1, 16800),
                "c": rng.choice([96, 192, 256, 512, 1024, 2048, _between(rng, 16, 2048), _between(rng, 16, 8192)]),
                "after": after, "before": before, "gate": rng.choice(["none", "none", "image", "full"]),
                "scale": rng.random() < 0.5, "affine": rng.random() < 0.8}
        shrink = ("b", "p")
    elif kind == "append":
        positions = rng.choice(["index", "index", "clip", "points"])
        long = rng.random() < 0.5
        case = {"op": "append", "dtype": dtype, "b": _between(rng, 1, 8 if long else 64),
                "n": _between(rng, 2, 4200) if long else 1, "hq": hq, "hkv": hkv, "d": d,
                "page": rng.choice([16, 32, 64, 128, rng.randrange(1, 100)]), "past": _between(rng, 1, 4200),
                "ragged": rng.random() < 0.5,
                "sections": _rotated(rng, d, {"index": 1, "clip": 3}.get(positions, 2)), "layout": layout,
                "positions": positions}
        shrink = ("b", "n", "past")
    else:
        case = {"op": "paged", "dtype": dtype, "b": _between(rng, 1, 64), "length": _between(rng, 1, 16800), "hq": hq,
                "hkv": hkv, "d": d, "page": rng.choice([16, 32, 64, 128, rng.randrange(1, 100)]),
                "lengths": rng.choice(["full", "ragged", "uneven"]), "heads_first": rng.random() < 0.4}
        shrink = ("b", "length")
    while _cost(case) > most:
        side = max(shrink, key=lambda s: case[s])
        case[side] = max(1, case[side] * 2 // 3)
    return case


# ---------------------------------------------------------------- inputs

def _sections(case):
    """How many pairs turn with each axis."""
    return [int(n) for n in case["sections"].split(",")]


def _lengths(case):
    """Lengths of the sequences, by the case (so that the work goes by it)."""
    b, most = case["b"], case["length"]
    rng = random.Random(most * 131 + b)
    if case["lengths"] == "full":
        return [most] * b
    if case["lengths"] == "ragged":
        return [max(1, round(most * rng.uniform(0.25, 1.0))) for _ in range(b)]
    lengths = [most if i == 0 else max(1, round(most * rng.uniform(0.0, 0.2))) for i in range(b)]   # one long among short
    if b > 1:
        lengths[b // 2] = 0                                       # and one that has nothing yet
    return lengths


def _counts(case):
    """How many of each sequence's n rows are tokens, and how many positions it held before."""
    b, n, past = case["b"], case["n"], case["past"]
    rng = random.Random(n * 257 + b)
    starts = [rng.randrange(0, past + 1) for _ in range(b)]
    if not case["ragged"]:
        return [n] * b, starts
    return [n if i == 0 else rng.randrange(0, n + 1) for i in range(b)], starts


def _pages(case, lengths):
    """For each sequence as many pages of the cache as it needs, in no order."""
    page = case["page"]
    need = [-(-n // page) for n in lengths]
    return need, max(1, max(need)), sum(need) + 3


def _tables(case, lengths, g):
    need, width, total = _pages(case, lengths)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["b"], width), -1, dtype=torch.int32, device="cuda")   # no page behind a sequence's last
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, total


def _positions(kind, b, l, g):
    """Positions [b,l,axes]: of text far in, of the map or clip with l positions, or of points on an image."""
    if kind == "points":
        return torch.rand((b, l, 2), generator=g, device="cuda") * torch.tensor([100.0, 168.0], device="cuda")
    at = torch.arange(l, device="cuda", dtype=torch.int32)
    if kind == "index":
        first = torch.randint(0, 1 << 20, (b, 1), generator=g, device="cuda", dtype=torch.int32)
        return (first + at)[:, :, None].contiguous()
    w = max(1, math.isqrt(l))
    if kind == "map":
        return torch.stack((at // w, at % w), -1)[None].expand(b, -1, -1)          # every image has the same
    w = max(1, math.isqrt(max(1, l // 8)))
    return torch.stack((at // (w * w), at // w % w, at % w), -1)[None].expand(b, -1, -1)


def _frequencies(kind, sections):
    base = {"index": 10000.0, "clip": 1000.0}.get(kind, 100.0)
    return torch.cat([base ** (-torch.arange(n, dtype=torch.float64) / n) for n in sections]).float().cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale + mean).to(dt)

    s = {"case": case}
    if case["op"] == "rotary":
        b, l, h, d = (case[k] for k in ("b", "l", "h", "d"))
        s["positions"] = _positions(case["positions"], b, l, g)
        s["frequencies"] = _frequencies(case["positions"], _sections(case))
        s["x"] = normal(b, l, 2, h, d)[:, :, 0] if case["packed"] else normal(b, l, h, d)
        if case["direction"] == "backward":
            s["grad"] = normal(b, l, h, d)
    elif case["op"] == "join":
        b, p, c = (case[k] for k in ("b", "p", "c"))
        # a stream that has grown over the blocks, with a mean of its own, and a block's output
        s["x"], s["y"] = normal(b, p, c, scale=2.0, mean=0.3), normal(b, p, c)
        s["gate"] = {"none": None, "image": normal(b, c, scale=0.3, mean=0.8),
                     "full": normal(b, p, c, scale=0.3, mean=0.5)}[case["gate"]] if case["gate"] != "none" else None
        s["scale"] = normal(c, scale=0.2, mean=0.5) if case["scale"] else None
        for side, kind in (("after", case["after"]), ("before", case["before"])):
            affine = case["affine"] and kind != "none"
            s[side + "_weight"] = normal(c, scale=0.2, mean=1.0) if affine else None
            s[side + "_bias"] = normal(c, scale=0.2) if affine and kind == "layer" else None
        if case["direction"] == "backward":
            s["stats"] = _plain_join(s, case)[2]                    # what the forward left
            s["grad_out"] = normal(b, p, c)
            s["grad_next"] = normal(b, p, c) if case["before"] != "none" else None
    elif case["op"] == "append":
        b, n, hq, hkv, d = (case[k] for k in ("b", "n", "hq", "hkv", "d"))
        counts, starts = _counts(case)
        s["table"], total = _tables(case, [a + c for a, c in zip(starts, counts)], g)
        qkv = normal(b, n, hq + 2 * hkv, d)                         # one projection's output
        s["q"], s["k"], s["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        s["key_pages"], s["value_pages"] = normal(total, case["page"], hkv, d), normal(total, case["page"], hkv, d)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda") if case["ragged"] else None
        # a text's tokens stand where they are appended
        s["positions"] = None if case["positions"] == "index" else _positions(case["positions"], b, n, g)
        s["frequencies"] = _frequencies(case["positions"], _sections(case))
    else:
        b, hq, hkv, d = (case[k] for k in ("b", "hq", "hkv", "d"))
        lengths = _lengths(case)
        s["table"], total = _tables(case, lengths, g)
        s["q"] = normal(b, hq, d, scale=1.5)
        if case["heads_first"]:                                     # each head's rows of a page side by side
            s["key_pages"], s["value_pages"] = (normal(total, hkv, case["page"], d).transpose(1, 2) for _ in range(2))
        else:
            s["key_pages"], s["value_pages"] = (normal(total, case["page"], hkv, d) for _ in range(2))
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- the plain forms

def _pair_columns(sections, layout):
    """For each pair its axis and its two elements."""
    axis, first, second, total = [], [], [], sum(sections)
    at = 0
    for a, n in enumerate(sections):
        for i in range(n):
            axis.append(a)
            if layout == "halves":
                e = (at + i, total + at + i)
            elif layout == "adjacent":
                e = (2 * (at + i), 2 * (at + i) + 1)
            else:
                e = (2 * at + i, 2 * at + n + i)
            first.append(e[0])
            second.append(e[1])
        at += n
    return axis, first, second


def _plain_angles(positions, frequencies, axis):
    """cos and sin [b,l,1,pairs] in 32 bits of angles in 64."""
    angle = positions[:, :, axis].double() * frequencies.double()
    return angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]


def _plain_rotate(x, cos, sin, first, second):
    """float32 [b,l,h,d] with the pairs rotated."""
    x = x.float()
    a, b = x[..., first], x[..., second]
    y = x.clone()
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def _plain_rotary(s, case):
    axis, first, second = _pair_columns(_sections(case), case["layout"])
    cos, sin = _plain_angles(s["positions"], s["frequencies"], axis)
    if case["direction"] == "forward":
        return _plain_rotate(s["x"], cos, sin, first, second).to(s["x"].dtype)
    gx = _plain_rotate(s["grad"], cos, -sin, first, second)
    if case["positions"] != "points":
        return gx.to(s["x"].dtype)
    x = s["x"].float()
    turn = ((gx[..., second] * x[..., first] - gx[..., first] * x[..., second]).sum(2)) * s["frequencies"]
    gp = torch.stack([turn[..., [i for i, a in enumerate(axis) if a == n]].sum(-1)
                      for n in range(len(_sections(case)))], -1)
    return gx.to(s["x"].dtype), gp


def _plain_normalise(x, kind):
    """The normed rows, their mean and 1 / standard deviation (root mean square for rms)."""
    one, zero = torch.ones_like(x[..., :1]), torch.zeros_like(x[..., :1])
    if kind == "none":
        return x, zero, one
    mean = x.mean(-1, keepdim=True) if kind == "layer" else zero
    r = 1 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + EPS)
    return (x - mean) * r, mean, r


def _plain_affine(x, weight, bias):
    x = x if weight is None else x * weight.float()
    return x if bias is None else x + bias.float()


def _plain_factor(s, case):
    """gate * scale, or 1, to multiply [b,p,c] by."""
    f = 1.0
    if s["gate"] is not None:
        f = s["gate"].float()
        f = f[:, None] if case["gate"] == "image" else f
    return f if s["scale"] is None else f * s["scale"].float()


def _plain_join(s, case):
    v, m1, r1 = _plain_normalise(s["y"].float(), case["after"])
    out = s["x"].float() + _plain_factor(s, case) * _plain_affine(v, s["after_weight"], s["after_bias"])
    u, m2, r2 = _plain_normalise(out, case["before"])
    stats = torch.cat((m1, r1, m2, r2), -1)
    dt = s["x"].dtype
    if case["before"] == "none":
        return out.to(dt), None, stats
    return out.to(dt), _plain_affine(u, s["before_weight"], s["before_bias"]).to(dt), stats


def _plain_norm_grad(g, x, r, kind):
    """Gradient at the rows that x (normed) came from."""
    if kind == "none":
        return g
    d = g - x * (g * x).mean(-1, keepdim=True)
    return r * (d - g.mean(-1, keepdim=True) if kind == "layer" else d)


def _plain_join_grad(s, case):
    m1, r1, m2, r2 = (s["stats"][..., i:i + 1] for i in range(4))
    v = (s["y"].float() - m1) * r1
    z = _plain_affine(v, s["after_weight"], s["after_bias"])
    factor = _plain_factor(s, case)
    d, grads = s["grad_out"].float(), {}
    if case["before"] != "none":
        u = (s["x"].float() + factor * z - m2) * r2
        gn = s["grad_next"].float()
        if s["before_weight"] is not None:
            grads["before_weight"] = (gn * u).sum((0, 1))
        if s["before_bias"] is not None:
            grads["before_bias"] = gn.sum((0, 1))
        d = d + _plain_norm_grad(gn if s["before_weight"] is None else gn * s["before_weight"].float(), u, r2,
                                 case["before"])
    if s["gate"] is not None:
        gg = d * z if s["scale"] is None else d * z * s["scale"].float()
        grads["gate"] = gg.sum(1) if case["gate"] == "image" else gg
    if s["scale"] is not None:
        gs = d * z
        if s["gate"] is not None:
            gs = gs * (s["gate"].float()[:, None] if case["gate"] == "image" else s["gate"].float())
        grads["scale"] = gs.sum((0, 1))
    h = d * factor
    if s["after_weight"] is not None:
        grads["after_weight"] = (h * v).sum((0, 1))
    if s["after_bias"] is not None:
        grads["after_bias"] = h.sum((0, 1))
    gy = _plain_norm_grad(h if s["after_weight"] is None else h * s["after_weight"].float(), v, r1, case["after"])
    names = ("gate", "scale", "after_weight", "after_bias", "before_weight", "before_bias")
    return tuple(t.to(s["x"].dtype) for t in (d, gy, *(grads[n] for n in names if n in grads)))


def _plain_append(s, case):
    b, n, page = case["b"], case["n"], case["page"]
    axis, first, second = _pair_columns(_sections(case), case["layout"])
    at = s["starts"][:, None] + torch.arange(n, device="cuda", dtype=torch.int32)
    positions = s["positions"]
    if positions is None:
        positions = at[:, :, None].expand(b, n, len(_sections(case)))
    cos, sin = _plain_angles(positions, s["frequencies"], axis)
    q = _plain_rotate(s["q"], cos, sin, first, second).to(s["q"].dtype)
    k = _plain_rotate(s["k"], cos, sin, first, second).to(s["q"].dtype)
    counts = torch.full_like(s["starts"], n) if s["counts"] is None else s["counts"]
    seq, row = (torch.arange(n, device="cuda") < counts[:, None]).nonzero(as_tuple=True)
    where = at[seq, row].long()
    pages = s["table"][seq, where // page].long()
    s["key_pages"][pages, where % page] = k[seq, row]
    s["value_pages"][pages, where % page] = s["v"][seq, row]
    return s["starts"] + counts, q, s["key_pages"], s["value_pages"]


def _plain_paged(s, case):
    b, hq, hkv, d = (case[k] for k in ("b", "hq", "hkv", "d"))
    rows = s["table"].clamp(min=0).long()

    def gathered(pages):                                            # [b, hkv, positions, d] float32
        return pages[rows].reshape(b, -1, hkv, d).permute(0, 2, 1, 3).float().contiguous()

    k, v = gathered(s["key_pages"]), gathered(s["value_pages"])
    q = s["q"].float().reshape(b, hkv, hq // hkv, d)
    scores = torch.matmul(q, k.transpose(-1, -2).contiguous()) / math.sqrt(d)
    kept = torch.arange(k.shape[2], device="cuda") < s["lengths"][:, None]
    scores = scores.masked_fill(~kept[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
    return out.reshape(b, hq, d).to(s["q"].dtype)


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "rotary":
        return _plain_rotary(state, case)
    if case["op"] == "join":
        if case["direction"] == "backward":
            return _plain_join_grad(state, case)
        return tuple(t for t in _plain_join(state, case)[:2] if t is not None)
    return _plain_append(state, case) if case["op"] == "append" else _plain_paged(state, case)


def _run_own(s, case):
    import deformable_convolution_vision_amd as dcn
    if case["op"] == "rotary":
        how = (s["positions"], s["frequencies"], _sections(case), case["layout"])
        if case["direction"] == "forward":
            return dcn.rotary_positions(s["x"], *how)
        if case["positions"] == "points":
            return dcn.rotary_positions_backward(s["grad"], *how, input=s["x"])
        return dcn.rotary_positions_backward(s["grad"], *how)
    if case["op"] == "join":
        how = {"gate": s["gate"], "scale": s["scale"], "branch_norm": case["after"], "branch_weight": s["after_weight"],
               "branch_bias": s["after_bias"], "next_norm": case["before"], "next_weight": s["before_weight"],
               "next_bias": s["before_bias"]}
        if case["direction"] == "forward":
            return tuple(t for t in dcn.residual_norm(s["x"], s["y"], eps=EPS, **how) if t is not None)
        grads = dcn.residual_norm_backward(s["grad_out"], s["grad_next"], s["x"], s["y"], s["stats"], **how)
        return tuple(t for t in grads if t is not None)
    if case["op"] == "append":
        lengths, q = dcn.paged_append(s["k"], s["v"], s["key_pages"], s["value_pages"], s["table"], s["starts"],
                                      counts=s["counts"], query=s["q"], positions=s["positions"],
                                      frequencies=s["frequencies"], sections=_sections(case), layout=case["layout"])
        return lengths, q, s["key_pages"], s["value_pages"]
    return dcn.paged_attention(s["q"], s["key_pages"], s["value_pages"], s["table"], s["lengths"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotary":
        b, l, h, d = (case[k] for k in ("b", "l", "h", "d"))
        n, pairs, axes = b * l * h * d, sum(_sections(case)), len(_sections(case))
        at = 4 * axes * l * (1 if case["positions"] in ("map", "clip") else b) + 4 * pairs
        points = case["direction"] == "backward" and case["positions"] == "points"
        return {"bytes": (3 if points else 2) * n * es + at + (4 * b * l * axes if points else 0),
                "flops": b * l * pairs * (h * (10 if points else 6) + 20)}
    if case["op"] == "join":
        n, c = case["b"] * case["p"] * case["c"], case["c"]
        gate = {"none": 0, "image": case["b"] * c, "full": n}[case["gate"]]
        vectors = int(case["scale"])
        if case["affine"]:
            vectors += sum({"none": 0, "rms": 1, "layer": 2}[case[k]] for k in ("after", "before"))
        then = case["before"] != "none"
        if case["direction"] == "backward":
            # both inputs, the gradients that come in and the two that go out; the gate and its gradient
            return {"bytes": ((6 if then else 5) * n + 2 * gate + 2 * vectors * c) * es + 16 * n // c, "flops": 40 * n}
        return {"bytes": ((4 if then else 3) * n + gate + vectors * c) * es, "flops": 20 * n}
    if case["op"] == "append":
        counts, _ = _counts(case)
        b, n, hq, hkv, d = (case[k] for k in ("b", "n", "hq", "hkv", "d"))
        pairs, axes = sum(_sections(case)), len(_sections(case))
        at = 0 if case["positions"] == "index" else 4 * axes * n * (b if case["positions"] == "points" else 1)
        new = sum(counts)
        return {"bytes": 2 * es * d * (2 * new * hkv + b * n * hq) + at + 4 * pairs + 12 * b + 4 * (-(-new // case["page"])),
                "flops": pairs * (6 * (new * hkv + b * n * hq) + 20 * b * n)}
    keys = sum(_lengths(case))
    b, hq, hkv, d = (case[k] for k in ("b", "hq", "hkv", "d"))
    pages = _pages(case, _lengths(case))[0]
    return {"bytes": 2 * es * d * (keys * hkv + b * hq) + 4 * sum(pages) + 4 * b, "flops": 4 * d * hq * keys}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "join": _exact_join, "append": _exact_append, "paged": _exact_paged}[case["op"]](case, s)


def _exact_turned(x, positions, frequencies, sections, layout):
    """Axis by axis as products of complex numbers."""
    parts, at, total = [], 0, sum(sections)
    x = x.double()
    rotated, rest = x[..., :2 * total], x[..., 2 * total:]
    turns = []
    for a, n in enumerate(sections):
        angle = positions[:, :, None, a:a + 1].double() * frequencies[at:at + n].double()
        turns.append(torch.polar(torch.ones_like(angle), angle))
        at += n
    if layout == "blocks":
        at = 0
        for n, turn in zip(sections, turns):
            block = rotated[..., at:at + 2 * n]
            z = torch.complex(block[..., :n].contiguous(), block[..., n:].contiguous()) * turn
            parts += [z.real, z.imag]
            at += 2 * n
        return torch.cat(parts + [rest], -1)
    turn = torch.cat(turns, -1)
    if layout == "adjacent":
        z = torch.view_as_complex(rotated.reshape(*x.shape[:3], total, 2).contiguous()) * turn
        return torch.cat((torch.view_as_real(z).flatten(-2), rest), -1)
    z = torch.complex(rotated[..., :total].contiguous(), rotated[..., total:].contiguous()) * turn
    return torch.cat((z.real, z.imag, rest), -1)


def _exact_rotary(case, s):
    how = (s["frequencies"], _sections(case), case["layout"])
    if case["direction"] == "forward":
        return _exact_turned(s["x"], s["positions"], *how)
    x = s["x"].double().detach().requires_grad_(True)
    positions = s["positions"].double().detach().requires_grad_(True)
    with torch.enable_grad():
        y = _exact_turned(x, positions, *how)
        gx, gp = torch.autograd.grad((y * s["grad"].double()).sum(), (x, positions))
    return (gx, gp) if case["positions"] == "points" else gx


def _exact_join(case, s):
    """Gradients by differentiation of the definition, one batch element at a time."""
    names = ("gate", "scale", "after_weight", "after_bias", "before_weight", "before_bias")
    shared = {n: s[n].double().requires_grad_(True) for n in names if s[n] is not None}

    def rows(t, kind, name):
        if kind == "none":
            return t
        t = t - t.sum(-1, keepdim=True) / t.shape[-1] if kind == "layer" else t
        t = t * ((t * t).sum(-1, keepdim=True) / t.shape[-1] + EPS) ** -0.5
        t = t * shared[name + "_weight"] if name + "_weight" in shared else t
        return t + shared[name + "_bias"] if name + "_bias" in shared else t

    outs, nexts, gxs, gys = [], [], [], []
    backward = case["direction"] == "backward"
    with torch.set_grad_enabled(backward):
        for i in range(case["b"]):
            x, y = (s[k][i].double().requires_grad_(True) for k in ("x", "y"))
            z = rows(y, case["after"], "after")
            for n in ("gate", "scale"):
                if n in shared:
                    z = z * (shared[n][i] if n == "gate" else shared[n])
            out = x + z
            then = rows(out, case["before"], "before")
            if backward:
                loss = (out * s["grad_out"][i].double()).sum()
                if case["before"] != "none":
                    loss = loss + (then * s["grad_next"][i].double()).sum()
                loss.backward()
                gxs.append(x.grad)
                gys.append(y.grad)
            else:
                outs.append(out)
                nexts.append(then)
    if backward:
        return (torch.stack(gxs), torch.stack(gys), *(shared[n].grad for n in names if n in shared))
    return (torch.stack(outs), torch.stack(nexts)) if case["before"] != "none" else (torch.stack(outs),)


def _exact_append(case, s):
    counts, starts = _counts(case)
    n, page, axes = case["n"], case["page"], len(_sections(case))
    positions = s["positions"]
    if positions is None:
        positions = torch.stack([a + torch.arange(n, device="cuda") for a in starts])[:, :, None].repeat(1, 1, axes)
    how = (positions, s["frequencies"], _sections(case), case["layout"])
    q, k, v = _exact_turned(s["q"], *how), _exact_turned(s["k"], *how), s["v"].double()
    key_pages, value_pages = s["key_pages"].double(), s["value_pages"].double()
    for i, (start, count) in enumerate(zip(starts, counts)):
        done = 0
        while done < count:                                         # page by page
            at = (start + done) % page
            m = min(page - at, count - done)
            to = int(s["table"][i, (start + done) // page])
            key_pages[to, at:at + m] = k[i, done:done + m]
            value_pages[to, at:at + m] = v[i, done:done + m]
            done += m
    return torch.tensor([a + c for a, c in zip(starts, counts)], dtype=torch.int32, device="cuda"), q, key_pages, value_pages


def _exact_paged(case, s):
    """Sequence by sequence and head by head; only a sequence's own positions enter."""
    b, hq, hkv, d = (case[k] for k in ("b", "hq", "hkv", "d"))
    out = torch.zeros((b, hq, d), dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        at = torch.arange(n, device="cuda")
        pages, places = s["table"][i].long()[at // case["page"]], at % case["page"]
        for h in range(hkv):
            k, v = s["key_pages"][pages, places, h].double(), s["value_pages"][pages, places, h].double()
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            out[i, heads] = torch.softmax((s["q"][i, heads].double() @ k.T.contiguous()) / d ** 0.5, -1) @ v
    return out
