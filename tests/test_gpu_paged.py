"""dcn_paged_append and dcn_paged_attention (through the binding) against the definition in 64 bits, element by
element, within the bounds that rotary_oracle and attention_oracle derive from the stated arithmetic."""

import math
import zlib

import numpy as np
import pytest
import torch

import deformable_convolution_vision_amd as dcn
import rotary_oracle
from attention_oracle import check, one_head

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.double().cpu().numpy()


def tables(need, total, width, g):
    """Pages in no order; entries behind a sequence's last page name none."""
    order = torch.randperm(total, generator=g).to(torch.int32)
    table, at = torch.full((len(need), width), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.cuda()


# ---------------------------------------------------------------- attention

# name: lengths, Hq, Hkv, D, page size
ATTENTION = {
    "one_position": ([1], 1, 1, 64, 16),
    "lengths": ([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 255, 256, 257, 300], 8, 2, 64, 32),
    "pages_of_one": ([5, 40, 0], 2, 1, 32, 1),
    "pages_of_seven": ([100, 3, 260], 4, 2, 128, 7),
    "pages_of_24": ([333, 24, 48, 1], 6, 3, 40, 24),
    "pages_of_100": ([777, 99, 100, 101], 3, 1, 72, 100),
    "one_long": ([5000], 8, 1, 128, 64),
    "one_long_among_short": ([3, 4100, 0, 17], 4, 4, 64, 64),
    "many_heads_of_a_key": ([200, 65], 40, 2, 32, 16),       # 20 heads: two tiles of 16 rows
    "sixteen_heads": ([513, 129], 16, 1, 128, 32),
    "odd_head": ([130, 77], 4, 2, 37, 16),                   # no vector fits a row
    "head_20": ([130, 77], 4, 2, 20, 16),
    "head_9": ([40, 3], 2, 2, 9, 16),
    "head_5": ([40, 3], 2, 1, 5, 16),                        # less than a vector in bf16
    "head_1": ([70], 2, 1, 1, 16),
    "head_33": ([90], 3, 1, 33, 8),
    "head_67": ([130, 77, 0], 8, 2, 67, 16),
    "head_98": ([90], 2, 1, 98, 16),
    "head_127": ([513, 31], 8, 4, 127, 32),
    "head_45_in_parts": ([2000, 30, 2900], 3, 3, 45, 16),
    "head_8": ([70], 2, 2, 8, 16),
    "head_96": ([300, 40], 6, 2, 96, 32),
    "many_short": ([(7 * i) % 50 for i in range(150)], 2, 1, 32, 16),
    "more_sequences_than_fill": ([40 + (13 * i) % 700 for i in range(70)], 8, 8, 64, 32),
    # more sequences than a wave has lanes, with tables for long ones: lists of the parts
    "lists": ([(131 * i) % 1700 for i in range(130)], 4, 2, 64, 32),
    "lists_65_one_long": ([5] * 40 + [7000] + [0] * 24, 1, 1, 128, 16),
    "lists_two_a_thread": ([(17 * i) % 40 for i in range(1500)] + [2500, 2000], 2, 1, 32, 8),
    "lists_more_heads_than_fill": ([(7 * i) % 30 for i in range(70)] + [1800], 270, 270, 8, 64),
}


def make(name, dtype, seed=0, heads_first=False, scale=1.0):
    lengths, hq, hkv, d, page = ATTENTION[name]
    g = torch.Generator().manual_seed(zlib.crc32(name.encode()) + seed)
    t = DT[dtype]
    need = [-(-n // page) for n in lengths]
    total, width = sum(need) + 2, max(1, max(need)) + 1

    def pages():
        shape = (total, hkv, page, d) if heads_first else (total, page, hkv, d)
        p = torch.randn(shape, generator=g).to(t).cuda()
        return p.transpose(1, 2) if heads_first else p

    k, v = pages(), pages()
    q = (torch.randn((len(lengths), hq, d), generator=g) * 1.5 * scale).to(t).cuda()
    return q, k, v, tables(need, total, width, g), torch.tensor(lengths, dtype=torch.int32).cuda()


def reference(q, k, v, table, lengths, dtype, scale=None):
    """out, lse and their bounds, sequence by sequence over the positions that the table names."""
    q, k, v, table, lengths = f64(q), f64(k), f64(v), table.cpu().numpy(), lengths.cpu().numpy()
    B, hq, d = q.shape
    total, page, hkv, _ = k.shape
    g = hq // hkv
    scale = d ** -0.5 if scale is None else scale
    out, tol, lse, ltol = np.zeros_like(q), np.zeros_like(q), np.zeros((B, hq)), np.zeros((B, hq))
    for b in range(B):
        j = np.arange(min(max(lengths[b], 0), table.shape[1] * page))
        at, place = table[b][j // page], j % page
        in_cache = (at >= 0) & (at < total)
        at, place = at[in_cache], place[in_cache]
        for h in range(hkv):
            r = one_head(q[b, h * g:(h + 1) * g], k[at, place, h], v[at, place, h], scale, dtype)
            rows = slice(h * g, (h + 1) * g)
            out[b, rows], tol[b, rows], lse[b, rows], ltol[b, rows] = r["out"], r["out_tol"], r["lse"], r["lse_tol"]
    return out, tol, lse, ltol


def compare(args, dtype, what, scale=None):
    out, lse = dcn.paged_attention(*args, scale=scale, return_lse=True)
    torch.cuda.synchronize()
    want, tol, wl, tl = reference(*args, dtype, scale)
    check(f64(out), want, tol, what + " out")
    check(f64(lse), wl, tl, what + " lse")
    return out, lse


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(ATTENTION))
def test_attention(name, dtype):
    print(f"[gpu-test] paged attention {name} {dtype}", flush=True)
    args = make(name, dtype)
    out, lse = compare(args, dtype, name)
    again = dcn.paged_attention(*args)
    assert torch.equal(again, out), "the same call gave other bits"
    args = make(name, dtype, heads_first=True)
    compare(args, dtype, name + " heads first", scale=0.31)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lists_of_equal_and_of_no_lengths(dtype):
    """Equal long ones (a quota that every sequence reaches), all empty, and lengths beyond the table."""
    q, k, v, table, _ = make("lists", dtype)
    width = table.shape[1] * k.shape[1]
    for n in (0, 1, width, width + 1000):
        compare((q, k, v, table, torch.full((len(q),), n, dtype=torch.int32, device="cuda")), dtype, f"{n} each")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_scores(dtype):
    """Scores of hundreds: the running maximum moves over blocks, waves and parts."""
    q, k, v, table, lengths = make("one_long", dtype, scale=30.0)
    ramp = torch.linspace(0.1, 3.0, k.shape[0], device="cuda")
    k = (k.float() * ramp[torch.argsort(table[0, :-1].clamp(min=0)).repeat(2)[:k.shape[0]]][:, None, None, None]).to(k.dtype)
    compare((q, k, v, table, lengths), dtype, "large scores")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_lies_behind_a_sequence_does_not_matter(dtype):
    for name in ("lengths", "pages_of_24", "odd_head"):
        q, k, v, table, lengths = make(name, dtype)
        want, wl = dcn.paged_attention(q, k, v, table, lengths, return_lse=True)
        page, used = k.shape[1], torch.zeros(k.shape[:2], dtype=torch.bool, device="cuda")
        for b, n in enumerate(lengths.tolist()):
            j = torch.arange(n, device="cuda")
            used[table[b].long()[j // page], j % page] = True
        k2, v2, t2 = k.clone(), v.clone(), table.clone()
        for t, bad in ((k2, float("nan")), (v2, float("inf"))):
            t[~used] = bad
        t2[t2 < 0] = 1 << 30                     # entries behind the last page are not looked at
        out, lse = dcn.paged_attention(q, k2, v2, t2, lengths, return_lse=True)
        assert torch.equal(out, want) and torch.equal(lse, wl), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_entries_that_are_no_page(dtype):
    q, k, v, table, lengths = make("pages_of_24", dtype)
    table[0, 1], table[0, 5], table[0, 9] = -7, k.shape[0], 1 << 30
    table[1, 0] = -1                             # its only page
    out, lse = compare((q, k, v, table, lengths), dtype, "bad entries")
    assert torch.all(out[1] == 0) and torch.all(lse[1] == -math.inf)
    # lengths beyond the table and below 0 are taken as its size and 0
    q, k, v, table, lengths = make("pages_of_seven", dtype)
    lengths[0], lengths[1] = 1 << 30, -5
    out, lse = compare((q, k, v, table, lengths), dtype, "lengths")
    assert torch.all(out[1] == 0) and torch.all(lse[1] == -math.inf)


def test_not_finite_values_in_the_sequence():
    q, k, v, table, lengths = make("pages_of_24", "bf16")
    v[int(table[0, 2]), 3, 1, 5] = float("inf")
    k[int(table[3, 0]), 0, 0, 0] = float("nan")
    out = dcn.paged_attention(q, k, v, table, lengths)
    assert torch.all(out[0, 2:4, 5] == float("inf")) and torch.isfinite(out[0, :2]).all()
    assert torch.isnan(out[3, :2]).all() and torch.isfinite(out[3, 2:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_key_of_minus_infinity_in_any_element(dtype):
    """The position has a weight of zero, whichever element of an odd head it is (reads of 16 bytes overlap there)."""
    for name in ("head_5", "head_9", "odd_head", "head_67"):
        q, k, v, table, lengths = make(name, dtype)
        q = q.abs() + 0.5
        for e in range(q.shape[2]):
            kk, vv = k.clone(), v.clone()
            kk[int(table[0, 0]), 3, :, e] = -float("inf")
            vv[int(table[0, 0]), 3] = 100.0
            out = dcn.paged_attention(q, kk, vv, table, lengths)
            vv[int(table[0, 0]), 3] = -100.0
            assert torch.isfinite(out).all() and torch.equal(out, dcn.paged_attention(q, kk, vv, table, lengths)), (name, e)


def test_strides():
    q, k, v, table, lengths = make("sixteen_heads", "bf16")
    want = dcn.paged_attention(q, k, v, table, lengths)
    both = torch.stack((k, v), 2)                # keys and values of a position side by side
    wide = torch.zeros((q.shape[0], 3, *q.shape[1:]), dtype=q.dtype, device="cuda")
    wide[:, 1] = q
    long = torch.full((table.shape[0], table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    long[:, :table.shape[1]] = table
    out = dcn.paged_attention(wide[:, 1], both[:, :, 0], both[:, :, 1], long[:, :table.shape[1]], lengths)
    assert torch.equal(out, want)
    shared = table[:1].expand(2, -1)             # two sequences of one beginning
    n = torch.tensor([513, 129], dtype=torch.int32, device="cuda")
    assert torch.equal(dcn.paged_attention(q, k, v, shared, n), dcn.paged_attention(q, k, v, shared.contiguous(), n))


def test_pages_beyond_32_bits():
    """Pages 2^26 elements apart: the last ones lie beyond 2^32 bytes and 2^31 elements."""
    step, n, page, hkv, d = 1 << 26, 40, 16, 2, 64
    buf = torch.empty(n * step, dtype=torch.bfloat16, device="cuda")
    k = buf.as_strided((n, page, hkv, d), (step, hkv * d, d, 1))
    v = buf.as_strided((n, page, hkv, d), (step, hkv * d, d, 1), 1 << 20)
    g = torch.Generator().manual_seed(5)
    kd, vd = (torch.randn((n, page, hkv, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    k.copy_(kd)
    v.copy_(vd)
    q = torch.randn((2, 4, d), generator=g).to(torch.bfloat16).cuda()
    table = torch.stack((torch.randperm(n, generator=g), torch.arange(n))).to(torch.int32).cuda()
    lengths = torch.tensor([n * page, n * page - 3], dtype=torch.int32, device="cuda")
    want = dcn.paged_attention(q, kd, vd, table, lengths)
    assert torch.equal(dcn.paged_attention(q, k, v, table, lengths), want)
    # and an append there
    rows = torch.randn((2, 5, hkv, d), generator=g).to(torch.bfloat16).cuda()
    starts = torch.tensor([3, n * page - 40], dtype=torch.int32, device="cuda")
    dcn.paged_append(rows, rows, k, v, table, starts)
    dcn.paged_append(rows, rows, kd, vd, table, starts)
    assert torch.equal(k, kd) and torch.equal(v, vd)


# ---------------------------------------------------------------- append

# name: B, L, Hq, Hkv, D, page size, starts (up to), counts, sections, positions
APPEND = {
    "tokens": (8, 1, 16, 4, 128, 64, 300, False, (64,), None),
    "one_token": (1, 1, 1, 1, 64, 16, 0, False, (32,), None),
    "prompt": (3, 133, 4, 2, 64, 24, 50, True, (12, 10, 10), "int"),
    "points": (2, 45, 0, 3, 40, 7, 30, True, (8, 12), "float"),
    "no_rotation": (2, 33, 2, 2, 32, 16, 10, True, (), None),
    "odd_head": (2, 21, 3, 1, 37, 5, 9, True, (17,), None),
    "rest": (2, 21, 6, 3, 96, 32, 9, False, (16, 16), "int"),
    "pages_of_one": (2, 9, 2, 1, 32, 1, 6, True, (16,), None),
    "many": (70, 3, 8, 8, 64, 16, 100, True, (32,), None),
    "far": (2, 4, 2, 1, 64, 4096, 60000, False, (32,), None),
}


def make_append(name, dtype, seed=0):
    B, L, hq, hkv, d, page, past, ragged, sections, positions = APPEND[name]
    g = torch.Generator().manual_seed(zlib.crc32(name.encode()) + seed)
    t = DT[dtype]
    starts = torch.randint(0, past + 1, (B,), generator=g)
    counts = torch.randint(0, L + 1, (B,), generator=g) if ragged else torch.full((B,), L)
    if ragged:
        counts[0], counts[-1] = 0, L
    need = [-(-int(s + n) // page) for s, n in zip(starts, counts)]
    total, width = sum(need) + 2, max(1, max(need))
    qkv = torch.randn((B, L, hq + 2 * hkv, d), generator=g).to(t).cuda()
    q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
    pages = [torch.randn((total, page, hkv, d), generator=g).to(t).cuda() for _ in range(2)]
    table = tables(need, total, width, g)
    how = {"counts": counts.to(torch.int32).cuda() if ragged else None, "query": q if hq else None}
    if sections:
        how["frequencies"] = torch.cat([1000.0 ** (-torch.arange(n, dtype=torch.float64) / n) for n in sections]).float().cuda()
        how["sections"] = sections
        if positions == "float":
            how["positions"] = (torch.rand((B, L, len(sections)), generator=g) * 100).cuda()
        elif positions == "int":
            how["positions"] = torch.randint(0, 200, (B, L, len(sections)), generator=g, dtype=torch.int32).cuda()
    return k, v, pages, table, starts.to(torch.int32).cuda(), counts, how


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(APPEND))
def test_append(name, dtype):
    for layout in ("halves", "adjacent", "blocks"):
        print(f"[gpu-test] append {name} {dtype} {layout}", flush=True)
        k, v, (kp, vp), table, starts, counts, how = make_append(name, dtype)
        B, L, hkv, d = k.shape
        page = kp.shape[1]
        wk, wv, wt = f64(kp), f64(vp), np.zeros(kp.shape)
        got = dcn.paged_append(k, v, kp, vp, table, starts, layout=layout, **how)
        torch.cuda.synchronize()
        lengths, qo = got if how["query"] is not None else (got, None)
        assert torch.equal(lengths.cpu(), (starts.cpu() + counts).to(torch.int32))
        rot, tol = f64(k), np.zeros(k.shape)
        if "sections" in how:
            pos = how.get("positions")
            if pos is None:
                pos = (starts[:, None] + torch.arange(L, device="cuda"))[:, :, None].expand(B, L, len(how["sections"]))
            r = (f64(pos), f64(how["frequencies"]), how["sections"], layout, dtype)
            rot, tol = rotary_oracle.rotate(f64(k), *r)
            if qo is not None:
                check(f64(qo), *rotary_oracle.rotate(f64(how["query"]), *r), "query")
        elif qo is not None:
            assert torch.equal(qo, how["query"])
        for b in range(B):
            for i in range(int(counts[b])):
                s = int(starts[b]) + i
                at = int(table[b, s // page]), s % page
                wk[at], wt[at], wv[at] = rot[b, i], tol[b, i], f64(v[b, i])
        check(f64(kp), wk, wt, "key_pages")
        assert np.array_equal(f64(vp), wv), "value_pages"
        if "sections" not in how:
            break


def test_rows_that_have_no_place():
    """Entries that are no page, positions outside the table, negative starts: not written, nothing else touched."""
    g = torch.Generator().manual_seed(3)
    B, L, H, D, page, total = 4, 6, 2, 32, 4, 9
    k, v = (torch.randn((B, L, H, D), generator=g).cuda() for _ in range(2))
    kp, vp = (torch.randn((total, page, H, D), generator=g).cuda() for _ in range(2))
    table = torch.tensor([[0, -1, 2], [3, total, 4], [5, 6, 7], [8, 1, -3]], dtype=torch.int32, device="cuda")
    starts = torch.tensor([2, 1, 9, -2], dtype=torch.int32, device="cuda")
    wk, wv = kp.clone(), vp.clone()
    for b in range(B):
        for i in range(L):
            s = int(starts[b]) + i
            if 0 <= s < 12 and 0 <= int(table[b, s // page]) < total:
                wk[int(table[b, s // page]), s % page] = k[b, i]
                wv[int(table[b, s // page]), s % page] = v[b, i]
    lengths = dcn.paged_append(k, v, kp, vp, table, starts)
    assert torch.equal(kp, wk) and torch.equal(vp, wv)
    assert torch.equal(lengths, starts + L)
    # counts below 0 and beyond the rows
    counts = torch.tensor([-1, 99, 0, 2], dtype=torch.int32, device="cuda")
    lengths = dcn.paged_append(v, k, kp, vp, table, starts, counts=counts)
    assert torch.equal(lengths, starts + counts.clamp(0, L))
    none = torch.empty((B, 0, H, D), device="cuda")
    before = kp.clone()
    lengths = dcn.paged_append(none, none, kp, vp, table, starts)
    assert torch.equal(lengths, starts) and torch.equal(kp, before)
    empty = torch.empty((0, L, H, D), device="cuda")
    assert dcn.paged_append(empty, empty, kp, vp, table[:0], starts[:0]).shape == (0,)
    no_pages = torch.empty((0, page, H, D), device="cuda")
    assert torch.equal(dcn.paged_append(k, v, no_pages, no_pages, table, starts), starts + L)
    q = torch.randn((B, 4, D), generator=g).cuda()
    out, lse = dcn.paged_attention(q, no_pages, no_pages, table, starts.abs(), return_lse=True)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
    out = dcn.paged_attention(q, kp, vp, table[:, :0], starts.abs())
    assert torch.all(out == 0)
    assert dcn.paged_attention(q[:0], kp, vp, table[:0], starts[:0]).shape == (0, 4, D)


def test_append_strides():
    for shift in (0, 1, 4):
        k, v, (kp, vp), table, starts, counts, how = make_append("prompt", "bf16")
        k2, v2 = k.contiguous(), v.contiguous()
        how2 = dict(how, query=how["query"].contiguous())
        n = kp.numel()
        buf = torch.zeros(2 * n + 8, dtype=kp.dtype, device="cuda")
        # heads first, keys and values in one allocation that starts `shift` elements in
        total, page, h, d = kp.shape
        both = buf[shift:shift + 2 * n].view(total, 2, h, page, d)
        a, b = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
        a.copy_(kp)
        b.copy_(vp)
        l1, q1 = dcn.paged_append(k, v, kp, vp, table, starts, **how)
        l2, q2 = dcn.paged_append(k2, v2, a, b, table, starts, **how2)
        assert torch.equal(kp, a) and torch.equal(vp, b) and torch.equal(q1, q2) and torch.equal(l1, l2)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_prompt_and_tokens(dtype):
    """A decoder's use: a ragged prompt goes to the cache, then token by token; every token's answer is
    that of cross attention over the same rotated keys kept densely."""
    g = torch.Generator().manual_seed(11)
    B, L, steps, hq, hkv, d, page, t = 3, 37, 4, 8, 2, 64, 16, DT[dtype]
    counts = torch.tensor([37, 5, 20], dtype=torch.int32, device="cuda")
    freq = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    width = -(-(L + steps) // page)
    kp, vp = (torch.zeros((B * width, page, hkv, d), dtype=t, device="cuda") for _ in range(2))
    table = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width).cuda()
    dense_k, dense_v = (torch.zeros((B, L + steps, hkv, d), dtype=t, device="cuda") for _ in range(2))
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    for step in range(steps + 1):
        n = L if step == 0 else 1
        qkv = torch.randn((B, n, hq + 2 * hkv, d), generator=g).to(t).cuda()
        q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        new = counts if step == 0 else None
        starts = lengths
        lengths, rq = dcn.paged_append(k, v, kp, vp, table, starts, counts=new, query=q, frequencies=freq, sections=(32,))
        pos = (starts[:, None] + torch.arange(n, device="cuda", dtype=torch.int32))[:, :, None].contiguous()
        rk = dcn.rotary_positions(k, pos, freq, (32,))
        assert torch.equal(rq, dcn.rotary_positions(q, pos, freq, (32,)))
        for b in range(B):
            c, s = int(counts[b]) if step == 0 else 1, int(starts[b])
            dense_k[b, s:s + c], dense_v[b, s:s + c] = rk[b, :c], v[b, :c]
        last = rq[torch.arange(B), (lengths - starts - 1).long()]
        out, lse = dcn.paged_attention(last, kp, vp, table, lengths, return_lse=True)
        mask = torch.arange(L + steps, device="cuda") < lengths[:, None]
        want, wl = dcn.cross_attention(last[:, None], dense_k, dense_v, key_mask=mask, return_lse=True)
        ref = reference(last, kp, vp, table, lengths, dtype)
        check(f64(out), ref[0], ref[1], "paged")
        check(f64(want[:, 0]), ref[0], ref[1], "dense")
        check(f64(lse), ref[2], ref[3], "lse")
        check(f64(wl[:, :, 0]), ref[2], ref[3], "dense lse")


@pytest.mark.parametrize("name", ["one_long_among_short", "lists"])
def test_on_a_side_stream_and_in_graphs(name):
    """A token's step (append, then attention) on another stream, and in two graphs that share a workspace;
    starts and lengths are read on the device at every replay."""
    q, kp, vp, table, lengths = make(name, "bf16")
    B, hq, d = q.shape
    hkv = kp.shape[2]
    g = torch.Generator().manual_seed(2)
    new = torch.randn((B, 1, 2 * hkv, d), generator=g).to(q.dtype).cuda()
    freq = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    desc = dcn.paged_desc(q, kp, vp, table, lengths)
    nb = dcn.dcn_paged_attention_workspace_bytes(desc)
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda")
    starts = (lengths - 1).clamp(min=0)

    def step(kp, vp, starts):
        n, rq = dcn.paged_append(new[:, :, :hkv], new[:, :, hkv:], kp, vp, table, starts, query=q[:, None],
                                 frequencies=freq, sections=(32,))
        return rq, dcn.paged_attention(rq[:, 0], kp, vp, table, n, workspace=ws)

    a, b = kp.clone(), vp.clone()
    want = step(a, b, starts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c, e = kp.clone(), vp.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(c, e, starts)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(s, t) for s, t in zip(want, got)) and torch.equal(a, c) and torch.equal(b, e)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(c, e, starts))
        graphs.append(graph)
    torch.cuda.synchronize()
    first = starts.clone()
    for back in (0, 1, 700, 2000):
        starts.copy_((first - back).clamp(min=0))
        for graph, out in zip(graphs, outs):
            q.mul_(-1)
            graph.replay()
            torch.cuda.synchronize()
            a.copy_(c)
            b.copy_(e)
            want = step(a, b, starts)
            assert all(torch.equal(s, t) for s, t in zip(want, out)), back
            assert torch.equal(a, c) and torch.equal(b, e)
    del graphs


def test_refusals():
    q, kp, vp, table, lengths = make("pages_of_24", "f32")
    f = dcn.paged_attention
    for bad in ((q.double(), kp, vp, table, lengths), (q, kp, vp.bfloat16(), table, lengths),
                (q, kp.bfloat16(), vp.bfloat16(), table, lengths)):
        with pytest.raises(TypeError):
            f(*bad)
    for bad in ((q[0], kp, vp, table, lengths), (q[:, :5], kp, vp, table, lengths), (q[..., :32], kp, vp, table, lengths),
                (q, kp[1:], vp, table, lengths), (q, kp, vp, table.long(), lengths), (q, kp, vp, table[1:], lengths),
                (q, kp, vp, table, lengths.long()), (q, kp, vp, table, lengths[1:]), (q, kp, vp, table[:, ::2], lengths),
                (q, kp.cpu(), vp, table, lengths), (q, kp, vp, table, lengths.cpu()), (q, kp[:, :0], vp[:, :0], table, lengths),
                (q, kp.transpose(2, 3).contiguous().transpose(2, 3), vp, table, lengths)):
        with pytest.raises(ValueError):
            f(*bad)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(dcn.DcnError) as e:
            f(q, kp, vp, table, lengths, scale=scale)
        assert e.value.status == dcn.E_ARG
    wide = torch.zeros((2, 4, 1, 129), device="cuda")
    with pytest.raises(dcn.DcnError) as e:
        f(wide[:, 0], wide, wide, table[:2], lengths[:2])
    assert e.value.status == dcn.E_UNSUPPORTED
    with pytest.raises(ValueError):
        f(*make("one_long", "f32"), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    k, v, (kp, vp), table, starts, counts, how = make_append("prompt", "f32")
    f = dcn.paged_append
    freq = how["frequencies"]
    for bad in ((k[:, 1:], v, kp, vp, table, starts), (k, v, kp, vp, table.long(), starts), (k, v, kp, vp, table, starts.long()),
                (k, v, kp[:, :, :1], vp[:, :, :1], table, starts), (k, v, kp, vp, table, starts[1:]),
                (k, v, kp[:1].expand(kp.shape), vp, table, starts), (k, v, kp.cpu(), vp, table, starts)):
        with pytest.raises(ValueError):
            f(*bad)
    for bad in (dict(counts=counts.cuda().long()), dict(query=how["query"][:, 1:]), dict(sections=(4,)),
                dict(positions=how["positions"]), dict(frequencies=freq, sections=(32, 1)),
                dict(frequencies=freq, sections=how["sections"], positions=how["positions"][..., :2]),
                dict(frequencies=freq, sections=how["sections"], layout="thirds"), dict(frequencies=freq)):
        with pytest.raises(ValueError):
            f(k, v, kp, vp, table, starts, **bad)
    with pytest.raises(TypeError):
        f(k, v.bfloat16(), kp, vp, table, starts)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_of_heads_far_apart(dtype):
    """Strides of heads at and beyond 2^24 elements, of the tokens and of the pages: the same bits as dense."""
    g = torch.Generator().manual_seed(4)
    t = DT[dtype]
    q, k, v = (torch.randn((2, 5, n, 16), generator=g).to(t).cuda() for n in (4, 2, 2))
    freq = torch.rand(8, generator=g).cuda()
    table = torch.tensor([[2, 0], [3, 1]], dtype=torch.int32, device="cuda")
    starts = torch.tensor([1, 3], dtype=torch.int32, device="cuda")

    def run(q, k, v, kp, vp):
        return dcn.paged_append(k, v, kp, vp, table, starts, query=q, frequencies=freq, sections=(8,))

    kp, vp = (torch.zeros((4, 4, 2, 16), dtype=t, device="cuda") for _ in range(2))
    want = run(q, k, v, kp, vp)
    for step in ((1 << 24) - 1, 1 << 24):
        def far(x):
            a, b, n, d = x.shape
            y = torch.empty(n * step + a * b * d, dtype=t, device="cuda").as_strided(x.shape, (b * d, d, step, 1))
            return y.copy_(x)

        for tokens, pages in ((True, False), (False, True), (True, True)):
            args = [far(x) if tokens else x for x in (q, k, v)]
            fk, fv = (far(torch.zeros_like(kp)) if pages else torch.zeros_like(kp) for _ in range(2))
            got = run(*args, fk, fv)
            assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(fk, kp) and torch.equal(fv, vp)
