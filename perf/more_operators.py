"""Serving operators over a KV cache held in 8 bits, and the choice of a token: the cases they are
measured on and their plain forms.

One serving iteration over such a cache, in the order a program runs it:

  append     rotary positions on the new tokens' queries and keys, and their K/V rows rounded to
             8 bits into the pages (kvs_rope_scatter_paged_q8)
  attention  attention of every sequence's new tokens over its pages (kvs_paged_attention_q8)
  sample     a token drawn from each row of logits under temperature, top-k, top-p and min-p with
             given random numbers (kvs_sample_logits)

Pages are [num_pages, Hkv, page_size, D] in float8_e4m3fn, scales [num_pages, Hkv, page_size / 16] in
float32: an element is its block's scale times the stored number.  A block is 16 positions of one kv
head; its scale is the smallest power of two (2^-60 at least) that keeps every row written to it
within 448.  Rows that were there before a larger one arrived are rounded again to the new scale.

Batches are ragged: sequence i brings n_i new tokens at positions p_i .. p_i + n_i - 1, its rows are
row_offsets[i] .. row_offsets[i + 1] of q, k, v and out.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
E4M3 = torch.float8_e4m3fn
BLOCK = 16  # positions that share a scale

# (query heads, kv heads, head size) of the decode workloads
HEADS = ((4, 2, 64), (14, 2, 64), (32, 8, 128), (40, 8, 128))
VOCAB = 152064


def listed():
    return [
        # a decode step of a batch of chats: one new token each, latency is all that counts
        dict(name="append decode", op="append", dtype="bf16", H=32, Hkv=8, D=128, page=64, M=32, new="one",
             rows=32, reach=8192, rot=128, interleaved=False),
        # prompts of a long-context model prefilled together, all of the head rotated
        dict(name="append prompts", op="append", dtype="bf16", H=32, Hkv=8, D=128, page=64, M=5, new="ragged",
             rows=8192, reach=131072, rot=128, interleaved=False),
        # the small model's prompt chunks in 32 bits, a quarter of each head rotated in pairs
        dict(name="append part f32", op="append", dtype="f32", H=14, Hkv=2, D=64, page=16, M=3, new="ragged",
             rows=1531, reach=2048, rot=16, interleaved=True),
        # the small model's decode step in 32 bits
        dict(name="decode small f32", op="attention", dtype="f32", H=14, Hkv=2, D=64, page=16, M=4, new="one",
             rows=4, reach=2048, lengths="uniform"),
        # a decode step of a batch of 32 chats
        dict(name="decode batch", op="attention", dtype="bf16", H=32, Hkv=8, D=128, page=64, M=32, new="one",
             rows=32, reach=8192, lengths="uniform"),
        # a decode step over long contexts: the cache is all that is read
        dict(name="decode long", op="attention", dtype="f16", H=32, Hkv=8, D=128, page=128, M=8, new="one",
             rows=8, reach=32768, lengths="full"),
        # a prompt's second chunk over the pages of its first
        dict(name="chunk long", op="attention", dtype="bf16", H=32, Hkv=8, D=128, page=64, M=1, new="ragged",
             rows=4096, reach=8192, lengths="full"),
        # prompt chunks beside sequences that decode, in one call
        dict(name="chunks and decodes", op="attention", dtype="f16", H=40, Hkv=8, D=128, page=32, M=9, new="mixed",
             rows=1700, reach=5000, lengths="uniform"),
        # the next token of one chat
        dict(name="sample one", op="sample", dtype="f32", M=1, V=VOCAB, k=True, p=True, least=False, probs=False),
        # a batch of chats, each with settings of its own
        dict(name="sample batch", op="sample", dtype="f32", M=32, V=VOCAB, k=True, p=True, least=True, probs=False),
        # a larger batch in 16 bits over an odd vocabulary, the nucleus alone
        dict(name="sample bf16 odd", op="sample", dtype="bf16", M=67, V=32001, k=False, p=True, least=False, probs=False),
        # a draft model's tokens with the distributions that the check against the large model needs
        dict(name="sample draft", op="sample", dtype="f16", M=24, V=VOCAB, k=True, p=False, least=True, probs=True),
    ]


def spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(("append", "attention", "attention", "sample"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    if op == "sample":
        return dict(op=op, dtype=dtype, M=spread(rng, 1, 64), V=spread(rng, 1000, VOCAB), k=rng.random() < 0.6,
                    p=rng.random() < 0.6, least=rng.random() < 0.4, probs=rng.random() < 0.25)
    H, Hkv, D = rng.choice(HEADS)
    page = rng.choice((16, 32, 64, 128, 256))
    case = dict(op=op, dtype=dtype, H=H, Hkv=Hkv, D=D, page=page)
    if op == "append":
        M = spread(rng, 1, 64)
        new = rng.choice(("one", "ragged", "mixed"))
        rows = M if new == "one" else M + spread(rng, 1, 8000)
        return dict(case, M=M, new=new, rows=rows, reach=max(spread(rng, 64, 131072), rows + 1),
                    rot=rng.choice((D, D, D // 2, D // 4, D - 8)), interleaved=rng.random() < 0.5)
    new = rng.choice(("one", "ragged", "mixed"))
    lengths = rng.choice(("uniform", "full"))
    if new == "one":
        M = spread(rng, 1, 64)
        return dict(case, M=M, new=new, rows=M, reach=spread(rng, 16, 240000 // M), lengths=lengths)
    M = spread(rng, 1, 16)
    rows = M + spread(rng, 1, 700 if dtype == "f32" else 1400)
    return dict(case, M=M, new=new, rows=rows, reach=max(rows + 1, spread(rng, 64, min(12000, 40000 // M + rows))),
                lengths=lengths)


def shares(case, seed):
    """New tokens and first position of each sequence: (n, p), lists of M."""
    r = random.Random("%s %s" % (sorted((k, v) for k, v in case.items() if k != "name"), seed))
    M, rows = case["M"], case["rows"]
    if case["new"] == "one":
        n = [1] * M
    else:
        # "mixed": two sequences in three decode, the others share the rest
        long = [i for i in range(M) if case["new"] == "ragged" or i % 3 == 1] or [0]
        n = [0 if i in long else 1 for i in range(M)]
        cuts = sorted(r.random() for _ in long[1:])
        left = rows - sum(n)
        ends = [0] + [int(c * left) for c in cuts] + [left]
        for j, i in enumerate(long):
            n[i] = ends[j + 1] - ends[j]
    full = case.get("lengths") == "full"
    p = [max(0, case["reach"] - k if full else r.randrange(0, max(1, case["reach"] - k + 1))) for k in n]
    return n, p


def normal(g, *shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def held(x):
    """Rows [pages, Hkv, page, D] as the cache holds them: the numbers in 8 bits and the scales."""
    b = x.unflatten(2, (-1, BLOCK))
    scale = scale_of(b.abs().amax((3, 4)).float())
    return (b / scale[..., None, None].to(x.dtype)).to(E4M3).flatten(2, 3), scale


def scale_of(most):
    """The power of two that keeps what is `most` in size within 448 = 0.875 2^9."""
    m, e = torch.frexp(most)
    k = (e - 9 + (m > 0.875)).clamp_min(-60)
    return torch.ldexp(torch.ones_like(most), torch.where(most > 0, k, -60))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    dtype = DTYPES[case["dtype"]]
    r = np.random.default_rng(seed)
    if case["op"] == "sample":
        # most tokens far behind, some dozens in front, as a model's logits are
        M, V = case["M"], case["V"]
        x = 2 * normal(g, M, V, dtype=torch.float32)
        front = torch.from_numpy(r.integers(0, V, (M, 40))).cuda()
        x.scatter_(1, front, torch.from_numpy(r.uniform(6, 14, (M, 40)).astype(np.float32)).cuda())
        s["logits"] = x.to(dtype)
        s["uniforms"] = torch.from_numpy(r.random(M, dtype=np.float32)).cuda()
        t = r.uniform(0.5, 1.5, M)
        t[np.arange(M) % 11 == 7] = 0.0  # one row in eleven is greedy
        s["temperature"] = torch.from_numpy(t.astype(np.float32)).cuda()
        s["top_k"] = torch.from_numpy(r.choice((0, 20, 50, 400, 3000), M).astype(np.int32)).cuda() if case["k"] else None
        p = np.where(np.arange(M) % 4 == 3, 1.0, r.uniform(0.7, 0.99, M))
        s["top_p"] = torch.from_numpy(p.astype(np.float32)).cuda() if case["p"] else None
        s["min_p"] = torch.from_numpy(r.choice((0.0, 0.02, 0.1), M).astype(np.float32)).cuda() if case["least"] else None
        s["token_ids"] = torch.empty(M, dtype=torch.int32, device="cuda")
        s["token_probs"] = torch.empty(M, dtype=torch.float32, device="cuda")
        s["out"] = torch.empty(M, V, dtype=torch.float32, device="cuda") if case["probs"] else None
        return s
    H, Hkv, D, page, M, rows = (case[k] for k in ("H", "Hkv", "D", "page", "M", "rows"))
    n, p = shares(case, seed)
    need = [-(-(a + b) // page) for a, b in zip(n, p)]
    table = np.full((M, max(need) + 1), -1, np.int32)
    if case["op"] == "append":  # page 0 stands for the prefix that all share; what is written has pages of its own
        first = [a // page for a in p]
        order = r.permutation(sum(max(0, b - a) for a, b in zip(first, need))) + 1
        at = 0
        for i in range(M):
            table[i, :first[i]] = 0
            table[i, first[i]:need[i]] = order[at:at + max(0, need[i] - first[i])]
            at += max(0, need[i] - first[i])
        num_pages = 1 + rows // page + 2 * M
    else:
        order, at = r.permutation(sum(need)), 0
        for i in range(M):
            table[i, :need[i]] = order[at:at + need[i]]
            at += need[i]
        num_pages = sum(need)
    s["page_table"] = torch.from_numpy(table).cuda()
    s["positions"] = torch.tensor(p, dtype=torch.int32, device="cuda")
    s["row_offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    s["max_new"] = max(n)
    for name in ("k", "v"):  # kv heads differ in size, and so do stretches of the context
        x = normal(g, num_pages, Hkv, page, D, dtype=torch.float16)
        x *= torch.rand(num_pages, Hkv, page // BLOCK, 1, device="cuda", generator=g).add_(0.5).half() \
            .repeat_interleave(BLOCK, 2)
        s[name + "_pages"], s[name + "_scales"] = held(x)
        del x
    s["out"] = torch.empty(rows, H, D, dtype=dtype, device="cuda")
    if case["op"] == "append":
        # q, k and v are column blocks of one product's rows
        qkv = normal(g, rows, (H + 2 * Hkv) * D, dtype=dtype)
        s["q"] = qkv[:, :H * D].unflatten(1, (H, D))
        s["k"] = qkv[:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (H + Hkv) * D:].unflatten(1, (Hkv, D))
        j = np.arange(case["rot"] // 2)
        s["inv_freq"] = torch.from_numpy((10000.0 ** (-2.0 * j / case["rot"])).astype(np.float32)).cuda()
        s["scale"] = 1.0
    else:
        s["q"] = normal(g, rows, H, D, dtype=dtype)
    if own:  # what a serving program makes once: the cache's and the batch's handles, the workspace
        import split_flash_decoding_kvcachescatter_gb300 as kvs
        s["cache"] = kvs.PagedCacheQ8(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        s["batch"] = kvs.PagedBatch(s["positions"], s["row_offsets"], s["page_table"], num_rows=rows, max_new=s["max_new"])
        if case["op"] == "attention":
            s["workspace"] = kvs.paged_attention_q8_workspace(s["cache"], s["batch"], H)
    return s


def run(s):
    if own:
        import split_flash_decoding_kvcachescatter_gb300 as kvs
        if s["op"] == "append":
            kvs.kvs_rope_scatter_paged_q8(s["q"], s["k"], s["v"], s["out"], s["cache"], s["batch"], s["inv_freq"],
                                          interleaved=s["interleaved"], scale=s["scale"])
            return s["out"], s["k_pages"], s["k_scales"], s["v_pages"], s["v_scales"]
        if s["op"] == "attention":
            kvs.kvs_paged_attention_q8(s["q"], s["cache"], s["batch"], s["out"], workspace=s["workspace"])
            return s["out"]
        kvs.kvs_sample_logits(s["logits"], s["uniforms"], token_ids=s["token_ids"], temperature=s["temperature"],
                              top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], token_probs=s["token_probs"],
                              probs=s["out"])
        return s["token_ids"], s["token_probs"], s["out"]
    return {"append": plain_append, "attention": plain_attention, "sample": plain_sample}[s["op"]](s)


def rows_of(offsets, count):
    """The row of the ragged list that each of `count` entries is in."""
    at = torch.arange(count, device="cuda", dtype=torch.int32)
    return torch.searchsorted(offsets, at, right=True) - 1, at


def rotated(x, cos, sin, rot, interleaved):
    """The heads of x [rows, heads, D] (32 bits) turned by the angles of [rows, rot / 2]."""
    part = x[..., :rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else part.chunk(2, -1)
    c, s = cos[:, None], sin[:, None]
    u, v = a * c - b * s, b * c + a * s
    turned = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def plain_append(s):
    seq, at = rows_of(s["row_offsets"], s["rows"])
    pos = s["positions"][seq] + at - s["row_offsets"][seq]
    angle = pos[:, None].double() * s["inv_freq"].double()
    cos, sin = angle.cos().float() * s["scale"], angle.sin().float() * s["scale"]
    s["out"].copy_(rotated(s["q"].float(), cos, sin, s["rot"], s["interleaved"]))
    page, slot = s["page_table"][seq, pos // s["page"]].long(), (pos % s["page"]).long()
    block = page * (s["page"] // BLOCK) + slot // BLOCK
    # a sequence's first new row that does not open its block finds older rows in it: so many
    first = torch.where(at == s["row_offsets"][seq], pos % BLOCK, 0)
    older = torch.zeros(s["k_scales"].shape[0] * (s["page"] // BLOCK), dtype=torch.int32, device="cuda")
    new = torch.zeros_like(older).index_add_(0, block, torch.ones_like(at)) > 0
    older.index_add_(0, block, first)
    shape = (s["k_scales"].shape[0], 1, -1)
    older, new = older.view(shape), new.view(shape)
    behind = torch.arange(s["page"], device="cuda") % BLOCK >= older.repeat_interleave(BLOCK, 2)
    for name, x in (("k", rotated(s["k"].float(), cos, sin, s["rot"], s["interleaved"])), ("v", s["v"].float())):
        pages, scales = s[name + "_pages"], s[name + "_scales"]
        most = torch.zeros(new.numel(), s["Hkv"], device="cuda").index_reduce_(0, block, x.abs().amax(2), "amax")
        need = scale_of(most).view(scales.shape[0], -1, s["Hkv"]).transpose(1, 2)
        scale = torch.where(new, torch.where(older > 0, torch.maximum(need, scales), need), scales)
        # older rows are rounded again where the scale has grown
        ratio = (scales / scale).repeat_interleave(BLOCK, 2)[..., None]
        values = pages.float()
        pages.copy_(torch.where((behind | (ratio[..., 0] >= 1))[..., None], values, values * ratio).to(E4M3))
        scales.copy_(scale)
        pages[page, :, slot] = (x / scale[page, :, slot // BLOCK][..., None]).to(E4M3)
    return s["out"], s["k_pages"], s["k_scales"], s["v_pages"], s["v_scales"]


def values_of(s, name, table):
    """The rows of every sequence's pages as the values they stand for, [M, Hkv, keys, D]."""
    x = s[name + "_pages"][table].float()
    x *= s[name + "_scales"][table].repeat_interleave(BLOCK, 3)[..., None]
    return x.transpose(1, 2).flatten(2, 3)


def plain_attention(s):
    H, Hkv, D, M, most = s["H"], s["Hkv"], s["D"], s["M"], s["max_new"]
    start, pos = s["row_offsets"][:-1], s["positions"]
    t = torch.arange(most, device="cuda", dtype=torch.int32)
    row = (start[:, None] + t).clamp_max(s["rows"] - 1)  # [M, most], those past n are left out at the end
    q = s["q"].float()[row].view(M, most, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(M, Hkv, -1, D)
    table = s["page_table"].clamp_min(0)
    k, v = values_of(s, "k", table), values_of(s, "v", table)
    score = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(M, Hkv, H // Hkv, most, -1)
    key = torch.arange(score.shape[-1], device="cuda", dtype=torch.int32)
    hidden = key > (pos[:, None] + t)[..., None]  # [M, most, keys]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    score = score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    out = (score.view(M, Hkv, -1, score.shape[-1]) @ v).view(M, Hkv, H // Hkv, most, D) / total
    seq, at = rows_of(s["row_offsets"], s["rows"])
    s["out"].copy_(out.permute(0, 3, 1, 2, 4).reshape(M, most, H, D)[seq, at - start[seq]])
    return s["out"]


def plain_sample(s):
    M, V = s["M"], s["V"]
    value, token = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    weight = ((value - value[:, :1]) / torch.where(t > 0, t, 1.0)).exp()
    place = torch.arange(V, device="cuda")
    weight = torch.where((t > 0) | (place == 0), weight, 0.0)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        weight = torch.where((k <= 0) | (place < k), weight, 0.0)
    keep = weight > 0
    if s["top_p"] is not None:
        p, before = s["top_p"].double()[:, None], weight.cumsum(1)
        keep &= (p >= 1) | (before - weight < p * before[:, -1:]) | (place == 0)
    if s["min_p"] is not None:
        keep &= weight >= s["min_p"].double()[:, None]
    kept = torch.zeros_like(weight).scatter_(1, token, torch.where(keep, weight, 0.0))
    run = kept.cumsum(1)
    mark = s["uniforms"].double()[:, None] * run[:, -1:]
    chosen = (run <= mark).sum(1, dtype=torch.int32)
    s["token_ids"].copy_(torch.minimum(chosen, (run < run[:, -1:]).sum(1, dtype=torch.int32)))
    kept /= run[:, -1:]
    s["token_probs"].copy_(kept.gather(1, s["token_ids"].long()[:, None])[:, 0])
    if s["out"] is not None:
        s["out"].copy_(kept)
    return s["token_ids"], s["token_probs"], s["out"]


def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] == "sample":
        M, V = case["M"], case["V"]
        return {"bytes": M * V * (size + (4 if case["probs"] else 0)) + 28 * M, "flops": 4 * M * V}
    H, Hkv, D, rows = case["H"], case["Hkv"], case["D"], case["rows"]
    if case["op"] == "append":
        return {"bytes": rows * ((2 * H + 2 * Hkv) * D * size + 2 * Hkv * D) + 8 * Hkv * (rows // BLOCK + case["M"])
                + 12 * case["M"] + 2 * case["rot"], "flops": 3 * rows * (H + Hkv) * case["rot"] + 4 * rows * Hkv * D}
    n, p = shares(case, 0)
    lengths = case["reach"] / 2 if case["lengths"] == "uniform" else None
    keys = sum((min(lengths, case["reach"] - a / 2) + a / 2) if lengths else b + a for a, b in zip(n, p) if a)
    pairs = sum(a * ((min(lengths, case["reach"] - a / 2) - a / 2 if lengths else b) + (a + 1) / 2) for a, b in zip(n, p))
    return {"bytes": 2 * keys * Hkv * (D + 4 / BLOCK) + 2 * rows * H * D * size, "flops": 4 * max(pairs, rows) * H * D}


def to_e4m3(x):
    """x in 64 bits to the nearest number of e4m3, ties to even: three bits behind the leading one, steps of 2^-9 at least."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    """What run() returns, by the definitions in 64 bits, a sequence, a block or a row at a time."""
    s = prepare(case, seed)
    if case["op"] == "sample":
        return exact_sample(s, case)
    n, p = shares(case, seed)
    D, page, Hkv = case["D"], case["page"], case["Hkv"]
    table = s["page_table"].cpu().tolist()
    ends = np.concatenate([[0], np.cumsum(n)])
    if case["op"] == "append":
        pos = torch.cat([torch.arange(a, a + b, dtype=torch.float64) for a, b in zip(p, n)]).cuda()
        w = s["inv_freq"].to(torch.float64)
        turn = torch.polar(torch.full((len(pos), len(w)), s["scale"], dtype=torch.float64, device="cuda"), torch.outer(pos, w))

        def turned(x):
            x = x.to(torch.float64).clone()
            half = case["rot"] // 2
            re, im = (slice(0, case["rot"], 2), slice(1, case["rot"], 2)) if case["interleaved"] else (slice(0, half), slice(half, 2 * half))
            z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * turn[:, None]
            x[..., re], x[..., im] = z.real, z.imag
            return x
        found = [turned(s["q"])]
        for name, x in (("k", turned(s["k"])), ("v", s["v"].to(torch.float64))):
            codes, scales = s[name + "_pages"].to(torch.float64), s[name + "_scales"].to(torch.float64)
            for i in range(case["M"]):
                a = p[i]
                while a < p[i] + n[i]:  # positions a .. b - 1 lie in one block
                    b = min(p[i] + n[i], a // BLOCK * BLOCK + BLOCK)
                    at, lo = table[i][a // page], a % page
                    j = lo // BLOCK
                    rows = x[int(ends[i]) + a - p[i]:int(ends[i]) + b - p[i]]
                    want = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((0, 2)) / 448)).clamp_min(-60))
                    if a % BLOCK:
                        want = torch.maximum(want, scales[at, :, j])
                        older = slice(j * BLOCK, lo)
                        codes[at, :, older] = to_e4m3(codes[at, :, older] * (scales[at, :, j] / want)[:, None, None])
                    scales[at, :, j] = want
                    codes[at, :, lo:lo + b - a] = to_e4m3(rows.transpose(0, 1) / want[:, None, None])
                    a = b
            found += [codes, scales]
        return tuple(found)
    G = case["H"] // Hkv
    out = torch.zeros(case["rows"], case["H"], D, dtype=torch.float64, device="cuda")
    for i in range(case["M"]):
        if not n[i]:
            continue
        L = p[i] + n[i]
        use = table[i][:-(-L // page)]
        for h in range(Hkv):
            k, v = (s[x + "_pages"][use, h].to(torch.float64).view(-1, BLOCK, D)
                    * s[x + "_scales"][use, h].to(torch.float64).view(-1, 1, 1) for x in ("k", "v"))
            k, v = k.view(-1, D)[:L], v.view(-1, D)[:L]
            for a in range(0, n[i], 512):
                b = min(n[i], a + 512)
                q = s["q"][int(ends[i]) + a:int(ends[i]) + b, h * G:(h + 1) * G].to(torch.float64)
                z = torch.einsum("tgd,ld->tgl", q, k) / D ** 0.5
                far = torch.arange(L, device="cuda")[None] > torch.arange(p[i] + a, p[i] + b, device="cuda")[:, None]
                w = torch.softmax(z.masked_fill(far[:, None], -torch.inf), -1)
                out[int(ends[i]) + a:int(ends[i]) + b, h * G:(h + 1) * G] = torch.einsum("tgl,ld->tgd", w, v)
    return out


def exact_sample(s, case):
    at = {k: None if s[k] is None else s[k].cpu().numpy() for k in ("uniforms", "temperature", "top_k", "top_p", "min_p")}
    x = s["logits"].cpu().to(torch.float64).numpy()
    M, V = x.shape
    ids, odds, probs = np.zeros(M, np.int64), np.zeros(M), np.zeros((M, V))
    for m in range(M):
        order = np.lexsort((np.arange(V), -x[m]))
        t = float(at["temperature"][m])
        if t > 0:
            if at["top_k"] is not None and at["top_k"][m] > 0:
                order = order[:at["top_k"][m]]
            w = np.exp((x[m, order] - x[m, order[0]]) / t)
            if at["top_p"] is not None and at["top_p"][m] < 1:
                sums = np.cumsum(w)
                count = int(np.searchsorted(sums, float(at["top_p"][m]) * sums[-1])) + 1
                order, w = order[:count], w[:count]
            if at["min_p"] is not None:
                order, w = order[w >= at["min_p"][m]], w[w >= at["min_p"][m]]
        else:
            order, w = order[:1], np.ones(1)
        probs[m, order] = w / w.sum()
        # the first id at which the running sum, in the order of ids, is above the random number
        ids[m] = min(int(np.searchsorted(np.cumsum(probs[m]), float(at["uniforms"][m]), side="right")), int(order.max()))
        odds[m] = probs[m, ids[m]]
    return ids, odds, probs if case["probs"] else None
