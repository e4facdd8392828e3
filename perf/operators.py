"""Paged-cache serving operators: the cases they are measured on and their plain forms.

One serving iteration over a paged KV cache, in the order a program runs it:

  rope       rotary positions on the new tokens' queries and keys, and their K/V rows written
             into the pages (kvs_rope_scatter_paged)
  attention  attention of every sequence's new tokens over its pages (kvs_paged_attention)
  logits     penalties, biases and grammar masks on the logits, and the greedy token
             (kvs_process_logits)

Batches are ragged: sequence i brings n_i new tokens at positions p_i .. p_i + n_i - 1, its rows are
row_offsets[i] .. row_offsets[i + 1] of q, k, v and out.  Pages are [num_pages, Hkv, page_size, D].
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}

# (query heads, kv heads, head size) of the decode workloads
HEADS = ((4, 2, 64), (14, 2, 64), (32, 8, 128), (40, 8, 128))
VOCAB = 152064


def listed():
    return [
        # a decode step of a batch of chats: one new token each, latency is all that counts
        dict(name="rope decode", op="rope", dtype="bf16", H=32, Hkv=8, D=128, page=64, M=32, new="one",
             rows=32, reach=8192, rot=128, interleaved=False),
        # prompts of a long-context model prefilled together, all of the head rotated
        dict(name="rope prompts", op="rope", dtype="bf16", H=32, Hkv=8, D=128, page=64, M=5, new="ragged",
             rows=8192, reach=131072, rot=128, interleaved=False),
        # the small model's prompt chunk in 32 bits, a quarter of each head rotated in pairs
        dict(name="rope part f32", op="rope", dtype="f32", H=14, Hkv=2, D=64, page=16, M=3, new="ragged",
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
        # a chunk of the small model's prompt in 32 bits
        dict(name="chunk f32", op="attention", dtype="f32", H=14, Hkv=2, D=64, page=32, M=3, new="ragged",
             rows=1001, reach=2048, lengths="uniform"),
        # a prompt's second chunk over the pages of its first
        dict(name="chunk long", op="attention", dtype="bf16", H=32, Hkv=8, D=128, page=64, M=1, new="ragged",
             rows=4096, reach=8192, lengths="full"),
        # prompt chunks beside sequences that decode, in one call
        dict(name="chunks and decodes", op="attention", dtype="f16", H=40, Hkv=8, D=128, page=32, M=9, new="mixed",
             rows=1700, reach=5000, lengths="uniform"),
        # greedy decoding of one chat under penalties
        dict(name="logits one", op="logits", dtype="f32", M=1, V=VOCAB, history=2048, bias=4, masked=False),
        # a batch of chats, half of them under a grammar
        dict(name="logits batch", op="logits", dtype="f32", M=32, V=VOCAB, history=4096, bias=64, masked=True),
        # a larger batch in 16 bits, over an odd vocabulary
        dict(name="logits bf16 odd", op="logits", dtype="bf16", M=67, V=32001, history=700, bias=17, masked=True),
    ]


def spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(("rope", "attention", "attention", "logits"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    if op == "logits":
        M = spread(rng, 1, 64)
        return dict(op=op, dtype=dtype, M=M, V=spread(rng, 1000, VOCAB), history=spread(rng, 1, 8192),
                    bias=rng.randrange(0, 100), masked=rng.random() < 0.5)
    H, Hkv, D = rng.choice(HEADS)
    page = rng.choice((16, 32, 64, 128, 256))
    case = dict(op=op, dtype=dtype, H=H, Hkv=Hkv, D=D, page=page)
    if op == "rope":
        M = spread(rng, 1, 64)
        new = rng.choice(("one", "ragged", "mixed"))
        rows = M if new == "one" else M + spread(rng, 1, 8000)
        return dict(case, M=M, new=new, rows=rows, reach=max(spread(rng, 64, 131072), rows + 1),
                    rot=rng.choice((D, D, D // 2, D // 4, D - 8)), interleaved=rng.random() < 0.5)
    new = rng.choice(("one", "ragged", "mixed"))
    lengths = rng.choice(("uniform", "full"))
    if new == "one":
        M = spread(rng, 1, 64)
        return dict(case, M=M, new=new, rows=M, reach=spread(rng, 16, 480000 // (M * SIZE[dtype])), lengths=lengths)
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


def pages_of(case, n, p):
    return [-(-(a + b) // case["page"]) for a, b in zip(n, p)]


def normal(g, *shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "logits":
        M, V = case["M"], case["V"]
        r = np.random.default_rng(seed)
        lens = r.integers(case["history"] // 2, case["history"] + 1, M)
        s["logits"] = 4 * normal(g, M, V, dtype=dtype)
        s["history"] = torch.from_numpy(np.minimum(r.zipf(1.3, int(lens.sum())) - 1, V - 1).astype(np.int32)).cuda()
        s["history_offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
        s["prompt_lens"] = torch.from_numpy((lens * r.random(M)).astype(np.int32)).cuda()
        s["repetition"] = torch.from_numpy(r.uniform(1.0, 1.4, M).astype(np.float32)).cuda()
        s["presence"] = torch.from_numpy(r.uniform(-0.5, 1.0, M).astype(np.float32)).cuda()
        s["frequency"] = torch.from_numpy(r.uniform(-0.1, 0.5, M).astype(np.float32)).cuda()
        ids = np.stack([np.sort(r.choice(V, case["bias"], replace=False)) for _ in range(M)])
        s["bias_ids"] = torch.from_numpy(ids.reshape(-1).astype(np.int32)).cuda()
        s["bias_values"] = torch.from_numpy(r.uniform(-8, 8, ids.size).astype(np.float32)).cuda()
        s["bias_offsets"] = torch.from_numpy((np.arange(M + 1) * case["bias"]).astype(np.int32)).cuda()
        s["mask"] = s["mask_rows"] = None
        if case["masked"]:  # a grammar leaves about a hundredth of the vocabulary
            rows = (M + 1) // 2
            words = (r.random((rows, (V + 31) // 32, 32)) < 0.01).astype(np.uint8)
            words[:, 0, 0] = 1
            s["mask"] = torch.from_numpy(np.packbits(words, axis=2, bitorder="little").view(np.int32)[..., 0].copy()).cuda()
            s["mask_rows"] = torch.from_numpy(np.where(np.arange(M) % 2 == 0, np.arange(M) // 2, -1).astype(np.int32)).cuda()
        s["out"] = torch.empty_like(s["logits"])
        s["token_ids"] = torch.empty(M, dtype=torch.int32, device="cuda")
        return s
    H, Hkv, D, page, M, rows = (case[k] for k in ("H", "Hkv", "D", "page", "M", "rows"))
    n, p = shares(case, seed)
    need = pages_of(case, n, p)
    r = np.random.default_rng(seed)
    table = np.full((M, max(need) + 1), -1, np.int32)
    if case["op"] == "rope":  # page 0 stands for the prefix that all share; what is written has pages of its own
        first = [a // page for a in p]
        order = r.permutation(sum(b - a for a, b in zip(first, need))) + 1
        at = 0
        for i in range(M):
            table[i, :first[i]] = 0
            table[i, first[i]:need[i]] = order[at:at + need[i] - first[i]]
            at += need[i] - first[i]
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
    s["k_pages"] = normal(g, num_pages, Hkv, page, D, dtype=dtype)
    s["v_pages"] = normal(g, num_pages, Hkv, page, D, dtype=dtype)
    if case["op"] == "rope":
        # q, k and v are column blocks of one product's rows
        qkv = normal(g, rows, (H + 2 * Hkv) * D, dtype=dtype)
        s["q"] = qkv[:, :H * D].unflatten(1, (H, D))
        s["k"] = qkv[:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (H + Hkv) * D:].unflatten(1, (Hkv, D))
        j = np.arange(case["rot"] // 2)
        s["inv_freq"] = torch.from_numpy((10000.0 ** (-2.0 * j / case["rot"])).astype(np.float32)).cuda()
        s["scale"] = 1.0
        s["out"] = torch.empty(rows, H, D, dtype=dtype, device="cuda")
    else:
        s["q"] = normal(g, rows, H, D, dtype=dtype)
        s["out"] = torch.empty(rows, H, D, dtype=dtype, device="cuda")
    if own:  # what a serving program makes once: the cache's and the batch's handles, the workspace
        import split_flash_decoding_kvcachescatter_gb300 as kvs
        s["cache"] = kvs.PagedCache(s["k_pages"], s["v_pages"])
        s["batch"] = kvs.PagedBatch(s["positions"], s["row_offsets"], s["page_table"], num_rows=rows, max_new=s["max_new"])
        if case["op"] == "attention":
            s["workspace"] = kvs.paged_attention_workspace(s["cache"], s["batch"], H)
    return s


def run(s):
    if own:
        import split_flash_decoding_kvcachescatter_gb300 as kvs
        if s["op"] == "rope":
            kvs.kvs_rope_scatter_paged(s["q"], s["k"], s["v"], s["out"], s["cache"], s["batch"], s["inv_freq"],
                                       interleaved=s["interleaved"], scale=s["scale"])
            return s["out"], s["k_pages"], s["v_pages"]
        if s["op"] == "attention":
            kvs.kvs_paged_attention(s["q"], s["cache"], s["batch"], s["out"], workspace=s["workspace"])
            return s["out"]
        kvs.kvs_process_logits(s["logits"], s["out"], token_ids=s["token_ids"], history=s["history"],
                               history_offsets=s["history_offsets"], prompt_lens=s["prompt_lens"],
                               repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                               bias_ids=s["bias_ids"], bias_values=s["bias_values"], bias_offsets=s["bias_offsets"],
                               mask=s["mask"], mask_rows=s["mask_rows"])
        return s["out"], s["token_ids"]
    return {"rope": plain_rope, "attention": plain_attention, "logits": plain_logits}[s["op"]](s)


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


def plain_rope(s):
    seq, at = rows_of(s["row_offsets"], s["rows"])
    pos = s["positions"][seq] + at - s["row_offsets"][seq]
    angle = pos[:, None].double() * s["inv_freq"].double()
    cos, sin = angle.cos().float() * s["scale"], angle.sin().float() * s["scale"]
    q = rotated(s["q"].float(), cos, sin, s["rot"], s["interleaved"])
    k = rotated(s["k"].float(), cos, sin, s["rot"], s["interleaved"])
    s["out"].copy_(q)
    page, slot = s["page_table"][seq, pos // s["page"]].long(), (pos % s["page"]).long()
    s["k_pages"][page, :, slot] = k.to(s["k_pages"].dtype)
    s["v_pages"][page, :, slot] = s["v"]
    return s["out"], s["k_pages"], s["v_pages"]


def plain_attention(s):
    H, Hkv, D, page, M, most = s["H"], s["Hkv"], s["D"], s["page"], s["M"], s["max_new"]
    start, pos = s["row_offsets"][:-1], s["positions"]
    n = s["row_offsets"][1:] - start
    t = torch.arange(most, device="cuda", dtype=torch.int32)
    row = (start[:, None] + t).clamp_max(s["rows"] - 1)  # [M, most], those past n are left out at the end
    q = s["q"].float()[row].view(M, most, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(M, Hkv, -1, D)
    table = s["page_table"].clamp_min(0)
    k = s["k_pages"][table].transpose(1, 2).reshape(M, Hkv, -1, D).float()
    v = s["v_pages"][table].transpose(1, 2).reshape(M, Hkv, -1, D).float()
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


def plain_logits(s):
    M, V = s["M"], s["V"]
    x = s["logits"].float()
    seq, at = rows_of(s["history_offsets"], s["history"].numel())
    made = at - s["history_offsets"][seq] >= s["prompt_lens"][seq]
    one = torch.ones_like(s["history"], dtype=torch.int32)
    token = s["history"].long()
    seen = torch.zeros(M, V, dtype=torch.int32, device="cuda").index_put_((seq, token), one, accumulate=True) > 0
    count = torch.zeros(M, V, dtype=torch.int32, device="cuda").index_put_((seq, token), made.int(), accumulate=True)
    rep = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * count.float()
    x = x - s["presence"][:, None] * (count > 0).float()
    brow, _ = rows_of(s["bias_offsets"], s["bias_ids"].numel())
    x = x.index_put((brow, s["bias_ids"].long()), s["bias_values"], accumulate=True)
    if s["mask"] is not None:
        v = torch.arange(V, device="cuda")
        bits = (s["mask"][s["mask_rows"].clamp_min(0)][:, v // 32] >> (v % 32).int()) & 1
        x = x.masked_fill((bits == 0) & (s["mask_rows"] >= 0)[:, None], -math.inf)
    s["out"].copy_(x)
    y = s["out"].float()
    best = torch.where(y == y.amax(1, keepdim=True), torch.arange(V, device="cuda", dtype=torch.int32), V)
    s["token_ids"].copy_(best.amin(1))
    return s["out"], s["token_ids"]


def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] == "logits":
        M, V = case["M"], case["V"]
        small = M * (case["history"] * 3 + case["bias"] * 8 + 40) + (M * V // 16 if case["masked"] else 0)
        return {"bytes": 2 * M * V * size + small, "flops": 2 * M * V}
    H, Hkv, D, rows = case["H"], case["Hkv"], case["D"], case["rows"]
    if case["op"] == "rope":
        return {"bytes": 2 * rows * (H + 2 * Hkv) * D * size + 12 * case["M"] + 2 * case["rot"],
                "flops": 3 * rows * (H + Hkv) * case["rot"]}
    n, p = shares(case, 0)
    lengths = case["reach"] / 2 if case["lengths"] == "uniform" else None
    keys = sum((min(lengths, case["reach"] - a / 2) + a / 2) if lengths else b + a for a, b in zip(n, p) if a)
    pairs = sum(a * ((min(lengths, case["reach"] - a / 2) - a / 2 if lengths else b) + (a + 1) / 2) for a, b in zip(n, p))
    return {"bytes": 2 * keys * Hkv * D * size + 2 * rows * H * D * size, "flops": 4 * max(pairs, rows) * H * D}


def exact(case, seed):
    """What run() returns, by the definitions in 64 bits, a sequence or a row at a time."""
    s = prepare(case, seed)
    if case["op"] == "logits":
        return exact_logits(s, case)
    n, p = shares(case, seed)
    D, page = case["D"], case["page"]
    table = s["page_table"].cpu().tolist()
    ends = np.concatenate([[0], np.cumsum(n)])
    if case["op"] == "rope":
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
        k, v = s["k_pages"].to(torch.float64), s["v_pages"].to(torch.float64)
        new = turned(s["k"])
        for i in range(case["M"]):
            for j in range(p[i] // page, -(-(p[i] + n[i]) // page) if n[i] else 0):
                a, b = max(p[i], j * page), min(p[i] + n[i], (j + 1) * page)
                rows = slice(int(ends[i]) + a - p[i], int(ends[i]) + b - p[i])
                k[table[i][j], :, a - j * page:b - j * page] = new[rows].transpose(0, 1)
                v[table[i][j], :, a - j * page:b - j * page] = s["v"][rows].transpose(0, 1).to(torch.float64)
        return turned(s["q"]), k, v
    G = case["H"] // case["Hkv"]
    out = torch.zeros(case["rows"], case["H"], D, dtype=torch.float64, device="cuda")
    for i in range(case["M"]):
        if not n[i]:
            continue
        L = p[i] + n[i]
        use = table[i][:-(-L // page)]
        for h in range(case["Hkv"]):
            k = s["k_pages"][use, h].reshape(-1, D)[:L].to(torch.float64)
            v = s["v_pages"][use, h].reshape(-1, D)[:L].to(torch.float64)
            for a in range(0, n[i], 512):
                b = min(n[i], a + 512)
                q = s["q"][int(ends[i]) + a:int(ends[i]) + b, h * G:(h + 1) * G].to(torch.float64)
                z = torch.einsum("tgd,ld->tgl", q, k) / D ** 0.5
                far = torch.arange(L, device="cuda")[None] > torch.arange(p[i] + a, p[i] + b, device="cuda")[:, None]
                w = torch.softmax(z.masked_fill(far[:, None], -torch.inf), -1)
                out[int(ends[i]) + a:int(ends[i]) + b, h * G:(h + 1) * G] = torch.einsum("tgl,ld->tgd", w, v)
    return out


def exact_logits(s, case):
    at = {k: s[k].cpu().numpy() for k in ("history", "history_offsets", "prompt_lens", "bias_ids", "bias_values", "bias_offsets")}
    rep, pres, freq = (s[k].cpu().numpy().astype(np.float64) for k in ("repetition", "presence", "frequency"))
    x = s["logits"].cpu().to(torch.float64).numpy()
    for m in range(case["M"]):
        h = at["history"][at["history_offsets"][m]:at["history_offsets"][m + 1]]
        seen = np.unique(h)
        x[m, seen] = np.where(x[m, seen] > 0, x[m, seen] / rep[m], x[m, seen] * rep[m])
        made, times = np.unique(h[at["prompt_lens"][m]:], return_counts=True)
        x[m, made] -= freq[m] * times + pres[m]
        b = slice(at["bias_offsets"][m], at["bias_offsets"][m + 1])
        np.add.at(x[m], at["bias_ids"][b], at["bias_values"][b].astype(np.float64))
        if s["mask"] is not None and m % 2 == 0:
            bits = np.unpackbits(s["mask"][m // 2].cpu().numpy().view(np.uint8), bitorder="little")[:case["V"]]
            x[m, bits == 0] = -np.inf
    return x, None
