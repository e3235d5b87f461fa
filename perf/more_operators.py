"""Attention for batches that share a prefix, and index keys held in 8 bits: calls as a user's program makes them, with
their plain forms.

Three operators:

prefix   attention of decode rows (1 to 8 a sequence) over every cached position, where groups of neighbouring sequences
         begin with the same cached positions, read once for the whole group
sparse   the block-sparse path (index scores, 16 blocks a row and key head, attention over them): over index keys of 8
         bits with a power of two for each position and head, and for groups that share a prefix
append   rotary positions and the store of new rows in the caches, index keys as 8-bit codes with their power of two

A case gives the batch as "rows/length" pairs, one for each sequence; the length counts the rows' own tokens.  `shared`
gives the groups as "sequences@positions" pairs, from the first sequence on; sequences after the last group are alone.
"""
import math
import random

import torch

own = False

D, DI, BLOCK, KEPT = 128, 64, 64, 16  # head and index dimensions, positions of a block, blocks that a row keeps
THETA = 1.0e6


def _case(name, op, seqs, H, G, shared=(), page=64, int8=False, index8=False, out="bf16", **more):
    return {"name": name, "op": op, "seqs": ",".join("%d/%d" % s for s in seqs), "H": H, "G": G, "page": page,
            "shared": ",".join("%d@%d" % s for s in shared), "int8": int8, "index8": index8, "out": out, **more}


def _after(seed, prefix, count, low, high, rows=1):
    """`count` sequences behind a prefix, their own lengths spread evenly over the logarithm."""
    r = random.Random(seed)
    return [(rows, prefix + rows + int(low * (high / low) ** r.random())) for _ in range(count)]


def listed():
    return [
        # the smallest: a few requests behind a system prompt
        _case("prefix_8_at_1984", "prefix", _after(1, 1984, 8, 1, 300), 4, 16, [(8, 1984)]),
        # a served batch behind one long document
        _case("prefix_64_at_32768", "prefix", _after(2, 32768, 64, 100, 2000), 4, 16, [(64, 32768)], page=256),
        # several system prompts, drafted windows, sequences that share nothing
        _case("prefix_groups_drafted", "prefix", _after(3, 9024, 5, 20, 900, 4) + _after(4, 1152, 17, 20, 900, 2) +
              _after(5, 40000, 2, 20, 900, 8) + [(1, 3), (3, 5001), (1, 700)], 8, 5, [(5, 9024), (17, 1152), (2, 40000)]),
        # many samples of one prompt: bound by its arithmetic
        _case("prefix_256_at_8192", "prefix", _after(6, 8192, 256, 64, 512), 4, 16, [(256, 8192)]),
        # an int8 cache
        _case("prefix_32_at_16384_int8", "prefix", _after(7, 16384, 32, 50, 1000), 4, 16, [(32, 16384)], page=128, int8=True),
        # outputs in 32 bits
        _case("prefix_16_at_8192_fp32", "prefix", _after(8, 8192, 16, 50, 1000), 4, 16, [(16, 8192)], out="fp32"),
        # one decoding step's cache write
        _case("append_8_index8", "append", _after(9, 0, 8, 500, 8000), 4, 16, index8=True, rope=64, axes=1),
        # a prompt chunk with image patches (time, height, width), keys and values in 8 bits too
        _case("append_4096_index8_axes", "append", [(4096, 4096)], 4, 16, page=256, int8=True, index8=True, rope=64, axes=3),
        # four long contexts
        _case("sparse_4x65536_index8", "sparse", [(1, 65536)] * 4, 4, 16, page=0, index8=True),
        # a prompt's chunk behind its prefix
        _case("sparse_1024_at_16384_index8", "sparse", [(1024, 17408)], 4, 16, index8=True),
        # a served batch behind one long document
        _case("sparse_32_at_65536", "sparse", _after(10, 65536, 32, 100, 2000), 4, 16, [(32, 65536)], page=256),
        # the same with drafted windows, two documents and index keys of 8 bits
        _case("sparse_groups_index8", "sparse", _after(11, 24576, 12, 100, 2000, 4) + _after(12, 50048, 9, 100, 2000, 3) +
              [(1, 9), (2, 12345)], 4, 16, [(12, 24576), (9, 50048)], index8=True),
    ]


def _log(rng, low, high):
    return int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "sparse", "append"])
    H, G, page = rng.choice([1, 2, 4, 8]), rng.randint(1, 16), rng.choice([64, 128, 512])
    c = {"op": op, "H": H, "G": G, "page": page, "shared": "", "int8": rng.random() < 0.3, "out": "bf16",
         "index8": op == "append"}
    if op == "append":
        B = _log(rng, 1, 12)
        seqs = [(n, n + rng.randint(0, 300)) for n in (_log(rng, 1, 4096 // B) for _ in range(B))]
        c.update(rope=rng.choice([0, 32, 64, 128]), axes=rng.choice([1, 1, 3]), interleaved=rng.random() < 0.3)
    elif op == "sparse" and rng.random() < 0.3:  # prompt chunks
        B = _log(rng, 1, 4)
        seqs = [(n, n + rng.randint(0, 12000)) for n in (_log(rng, 9, 1024 // B) for _ in range(B))]
        c["index8"] = True
    else:
        groups, seqs, most = [], [], rng.choice([1, 1, 4, 8])
        counts = [_log(rng, 2, 256 if op == "prefix" else 48) for _ in range(rng.choice([1, 1, 2, 3]))]
        for count in counts:
            prefix = max(1, _log(rng, 64, min(65536, 8000000 // (H * sum(counts)))) // page) * page
            groups.append((count, prefix))
            for _ in range(count):
                n = rng.randint(1, most)
                seqs.append((n, prefix + n + _log(rng, 1, 1000) - 1))
        seqs += [(1, _log(rng, 1, 8000)) for _ in range(rng.choice([0, 0, 1, 3]))]
        c["shared"] = ",".join("%d@%d" % s for s in groups)
        c["index8"] = op == "sparse" and rng.random() < 0.6
        if op == "prefix":
            c["out"] = rng.choice(["bf16", "bf16", "fp32"])
    c["seqs"] = ",".join("%d/%d" % s for s in seqs)
    return c


def _seqs(case):
    return [tuple(int(x) for x in s.split("/")) for s in case["seqs"].split(",")]


def _groups(case):
    return [tuple(int(x) for x in s.split("@")) for s in case["shared"].split(",")] if case["shared"] else []


def _values(gen, *shape):
    """Values with a mean of their own in every channel, as keys and values have."""
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return x.add_(0.5 * torch.randn(*shape[1:], generator=gen, device="cuda", dtype=torch.bfloat16))


def _grid(gen, *shape):
    """Normal values on a grid of 1/16, at most 4: sums of their products are exact in 32 bits in any order, so that
    every way to compute the index scores chooses the same blocks."""
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return x.mul_(16).round_().clamp_(-64, 64).div_(16)


def _tables(host, seqs, groups, page):
    """Page numbers of a pool in any order, the pages of a group's prefix the same for its sequences; pages in all."""
    prefix, lead = [0] * len(seqs), list(range(len(seqs)))
    first = 0
    for count, positions in groups:
        for b in range(first, first + count):
            prefix[b], lead[b] = positions // page, first
        first += count
    need = [-(-L // page) for _, L in seqs]
    ids = list(range(sum(k if lead[b] == b else k - prefix[b] for b, k in enumerate(need)) + 3))
    host.shuffle(ids)
    table, at = [[0] * max(need) for _ in seqs], 0
    for b, k in enumerate(need):
        keep = 0 if lead[b] == b else prefix[b]
        table[b][:keep] = table[lead[b]][:keep]
        table[b][keep:k] = ids[at:at + k - keep]
        at += k - keep
    return table, len(ids)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    seqs, groups, H, G, page = _seqs(case), _groups(case), case["H"], case["G"], case["page"]
    B, R = len(seqs), sum(n for n, _ in seqs)
    s = {"case": case, "H": H, "G": G, "page": page, "R": R, "rows_most": max(n for n, _ in seqs),
         "len_most": max(L for _, L in seqs)}
    ints = lambda v, t: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    s["n"], s["L"] = ints([n for n, _ in seqs], torch.int64), ints([L for _, L in seqs], torch.int64)
    s["first"] = torch.cumsum(s["n"], 0) - s["n"]
    s["seq"] = torch.repeat_interleave(torch.arange(B, device="cuda"), s["n"])
    s["pos"] = torch.arange(R, device="cuda") - s["first"][s["seq"]] + (s["L"] - s["n"])[s["seq"]]
    if page:
        table, pages = _tables(host, seqs, groups, page)
        s["table"], T = ints(table, torch.int32), pages * page
    else:
        starts = [sum(L for _, L in seqs[:b]) for b in range(B)]
        s["starts"], T = ints(starts, torch.int64), sum(L for _, L in seqs)
    s["T"] = T
    if case["op"] == "append":
        # the projections of the new rows, side by side in one buffer as a fused product leaves them
        widths = [H * G * D, H * D, H * D, H * DI, H * DI]
        x = torch.randn(R, sum(widths), generator=gen, device="cuda", dtype=torch.bfloat16)
        q, k, v, iq, ik = torch.split(x, widths, dim=1)
        s.update(q=q.view(R, H * G, D), new_k=k.view(R, H, D), new_v=v.view(R, H, D), iq=iq.view(R, H, DI),
                 new_ik=ik.view(R, H, DI))
        held = torch.int8 if case["int8"] else torch.bfloat16
        s["k"], s["v"] = (torch.zeros(T, H, D, dtype=held, device="cuda") for _ in range(2))
        if case["int8"]:
            s["k_scale"], s["v_scale"] = (torch.zeros(T, H, dtype=torch.float32, device="cuda") for _ in range(2))
        s["ik"] = torch.zeros(T, H, DI, dtype=torch.int8, device="cuda")
        s["ik_exp"] = torch.zeros(T, H, dtype=torch.int8, device="cuda")
        half, axes = case["rope"] // 2, case["axes"]
        if half and axes > 1:  # text, then patches of an image: time stands, height and width run
            t = torch.arange(R, device="cuda")
            s["positions"] = torch.stack([t // 1024, t // 32 % 32, t % 32][:axes]).int() + host.randint(0, 100000)
            s["axis"] = ints([0] * (half - 2 * (half * 3 // 8)) + [1] * (half * 3 // 8) + [2] * (half * 3 // 8), torch.int32)
    else:
        s["q"] = 2 * torch.randn(R, H * G, D, generator=gen, device="cuda", dtype=torch.bfloat16)
        if case["int8"]:
            for x in ("k", "v"):
                s[x] = torch.randint(-127, 128, (T, H, D), generator=gen, device="cuda", dtype=torch.int8)
                s[x + "_scale"] = (0.5 + torch.rand(T, H, generator=gen, device="cuda")) / 64
        else:
            s["k"], s["v"] = _values(gen, T, H, D), _values(gen, T, H, D)
        if case["op"] == "sparse":
            s["iq"] = _grid(gen, R, H, DI)
            if case["index8"]:  # codes about as a normal vector's, the largest of 64 near 127
                x = torch.randn(T, H, DI, generator=gen, device="cuda", dtype=torch.bfloat16)
                s["ik"] = x.mul_(36).round_().clamp_(-127, 127).to(torch.int8)
                s["ik_exp"] = torch.randint(-7, -4, (T, H), generator=gen, device="cuda", dtype=torch.int8)
            else:
                s["ik"] = _grid(gen, T, H, DI)
    if own:
        import block_sparse_attention_index_gb300 as msa
        kw = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]} if case["int8"] else {}
        if case["index8"]:
            kw["ik_exp"] = s["ik_exp"]
        if groups:
            kw["shared"] = groups
        if page:
            kw.update(block_table=s["table"], page_size=page)
        else:
            kw.update(cache_starts=starts)
        s["problem"] = msa.Problem(H, G, seqs, "cuda", out_dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16,
                                   cache_tokens=T, **kw)
        if case["op"] == "append":
            s["workspace"] = torch.empty(256, dtype=torch.uint8, device="cuda")
            s["rope"] = None if not case["rope"] else msa.Rope(
                case["rope"], index_dim=min(case["rope"], DI), theta=THETA, device="cuda", axes=axes,
                axis=s.get("axis"), index_axis=s["axis"][:min(case["rope"], DI) // 2] if "axis" in s else None,
                interleaved=case.get("interleaved", False))
        else:
            s["workspace"] = s["problem"].dense_workspace() if case["op"] == "prefix" else s["problem"].workspace()
    return s


def _cache_rows(s, seq, t):
    """The cache rows of positions t [N, M] of sequences seq [N]; of positions past the end, some row."""
    t = torch.minimum(t, s["L"][seq][:, None] - 1)
    if s["page"]:
        return torch.gather(s["table"].long()[seq], 1, t // s["page"]) * s["page"] + t % s["page"]
    return s["starts"][seq][:, None] + t


def _held(s, x, rows):
    """The cached values at `rows`, in 32 bits."""
    got = s[x][rows].float()
    return got * s[x + "_scale"][rows][..., None] if x + "_scale" in s else got


def _power(e):
    """2^e in 32 bits, of 8-bit exponents."""
    return torch.ldexp(torch.ones((), device=e.device), e.int())


def _prefix(s):
    B, H, G = len(s["L"]), s["H"], s["G"]
    t = torch.arange(s["len_most"], device="cuda").expand(B, -1)
    i = torch.arange(s["rows_most"], device="cuda").expand(B, -1)
    rows = _cache_rows(s, torch.arange(B, device="cuda"), t)
    live = (t < s["L"][:, None])[:, :, None, None]
    k = torch.where(live, _held(s, "k", rows), 0).permute(0, 2, 3, 1)  # [B, H, D, L]
    v = torch.where(live, _held(s, "v", rows), 0).transpose(1, 2)      # [B, H, L, D]
    q = s["q"][torch.minimum(s["first"][:, None] + i, s["first"][:, None] + s["n"][:, None] - 1)].float()
    q = q.view(B, -1, H, G, D).transpose(1, 2).reshape(B, H, -1, D)    # [B, H, rows G, D]
    w = torch.matmul(q, k).mul_(1 / math.sqrt(D))
    hidden = t[:, None] > (s["L"] - s["n"])[:, None, None] + i[:, :, None]  # [B, rows, L]
    w.view(B, H, -1, G, t.shape[1]).masked_fill_(hidden[:, None, :, None], -math.inf)
    w.sub_(w.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(w, v).div_(w.sum(-1, keepdim=True))
    o = o.view(B, H, -1, G, D).transpose(1, 2).reshape(B, -1, H * G, D)
    return o[s["seq"], torch.arange(s["R"], device="cuda") - s["first"][s["seq"]]]


def _sparse(s):
    B, R, H, G = len(s["L"]), s["R"], s["H"], s["G"]
    blocks = -(-s["len_most"] // BLOCK)
    t = torch.arange(blocks * BLOCK, device="cuda")
    rows = _cache_rows(s, torch.arange(B, device="cuda"), t.expand(B, -1))
    ik = s["ik"][rows].float()
    if s["case"]["index8"]:
        ik *= _power(s["ik_exp"][rows])[..., None]
    i = torch.arange(s["rows_most"], device="cuda")
    iq = s["iq"][torch.minimum(s["first"][:, None] + i, s["first"][:, None] + s["n"][:, None] - 1)].float()
    score = torch.matmul(iq.permute(0, 2, 1, 3), ik.permute(0, 2, 3, 1))  # [B, H, rows, L]
    score = score.transpose(1, 2)[s["seq"], torch.arange(R, device="cuda") - s["first"][s["seq"]]]  # [R, H, L]
    score = score.masked_fill(t > s["pos"][:, None, None], -math.inf)
    best = score.view(R, H, blocks, BLOCK).amax(-1)
    last = s["pos"] // BLOCK
    best[torch.arange(R, device="cuda"), :, last] = math.inf  # the block of the row's own position
    order = torch.sort(best, dim=-1, descending=True, stable=True).indices[..., :KEPT]
    order = torch.nn.functional.pad(order, (0, KEPT - order.shape[-1]), value=blocks)
    count = torch.clamp(last + 1, max=KEPT)
    order = torch.where(torch.arange(KEPT, device="cuda") < count[:, None, None], order, blocks)
    order = torch.sort(order, dim=-1).values
    sel = torch.where(order < blocks, order, -1).int()
    at = (order[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).view(R, H, -1)  # positions of the kept blocks
    seen = at <= s["pos"][:, None, None]
    at = torch.where(seen, at, 0).view(R, -1)
    row = _cache_rows(s, s["seq"], at).view(R, H, -1)
    head = torch.arange(H, device="cuda")[None, :, None]
    k, v = s["k"][row, head].float(), s["v"][row, head].float()
    if s["case"]["int8"]:
        k, v = k * s["k_scale"][row, head][..., None], v * s["v_scale"][row, head][..., None]
    w = torch.matmul(s["q"].float().view(R, H, G, D), k.transpose(2, 3)).mul_(1 / math.sqrt(D))
    w.masked_fill_(~seen[:, :, None], -math.inf)
    w.sub_(w.amax(-1, keepdim=True)).exp_()
    out = torch.matmul(w, v).div_(w.sum(-1, keepdim=True))
    return out.view(R, H * G, D), sel, count[:, None].expand(R, H).int()


def _rotated(s, x, dim, axis):
    """x [R, heads, .] with its first `dim` dimensions rotated, in 64 bits (far positions need them)."""
    x = x.double()
    if not dim:
        return x
    j = torch.arange(dim // 2, device="cuda")
    turn = THETA ** (-2.0 * j.double() / dim)
    where = s["positions"].double()[axis.long()].T if "positions" in s else s["pos"].double()[:, None]
    angle = (where * turn)[:, None]
    a, b = (2 * j, 2 * j + 1) if s["case"].get("interleaved") else (j, j + dim // 2)
    y = x.clone()
    y[..., a] = x[..., a] * angle.cos() - x[..., b] * angle.sin()
    y[..., b] = x[..., b] * angle.cos() + x[..., a] * angle.sin()
    return y


def _append(s):
    dim = s["case"]["rope"]
    axis = s.get("axis")
    index = min(dim, DI)
    index_axis = axis[:index // 2] if axis is not None else None
    rows = _cache_rows(s, s["seq"], s["pos"][:, None])[:, 0]
    q = _rotated(s, s["q"], dim, axis).bfloat16()
    iq = _rotated(s, s["iq"], index, index_axis).bfloat16()
    y = _rotated(s, s["new_ik"], index, index_axis)
    big = y.abs().amax(-1)
    e = torch.ceil(torch.log2(torch.where(big > 0, big / 127, 1)))
    e = torch.where(big > 0, e, -126).clamp(min=-126)
    s["ik_exp"][rows] = e.to(torch.int8)
    s["ik"][rows] = torch.ldexp(y, -e[..., None]).round().to(torch.int8)
    k, v = _rotated(s, s["new_k"], dim, axis), s["new_v"].double()
    if s["case"]["int8"]:
        scale = (torch.stack([k, v]).abs().amax(-1) / 127).float()
        s["k_scale"][rows], s["v_scale"][rows] = scale[0], scale[1]
        code = (torch.stack([k, v]) / torch.where(scale > 0, scale, 1)[..., None].double()).round().clamp(-127, 127)
        s["k"][rows], s["v"][rows] = code[0].to(torch.int8), code[1].to(torch.int8)
    else:
        s["k"][rows], s["v"][rows] = k.bfloat16(), v.bfloat16()
    return q, iq


def run(s):
    case = s["case"]
    if own:
        import block_sparse_attention_index_gb300 as msa
        if case["op"] == "prefix":
            return msa.dense_forward(s["problem"], s["q"], s["k"], s["v"], workspace=s["workspace"])
        if case["op"] == "sparse":
            out, sel, count = msa.forward(s["problem"], s["q"], s["iq"], s["k"], s["v"], s["ik"], workspace=s["workspace"])
            return {"out": out, "sel": sel, "count": count}
        q, iq = msa.append_cache(s["problem"], s["new_k"], s["new_v"], s["k"], s["v"], new_ik=s["new_ik"], ik=s["ik"],
                                 q=s["q"], iq=s["iq"], rope=s["rope"], positions=s.get("positions"),
                                 workspace=s["workspace"])
    elif case["op"] == "prefix":
        return _prefix(s).to(torch.float32 if case["out"] == "fp32" else torch.bfloat16)
    elif case["op"] == "sparse":
        out, sel, count = _sparse(s)
        return {"out": out.bfloat16(), "sel": sel, "count": count}
    else:
        q, iq = _append(s)
    # the values that the codes stand for
    got = {"q": q, "iq": iq, "ik": torch.mul(s["ik"], _power(s["ik_exp"])[..., None], out=torch.empty(
        s["ik"].shape, dtype=torch.bfloat16, device="cuda"))}
    got["k"], got["v"] = (torch.mul(s[x], s[x + "_scale"][..., None], out=torch.empty(
        s[x].shape, dtype=torch.bfloat16, device="cuda")) if case["int8"] else s[x] for x in ("k", "v"))
    return got


def work(case):
    seqs, groups, H, G = _seqs(case), _groups(case), case["H"], case["G"]
    R = sum(n for n, _ in seqs)
    held = H * (2 * D + 8) if case["int8"] else H * 4 * D     # bytes of a position's key and value
    index = H * (DI + 1) if case["index8"] else H * 2 * DI    # and of its index keys
    if case["op"] == "append":
        new = 2 * (H * G * D + 2 * H * D + 2 * H * DI)
        return {"bytes": R * (new + 2 * (H * G * D + H * DI) + held + index), "flops": 6 * R * H * (G + 1) * case["rope"]}
    first, cached = 0, sum(L for _, L in seqs)
    for count, positions in groups:
        cached -= (count - 1) * positions  # read once
    out = 4 if case["out"] == "fp32" else 2
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for n, L in seqs)
    rows = R * H * G * D * (2 + out)
    if case["op"] == "prefix":
        return {"bytes": cached * held + rows, "flops": 4 * D * H * G * pairs}
    kept = sum(min(KEPT * BLOCK, p + 1) for n, L in seqs for p in range(L - n, L))
    # kept blocks: read at least once each, at most the whole cache
    return {"bytes": cached * index + min(cached, kept) * held + rows + 2 * R * H * DI,
            "flops": 2 * DI * H * pairs + 4 * D * H * G * kept}


def exact(case, seed):
    """The same from the definitions, one sequence after another, in 64 bits."""
    s = prepare(case, seed)
    H, G, page = s["H"], s["G"], s["page"]
    table = s["table"].tolist() if page else None
    starts = s["starts"].tolist() if not page else None

    def rows_of(b, t):
        if page:
            return torch.tensor(table[b], device="cuda")[t.div(page, rounding_mode="floor")] * page + t.remainder(page)
        return starts[b] + t

    if case["op"] == "append":
        return _exact_append(case, s, rows_of)
    out, first = torch.empty(s["R"], H * G, D, dtype=torch.float64, device="cuda"), 0
    for b, (n, L) in enumerate(_seqs(case)):
        rows = rows_of(b, torch.arange(L, device="cuda"))
        t = torch.arange(L, device="cuda")
        for h in range(H):
            k, v = s["k"][rows, h].double(), s["v"][rows, h].double()
            if case["int8"]:
                k, v = k * s["k_scale"][rows, h].double()[:, None], v * s["v_scale"][rows, h].double()[:, None]
            chosen = _exact_blocks(s, rows, first, n, L, h) if case["op"] == "sparse" else None
            for i in range(n):
                p = L - n + i
                q = s["q"][first + i, h * G:(h + 1) * G].double()
                seen = t[:p + 1] if chosen is None else chosen[i]
                x = (q @ k[seen].T) / D ** 0.5
                out[first + i, h * G:(h + 1) * G] = torch.softmax(x, 1) @ v[seen]
        first += n
    return out if case["op"] == "prefix" else {"out": out, "sel": None, "count": None}


def _exact_blocks(s, rows, first, n, L, h):
    """The positions that each of the sequence's rows keeps: those of its own block and of the 15 others whose largest
    index score is best, the earlier block where two are the same."""
    ik = s["ik"][rows, h].double()
    if s["case"]["index8"]:
        ik = ik * 2.0 ** s["ik_exp"][rows, h].double()[:, None]
    score = (s["iq"][first:first + n, h].double() @ ik.T).cpu()
    kept = []
    for i in range(n):
        p = L - n + i
        top = [float(x.max()) for x in score[i, :p // BLOCK * BLOCK].split(BLOCK)] if p >= BLOCK else []
        best = sorted(range(len(top)), key=lambda j: (-top[j], j))[:KEPT - 1]
        at = [torch.arange(j * BLOCK, min(p + 1, (j + 1) * BLOCK)) for j in sorted(best + [p // BLOCK])]
        kept.append(torch.cat(at).cuda())
    return kept


def _exact_append(case, s, rows_of):
    def turned(x, where, axis):
        x, dim = x.double(), min(case["rope"], x.shape[-1])
        for j in range(dim // 2):
            a, b = (2 * j, 2 * j + 1) if case.get("interleaved") else (j, j + dim // 2)
            angle = where[axis[j]].double() / THETA ** (2 * j / dim)
            z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, None]
            x[..., a], x[..., b] = z.real, z.imag
        return x

    rows, where = [], []
    for b, (n, L) in enumerate(_seqs(case)):
        rows.append(rows_of(b, torch.arange(L - n, L, device="cuda")))
        where.append(torch.arange(L - n, L, device="cuda"))
    rows, where = torch.cat(rows), torch.cat(where)[None]
    axis = [0] * 64
    if "positions" in s:
        where, axis = s["positions"], s["axis"].tolist()
    got = {"q": turned(s["q"], where, axis), "iq": turned(s["iq"], where, axis)}
    y = turned(s["new_ik"], where, axis)
    step = 2.0 ** torch.ceil(torch.log2(y.abs().max(-1, keepdim=True).values.clamp_min(1e-300) / 127))
    got["ik"] = torch.zeros(s["T"], s["H"], DI, dtype=torch.float64, device="cuda")
    got["ik"][rows] = torch.round(y / step) * step
    for x, y in (("k", turned(s["new_k"], where, axis)), ("v", s["new_v"].double())):
        got[x] = torch.zeros(s["T"], s["H"], D, dtype=torch.float64, device="cuda")
        if case["int8"]:
            scale = y.abs().max(-1).values / 127
            y = torch.round(y / scale.clamp_min(1e-300)[..., None]) * scale[..., None]
        got[x][rows] = y
    return got
