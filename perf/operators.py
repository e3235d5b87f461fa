"""The cache writer and the dense attention, as a user's program calls them, with their plain forms.

Three operators over the same caches:

append   rotary positions on the new rows' queries, keys and index keys, and the store of keys, values and index keys
         into the paged or contiguous caches (bf16, or int8 with a scale per position and head)
decode   attention of 1 to 8 new rows a sequence over all of the sequence's cached positions
prompt   causal attention of whole prompt chunks, packed sequences of different lengths, with their cached prefixes

A case gives the batch as "rows/length" pairs, one for each sequence; the length counts the rows' own tokens.
"""
import math
import random

import torch

own = False

D, DI = 128, 64  # head and index dimensions of the caches
THETA = 1.0e6


def _case(name, op, seqs, H, G, int8=False, page=0, out="bf16", **more):
    return {"name": name, "op": op, "seqs": ",".join("%d/%d" % s for s in seqs), "H": H, "G": G, "int8": int8,
            "page": page, "out": out, **more}


def _spread(seed, count, low, high):
    """`count` lengths, spread evenly over their logarithm."""
    r = random.Random(seed)
    return [int(low * (high / low) ** r.random()) for _ in range(count)]


def listed():
    return [
        # one decoding step's cache write: 8 sequences, one token each, paged
        _case("append_8_rows", "append", [(1, L) for L in _spread(1, 8, 500, 8000)], 4, 16, page=64, rope=64, axes=1),
        # a prompt chunk with image patches (time, height, width), int8 cache
        _case("append_4096_int8_axes", "append", [(4096, 4096)], 4, 16, int8=True, page=256, rope=64, axes=3),
        # packed short prompts behind their prefixes, contiguous bf16 cache, neighbouring pairs rotated
        _case("append_packed", "append", [(n, n + 7) for n in _spread(2, 7, 20, 900)], 8, 5, rope=128, axes=1,
              interleaved=True),
        # the smallest step: one token, one key head, a short context
        _case("decode_1x4096", "decode", [(1, 4096)], 1, 16, out="fp32"),
        # four long contexts
        _case("decode_4x65536", "decode", [(1, 65536)] * 4, 4, 16),
        # long contexts of very different lengths, int8 and paged
        _case("decode_8_ragged_int8", "decode", [(1, L) for L in _spread(3, 8, 1024, 196608)], 4, 16, int8=True, page=64),
        # drafted windows: four rows a sequence
        _case("decode_4x4_65536", "decode", [(4, 65536)] * 4, 4, 16, page=256),
        # a served batch: many short contexts, few query heads a key head
        _case("decode_64_short", "decode", [(1, L) for L in _spread(4, 64, 3, 4096)], 8, 4, page=64),
        # a long prompt's chunk behind its prefix
        _case("prompt_4096_at_8192", "prompt", [(4096, 12288)], 4, 16),
        # the same behind an int8 cache
        _case("prompt_2048_at_8192_int8", "prompt", [(2048, 10240)], 4, 16, int8=True, page=64),
        # whole prompts of odd lengths, packed, paged
        _case("prompt_packed", "prompt", [(n, n) for n in (1, 77, 1023, 130, 2047, 9, 640, 1511)], 8, 5, page=64),
        # a short chunk behind a long prefix, outputs in 32 bits
        _case("prompt_512_at_32768_fp32", "prompt", [(512, 33280)], 4, 16, out="fp32"),
    ]


def _log(rng, low, high):
    return int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))


def draw(rng):
    op = rng.choice(["append", "decode", "prompt"])
    H, G = rng.choice([1, 2, 4, 8]), rng.randint(1, 16)
    c = {"H": H, "G": G, "int8": rng.random() < 0.4, "page": rng.choice([0, 64, 128, 512]),
         "out": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "append":
        B = _log(rng, 1, 12)
        seqs = [(n, n + rng.randint(0, 300)) for n in (_log(rng, 1, 4096 // B) for _ in range(B))]
        c.update(rope=rng.choice([0, 32, 64, 128]), axes=rng.choice([1, 1, 3]), interleaved=rng.random() < 0.3)
    elif op == "decode":
        most = rng.choice([1, 1, 8])
        B = _log(rng, 1, 64)
        top = min(196608, 4 * 4 * 65536 // (H * B))
        seqs = [(min(rng.randint(1, most), L), L) for L in (_log(rng, 1, top) for _ in range(B))]
    else:
        B = _log(rng, 1, 8)
        rows = [_log(rng, 9, 4096 // B) for _ in range(B)]
        room = max(1, min(32768, (1 << 31) // (B * max(rows) * H * G) - max(rows)))
        seqs = [(n, n + (rng.randint(0, room) if rng.random() < 0.7 else 0)) for n in rows]
    c.update(op=op, seqs=",".join("%d/%d" % s for s in seqs))
    return c


def _seqs(case):
    return [tuple(int(x) for x in s.split("/")) for s in case["seqs"].split(",")]


def _values(gen, *shape):
    """Values with a mean of their own in every channel, as keys and values have."""
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return x.add_(0.5 * torch.randn(*shape[1:], generator=gen, device="cuda", dtype=torch.bfloat16))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    seqs, H, G, page = _seqs(case), case["H"], case["G"], case["page"]
    B, R = len(seqs), sum(n for n, _ in seqs)
    s = {"case": case, "H": H, "G": G, "page": page, "R": R, "rows_most": max(n for n, _ in seqs),
         "len_most": max(L for _, L in seqs)}
    ints = lambda v, t: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    s["n"], s["L"] = ints([n for n, _ in seqs], torch.int64), ints([L for _, L in seqs], torch.int64)
    s["first"] = torch.cumsum(s["n"], 0) - s["n"]
    s["seq"] = torch.repeat_interleave(torch.arange(B, device="cuda"), s["n"])
    s["pos"] = torch.arange(R, device="cuda") - s["first"][s["seq"]] + (s["L"] - s["n"])[s["seq"]]
    if page:  # a pool of pages in any order, some of them nobody's
        need = [-(-L // page) for _, L in seqs]
        ids = list(range(sum(need) + 3))
        host.shuffle(ids)
        table, at = [[0] * max(need) for _ in seqs], 0
        for b, k in enumerate(need):
            table[b][:k] = ids[at:at + k]
            at += k
        s["table"], T = ints(table, torch.int32), len(ids) * page
    else:
        starts = [sum(L for _, L in seqs[:b]) for b in range(B)]
        s["starts"], T = ints(starts, torch.int64), sum(L for _, L in seqs)
    s["T"] = T
    if case["op"] == "append":
        # the projections of the new rows, side by side in one buffer as a fused product leaves them
        widths = [H * G * D, H * D, H * D, H * DI, H * DI]
        x = torch.randn(R, sum(widths), generator=gen, device="cuda", dtype=torch.bfloat16)
        q, k, v, iq, ik = torch.split(x, widths, dim=1)
        s.update(q=q.view(R, H * G, D), k=k.view(R, H, D), v=v.view(R, H, D), iq=iq.view(R, H, DI), ik=ik.view(R, H, DI))
        held = torch.int8 if case["int8"] else torch.bfloat16
        s["k_cache"], s["v_cache"] = (torch.zeros(T, H, D, dtype=held, device="cuda") for _ in range(2))
        s["ik_cache"] = torch.zeros(T, H, DI, dtype=torch.bfloat16, device="cuda")
        if case["int8"]:
            s["k_scale"], s["v_scale"] = (torch.zeros(T, H, dtype=torch.float32, device="cuda") for _ in range(2))
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
    if own:
        import block_sparse_attention_index_gb300 as msa
        kw = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]} if case["int8"] else {}
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
            s["workspace"] = s["problem"].dense_workspace()
    return s


def _cache_rows(s, t):
    """The cache rows of positions t [B, N]; of positions past the end, some row."""
    t = torch.minimum(t, s["L"][:, None] - 1)
    if s["page"]:
        return torch.gather(s["table"].long(), 1, t // s["page"]) * s["page"] + t % s["page"]
    return s["starts"][:, None] + t


def _held(s, x, rows):
    """The cached values at `rows`, in 32 bits."""
    got = s[x][rows].float()
    return got * s[x + "_scale"][rows][..., None] if x + "_scale" in s else got


def _rotated(s, x, dim, axis):
    """x [R, heads, .] with its first `dim` dimensions rotated, in 64 bits (far positions need them)."""
    x = x.double()
    if not dim:
        return x
    j = torch.arange(dim // 2, device="cuda")
    where = s["positions"].double()[axis.long()].T if "positions" in s else s["pos"].double()[:, None]
    angle = (where * THETA ** (-2.0 * j.double() / dim))[:, None]
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
    at = s["pos"]
    if s["page"]:
        rows = s["table"].long()[s["seq"], at // s["page"]] * s["page"] + at % s["page"]
    else:
        rows = s["starts"][s["seq"]] + at
    q = _rotated(s, s["q"], dim, axis).bfloat16()
    iq = _rotated(s, s["iq"], index, index_axis).bfloat16()
    s["ik_cache"][rows] = _rotated(s, s["ik"], index, index_axis).bfloat16()
    for x, y in (("k", _rotated(s, s["k"], dim, axis)), ("v", s["v"].double())):
        if s["case"]["int8"]:
            scale = (y.abs().amax(-1) / 127).float()
            s[x + "_scale"][rows] = scale
            code = (y / torch.where(scale > 0, scale, 1)[..., None].double()).round().clamp(-127, 127)
            s[x + "_cache"][rows] = code.to(torch.int8)
        else:
            s[x + "_cache"][rows] = y.bfloat16()
    return q, iq


def _attend(s):
    B, H, G = len(s["L"]), s["H"], s["G"]
    t = torch.arange(s["len_most"], device="cuda").expand(B, -1)
    i = torch.arange(s["rows_most"], device="cuda").expand(B, -1)
    rows = _cache_rows(s, t)
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


def run(s):
    case = s["case"]
    if case["op"] == "append":
        if own:
            import block_sparse_attention_index_gb300 as msa
            q, iq = msa.append_cache(s["problem"], s["k"], s["v"], s["k_cache"], s["v_cache"], new_ik=s["ik"],
                                     ik=s["ik_cache"], q=s["q"], iq=s["iq"], rope=s["rope"],
                                     positions=s.get("positions"), workspace=s["workspace"])
        else:
            q, iq = _append(s)
        got = {"q": q, "iq": iq, "ik": s["ik_cache"]}
        for x in ("k", "v"):
            got[x] = s[x + "_cache"]
            if case["int8"]:  # the values that the codes stand for
                got[x + "_scale"] = s[x + "_scale"]
                got[x] = torch.mul(got[x], s[x + "_scale"][..., None], out=torch.empty(
                    got[x].shape, dtype=torch.bfloat16, device="cuda"))
        return got
    if own:
        import block_sparse_attention_index_gb300 as msa
        return msa.dense_forward(s["problem"], s["q"], s["k"], s["v"], workspace=s["workspace"])
    return _attend(s).to(torch.float32 if case["out"] == "fp32" else torch.bfloat16)


def work(case):
    seqs, H, G = _seqs(case), case["H"], case["G"]
    R = sum(n for n, _ in seqs)
    held = H * (2 * D + 8) if case["int8"] else H * 4 * D  # bytes of a position's key and value
    if case["op"] == "append":
        new = 2 * (H * G * D + 2 * H * D + 2 * H * DI)
        return {"bytes": R * (new + 2 * (H * G * D + 2 * H * DI) + held), "flops": 6 * R * H * (G + 1) * case["rope"]}
    out = 4 if case["out"] == "fp32" else 2
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for n, L in seqs)
    return {"bytes": sum(L for _, L in seqs) * held + R * H * G * D * (2 + out), "flops": 4 * D * H * G * pairs}


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
        p = torch.arange(L - n, L, device="cuda")
        for h in range(H):
            k, v = s["k"][rows, h].double(), s["v"][rows, h].double()
            if case["int8"]:
                k, v = k * s["k_scale"][rows, h].double()[:, None], v * s["v_scale"][rows, h].double()[:, None]
            for g in range(G):
                for lo in range(0, n, 8192):
                    q = s["q"][first + lo:first + min(n, lo + 8192), h * G + g].double()
                    x = (q @ k.T) / D ** 0.5
                    x[torch.arange(L, device="cuda")[None] > p[lo:lo + 8192, None]] = -math.inf
                    out[first + lo:first + lo + len(q), h * G + g] = torch.softmax(x, 1) @ v
        first += n
    return out


def _exact_append(case, s, rows_of):
    def turned(x, where, axis):
        x, dim = x.double(), min(case["rope"], x.shape[-1])
        for j in range(dim // 2):
            a, b = (2 * j, 2 * j + 1) if case.get("interleaved") else (j, j + dim // 2)
            angle = where[axis[j]].double() / THETA ** (2 * j / dim)
            z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, None]
            x[..., a], x[..., b] = z.real, z.imag
        return x

    rows, first, where = [], 0, []
    for b, (n, L) in enumerate(_seqs(case)):
        rows.append(rows_of(b, torch.arange(L - n, L, device="cuda")))
        where.append(torch.arange(L - n, L, device="cuda"))
        first += n
    rows, where = torch.cat(rows), torch.cat(where)[None]
    axis = [0] * 64
    if "positions" in s:
        where, axis = s["positions"], s["axis"].tolist()
    got = {"q": turned(s["q"], where, axis), "iq": turned(s["iq"], where, axis)}
    got["ik"] = torch.zeros(s["T"], s["H"], DI, dtype=torch.float64, device="cuda")
    got["ik"][rows] = turned(s["ik"], where, axis)
    for x, y in (("k", turned(s["k"], where, axis)), ("v", s["v"].double())):
        got[x] = torch.zeros(s["T"], s["H"], D, dtype=torch.float64, device="cuda")
        if case["int8"]:
            scale = y.abs().max(-1).values / 127
            got[x + "_scale"] = torch.zeros(s["T"], s["H"], dtype=torch.float64, device="cuda")
            got[x + "_scale"][rows] = scale
            y = torch.round(y / scale.clamp_min(1e-300)[..., None]) * scale[..., None]
        got[x][rows] = y
    return got
