"""Workloads of the 4-bit paged key/value cache and the attention that reads it, with plain forms.

Four families of calls:
  append    q, k and v rows rotated by positions of one or more axes; k and v go to the cache in 4 bits
  read      rows of the cache as values
  decode    attention of up to eight query tokens a sequence over the cache, its Q8_1 image for the output projection
  prefill   the same for prompts and chunks of prompts, with the Q8_0 planes

`own` False computes each in elementary torch operations in binary32 (angles in binary64); True makes the library's
calls. `exact` is the definition in binary64.

The cache: pages of P tokens, [n_pages][Hkv][P / 16] groups of 16 tokens, 18 * D bytes each: codes of k (8 D bytes),
scales of k (D bytes, halves), codes of v, scales of v. `_unpack` and `_offsets` give the places inside a group.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one sequence through a small layer: launch latency
        dict(name="append 1 token", op="append", T=1, live=1, Hq=4, Hkv=1, D=64, P=16, axes=1, kind="halves", R=64,
             q="bf16", x="f32"),
        # the new tokens of a decode batch
        dict(name="append 200 tokens", op="append", T=200, live=187, Hq=28, Hkv=4, D=128, P=64, axes=1, kind="halves",
             R=128, q="bf16", x="f32"),
        # a prompt with image positions: time, height and width, three quarters of a head rotated
        dict(name="append 3325 tokens 3 axes", op="append", T=3325, live=3325, Hq=28, Hkv=4, D=128, P=64, axes=3,
             kind="adjacent", R=96, q="bf16", x="f32"),
        # a shared prefix read back: odd count; and a long one
        dict(name="read 45 tokens", op="read", n=45, Hkv=4, D=64, P=16, dtype="f32"),
        dict(name="read 16384 tokens", op="read", n=16384, Hkv=8, D=128, P=64, dtype="bf16"),
        # one sequence with a short past: latency
        dict(name="decode 1 x 77", op="decode", B=1, live=1, T=1, lo=77, hi=77, Hq=8, Hkv=2, D=64, P=16, window=0,
             sinks=False, q="bf16", out="f16image"),
        # a decode bucket of ragged lengths, heads in groups of seven
        dict(name="decode 8 ragged", op="decode", B=8, live=7, T=1, lo=100, hi=8000, Hq=28, Hkv=4, D=128, P=64, window=0,
             sinks=False, q="bf16", out="bf16"),
        # a large decode batch: the cache is larger than the L2 cache
        dict(name="decode 64 x 8192", op="decode", B=64, live=64, T=1, lo=8192, hi=8192, Hq=28, Hkv=4, D=128, P=64,
             window=0, sinks=False, q="bf16", out="bf16"),
        # eight drafted tokens a sequence checked at once, with sinks
        dict(name="decode 16 x 8 tokens", op="decode", B=16, live=16, T=8, lo=1500, hi=9000, Hq=32, Hkv=8, D=128, P=32,
             window=0, sinks=True, q="bf16", out="bf16"),
        # two short prompts, one of them behind a past, wide heads, a window
        dict(name="prefill 2 x 150", op="prefill", B=2, nq=150, step=37, past=200, Hq=8, Hkv=2, D=256, P=16, window=100,
             sinks=True, q="bf16", out="bf16"),
        # a whole prompt, with the planes of the output projection
        dict(name="prefill 3325", op="prefill", B=1, nq=3325, step=0, past=0, Hq=28, Hkv=4, D=128, P=64, window=0,
             sinks=False, q="bf16", out="f16planes"),
        # a chunk of a long prompt behind its past
        dict(name="prefill 1024 behind 32000", op="prefill", B=1, nq=1024, step=0, past=32000, Hq=28, Hkv=4, D=128, P=64,
             window=0, sinks=False, q="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8, 16])
    return D, Hkv, Hkv * (G if Hkv * G <= 64 else 1)


def draw(rng):
    op = rng.choice(["append", "append", "read", "decode", "decode", "decode", "prefill", "prefill"])
    D, Hkv, Hq = _heads(rng)
    P = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        T = _log(rng, 1, max(2, 3325 * 36 * 128 // ((Hq + 2 * Hkv) * D)))
        kind = rng.choice(["halves", "adjacent"])
        return dict(op=op, T=T, live=rng.randint(max(1, T // 2), T), Hq=Hq, Hkv=Hkv, D=D, P=P, axes=rng.randint(1, 4),
                    kind=kind, R=8 * rng.randint(1, D // 8), q=rng.choice(["bf16", "f32"]), x=rng.choice(["f32", "bf16"]))
    if op == "read":
        return dict(op=op, n=_log(rng, 1, 16384 * 8 * 128 // (Hkv * D)), Hkv=Hkv, D=D, P=P,
                    dtype=rng.choice(["bf16", "f32"]))
    sinks, window = rng.choice([False, True]), rng.choice([0, 0, _log(rng, 1, 4096)])
    q, out = rng.choice(["bf16", "f32"]), "bf16"
    if op == "decode":
        T = rng.choice([1, 1, 1, rng.randint(2, 8)])
        B = _log(rng, 1, 64)
        most = 64 * 8192 * 4 * 128 // (B * Hkv * D)                    # the largest case's cache
        most = min(most, 131072, 64 * 8192 * 28 * 128 // (B * T * Hq * D))   # and its products
        hi = _log(rng, 1, max(2, most))
        return dict(op=op, B=B, live=rng.randint(max(1, B // 2), B), T=T, lo=_log(rng, 1, hi) if hi > 1 else 1, hi=hi,
                    Hq=Hq, Hkv=Hkv, D=D, P=P, window=window, sinks=sinks, q=q, out=rng.choice([out, out, "f16image"]))
    B = rng.choice([1, 1, 2, 3])
    nq = _log(rng, 2, 3325 // B)
    most = min(64000, 1024 * 33000 * 28 * 128 // (B * nq * Hq * D))
    past = min(rng.choice([0, _log(rng, 1, 32000)]), max(0, most - nq))
    return dict(op=op, B=B, nq=nq, step=rng.randint(0, nq // 4), past=past, Hq=Hq, Hkv=Hkv, D=D, P=P, window=window,
                sinks=sinks, q=q, out=rng.choice([out, out, "f16planes"]))


def _lens(case):
    """Key counts of the sequences, by the case alone: spread from hi to lo; a prompt's rows behind its past."""
    B = case["B"]
    if case["op"] == "decode":
        lo, hi = case["lo"], case["hi"]
        return [int(round(hi * (lo / hi) ** (b / max(1, B - 1)))) for b in range(B)]
    return [n + case["past"] // (b + 1) for b, n in enumerate(_rows(case))]


def _rows(case):
    """Query rows of the sequences."""
    if case["op"] == "decode":
        return [case["T"]] * case["B"]
    return [max(1, case["nq"] - b * case["step"]) for b in range(case["B"])]


def _visible(case):
    """(query, key) pairs, and keys that some query of a sequence sees, over the live sequences."""
    pairs = keys = 0
    w = case["window"]
    for n, L in list(zip(_rows(case), _lens(case)))[:case.get("live", case["B"])]:
        ends = [L - n + i + 1 for i in range(n)]
        pairs += sum(min(max(e, 0), w) if w else max(e, 0) for e in ends)
        keys += max(0, L - max(0, ends[0] - w)) if w else L
    return pairs, keys


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6151 + 17)
    return g


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _pages(g, n, Hkv, P, D):
    """Pages with random codes and scales of either sign: values of about unit size."""
    pages = torch.randint(0, 256, (n, Hkv, P // 16, 18 * D), dtype=torch.uint8, device="cuda", generator=g)
    for lo in (8 * D, 17 * D):
        d = torch.empty((n, Hkv, P // 16, D // 2), device="cuda").uniform_(0.1, 0.3, generator=g)
        d *= 1 - 2 * torch.randint(0, 2, d.shape, device="cuda", generator=g)
        pages[..., lo:lo + D] = d.half().view(torch.uint8)
    return pages


def prepare(case, seed):
    g = _gen(seed)
    op, Hkv, D, P = case["op"], case["Hkv"], case["D"], case["P"]
    s = dict(case=case)
    if op in ("append", "read"):
        n = case["T"] if op == "append" else case["n"]
        n_pages = -(-n // P) + 3
        s["pages"] = _pages(g, n_pages, Hkv, P, D)
        # consecutive tokens of pages in any order
        order = torch.randperm(n_pages, device="cuda", generator=g)
        t = torch.arange(n, device="cuda") + 5
        s["slots"] = (order[t // P] * P + t % P).to(torch.int32)
    if op == "read":
        s["out"] = torch.zeros((n, 2 * Hkv * D), dtype=_type(case["dtype"]), device="cuda")
    elif op == "append":
        T, Hq, R, A = case["T"], case["Hq"], case["R"], case["axes"]
        width = (Hq + 2 * Hkv) * D
        x = torch.randn((T, width), device="cuda", generator=g)
        x[:, (Hq + Hkv) * D:] *= 2
        s["x"] = x.to(_type(case["x"]))                      # the projections' rows, q | k | v
        if A == 1:
            far = torch.randint(0, 200000, (1,), device="cuda", generator=g)
            s["pos"] = (torch.arange(T, device="cuda") + far).to(torch.int32).unsqueeze(0)
        else:
            s["pos"] = torch.randint(0, 30000, (A, T), dtype=torch.int32, device="cuda", generator=g)
        i = torch.arange(R // 2, device="cuda")
        f = 10000.0 ** (-2.0 * i.double() / R)
        axis = i * A // (R // 2)                              # consecutive pairs turn with one axis
        s["freqs"] = torch.where(axis == torch.arange(A, device="cuda").unsqueeze(1), f, 0.0).float()
        s["q_out"] = torch.zeros((T, Hq * D), dtype=_type(case["q"]), device="cuda")
        s["kv"] = torch.zeros((T, 2 * Hkv * D), dtype=torch.bfloat16, device="cuda")
        s["live"] = torch.tensor([case["live"]], dtype=torch.int32, device="cuda")
    elif op in ("decode", "prefill"):
        B, Hq, lens, rows = case["B"], case["Hq"], _lens(case), _rows(case)
        need = [-(-L // P) for L in lens]
        n_pages = sum(need) + 2
        s["pages"] = _pages(g, n_pages, Hkv, P, D)
        order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
        table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        s["table"] = table
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["most"] = max(lens)
        s["total"] = sum(rows)
        first = [sum(rows[:b]) for b in range(B + 1)]
        s["first"] = torch.tensor(first, dtype=torch.int32, device="cuda")
        s["q"] = (1.5 * torch.randn((s["total"], Hq * D), device="cuda", generator=g)).to(_type(case["q"]))
        s["sinks"] = torch.randn((Hq,), device="cuda", generator=g) if case["sinks"] else None
        s["live"] = torch.tensor([case.get("live", B)], dtype=torch.int32, device="cuda")
        width = Hq * D
        s["out"] = torch.zeros((s["total"], width), dtype=torch.bfloat16, device="cuda") if case["out"] == "bf16" else None
        if case["out"] == "f16image":
            s["img"] = torch.zeros((s["total"], width // 32, 36), dtype=torch.uint8, device="cuda")
        elif case["out"] == "f16planes":
            s["qs"] = torch.zeros((s["total"], width // 32, 32), dtype=torch.int8, device="cuda")
            s["d"] = torch.zeros((s["total"], width // 32, 1), dtype=torch.float16, device="cuda")
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a user of the library keeps: the descriptors of the cache, the rotation and the attention, a workspace."""
    from quantized_activation_q4_gb300 import binding as qk
    case = s["case"]
    op, Hkv, D, P = case["op"], case["Hkv"], case["D"], case["P"]
    s["cache"] = qk.make_kv_cache(s["pages"], s["pages"].shape[0], P, Hkv, D)
    if op == "append":
        s["rope"] = qk.make_rope(case["kind"], case["R"], case["axes"], s["pos"], s["freqs"])
    elif op in ("decode", "prefill"):
        width = case["Hq"] * D
        s["attn"] = qk.make_attn(s["q"], case["q"], width, case["Hq"], s["table"], s["table"].shape[1], s["lens"],
                                 1 / math.sqrt(D), case["window"], s["sinks"], s["out"], "bf16", width)
        if op == "decode":
            s["ws_bytes"] = qk.qk_attn_decode_workspace_bytes(s["cache"], case["Hq"], case["B"], case["T"])
        else:
            s["ws_bytes"] = qk.qk_attn_prefill_workspace_bytes(s["cache"], case["B"], s["most"])
        s["ws"] = torch.empty((max(16, s["ws_bytes"]),), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from quantized_activation_q4_gb300 import binding as qk
    case = s["case"]
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    if op == "read":
        qk.qk_kv_read(s["cache"], s["slots"], case["n"], case["dtype"], s["out"], 2 * Hkv * D)
        return s["out"]
    if op == "append":
        Hq, width, x = case["Hq"], s["x"].shape[1], s["x"]
        qk.qk_kv_append(s["cache"], case["x"], x, width, Hq, x[:, Hq * D:], width, x[:, (Hq + Hkv) * D:], width,
                        case["T"], s["slots"], s["rope"], case["q"], s["q_out"], Hq * D, s["live"])
        # the values that the new tokens' codes stand for
        qk.qk_kv_read(s["cache"], s["slots"], case["T"], "bf16", s["kv"], 2 * Hkv * D, s["live"])
        return dict(q=s["q_out"], kv=s["kv"])
    width = case["Hq"] * D
    if op == "decode":
        qk.qk_attn_decode(s["cache"], s["attn"], case["B"], case["T"], s.get("img"), width // 32, s["ws"], s["ws_bytes"],
                          s["live"])
    else:
        qk.qk_attn_prefill(s["cache"], s["attn"], case["B"], s["total"], s["first"], s["most"], s.get("qs"), s.get("d"),
                           width // 32, s["ws"], s["ws_bytes"], s["live"])
    if case["out"] == "f16image":
        return s["img"][..., 4:].view(torch.int8) * s["img"][..., 0:2].view(torch.float16)
    if case["out"] == "f16planes":
        return s["qs"] * s["d"]
    return s["out"]


def _unpack(groups, D):
    """Groups [..., 18 D] -> k and v [..., 16, D] in binary32."""
    lead, nb = groups.shape[:-1], D // 32
    n = len(lead)
    W = min(4, nb)
    at = lambda *axes: [*range(n), *(n + a for a in axes)]
    c = groups[..., :8 * D].unflatten(-1, (nb // W, 16, 4, W, 4))             # block quad, token, t, block, j
    c = torch.stack([c & 15, c >> 4], n)                                      # nibble first
    k = c.permute(at(2, 1, 4, 0, 3, 5)).reshape(*lead, 16, nb, 32).float() - 8
    k = k * groups[..., 8 * D:9 * D].contiguous().view(torch.float16).unflatten(-1, (16, nb, 1)).float()
    c = groups[..., 9 * D:17 * D].unflatten(-1, (D // 64, 8, 4, 4, 2, 2))     # quad, g, t, tile, token & 1, token >> 3
    c = torch.stack([c & 15, c >> 4], n)
    v = c.permute(at(6, 3, 5, 1, 4, 0, 2)).reshape(*lead, 16, nb, 32).float() - 8
    d = groups[..., 17 * D:].contiguous().view(torch.float16).unflatten(-1, (4, nb, 2, 2))   # t, block, token >> 3, token & 1
    v = v * d.permute(at(2, 0, 3, 1)).reshape(*lead, 16, nb, 1).float()
    return k.flatten(-2), v.flatten(-2)


def _four_bits(x):
    """The values that 4-bit codes of x [..., 32] stand for."""
    first = x.abs().argmax(-1, keepdim=True)
    d = x.gather(-1, first) / -8
    code = torch.where(d != 0, torch.clamp(torch.round(x / torch.where(d != 0, d, 1.0)), -8, 7), 0.0)
    return code * d.clamp(-65504, 65504).half().to(x.dtype)


def _run_plain(s):
    case = s["case"]
    op, Hkv, D, P = case["op"], case["Hkv"], case["D"], case["P"]
    if op == "read":
        slot = s["slots"].long()
        k, v = _unpack(s["pages"][slot // P, :, slot % P // 16], D)            # [n, Hkv, 16, D]
        at = (slot % 16).view(-1, 1, 1, 1).expand(-1, Hkv, 1, D)
        return torch.cat([k.gather(2, at).flatten(1), v.gather(2, at).flatten(1)], 1).to(s["out"].dtype)
    if op == "append":
        T, Hq, R = case["T"], case["Hq"], case["R"]
        keep = (torch.arange(T, device="cuda") < s["live"]).unsqueeze(1)
        x = s["x"].float().unflatten(1, (-1, D))
        angle = s["pos"].double().T @ s["freqs"].double()                      # [T, R/2]
        c, sn = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
        r = x[:, :Hq + Hkv]
        if case["kind"] == "halves":
            a, b = r[..., :R // 2], r[..., R // 2:R]
            r = torch.cat([a * c - b * sn, b * c + a * sn, r[..., R:]], -1)
        else:
            a, b = r[..., 0:R:2], r[..., 1:R:2]
            r = torch.cat([torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2), r[..., R:]], -1)
        kv = torch.cat([r[:, Hq:], x[:, Hq + Hkv:]], 1)
        kv = _four_bits(kv.unflatten(-1, (-1, 32))).flatten(1).bfloat16()
        return dict(q=(r[:, :Hq].flatten(1) * keep).to(s["q_out"].dtype), kv=kv * keep)
    B, Hq, L = case["B"], case["Hq"], s["most"]
    G, n = Hq // Hkv, max(_rows(case))
    k, v = _unpack(s["pages"][s["table"].clamp(min=0).long()], D)              # [B, pages, Hkv, P/16, 16, D]
    k, v = (z.transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L] for z in (k, v))
    # every sequence's rows at the end of a batch of n
    count = s["first"][1:] - s["first"][:-1]
    j = torch.arange(n, device="cuda")
    row = (s["first"][1:, None] - n + j).long()                                # [B, n]
    there = j >= n - count[:, None]
    q = s["q"][row.clamp(min=0)].float() / math.sqrt(D)
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    score = (q @ k.transpose(2, 3)).view(B, Hkv, G, n, L)
    end = (s["lens"][:, None] - n + 1 + j).view(B, 1, 1, n, 1)                 # keys below it are seen
    key = torch.arange(L, device="cuda")
    seen = key < end
    if case["window"]:
        seen = seen & (key >= end - case["window"])
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, Hkv, G, 1, 1)
        top = torch.maximum(top, sink)
    top = top.clamp(min=-1e30)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(sink - top)
    o = (p.view(B, Hkv, G * n, L) @ v).view(B, Hkv, G, n, D) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq * D)
    live = torch.arange(B, device="cuda") < s["live"]
    out = torch.zeros((s["total"], Hq * D), device="cuda")
    out[row[there]] = (o * live.view(B, 1, 1))[there]
    if case["out"] == "bf16":
        return out.bfloat16()
    ob = out.unflatten(1, (-1, 32))
    d = ob.abs().amax(-1, keepdim=True) / 127
    code = torch.where(d > 0, torch.round(ob / torch.where(d > 0, d, 1.0)), 0.0)
    return (code * d.half().float()).half()


# ------------------------------------------------------------------ the definitions in 64 bits
def _offsets(D):
    """Byte and shift of the codes of k and v, byte of their scales, for token i and column x of a group: [16, D]."""
    i, x = torch.arange(16).view(16, 1), torch.arange(D).view(1, D)
    nb = D // 32
    W = min(4, nb)
    block, r = x // 32, x % 32
    kb = ((block // W * 16 + i) * 4 + r % 16 // 4) * 4 * W + block % W * 4 + r % 4
    m, u, t = x // 16, x % 16, i % 8 // 2
    vb = 9 * D + ((m // 4 * 8 + u % 8) * 4 + t) * 16 + m % 4 * 4 + 2 * (i % 2) + i // 8
    ks, vs = 8 * D + 2 * (i * nb + block), 17 * D + 2 * ((t * nb + block) * 4 + i % 2 + 2 * (i // 8))
    whole = lambda z: (z + torch.zeros((16, D), dtype=torch.int64)).cuda()
    return [(whole(kb), whole(r // 16 * 4), whole(ks)), (whole(vb), whole(u // 8 * 4), whole(vs))]


def _exact_values(groups, D):
    """Groups [..., 18 D] -> [k, v], each [..., 16, D] in binary64."""
    out = []
    for byte, shift, scale in _offsets(D):
        code = (groups[..., byte].int() >> shift) & 15
        d = groups[..., scale].int() + 256 * groups[..., scale + 1].int()
        d = torch.where(d >= 32768, d - 65536, d).to(torch.int16).view(torch.float16).double()
        out.append((code - 8).double() * d)
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, Hkv, D, P = case["op"], case["Hkv"], case["D"], case["P"]
    if op == "read":
        slot = s["slots"].long()
        parts = []
        for z in _exact_values(s["pages"][slot // P, :, (slot % P) // 16], D):
            parts.append(z[torch.arange(len(slot), device="cuda"), :, slot % 16].reshape(len(slot), -1))
        return torch.cat(parts, 1)
    if op == "append":
        T, Hq, R, live = case["T"], case["Hq"], case["R"], case["live"]
        x = s["x"].double().reshape(T, -1, D)
        turn = torch.zeros((T, R // 2), dtype=torch.float64, device="cuda")
        for a in range(case["axes"]):
            turn += s["pos"][a, :, None].double() * s["freqs"][a].double()
        z = torch.polar(torch.ones_like(turn), turn)[:, None]
        first = torch.arange(R // 2, device="cuda")
        first, second = (first, first + R // 2) if case["kind"] == "halves" else (2 * first, 2 * first + 1)
        w = torch.complex(x[:, :Hq + Hkv, first], x[:, :Hq + Hkv, second]) * z
        x[:, :Hq + Hkv, first], x[:, :Hq + Hkv, second] = w.real, w.imag
        q, kv = x[:, :Hq].reshape(T, -1), x[:, Hq:].reshape(T, -1, 32)
        top, low = kv.max(-1, keepdim=True).values, kv.min(-1, keepdim=True).values
        d = torch.where(top >= -low, top, low) / -8
        safe = torch.where(d == 0, torch.ones_like(d), d)
        kv = (kv / safe).round().clamp(-8, 7) * d.half().double() * (d != 0)
        q, kv = q.clone(), kv.reshape(T, -1)
        q[live:] = 0
        kv[live:] = 0
        return dict(q=q, kv=kv)
    G = case["Hq"] // Hkv
    out = torch.zeros((s["total"], case["Hq"] * D), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, L) in enumerate(zip(_rows(case), _lens(case))):
        if b < case.get("live", case["B"]):
            pages = s["table"][b, :-(-L // P)].long()
            end = torch.arange(n, device="cuda")[:, None] + (L - n + 1)
            key = torch.arange(L, device="cuda")[None]
            hide = key >= end
            if case["window"]:
                hide |= key < end - case["window"]
            for h in range(Hkv):
                k, v = (z.reshape(-1, D)[:L] for z in _exact_values(s["pages"][pages, h], D))
                for head in range(h * G, h * G + G):
                    q = s["q"][at:at + n, head * D:(head + 1) * D].double()
                    logit = (q @ k.T / math.sqrt(D)).masked_fill(hide, -math.inf)
                    if s["sinks"] is not None:
                        logit = torch.cat([logit, s["sinks"][head].double().expand(n, 1)], 1)
                    p = torch.nan_to_num(torch.softmax(logit, 1), nan=0.0)[:, :L]
                    out[at:at + n, head * D:(head + 1) * D] = p @ v
        at += n
    if case["out"] == "bf16":
        return out
    blocks = out.reshape(s["total"], -1, 32)
    step = blocks.abs().max(-1, keepdim=True).values / 127
    code = torch.where(step > 0, (blocks / step).round(), torch.zeros_like(blocks))
    return code * step.half().double()


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    size = lambda name: 2 if name == "bf16" else 4
    token = 2 * Hkv * D * 9 / 16                       # a token's keys and values in the cache
    if op == "read":
        return dict(bytes=case["n"] * (token + 2 * Hkv * D * size(case["dtype"])), flops=2 * case["n"] * Hkv * D)
    if op == "append":
        n, Hq = case["live"], case["Hq"]
        return dict(bytes=n * ((Hq + 2 * Hkv) * D * size(case["x"]) + Hq * D * size(case["q"]) + token +
                               2 * Hkv * D * 2 + 4 * case["axes"]), flops=n * (6 * Hq + 20 * Hkv) * D)
    pairs, keys = _visible(case)
    n = sum(_rows(case)[:case.get("live", case["B"])])
    return dict(bytes=keys * token + n * case["Hq"] * D * (size(case["q"]) + (2 if case["out"] == "bf16" else 9 / 8)),
                flops=4 * D * case["Hq"] * pairs)
