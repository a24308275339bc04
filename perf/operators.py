"""Workloads of the group-scaled 4-bit weights and of the routed prefill, with plain forms.

Four families of calls:
  mmvq / mmvq_id      projections of one Q8_1 image through 4-bit weights with group scales and zero points
  mmq_id              routed products of a prompt's Q8_0 planes, grouped by expert with ragged sizes
  glu                 act(gate) * up emitting the Q8_0 planes of the next projection
  combine             weighted sum of the routed pair rows

`own` False computes each in elementary torch operations in binary32; True makes the library's
calls. `exact` is the definition in binary64.
"""
import math

import torch

own = False

GLU_KINDS = ("swiglu", "geglu_tanh", "reglu", "geglu_erf", "geglu_quick", "swiglu_oai", "swiglu_clamp")
ALPHA, LIMIT = 1.702, 7.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token through one small projection: launch latency
        dict(name="mmvq one token 256x256", op="mmvq", T=1, live=1, K=256, N=256, N2=0, N3=0, G=64),
        # the q/k/v projections of a decode batch of eight
        dict(name="mmvq qkv 8 tokens", op="mmvq", T=8, live=8, K=3584, N=3584, N2=512, N3=512, G=128),
        # an output head: one weight matrix much larger than the L2 cache
        dict(name="mmvq head 4 tokens", op="mmvq", T=4, live=4, K=8192, N=65536, N2=0, N3=0, G=128),
        # gate and up of 128 experts for a decode bucket of 16 rows of which 13 are live
        dict(name="mmvq_id gate/up 16 rows", op="mmvq_id", rows=16, live=13, k=8, E=128, K=2560, N=768, N2=768, G=64,
             slots=False),
        # a short prompt over eight small experts, odd width
        dict(name="mmq_id 37 rows", op="mmq_id", rows=37, live=37, k=2, E=8, K=320, N=203, N2=0, wtype="q4_g64",
             slots=False, skew=0.5),
        # gate and up of a 512-token prompt chunk: about 32 pairs per expert, bound by the weights
        dict(name="mmq_id gate/up 512 rows", op="mmq_id", rows=512, live=512, k=8, E=128, K=2560, N=768, N2=768,
             wtype="q4_0", slots=False, skew=0.5),
        # gate and up of a long prompt: a few hundred pairs per expert, bound by the products
        dict(name="mmq_id gate/up 4096 rows", op="mmq_id", rows=4096, live=4096, k=8, E=128, K=2560, N=768, N2=768,
             wtype="q4_g128", slots=False, skew=0.5),
        # the down projection of a 3325-token prompt, one image row per pair
        dict(name="mmq_id down 3325 rows", op="mmq_id", rows=3325, live=3325, k=8, E=128, K=768, N=2560, N2=0,
             wtype="q4_0", slots=True, skew=0.5),
        # SwiGLU between the two routed products of that prompt: 16-bit pair rows, gate and up side by side
        dict(name="glu 26600 pairs bf16", op="glu", T=26600, live=26600, N=768, kind="swiglu", layout="packed",
             dtype="bf16", out=False),
        # the same producer in a dense FFN of binary32 rows, its output kept
        dict(name="glu 700 rows f32", op="glu", T=700, live=651, N=18944, kind="geglu_tanh", layout="separate",
             dtype="f32", out=True),
        # combine of a decode bucket and of a prompt
        dict(name="combine 24 rows", op="combine", rows=24, live=17, k=8, N=2560),
        dict(name="combine 3325 rows", op="combine", rows=3325, live=3325, k=8, N=2560),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mmvq", "mmvq_id", "mmq_id", "mmq_id", "glu", "combine"])
    if op == "mmvq":
        G = rng.choice([64, 128])
        K = G * _log(rng, 1, 20480 // G)
        n_max = min(65536, 8192 * 65536 // K)
        T = rng.randint(1, 8)
        return dict(op=op, T=T, live=rng.randint(1, T), K=K, N=_log(rng, 1, n_max), N2=rng.choice([0, rng.randint(1, 1024)]),
                    N3=rng.choice([0, rng.randint(1, 1024)]), G=G)
    if op == "mmvq_id":
        G = rng.choice([64, 128])
        E = _log(rng, 1, 192)
        rows = _log(rng, 1, 32)
        return dict(op=op, rows=rows, live=rng.randint(1, rows), k=rng.randint(1, min(8, E)), E=E,
                    K=G * _log(rng, 1, 4096 // G), N=_log(rng, 1, 1536), N2=rng.choice([0, _log(rng, 1, 1536)]), G=G,
                    slots=rng.choice([False, True]))
    if op == "mmq_id":
        wtype = rng.choice(["q4_0", "q4_g64", "q4_g128"])
        step = {"q4_0": 32, "q4_g64": 64, "q4_g128": 128}[wtype]
        E = _log(rng, 1, 160)
        rows = _log(rng, 1, 4096)
        k = rng.randint(1, min(8, E))
        N = _log(rng, 1, 2560)
        k_max = max(step, min(4096, 4096 * 8 * 1536 * 2560 // (rows * k * N), 128 * 1536 * 2560 // (E * N)))
        return dict(op=op, rows=rows, live=rng.randint(max(1, rows // 2), rows), k=k, E=E,
                    K=step * _log(rng, 1, k_max // step), N=N, N2=0, wtype=wtype, slots=rng.choice([False, True]),
                    skew=round(rng.uniform(0.0, 1.5), 2))
    if op == "glu":
        N = 32 * _log(rng, 1, 640)
        T = _log(rng, 1, max(2, 26600 * 768 // N))
        return dict(op=op, T=T, live=rng.randint(max(1, T // 2), T), N=N, kind=rng.choice(GLU_KINDS),
                    layout=rng.choice(["separate", "packed", "packed_swapped"]), dtype=rng.choice(["bf16", "f32"]),
                    out=rng.choice([False, True]))
    k = rng.randint(1, 8)
    N = 4 * _log(rng, 1, 2048)
    rows = _log(rng, 1, max(2, 3325 * 8 * 2560 // (k * N)))
    rows = min(rows, 8192)
    return dict(op=op, rows=rows, live=rng.randint(max(1, rows // 2), rows), k=k, N=N)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _group(wtype):
    return {"q4_0": 32, "q4_g64": 64, "q4_g128": 128}[wtype]


def _weights(g, wtype, E, N, K):
    """Canonical blocks [E, N, K/G, bytes]: q4_0 [half d][16 bytes]; q4_g* [half d][zero point][0][G/2 bytes]."""
    G = _group(wtype)
    head = 2 if wtype == "q4_0" else 4
    w = torch.randint(0, 256, (E, N, K // G, head + G // 2), dtype=torch.uint8, device="cuda", generator=g)
    d = torch.empty((E, N, K // G), device="cuda").uniform_(0.002, 0.02, generator=g).half()
    w[..., 0:2] = d.unsqueeze(-1).view(torch.uint8)
    if wtype != "q4_0":
        w[..., 2] = torch.randint(4, 12, (E, N, K // G), dtype=torch.uint8, device="cuda", generator=g)
        w[..., 3] = 0
    return w


def _codes(g, rows, K):
    """int8 codes [rows, K] and half scales [rows, K/32] of the 32-blocks of rows ~ N(0, 1)."""
    x = torch.randn((rows, K // 32, 32), device="cuda", generator=g)
    d = x.abs().amax(-1, keepdim=True) / 127
    q = torch.round(x / d).to(torch.int8)
    return q.reshape(rows, K), d.squeeze(-1).half()


def _image(q, d):
    """The Q8_1 image's bytes: [half d][half d * sum q][32 codes] per block."""
    rows, K = q.shape
    qb = q.view(rows, K // 32, 32)
    s = (d.float() * qb.float().sum(-1)).half()
    return torch.cat([d.unsqueeze(-1).view(torch.uint8), s.unsqueeze(-1).view(torch.uint8), qb.view(torch.uint8)],
                     -1).contiguous()


def _route(g, case):
    """A router's picks and their plan: ids [rows, k], counts, offsets, items (pairs by expert, ascending)."""
    rows, k, E, live = case["rows"], case["k"], case["E"], case["live"]
    logits = torch.randn((rows, E), device="cuda", generator=g)
    logits += case.get("skew", 0.5) * torch.randn((E,), device="cuda", generator=g)
    ids = logits.topk(k, dim=-1).indices.to(torch.int32)
    flat = ids[:live].reshape(-1).long()
    items = torch.full((rows * k,), -1, dtype=torch.int32, device="cuda")
    items[:live * k] = torch.sort(flat, stable=True).indices.to(torch.int32)
    counts = torch.bincount(flat, minlength=E).to(torch.int32)
    offsets = torch.zeros((E + 1,), dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return ids, counts, offsets, items


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "mmvq":
        s["img"] = _image(*_codes(g, case["T"], case["K"]))
        s["Ns"] = [n for n in (case["N"], case["N2"], case["N3"]) if n]
        s["w"] = [_weights(g, "q4_g%d" % case["G"], 1, n, case["K"]) for n in s["Ns"]]
        s["y"] = [torch.zeros((case["T"], n), device="cuda") for n in s["Ns"]]
        s["live"] = torch.tensor([case["live"]], dtype=torch.int32, device="cuda")
    elif op in ("mmvq_id", "mmq_id"):
        wtype = case["wtype"] if op == "mmq_id" else "q4_g%d" % case["G"]
        pairs = case["rows"] * case["k"]
        s["q"], s["d"] = _codes(g, pairs if case["slots"] else case["rows"], case["K"])
        if op == "mmvq_id":
            s["img"] = _image(s.pop("q"), s.pop("d"))
        s["wtype"], s["Ns"] = wtype, [n for n in (case["N"], case["N2"]) if n]
        s["w"] = [_weights(g, wtype, case["E"], n, case["K"]) for n in s["Ns"]]
        s["ids"], s["counts"], s["offsets"], s["items"] = _route(g, case)
        s["most"] = int(s["counts"].max())
        # gate and up share one buffer of pair rows, as the GLU's packed input
        s["y"] = torch.zeros((pairs, sum(s["Ns"])), dtype=torch.bfloat16 if op == "mmq_id" else torch.float32,
                             device="cuda")
        if op == "mmvq_id":
            s["y"] = [torch.zeros((pairs, n), device="cuda") for n in s["Ns"]]
    elif op == "glu":
        T, N = case["T"], case["N"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case["layout"] == "separate":
            s["a"] = (2 * torch.randn((T, N), device="cuda", generator=g)).to(dt)
            s["b"] = (2 * torch.randn((T, N), device="cuda", generator=g)).to(dt)
        else:
            s["a"] = (2 * torch.randn((T, 2 * N), device="cuda", generator=g)).to(dt)
            s["b"] = None
        s["out"] = torch.zeros((T, N), device="cuda") if case["out"] else None
        s["qs"] = torch.zeros((T, N), dtype=torch.int8, device="cuda")
        s["dh"] = torch.zeros((T, N // 32), dtype=torch.float16, device="cuda")
        s["live"] = torch.tensor([case["live"]], dtype=torch.int32, device="cuda")
    else:
        rows, k, N = case["rows"], case["k"], case["N"]
        s["e"] = torch.randn((rows * k, N), device="cuda", generator=g).bfloat16()
        s["wts"] = torch.softmax(torch.randn((rows, max(k, 8)), device="cuda", generator=g), -1)[:, :k].contiguous()
        s["y"] = torch.zeros((rows, N), device="cuda")
        s["live"] = torch.tensor([case["live"]], dtype=torch.int32, device="cuda")
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a user of the library keeps: the packed weights, the projections' descriptors and a workspace."""
    from quantized_activation_q4_gb300 import binding as qk
    case = s["case"]
    op = case["op"]
    if "w" not in s:
        return
    E = case.get("E", 1)
    wtype = s.get("wtype", "q4_g%d" % case.get("G", 0))
    s["packed"], s["projs"] = [], []
    for j, n in enumerate(s["Ns"]):
        K = case["K"]
        per = qk.qk_weight_packed_bytes(wtype, n, K)
        buf = torch.empty((E * per,), dtype=torch.uint8, device="cuda")
        for e in range(E):
            qk.qk_weight_pack(wtype, s["w"][j][e], n, K, buf[e * per:(e + 1) * per], per)
        s["packed"].append(buf)
        if op == "mmvq":
            s["projs"].append(qk.make_proj(wtype, buf, n, K, s["y"][j], n))
        elif op == "mmvq_id":
            s["projs"].append(qk.make_proj_id(wtype, E, buf, n, K, s["y"][j]))
        else:
            width = sum(s["Ns"])
            s["projs"].append(qk.make_proj_id16(wtype, E, buf, n, K, s["y"][:, sum(s["Ns"][:j]):], width))
    del s["w"]
    if op == "mmvq":
        s["ws_bytes"] = qk.qk_mmvq_workspace_bytes(s["projs"])
        s["ws"] = torch.zeros((max(16, s["ws_bytes"]),), dtype=torch.uint8, device="cuda")
    elif op == "mmq_id":
        # room for every pair's activation row, so the size depends on the rows and the slots per row
        s["ws_bytes"] = qk.qk_mmq_id_workspace_bytes(case["rows"], case["k"], s["projs"])
        s["ws"] = torch.empty((s["ws_bytes"],), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from quantized_activation_q4_gb300 import binding as qk
    case = s["case"]
    op = case["op"]
    if op == "mmvq":
        qk.qk_mmvq(s["img"], case["K"] // 32, case["T"], s["projs"], s["ws"], s["ws_bytes"], s["live"])
        return s["y"]
    if op == "mmvq_id":
        call = qk.qk_mmvq_id_slots if case["slots"] else qk.qk_mmvq_id
        call(s["img"], case["K"] // 32, case["rows"], case["k"], s["projs"], s["counts"], s["offsets"], s["items"])
        return s["y"]
    if op == "mmq_id":
        call = qk.qk_mmq_id_slots if case["slots"] else qk.qk_mmq_id
        call(s["q"], s["d"], case["K"] // 32, case["rows"], case["k"], s["projs"], s["counts"], s["offsets"],
             s["items"], s["ws"], s["ws_bytes"])
        return s["y"]
    if op == "glu":
        N = case["N"]
        stride = N if case["layout"] == "separate" else 2 * N
        qk.qk_glu_q8_0(case["kind"], case["layout"], case["dtype"], s["a"], stride, s["b"], N, case["T"], N, s["out"],
                       N, s["qs"], s["dh"], N // 32, ALPHA, LIMIT, s["live"])
        return dict(planes=_plane_values(s["qs"], s["dh"]), out=s["out"])
    qk.qk_moe_combine_bf16(s["e"], case["N"], s["wts"], case["rows"], case["k"], case["N"], s["y"], case["N"],
                           s["live"])
    return s["y"]


def _plane_values(qs, dh):
    """The values that the planes' codes stand for; 16 bits hold more than their 8."""
    T, N = qs.shape
    return (qs.view(T, N // 32, 32) * dh.unsqueeze(-1)).view(T, N)


def _dequant(w, dtype):
    """Blocks [..., K/G, bytes] -> values [..., K]."""
    head = 2 if w.shape[-1] == 18 else 4
    d = w[..., 0:2].contiguous().view(torch.float16).to(dtype)
    z = 8 if head == 2 else w[..., 2:3].to(dtype).unsqueeze(-2)
    c = w[..., head:].unflatten(-1, (-1, 16))
    c = torch.cat([c & 15, c >> 4], -1).to(dtype)          # [..., K/G, G/32, 32]
    return ((c - z) * d.unsqueeze(-1)).flatten(-3)


def _image_values(img):
    d = img[..., 0:2].contiguous().view(torch.float16).float()
    return (img[..., 4:].view(torch.int8).float() * d).flatten(-2)


def _plane_rows(q, d):
    return (q.float().unflatten(-1, (-1, 32)) * d.float().unsqueeze(-1)).flatten(-2)


def _act(kind, g, u):
    if kind == "swiglu":
        return g / (1 + torch.exp(-g)) * u
    if kind == "geglu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))) * u
    if kind == "reglu":
        return torch.clamp(g, min=0) * u
    if kind == "geglu_erf":
        return 0.5 * g * (1 + torch.erf(g / math.sqrt(2))) * u
    if kind == "geglu_quick":
        return g / (1 + torch.exp(-1.702 * g)) * u
    g, u = torch.clamp(g, max=LIMIT), torch.clamp(u, -LIMIT, LIMIT)
    if kind == "swiglu_oai":
        return g / (1 + torch.exp(-ALPHA * g)) * (u + 1)
    return g / (1 + torch.exp(-g)) * u


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "mmvq":
        x = _image_values(s["img"])
        x = x * (torch.arange(case["T"], device="cuda") < s["live"]).unsqueeze(-1)
        return [x @ _dequant(w[0], torch.float32).T for w in s["w"]]
    if op in ("mmvq_id", "mmq_id"):
        x = _image_values(s["img"]) if op == "mmvq_id" else _plane_rows(s["q"], s["d"])
        # each expert's pairs as one batch of `most` rows, the rest of it zero
        E, k, total, most = case["E"], case["k"], case["live"] * case["k"], s["most"]
        pair = s["items"][:total].long()
        expert = s["ids"].reshape(-1)[pair].long()
        place = expert * most + torch.arange(total, device="cuda") - s["offsets"][expert]
        xe = torch.zeros((E * most, x.shape[1]), device="cuda")
        xe[place] = x[pair if case["slots"] else pair // k]
        ys = []
        for w in s["w"]:
            ye = torch.bmm(xe.view(E, most, -1), _dequant(w, torch.float32).transpose(1, 2)).flatten(0, 1)
            y = torch.zeros((case["rows"] * k, w.shape[1]), device="cuda")
            y[pair] = ye[place]
            ys.append(y)
        return ys if op == "mmvq_id" else torch.cat(ys, 1).bfloat16()
    if op == "glu":
        N = case["N"]
        a = s["a"].float()
        g, u = (a, s["b"].float()) if case["layout"] == "separate" else (a[:, :N], a[:, N:])
        if case["layout"] == "packed_swapped":
            g, u = u, g
        h = _act(case["kind"], g, u) * (torch.arange(case["T"], device="cuda") < s["live"]).unsqueeze(-1)
        hb = h.unflatten(-1, (-1, 32))
        d = hb.abs().amax(-1, keepdim=True) / 127
        q = torch.where(d > 0, torch.round(hb / d), 0.0)
        return dict(planes=(q * d.half().float()).flatten(-2).half(), out=h if case["out"] else None)
    e = s["e"].float().unflatten(0, (-1, case["k"]))
    y = (e * s["wts"].unsqueeze(-1)).sum(1)
    return y * (torch.arange(case["rows"], device="cuda") < s["live"]).unsqueeze(-1)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_weight(blocks, wtype):
    """One matrix [N, K] from its blocks, element j of a 32-run in byte j % 16, nibble j // 16."""
    G = _group(wtype)
    N, nb, _ = blocks.shape
    head = 2 if wtype == "q4_0" else 4
    out = torch.empty((N, nb, G), dtype=torch.float64, device="cuda")
    scale = blocks[:, :, :2].contiguous().view(torch.float16).double()[:, :, 0]
    zero = torch.full_like(scale, 8.0) if wtype == "q4_0" else blocks[:, :, 2].double()
    for run_ in range(G // 32):
        by = blocks[:, :, head + 16 * run_:head + 16 * (run_ + 1)].int()
        for half, v in enumerate((by % 16, by // 16)):
            lo = 32 * run_ + 16 * half
            out[:, :, lo:lo + 16] = (v.double() - zero[:, :, None]) * scale[:, :, None]
    return out.reshape(N, nb * G)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, live = case["op"], case["live"]
    if op in ("mmvq", "mmvq_id"):
        blocks = s["img"].reshape(s["img"].shape[0], -1, 36)
        x = blocks[:, :, 4:].view(torch.int8).double() * blocks[:, :, :2].contiguous().view(torch.float16).double()
        x = x.reshape(blocks.shape[0], -1)
    elif op == "mmq_id":
        x = (s["q"].double().reshape(s["q"].shape[0], -1, 32) * s["d"].double()[:, :, None]).reshape(s["q"].shape)
    if op == "mmvq":
        ys = []
        for w, n in zip(s["w"], s["Ns"]):
            y = torch.zeros((case["T"], n), dtype=torch.float64, device="cuda")
            for lo in range(0, n, 8192):
                y[:live, lo:lo + 8192] = x[:live] @ _exact_weight(w[0, lo:lo + 8192], "q4_g%d" % case["G"]).T
            ys.append(y)
        return ys
    if op in ("mmvq_id", "mmq_id"):
        pairs = torch.arange(live * case["k"], device="cuda")
        ids = s["ids"].reshape(-1)[:live * case["k"]]
        ys = [torch.zeros((case["rows"] * case["k"], n), dtype=torch.float64, device="cuda") for n in s["Ns"]]
        for e in range(case["E"]):
            p = pairs[ids == e]
            if p.numel():
                xe = x[p if case["slots"] else torch.div(p, case["k"], rounding_mode="floor")]
                for y, w in zip(ys, s["w"]):
                    y[p] = xe @ _exact_weight(w[e], s["wtype"]).T
        return ys if op == "mmvq_id" else torch.cat(ys, 1)
    if op == "glu":
        N, T = case["N"], case["T"]
        a = s["a"].double()
        parts = (a, s["b"].double()) if case["layout"] == "separate" else (a[:, :N], a[:, N:])
        g, u = parts[::-1] if case["layout"] == "packed_swapped" else parts
        kind = case["kind"]
        if kind in ("swiglu_oai", "swiglu_clamp"):
            g, u = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
        if kind in ("swiglu", "swiglu_clamp"):
            h = g * torch.sigmoid(g) * u
        elif kind == "swiglu_oai":
            h = g * torch.sigmoid(ALPHA * g) * (u + 1)
        elif kind == "geglu_quick":
            h = g * torch.sigmoid(1.702 * g) * u
        elif kind == "reglu":
            h = torch.relu(g) * u
        elif kind == "geglu_erf":
            h = g * 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) * u
        else:
            h = g * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * g * (1 + 0.044715 * g * g))) * u
        h[live:] = 0
        hb = h.reshape(T, N // 32, 32)
        step = hb.abs().max(-1, keepdim=True).values / 127
        q = torch.where(step > 0, (hb / step).round(), torch.zeros_like(hb))
        return dict(planes=(q * step.half().double()).reshape(T, N), out=h if case["out"] else None)
    y = torch.zeros((case["rows"], case["N"]), dtype=torch.float64, device="cuda")
    e = s["e"].double().reshape(case["rows"], case["k"], case["N"])
    for slot in range(case["k"]):
        y += e[:, slot] * s["wts"][:, slot, None].double()
    y[live:] = 0
    return y


# ------------------------------------------------------------------ what a pass cannot do without
def _block_bytes(wtype):
    return {"q4_0": 18 / 32, "q4_g64": 36 / 64, "q4_g128": 68 / 128}[wtype]


def work(case):
    op = case["op"]
    if op == "mmvq":
        n = case["N"] + case["N2"] + case["N3"]
        return dict(bytes=n * case["K"] * _block_bytes("q4_g%d" % case["G"]) + case["live"] * case["K"] * 36 / 32 +
                    4 * case["live"] * n, flops=2 * case["live"] * n * case["K"])
    if op in ("mmvq_id", "mmq_id"):
        wtype = case["wtype"] if op == "mmq_id" else "q4_g%d" % case["G"]
        n, pairs = case["N"] + case["N2"], case["live"] * case["k"]
        touched = case["E"] * (1 - (1 - case["k"] / case["E"]) ** case["live"])   # experts with a pair, expected
        rows = pairs if case["slots"] else case["live"]
        return dict(bytes=touched * n * case["K"] * _block_bytes(wtype) +
                    rows * case["K"] * (36 if op == "mmvq_id" else 34) / 32 +
                    pairs * n * (4 if op == "mmvq_id" else 2), flops=2 * pairs * n * case["K"])
    if op == "glu":
        n = case["live"] * case["N"]
        return dict(bytes=n * (2 * (2 if case["dtype"] == "bf16" else 4) + 34 / 32 + (4 if case["out"] else 0)),
                    flops=20 * n)
    n = case["live"] * case["N"]
    return dict(bytes=n * (2 * case["k"] + 4) + 4 * case["live"] * case["k"], flops=2 * n * case["k"])
