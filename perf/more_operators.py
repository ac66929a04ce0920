"""Serving from a paged 8-bit KV cache: the three operators' plain forms, the
calls of the library that compute them, and the cases they are measured at.

* ``rotate``  rotary positions on a projection's output (or, turned back, on
              the gradient of the rotated tensor)
* ``append``  new tokens' K (rotated on the way) and V into the pages of their
              sequences, as 8-bit codes with one scale for each page and head;
              the tokens' Q rotated beside them
* ``attend``  attention of the new tokens (one, a few, a chunk, a whole prompt)
              over the pages of their sequences
"""
import math

import torch

own = False

LOG2E = 1.4426950408889634
DEV = "cuda"
#: the largest magnitude of a code; a block with nothing above FLUSH holds zeros
TOP = {"int8": 127.0, "e4m3": 448.0}
FLUSH = 2.0 ** -64
#: most score elements (padded) of a drawn case
MOST = 2 ** 31


# --------------------------------------------------------------------- cases
def listed():
    return [
        # Q of an 8K prompt
        dict(name="rotate_prompt", op="rotate", B=1, H=32, T=8192, d=128, rot=128, inter=False, back=False,
             pos="none", dt="bf16"),
        # training: the gradient turned back, neighbouring pairs, half of the head, documents packed
        dict(name="rotate_gradient", op="rotate", B=8, H=12, T=1021, d=64, rot=32, inter=True, back=True,
             pos="given", dt="bf16"),
        # one chat user's next token: launch latency counts
        dict(name="append_one", op="append", B=1, Hq=32, Hkv=8, d=128, page=64, code="int8", lo=4097, hi=4097,
             T=1, ragged=False, rot=128, inter=False),
        # a serving batch's next tokens, each sequence at its own place in its last page
        dict(name="append_batch", op="append", B=64, Hq=32, Hkv=8, d=128, page=64, code="int8", lo=201, hi=4500,
             T=1, ragged=False, rot=128, inter=False),
        # prompts of uneven length into empty sequences
        dict(name="append_prompts", op="append", B=4, Hq=32, Hkv=8, d=128, page=128, code="int8", lo=0, hi=0,
             T=4099, ragged=True, rot=128, inter=False),
        # a chunk of a long prompt behind what is there, e4m3 codes, part of the head rotated in pairs
        dict(name="append_chunk_e4m3", op="append", B=2, Hq=16, Hkv=16, d=64, page=32, code="e4m3", lo=1003,
             hi=2048, T=2048, ragged=False, rot=32, inter=True),
        # one token of a chat reply: launch latency counts
        dict(name="attend_one", op="attend", B=1, Hq=32, Hkv=8, d=128, page=64, code="int8", lo=4097, hi=4097,
             T=1, ragged=False, causal=True),
        # a decode step of a serving batch at uneven lengths
        dict(name="attend_batch", op="attend", B=32, Hq=32, Hkv=8, d=128, page=64, code="int8", lo=211, hi=8191,
             T=1, ragged=False, causal=True),
        # long contexts, e4m3 codes
        dict(name="attend_long_e4m3", op="attend", B=8, Hq=32, Hkv=8, d=128, page=128, code="e4m3", lo=16385,
             hi=32768, T=1, ragged=False, causal=True),
        # a few tokens of each sequence (short questions behind cached documents), small model
        dict(name="attend_few_d64", op="attend", B=8, Hq=32, Hkv=8, d=64, page=32, code="int8", lo=1023, hi=16000,
             T=24, ragged=True, causal=True),
        # the largest: a chunk of 2048 tokens at the end of 32K
        dict(name="attend_chunk", op="attend", B=1, Hq=32, Hkv=8, d=128, page=64, code="int8", lo=32768, hi=32768,
             T=2048, ragged=False, causal=True),
        # whole prompts, uneven, from an e4m3 cache
        dict(name="attend_prompts", op="attend", B=4, Hq=12, Hkv=12, d=64, page=64, code="e4m3", lo=1777, hi=4099,
             T=4099, ragged=True, causal=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _time_floor(case):
    w = work(case)
    return w["bytes"] / 6.7e12 + w["flops"] / 1.9e15


def draw(rng):
    top = max(_time_floor(c) for c in listed())
    while True:
        op = rng.choice(["rotate", "append", "append", "attend", "attend", "attend"])
        B = _log(rng, 1, 64)
        d = rng.choice([64, 128, 128])
        rot = rng.choice([d, d, d // 2, 24])
        Hkv, G = rng.choice([(8, 4), (8, 4), (12, 1), (4, 8), (2, 3), (1, 16), (16, 2), (8, 1)])
        if op == "rotate":
            case = dict(op=op, B=B, H=Hkv * G, T=_log(rng, 1, 8192), d=d, rot=rot, inter=rng.random() < 0.5,
                        back=rng.random() < 0.5, pos=rng.choice(["none", "given"]), dt=rng.choice(["bf16", "bf16", "f32"]))
        else:
            hi = _log(rng, 1, 32768)
            case = dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, page=rng.choice([32, 64, 128]),
                        code=rng.choice(["int8", "e4m3"]), lo=_log(rng, 1, hi), hi=hi)
            if op == "append":
                if rng.random() < 0.3:
                    case.update(lo=0, hi=0)
                case.update(T=_log(rng, 1, 8192), ragged=rng.random() < 0.5, rot=rot, inter=rng.random() < 0.5)
                if B * (hi + case["T"]) * Hkv * d > 2 ** 29:  # the pool's codes
                    continue
            else:
                case.update(T=_log(rng, 1, min(hi, 8192)), ragged=rng.random() < 0.5, causal=rng.random() < 0.8)
                if B * case["Hq"] * case["T"] * hi > MOST or B * hi * Hkv * d > 2 ** 30:
                    continue
        if _time_floor(case) <= top:
            return case


def _spread(lo, hi, B):
    """B whole numbers spread over [lo, hi], the last at hi."""
    return [hi - (hi - lo) * ((7 * (B - 1 - b)) % B) // max(B - 1, 1) for b in range(B)]


def _new(case):
    """New tokens of each sequence."""
    B, T = case["B"], case["T"]
    return _spread(1 + T // 3, T, B)[::-1] if case["ragged"] else [T] * B


def _before(case):
    """Rows in use before the new tokens (append)."""
    return _spread(case["lo"], case["hi"], case["B"])


def _lengths(case):
    """Rows in use, the new tokens' among them."""
    if case["op"] == "append":
        return [a + n for a, n in zip(_before(case), _new(case))]
    return [max(a, n) for a, n in zip(_spread(case["lo"], case["hi"], case["B"]), _new(case))]


def _pairs(case):
    """(query, row) pairs of one head that are visible, over the batch."""
    total = 0
    for L, n in zip(_lengths(case), _new(case)):
        total += n * L - (n * (n - 1) // 2 if case["causal"] else 0)
    return total


def work(case):
    op, B, d = case["op"], case["B"], case["d"]
    if op == "rotate":
        size = 2 if case["dt"] == "bf16" else 4
        tokens = B * case["T"]
        table = (case["T"] if case["pos"] == "none" else tokens) * case["rot"] * 4
        return {"bytes": 2 * size * tokens * case["H"] * d + table + (4 * tokens if case["pos"] == "given" else 0),
                "flops": 3 * tokens * case["H"] * case["rot"]}
    Hkv, page = case["Hkv"], case["page"]
    n = sum(_new(case))
    if op == "append":
        pages = sum((L - 1) // page - (L - m) // page + 1 for L, m in zip(_lengths(case), _new(case)))
        byts = (n * Hkv * d * 6                        # K and V in, codes out
                + n * case["Hq"] * d * 4               # Q in and out
                + n * case["rot"] * 4                  # angles
                + pages * (2 * Hkv * 4 + 4) + 8 * B)   # scales, page numbers, lengths
        return {"bytes": byts, "flops": n * (case["Hq"] + Hkv) * case["rot"] * 3 + 4 * n * Hkv * d}
    rows = sum(_lengths(case))
    pages = sum(-(-L // page) for L in _lengths(case))
    byts = (2 * rows * Hkv * d + pages * (8 * Hkv + 4) + 8 * B
            + n * case["Hq"] * (4 * d + 4))
    return {"bytes": byts, "flops": 4 * d * case["Hq"] * _pairs(case)}


# -------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(2000003 + seed)
    return g


def _table(n, rot, stretch=4.0, base=10000.0):
    """Cosines and sines [n, rot] of n positions, stretched for a longer context:
    the slow channels' angles divided by `stretch`, the fast ones' as they are, a
    ramp between."""
    half = rot // 2
    i = torch.arange(half, dtype=torch.float64, device=DEV)
    freq = base ** (-2.0 * i / rot)
    turns = freq * 2048.0 / (2.0 * math.pi)             # over the context trained on
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    freq = freq * keep + freq / stretch * (1.0 - keep)
    a = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * freq
    mscale = 0.1 * math.log(stretch) + 1.0
    return (torch.cat([a.cos(), a.sin()], dim=1) * mscale).to(torch.float32).contiguous()


def _projection(g, B, T, H, d, dt=torch.bfloat16, outliers=False):
    """A projection's output [B, T, H, d], seen as [B, H, T, d]."""
    x = torch.randn(B, T, H, d, generator=g, device=DEV)
    if outliers:  # the channels that an LLM's keys have far above the others
        for c in (7, 35, 62):
            x[..., c] *= 9.0
    return x.to(dt).transpose(1, 2)


def _codes(g, code, *shape):
    """Codes shaped by N(0, 1), the largest near the type's top."""
    out = torch.empty(shape, dtype=torch.int8 if code == "int8" else torch.uint8, device=DEV)
    flat = out.view(shape[0], -1)
    step = max(1, 2 ** 26 // flat.shape[1])
    for i in range(0, shape[0], step):
        z = torch.randn(flat[i:i + step].shape, generator=g, device=DEV) * (TOP[code] / 4.5)
        z = z.clamp(-TOP[code], TOP[code])
        flat[i:i + step] = z.round().to(torch.int8) if code == "int8" else z.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _paged(case, g, st):
    """A pool whose pages lie in no order, with the sequences' page table."""
    B, page, L = case["B"], case["page"], _lengths(case)
    need = [-(-x // page) for x in L]
    n_pages, width = sum(need) + 3, max(need) + 1
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    st.update(n_pages=n_pages, width=width, pt=table,
              lengths=torch.tensor(L, dtype=torch.int32, device=DEV),
              n_new=torch.tensor(_new(case), dtype=torch.int32, device=DEV))
    shape = (n_pages, case["Hkv"], page, case["d"])
    st["kp"], st["vp"] = _codes(g, case["code"], *shape), _codes(g, case["code"], *shape)
    for name in ("ks", "vs"):
        st[name] = (0.5 + torch.rand(n_pages, case["Hkv"], generator=g, device=DEV)) * (4.5 / TOP[case["code"]])


def _inputs(case, seed):
    g = _gen(seed)
    op, B, T, d = case["op"], case["B"], case["T"], case["d"]
    st = dict(case=case)
    if op == "rotate":
        dt = torch.bfloat16 if case["dt"] == "bf16" else torch.float32
        st["x"] = _projection(g, B, T, case["H"], d, dt)
        st["y"] = torch.empty(B, case["H"], T, d, dtype=dt, device=DEV)
        st["table"] = _table(T, case["rot"])
        st["pos"] = None
        if case["pos"] == "given":  # documents packed one behind the other
            start = torch.randint(0, max(1, T // 2), (B, 1), generator=g, device=DEV)
            st["pos"] = ((torch.arange(T, device=DEV)[None] + start) % T).to(torch.int32).contiguous()
        return st
    Hq, Hkv = case["Hq"], case["Hkv"]
    _paged(case, g, st)
    st["q"] = _projection(g, B, T, Hq, d)
    if op == "append":
        st["k"], st["v"] = _projection(g, B, T, Hkv, d, outliers=True), _projection(g, B, T, Hkv, d)
        # what a sequence holds at first was met by smaller outliers: some pages' scales have to grow
        st["ks"] *= 2.0
        st["table"] = _table(max(_lengths(case)), case["rot"])
        st["q_out"] = torch.zeros(B, Hq, T, d, dtype=torch.bfloat16, device=DEV)
    else:
        st["o"] = torch.zeros(B, Hq, T, d, dtype=torch.bfloat16, device=DEV)
        st["lse"] = torch.zeros(B, Hq, T, device=DEV)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from quantized_attention_gb300 import binding as qb
        if "table" in st:
            st["rope"] = qb.make_rope(st["table"], interleaved=case["inter"], inverse=case.get("back", False))
        if case["op"] != "rotate":
            st["paging"] = qb.make_paging(st["n_pages"], case["page"], st["width"],
                                          qb.DT_I8 if case["code"] == "int8" else qb.DT_E4M3)
            st["shape"] = qb.make_shape(case["B"], case["Hq"], case["Hkv"], case["T"], max(_lengths(case)), case["d"])
        if case["op"] == "attend":
            st["params"] = qb.make_params(causal=case["causal"], out_dtype=qb.DT_BF16)
            need = qb.paged_workspace_size(st["shape"], st["params"], st["paging"])
            st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return st


# --------------------------------------------------------------- plain forms
def _turn(x, cs, inter, back):
    """x [B, H, T, d] turned by the angles of cs [B or 1, T, rot]; every product and
    sum rounded to 32 bits."""
    rot = cs.shape[-1]
    c, s = cs[:, None, :, :rot // 2], cs[:, None, :, rot // 2:]
    if back:
        s = -s
    x = x.float()
    y = x.clone()
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * c - b * s, b * c + a * s
    if inter:
        y[..., :rot:2], y[..., 1:rot:2] = u, v
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = u, v
    return y


def _plain_rotate(st):
    c = st["case"]
    cs = st["table"][None] if st["pos"] is None else st["table"][st["pos"].long()]
    st["y"].copy_(_turn(st["x"], cs, c["inter"], c["back"]))
    return st["y"]


def _values(p, code):
    return p.float() if code == "int8" else p.view(torch.float8_e4m3fn).float()


def _encode(y, code):
    if code == "int8":
        return y.round().clamp(-127.0, 127.0).to(torch.int8)
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_store(st, x, pages, scales):
    """x [B, Hkv, T, d] fp32 into the pages.  The scale of a page: its largest
    magnitude over the type's top; one that holds rows already keeps its scale, or
    doubles it until the new rows fit, its rows' codes divided along."""
    c = st["case"]
    B, Hkv, T, d, page, top = c["B"], c["Hkv"], c["T"], c["d"], c["page"], TOP[c["code"]]
    first = st["lengths"].long() - st["n_new"].long()
    t = torch.arange(T, device=DEV)
    live = t[None] < st["n_new"][:, None]                       # [B, T]
    row = first[:, None] + t[None]
    slot = torch.where(live, row // page - (first // page)[:, None], 0)
    J = (T + page - 2) // page + 1                                # touched pages, at most
    a = torch.where(live[:, None], x.abs().amax(dim=3), 0.0)      # [B, Hkv, T]
    amax = torch.zeros(B, Hkv, J, device=DEV).scatter_reduce(2, slot[:, None].expand(B, Hkv, T), a, "amax")
    j = (first // page)[:, None] + torch.arange(J, device=DEV)[None]
    used = j * page < st["lengths"][:, None]                      # [B, J]
    no = st["pt"].gather(1, j.clamp(max=st["width"] - 1)).long().clamp(min=0)
    fresh = torch.where(amax < FLUSH, torch.zeros_like(amax), amax / top)
    old = scales[no].transpose(1, 2)                              # [B, Hkv, J]
    held = ((j * page < first[:, None]) & used)[:, None] & (old > 0)
    (ma, ea), (mb, eb) = torch.frexp(amax), torch.frexp(old * top)
    up = torch.where(amax > old * top, ea - eb + (ma > mb).int(), torch.zeros_like(ea))
    s = torch.where(held, torch.ldexp(old, up), fresh)
    # the codes of the first page's rows, where its scale has grown
    grow = torch.where(held[:, :, 0], up[:, :, 0], torch.zeros_like(up[:, :, 0]))
    was = pages[no[:, 0]]
    again = _encode(_values(was, c["code"]) * torch.ldexp(torch.ones_like(s[:, :, 0]), -grow)[:, :, None, None], c["code"])
    keep = (grow[:, :, None] == 0) | (torch.arange(page, device=DEV) >= (first % page)[:, None, None])
    bi = st["n_new"] > 0
    pages[no[bi, 0]] = torch.where(keep[..., None], was, again)[bi]
    scales[no[used]] = s.transpose(1, 2)[used]
    # the new rows
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s)).gather(2, slot[:, None].expand(B, Hkv, T))
    codes = _encode(x * inv[..., None], c["code"])
    b, i = live.nonzero(as_tuple=True)
    pages[no[b, slot[b, i]], :, row[b, i] % page] = codes[b, :, i]


def _plain_append(st):
    c = st["case"]
    pos = (st["lengths"] - st["n_new"]).long()[:, None] + torch.arange(c["T"], device=DEV)[None]
    cs = st["table"][pos.clamp(max=st["table"].shape[0] - 1)]
    live = (torch.arange(c["T"], device=DEV)[None] < st["n_new"][:, None])[:, None, :, None]
    st["q_out"].copy_(torch.where(live, _turn(st["q"], cs, c["inter"], False).to(torch.bfloat16), st["q_out"]))
    _plain_store(st, _turn(st["k"], cs, c["inter"], False), st["kp"], st["ks"])
    _plain_store(st, st["v"].float(), st["vp"], st["vs"])
    return _appended(st)


def _appended(st):
    if st["case"]["code"] == "int8":
        kp, vp = st["kp"], st["vp"]
    else:
        kp, vp = st["kp"].view(torch.float8_e4m3fn), st["vp"].view(torch.float8_e4m3fn)
    return {"q": st["q_out"], "kp": kp, "vp": vp, "ks": st["ks"], "vs": st["vs"]}


def _gathered(st, pages, scales):
    """The sequences' rows [B, Hkv, Lmax, d] as fp32."""
    c = st["case"]
    no = st["pt"][:, :-1].long().clamp(min=0)
    x = _values(pages[no], c["code"]) * scales[no][..., None, None]   # [B, pages, Hkv, page, d]
    B, n, Hkv, page, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * page, d)


def _plain_attend(st):
    c = st["case"]
    B, Hq, Hkv, d, T = c["B"], c["Hq"], c["Hkv"], c["d"], c["T"]
    G = Hq // Hkv
    k = _gathered(st, st["kp"], st["ks"])
    L = k.shape[2]
    s = st["q"].float().reshape(B, Hkv, G * T, d) @ k.transpose(2, 3)
    del k
    s = s.mul_(1.0 / math.sqrt(d)).view(B, Hkv, G, T, L)
    r = torch.arange(L, device=DEV)
    see = (r[None] < st["lengths"][:, None])[:, None].expand(B, T, L)
    if c["causal"]:
        p = (st["lengths"] - st["n_new"])[:, None] + torch.arange(T, device=DEV)[None]
        see = see & (r[None, None] <= p[:, :, None])
    s.masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    s.sub_(m).exp_()
    l = s.sum(dim=-1, keepdim=True)
    o = s.view(B, Hkv, G * T, L) @ _gathered(st, st["vp"], st["vs"])
    o = (o.view(B, Hkv, G, T, d) / l).view(B, Hq, T, d)
    lse = (m + l.log()).view(B, Hq, T)
    live = (torch.arange(T, device=DEV)[None] < st["n_new"][:, None])[:, None]
    st["o"].copy_(torch.where(live[..., None], o.to(torch.bfloat16), st["o"]))
    st["lse"].copy_(torch.where(live, lse, st["lse"]))
    return {"o": st["o"], "lse": st["lse"]}


# ----------------------------------------------------------------- one pass
def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"rotate": _plain_rotate, "append": _plain_append, "attend": _plain_attend}[op](s)
    from quantized_attention_gb300 import binding as qb
    if op == "rotate":
        qb.rotate(s["x"], s["y"], s["rope"], positions=s["pos"])
        return s["y"]
    if op == "append":
        qb.paged_append(s["k"], s["v"], s["shape"], s["paging"], s["pt"], s["lengths"], s["kp"], s["vp"], s["ks"],
                        s["vs"], n_new=s["n_new"], rope=s["rope"], Q=s["q"], Q_out=s["q_out"])
        return _appended(s)
    qb.paged_fwd(s["q"], s["shape"], s["params"], s["paging"], s["pt"], s["lengths"], s["kp"], s["vp"], s["ks"],
                 s["vs"], s["o"], s["lse"], s["ws"], n_new=s["n_new"])
    return {"o": s["o"], "lse": s["lse"]}


# ----------------------------------------------------------- in 64 bits
def _exact_turn(x, cos, sin, inter):
    """As complex numbers: the pair (a, b) times cos + i sin."""
    rot = 2 * cos.shape[-1]
    x = x.double()
    a = x[..., :rot]
    z = (torch.view_as_complex(a.unflatten(-1, (rot // 2, 2)).contiguous()) if inter else
         torch.complex(*a.chunk(2, dim=-1)))
    w = z * torch.complex(cos, sin)
    turned = torch.view_as_real(w).flatten(-2) if inter else torch.cat([w.real, w.imag], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _exact_rotate(st):
    c = st["case"]
    out = torch.empty(st["y"].shape, dtype=torch.float64, device=DEV)
    cos, sin = st["table"].double().chunk(2, dim=1)
    for b in range(c["B"]):
        p = torch.arange(c["T"], device=DEV) if st["pos"] is None else st["pos"][b].long()
        out[b] = _exact_turn(st["x"][b], cos[p], -sin[p] if c["back"] else sin[p], c["inter"])
    return out


def _exact_append(st):
    """The turned queries, and the pages' scales by their rule; the codes are whole numbers."""
    c = st["case"]
    top, page = TOP[c["code"]], c["page"]
    cos, sin = st["table"].double().chunk(2, dim=1)
    q = st["q_out"].double()
    ks, vs = st["ks"].double(), st["vs"].double()
    for b, (L, n) in enumerate(zip(_lengths(c), _new(c))):
        p = torch.arange(L - n, L, device=DEV)
        q[b, :, :n] = _exact_turn(st["q"][b, :, :n], cos[p], sin[p], c["inter"])
        k = _exact_turn(st["k"][b, :, :n], cos[p], sin[p], c["inter"])
        for j in range((L - n) // page, (L - 1) // page + 1):
            rows = slice(max(0, j * page - (L - n)), (j + 1) * page - (L - n))
            for x, s in ((k, ks), (st["v"][b, :, :n].double(), vs)):
                a = x[:, rows].abs().amax(dim=(1, 2))
                no = int(st["pt"][b, j])
                if j * page < L - n:
                    doublings = torch.ceil(torch.log2(a / (s[no] * top))).clamp(min=0.0)
                    s[no] = s[no] * 2.0 ** doublings
                else:
                    s[no] = a / top
    return {"q": q, "kp": None, "vp": None, "ks": ks, "vs": vs}


def _exact_attend(st):
    """Head by head, from softmax's definition over the visible rows."""
    c = st["case"]
    d, G, page = c["d"], c["Hq"] // c["Hkv"], c["page"]
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device=DEV)

    def rows(pages, scales, b, h, L):
        no = st["pt"][b, :-(-L // page)].long()
        p = pages[no, h]
        p = p if c["code"] == "int8" else p.view(torch.float8_e4m3fn).float()
        return (p.double() * scales[no, h].double()[:, None, None]).reshape(-1, d)[:L]

    for b, (L, n) in enumerate(zip(_lengths(c), _new(c))):
        hide = torch.arange(L, device=DEV)[None] > (L - n + torch.arange(n, device=DEV))[:, None]
        for h in range(c["Hkv"]):
            k, v = rows(st["kp"], st["ks"], b, h, L), rows(st["vp"], st["vs"], b, h, L)
            for g in range(h * G, (h + 1) * G):
                s = st["q"][b, g, :n].double() @ k.T / math.sqrt(d)
                if c["causal"]:
                    s = s.masked_fill(hide, -math.inf)
                lse[b, g, :n] = torch.logsumexp(s, dim=1)
                o[b, g, :n] = torch.exp(s - lse[b, g, :n, None]) @ v
    return {"o": o, "lse": lse}


def exact(case, seed):
    st = _inputs(case, seed)
    return {"rotate": _exact_rotate, "append": _exact_append, "attend": _exact_attend}[case["op"]](st)
