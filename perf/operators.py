"""Speculative decoding on, and eviction from, the int8 KV cache: the four
operators' plain forms, the calls of the library that compute them, and the
cases they are measured at.

* ``tree``    attention of T drafted tokens (a tree, given by its ancestor
              masks) over a ragged int8 cache and over the drafts themselves
* ``commit``  the accepted path appended to the cache, its header updated
* ``weights`` the attention weight that each cached row has received
* ``evict``   the rows with the most weight gathered into a shorter cache
"""
import math

import numpy as np
import torch

own = False

LOG2E = 1.4426950408889634
#: device, and the most score elements a plain form holds at once
DEV = "cuda"
CHUNK = 1 << 28


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a chat reply on a short prompt: launch latency counts
        dict(name="tree_one_token", op="tree", B=1, Hq=32, Hkv=8, d=128, lo=4097, hi=4097, T=1),
        # a serving batch verifying four-token drafts at uneven prompt lengths
        dict(name="tree_chat_batch", op="tree", B=16, Hq=32, Hkv=8, d=128, lo=211, hi=4501, T=4),
        # a 64-node tree at long context, batch one
        dict(name="tree_64_long", op="tree", B=1, Hq=32, Hkv=8, d=128, lo=32768, hi=32768, T=64),
        # the largest: 26-node trees, ragged long contexts
        dict(name="tree_26_ragged", op="tree", B=8, Hq=32, Hkv=8, d=128, lo=5003, hi=32768, T=26),
        # a small model: one KV head per query head, d = 64
        dict(name="tree_d64_heads", op="tree", B=4, Hq=12, Hkv=12, d=64, lo=197, hi=2049, T=16),
        # weight received in one decode step over a long cache
        dict(name="weights_step", op="weights", B=1, Hq=32, Hkv=8, d=128, lo=32768, hi=32768, T=1,
             causal=False),
        # the last 32 prompt tokens as the window that votes on the prompt's rows
        dict(name="weights_window", op="weights", B=2, Hq=32, Hkv=8, d=128, lo=20011, hi=32001,
             T=32, causal=True),
        # the whole 8K prefill
        dict(name="weights_prefill", op="weights", B=1, Hq=32, Hkv=8, d=128, lo=8192, hi=8192,
             T=8192, causal=True),
        # a 32K prompt cut to 4K rows
        dict(name="evict_prompt", op="evict", B=1, Hkv=8, d=128, lo=32768, hi=32768, budget=4096,
             sink=4, recent=64),
        # steady state of a batch: each cache a little over its budget
        dict(name="evict_steady", op="evict", B=16, Hkv=8, d=64, lo=1801, hi=2305, budget=1999,
             sink=4, recent=128),
        # one sequence accepts a few of eight drafts
        dict(name="commit_one", op="commit", B=1, Hkv=8, d=128, lo=4097, hi=4097, T=8, accept=3),
        # a batch of 64-node trees, each with its own accepted path
        dict(name="commit_batch", op="commit", B=32, Hkv=8, d=128, lo=301, hi=2048, T=64, accept=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _time_floor(case):
    w = work(case)
    return w["bytes"] / 6.6e12 + w["flops"] / 1.9e15


def draw(rng):
    top = max(_time_floor(c) for c in listed())
    while True:
        op = rng.choice(["tree", "tree", "weights", "weights", "evict", "commit"])
        B = _log(rng, 1, 32)
        Hkv, G = rng.choice([(8, 4), (8, 4), (12, 1), (4, 8), (2, 3), (1, 16), (16, 2), (8, 1)])
        d = rng.choice([64, 128, 128])
        hi = _log(rng, 1, 32768)
        lo = _log(rng, 1, hi)
        case = dict(op=op, B=B, Hkv=Hkv, d=d, lo=lo, hi=hi)
        if op == "tree":
            case.update(Hq=Hkv * G, T=_log(rng, 1, 128))
        elif op == "weights":
            causal = rng.random() < 0.5
            case.update(Hq=Hkv * G, T=_log(rng, 1, hi if causal else min(hi, 512)), causal=causal)
        elif op == "evict":
            budget = _log(rng, 1, max(1, hi))
            sink = min(rng.choice([0, 1, 4]), budget)
            case.update(budget=budget, sink=sink, recent=min(rng.choice([0, 16, 100]), budget - sink))
        else:
            T = _log(rng, 1, 128)
            case.update(T=T, accept=rng.randint(1, min(T, 16)))
        if _time_floor(case) <= top:
            return case


def _lengths(case):
    """Rows in use per sequence: spread over [lo, hi], the last sequence at hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi - (hi - lo) * ((7 * (B - 1 - b)) % B) // max(B - 1, 1) for b in range(B)]


def _accepted(case):
    return [1 + (5 * b + case["accept"] - 1) % case["accept"] for b in range(case["B"])]


def _visible_pairs(case):
    """(query, row) pairs of one head, over the batch."""
    n = 0
    for L in _lengths(case):
        for_causal = case.get("causal", False)
        T = case["T"]
        if not for_causal:
            n += T * L
        else:  # query i sees rows 0 .. L - T + i
            first = max(0, T - L)  # the queries before see nothing
            k = T - first
            n += k * (L - T + first + 1) + k * (k - 1) // 2
    return n


def work(case):
    op, B, Hkv, d = case["op"], case["B"], case["Hkv"], case["d"]
    rows = sum(_lengths(case))
    if op == "tree":
        Hq, T = case["Hq"], case["T"]
        byts = (2 * rows * Hkv * d                   # K and V codes
                + B * Hq * T * (d + 4)               # query codes, scales
                + 2 * B * Hkv * T * d * 2            # the drafts' K and V
                + 3 * B * Hkv * d * 4                # header: scales and mean
                + B * T * 4 * ((T + 31) // 32) + 4 * B
                + B * Hq * T * (2 * d + 4))          # O, lse
        return {"bytes": byts, "flops": 4 * d * Hq * (_visible_pairs(case) + B * T)}
    if op == "weights":
        Hq, T = case["Hq"], case["T"]
        byts = rows * Hkv * (d + 8) + B * Hq * T * (d + 4) + 4 * B
        return {"bytes": byts, "flops": 2 * d * Hq * _visible_pairs(case)}
    if op == "evict":
        kept = sum(min(L, case["budget"]) for L in _lengths(case))
        byts = 4 * rows * Hkv + kept * Hkv * (4 * d + 8) + 4 * B * Hkv * d + 8 * B
        return {"bytes": byts, "flops": rows * Hkv}
    n = sum(_accepted(case))
    byts = n * Hkv * (6 * d + 4) + 6 * B * Hkv * d * 4 + 4 * n + 16 * B
    return {"bytes": byts, "flops": 8 * n * Hkv * d}


# -------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 + seed)
    return g


def _codes(g, *shape):
    """int8 codes shaped by N(0, 1) over +-4.5 sigma, as an int8 cache holds them."""
    out = torch.empty(shape, dtype=torch.int8, device=DEV)
    flat = out.view(shape[0], -1)
    for b in range(shape[0]):
        z = torch.randn(flat.shape[1], generator=g, device=DEV)
        flat[b] = (z * (127.0 / 4.5)).round().clamp(-127, 127).to(torch.int8)
    return out


def _quantize(x):
    """Symmetric int8 codes per (batch, head, 128 tokens), scale = amax / 127."""
    B, H, N, d = x.shape
    nb = (N + 127) // 128
    pad = torch.zeros(B, H, nb * 128, d, device=x.device)
    pad[:, :, :N] = x
    blk = pad.view(B, H, nb, 128, d)
    s = (blk.abs().amax(dim=(3, 4)) / 127.0).clamp_min(1e-20)
    codes = (blk / s[..., None, None]).round().clamp(-127, 127).to(torch.int8)
    return codes.view(B, H, nb * 128, d)[:, :, :N].contiguous(), s.contiguous()


def _header(g, B, Hkv, d):
    """Channel scales and K mean with the outlier channels of an LLM's keys."""
    sig = torch.rand(B, Hkv, d, generator=g, device=DEV) + 0.5
    mean = 0.5 * torch.randn(B, Hkv, d, generator=g, device=DEV)
    for i, c in enumerate((7, 35, 62)):
        sig[:, :, c] = 2.2 + 0.8 * i
        mean[:, :, c] = (-1.0) ** i * (54.0 + 60.0 * i)
    vsig = 0.8 + 0.4 * torch.rand(B, Hkv, d, generator=g, device=DEV)
    return dict(ks=sig * (4.5 / 127), vs=vsig * (4.5 / 127), mean=mean, sig=sig, vsig=vsig)


def _tree_masks(case, seed):
    """Ancestor masks of random trees: bit j of token i's words is set iff j is
    i or an ancestor of i."""
    B, T = case["B"], case["T"]
    W = (T + 31) // 32
    rng = np.random.default_rng(seed)
    words = np.zeros((B, T, W), dtype=np.uint32)
    for b in range(B):
        for j in range(T):
            p = int(rng.integers(max(-1, j - 9), j)) if j else -1  # -1: child of the last cached token
            if p >= 0:
                words[b, j] = words[b, p]
            words[b, j, j // 32] |= np.uint32(1 << (j % 32))
    return torch.from_numpy(words.view(np.int32)).to(DEV)


def _inputs(case, seed):
    g = _gen(seed)
    op, B, Hkv, d = case["op"], case["B"], case["Hkv"], case["d"]
    L = _lengths(case)
    st = dict(case=case, L=L, Lmax=max(L), lengths=torch.tensor(L, dtype=torch.int32, device=DEV))
    if op == "tree":
        Hq, T, cap = case["Hq"], case["T"], max(L) + 128
        st.update(_header(g, B, Hkv, d))
        q = 1.5 * torch.randn(B, Hq, T, d, generator=g, device=DEV)
        kfold = st["ks"].repeat_interleave(Hq // Hkv, dim=1)[:, :, None, :]
        st["qc"], st["qs"] = _quantize(q * kfold)
        st["kc"], st["vc"] = _codes(g, B, Hkv, cap, d), _codes(g, B, Hkv, cap, d)
        k = st["mean"][:, :, None] + torch.randn(B, Hkv, T, d, generator=g, device=DEV) * st["sig"][:, :, None]
        v = torch.randn(B, Hkv, T, d, generator=g, device=DEV) * st["vsig"][:, :, None]
        st["K"], st["V"] = k.to(torch.bfloat16), v.to(torch.bfloat16)
        st["mask"] = _tree_masks(case, seed)
        st["O"] = torch.empty(B, Hq, T, d, dtype=torch.bfloat16, device=DEV)
        st["lse"] = torch.empty(B, Hq, T, device=DEV)
    elif op == "weights":
        Hq, T, cap = case["Hq"], case["T"], max(L)
        q = 1.5 * torch.randn(B, Hq, T, d, generator=g, device=DEV)
        st["qc"], st["qs"] = _quantize(q)
        st["kc"] = _codes(g, B, Hkv, cap, d)
        nkb = (cap + 127) // 128
        st["ks"] = (0.9 + 0.2 * torch.rand(B, Hkv, nkb, generator=g, device=DEV)) * (4.5 / 127)
        st["base"] = torch.rand(B, Hkv, cap, generator=g, device=DEV)
        st["out"] = torch.zeros(B, Hkv, cap, device=DEV)
        st["lse"] = torch.empty(B, Hq, T, device=DEV)
        _attn_chunks(st, torch.float32, _lse_chunk)
    elif op == "evict":
        cap, bud = max(L), case["budget"]
        st["kc"], st["vc"] = _codes(g, B, Hkv, cap, d), _codes(g, B, Hkv, cap, d)
        # accumulated weights: heavy-tailed, and equal for rows nothing looked at
        w = torch.randn(B, Hkv, cap, generator=g, device=DEV).mul_(2.0).exp_()
        st["w"] = torch.where(w < 0.05, torch.zeros_like(w), w)
        st["ko"] = torch.zeros(B, Hkv, bud, d, dtype=torch.int8, device=DEV)
        st["vo"] = torch.zeros_like(st["ko"])
        st["wo"] = torch.zeros(B, Hkv, bud, device=DEV)
        st["kept"] = torch.zeros(B, Hkv, bud, dtype=torch.int32, device=DEV)
        st["lo"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        st["am"] = torch.zeros(B, Hkv, d, device=DEV)
    else:
        T, cap = case["T"], max(L) + 128
        st.update(_header(g, B, Hkv, d))
        st["kc"], st["vc"] = _codes(g, B, Hkv, cap, d), _codes(g, B, Hkv, cap, d)
        k = st["mean"][:, :, None] + torch.randn(B, Hkv, T, d, generator=g, device=DEV) * st["sig"][:, :, None]
        v = torch.randn(B, Hkv, T, d, generator=g, device=DEV) * st["vsig"][:, :, None]
        st["K"], st["V"] = k.to(torch.bfloat16), v.to(torch.bfloat16)
        st["amax"] = torch.full((B, Hkv, d), 100.0, device=DEV)
        st["w"] = torch.rand(B, Hkv, cap, generator=g, device=DEV)
        rng = np.random.default_rng(seed)
        path = np.zeros((B, T), dtype=np.int32)
        for b, n in enumerate(_accepted(case)):
            path[b, :n] = np.sort(rng.choice(T, n, replace=False))
        st["path"] = torch.from_numpy(path).to(DEV)
        st["n"] = torch.tensor(_accepted(case), dtype=torch.int32, device=DEV)
        st["lengths_out"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        st["mean_out"], st["amax_out"] = torch.zeros_like(st["mean"]), torch.zeros_like(st["amax"])
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from quantized_attention_gb300 import binding as qb
        op, B, Hkv, d = case["op"], case["B"], case["Hkv"], case["d"]
        if op in ("tree", "weights"):
            cap = st["kc"].shape[2]
            st["shape"] = qb.make_shape(B, case["Hq"], Hkv, case["T"], st["Lmax"], d)
            st["params"] = qb.make_params(causal=case.get("causal", False), out_dtype=qb.DT_BF16,
                                          kv_capacity=cap)
        if op == "tree":
            need = qb.tree_workspace_size(st["shape"], st["params"])
            st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return st


# --------------------------------------------------------------- plain forms
def _bits(mask, T):
    """[B, T, T] truth values of the ancestor words."""
    j = torch.arange(T, device=mask.device)
    return ((mask[:, :, j // 32] >> (j % 32).to(torch.int32)) & 1).bool()


def _draft_codes(st):
    """The drafts as the cache would hold them (fp32, one rounding a step)."""
    k = ((st["K"].float() - st["mean"][:, :, None]) / st["ks"][:, :, None]).round().clamp(-127, 127)
    v = (st["V"].float() / st["vs"][:, :, None]).round().clamp(-127, 127)
    return k, v


def _plain_tree(st):
    c = st["case"]
    B, Hq, Hkv, d, T = c["B"], c["Hq"], c["Hkv"], c["d"], c["T"]
    G, L = Hq // Hkv, st["Lmax"]
    dk, dv = _draft_codes(st)
    k = torch.cat([st["kc"][:, :, :L].float(), dk], dim=2)
    v = torch.cat([st["vc"][:, :, :L].float(), dv], dim=2) * st["vs"][:, :, None]
    q = st["qc"].float().view(B, Hkv, G * T, d)
    s = (q @ k.transpose(2, 3)).view(B, Hkv, G, T, L + T)
    s = s * (st["qs"].view(B, Hkv, G, 1, 1) * (1.0 / math.sqrt(d)))
    see = torch.zeros(B, T, L + T, dtype=torch.bool, device=s.device)
    see[:, :, :L] = (torch.arange(L, device=s.device)[None] < st["lengths"][:, None])[:, None]
    see[:, :, L:] = _bits(st["mask"], T)
    s.masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = (s - m).exp_()
    l = p.sum(dim=-1, keepdim=True)
    o = (p.view(B, Hkv, G * T, L + T) @ v).view(B, Hkv, G, T, d) / l
    lse = (m + l.log()).view(B, Hq, T)
    return {"O": o.view(B, Hq, T, d).to(torch.bfloat16), "lse": lse}


def _attn_chunks(st, dt, fn):
    """fn(st, b, h0, h1, s) on the masked scores s [h1 - h0, T, L] of query
    heads h0 .. h1 - 1 (of one KV head) of sequence b."""
    c = st["case"]
    B, Hq, Hkv, d, T = c["B"], c["Hq"], c["Hkv"], c["d"], c["T"]
    G = Hq // Hkv
    dev = st["qc"].device
    for b in range(B):
        L = st["L"][b]
        sk = st["ks"][b].to(dt).repeat_interleave(128, dim=1)[:, :L]
        sq = st["qs"][b].to(dt).repeat_interleave(128, dim=1)[:, :T]
        hide = None
        if c["causal"]:
            hide = (torch.arange(L, device=dev)[None] > (L - T + torch.arange(T, device=dev))[:, None])
        step = max(1, min(G, CHUNK // max(1, T * L)))
        for hk in range(Hkv):
            k = st["kc"][b, hk, :L].to(dt)
            for g0 in range(0, G, step):
                h0, h1 = hk * G + g0, hk * G + min(G, g0 + step)
                s = st["qc"][b, h0:h1].to(dt).view(-1, d) @ k.T
                s = s.view(h1 - h0, T, L)
                s *= sq[h0:h1, :, None] / math.sqrt(d)
                s *= sk[hk]
                if hide is not None:
                    s.masked_fill_(hide, -math.inf)
                fn(st, b, h0, h1, s)


def _lse_chunk(st, b, h0, h1, s):
    st["lse"][b, h0:h1] = torch.logsumexp(s, dim=-1)


def _plain_weights(st):
    c = st["case"]
    G = c["Hq"] // c["Hkv"]
    acc = st["base"].clone()

    def add(st, b, h0, h1, s):
        lse = st["lse"][b, h0:h1, :, None]
        s -= torch.where(lse == -math.inf, torch.zeros_like(lse), lse)
        acc[b, h0 // G, :s.shape[-1]] += s.exp_().sum(dim=(0, 1))

    _attn_chunks(st, torch.float32, add)
    out = st["out"]
    live = torch.arange(out.shape[2], device=out.device)[None] < st["lengths"][:, None]
    out.copy_(torch.where(live[:, None], acc, out))
    return out


def _plain_evict(st):
    c = st["case"]
    for b, L in enumerate(st["L"]):
        n = min(L, c["budget"])
        w = st["w"][b, :, :L]
        key = torch.where(torch.isnan(w), torch.full_like(w, -math.inf), w)
        key[:, :c["sink"]] = math.inf
        key[:, max(0, L - c["recent"]):] = math.inf
        order = key.sort(dim=1, descending=True, stable=True).indices[:, :n]
        rows = order.sort(dim=1).values
        st["kept"][b, :, :n] = rows.int()
        st["wo"][b, :, :n] = w.gather(1, rows)
        idx = rows[:, :, None].expand(-1, -1, c["d"])
        st["ko"][b, :, :n] = st["kc"][b].gather(1, idx)
        vk = st["vc"][b].gather(1, idx)
        st["vo"][b, :, :n] = vk
        st["am"][b] = vk.float().abs().amax(dim=1)
        st["lo"][b] = n
    return {k: st[k] for k in ("ko", "vo", "wo", "kept", "lo", "am")}


def _plain_commit(st):
    c = st["case"]
    B = c["B"]
    dev = st["K"].device
    bi = torch.arange(B, device=dev)
    mu, am = st["mean"].clone(), st["amax"].clone()
    for t in range(c["accept"]):
        live = (t < st["n"])[:, None, None]
        j = st["path"][:, t].long()
        row = st["lengths"].long() + t
        k, v = st["K"][bi, :, j].float(), st["V"][bi, :, j].float()
        diff = k - mu
        qk = (diff / st["ks"]).round().clamp(-127, 127)
        qv = (v / st["vs"]).round().clamp(-127, 127)
        mu = torch.where(live, mu + diff / (row + 1).float()[:, None, None], mu)
        am = torch.where(live, torch.maximum(am, qv.abs()), am)
        st["kc"][bi, :, row] = torch.where(live, qk.to(torch.int8), st["kc"][bi, :, row])
        st["vc"][bi, :, row] = torch.where(live, qv.to(torch.int8), st["vc"][bi, :, row])
        w = st["w"][bi, :, row]
        st["w"][bi, :, row] = torch.where(live[:, :, 0], torch.zeros_like(w), w)
    st["mean_out"].copy_(mu)
    st["amax_out"].copy_(am)
    st["lengths_out"].copy_(st["lengths"] + st["n"])
    return {k: st[k] for k in ("kc", "vc", "lengths_out", "mean_out", "amax_out", "w")}


# ----------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"tree": _plain_tree, "weights": _plain_weights, "evict": _plain_evict,
                "commit": _plain_commit}[op](state)
    from quantized_attention_gb300 import binding as qb
    s = state
    if op == "tree":
        qb.tree_decode(s["qc"], s["qs"], s["kc"], s["vc"], s["ks"], s["vs"], s["shape"], s["params"],
                       s["O"], s["lse"], s["ws"], lengths=s["lengths"], K_new=s["K"], V_new=s["V"],
                       k_mean=s["mean"], tree_mask=s["mask"])
        return {"O": s["O"], "lse": s["lse"]}
    if op == "weights":
        qb.kv_weights(s["qc"], s["qs"], s["kc"], s["ks"], s["lse"], s["shape"], s["params"], s["out"],
                      base=s["base"], lengths=s["lengths"])
        return s["out"]
    if op == "evict":
        c = s["case"]
        qb.kv_evict(s["kc"], s["vc"], s["w"], c["budget"], s["ko"], s["vo"], s["wo"], s["kept"], s["lo"],
                    s["am"], lengths=s["lengths"], n_sink=c["sink"], n_recent=c["recent"])
        return {k: s[k] for k in ("ko", "vo", "wo", "kept", "lo", "am")}
    qb.tree_commit(s["K"], s["V"], s["path"], s["n"], s["ks"], s["vs"], s["lengths"], s["mean"],
                   s["amax"], s["kc"], s["vc"], lengths_out=s["lengths_out"], k_mean_out=s["mean_out"],
                   v_code_amax_out=s["amax_out"], weights=s["w"])
    return {k: s[k] for k in ("kc", "vc", "lengths_out", "mean_out", "amax_out", "w")}


# ----------------------------------------------------------- in 64 bits
def _exact_tree(st):
    """Sequence by sequence, from softmax's definition over the visible rows."""
    c = st["case"]
    B, Hq, Hkv, d, T = c["B"], c["Hq"], c["Hkv"], c["d"], c["T"]
    G = Hq // Hkv
    O = torch.zeros(B, Hq, T, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    words = st["mask"].cpu().numpy().view(np.uint32)
    for b in range(B):
        L = st["L"][b]
        see = np.ones((T, L + T), dtype=bool)
        for i in range(T):
            for j in range(T):
                see[i, L + j] = bool((int(words[b, i, j // 32]) >> (j % 32)) & 1)
        see = torch.from_numpy(see).to(DEV)
        for h in range(Hkv):
            # the drafts' codes are defined by their fp32 steps
            nk = torch.clamp(torch.round((st["K"][b, h].float() - st["mean"][b, h]) / st["ks"][b, h]), -127, 127)
            nv = torch.clamp(torch.round(st["V"][b, h].float() / st["vs"][b, h]), -127, 127)
            k = torch.cat([st["kc"][b, h, :L].double(), nk.double()])
            v = torch.cat([st["vc"][b, h, :L].double(), nv.double()]) * st["vs"][b, h].double()
            for g in range(h * G, (h + 1) * G):
                scale = st["qs"][b, g, 0].double() / math.sqrt(d)
                s = torch.where(see, (st["qc"][b, g].double() @ k.T) * scale, -math.inf)
                top = s.max(dim=1, keepdim=True).values
                e = torch.exp(s - top)
                z = e.sum(dim=1, keepdim=True)
                O[b, g] = (e / z) @ v
                lse[b, g] = (top + torch.log(z))[:, 0]
    return {"O": O, "lse": lse}


def _exact_weights(st):
    c = st["case"]
    Hkv, T, d = c["Hkv"], c["T"], c["d"]
    G = c["Hq"] // Hkv
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        L = st["L"][b]
        row = torch.arange(L, device=DEV)
        for h in range(Hkv):
            total = st["base"][b, h, :L].double()
            k = st["kc"][b, h, :L].double() * st["ks"][b, h].double()[row // 128][:, None]
            for g in range(h * G, (h + 1) * G):
                for i0 in range(0, T, 2048):
                    i = torch.arange(i0, min(T, i0 + 2048), device=DEV)
                    q = st["qc"][b, g, i].double() * st["qs"][b, g].double()[i // 128][:, None]
                    x = torch.exp(q @ k.T / math.sqrt(d) - st["lse"][b, g, i].double()[:, None])
                    if c["causal"]:
                        x = x * (row[None] <= (L - T + i)[:, None])
                    # a query that sees nothing gives nothing
                    ok = st["lse"][b, g, i] > -math.inf
                    total += x[ok].sum(dim=0)
            out[b, h, :L] = total
    return out


def _exact_evict(st):
    """Keys and rows in NumPy: sorted by (protected, weight, -row)."""
    c = st["case"]
    out = {k: np.zeros(st[k].shape, dtype=np.float64) for k in ("ko", "vo", "wo", "kept", "lo", "am")}
    kc, vc, w = (st[k].cpu().numpy() for k in ("kc", "vc", "w"))
    for b, L in enumerate(st["L"]):
        n = min(L, c["budget"])
        out["lo"][b] = n
        for h in range(c["Hkv"]):
            r = np.arange(L)
            guard = (r < c["sink"]) | (r >= L - c["recent"])
            val = np.where(np.isnan(w[b, h, :L]), -np.inf, w[b, h, :L])
            sel = np.sort(np.lexsort((r, -val, ~guard))[:n])
            out["kept"][b, h, :n], out["wo"][b, h, :n] = sel, w[b, h, sel]
            out["ko"][b, h, :n], out["vo"][b, h, :n] = kc[b, h, sel], vc[b, h, sel]
            out["am"][b, h] = np.abs(vc[b, h, sel].astype(np.float64)).max(axis=0)
    return {k: torch.from_numpy(v) for k, v in out.items()}


def _exact_commit(st):
    """The running mean in 64 bits; codes, maxima and lengths are whole numbers."""
    c = st["case"]
    mean = st["mean"].double().cpu().numpy()
    K = st["K"].double().cpu().numpy()
    path = st["path"].cpu().numpy()
    for b, n in enumerate(_accepted(c)):
        for t in range(n):
            mean[b] += (K[b, :, path[b, t]] - mean[b]) / (st["L"][b] + t + 1)
    return {"kc": None, "vc": None, "lengths_out": None, "mean_out": torch.from_numpy(mean),
            "amax_out": None, "w": None}


def exact(case, seed):
    st = _inputs(case, seed)
    return {"tree": _exact_tree, "weights": _exact_weights, "evict": _exact_evict,
            "commit": _exact_commit}[case["op"]](st)
