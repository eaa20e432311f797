"""The selection attention's training and serving operators, and the cases they are measured at.

Three operators around ``nsa_select_forward``:

* ``append``   -- ``nsa_cache_append``: the keys and values of new tokens, keys (and queries) rotated by position, into
  a paged cache of e4m3 codes with one power-of-two scale for each page and head.
* ``decode``   -- ``nsa_select_decode``: one query token per sequence over that cache, either over the blocks that a
  selection lists or over every block of the sequence.
* ``backward`` -- ``nsa_select_backward``: dq, dk and dv of the selection attention, the probabilities recomputed from
  the forward's log-sum-exp.

``run`` computes them in plain torch operations, or with ``own`` through the package.
"""

import torch

own = False

E_MIN = -96  # exponent of the smallest page scale, 2^-96


def _append(name, B, n, Hq, Hkv, D, page, len_min, len_max, dtype="bf16", rotary=None, interleaved=False):
    return {"name": name, "op": "append", "B": B, "n": n, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
            "len_min": len_min, "len_max": len_max, "dtype": dtype, "rotary": D if rotary is None else rotary,
            "interleaved": interleaved}


def _decode(name, B, Hq, Hkv, D, page, S, len_min, len_max):
    return {"name": name, "op": "decode", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "S": S,
            "len_min": len_min, "len_max": len_max}


def _backward(name, B, Hq, Hkv, T, D, block, S, pad=0):
    return {"name": name, "op": "backward", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "D": D, "block": block, "S": S,
            "pad": pad}


def listed():
    return [
        # one user's next token, its page begun: the latency of a serving step
        _append("append_1_token", 1, 1, 32, 2, 128, 64, 4095, 4095),
        # a full batch's next tokens at ragged lengths
        _append("append_128_tokens", 128, 1, 64, 4, 128, 64, 1, 4096),
        # fp32 activations, interleaved pairs, part of the head rotated, chunked prompts that end inside pages
        _append("append_4_chunks_f32", 4, 1031, 16, 2, 64, 32, 5, 777, dtype="f32", rotary=32, interleaved=True),
        # a long prompt into an empty cache
        _append("append_prompt_32768", 1, 32768, 64, 4, 128, 64, 0, 0),
        # one user, the selected blocks of a long context: latency
        _decode("decode_selected_1", 1, 32, 2, 128, 64, 16, 8191, 8191),
        # a full batch on the selected blocks of ragged contexts
        _decode("decode_selected_128", 128, 64, 4, 128, 64, 16, 700, 32768),
        # small heads and small pages, every block, odd lengths with an empty sequence
        _decode("decode_all_17_d64", 17, 24, 3, 64, 32, 0, 0, 5003),
        # four long ragged contexts, every block (a layer without selection)
        _decode("decode_all_4_long", 4, 32, 2, 128, 64, 0, 20011, 131072),
        # a short sequence of a small model
        _backward("backward_256_d32", 1, 8, 2, 256, 32, 32, 4),
        # 64-wide heads in groups of four, a padded tail
        _backward("backward_4096_d64", 1, 16, 4, 4096, 64, 64, 16, pad=100),
        # a training step's sequence at the head layout of the selection workloads
        _backward("backward_4096_d128", 1, 32, 2, 4096, 128, 64, 16),
        # the selection workload itself
        _backward("backward_8192_d128", 2, 32, 2, 8192, 128, 64, 16),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "decode", "backward"])
    D = rng.choice([32, 64, 128, 128])
    page = rng.choice([16, 32, 64, 64, 128])
    Hkv = rng.randint(1, 4)
    Hq = Hkv * rng.choice([1, 3, 4, 8, 16, 16])
    if op == "append":
        B = _spread(rng, 1, 128)
        n = 1 if rng.random() < 0.4 else _spread(rng, 2, max(2, 16384 // B))
        lo = rng.randint(0, 200)
        c = _append("", B, n, Hq, Hkv, D, page, lo, lo + _spread(rng, 1, 4000), rng.choice(["bf16", "bf16", "f32"]),
                    rng.choice([D, D // 2]), rng.random() < 0.3)
    elif op == "decode":
        B = _spread(rng, 1, 128)
        S = rng.choice([0, rng.randint(1, 32)])
        hi = _spread(rng, 64, 131072 if B <= 4 else 262144 // B)
        c = _decode("", B, Hq, Hkv, D, page, S, rng.randint(0, hi // 2), hi)
    else:
        blocks = _spread(rng, 2, 2560 // page)
        c = _backward("", rng.randint(1, 2), Hq, Hkv, blocks * page, D, page, rng.randint(1, 24),
                      pad=rng.choice([0, rng.randint(1, page)]))
    del c["name"]
    return c


def _lengths(case):
    """Cached lengths of the batch: evenly spread over [len_min, len_max], long and short ones mixed."""
    B, lo, hi = case["B"], case["len_min"], case["len_max"]
    step = next(s for s in (7, 11, 13, 1) if s == 1 or B % s)
    return [hi if B == 1 else lo + (hi - lo) * ((b * step) % B) // (B - 1) for b in range(B)]


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _channels(g, D):
    """Per-channel magnitudes of keys: mostly 1, a few strong ones, as in trained heads."""
    w = torch.ones(D, device="cuda")
    w[torch.randperm(D, generator=g, device="cuda")[: max(1, D // 32)]] = 6.0
    return w


def _scale_exponent(amax):
    """The least e >= E_MIN with amax <= 448 * 2^e (448 = 0.875 * 2^9 is the largest e4m3 value)."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp_min(E_MIN)


def _table(g, B, per_seq):
    """A page table that scatters the sequences' pages over the pool."""
    return torch.randperm(B * per_seq, generator=g, device="cuda").view(B, per_seq).to(torch.int32)


def _filled(g, pages, Hkv, page, D, channels):
    """A cache of `pages` pages whose every slot holds a value, and its scales: what a running server's pool holds."""
    x = torch.randn((pages, Hkv, page, D), generator=g, device="cuda") * channels
    e = _scale_exponent(x.abs().amax((-1, -2)))
    scale = torch.exp2(e.float())
    return (x / scale[..., None, None]).to(torch.float8_e4m3fn), scale


def _prepare_append(case, g):
    B, n, Hq, Hkv, D, page = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "page"))
    t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    lens = _lengths(case)
    per_seq = max((x + n - 1) // page for x in lens) + 2
    ch = _channels(g, D)
    kc, ks = _filled(g, B * per_seq, Hkv, page, D, ch)
    vc, vs = _filled(g, B * per_seq, Hkv, page, D, torch.ones_like(ch))
    r = case["rotary"]
    return {
        "case": case,
        "q": torch.randn((B, Hq, n, D), generator=g, device="cuda").to(t),
        "k": (torch.randn((B, Hkv, n, D), generator=g, device="cuda") * ch).to(t),
        "v": torch.randn((B, Hkv, n, D), generator=g, device="cuda").to(t),
        "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs,
        "table": _table(g, B, per_seq),
        "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
        "inv_freq": (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda(),
    }


def _select(g, current, n_blk, S):
    """Selected blocks [..., S] of rows whose current block is `current` [...]: the current block, block 0, then distinct
    earlier blocks, -1 behind them."""
    blk = torch.arange(n_blk, device="cuda")
    u = torch.rand((*current.shape, n_blk), generator=g, device="cuda")
    u = torch.where(blk == 0, -1.0, u)  # block 0 comes first
    u = torch.where(blk < current[..., None], u, 2.0)
    u = torch.where(blk == current[..., None], -2.0, u)  # behind the current block only
    val, pick = torch.topk(u, min(S, n_blk), dim=-1, largest=False)
    pick = torch.where(val < 2.0, pick, -1)
    out = torch.full((*current.shape, S), -1, dtype=torch.int32, device="cuda")
    out[..., : pick.shape[-1]] = pick.to(torch.int32)
    return out


def _prepare_decode(case, g):
    B, Hq, Hkv, D, page, S = (case[x] for x in ("B", "Hq", "Hkv", "D", "page", "S"))
    lens = _lengths(case)
    per_seq = max(1, max(-(-x // page) for x in lens))
    ch = _channels(g, D)
    kc, ks = _filled(g, B * per_seq, Hkv, page, D, ch)
    vc, vs = _filled(g, B * per_seq, Hkv, page, D, torch.ones_like(ch))
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    idx = None
    if S:
        current = ((lens - 1).clamp_min(0) // page)[:, None].expand(B, Hkv)
        idx = _select(g, current, per_seq, S)[:, :, None, :].contiguous()
    return {
        "case": case,
        "q": (torch.randn((B, Hq, 1, D), generator=g, device="cuda") / ch.square()).to(torch.bfloat16),
        "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs, "table": _table(g, B, per_seq), "lens": lens,
        "idx": idx,
    }


def _prepare_backward(case, g):
    B, Hq, Hkv, T, D, bs, S = (case[x] for x in ("B", "Hq", "Hkv", "T", "D", "block", "S"))
    G = Hq // Hkv
    bf = torch.bfloat16
    q, dout = (torch.randn((B, Hq, T, D), generator=g, device="cuda").to(bf) for _ in range(2))
    k, v = (torch.randn((B, Hkv, T, D), generator=g, device="cuda").to(bf) for _ in range(2))
    current = (torch.arange(T, device="cuda") // bs).expand(B, Hkv, T)
    idx = _select(g, current, T // bs, S)
    if case["pad"]:  # the padded tail of the first sequence selects nothing
        idx[0, :, T - case["pad"]:] = -1
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, T), device="cuda")
    for b in range(B):  # the forward's results, a key head at a time
        for h in range(Hkv):
            heads = slice(h * G, h * G + G)
            m = _mask(idx[b:b + 1, h:h + 1], T, bs)[0, 0]
            s = (q[b, heads].float() @ k[b, h].float().T * D ** -0.5).masked_fill_(~m, -torch.inf)
            some = m.any(-1)
            lse[b, heads] = torch.where(some, s.logsumexp(-1), -1.0e9)
            p = s.softmax(-1).masked_fill_(~m, 0.0)
            out[b, heads] = (p @ v[b, h].float()).to(bf)
            del s, p
    return {"case": case, "q": q, "k": k, "v": v, "idx": idx, "out": out, "lse": lse, "dout": dout}


def prepare(case, seed):
    g = _generator(seed)
    return {"append": _prepare_append, "decode": _prepare_decode, "backward": _prepare_backward}[case["op"]](case, g)


def _rotate(x, pos, inv_freq, interleaved):
    """Rotates the first 2 * len(inv_freq) of x [B, H, n, D] (32 bits) by pos [B, n]; angles in 64 bits."""
    r = 2 * inv_freq.numel()
    a = (pos.double()[..., None] * inv_freq.double())[:, None]
    c, s = torch.cos(a).float(), torch.sin(a).float()
    if interleaved:
        x0, x1 = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([x0 * c - x1 * s, x0 * s + x1 * c], -1).flatten(-2)
    else:
        x0, x1 = x[..., : r // 2], x[..., r // 2: r]
        y = torch.cat([x0 * c - x1 * s, x0 * s + x1 * c], -1)
    return torch.cat([y, x[..., r:]], -1)


def _store(x, cache, scale, phys, lens, page):
    """Writes x [B, H, n, D] (32 bits) behind `lens` cached tokens into the pages `phys` [B, P] that it touches."""
    B, H, n, D = x.shape
    P = phys.shape[1]
    off = lens.long() % page  # tokens the first page holds already
    at = off[:, None] + torch.arange(n, device=x.device)
    new = torch.zeros((B, P * page, H, D), device=x.device)
    new[torch.arange(B, device=x.device)[:, None], at] = x.transpose(1, 2)
    new = new.view(B, P, page, H, D).transpose(2, 3)
    row = torch.arange(P * page, device=x.device).view(P, page)
    kept = row < off[:, None, None]
    ours = ~kept & (row < off[:, None, None] + n)
    touched = ours.any(-1)[..., None]
    e = _scale_exponent(new.abs().amax((-1, -2)))
    old = scale[phys]
    e_old = torch.frexp(old)[1] - 1
    e = torch.where(kept.any(-1)[..., None], torch.maximum(e, e_old), e)
    got = cache.view(torch.uint8)[phys]
    moved = got.view(torch.float8_e4m3fn).float() * torch.exp2((e_old - e).float())[..., None, None]
    codes = torch.where(ours[:, :, None, :, None], new * torch.exp2(-e.float())[..., None, None], moved)
    codes = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    change = (touched[..., None, None] & (kept | ours)[:, :, None, :, None])
    cache.view(torch.uint8)[phys] = torch.where(change, codes, got)
    scale[phys] = torch.where(touched, torch.exp2(e.float()), old)


def _append_plain(s):
    case = s["case"]
    n, page = case["n"], case["page"]
    pos = s["lens"].long()[:, None] + torch.arange(n, device="cuda")
    P = (n + page - 2) // page + 1
    phys = s["table"].gather(1, s["lens"].long()[:, None] // page + torch.arange(P, device="cuda")).long()
    _store(_rotate(s["k"].float(), pos, s["inv_freq"], case["interleaved"]), s["k_cache"], s["k_scale"], phys,
           s["lens"], page)
    _store(s["v"].float(), s["v_cache"], s["v_scale"], phys, s["lens"], page)
    return _rotate(s["q"].float(), pos, s["inv_freq"], case["interleaved"]).to(s["q"].dtype)


def _decode_plain(s):
    case = s["case"]
    B, Hq, Hkv, D, page = (case[x] for x in ("B", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    table, lens, idx = s["table"].long(), s["lens"].long(), s["idx"]
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    if idx is None:
        blk = torch.arange(table.shape[1], device="cuda").expand(B, Hkv, -1)
    else:
        blk = idx[:, :, 0].long()
        again = (blk[..., :, None] == blk[..., None, :]).tril(-1).any(-1)  # a block counts once
        blk = torch.where(again, -1, blk)
    phys = table[:, None, :].expand(B, Hkv, -1).gather(2, blk.clamp_min(0))
    k = s["k_cache"].view(torch.uint8)[phys, head].view(torch.float8_e4m3fn).float()
    v = s["v_cache"].view(torch.uint8)[phys, head].view(torch.float8_e4m3fn).float()
    k = (k * s["k_scale"][phys, head][..., None, None]).flatten(2, 3)
    v = (v * s["v_scale"][phys, head][..., None, None]).flatten(2, 3)
    tok = (blk[..., None] * page + torch.arange(page, device="cuda"))
    live = ((blk[..., None] >= 0) & (tok < lens[:, None, None, None])).flatten(2)[:, :, None]
    sc = (s["q"].float().view(B, Hkv, G, D) @ k.transpose(-1, -2) * D ** -0.5).masked_fill(~live, -torch.inf)
    m = sc.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(sc - m)
    total = p.sum(-1, keepdim=True)
    some = total > 0
    out = torch.where(some, (p @ v) / total, 0.0)
    lse = torch.where(some, m + torch.log(total), -1.0e9)
    return out.view(B, Hq, 1, D).to(torch.bfloat16), lse.view(B, Hq, 1)


def _mask(idx, T, bs):
    """[B, Hkv, T, T]: whether query i reads key j under the index rows idx [B, Hkv, T, S]."""
    sel = torch.zeros((*idx.shape[:3], T // bs + 1), dtype=torch.bool, device=idx.device)
    sel.scatter_(-1, torch.where(idx >= 0, idx, T // bs).long(), True)
    return sel[..., :-1].repeat_interleave(bs, -1).tril_()


def _backward_plain(s):
    case = s["case"]
    B, Hq, Hkv, T, D, bs = (case[x] for x in ("B", "Hq", "Hkv", "T", "D", "block"))
    G, scale = Hq // Hkv, D ** -0.5
    hidden = ~_mask(s["idx"], T, bs)[:, :, None]
    q, do = (s[x].float().view(B, Hkv, G * T, D) for x in ("q", "dout"))
    k, v = s["k"].float(), s["v"].float()
    delta = (s["dout"].float() * s["out"].float()).sum(-1)
    p = (q @ k.transpose(-1, -2)).view(B, Hkv, G, T, T)
    p.mul_(scale).sub_(s["lse"].view(B, Hkv, G, T, 1)).exp_().masked_fill_(hidden, 0.0)
    dv = p.view(B, Hkv, G * T, T).transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).view(B, Hkv, G, T, T)
    ds = ds.sub_(delta.view(B, Hkv, G, T, 1)).mul_(p).mul_(scale).view(B, Hkv, G * T, T)
    del p
    dq = ds @ k
    dk = ds.transpose(-1, -2) @ q
    return tuple(x.to(torch.bfloat16) for x in (dq.view(B, Hq, T, D), dk, dv))


def run(state):
    s, case = state, state["case"]
    if own:
        import block_sparse_attention_tra_gb300 as bsa
    if case["op"] == "append":
        if own:
            q = bsa.nsa_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                     s["lens"], inv_freq=s["inv_freq"], interleaved=case["interleaved"], q=s["q"])
        else:
            q = _append_plain(s)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"],
                "v_scale": s["v_scale"]}
    if case["op"] == "decode":
        if own:
            out, lse = bsa.nsa_select_decode(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                             s["lens"], block_idx=s["idx"], return_lse=True)
        else:
            out, lse = _decode_plain(s)
        return {"out": out, "lse": lse}
    if own:
        dq, dk, dv = bsa.nsa_select_backward(s["q"], s["k"], s["v"], s["idx"], s["out"], s["lse"], s["dout"],
                                             case["block"])
    else:
        dq, dk, dv = _backward_plain(s)
    return {"dq": dq, "dk": dk, "dv": dv}


def _selected_tokens(length, page, S):
    """Tokens that a query at position length - 1 reads through S slots of _select."""
    if length <= 0:
        return 0
    c = (length - 1) // page
    return length - c * page + page * min(S - 1, c)


def work(case):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        n, el = case["n"], 2 if case["dtype"] == "bf16" else 4
        new = B * Hkv * n * D
        pages = sum((x + n - 1) // case["page"] - x // case["page"] + 1 for x in _lengths(case))
        return {"bytes": 2 * new * (el + 1) + 2 * el * B * Hq * n * D + pages * (2 * 4 * Hkv + 4) + 4 * B,
                "flops": 3 * B * (Hq + Hkv) * n * case["rotary"] + 4 * new}
    if case["op"] == "decode":
        S = case["S"]
        tokens = sum(x if not S else _selected_tokens(x, case["page"], S) for x in _lengths(case))
        pages = tokens / case["page"] * (2 * 4 * Hkv + 4 * (Hkv if S else 1))
        return {"bytes": 2 * Hkv * tokens * D + pages + 4 * B * Hq * D + 4 * B * Hq, "flops": 4 * Hq * tokens * D}
    T, bs, S = case["T"], case["block"], case["S"]
    pairs = B * sum(_selected_tokens(i + 1, bs, S) for i in range(T))
    pairs -= sum(_selected_tokens(i + 1, bs, S) for i in range(T - case["pad"], T))
    return {"bytes": 2 * D * T * B * (4 * Hq + 4 * Hkv) + 4 * T * B * (Hq + Hkv * S), "flops": 10 * D * Hq * pairs}


def _exact_append(case, s):
    """In 64 bits and not rounded to codes: every value that the cache ends up holding, over its page's scale."""
    n, page, H = case["n"], case["page"], case["Hkv"]
    inv = s["inv_freq"].double()
    r = 2 * inv.numel()
    i = torch.arange(r // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
    turned = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        angle = (s["lens"].double()[:, None] + torch.arange(n, device="cuda").double())[:, None, :, None] * inv
        z = torch.polar(torch.ones_like(angle), angle) * torch.complex(x[..., first], x[..., second])
        y[..., first], y[..., second] = z.real, z.imag
        turned[name] = y
    got = {"q": turned["q"]}
    for name, x in (("k", turned["k"]), ("v", s["v"].double())):
        cache, scale = s[name + "_cache"].to(torch.float64), s[name + "_scale"].double()
        for b, held in enumerate(s["lens"].tolist()):
            for p in range(held // page, (held + n - 1) // page + 1):
                page_id = int(s["table"][b, p])
                t0, t1 = max(0, p * page - held), min(n, (p + 1) * page - held)
                r0 = held + t0 - p * page
                most = x[b, :, t0:t1].abs().amax((-1, -2))
                least = torch.ceil(torch.log2(most / 448)).clamp_min(E_MIN)
                was = torch.log2(scale[page_id])
                if r0:
                    least = torch.maximum(least, was)
                    cache[page_id, :, :r0] *= torch.exp2(was - least)[:, None, None]
                cache[page_id, :, r0:r0 + t1 - t0] = x[b, :, t0:t1] * torch.exp2(-least)[:, None, None]
                scale[page_id] = torch.exp2(least)
        got[name + "_cache"], got[name + "_scale"] = cache, scale
    return got


def _exact_decode(case, s):
    B, Hq, Hkv, D, page = (case[x] for x in ("B", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    out = torch.zeros((B, Hq, 1, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, 1), -1.0e9, dtype=torch.float64, device="cuda")
    lens, table = s["lens"].tolist(), s["table"].cpu()
    picks = None if s["idx"] is None else s["idx"][:, :, 0].cpu()
    for b in range(B):
        for h in range(Hkv):
            blocks = range(-(-lens[b] // page)) if picks is None else sorted({int(j) for j in picks[b, h] if j >= 0})
            rows = [j for j in blocks if j * page < lens[b]]
            if not rows:
                continue
            at = table[b, rows].long().cuda()
            tok = (torch.tensor(rows, device="cuda")[:, None] * page + torch.arange(page, device="cuda")).flatten()
            use = tok < lens[b]
            k = (s["k_cache"].view(torch.uint8)[at, h].view(torch.float8_e4m3fn).double()
                 * s["k_scale"][at, h].double()[:, None, None]).flatten(0, 1)[use]
            v = (s["v_cache"].view(torch.uint8)[at, h].view(torch.float8_e4m3fn).double()
                 * s["v_scale"][at, h].double()[:, None, None]).flatten(0, 1)[use]
            x = s["q"][b, h * G:h * G + G, 0].double() @ k.T / D ** 0.5
            lse[b, h * G:h * G + G, 0] = torch.logsumexp(x, -1)
            out[b, h * G:h * G + G, 0] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}


def _exact_backward(case, s):
    """Query by query over the gathered keys of its set, in 64 bits."""
    B, Hq, Hkv, T, D, bs, S = (case[x] for x in ("B", "Hq", "Hkv", "T", "D", "block", "S"))
    G = Hq // Hkv
    dq = torch.zeros((B, Hq, T, D), dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros((B, Hkv, T, D), dtype=torch.float64, device="cuda") for _ in range(2))
    step = max(1, (1 << 28) // (S * bs * max(D, G)) // 4)
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * G, h * G + G)
            k, v = s["k"][b, h].double(), s["v"][b, h].double()
            for i0 in range(0, T, step):
                i = torch.arange(i0, min(T, i0 + step), device="cuda")
                tok = (s["idx"][b, h, i].long()[..., None] * bs + torch.arange(bs, device="cuda")).flatten(1)
                use = (tok >= 0) & (tok <= i[:, None])
                tok = tok.clamp_min(0)
                kk, vv = k[tok], v[tok]
                q, do, o = (s[x][b, heads, i].double().transpose(0, 1) for x in ("q", "dout", "out"))
                x = torch.einsum("igd,itd->igt", q, kk) / D ** 0.5 - s["lse"][b, heads, i].double().T[..., None]
                p = torch.where(use[:, None], torch.exp(x), 0.0)
                g = torch.einsum("igd,itd->igt", do, vv) - (do * o).sum(-1)[..., None]
                ds = torch.where(use[:, None], p * g, 0.0) / D ** 0.5
                dq[b, heads, i] = torch.einsum("igt,itd->gid", ds, kk)
                dk[b, h].index_add_(0, tok.flatten(), torch.einsum("igt,igd->itd", ds, q).flatten(0, 1))
                dv[b, h].index_add_(0, tok.flatten(), torch.einsum("igt,igd->itd", p, do).flatten(0, 1))
    return {"dq": dq, "dk": dk, "dv": dv}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "backward": _exact_backward}[case["op"]](case, s)
