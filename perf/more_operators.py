"""What stands between a projection and the attention, and the 4-bit cache behind it: operators and measured cases.

* ``rows``      -- ``qk_norm_rope_forward``: the RMS norm of every query and key head and the rotation by position.
* ``rows_grad`` -- ``qk_norm_rope_backward``: its gradients, those of the norms' weights among them.
* ``append``    -- ``nsa_cache4_append`` and ``nsa_cache4_read``: new tokens into a paged cache of e2m1 codes with an
  e4m3 scale for every 16 elements, keys (and queries) normalised and rotated on the way, and the values they got.
* ``decode``    -- ``nsa_cache4_decode``: one query token per sequence over that cache, over the blocks that a selection
  lists or over every block.

``run`` computes them in plain torch operations, or with ``own`` through the package.
"""

import torch

own = False

EPS = 1e-6
GROUP = 16  # elements under one scale


def _rows(name, op, B, T, Hq, Hkv, D, rotary=None, interleaved=False, dtype="bf16", fused=False, norm=True, scale=1.0,
          first=0):
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D,
            "rotary": D if rotary is None else rotary, "interleaved": interleaved, "dtype": dtype, "fused": fused,
            "norm": norm, "scale": scale, "first": first}


def _append(name, B, n, Hq, Hkv, D, page, len_min, len_max, rotary=None, interleaved=False, dtype="bf16"):
    """rotary 0: keys that are normalised and rotated already, no queries."""
    return {"name": name, "op": "append", "B": B, "n": n, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
            "len_min": len_min, "len_max": len_max, "rotary": D if rotary is None else rotary,
            "interleaved": interleaved, "dtype": dtype}


def _decode(name, B, Hq, Hkv, D, page, S, len_min, len_max):
    return {"name": name, "op": "decode", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "S": S,
            "len_min": len_min, "len_max": len_max}


def listed():
    return [
        # one user's next token: the latency of a serving step
        _rows("rows_1_token", "rows", 1, 1, 32, 2, 128, fused=True, first=8191),
        # fp32, interleaved pairs, part of the head, odd length, frequencies of a stretched context
        _rows("rows_4x1031_f32", "rows", 4, 1031, 16, 2, 64, rotary=32, interleaved=True, dtype="f32", scale=1.1386),
        # the selection workload's sequences, read out of the fused projection
        _rows("rows_2x8192_d128", "rows", 2, 8192, 32, 2, 128, fused=True),
        # a short batch of odd heads and sizes
        _rows("rows_grad_3x257_d48", "rows_grad", 3, 257, 6, 3, 48, rotary=32, dtype="f32"),
        # a training step of the selection workload
        _rows("rows_grad_2x8192_d128", "rows_grad", 2, 8192, 32, 2, 128, fused=True),
        # one user's next token, normalised and rotated into a begun page
        _append("append_1_token", 1, 1, 32, 2, 128, 64, 4095, 4095),
        # a full batch's next tokens at ragged lengths
        _append("append_128_tokens", 128, 1, 64, 4, 128, 64, 1, 4096),
        # a long prompt whose attention has taken the rotated keys already
        _append("append_prompt_32768", 1, 32768, 64, 4, 128, 64, 0, 0, rotary=0),
        # one user, the selected blocks of a long context: latency
        _decode("decode_selected_1", 1, 32, 2, 128, 64, 16, 8191, 8191),
        # a full batch on the selected blocks of ragged contexts
        _decode("decode_selected_128", 128, 64, 4, 128, 64, 16, 700, 32768),
        # small heads and small pages, every block, odd lengths with an empty sequence
        _decode("decode_all_17_d64", 17, 24, 3, 64, 32, 0, 0, 5003),
        # four long ragged contexts, every block (a layer without selection)
        _decode("decode_all_4_long", 4, 32, 2, 128, 64, 0, 20011, 131072),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rows", "rows_grad", "append", "decode", "decode"])
    Hkv = rng.randint(1, 4)
    Hq = Hkv * rng.choice([1, 3, 4, 8, 16, 16])
    if op in ("rows", "rows_grad"):
        D = rng.choice([32, 48, 64, 80, 96, 128, 128])
        B = _spread(rng, 1, 32)
        T = _spread(rng, 1, 16384 // B)
        rotary = rng.choice([D, D, 16 * rng.randint(1, D // 16)])
        c = _rows("", op, B, T, Hq, min(Hkv, 2), D, rotary, rng.random() < 0.3, rng.choice(["bf16", "bf16", "f32"]),
                  rng.random() < 0.5, rng.random() < 0.8, rng.choice([1.0, 1.0, 1.2]), rng.choice([0, 0, 5000]))
        c["Hq"] = min(c["Hq"], 32)
        if c["dtype"] == "f32":
            c["T"] = max(1, T // 2)
        del c["name"]
        return c
    D = rng.choice([16, 32, 64, 128, 128])
    page = rng.choice([16, 32, 64, 64, 128])
    if op == "append":
        B = _spread(rng, 1, 128)
        lo = rng.randint(0, 200)
        hi = lo + _spread(rng, 1, 4000)
        if rng.random() < 0.5:  # a step: a token or a few
            c = _append("", B, rng.choice([1, 1, 1, 2, 5]), Hq, Hkv, D, page, lo, hi,
                        rng.choice([D, D, 16 * rng.randint(1, D // 16)]), rng.random() < 0.3,
                        rng.choice(["bf16", "bf16", "f32"]))
        else:
            c = _append("", B, _spread(rng, 2, max(2, 16384 // B)), Hq, Hkv, D, page, lo, hi, 0, False,
                        rng.choice(["bf16", "bf16", "f32"]))
    else:
        B = _spread(rng, 1, 128)
        S = rng.choice([0, rng.randint(1, 32)])
        hi = _spread(rng, 64, min(131072, 786432 // (B * Hkv)))
        c = _decode("", B, Hq, Hkv, D, page, S, rng.randint(0, hi // 2), hi)
    del c["name"]
    return c


def _lengths(case):
    """Cached lengths of the batch: evenly spread over [len_min, len_max], long and short ones mixed."""
    B, lo, hi = case["B"], case["len_min"], case["len_max"]
    step = next(s for s in (7, 11, 13, 1) if s == 1 or B % s)
    return [hi if B == 1 else lo + (hi - lo) * ((b * step) % B) // (B - 1) for b in range(B)]


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _channels(g, D):
    """Per-channel magnitudes of keys: mostly 1, a few strong ones, as in trained heads."""
    w = torch.ones(D, device="cuda")
    w[torch.randperm(D, generator=g, device="cuda")[: max(1, D // 32)]] = 6.0
    return w


def _frequencies(rotary, stretch=1.0):
    f = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / max(1, rotary))
    # a stretched context: the slow pairs turn slower, the fast ones as before
    slow = (f < 0.01).double()
    return (f * (1.0 - slow) + f * slow / (1.0 if stretch == 1.0 else 4.0)).float().cuda()


def _weights(g, D):
    return 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")


def _prepare_rows(case, g):
    B, T, Hq, Hkv, D = (case[x] for x in ("B", "T", "Hq", "Hkv", "D"))
    t = _type(case)
    if case["fused"]:  # [B, T, heads of q, k and v, D], as a projection leaves them
        x = (torch.randn((B, T, Hq + 2 * Hkv, D), generator=g, device="cuda") * 1.5).to(t).transpose(1, 2)
        q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    else:
        q, k = ((torch.randn((B, h, T, D), generator=g, device="cuda") * 1.5).to(t) for h in (Hq, Hkv))
    s = {"case": case, "q": q, "k": k, "wq": None, "wk": None,
         "inv_freq": _frequencies(case["rotary"], case["scale"]),
         "pos": None if not case["first"] else (
             torch.arange(T, device="cuda") + case["first"]).expand(B, T).to(torch.int32).contiguous()}
    if case["norm"]:
        s["wq"], s["wk"] = _weights(g, D), _weights(g, D)
    if case["op"] == "rows_grad":
        s["dq"], s["dk"] = (torch.randn((B, h, T, D), generator=g, device="cuda").to(t) for h in (Hq, Hkv))
    return s


def _encode(x):
    """Rows x [..., D] (32 bits) as (codes [..., D / 2], two to a byte, and scales [..., D / 16])."""
    grp = x.unflatten(-1, (-1, GROUP))
    scale = (grp.abs().amax(-1) / 6.0).clamp_max(448.0).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    y = torch.where(s > 0, grp / s, 0.0)
    a = y.abs()
    # the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; ties to the even code
    c = (a > 0.25).to(torch.uint8)
    for border, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (a >= border) if up else (a > border)
    c += (torch.signbit(x).unflatten(-1, (-1, GROUP))) * 8
    c = c.flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), scale


def _values(codes, scale):
    """What codes [..., D / 2] and scales [..., D / 16] stand for, in 32 bits."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    m = (c & 7).float()
    # 0, 0.5, then (1 + m / 2) 2^(e - 1) of two exponent bits and one of the mantissa
    v = torch.where(m < 2, m * 0.5, (1.0 + 0.5 * (m % 2)) * torch.exp2(torch.floor(m / 2) - 1.0))
    v = torch.where(c >= 8, -v, v)
    return (v.unflatten(-1, (-1, GROUP)) * scale.float()[..., None]).flatten(-2)


def _filled(g, pages, Hkv, page, D, channels):
    """A cache of `pages` pages whose every slot holds a value: what a running server's pool holds."""
    codes = torch.empty((pages, Hkv, page, D // 2), dtype=torch.uint8, device="cuda")
    scale = torch.empty((pages, Hkv, page, D // GROUP), dtype=torch.float8_e4m3fn, device="cuda")
    step = max(1, (1 << 27) // (Hkv * page * D))
    for i in range(0, pages, step):
        x = torch.randn((min(step, pages - i), Hkv, page, D), generator=g, device="cuda") * channels
        codes[i:i + step], s = _encode(x)
        scale.view(torch.uint8)[i:i + step] = s.view(torch.uint8)
    return codes, scale


def _table(g, B, per_seq):
    """A page table that scatters the sequences' pages over the pool."""
    return torch.randperm(B * per_seq, generator=g, device="cuda").view(B, per_seq).to(torch.int32)


def _prepare_append(case, g):
    B, n, Hq, Hkv, D, page = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "page"))
    t, r = _type(case), case["rotary"]
    lens = _lengths(case)
    per_seq = max((x + n - 1) // page for x in lens) + 2
    ch = _channels(g, D)
    kc, ks = _filled(g, B * per_seq, Hkv, page, D, ch)
    vc, vs = _filled(g, B * per_seq, Hkv, page, D, torch.ones_like(ch))
    s = {"case": case, "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs, "table": _table(g, B, per_seq),
         "k": (torch.randn((B, Hkv, n, D), generator=g, device="cuda") * ch).to(t),
         "v": torch.randn((B, Hkv, n, D), generator=g, device="cuda").to(t),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "q": None, "wq": None, "wk": None,
         "inv_freq": None}
    s["lens_after"] = s["lens"] + n
    if r:
        s["q"] = torch.randn((B, Hq, n, D), generator=g, device="cuda").to(t)
        s["wq"], s["wk"] = _weights(g, D), _weights(g, D)
        s["inv_freq"] = _frequencies(r)
    return s


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


def prepare(case, seed):
    g = _generator(seed)
    return {"rows": _prepare_rows, "rows_grad": _prepare_rows, "append": _prepare_append,
            "decode": _prepare_decode}[case["op"]](case, g)


def _angles(pos, inv_freq):
    """Cosines and sines [B, 1, n, r / 2] (32 bits) at positions [B, n]; angles in 64 bits."""
    a = (pos.double()[..., None] * inv_freq.double())[:, None]
    return torch.cos(a).float(), torch.sin(a).float()


def _turn(x, c, s, interleaved):
    """Rotates the first 2 * c.shape[-1] of x [B, H, n, D] (32 bits)."""
    r = 2 * c.shape[-1]
    if interleaved:
        x0, x1 = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([x0 * c - x1 * s, x0 * s + x1 * c], -1).flatten(-2)
    else:
        x0, x1 = x[..., : r // 2], x[..., r // 2: r]
        y = torch.cat([x0 * c - x1 * s, x0 * s + x1 * c], -1)
    return torch.cat([y, x[..., r:]], -1)


def _norm(x, w):
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _positions(s):
    case = s["case"]
    return torch.arange(case["T"], device="cuda").expand(case["B"], -1) if s["pos"] is None else s["pos"]


def _rows_plain(s):
    case = s["case"]
    c, w = (x * case["scale"] for x in _angles(_positions(s), s["inv_freq"]))
    return {n: _turn(_norm(s[n].float(), s["w" + n]), c, w, case["interleaved"]).to(s[n].dtype) for n in ("q", "k")}


def _rows_grad_plain(s):
    case = s["case"]
    c, w = (x * case["scale"] for x in _angles(_positions(s), s["inv_freq"]))
    got = {}
    for n in ("q", "k"):
        dn = _turn(s["d" + n].float(), c, -w, case["interleaved"])
        if s["w" + n] is None:
            got["d" + n] = dn.to(s[n].dtype)
            continue
        x = s[n].float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        x = x * r
        got["dw" + n] = (dn * x).sum((0, 1, 2))
        dn = dn * s["w" + n]
        got["d" + n] = (r * (dn - x * (dn * x).mean(-1, keepdim=True))).to(s[n].dtype)
    return got


def _append_plain(s):
    case = s["case"]
    n, page = case["n"], case["page"]
    pos = s["lens"].long()[:, None] + torch.arange(n, device="cuda")
    page_id = s["table"].long().gather(1, pos // page)[:, None]
    at = (page_id, torch.arange(case["Hkv"], device="cuda")[:, None], (pos % page)[:, None])
    c, w = _angles(pos, s["inv_freq"]) if case["rotary"] else (None, None)
    out = {}
    for name in ("k", "v"):
        x = s[name].float()
        if name == "k" and case["rotary"]:
            x = _turn(_norm(x, s["wk"]), c, w, case["interleaved"])
        codes, scale = _encode(x)
        s[name + "_cache"][at] = codes
        s[name + "_scale"].view(torch.uint8)[at] = scale.view(torch.uint8)
        back = _values(s[name + "_cache"][at], s[name + "_scale"].view(torch.uint8)[at].view(torch.float8_e4m3fn))
        out[name] = back.to(torch.bfloat16)
    if case["rotary"]:
        out["q"] = _turn(_norm(s["q"].float(), s["wq"]), c, w, case["interleaved"]).to(s["q"].dtype)
    return out


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
    k, v = (_values(s[x + "_cache"][phys, head], s[x + "_scale"].view(torch.uint8)[phys, head].view(
        torch.float8_e4m3fn)).flatten(2, 3) for x in ("k", "v"))
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


def run(state):
    s, case = state, state["case"]
    if own:
        import block_sparse_attention_tra_gb300 as bsa
    if case["op"] == "rows":
        if own:
            q, k = bsa.qk_norm_rope_forward(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], positions=s["pos"],
                                            interleaved=case["interleaved"], rotary_scale=case["scale"], eps=EPS)
            return {"q": q, "k": k}
        return _rows_plain(s)
    if case["op"] == "rows_grad":
        if own:
            dq, dk, dwq, dwk = bsa.qk_norm_rope_backward(
                s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], s["inv_freq"], positions=s["pos"],
                interleaved=case["interleaved"], rotary_scale=case["scale"], eps=EPS)
            return {"dq": dq, "dk": dk} | ({"dwq": dwq, "dwk": dwk} if case["norm"] else {})
        return _rows_grad_plain(s)
    if case["op"] == "append":
        if own:
            cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"])
            q = bsa.nsa_cache4_append(s["k"], s["v"], *cache, s["lens"], inv_freq=s["inv_freq"],
                                      interleaved=case["interleaved"], q=s["q"], q_weight=s["wq"], k_weight=s["wk"],
                                      eps=EPS)
            k, v = bsa.nsa_cache4_read(*cache, s["lens_after"], case["n"], starts=s["lens"])
            return {"k": k, "v": v} | ({"q": q} if case["rotary"] else {})
        return _append_plain(s)
    if own:
        out, lse = bsa.nsa_cache4_decode(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                         s["lens"], block_idx=s["idx"], return_lse=True)
    else:
        out, lse = _decode_plain(s)
    return {"out": out, "lse": lse}


def _selected_tokens(length, page, S):
    """Tokens that a query at position length - 1 reads through S slots of _select."""
    if length <= 0:
        return 0
    c = (length - 1) // page
    return length - c * page + page * min(S - 1, c)


def work(case):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] in ("rows", "rows_grad"):
        el, n = 2 if case["dtype"] == "bf16" else 4, B * case["T"] * (Hq + Hkv) * D
        side = (8 * D if case["norm"] else 0) + 2 * case["rotary"] + (4 * B * case["T"] if case["first"] else 0)
        turn = 3 * B * case["T"] * (Hq + Hkv) * case["rotary"]
        if case["op"] == "rows":
            return {"bytes": 2 * el * n + side, "flops": turn + (4 * n if case["norm"] else 0)}
        if not case["norm"]:
            return {"bytes": 2 * el * n + side, "flops": turn}
        return {"bytes": 3 * el * n + side + 8 * D, "flops": turn + 12 * n}
    if case["op"] == "append":
        n, el = case["n"], 2 if case["dtype"] == "bf16" else 4
        new = B * Hkv * n * D
        q = B * Hq * n * D if case["rotary"] else 0
        # new rows read, their codes written and read back, their values written
        return {"bytes": 2 * new * (el + 2 * 0.5625 + 2) + 2 * el * q + 4 * B * (n + 1),
                "flops": 3 * B * (Hq + Hkv) * n * case["rotary"] + 6 * new + (4 * (q + new) if q else 0)}
    S = case["S"]
    tokens = sum(x if not S else _selected_tokens(x, case["page"], S) for x in _lengths(case))
    pages = tokens / case["page"] * 4 * (Hkv if S else 1)
    return {"bytes": 2 * Hkv * tokens * D * 0.5625 + pages + 4 * B * Hq * D + 4 * B * Hq,
            "flops": 4 * Hq * tokens * D}


# ---- the definitions in 64 bits

def _turned64(x, pos, inv_freq, interleaved, factor):
    """x [B, H, n, D] in 64 bits with its first pairs turned, as complex numbers."""
    inv = inv_freq.double()
    i = torch.arange(inv.numel(), device="cuda")
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + inv.numel())
    angle = pos.double()[:, None, :, None] * inv
    z = torch.polar(torch.full_like(angle, factor), angle) * torch.complex(x[..., first], x[..., second])
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _normed64(x, w):
    return x if w is None else torch.einsum("bhtd,bht,d->bhtd", x, (torch.linalg.vector_norm(x, dim=-1).square()
                                                                    / x.shape[-1] + EPS) ** -0.5, w.double())


def _exact_rows(case, s):
    pos = _positions(s)
    return {n: _turned64(_normed64(s[n].double(), s["w" + n]), pos, s["inv_freq"], case["interleaved"], case["scale"])
            for n in ("q", "k")}


def _exact_rows_grad(case, s):
    """By autograd through the 64-bit forward, a batch at a time."""
    pos, out = _positions(s), {}
    for n in ("q", "k"):
        w = None if s["w" + n] is None else s["w" + n].double().requires_grad_()
        parts, dw = [], 0.0
        for b in range(case["B"]):
            x = s[n][b:b + 1].double().requires_grad_()
            y = x
            if w is not None:
                y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
            inv = s["inv_freq"].double()
            angle = pos[b:b + 1].double()[:, None, :, None] * inv
            i = torch.arange(inv.numel(), device="cuda")
            first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + inv.numel())
            z = torch.polar(torch.full_like(angle, case["scale"]), angle) * torch.complex(y[..., first], y[..., second])
            dy = s["d" + n][b:b + 1].double()
            loss = (z.real * dy[..., first]).sum() + (z.imag * dy[..., second]).sum()
            r = 2 * inv.numel()
            loss = loss + (y[..., r:] * dy[..., r:]).sum()
            grads = torch.autograd.grad(loss, [x] if w is None else [x, w])
            parts.append(grads[0])
            if w is not None:
                dw = dw + grads[1]
        out["d" + n] = torch.cat(parts)
        if w is not None:
            out["dw" + n] = dw
    return out


def _e4m3_table():
    v = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")


def _nearest(x, table):
    """Index of the nearest of the ascending table for x >= 0, ties to the even index."""
    x = x.clamp_max(table[-1].item())
    hi = torch.searchsorted(table, x.contiguous()).clamp_max(table.numel() - 1)
    lo = (hi - 1).clamp_min(0)
    a, b = x - table[lo], table[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def _held64(x):
    """What the cache holds of rows x [..., D]: 64-bit values."""
    e4, e2 = _e4m3_table(), torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    parts = x.unflatten(-1, (-1, GROUP))
    scale = e4[_nearest(parts.abs().max(-1).values / 6.0, e4)][..., None]
    code = e2[_nearest(torch.nan_to_num(parts.abs() / scale, 0.0, 6.0), e2)]
    return (torch.sign(parts) * code * scale).flatten(-2)


def _exact_append(case, s):
    pos = s["lens"].double()[:, None] + torch.arange(case["n"], device="cuda")
    out = {}
    k = s["k"].double()
    if case["rotary"]:
        k = _turned64(_normed64(k, s["wk"]), pos, s["inv_freq"], case["interleaved"], 1.0)
        out["q"] = _turned64(_normed64(s["q"].double(), s["wq"]), pos, s["inv_freq"], case["interleaved"], 1.0)
    return out | {"k": _held64(k), "v": _held64(s["v"].double())}


def _exact_decode(case, s):
    B, Hq, Hkv, D, page = (case[x] for x in ("B", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    e2 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    e2 = torch.cat([e2, -e2])
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
            kv = []
            for name in ("k", "v"):
                byte = s[name + "_cache"][at, h].flatten(0, 1)[use].long()
                code = torch.empty((byte.shape[0], D), dtype=torch.float64, device="cuda")
                code[:, 0::2], code[:, 1::2] = e2[byte % 16], e2[byte // 16]
                scale = s[name + "_scale"].view(torch.uint8)[at, h].view(torch.float8_e4m3fn).double().flatten(0, 1)[use]
                kv.append(code * scale.repeat_interleave(GROUP, -1))
            x = s["q"][b, h * G:h * G + G, 0].double() @ kv[0].T / D ** 0.5
            lse[b, h * G:h * G + G, 0] = torch.logsumexp(x, -1)
            out[b, h * G:h * G + G, 0] = torch.softmax(x, -1) @ kv[1]
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rows": _exact_rows, "rows_grad": _exact_rows_grad, "append": _exact_append,
            "decode": _exact_decode}[case["op"]](case, s)
