"""GPU: the selection operators on sequences of more than 2048 blocks and on
tensors of more than 2**31 elements.

The long sequences are checked whole against the float64 oracle, under the
element-wise bounds of ``test_gpu_nsa_backward.py``.  Tensors whose last rows
lie past element 2**31 are drawn on the device, and rows and blocks at both
ends are computed anew in float64; the backward at the large shapes' bar
(max|gpu - ref| <= 2e-2 max|ref|), the cache's values within half a step of
e4m3 (2^-4 of the value, 2^-10 scales where it is subnormal) and the 2^-21 of
a rotation's fp32 roundings.
"""

import gc

import pytest
import torch

from block_sparse_attention_tra_gb300 import bsa
from oracle import cache as ocache
from test_gpu_nsa_backward import run
from test_gpu_nsa_cache import Pool, check_decode, freqs

pytestmark = pytest.mark.gpu
TOL = 2e-2


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_tra_gb300 import build

    build.build()
    bsa.load_library()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    assert bsa.device_error() == 0


@pytest.fixture(autouse=True)
def _release():
    yield
    gc.collect()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,D,bs", [(33024, 64, 16), (33024, 16, 16), (5248, 128, 64)])
def test_backward_of_many_blocks_and_chunks(T, D, bs):
    """More than 2048 blocks (16-token ones) and more than 32 chunks of 128 rows; a list as long as the sequence, rows
    that read nothing, and blocks that no row reads."""

    def change(idx):
        idx[:, :, :, 2] = 0
        idx[:, :, 700:900] = -1
        idx[idx == 40] = -1
        return idx

    dq, dk, dv = run(1, 2, 1, T, D, bs, 3, seed=D, change=change)
    assert not dq[:, :, 700:900].any() and dk[:, :, :bs].any() and dk[:, :, -bs:].any()
    assert not dk[:, :, 40 * bs:41 * bs].any() and not dv[:, :, 40 * bs:41 * bs].any()


def rel(got, ref):
    return float((got.double() - ref).abs().max() / ref.abs().max())


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (63, 9)])  # bulk copies, and cp.async for the other group sizes
def test_backward_past_2_31_elements(Hq, Hkv):
    T, D, bs, S, G = 271360, 128, 64, 2, Hq // Hkv
    g = torch.Generator(device="cuda").manual_seed(Hq)
    q, dout = (torch.randn((1, Hq, T, D), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.randn((1, Hkv, T, D), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    assert q.numel() > 2 ** 31
    own = (torch.arange(T, device="cuda") // bs).expand(1, Hkv, T)
    other = (torch.rand((1, Hkv, T), generator=g, device="cuda") * own).long()
    idx = torch.stack([own, other], -1).to(torch.int32)
    out, lse = bsa.nsa_select_forward(q, k, v, idx, bs, return_lse=True)
    dq, dk, dv = bsa.nsa_select_backward(q, k, v, idx, out, lse, dout, bs)
    torch.cuda.synchronize()
    c = D ** -0.5

    def pairs(h, i, tok):
        """p and dS [rows, G, tokens] of rows i of kv head h over tokens [rows, tokens]."""
        heads = slice(h * G, h * G + G)
        qi, di, oi = (t[0, heads, i].double().transpose(0, 1) for t in (q, dout, out))
        p = torch.exp(c * torch.einsum("igd,itd->igt", qi, k[0, h][tok].double())
                      - lse[0, heads, i].double().T[..., None])
        p = torch.where((tok <= i[:, None])[:, None], p, 0.0)
        dp = torch.einsum("igd,itd->igt", di, v[0, h][tok].double())
        return p, c * p * (dp - (di * oi).sum(-1)[..., None]), qi, di

    for h in (0, Hkv - 1):
        i = torch.tensor([0, 63, 64, 200, T // 2, T - 65, T - 1], device="cuda")
        tok = (idx[0, h, i].long()[..., None] * bs + torch.arange(bs, device="cuda")).flatten(1)
        tok[own[0, h, i] == other[0, h, i], bs:] = T  # a block listed twice is read once
        dead = tok == T
        _, ds, _, _ = pairs(h, i, torch.where(dead, T - 1, tok))
        ds = torch.where(dead[:, None], 0.0, ds)
        want = torch.einsum("igt,itd->gid", ds, k[0, h][tok.clamp_max(T - 1)].double())
        assert rel(dq[0, h * G:h * G + G, i], want) <= TOL
        for blk in (0, 1, T // bs // 2, T // bs - 1):
            i = (idx[0, h] == blk).any(-1).nonzero()[:, 0]
            tok = (blk * bs + torch.arange(bs, device="cuda")).expand(len(i), bs)
            p, ds, qi, di = pairs(h, i, tok)
            block = slice(blk * bs, blk * bs + bs)
            assert rel(dk[0, h, block], torch.einsum("igt,igd->td", ds, qi)) <= TOL
            assert rel(dv[0, h, block], torch.einsum("igt,igd->td", p, di)) <= TOL


def test_append_past_2_31_elements():
    """A prompt of more than 2**31 elements of k, v and q into pools of as many codes."""
    Hkv, n, D, page, held = 8, 2097152 + 37, 128, 64, 50
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v, q = (torch.randn((1, Hkv, n, D), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    pages = (held + n + page - 1) // page
    kc, vc = (torch.zeros((pages, Hkv, page, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, Hkv), 2.0 ** -9, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31 and kc.numel() > 2 ** 31
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    f = freqs(D)
    qr = bsa.nsa_cache_append(k, v, kc, vc, ks, vs, table, torch.tensor([held], device="cuda"), inv_freq=f, q=q)
    torch.cuda.synchronize()
    at = table[0].cpu()
    ends = {int(x) for x in at.argsort()[-3:]}  # the logical pages in the pools' last ones
    for lp in sorted({0, 1, pages // 2, pages - 2, pages - 1} | ends):
        t0, t1 = max(0, lp * page - held), min(n, (lp + 1) * page - held)
        slot, pid = t0 + held - lp * page, int(at[lp])
        pos = held + torch.arange(t0, t1).numpy()

        def turned(x):
            x = x[0, :, t0:t1].double().cpu().numpy()
            return torch.from_numpy(ocache.rotate(x, pos, f.double().cpu().numpy(), False))

        for want, codes, scale in ((turned(k), kc, ks), (v[0, :, t0:t1].double().cpu(), vc, vs)):
            s = scale[pid].double().cpu()[:, None, None]
            got = codes[pid, :, slot:slot + t1 - t0].view(torch.float8_e4m3fn).double().cpu() * s
            top = want.abs().amax((1, 2), keepdim=True)
            assert (top <= 448 * s * (1 + 2.0 ** -20)).all() and (top > 224 * s * (1 - 2.0 ** -20)).all()
            assert ((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * s + 2.0 ** -20 * top).all()
        want = turned(q)
        assert ((qr[0, :, t0:t1].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * 8).all()


@pytest.mark.parametrize("S", [0, 4])
@pytest.mark.parametrize("D,page,Hkv", [(128, 64, 5), (16, 16, 33)])
def test_decode_over_pools_past_2_32_bytes(D, page, Hkv, S):
    """Pages at both ends of pools of more than 2**32 codes."""
    B, Hq, per = 3, 2 * Hkv, 6
    used = Pool(B, Hkv, D, page, per, seed=D + S, spare=0).clean()
    pages = (1 << 32) // (Hkv * page * D) + 1000
    where = torch.randperm(used.pages, generator=torch.Generator().manual_seed(S))
    where = torch.where(where < used.pages // 2, where, pages - 1 - where).cuda()  # of each used page
    big = [torch.full((pages, Hkv, page, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, Hkv), float("nan"), device="cuda") for _ in range(2)]
    for b, x in zip((*big, *scales), (used.k, used.v, used.ks, used.vs)):
        b[where] = x
    assert big[0].numel() > 2 ** 32 and int(where.max()) == pages - 1 - used.pages // 2
    lens = [per * page, 3 * page + 5, 1]
    q = torch.randn((B, Hq, 1, D), generator=torch.Generator().manual_seed(D)).to(torch.bfloat16).cuda()
    idx = torch.tensor([0, 2, 5, 3], dtype=torch.int32, device="cuda").expand(B, Hkv, 1, S).contiguous() if S else None
    table = where[used.table.long()].to(torch.int32)
    out, lse = bsa.nsa_select_decode(q, *big, *scales, table, torch.tensor(lens, device="cuda"), block_idx=idx,
                                     return_lse=True)
    torch.cuda.synchronize()
    check_decode(out, lse, q, used, lens, idx)
