"""The operators of the paged 4-bit KV cache, their cases, plain forms and exact values.

The cache holds keys and values as e2m1 codes (two per byte, the even channel in the low half) with
one e4m3 scale per 16 consecutive channels, in pages of 16 to 128 positions; a value is
code * scale * k_scale (or v_scale).  Three operators work on it:

  append  rotates queries and keys by their positions, quantises keys and values and writes them into
          the sequences' pages (optionally the means of the touched blocks of keys)
  attn    attention of a block's queries over the whole cache and the block's own bf16 keys
  gather  rows of the cache at given positions as bf16 (the sparse pool, or staged candidates)

`own` False: elementary torch operations in fp32.  `own` True: the framework's kernels.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a small layer: nothing but latency
        dict(name="attn token tiny", op="attn", N=1, Hq=4, Hkv=1, d=64, B=1, ctx=2048, ragged=False,
             page=16, block=True),
        # single-token serving of a ragged batch, one sequence still empty
        dict(name="attn token batch", op="attn", N=64, Hq=32, Hkv=8, d=128, B=1, ctx=8192,
             ragged=True, page=64, block=True),
        # single-token serving of one long context (split over the whole GPU)
        dict(name="attn token 128k", op="attn", N=1, Hq=32, Hkv=8, d=128, B=1, ctx=131071,
             ragged=False, page=128, block=True),
        # a handful of drafted tokens, keys already in the cache
        dict(name="attn draft", op="attn", N=7, Hq=28, Hkv=4, d=128, B=5, ctx=12001, ragged=True,
             page=32, block=False),
        # a denoising step with full attention on the 32K layer
        dict(name="attn block 32k", op="attn", N=1, Hq=28, Hkv=4, d=128, B=32, ctx=32768,
             ragged=False, page=64, block=True),
        # the same on the 4 x 64K layer: the largest call
        dict(name="attn block 4x64k", op="attn", N=4, Hq=32, Hkv=8, d=128, B=32, ctx=65536,
             ragged=False, page=128, block=True),
        # one new token of every sequence of a serving batch
        dict(name="append token batch", op="append", N=64, Hq=32, Hkv=8, d=128, T=1, ctx=63,
             ragged=True, page=16, rot=128, interleaved=False, pooled=0, fused=True),
        # a decoded block joins the cache and the block means stage 1 scans
        dict(name="append block", op="append", N=1, Hq=28, Hkv=4, d=128, T=32, ctx=4077,
             ragged=False, page=64, rot=128, interleaved=False, pooled=64, fused=False),
        # prompts of a padded batch
        dict(name="append prompts", op="append", N=4, Hq=32, Hkv=8, d=128, T=4096, ctx=0,
             ragged=True, page=64, rot=128, interleaved=True, pooled=0, fused=True),
        # the selected rows of the 32K layer into the sparse pool
        dict(name="gather pool 32k", op="gather", N=1, Hq=28, Hkv=4, d=128, ctx=32768, ragged=False,
             page=64, rows=1344, values=True),
        # stage 2's candidate keys of the 4 x 64K layer
        dict(name="gather candidates 4x64k", op="gather", N=4, Hq=32, Hkv=8, d=128, ctx=65536,
             ragged=False, page=128, rows=4096, values=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attn", "attn", "append", "gather"))
    d = rng.choice((64, 128, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    G = rng.choice((1, 2, 4, 7, 8))
    c = dict(op=op, Hq=Hkv * G, Hkv=Hkv, d=d, ragged=rng.random() < 0.6,
             page=rng.choice((16, 32, 64, 128)))
    if op == "attn":
        c["B"] = 1 if rng.random() < 0.4 else _log(rng, 1, min(64, 256 // G))
        c["ctx"] = _log(rng, 1, 131072)
        c["N"] = _log(rng, 1, max(1, min(64, (1 << 21) // (Hkv * c["ctx"]))))
        c["block"] = rng.random() < 0.7
    elif op == "append":
        c["T"] = _log(rng, 1, 4096)
        c["N"] = _log(rng, 1, max(1, min(64, (1 << 14) // c["T"])))
        c["ctx"] = rng.randrange(0, 300)
        c["rot"] = rng.choice((0, 32, 64, d))
        c["interleaved"] = rng.random() < 0.5
        c["pooled"] = rng.choice((0, 32, 64)) if c["T"] <= 64 else 0
        c["fused"] = rng.random() < 0.5
    else:
        c["ctx"] = _log(rng, 16, 131072)
        c["N"] = _log(rng, 1, max(1, min(16, (1 << 21) // (Hkv * c["ctx"]))))
        c["rows"] = _log(rng, 1, min(4096, c["ctx"]))
        c["values"] = rng.random() < 0.5
    return c


def _lengths(case, top, salt):
    """Lengths of the sequences: all `top`, or ragged between none and `top`, one of them `top`."""
    n = case["N"]
    if not case["ragged"]:
        return [top] * n
    r = random.Random("%s %d %d" % (salt, n, top))
    got = [r.randrange(0, top + 1) for _ in range(n)]
    got[r.randrange(n)] = top
    if n > 2:
        got[(got.index(top) + 1) % n] = 0
    return got


def work(case):
    n, hq, hkv, d = case["N"], case["Hq"], case["Hkv"], case["d"]
    row = d // 2 + d // 16  # bytes of one held row
    if case["op"] == "attn":
        keys, b = sum(_lengths(case, case["ctx"], "ctx")), case["B"]
        own_keys = n * b if case["block"] else 0
        return {"bytes": 2 * hkv * keys * row + 4 * n * b * hq * d + 4 * own_keys * hkv * d,
                "flops": 4 * hq * b * d * (keys + own_keys)}
    if case["op"] == "append":
        toks = sum(_lengths(case, case["T"], "tok"))
        table = 4 * case["rot"] * toks if case["rot"] else 0
        means = 0
        if case["pooled"]:
            means = n * hkv * d * 4 * (-(-case["T"] // case["pooled"]))
        return {"bytes": toks * (2 * (hq + 2 * hkv) * d + 2 * (hq + hkv) * d + 2 * hkv * row) + table + means,
                "flops": toks * d * (3 * hq + 10 * hkv)}
    rows = n * hkv * case["rows"]
    return {"bytes": rows * (4 + (2 if case["values"] else 1) * (row + 2 * d)), "flops": 0}


# ------------------------------------------------------- the cache's format

def _quantise(x, scale):
    """x [..., d] fp32 -> (codes [..., d/2] uint8, scales [..., d/16] e4m3 as uint8), one IEEE fp32
    operation at a time.  `scale`: a tensor of one fp32 (a tensor, so that divisions divide)."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    s = (g.abs().amax(-1) / (6.0 * scale)).clamp(max=448.0).to(torch.float8_e4m3fn)
    full = (s.float() * scale).unsqueeze(-1)
    y = torch.where(full == 0, torch.zeros_like(g), g / full)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).reshape(x.shape)
    return code[..., 0::2] + 16 * code[..., 1::2], s.view(torch.uint8)


def _held(codes, scales, scale, lut):
    """codes [..., d/2], scales [..., d/16] (uint8) -> fp32 values [..., d]."""
    v = lut[codes.long()].reshape(*codes.shape[:-1], codes.shape[-1] * 2 // 16, 16)
    s = scales.view(torch.float8_e4m3fn).float()
    return (v * s.unsqueeze(-1) * scale).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _pair_table(dev):
    """[256][2] fp32: the two values of a byte of codes."""
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=dev)
    b = torch.arange(256, device=dev)
    return torch.stack((v[b & 15], v[b >> 4]), 1)


def _paged(x, table):
    """The pages [n_pages, Hkv, page, w] of every sequence in order: [N, Hkv, max_pages*page, w]
    (entries without a page read page 0)."""
    g = x[table.clamp(min=0).long()]  # [N, max_pages, Hkv, page, w]
    return g.permute(0, 2, 1, 3, 4).reshape(g.shape[0], g.shape[2], -1, g.shape[4])


# ------------------------------------------------------------------ inputs

def _pool(case, lengths, gen, dev):
    """A paged cache with room for `lengths`, its pages in random order.  Where no row is held it has
    arbitrary bytes (NaN scales among them); zeros for the append, whose pages are outputs."""
    n, hkv, d, page = case["N"], case["Hkv"], case["d"], case["page"]
    need = [-(-x // page) for x in lengths]
    max_pages, used = max(1, max(need)), sum(need)
    n_pages = used + 3
    order = torch.randperm(n_pages, generator=gen, device=dev)[:used].to(torch.int32)
    want = torch.arange(max_pages, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
    table = torch.full((n, max_pages), -1, dtype=torch.int32, device=dev)
    table[want] = order
    codes = torch.randint(0, 256, (2, n_pages, hkv, page, d // 2), generator=gen, device=dev,
                          dtype=torch.uint8)
    scales = torch.randint(0, 256, (2, n_pages, hkv, page, d // 16), generator=gen, device=dev,
                           dtype=torch.uint8)
    if case["op"] == "append":
        codes.zero_()
        scales.zero_()
    return dict(table=table, codes=codes, scales=scales, page=page, max_pages=max_pages, want=want,
                lengths=torch.tensor(lengths, device=dev), k_scale=1.0, v_scale=0.25)


def _fill(c, case, topic, gen, dev):
    """Every row below the lengths holds quantised keys and values: normal keys with a hundredth of
    them near the queries' common direction, smaller values."""
    hkv, d, page = case["Hkv"], case["d"], case["page"]
    n, mp = c["table"].shape
    held = (torch.arange(mp * page, device=dev) < c["lengths"][:, None]).reshape(n, mp, 1, page, 1)
    held, at = held[c["want"]], c["table"][c["want"]].long()
    for kv in (0, 1):
        x = torch.randn((n, hkv, mp * page, d), generator=gen, device=dev)
        if kv == 0:
            hot = torch.rand((n, hkv, mp * page, 1), generator=gen, device=dev) < 0.01
            x += torch.where(hot, 2.0 * topic[None, :, None], torch.zeros((), device=dev))
        else:
            x *= 0.5
        x = x.bfloat16().float()
        scale = torch.tensor([c["k_scale"], c["v_scale"]][kv], device=dev)
        for part, to in zip(_quantise(x, scale), (c["codes"], c["scales"])):
            part = part.reshape(n, hkv, mp, page, -1).permute(0, 2, 1, 3, 4)
            to[kv][at] = torch.where(held, part[c["want"]], to[kv][at])


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(int(seed))
    n, hq, hkv, d = case["N"], case["Hq"], case["Hkv"], case["d"]
    topic = torch.randn((hkv, d), generator=gen, device=dev)
    s = dict(case=case, lut=_pair_table(dev))

    def queries(rows):
        x = torch.randn((n, rows, hkv, hq // hkv, d), generator=gen, device=dev)
        return (0.7 * topic[:, None] + 0.7 * x).reshape(n, rows, hq, d).bfloat16()

    if case["op"] == "append":
        toks = _lengths(case, case["T"], "tok")
        ctx = _lengths(case, case["ctx"], "ctx")
        s["L_max"] = case["ctx"] + case["T"]
        c = _pool(case, [x + case["T"] for x in ctx], gen, dev)
        _fill(c, case, topic, gen, dev)
        T = case["T"]
        s["n_tok"] = torch.tensor(toks, dtype=torch.int32, device=dev)
        k = torch.randn((n, T, hkv, d), generator=gen, device=dev).bfloat16()
        v = (0.5 * torch.randn((n, T, hkv, d), generator=gen, device=dev)).bfloat16()
        q = queries(T)
        if case["fused"]:  # views of one projection's output
            qkv = torch.cat((q, k, v), 2).contiguous()
            q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        s.update(q=q, k=k, v=v, q_rot=torch.zeros((n, T, hq, d), dtype=torch.bfloat16, device=dev),
                 k_rot=torch.zeros((n, T, hkv, d), dtype=torch.bfloat16, device=dev))
        if case["rot"]:
            inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"])
            a = torch.arange(s["L_max"], dtype=torch.float64, device=dev)[:, None] * inv
            s["cos_sin"] = torch.stack((a.cos(), a.sin()), -1).float().contiguous()
        if case["pooled"]:
            blocks = -(-s["L_max"] // case["pooled"])
            s["pooled"] = torch.zeros((n, hkv, blocks, d), device=dev)
    else:
        ctx = _lengths(case, case["ctx"], "ctx")
        s["L_max"] = max(1, case["ctx"])
        c = _pool(case, ctx, gen, dev)
        _fill(c, case, topic, gen, dev)
        if case["op"] == "attn":
            s["q"] = queries(case["B"])
            s["out"] = torch.zeros_like(s["q"])
            if case["block"]:
                s["bk"] = torch.randn((n, case["B"], hkv, d), generator=gen, device=dev).bfloat16()
                s["bv"] = (0.5 * torch.randn((n, case["B"], hkv, d), generator=gen, device=dev)).bfloat16()
        else:
            P = case["rows"]
            idx = torch.full((n, hkv, P), -1, dtype=torch.int32, device=dev)
            n_sel = torch.zeros((n, hkv), dtype=torch.int32, device=dev)
            for i, L in enumerate(ctx):  # ascending, distinct, fewer where the context is short
                m = min(P, L)
                if m:
                    r = torch.rand((hkv, L), generator=gen, device=dev).topk(m, -1).indices
                    idx[i, :, :m] = r.sort(-1).values.to(torch.int32)
                    n_sel[i] = m
            s.update(idx=idx, n_sel=n_sel,
                     pool_k=torch.zeros((n, hkv, P, d), dtype=torch.bfloat16, device=dev))
            s["pool_v"] = torch.zeros_like(s["pool_k"]) if case["values"] else None
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    s["cache"] = c
    if own:  # what a program keeps between calls: the argument structs and the workspace
        from block_diffusion_sparse_gb300 import herald as H
        s["dims"] = H.dims(n, hq, hkv, d, case.get("B", 1), s["L_max"])
        s["kv4"] = H.kv4(c["page"], c["table"], c["codes"][0], c["scales"][0], c["codes"][1],
                         c["scales"][1], c["k_scale"], c["v_scale"])
        if case["op"] == "attn":
            s["ws"] = torch.zeros(H.herald_workspace_size_kv4(s["dims"]), dtype=torch.uint8, device=dev)
        if "cos_sin" in s:
            s["rope"] = H.rope(s["cos_sin"], case["rot"], case["interleaved"])
    return s


# ------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        from block_diffusion_sparse_gb300 import herald as H
        st = torch.cuda.current_stream()
        if op == "attn":
            H.herald_kv4_attn(s["dims"], s["q"], s["kv4"], s["ctx"], s.get("bk"), s.get("bv"),
                              s["out"], ws=s["ws"], stream=st)
            return s["out"]
        if op == "gather":
            H.herald_kv4_gather(s["dims"], s["idx"], s["n_sel"], s["case"]["rows"], s["kv4"],
                                s["pool_k"], s["pool_v"], stream=st)
            return [s["pool_k"], s["pool_v"]]
        H.herald_kv4_append(s["dims"], s["case"]["T"], s["q"], s["k"], s["v"], s["ctx"], s["kv4"],
                            s["q_rot"], s["k_rot"], rope=s.get("rope"), n_tok=s["n_tok"],
                            pooled=s.get("pooled"), Bk=s["case"]["pooled"], stream=st)
        return _appended(s)
    if op == "attn":
        return _attn(s)
    if op == "gather":
        return _gather(s)
    _append(s)
    return _appended(s)


def _appended(s):
    """The append's outputs, the held codes and scales as the numbers they stand for."""
    c = s["cache"]
    values = s["lut"].index_select(0, c["codes"].view(-1).int())
    return [s["q_rot"], s["k_rot"], values, c["scales"].view(torch.float8_e4m3fn), s.get("pooled")]


def _attn(s):
    case, c = s["case"], s["cache"]
    n, hq, hkv, d, b = case["N"], case["Hq"], case["Hkv"], case["d"], case["B"]
    k = _held(_paged(c["codes"][0], c["table"]), _paged(c["scales"][0], c["table"]), c["k_scale"], s["lut"])
    v = _held(_paged(c["codes"][1], c["table"]), _paged(c["scales"][1], c["table"]), c["v_scale"], s["lut"])
    seen = torch.arange(k.shape[2], device=k.device)[None] < s["ctx"][:, None]
    if "bk" in s:
        k = torch.cat((k, s["bk"].float().transpose(1, 2)), 2)
        v = torch.cat((v, s["bv"].float().transpose(1, 2)), 2)
        seen = torch.cat((seen, seen.new_ones((n, b))), 1)
    seen = seen[:, None, None]
    v = torch.where(seen.transpose(2, 3), v, torch.zeros((), device=v.device))
    q = s["q"].float().reshape(n, b, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, d)
    x = q @ k.transpose(2, 3) * (1.0 / math.sqrt(d))
    x = torch.where(seen, x, torch.full((), -math.inf, device=x.device))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = e.sum(-1, keepdim=True)
    o = e @ v / torch.where(total == 0, torch.ones_like(total), total)
    o = o.reshape(n, hkv, b, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, b, hq, d)
    return o.bfloat16()


def _gather(s):
    case, c = s["case"], s["cache"]
    pos = s["idx"].long().clamp(min=0)
    page = torch.gather(c["table"].long()[:, None].expand(-1, case["Hkv"], -1), 2, pos // c["page"])
    page = page.clamp(min=0)
    head = torch.arange(case["Hkv"], device=pos.device)[None, :, None]
    used = torch.arange(case["rows"], device=pos.device) < s["n_sel"][..., None]
    got = []
    for kv in range(2 if case["values"] else 1):
        x = _held(c["codes"][kv][page, head, pos % c["page"]], c["scales"][kv][page, head, pos % c["page"]],
                  (c["k_scale"], c["v_scale"])[kv], s["lut"])
        got.append(torch.where(used[..., None], x, torch.zeros((), device=x.device)).bfloat16())
    return got + [None] * (2 - len(got))


def _rotated(x, cos, sin, case):
    """x [N, T, H, d] fp32, cos and sin [N, T, 1, rot/2]."""
    r = case["rot"]
    if not r:
        return x
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
    u, w = a * cos - b * sin, b * cos + a * sin
    front = torch.stack((u, w), -1).flatten(-2) if case["interleaved"] else torch.cat((u, w), -1)
    return torch.cat((front, x[..., r:]), -1)


def _append(s):
    case, c = s["case"], s["cache"]
    n, hkv, d, T = case["N"], case["Hkv"], case["d"], case["T"]
    dev = s["ctx"].device
    t = torch.arange(T, device=dev)
    pos = s["ctx"].long()[:, None] + t
    live = (t < s["n_tok"][:, None]) & (pos < s["L_max"])
    cos = sin = None
    if case["rot"]:
        cs = s["cos_sin"][pos.clamp(max=s["L_max"] - 1)][:, :, None]
        cos, sin = cs[..., 0], cs[..., 1]
    k = _rotated(s["k"].float(), cos, sin, case)
    for x, to in ((_rotated(s["q"].float(), cos, sin, case), s["q_rot"]), (k, s["k_rot"])):
        to.copy_(torch.where(live[..., None, None], x.bfloat16(), to))
    page = torch.gather(c["table"].long(), 1, (pos // c["page"]).clamp(max=c["max_pages"] - 1))
    at = (page[live], (pos % c["page"])[live])
    for kv, x in ((0, k), (1, s["v"].float())):
        scale = torch.tensor((c["k_scale"], c["v_scale"])[kv], device=dev)
        for part, to in zip(_quantise(x[live], scale), (c["codes"], c["scales"])):
            to[kv].transpose(1, 2)[at] = part
    if case["pooled"]:
        bk, blocks = case["pooled"], s["pooled"].shape[2]
        end = torch.minimum(s["ctx"] + s["n_tok"], torch.full_like(s["ctx"], s["L_max"])).long()
        held = _held(_paged(c["codes"][0], c["table"]), _paged(c["scales"][0], c["table"]), c["k_scale"], s["lut"])
        at = torch.arange(held.shape[2], device=dev)
        held = torch.where((at < end[:, None])[:, None, :, None], held, torch.zeros((), device=dev))
        fit = blocks * bk
        if held.shape[2] < fit:
            held = torch.cat((held, held.new_zeros((n, hkv, fit - held.shape[2], d))), 2)
        first = torch.arange(blocks, device=dev) * bk
        count = (end[:, None] - first).clamp(0, bk)
        mean = held[:, :, :fit].reshape(n, hkv, blocks, bk, d).sum(3) / count.clamp(min=1)[:, None, :, None].float()
        touched = (first < end[:, None]) & (first + bk > s["ctx"][:, None]) & (s["n_tok"][:, None] > 0)
        s["pooled"].copy_(torch.where(touched[:, None, :, None], mean, s["pooled"]))


# -------------------------------------------------- exact values, in 64 bits

def _e2m1_64(nibble):
    """The number of a 4-bit code: sign, two exponent bits (bias 1), one mantissa bit."""
    n = nibble.to(torch.int64)
    e, m = ((n >> 1) & 3).double(), (n & 1).double()
    mag = torch.where(e == 0, m * 0.5, (1 + m / 2) * 2.0 ** (e - 1))
    return torch.where(n >= 8, -mag, mag)


def _e4m3_64(byte):
    """The number of an 8-bit scale: sign, four exponent bits (bias 7), three mantissa bits."""
    b = byte.to(torch.int64)
    e, m = ((b >> 3) & 15).double(), (b & 7).double()
    mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7))
    mag = torch.where((b & 127) == 127, torch.full_like(mag, math.nan), mag)
    return torch.where(b >= 128, -mag, mag)


def _rows_64(c, kv, pages, hkv):
    """All rows of the given pages, one KV head after another: [Hkv, len(pages)*page, d]."""
    codes, scales = c["codes"][kv][pages], c["scales"][kv][pages]  # [P, Hkv, page, .]
    x = torch.empty((*codes.shape[:3], codes.shape[3] * 2), dtype=torch.float64, device=codes.device)
    x[..., 0::2] = _e2m1_64(codes & 15)
    x[..., 1::2] = _e2m1_64(codes >> 4)
    x *= _e4m3_64(scales).repeat_interleave(16, -1)
    x *= (c["k_scale"], c["v_scale"])[kv]
    return x.transpose(0, 1).reshape(hkv, -1, x.shape[-1])


def _round_64(x, sizes):
    """x to the nearest of `sizes` (ascending, from 0), ties to the even place, larger ones to the last."""
    mids = (sizes[1:] + sizes[:-1]) / 2
    a = x.abs()
    low = torch.searchsorted(mids, a)           # ties go down ...
    high = torch.searchsorted(mids, a, right=True)  # ... or up
    at = torch.where((low != high) & (low % 2 == 1), high, low)
    return torch.copysign(sizes[at], x)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["cache"]
    n, hq, hkv, d = case["N"], case["Hq"], case["Hkv"], case["d"]
    dev = s["ctx"].device
    lengths = [int(x) for x in s["ctx"].tolist()]
    if case["op"] == "attn":
        out = torch.zeros((n, case["B"], hq, d), dtype=torch.float64, device=dev)
        g = hq // hkv
        for i, L in enumerate(lengths):
            pages = c["table"][i][:-(-L // c["page"])].long()
            k, v = (_rows_64(c, kv, pages, hkv)[:, :L] for kv in (0, 1))
            if case["block"]:
                k = torch.cat((k, s["bk"][i].double().transpose(0, 1)), 1)
                v = torch.cat((v, s["bv"][i].double().transpose(0, 1)), 1)
            if not k.shape[1]:
                continue
            for h in range(hq):
                p = torch.softmax(s["q"][i, :, h].double() @ k[h // g].T / math.sqrt(d), -1)
                out[i, :, h] = p @ v[h // g]
        return out
    if case["op"] == "gather":
        got = []
        for kv in range(2 if case["values"] else 1):
            x = torch.zeros((n, hkv, case["rows"], d), dtype=torch.float64, device=dev)
            for i, L in enumerate(lengths):
                if L:
                    rows = _rows_64(c, kv, c["table"][i][:-(-L // c["page"])].long(), hkv)
                    m = int(s["n_sel"][i, 0])
                    at = s["idx"][i, :, :m].long()[..., None].expand(-1, -1, d)
                    x[i, :, :m] = torch.gather(rows, 1, at)
            got.append(x)
        return got + [None] * (2 - len(got))
    toks = [int(x) for x in s["n_tok"].tolist()]
    r, T = case["rot"], case["T"]
    e2 = torch.tensor(E2M1, dtype=torch.float64, device=dev)
    e4 = _e4m3_64(torch.arange(127, device=dev))  # every scale that is not negative, 0 to 448
    q_rot, k_rot = s["q_rot"].double(), s["k_rot"].double()
    b = c["codes"].reshape(-1)
    values = torch.stack((_e2m1_64(b & 15), _e2m1_64(b >> 4)), 1).reshape(*c["codes"].shape, 2)
    scales = _e4m3_64(c["scales"])
    for i, (L, m) in enumerate(zip(lengths, toks)):
        m = min(m, s["L_max"] - L)
        if m <= 0:
            continue
        at = torch.arange(L, L + m, device=dev)

        def turn(x):
            x = x[i, :m].double()
            if not r:
                return x
            z = torch.view_as_complex(s["cos_sin"][at].double().contiguous())[:, None]
            f = x[..., :r]
            f = f.reshape(*f.shape[:-1], r // 2, 2) if case["interleaved"] else f.reshape(*f.shape[:-1], 2, r // 2).transpose(-1, -2)
            f = torch.view_as_real(torch.view_as_complex(f.contiguous()) * z)
            f = f if case["interleaved"] else f.transpose(-1, -2)
            return torch.cat((f.reshape(*x.shape[:-1], r), x[..., r:]), -1)

        k = turn(s["k"])
        q_rot[i, :m], k_rot[i, :m] = turn(s["q"]), k
        page, row = c["table"][i][at // c["page"]].long(), at % c["page"]
        for kv, x in ((0, k), (1, s["v"][i, :m].double())):
            scale = (c["k_scale"], c["v_scale"])[kv]
            x = x.reshape(m, hkv, d // 16, 16)
            sc = _round_64(x.abs().amax(-1) / (6 * scale), e4)
            y = torch.where(sc[..., None] == 0, torch.zeros_like(x), x / (sc[..., None] * scale))
            values[kv].transpose(1, 2)[page, row] = _round_64(y, e2).reshape(m, hkv, d // 2, 2)
            scales[kv].transpose(1, 2)[page, row] = sc
    pooled = None
    if case["pooled"]:
        pooled = s["pooled"].double()
        for i, (L, m) in enumerate(zip(lengths, toks)):
            end = min(L + m, s["L_max"])
            for blk in range(L // case["pooled"], -(-end // case["pooled"]) if m else 0):
                at = torch.arange(blk * case["pooled"], min(end, (blk + 1) * case["pooled"]), device=dev)
                page, row = c["table"][i][at // c["page"]].long(), at % c["page"]
                x = values[0].transpose(1, 2)[page, row].reshape(len(at), hkv, d // 16, 16)
                x = x * scales[0].transpose(1, 2)[page, row][..., None] * c["k_scale"]
                pooled[i, :, blk] = x.reshape(len(at), hkv, d).mean(0)
    return [q_rot, k_rot, values.reshape(-1, 2), scales, pooled]
