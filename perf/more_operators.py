"""The operators of the paged 8-bit KV cache, their cases, plain forms and exact values.

The cache holds keys and values as e4m3 codes, one byte a value, with one power-of-two scale (a biased
exponent in a byte: 2^(byte - 127)) per block of consecutive positions and KV head, in pages of 16 to 128
positions; a value is code * scale.  Three operators work on it:

  append  rotates queries and keys by their positions, quantises keys and values and writes them into
          the sequences' pages; a block that holds older rows keeps the larger of its scale and the new
          rows', and its older rows follow (optionally the means of the touched blocks of keys)
  attn    attention of a block's queries over the whole cache and the block's own bf16 keys
  gather  rows of the cache at given positions as bf16 (the sparse pool, or staged candidates)

`own` False: elementary torch operations in fp32.  `own` True: the framework's kernels.
"""
import math
import random

import torch

own = False

TOP = 448.0  # the largest e4m3 number
E_MIN, E_MAX = -32, 32  # exponents of the scales


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a small layer: nothing but latency
        dict(name="attn token tiny", op="attn", N=1, Hq=4, Hkv=1, d=64, B=1, ctx=2048, ragged=False,
             page=16, block=16, own_keys=True),
        # single-token serving of a ragged batch, one sequence still empty
        dict(name="attn token batch", op="attn", N=64, Hq=32, Hkv=8, d=128, B=1, ctx=8192, ragged=True,
             page=64, block=32, own_keys=True),
        # single-token serving of one long context (split over the whole GPU)
        dict(name="attn token 128k", op="attn", N=1, Hq=32, Hkv=8, d=128, B=1, ctx=131071, ragged=False,
             page=128, block=64, own_keys=True),
        # four drafted tokens of every sequence of a batch, keys already in the cache
        dict(name="attn draft batch", op="attn", N=16, Hq=32, Hkv=8, d=128, B=4, ctx=8190, ragged=True,
             page=16, block=16, own_keys=False),
        # a handful of drafted tokens at seven heads a group, odd lengths
        dict(name="attn draft", op="attn", N=7, Hq=28, Hkv=4, d=128, B=5, ctx=12001, ragged=True,
             page=32, block=16, own_keys=False),
        # a denoising step with full attention on the 32K layer
        dict(name="attn block 32k", op="attn", N=1, Hq=28, Hkv=4, d=128, B=32, ctx=32768, ragged=False,
             page=64, block=64, own_keys=True),
        # the same on the 4 x 64K layer: the largest call
        dict(name="attn block 4x64k", op="attn", N=4, Hq=32, Hkv=8, d=128, B=32, ctx=65536,
             ragged=False, page=128, block=128, own_keys=True),
        # one new token of every sequence of a serving batch, most of them into a block in use
        dict(name="append token batch", op="append", N=64, Hq=32, Hkv=8, d=128, T=1, ctx=63, ragged=True,
             page=32, block=16, rot=128, interleaved=False, pooled=0, fused=True),
        # a decoded block joins the cache and the block means stage 1 scans
        dict(name="append block", op="append", N=1, Hq=28, Hkv=4, d=128, T=32, ctx=4077, ragged=False,
             page=64, block=32, rot=128, interleaved=False, pooled=64, fused=False),
        # prompts of a padded batch
        dict(name="append prompts", op="append", N=4, Hq=32, Hkv=8, d=128, T=4096, ctx=0, ragged=True,
             page=64, block=64, rot=128, interleaved=True, pooled=0, fused=True),
        # the selected rows of the 32K layer into the sparse pool
        dict(name="gather pool 32k", op="gather", N=1, Hq=28, Hkv=4, d=128, ctx=32768, ragged=False,
             page=64, block=32, rows=1344, values=True),
        # stage 2's candidate keys of the 4 x 64K layer
        dict(name="gather candidates 4x64k", op="gather", N=4, Hq=32, Hkv=8, d=128, ctx=65536,
             ragged=False, page=128, block=64, rows=4096, values=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attn", "attn", "append", "gather"))
    Hkv = rng.choice((1, 2, 4, 8))
    G = rng.choice((1, 2, 4, 7, 8))
    page = rng.choice((16, 32, 64, 128))
    c = dict(op=op, Hq=Hkv * G, Hkv=Hkv, d=rng.choice((64, 128, 128)), ragged=rng.random() < 0.6,
             page=page, block=rng.choice([b for b in (16, 32, 64, 128) if b <= page]))
    if op == "attn":
        c["B"] = 1 if rng.random() < 0.4 else _log(rng, 1, min(64, 256 // G))
        c["ctx"] = _log(rng, 1, 131072)
        c["N"] = _log(rng, 1, max(1, min(64, (1 << 21) // (Hkv * c["ctx"]))))
        c["own_keys"] = rng.random() < 0.7
    elif op == "append":
        c["T"] = _log(rng, 1, 4096)
        c["N"] = _log(rng, 1, max(1, min(64, (1 << 14) // c["T"])))
        c["ctx"] = rng.randrange(0, 300)
        c["rot"] = rng.choice((0, 32, 64, c["d"]))
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
    n, hq, hkv, d, blk = case["N"], case["Hq"], case["Hkv"], case["d"], case["block"]
    if case["op"] == "attn":
        lengths, b = _lengths(case, case["ctx"], "ctx"), case["B"]
        keys, own_keys = sum(lengths), n * b if case["own_keys"] else 0
        scales = sum(-(-x // blk) for x in lengths)
        return {"bytes": 2 * hkv * (keys * d + scales) + 4 * n * b * hq * d + 4 * own_keys * hkv * d,
                "flops": 4 * hq * b * d * (keys + own_keys)}
    if case["op"] == "append":
        toks, ctx = _lengths(case, case["T"], "tok"), _lengths(case, case["ctx"], "ctx")
        places = set()  # positions whose angles are read
        scales = means = earlier = 0
        for c, t in zip(ctx, toks):
            if not t:
                continue
            places.update(range(c, c + t))
            scales += (c + t - 1) // blk - c // blk + 1
            if case["pooled"]:
                means += (c + t - 1) // case["pooled"] - c // case["pooled"] + 1
                earlier += c % case["pooled"]
        row = 2 * (2 * hq + 3 * hkv) * d + 2 * hkv * d  # q, k, v in; q_rot, k_rot and the codes out
        angles = 4 * case["rot"] * len(places) if case["rot"] else 0
        return {"bytes": sum(toks) * row + 2 * hkv * scales + angles + hkv * d * (4 * means + earlier),
                "flops": sum(toks) * d * (3 * hq + 8 * hkv)}
    rows = n * hkv * case["rows"]
    return {"bytes": rows * (4 + (2 if case["values"] else 1) * 3 * d), "flops": 0}


# ------------------------------------------------------- the cache's format

def _exponent(top):
    """The scale exponent of a block whose largest magnitude is `top`: the smallest e with
    top <= 448 * 2^e, within the exponents that a scale may have."""
    f, e = torch.frexp(top)  # top = f * 2^e, f in [1/2, 1); 448 = 7/8 * 2^9
    e = e - 9 + (f > 0.875).to(e.dtype)
    return torch.where(top == 0, torch.full_like(e, E_MIN), e.clamp(E_MIN, E_MAX))


def _codes(x, e):
    """x fp32 and exponents e that broadcast over it -> e4m3 codes as bytes."""
    y = torch.ldexp(x, -e).clamp(-TOP, TOP)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _held(codes, scales, block):
    """codes [..., rows, d], scales [..., rows / block] (bytes) -> fp32 values [..., rows, d]."""
    v = codes.view(torch.float8_e4m3fn).float()
    s = torch.exp2(scales.float() - 127.0).repeat_interleave(block, -1)
    return v * s.unsqueeze(-1)


def _paged(x, table):
    """The pages [n_pages, Hkv, ...] of every sequence in order: [N, Hkv, max_pages, ...] (entries
    without a page read page 0)."""
    return x[table.clamp(min=0).long()].transpose(1, 2)


def _dense(c, kv):
    """The held rows of all sequences: fp32 [N, Hkv, max_pages * page, d]."""
    codes, scales = _paged(c["codes"][kv], c["table"]), _paged(c["scales"][kv], c["table"])
    return _held(codes.flatten(2, 3), scales.flatten(2, 3), c["block"])


# ------------------------------------------------------------------ inputs

def _pool(case, lengths, gen, dev):
    """A paged cache with room for `lengths`, its pages in random order.  Where no row is held it has
    arbitrary bytes (NaN codes among them); zeros for the append, whose pages are outputs."""
    n, hkv, d, page, block = case["N"], case["Hkv"], case["d"], case["page"], case["block"]
    need = [-(-x // page) for x in lengths]
    max_pages, used = max(1, max(need)), sum(need)
    n_pages = used + 3
    order = torch.randperm(n_pages, generator=gen, device=dev)[:used].to(torch.int32)
    want = torch.arange(max_pages, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
    table = torch.full((n, max_pages), -1, dtype=torch.int32, device=dev)
    table[want] = order
    codes = torch.randint(0, 256, (2, n_pages, hkv, page, d), generator=gen, device=dev, dtype=torch.uint8)
    scales = torch.randint(0, 256, (2, n_pages, hkv, page // block), generator=gen, device=dev,
                           dtype=torch.uint8)
    if case["op"] == "append":
        codes.zero_()
        scales.fill_(127)
    return dict(table=table, codes=codes, scales=scales, page=page, block=block, max_pages=max_pages,
                want=want)


def _fill(c, case, lengths, topic, gen, dev):
    """Every row below `lengths` holds quantised keys and values: normal keys, a few channels and the
    first four positions larger than the rest (a model's outlier channels and sink tokens), a hundredth
    near the queries' common direction; smaller values."""
    hkv, d, page, block = case["Hkv"], case["d"], case["page"], case["block"]
    n, mp = c["table"].shape
    wide = 1.0 + 3.0 * (torch.rand((hkv, 1, d), generator=gen, device=dev) < 0.03).float()
    pos = torch.arange(mp * page, device=dev)
    held = pos < torch.tensor(lengths, device=dev)[:, None]  # [N, rows]
    at = c["table"][c["want"]].long()
    for kv in (0, 1):
        x = torch.randn((n, hkv, mp * page, d), generator=gen, device=dev)
        if kv == 0:
            hot = torch.rand((n, hkv, mp * page, 1), generator=gen, device=dev) < 0.01
            x += torch.where(hot, 2.0 * topic[None, :, None], torch.zeros((), device=dev))
            x *= wide
            x[:, :, :4] *= 2.0
        else:
            x *= 0.5
        x = torch.where(held[:, None, :, None], x.bfloat16().float(), torch.zeros((), device=dev))
        b = x.view(n, hkv, -1, block, d)
        e = _exponent(b.abs().amax((3, 4)))
        codes = _codes(b, e[..., None, None]).view(n, hkv, mp, page, d).transpose(1, 2)
        scales = (e + 127).to(torch.uint8).view(n, hkv, mp, page // block).transpose(1, 2)
        rows = held.view(n, mp, 1, page, 1)[c["want"]]
        blocks = held.view(n, mp, 1, page // block, block)[..., 0][c["want"]]
        c["codes"][kv][at] = torch.where(rows, codes[c["want"]], c["codes"][kv][at])
        c["scales"][kv][at] = torch.where(blocks, scales[c["want"]], c["scales"][kv][at])


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(int(seed))
    n, hq, hkv, d = case["N"], case["Hq"], case["Hkv"], case["d"]
    topic = torch.randn((hkv, d), generator=gen, device=dev)
    s = dict(case=case)

    def queries(rows):
        x = torch.randn((n, rows, hkv, hq // hkv, d), generator=gen, device=dev)
        return (0.7 * topic[:, None] + 0.7 * x).reshape(n, rows, hq, d).bfloat16()

    if case["op"] == "append":
        toks, T = _lengths(case, case["T"], "tok"), case["T"]
        ctx = _lengths(case, case["ctx"], "ctx")
        s["L_max"] = case["ctx"] + T
        c = _pool(case, [x + T for x in ctx], gen, dev)
        _fill(c, case, ctx, topic, gen, dev)
        s["n_tok"] = torch.tensor(toks, dtype=torch.int32, device=dev)
        k = torch.randn((n, T, hkv, d), generator=gen, device=dev)
        k *= 1.0 + 3.0 * (torch.rand((hkv, d), generator=gen, device=dev) < 0.03).float()
        k = k.bfloat16()
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
        _fill(c, case, ctx, topic, gen, dev)
        if case["op"] == "attn":
            s["q"] = queries(case["B"])
            s["out"] = torch.zeros_like(s["q"])
            if case["own_keys"]:
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
        s["kv8"] = H.kv8(c["page"], c["block"], c["table"], c["codes"][0], c["scales"][0], c["codes"][1],
                         c["scales"][1])
        if case["op"] == "attn":
            s["ws"] = torch.zeros(H.herald_workspace_size_kv8(s["dims"]), dtype=torch.uint8, device=dev)
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
            H.herald_kv8_attn(s["dims"], s["q"], s["kv8"], s["ctx"], s.get("bk"), s.get("bv"),
                              s["out"], ws=s["ws"], stream=st)
            return s["out"]
        if op == "gather":
            H.herald_kv8_gather(s["dims"], s["idx"], s["n_sel"], s["case"]["rows"], s["kv8"],
                                s["pool_k"], s["pool_v"], stream=st)
            return [s["pool_k"], s["pool_v"]]
        H.herald_kv8_append(s["dims"], s["case"]["T"], s["q"], s["k"], s["v"], s["ctx"], s["kv8"],
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
    return [s["q_rot"], s["k_rot"], c["codes"].view(torch.float8_e4m3fn),
            c["scales"].view(torch.float8_e8m0fnu), s.get("pooled")]


def _attn(s):
    case, c = s["case"], s["cache"]
    n, hq, hkv, d, b = case["N"], case["Hq"], case["Hkv"], case["d"], case["B"]
    k, v = _dense(c, 0), _dense(c, 1)
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
        x = c["codes"][kv][page, head, pos % c["page"]].view(torch.float8_e4m3fn).float()
        x = x * torch.exp2(c["scales"][kv][page, head, pos % c["page"] // c["block"]].float() - 127.0)[..., None]
        got.append(torch.where(used[..., None], x, torch.zeros((), device=x.device)).bfloat16())
    return got + [None] * (2 - len(got))


def _rotated(x, cos, sin, case):
    """x [N, T, H, d] fp32, cos and sin [N, T, 1, rot/2] -> bf16."""
    r = case["rot"]
    if not r:
        return x.bfloat16()
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
    u, w = a * cos - b * sin, b * cos + a * sin
    front = torch.stack((u, w), -1).flatten(-2) if case["interleaved"] else torch.cat((u, w), -1)
    return torch.cat((front, x[..., r:]), -1).bfloat16()


def _append(s):
    case, c = s["case"], s["cache"]
    n, hkv, d, T = case["N"], case["Hkv"], case["d"], case["T"]
    dev, block, page = s["ctx"].device, c["block"], c["page"]
    t = torch.arange(T, device=dev)
    ctx = s["ctx"].long()
    end = torch.minimum(ctx + s["n_tok"].clamp(0, T), torch.full_like(ctx, s["L_max"]))
    pos = ctx[:, None] + t
    live = pos < end[:, None]
    cos = sin = None
    if case["rot"]:
        cs = s["cos_sin"][pos.clamp(max=s["L_max"] - 1)][:, :, None]
        cos, sin = cs[..., 0], cs[..., 1]
    k = _rotated(s["k"].float(), cos, sin, case)
    for x, to in ((_rotated(s["q"].float(), cos, sin, case), s["q_rot"]), (k, s["k_rot"])):
        to.copy_(torch.where(live[..., None, None], x, to))
    # the touched blocks, from the one that the first new token falls into
    nb = -(-(T - 1) // block) + 1
    at = (ctx // block)[:, None] * block + torch.arange(nb * block, device=dev)  # [N, nb * block]
    new = (at >= ctx[:, None]) & (at < end[:, None])
    touched = new.view(n, nb, block).any(2)
    older = (at < ctx[:, None]) & touched.repeat_interleave(block, 1)
    ph = torch.gather(c["table"].long(), 1, (at // page).clamp(max=c["max_pages"] - 1)).clamp(min=0)
    head = torch.arange(hkv, device=dev)
    bph, bat = ph[:, ::block, None], (at[:, ::block] % page // block)[..., None]
    used = older.view(n, nb, block).any(2)[..., None]  # the block's scale stands for older rows
    for kv, x in ((0, k), (1, s["v"])):
        x = x.float()[torch.arange(n, device=dev)[:, None], (at - ctx[:, None]).clamp(0, T - 1)]
        x = torch.where(new[..., None, None], x, torch.zeros((), device=dev))  # [N, nb * block, Hkv, d]
        e = _exponent(x.view(n, nb, block, hkv, d).abs().amax((2, 4)))  # [N, nb, Hkv]
        was = c["scales"][kv][bph, head, bat].to(torch.int32) - 127
        e = torch.where(used, torch.maximum(e, was), e)
        row_e = e.repeat_interleave(block, 1)[..., None]
        codes = c["codes"][kv].transpose(1, 2)  # [n_pages, page, Hkv, d]
        held = codes[ph, at % page]
        moved = held.view(torch.float8_e4m3fn).float()
        moved = _codes(moved, row_e - was.repeat_interleave(block, 1)[..., None])
        put = torch.where(new[..., None, None], _codes(x, row_e), moved)
        codes[ph[new | older], (at % page)[new | older]] = put[new | older]
        scales = c["scales"][kv].transpose(1, 2)  # [n_pages, page / block, Hkv]
        scales[bph[..., 0][touched], bat[..., 0][touched]] = (e + 127).to(torch.uint8)[touched]
    if case["pooled"]:
        bk, blocks = case["pooled"], s["pooled"].shape[2]
        held = _dense(c, 0)
        at = torch.arange(held.shape[2], device=dev)
        held = torch.where((at < end[:, None])[:, None, :, None], held, torch.zeros((), device=dev))
        fit = blocks * bk
        if held.shape[2] < fit:
            held = torch.cat((held, held.new_zeros((n, hkv, fit - held.shape[2], d))), 2)
        first = torch.arange(blocks, device=dev) * bk
        count = (end[:, None] - first).clamp(0, bk)
        mean = held[:, :, :fit].reshape(n, hkv, blocks, bk, d).sum(3) / count.clamp(min=1)[:, None, :, None].float()
        some = (first < end[:, None]) & (first + bk > ctx[:, None]) & (end > ctx)[:, None]
        s["pooled"].copy_(torch.where(some[:, None, :, None], mean, s["pooled"]))


# -------------------------------------------------- exact values, in 64 bits

def _e4m3_64(byte):
    """The number of a code: sign, four exponent bits (bias 7), three mantissa bits."""
    b = byte.to(torch.int64)
    e, m = ((b >> 3) & 15).double(), (b & 7).double()
    mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7))
    mag = torch.where((b & 127) == 127, torch.full_like(mag, math.nan), mag)
    return torch.where(b >= 128, -mag, mag)


def _power(e):
    """2^e of whole numbers, without a rounding."""
    return torch.ldexp(torch.ones_like(e), e.round().to(torch.int32))


def _rows_64(c, kv, pages, hkv):
    """All rows of the given pages, one KV head after another: [Hkv, len(pages)*page, d]."""
    x = _e4m3_64(c["codes"][kv][pages])  # [P, Hkv, page, d]
    x *= _power(c["scales"][kv][pages].double() - 127).repeat_interleave(c["block"], -1)[..., None]
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
    dev, page, block = s["ctx"].device, c["page"], c["block"]
    lengths = [int(x) for x in s["ctx"].tolist()]
    if case["op"] == "attn":
        out = torch.zeros((n, case["B"], hq, d), dtype=torch.float64, device=dev)
        g = hq // hkv
        for i, L in enumerate(lengths):
            pages = c["table"][i][:-(-L // page)].long()
            k, v = (_rows_64(c, kv, pages, hkv)[:, :L] for kv in (0, 1))
            if case["own_keys"]:
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
                    rows = _rows_64(c, kv, c["table"][i][:-(-L // page)].long(), hkv)
                    m = int(s["n_sel"][i, 0])
                    at = s["idx"][i, :, :m].long()[..., None].expand(-1, -1, d)
                    x[i, :, :m] = torch.gather(rows, 1, at)
            got.append(x)
        return got + [None] * (2 - len(got))
    toks = [int(x) for x in s["n_tok"].tolist()]
    r, T = case["rot"], case["T"]
    e4 = _e4m3_64(torch.arange(127, device=dev))  # every code that is not negative, 0 to 448
    q_rot, k_rot = s["q_rot"].double(), s["k_rot"].double()
    codes = _e4m3_64(c["codes"])
    scales = _power(c["scales"].double() - 127)
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
        first, n_blk = L // block, (L + m - 1) // block - L // block + 1
        of = at // block - first  # which of the touched blocks
        bpos = (torch.arange(n_blk, device=dev) + first) * block
        bpage, bwhich = c["table"][i][bpos // page].long(), bpos % page // block
        prior = torch.arange(first * block, L, device=dev)  # older rows of the first block
        ppage, prow = c["table"][i][prior // page].long(), prior % page
        ph, row = c["table"][i][at // page].long(), at % page
        for kv, x in ((0, k.bfloat16().double()), (1, s["v"][i, :m].double())):  # held is what k_rot says
            top = torch.zeros((n_blk, hkv), dtype=torch.float64, device=dev)
            top.scatter_reduce_(0, of[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
            e = torch.ceil(torch.log2(top / TOP)).clamp(E_MIN, E_MAX)
            was = scales[kv][bpage[:1], :, bwhich[:1]].log2().round()[0]
            if len(prior):
                e[0] = torch.maximum(e[0], was)
                moved = codes[kv].transpose(1, 2)[ppage, prow] * _power(was - e[0])[None, :, None]
                codes[kv].transpose(1, 2)[ppage, prow] = _round_64(moved, e4)
            codes[kv].transpose(1, 2)[ph, row] = _round_64(x * _power(-e[of])[..., None], e4)
            scales[kv].transpose(1, 2)[bpage, bwhich] = _power(e)
    pooled = None
    if case["pooled"]:
        pooled = s["pooled"].double()
        for i, (L, m) in enumerate(zip(lengths, toks)):
            end = min(L + m, s["L_max"])
            for blk in range(L // case["pooled"], -(-end // case["pooled"]) if m else 0):
                at = torch.arange(blk * case["pooled"], min(end, (blk + 1) * case["pooled"]), device=dev)
                ph, row = c["table"][i][at // page].long(), at % page
                x = codes[0].transpose(1, 2)[ph, row] * scales[0].transpose(1, 2)[ph, row // block][..., None]
                pooled[i, :, blk] = x.mean(0)
    return [q_rot, k_rot, codes, scales, pooled]
