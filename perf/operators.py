"""Cases of the 4-bit KV block store: writing it, reading it back and attending over it.

A store holds units x max_blocks blocks of 64 tokens of one (sequence, kv head) each.  A block is
four tiles of 16 tokens; a tile is 2560 bytes: 1024 of K codes, 1024 of V codes, 256 of K scales
and 256 of V scales.  A token's 128 values of K (or V) fall into four groups of 32; a group is held
as m = f16(min), s = f16((max - min) / 15) and 32 codes n = clamp(rint((x - m) / s), 0, 15) and
stands for n s + m.  include/nosa.h (nosa_quant_append) gives the place of every code.

The sizes are this repository's workloads (synth/inputs.py): 2 kv heads with 8 query heads each at
16K and 64K tokens, 8 kv heads with 4 query heads each at 32K, and the one-sequence 4K case.
"""
import math

import numpy as np
import torch

own = False

TILE = 2560
BLOCK = 4 * TILE
D = 128


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's new token of 32 sequences, 8 kv heads, contexts of different lengths
        dict(name="append-token-8b-b32", op="append", batch=32, heads=8, tokens=1, start=32700, ragged=True),
        # prompts of 8 sequences written into an empty store
        dict(name="append-prompt-1b-16k", op="append", batch=8, heads=2, tokens=16384, start=0, ragged=False),
        # a padded batch of prompt chunks that continue contexts at odd positions
        dict(name="append-chunk-8b-ragged", op="append", batch=8, heads=8, tokens=2047, start=1001, ragged=True),
        # one small selection turned back to bf16 blocks
        dict(name="read-few-4k", op="read", batch=1, heads=2, context=4096, blocks=21, ragged=False),
        # a batch's selections (sink, 64 picked, 16 window blocks) turned back to bf16 blocks
        dict(name="read-selection-8b-32k", op="read", batch=32, heads=8, context=32768, blocks=81, ragged=True),
        # full attention of one sequence: latency counts
        dict(name="dense-4k-b1", op="dense", batch=1, heads=2, group=8, queries=1, context=4096, ragged=False),
        # full attention, small batch
        dict(name="dense-1b-16k-b8", op="dense", batch=8, heads=2, group=8, queries=1, context=16384, ragged=False),
        # full attention over a padded batch
        dict(name="dense-8b-32k-b32", op="dense", batch=32, heads=8, group=4, queries=1, context=32768, ragged=True),
        # four drafted tokens a sequence checked at once over a long context of odd length
        dict(name="dense-draft-1b-64k", op="dense", batch=8, heads=2, group=8, queries=4, context=65521, ragged=False),
        # sparse attention of one sequence: latency counts
        dict(name="sparse-4k-b1", op="sparse", batch=1, heads=2, group=8, queries=1, context=4096, blocks=21,
             ragged=False),
        # sparse attention, large batch
        dict(name="sparse-1b-16k-b128", op="sparse", batch=128, heads=2, group=8, queries=1, context=16384,
             blocks=81, ragged=False),
        # sparse attention over a padded batch
        dict(name="sparse-8b-32k-b32", op="sparse", batch=32, heads=8, group=4, queries=1, context=32768, blocks=81,
             ragged=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "read", "dense", "sparse"])
    heads = rng.choice([1, 2, 4, 8])
    batch = _spread(rng, 1, 128 if heads <= 2 else 32)
    units = batch * heads
    ragged = rng.random() < 0.6
    if op == "append":
        tokens = _spread(rng, 1, min(16384, 262144 // units))
        start = 0 if rng.random() < 0.3 else _spread(rng, 1, 4096)
        return dict(op=op, batch=batch, heads=heads, tokens=tokens, start=start, ragged=ragged)
    if op == "read":
        context = _spread(rng, 1, 32768)
        blocks = _spread(rng, 1, max(1, min(256, 20736 // units)))
        return dict(op=op, batch=batch, heads=heads, context=context, blocks=blocks, ragged=ragged)
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    queries = rng.choice([1, 1, 1, 2, 3, 4]) if group * 4 <= 32 else 1
    context = _spread(rng, 1, min(65536, 4194304 // units))
    case = dict(op=op, batch=batch, heads=heads, group=group, queries=queries, context=context, ragged=ragged)
    if op == "sparse":
        case["blocks"] = _spread(rng, 1, 128)
    return case


def _lengths(case, most):
    """Sequence lengths: `most`, or spread from a quarter of it to all of it (the same total for every seed)."""
    b = case["batch"]
    if not case["ragged"] or b == 1:
        return np.full(b, most, dtype=np.int64)
    return np.maximum(1, np.round(most * (0.25 + 0.75 * np.arange(b) / (b - 1)))).astype(np.int64)


# -------------------------------------------------------------------------------- the store
def _quantise(x):
    """x [..., 128] float32: codes [..., 4, 32] as float32, s and m [..., 4] as float16."""
    g = x.unflatten(-1, (4, 32))
    lo, hi = g.amin(-1), g.amax(-1)
    m = lo.to(torch.float16)
    s = ((hi - lo) / torch.full_like(lo, 15.0)).to(torch.float16)
    bad = ~(torch.isfinite(m) & torch.isfinite(s))
    m, s = m.masked_fill(bad, math.nan), s.masked_fill(bad, math.nan)
    wide = s.float().unsqueeze(-1)
    n = torch.round((g - m.float().unsqueeze(-1)) / torch.where(wide > 0, wide, 1.0))
    return torch.where(wide > 0, n.clamp(0, 15), 0.0), s, m


def _pack(k, v):
    """k, v [N, 64, 128] float32: the blocks' bytes, uint8 [N, 4, 2560]."""
    n = k.shape[0]
    out = torch.empty((n, 4, TILE), dtype=torch.uint8, device=k.device)
    c, s, m = _quantise(k)
    c = c.to(torch.uint8).view(n, 4, 16, 4, 4, 4, 2)  # tile, token, group, lane, byte, nibble
    c = (c[..., 0] | (c[..., 1] << 4)).transpose(3, 4)
    out[..., :1024] = c.reshape(n, 4, 1024)
    out[..., 2048:2304] = torch.cat((s, m), -1).view(n, 4, 16 * 8).contiguous().view(torch.uint8)
    c, s, m = _quantise(v)
    c = c.to(torch.uint8).view(n, 4, 2, 4, 2, 4, 8, 2, 2)  # tile, half, pair, parity, group, lane, byte, nibble
    c = (c[..., 0] | (c[..., 1] << 4)).permute(0, 1, 2, 6, 3, 5, 4, 7)
    out[..., 1024:2048] = c.reshape(n, 4, 1024)
    s, m = (z.view(n, 4, 8, 2, 4).transpose(3, 4).reshape(n, 4, 64) for z in (s, m))
    out[..., 2304:] = torch.cat((s, m), -1).contiguous().view(torch.uint8)
    return out


def _unpack(blocks):
    """Blocks' bytes, uint8 [N, 4, 2560]: the K and V that they stand for, float32 [N, 64, 128] each."""
    n = blocks.shape[0]
    c = blocks[..., :1024].reshape(n, 4, 16, 4, 4, 4)
    c = torch.stack((c & 15, c >> 4), -1).transpose(3, 4).reshape(n, 64, 4, 32)
    h = blocks[..., 2048:2304].contiguous().view(torch.float16).view(n, 64, 8, 1).float()
    k = (c * h[:, :, :4] + h[:, :, 4:]).view(n, 64, D)
    c = blocks[..., 1024:2048].reshape(n, 4, 2, 8, 4, 4, 2, 2)  # tile, half, lane, pair, group, parity, byte
    c = torch.stack((c & 15, c >> 4), -1).permute(0, 1, 2, 4, 6, 5, 3, 7, 8).reshape(n, 64, 4, 32)
    h = blocks[..., 2304:].contiguous().view(torch.float16).view(n, 4, 2, 8, 4, 2)
    h = h.permute(2, 0, 1, 3, 5, 4).reshape(2, n, 64, 4, 1).float()
    return k, (c * h[0] + h[1]).view(n, 64, D)


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    op, units = case["op"], case["batch"] * case["heads"]
    order = torch.randperm(case["batch"], generator=gen, device="cuda")

    def per_unit(values):
        values = torch.from_numpy(np.ascontiguousarray(values)).cuda()[order]
        return values.repeat_interleave(case["heads"]).to(torch.int32)

    st = dict(op=op, units=units)
    if op == "append":
        n, nb = case["tokens"], -(-(case["start"] + case["tokens"]) // 64)
        count = _lengths(case, n)
        pos = np.minimum(_lengths(case, case["start"])[::-1], case["start"]) if case["start"] else 0 * count
        touched = int(max((p + c - 1) // 64 - p // 64 + 1 for p, c in zip(pos, count)))
        st |= dict(nb=nb, n=n, pos=per_unit(pos), count=per_unit(count), n_blocks=touched)
        st["k"], st["v"] = (normal(units, n, D).to(torch.bfloat16) for _ in range(2))
        st["store"] = torch.zeros((units, nb, 4, TILE), dtype=torch.uint8, device="cuda")
        ids = (st["pos"] // 64)[:, None] + torch.arange(touched, dtype=torch.int32, device="cuda")
        last = ((st["pos"] + st["count"] - 1) // 64)[:, None]
        st["blocks"] = torch.where(ids <= last, ids, -1).contiguous()
        st["lens"] = st["pos"] + st["count"]
        head = (st["pos"] // 64).long()  # the block that the context ends in holds its earlier tokens
        old = _pack(*(normal(units, 64, D).to(torch.bfloat16).float() for _ in range(2)))
        st["store"][torch.arange(units, device="cuda"), head] = old
        st["kv"] = torch.zeros((units, touched, 2, 64, D), dtype=torch.bfloat16, device="cuda")
        return st
    context, nb = case["context"], -(-case["context"] // 64)
    lens = _lengths(case, context)
    st |= dict(nb=nb, lens=per_unit(lens))
    st["store"] = torch.empty((units, nb, 4, TILE), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 14) // nb)
    for u in range(0, units, step):  # a few GB of float32 at a time
        w = min(step, units - u)
        k, v = (normal(w * nb, 64, D).to(torch.bfloat16).float() for _ in range(2))
        st["store"][u:u + w] = _pack(k, v).view(w, nb, 4, TILE)
    if op in ("read", "sparse"):
        # sink, 16 (or fewer) window blocks, the others anywhere between; the list ascends, -1 pads it
        most = case["blocks"]
        nbl = ((st["lens"] + 63) // 64)[:, None]
        ids = torch.arange(nb, dtype=torch.int32, device="cuda")
        rank = torch.rand((units, nb), generator=gen, device="cuda")
        window = min(16, (most + 3) // 4)
        rank = torch.where((ids == 0) | (ids >= nbl - window), rank + 1, rank)
        rank = torch.where(ids < nbl, rank, -1.0)
        top = torch.topk(rank, min(most, nb), dim=1)
        picked = torch.where(top.values >= 0, top.indices, nb).sort(1).values
        sel = torch.full((units, most), -1, dtype=torch.int32, device="cuda")
        sel[:, :picked.shape[1]] = torch.where(picked < nb, picked, -1)
        st |= dict(blocks=sel, n_blocks=most)
        if op == "read":
            st["kv"] = torch.zeros((units, most, 2, 64, D), dtype=torch.bfloat16, device="cuda")
            return st
    rows = case["group"] * case["queries"]
    q = normal(units, rows, D)
    st["q"] = (q / q.norm(dim=-1, keepdim=True) * math.sqrt(D)).to(torch.bfloat16)
    st["out"] = torch.zeros((units, rows, D), dtype=torch.bfloat16, device="cuda")
    st |= dict(group=case["group"], queries=case["queries"], context=context)
    # the header's bound of nosa_quant_scratch_bytes for 256 SMs
    st["scratch"] = torch.zeros(256 + 520 * rows * (units + 4096), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def _run_own(st):
    from offloadable_block_sparse_gb300 import nosa as N
    stream = torch.cuda.current_stream().cuda_stream
    op, units, nb = st["op"], st["units"], st["nb"]
    if op == "append":
        N.nosa_quant_append(st["k"], st["v"], st["store"], units, st["n"], nb, pos=st["pos"], count=st["count"],
                            stream=stream)
    if op in ("append", "read"):
        N.nosa_quant_read(st["store"], units, nb, st["blocks"], st["n_blocks"], st["kv"], lens=st["lens"],
                          stream=stream)
        return st["kv"]
    if op == "dense":
        N.nosa_quant_dense_attend(st["q"], st["store"], units, st["group"], st["queries"], nb, st["lens"],
                                  st["context"], st["out"], st["scratch"], st["scratch"].numel(), stream=stream)
    else:
        N.nosa_quant_attend(st["q"], st["store"], st["blocks"], None, units, st["group"], st["queries"], nb,
                            st["n_blocks"], st["lens"], st["out"], st["scratch"], st["scratch"].numel(),
                            stream=stream)
    return st["out"]


def _gather(st):
    """The listed blocks' values, float32 [units, blocks, 64, 128] each, and the tokens' positions (-1: none)."""
    ids = st["blocks"].long()
    flat = torch.arange(st["units"], device="cuda")[:, None] * st["nb"] + ids.clamp(min=0)
    k, v = _unpack(st["store"].view(-1, 4, TILE)[flat.view(-1)])
    at = ids[:, :, None] * 64 + torch.arange(64, device="cuda")
    at = torch.where((ids[:, :, None] >= 0) & (at < st["lens"][:, None, None]), at, -1)
    return k.view(*ids.shape, 64, D), v.view(*ids.shape, 64, D), at


def _run_plain(st):
    op = st["op"]
    if op == "append":
        # the blocks as they were, with the new tokens' values in their rows
        k, v, at = _gather(st)
        i = at - st["pos"][:, None, None]
        new = (i >= 0) & (at >= 0)
        row = torch.arange(st["units"], device="cuda")[:, None, None] * st["n"] + i.clamp(0, st["n"] - 1)
        ck, sk, mk = _quantise(st["k"].float())
        cv, sv, mv = _quantise(st["v"].float())
        xk = (ck * sk.float().unsqueeze(-1) + mk.float().unsqueeze(-1)).view(-1, D)
        xv = (cv * sv.float().unsqueeze(-1) + mv.float().unsqueeze(-1)).view(-1, D)
        k = torch.where(new.unsqueeze(-1), xk[row], k)
        v = torch.where(new.unsqueeze(-1), xv[row], v)
        return (torch.stack((k, v), 2) * (at >= 0)[:, :, None, :, None]).to(torch.bfloat16)
    if op == "read":
        k, v, at = _gather(st)
        return (torch.stack((k, v), 2) * (at >= 0)[:, :, None, :, None]).to(torch.bfloat16)
    units, rows = st["units"], st["group"] * st["queries"]
    if op == "dense":
        k, v = _unpack(st["store"].view(-1, 4, TILE))
        at = torch.arange(st["nb"] * 64, device="cuda").expand(units, -1)
        at = torch.where(at < st["lens"][:, None], at, -1)
    else:
        k, v, at = _gather(st)
    k, v, at = k.view(units, -1, D), v.view(units, -1, D), at.reshape(units, 1, -1)
    # row h * queries + i is query token i of the last `queries` tokens: it sees the tokens up to its own
    late = st["queries"] - 1 - torch.arange(rows, device="cuda") % st["queries"]
    seen = (at >= 0) & (at < (st["lens"][:, None] - late)[:, :, None])
    z = torch.matmul(st["q"].float(), k.transpose(1, 2)) * (1.0 / math.sqrt(D))
    z = z.masked_fill(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return out.to(torch.bfloat16)


# ------------------------------------------------------------------------------ work
def work(case):
    """Each byte that has to move once: 160 bytes a token and unit in the store, 512 in bf16."""
    heads = case["heads"]
    if case["op"] == "append":
        # written, then read back; the block that the context ended in gives its earlier tokens too
        tokens = int(_lengths(case, case["tokens"]).sum()) * heads
        return {"bytes": tokens * (512 + 160 + 160 + 512), "flops": tokens * 2 * D * 4}
    lens = _lengths(case, case["context"])
    if "blocks" in case:
        lens = np.minimum(lens, case["blocks"] * 64)
    tokens = int(lens.sum()) * heads
    if case["op"] == "read":
        return {"bytes": tokens * (160 + 512), "flops": tokens * 2 * D * 2}
    rows = case["group"] * case["queries"]
    io = case["batch"] * heads * rows * D * 2 * 2
    return {"bytes": tokens * 160 + io, "flops": tokens * rows * 4 * D}


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    units, nb = st["units"], st["nb"]
    tok, dim = np.arange(64)[:, None], np.arange(D)[None, :]
    tile, i, grp = tok // 16 * TILE, tok % 16, dim // 32
    g8, e4 = dim % 32 // 4, dim % 4
    k_byte = tile + i * 64 + dim % 32 // 8 * 16 + grp * 4 + dim % 8 // 2
    v_byte = tile + 1024 + i // 8 * 512 + (g8 * 4 + i % 8 // 2) * 16 + grp * 4 + i % 2 * 2 + e4 // 2
    k_half = (tile + 2048) // 2 + i * 8 + grp
    v_half = (tile + 2304) // 2 + (i // 2 * 4 + grp) * 2 + i % 2
    cuda = {n: torch.from_numpy(np.broadcast_to(a, (64, D)).reshape(-1).copy()).cuda()
            for n, a in dict(kb=k_byte, vb=v_byte, kh=k_half, vh=v_half, sh=(dim % 2) * 4).items()}

    def values(blocks):
        """K and V of blocks given as bytes [n, 10240], float64 [n, 64, 128]."""
        half = blocks.view(torch.float16)
        got = []
        for byte, at, far in ((cuda["kb"], cuda["kh"], 4), (cuda["vb"], cuda["vh"], 64)):
            code = (blocks[:, byte].to(torch.int16) >> cuda["sh"].to(torch.int16)) & 15
            got.append((code.double() * half[:, at].double() + half[:, at + far].double()).view(-1, 64, D))
        return got

    def held(x):
        """What the store holds for x [..., 128], in float64."""
        x = x.double().reshape(*x.shape[:-1], 4, 32)
        low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        m, s = low.half().double(), ((high - low) / 15).half().double()
        return (torch.clamp(torch.round((x - m) / s), 0, 15) * s + m).flatten(-2)

    store = st["store"].view(units, nb, BLOCK)
    lens = st["lens"].tolist()
    if st["op"] in ("append", "read"):
        out = torch.zeros(st["kv"].shape, dtype=torch.float64, device="cuda")
        blocks = st["blocks"].tolist()
        for u in range(units):
            keep = [j for j, b in enumerate(blocks[u]) if b >= 0]
            ids = torch.tensor([blocks[u][j] for j in keep], device="cuda")
            k, v = values(store[u, ids])
            if st["op"] == "append":
                p, c = int(st["pos"][u]), int(st["count"][u])
                first = blocks[u][0] * 64
                for x, new in ((k, st["k"]), (v, st["v"])):
                    x.view(-1, D)[p - first:p - first + c] = held(new[u, :c])
            for x in (k, v):
                at = ids[:, None] * 64 + torch.arange(64, device="cuda")
                x[at >= lens[u]] = 0
            out[u, keep, 0], out[u, keep, 1] = k, v
        return out
    nq, rows = st["queries"], st["group"] * st["queries"]
    out = torch.zeros((units, rows, D), dtype=torch.float64, device="cuda")
    for u in range(units):
        ids = torch.arange(nb, device="cuda") if st["op"] == "dense" else st["blocks"][u][st["blocks"][u] >= 0].long()
        k, v = (x.reshape(-1, D) for x in values(store[u, ids]))
        at = (ids[:, None] * 64 + torch.arange(64, device="cuda")).view(-1)
        for late in range(nq):
            see = at < lens[u] - late
            if not bool(see.any()):
                continue
            r = torch.arange(nq - 1 - late, rows, nq, device="cuda")
            w = torch.softmax(st["q"][u, r].double() @ k[see].T / math.sqrt(D), dim=-1)
            out[u, r] = w @ v[see]
    return out
