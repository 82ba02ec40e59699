"""Cases of the path from projections to an 8-bit KV store that evicts: rotary positions, writing the
store, attending over it with each block's attention mass, and dropping the blocks of least mass.

An 8-bit store holds units x rows blocks of 64 tokens of one (sequence, kv head) each.  Values are e4m3
codes times a power of two, one for the block's K and one for its V: the smallest s with max|x| <= 448 s.
A block is four tiles of 16 tokens (2048 bytes of K codes, 2048 of V codes) and 128 bytes that begin with
the two scales as float32.  include/nosa.h (nosa_byte_append) gives the place of every code.

The sizes are this repository's workloads (synth/inputs.py): 2 kv heads with 8 query heads each at 16K
and 64K tokens, 8 kv heads with 4 query heads each at 32K, and the one-sequence 4K case.
"""
import math

import numpy as np
import torch

own = False

TILE = 4096
BLOCK = 4 * TILE + 128
D = 128
LEAST = -118  # the smallest exponent of a scale


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's q and k of 32 sequences at far positions: latency counts
        dict(name="rope-token-8b-b32", op="rope", batch=32, heads=8, group=4, tokens=1, start=32700, rot=128,
             pairs="half", scaling="none", ragged=True),
        # the prompts of 8 sequences
        dict(name="rope-prompt-1b-16k", op="rope", batch=8, heads=2, group=8, tokens=16384, start=0, rot=128,
             pairs="half", scaling="none", ragged=False),
        # a padded batch of prompt chunks of a context far beyond the trained one, half of each head rotated
        dict(name="rope-chunk-8b-ragged", op="rope", batch=8, heads=8, group=4, tokens=2047, start=1000003, rot=64,
             pairs="interleaved", scaling="parts", ragged=True),
        # one decode step's new token of 32 sequences, written among earlier tokens and read back
        dict(name="append-token-8b-b32", op="append", batch=32, heads=8, tokens=1, start=32700, ragged=True),
        # a padded batch of prompt chunks that continue contexts at odd positions
        dict(name="append-chunk-8b-ragged", op="append", batch=8, heads=8, tokens=2047, start=1001, ragged=True),
        # full attention of one sequence: latency counts
        dict(name="dense-4k-b1", op="dense", batch=1, heads=2, group=8, queries=1, context=4096, ragged=False),
        # full attention over a padded batch
        dict(name="dense-8b-32k-b32", op="dense", batch=32, heads=8, group=4, queries=1, context=32768, ragged=True),
        # four drafted tokens a sequence checked at once over a long context of odd length
        dict(name="dense-draft-1b-64k", op="dense", batch=8, heads=2, group=8, queries=4, context=65521, ragged=False),
        # sparse attention over a batch's selections (sink, 64 picked, 16 window blocks)
        dict(name="sparse-1b-16k-b128", op="sparse", batch=128, heads=2, group=8, queries=1, context=16384, blocks=81,
             ragged=False),
        # a decode step over a padded batch's evicting stores, with the mass of each block
        dict(name="mass-8b-32k-b32", op="mass", batch=32, heads=8, group=4, queries=1, context=32768, blocks=128,
             ragged=True),
        # the same step's eviction: a block goes where the next one needs its row
        dict(name="evict-step-8b-b32", op="evict", batch=32, heads=8, slots=128, budget=128, context=32768, ragged=True),
        # contexts of many sequences cut to a quarter after their prompts
        dict(name="evict-prompt-1b-64k", op="evict", batch=128, heads=2, slots=1025, budget=256, context=65536,
             ragged=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "dense", "sparse", "mass", "evict", "evict"])
    heads = rng.choice([1, 2, 4, 8])
    batch = _spread(rng, 1, 128 if heads <= 2 else 32)
    units = batch * heads
    ragged = rng.random() < 0.6
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if op == "rope":
        tokens = _spread(rng, 1, min(16384, 2359296 // (units * (group + 1))))
        return dict(op=op, batch=batch, heads=heads, group=group, tokens=tokens, start=_spread(rng, 1, 1 << 20) - 1,
                    rot=rng.choice([128, 128, 64, 96, 32, 2 * rng.randint(1, 64)]),
                    pairs=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "base", "parts"]), ragged=ragged)
    if op == "append":
        tokens = _spread(rng, 1, min(16384, 131072 // units))
        start = 0 if rng.random() < 0.3 else _spread(rng, 1, 4096)
        return dict(op=op, batch=batch, heads=heads, tokens=tokens, start=start, ragged=ragged)
    if op == "evict":
        slots = _spread(rng, 1, 1025)
        budget = rng.randint(1, slots)
        return dict(op=op, batch=batch, heads=heads, slots=slots, budget=budget,
                    context=_spread(rng, 1, 65536), ragged=ragged)
    queries = rng.choice([1, 1, 1, 2, 3, 4]) if group * 4 <= 32 else 1
    context = _spread(rng, 1, min(65536, 4194304 // units))
    case = dict(op=op, batch=batch, heads=heads, group=group, queries=queries, context=context, ragged=ragged)
    if op != "dense":
        case["blocks"] = _spread(rng, 1, 128)
    return case


def _lengths(case, most):
    """Sequence lengths: `most`, or spread from a quarter of it to all of it (the same total for every seed)."""
    b = case["batch"]
    if not case["ragged"] or b == 1:
        return np.full(b, most, dtype=np.int64)
    return np.maximum(1, np.round(most * (0.25 + 0.75 * np.arange(b) / (b - 1)))).astype(np.int64)


# ---------------------------------------------------------------------------------- rotary
def _rope_config(case):
    """What a program says of its rotary positions."""
    kind = case["scaling"]
    return dict(rot_dims=case["rot"], interleaved=case["pairs"] == "interleaved", scaling=kind, base=500000.0,
                factor=1.0 if kind == "none" else 8.0, low=1.0, high=32.0, original=32768.0,
                attention_factor=0.1 * math.log(8.0) + 1.0 if kind == "parts" else 1.0)


def _frequencies(c):
    """Radians per position of each pair, float64."""
    i = np.arange(c["rot_dims"] // 2, dtype=np.float64)
    base = c["base"]
    if c["scaling"] == "base" and c["rot_dims"] > 2:
        base *= c["factor"] ** (c["rot_dims"] / (c["rot_dims"] - 2))
    f = base ** (-2.0 * i / c["rot_dims"])
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "parts":
        turns = c["original"] * f / (2 * math.pi)
        keep = np.clip((turns - c["low"]) / (c["high"] - c["low"]), 0.0, 1.0)
        f = f * (keep + (1 - keep) / c["factor"])
    return f


# -------------------------------------------------------------------------------- the store
def _scale(top):
    """The block scale for values up to `top`: a power of two, 0 for 0."""
    m, e = torch.frexp(top / 448.0)
    e = torch.where(m == 0.5, e - 1, e).clamp(min=LEAST)
    return torch.where(top > 0, ((e + 127) << 23).to(torch.int32).view(torch.float32), 0.0)


def _codes(x, s):
    """x [N, 64, 128] float32 with scales s [N]: e4m3 codes."""
    s = torch.where(s > 0, s, 1.0)[:, None, None]
    return (x / s).to(torch.float8_e4m3fn)


def _pack(k, v):
    """k, v [N, 64, 128] float32: the blocks' bytes, uint8 [N, BLOCK]."""
    n = k.shape[0]
    out = torch.zeros((n, BLOCK), dtype=torch.uint8, device=k.device)
    ks, vs = (_scale(x.abs().amax((1, 2))) for x in (k, v))
    tiles = out[:, :4 * TILE].view(n, 4, 2, TILE // 2)
    # K: tile, 8 tokens' half, token, 32 dims' quarter, half of it, dim
    c = _codes(k, ks).view(torch.uint8).view(n, 4, 2, 8, 4, 2, 16)
    tiles[:, :, 0] = c.permute(0, 1, 2, 5, 3, 4, 6).reshape(n, 4, 2048)
    # V: tile, half, pair of tokens, parity, 16 dims' group, quarter of it, pair of dims, parity
    c = _codes(v, vs).view(torch.uint8).view(n, 4, 2, 4, 2, 8, 4, 2, 2)
    tiles[:, :, 1] = c.permute(0, 1, 6, 5, 3, 7, 2, 8, 4).reshape(n, 4, 2048)
    out[:, 4 * TILE:4 * TILE + 8] = torch.stack((ks, vs), 1).view(torch.uint8)
    return out


def _unpack(blocks):
    """Blocks' bytes, uint8 [N, BLOCK]: the K and V that they stand for, float32 [N, 64, 128] each, and their scales."""
    n = blocks.shape[0]
    tiles = blocks[:, :4 * TILE].reshape(n, 4, 2, TILE // 2)
    s = blocks[:, 4 * TILE:4 * TILE + 8].contiguous().view(torch.float32)
    c = tiles[:, :, 0].reshape(n, 4, 2, 2, 8, 4, 16).permute(0, 1, 2, 4, 5, 3, 6).reshape(n, 64, D)
    k = c.contiguous().view(torch.float8_e4m3fn).float() * s[:, 0, None, None]
    c = tiles[:, :, 1].reshape(n, 4, 4, 8, 4, 2, 2, 2, 2).permute(0, 1, 6, 4, 8, 3, 2, 5, 7).reshape(n, 64, D)
    v = c.contiguous().view(torch.float8_e4m3fn).float() * s[:, 1, None, None]
    return k, v, s[:, 0], s[:, 1]


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    op, batch, heads = case["op"], case["batch"], case["heads"]
    units = batch * heads
    order = torch.randperm(batch, generator=gen, device="cuda")

    def per_sequence(values):
        return torch.from_numpy(np.ascontiguousarray(values)).cuda()[order].to(torch.int32)

    def per_unit(values):
        return per_sequence(values).repeat_interleave(heads)

    st = dict(op=op, units=units)
    if op == "rope":
        n, hq = case["tokens"], heads * case["group"]
        st |= dict(batch=batch, n=n, config=_rope_config(case))
        # a projection's output: [sequence][token][q heads, k heads][dim]
        st["x"] = normal(batch, n, hq + heads, D).to(torch.bfloat16)
        st["pos"] = per_sequence(case["start"] - np.arange(batch) * (case["start"] // (2 * batch)))
        st["count"] = per_sequence(_lengths(case, n))
        # q and k in the layout of the attention and append calls; rows behind a sequence's tokens stay zero
        st["q"] = torch.zeros((batch, hq, n, D), dtype=torch.bfloat16, device="cuda")
        st["k"] = torch.zeros((batch, heads, n, D), dtype=torch.bfloat16, device="cuda")
        return st
    if op == "evict":
        slots, context = case["slots"], case["context"]
        lens = per_unit(_lengths(case, context))
        nbl = (lens + 63) // 64
        nb = -(-context // 64)
        ids = torch.arange(nb, dtype=torch.int32, device="cuda")
        rank = torch.rand((units, nb), generator=gen, device="cuda")
        # the sink and the last 16 blocks are held where there is room, others by chance; every other sequence has
        # just begun a block that no row holds yet
        new = (torch.arange(units, device="cuda") // heads % 2 == 0) & (nbl > 1)
        rank = torch.where((ids == 0) | (ids >= nbl[:, None] - 16), rank + 1, rank)
        rank = torch.where(ids < (nbl - new.int())[:, None], rank, -1.0)
        top = torch.topk(rank, min(slots, nb), dim=1)
        blk = torch.full((units, slots), -1, dtype=torch.int32, device="cuda")
        blk[:, :top.indices.shape[1]] = torch.where(top.values >= 0, top.indices, -1).to(torch.int32)
        shuffle = torch.rand((units, slots), generator=gen, device="cuda").argsort(1)
        st["slot_blk"] = blk.gather(1, shuffle).contiguous()
        st["acc"] = torch.where(st["slot_blk"] >= 0, torch.exp(2 * normal(units, slots)), 0.0)
        st["mass"] = torch.where(st["slot_blk"] >= 0, torch.exp(3 * normal(units, slots) - 4), 0.0)
        st |= dict(slots=slots, budget=case["budget"], lens=lens, next=nbl - 1, sink=1, window=16, decay=0.97)
        st["acc_out"], st["slot_out"] = torch.zeros_like(st["acc"]), torch.zeros_like(st["slot_blk"])
        st["row"] = torch.zeros(units, dtype=torch.int32, device="cuda")
        return st
    if op == "append":
        n, nb = case["tokens"], -(-(case["start"] + case["tokens"]) // 64)
        count = _lengths(case, n)
        pos = np.minimum(_lengths(case, case["start"])[::-1], case["start"]) if case["start"] else 0 * count
        touched = int(max((p + c - 1) // 64 - p // 64 + 1 for p, c in zip(pos, count)))
        st |= dict(nb=nb, n=n, pos=per_unit(pos), count=per_unit(count), n_blocks=touched)
        # tokens differ in size, so that some blocks need a larger scale than they have
        st["k"], st["v"] = ((normal(units, n, D) * torch.exp(0.5 * normal(units, n, 1))).to(torch.bfloat16)
                            for _ in range(2))
        st["store"] = torch.zeros((units, nb, BLOCK), dtype=torch.uint8, device="cuda")
        ids = (st["pos"] // 64)[:, None] + torch.arange(touched, dtype=torch.int32, device="cuda")
        last = ((st["pos"] + st["count"] - 1) // 64)[:, None]
        st["blocks"] = torch.where(ids <= last, ids, -1).contiguous()
        st["lens"] = st["pos"] + st["count"]
        head = (st["pos"] // 64).long()  # the block that the context ends in holds its earlier tokens
        old = _pack(*(normal(units, 64, D).to(torch.bfloat16).float() for _ in range(2)))
        st["store"][torch.arange(units, device="cuda"), head] = old
        st["kv"] = torch.zeros((units, touched, 2, 64, D), dtype=torch.bfloat16, device="cuda")
        return st
    context = case["context"]
    nbc = -(-context // 64)
    lens = _lengths(case, context)
    st |= dict(lens=per_unit(lens), context=context)
    # an evicting store has a row for each block that it may hold, the others one for each block there is
    st["nb"] = nb = case["blocks"] if op == "mass" else nbc
    st["store"] = torch.empty((units, nb, BLOCK), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 14) // nb)
    for u in range(0, units, step):  # a few GB of float32 at a time
        w = min(step, units - u)
        k, v = (normal(w * nb, 64, D).to(torch.bfloat16).float() for _ in range(2))
        st["store"][u:u + w] = _pack(k, v).view(w, nb, BLOCK)
    st["slots"] = None
    if op != "dense":
        # sink, 16 (or fewer) window blocks, the others anywhere between
        most = case["blocks"]
        nbl = ((st["lens"] + 63) // 64)[:, None]
        ids = torch.arange(nbc, dtype=torch.int32, device="cuda")
        rank = torch.rand((units, nbc), generator=gen, device="cuda")
        window = min(16, (most + 3) // 4)
        rank = torch.where((ids == 0) | (ids >= nbl - window), rank + 1, rank)
        rank = torch.where(ids < nbl, rank, -1.0)
        top = torch.topk(rank, min(most, nbc), dim=1)
        picked = torch.where(top.values >= 0, top.indices, nbc).sort(1).values
        sel = torch.full((units, most), -1, dtype=torch.int32, device="cuda")
        sel[:, :picked.shape[1]] = torch.where(picked < nbc, picked, -1)
        if op == "mass":  # rows hold their blocks in any order
            sel = sel.gather(1, torch.rand((units, most), generator=gen, device="cuda").argsort(1)).contiguous()
            st["slots"] = torch.arange(most, dtype=torch.int32, device="cuda").repeat(units, 1)
        st |= dict(sel=sel, n_blocks=most)
    rows = case["group"] * case["queries"]
    q = normal(units, rows, D)
    st["q"] = (q / q.norm(dim=-1, keepdim=True) * math.sqrt(D)).to(torch.bfloat16)
    st["out"] = torch.zeros((units, rows, D), dtype=torch.bfloat16, device="cuda")
    st["mass"] = torch.zeros((units, case["blocks"]), dtype=torch.float32, device="cuda") if op == "mass" else None
    st |= dict(group=case["group"], queries=case["queries"])
    # the header's bound of nosa_byte_scratch_bytes for 256 SMs
    need = 512 + 536 * rows * (units + 4096) + (16 * (rows + 1) * units * case["blocks"] if op == "mass" else 0)
    st["scratch"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def _run_own(st):
    from offloadable_block_sparse_gb300 import nosa as N
    stream = torch.cuda.current_stream().cuda_stream
    op, units = st["op"], st["units"]
    if op == "rope":
        if "table" not in st:  # made once by a program
            c = dict(st["config"])
            kind = dict(none=N.NOSA_ROPE_PLAIN, linear=N.NOSA_ROPE_LINEAR, base=N.NOSA_ROPE_BASE, parts=N.NOSA_ROPE_PARTS)
            st["table"] = N.nosa_rope_make(**(c | dict(scaling=kind[c["scaling"]])))
        x, q, k, hq = st["x"], st["q"], st["k"], st["q"].shape[1]
        N.nosa_rope(st["table"], [(x[:, :, :hq].transpose(1, 2), q), (x[:, :, hq:].transpose(1, 2), k)], pos=st["pos"],
                    count=st["count"], stream=stream)
        return q, k
    if op == "evict":
        N.nosa_evict(st["acc"], st["slot_blk"], st["mass"], units, st["slots"], st["lens"], st["budget"], st["sink"],
                     st["window"], st["decay"], st["acc_out"], st["slot_out"], next_block=st["next"],
                     next_slot=st["row"], stream=stream)
        return st["acc_out"], st["slot_out"], st["row"]
    nb = st["nb"]
    if op == "append":
        N.nosa_byte_append(st["k"], st["v"], st["store"], units, st["n"], nb, pos=st["pos"], count=st["count"],
                          stream=stream)
        N.nosa_byte_read(st["store"], units, nb, st["blocks"], st["n_blocks"], st["kv"], lens=st["lens"], stream=stream)
        return st["kv"]
    if op == "dense":
        N.nosa_byte_dense_attend(st["q"], st["store"], units, st["group"], st["queries"], nb, st["lens"], st["context"],
                                st["out"], st["scratch"], st["scratch"].numel(), stream=stream)
        return st["out"]
    N.nosa_byte_attend(st["q"], st["store"], st["sel"], st["slots"], units, st["group"], st["queries"], nb,
                      st["n_blocks"], st["lens"], st["out"], st["scratch"], st["scratch"].numel(), mass=st["mass"],
                      stream=stream)
    return st["out"] if st["mass"] is None else (st["out"], st["mass"])


def _gather(st, ids, rows=None):
    """The values and scales of blocks ids [units, n] (kept in rows `rows`), and their tokens' positions (-1: none)."""
    ids = ids.long()
    rows = ids if rows is None else rows.long()
    flat = torch.arange(st["units"], device="cuda")[:, None] * st["nb"] + torch.where(ids >= 0, rows, 0)
    k, v, ks, vs = _unpack(st["store"].view(-1, BLOCK)[flat.view(-1)])
    at = ids[:, :, None] * 64 + torch.arange(64, device="cuda")
    at = torch.where((ids[:, :, None] >= 0) & (at < st["lens"][:, None, None]), at, -1)
    return k, v, ks, vs, at


def _plain_rope(st):
    c = st["config"]
    r = c["rot_dims"]
    f = torch.from_numpy(_frequencies(c)).cuda()
    at = st["pos"][:, None] + torch.arange(st["n"], device="cuda")
    angle = at.double()[:, :, None] * f
    cos, sin = (z.float()[:, None] * c["attention_factor"] for z in (torch.cos(angle), torch.sin(angle)))
    x = st["x"].float().transpose(1, 2)
    if c["interleaved"]:
        x1, x2 = x[..., 0:r:2], x[..., 1:r:2]
    else:
        x1, x2 = x[..., :r // 2], x[..., r // 2:r]
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    turned = torch.stack((y1, y2), -1).flatten(-2) if c["interleaved"] else torch.cat((y1, y2), -1)
    y = torch.cat((turned, x[..., r:]), -1)
    real = (torch.arange(st["n"], device="cuda") < st["count"][:, None])[:, None, :, None]
    y = torch.where(real, y, 0.0).to(torch.bfloat16)
    hq = st["q"].shape[1]
    return y[:, :hq].contiguous(), y[:, hq:].contiguous()


def _plain_evict(st):
    blk, slots = st["slot_blk"], st["slots"]
    held = blk >= 0
    acc = st["acc"] * st["decay"] + st["mass"]
    acc = torch.where(held & ~torch.isnan(acc), acc, 0.0)
    nbl = ((st["lens"] + 63) // 64)[:, None]
    free = held & (blk >= st["sink"]) & (blk < nbl - st["window"]) & (blk != st["next"][:, None])
    has = (blk == st["next"][:, None]).any(1)
    over = held.sum(1) + (~has).int() - st["budget"]
    # smallest mass first, of equal ones the later block
    order = torch.argsort(blk, dim=1, descending=True, stable=True)
    key = torch.where(free, acc, math.inf).gather(1, order)
    order = order.gather(1, torch.argsort(key, dim=1, stable=True))
    rank = torch.empty_like(order).scatter_(1, order, torch.arange(slots, device="cuda").expand_as(order).contiguous())
    gone = free & (rank < over[:, None])
    blk = torch.where(gone, -1, blk)
    acc = torch.where(gone, 0.0, acc)
    # the next block takes the lowest empty row
    index = torch.arange(slots, device="cuda")
    empty = torch.where(blk < 0, index, slots).amin(1)
    there = torch.where(blk == st["next"][:, None], index, slots).amin(1)
    row = torch.where(has, there, empty)
    row = torch.where(row < slots, row, -1)
    put = (index == row[:, None]) & ~has[:, None]
    return acc, torch.where(put, st["next"][:, None], blk), row.to(torch.int32)


def _run_plain(st):
    op = st["op"]
    if op == "rope":
        return _plain_rope(st)
    if op == "evict":
        return _plain_evict(st)
    units = st["units"]
    if op == "append":
        ids = st["blocks"]
        k, v, ks, vs, at = _gather(st, ids)
        i = at - st["pos"][:, None, None]
        new = ((i >= 0) & (at >= 0)).view(-1, 64)[:, :, None]
        row = (torch.arange(units, device="cuda")[:, None, None] * st["n"] + i.clamp(0, st["n"] - 1)).view(-1, 64)
        # a block that the call does not begin keeps its tokens, under a scale that is at least its own
        begun = (ids.long() * 64 < st["pos"][:, None]).view(-1)
        got = []
        for old, s, x in ((k, ks, st["k"]), (v, vs, st["v"])):
            x = torch.where(new, x.float().view(-1, D)[row], 0.0)
            s = torch.maximum(torch.where(begun, s, 0.0), _scale(x.abs().amax((1, 2))))
            x = torch.where(new, x, old)
            got.append(_codes(x, s).float() * s[:, None, None])
        kv = torch.where((at >= 0).view(-1, 1, 64, 1), torch.stack(got, 1), 0.0)
        return kv.view(st["kv"].shape).to(torch.bfloat16)
    rows = st["group"] * st["queries"]
    if op == "dense":
        k, v, _, _ = _unpack(st["store"].view(-1, BLOCK))
        at = torch.arange(st["nb"] * 64, device="cuda").expand(units, -1)
        at = torch.where(at < st["lens"][:, None], at, -1)
    else:
        k, v, _, _, at = _gather(st, st["sel"], st["slots"])
    k, v, at = k.view(units, -1, D), v.view(units, -1, D), at.reshape(units, 1, -1)
    # row h * queries + i is query token i of the last `queries` tokens: it sees the tokens up to its own
    late = st["queries"] - 1 - torch.arange(rows, device="cuda") % st["queries"]
    seen = (at >= 0) & (at < (st["lens"][:, None] - late)[:, :, None])
    z = torch.matmul(st["q"].float(), k.transpose(1, 2)) * (1.0 / math.sqrt(D))
    z = z.masked_fill(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    out = (torch.matmul(p, v) / total).to(torch.bfloat16)
    if st["mass"] is None:
        return out
    return out, (p / total).view(units, rows, -1, 64).sum((1, 3))


# ------------------------------------------------------------------------------ work
def work(case):
    """Each byte that has to move once: 256 bytes a token and unit in the store, 512 in bf16."""
    heads = case["heads"]
    if case["op"] == "rope":
        rows = int(_lengths(case, case["tokens"]).sum()) * heads * (case["group"] + 1)
        return {"bytes": rows * 512, "flops": rows * 3 * case["rot"]}
    if case["op"] == "evict":
        slots = case["batch"] * heads * case["slots"]
        return {"bytes": slots * 20, "flops": slots * 4}
    if case["op"] == "append":
        # written, then read back
        tokens = int(_lengths(case, case["tokens"]).sum()) * heads
        return {"bytes": tokens * (512 + 256 + 256 + 512), "flops": tokens * 2 * D * 2}
    lens = _lengths(case, case["context"])
    if "blocks" in case:
        lens = np.minimum(lens, case["blocks"] * 64)
    tokens = int(lens.sum()) * heads
    rows = case["group"] * case["queries"]
    io = case["batch"] * heads * (rows * D * 2 * 2 + (4 * case["blocks"] if case["op"] == "mass" else 0))
    return {"bytes": tokens * 256 + io, "flops": tokens * rows * 4 * D}


# ------------------------------------------------------------------------------ 64 bits
def _round_e4m3(y):
    """y float64, at most 448 in size: to the nearest e4m3 value, ties to even."""
    _, e = torch.frexp(y)  # |y| in [2^(e-1), 2^e)
    step = (((e - 1).clamp(min=-6) - 3 + 1023).long() << 52).view(torch.float64)
    return torch.round(y / step) * step


def _block_values(block):
    """K and V of one block's bytes, float64 [64, 128] each, code by code, and the two scales."""
    size = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    value = torch.tensor(size + [-x for x in size], dtype=torch.float64, device="cuda")
    i, d = torch.arange(64, device="cuda")[:, None], torch.arange(D, device="cuda")[None]
    tile, i = i // 16 * TILE, i % 16
    k_at = tile + i // 8 * 1024 + d % 32 // 16 * 512 + (i % 8 * 4 + d // 32) * 16 + d % 16
    v_at = (tile + 2048 + d % 16 // 4 * 512 + (d // 16 * 4 + i % 8 // 2) * 16 + d % 4 // 2 * 8 + i // 8 * 4 + d % 2 * 2
            + i % 2)
    s = block[:, 4 * TILE:4 * TILE + 8].contiguous().view(torch.float32).double()
    return (value[block[:, k_at].long()] * s[:, :1, None], value[block[:, v_at].long()] * s[:, 1:, None], s)


def exact(case, seed):
    st = prepare(case, seed)
    units = st["units"]
    if st["op"] == "rope":
        c, n = st["config"], st["n"]
        r, f = c["rot_dims"], torch.from_numpy(_frequencies(c)).cuda()
        y = st["x"].double().permute(0, 2, 1, 3).contiguous()
        a = torch.arange(r // 2, device="cuda")
        one, two = (2 * a, 2 * a + 1) if c["interleaved"] else (a, a + r // 2)
        for b in range(y.shape[0]):
            angle = (int(st["pos"][b]) + torch.arange(n, dtype=torch.float64, device="cuda"))[:, None] * f
            z = torch.polar(torch.full_like(angle, c["attention_factor"]), angle)
            z = torch.complex(y[b][:, :, one], y[b][:, :, two]) * z
            y[b][:, :, one], y[b][:, :, two] = z.real, z.imag
            y[b][:, int(st["count"][b]):] = 0
        hq = st["q"].shape[1]
        return y[:, :hq].contiguous(), y[:, hq:].contiguous()
    if st["op"] == "evict":
        blk, acc, mass = (st[x].cpu().numpy() for x in ("slot_blk", "acc", "mass"))
        lens, nxt = st["lens"].cpu().numpy(), st["next"].cpu().numpy()
        # the order is decided on the sums as float32 holds them
        rank = acc * np.float32(st["decay"]) + mass
        out = acc.astype(np.float64) * float(np.float32(st["decay"])) + mass
        out[blk < 0] = 0
        for u in range(units):
            last = -(-int(lens[u]) // 64) - st["window"]
            may = [s for s in range(st["slots"]) if st["sink"] <= blk[u, s] < last and blk[u, s] != nxt[u]]
            over = int((blk[u] >= 0).sum()) + int(nxt[u] not in blk[u]) - st["budget"]
            for s in sorted(may, key=lambda s: (rank[u, s], -blk[u, s]))[:max(over, 0)]:
                out[u, s] = 0
        return torch.from_numpy(out).cuda(), None, None
    store, lens = st["store"], st["lens"].tolist()
    if st["op"] == "append":
        out = torch.zeros(st["kv"].shape, dtype=torch.float64, device="cuda")
        blocks, poss, counts = (st[x].tolist() for x in ("blocks", "pos", "count"))
        for u in range(units):
            p, c = poss[u], counts[u]
            for j, b in enumerate(blocks[u]):
                if b < 0:
                    continue
                lo, hi = max(p, 64 * b), min(p + c, 64 * b + 64)
                k, v, s = _block_values(store[u, b][None])
                for n, (old, new) in enumerate(((k, st["k"]), (v, st["v"]))):
                    x = old[0].clone() if 64 * b < p else torch.zeros_like(old[0])
                    have = float(s[0, n]) if 64 * b < p else 0.0
                    x[lo - 64 * b:hi - 64 * b] = new[u, lo - p:hi - p].double()
                    top = float(new[u, lo - p:hi - p].double().abs().max())
                    need = 2.0 ** max(math.ceil(math.log2(top / 448)), LEAST) if top > 0 else 0.0
                    scale = max(have, need)
                    x = _round_e4m3(x / scale) * scale if scale > 0 else 0 * x
                    x[max(0, lens[u] - 64 * b):] = 0
                    out[u, j, n] = x
        return out
    nq, rows = st["queries"], st["group"] * st["queries"]
    out = torch.zeros((units, rows, D), dtype=torch.float64, device="cuda")
    mass = None if st["mass"] is None else torch.zeros(st["mass"].shape, dtype=torch.float64, device="cuda")
    for u in range(units):
        ids = torch.arange(st["nb"], device="cuda") if st["op"] == "dense" else st["sel"][u].long()
        which = torch.nonzero(ids >= 0)[:, 0]
        ids = ids[which]
        held = ids if st["slots"] is None else st["slots"][u].long()[which]
        k, v, _ = _block_values(store[u, held])
        k, v = k.view(-1, D), v.view(-1, D)
        at = (ids[:, None] * 64 + torch.arange(64, device="cuda")).view(-1)
        for late in range(nq):
            see = at < lens[u] - late
            if not bool(see.any()):
                continue
            r = torch.arange(nq - 1 - late, rows, nq, device="cuda")
            z = (st["q"][u, r].double() @ k.T / math.sqrt(D)).masked_fill(~see, -math.inf)
            w = torch.softmax(z, dim=-1)
            out[u, r] = w @ v
            if mass is not None:
                mass[u, which] += w.view(len(r), -1, 64).sum((0, 2))
    return out if mass is None else (out, mass)
