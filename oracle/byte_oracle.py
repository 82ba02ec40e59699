"""Oracle of the 8-bit KV block store, of eviction and of rotary positions (include/nosa.h, nosa_byte_append and what
follows it): their definitions in float64 NumPy, for the tests.  Shares no code with the kernels or the binding."""
from __future__ import annotations

import math

import numpy as np

BLOCK_BYTES = 16512
TILE_BYTES = 4096
SCALES = 4 * TILE_BYTES
LEAST, MOST = -118, 119

# what each code stands for under a scale of 1
E4M3 = np.array([s * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)) for s in (1, -1) for e in range(16) for m in range(8)])
E4M3[0x7F] = E4M3[0xFF] = np.nan


def encode(y):
    """float64 y: e4m3 codes, to nearest, ties to even; sizes above 448 become 448, NaN and infinities 0x7F."""
    y = np.asarray(y, np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(y), y, 0)), 448.0)
    e = np.maximum(np.frexp(a)[1] - 1, -6)
    n = np.rint(a / np.exp2(e - 3.0)).astype(np.int64)  # 8 .. 16 of a normal, 0 .. 8 of a subnormal
    code = np.where(n >= 8, (e + 7) * 8 + n - 8, n)     # 16 carries into the next exponent
    code = np.where(np.isfinite(y), code | np.where(np.signbit(y), 0x80, 0), 0x7F)
    return code.astype(np.uint8)


def need(x):
    """The scale for finite values of x: the smallest power of two s with |x| <= 448 s, within the range; 0 for zeros."""
    x = np.abs(x[np.isfinite(x)])
    if not x.size or x.max() == 0:
        return 0.0
    m, e = math.frexp(float(x.max()) / 448.0)
    return 2.0 ** min(max(e - (m == 0.5), LEAST), MOST)


def place(kind, i, d):
    """Byte within the tile of the code of dim d of the tile's token i; kind 'k' or 'v'."""
    if kind == "k":
        return 1024 * (i // 8) + 512 * ((d % 32) // 16) + 16 * (4 * (i % 8) + d // 32) + d % 16
    return (2048 + 512 * ((d % 16) // 4) + 16 * (4 * (d // 16) + (i % 8) // 2) + 8 * ((d % 4) // 2) + 4 * (i // 8)
            + 2 * (d % 2) + i % 2)


_T, _D = np.arange(64)[:, None], np.arange(128)[None]
AT = {kind: _T // 16 * TILE_BYTES + place(kind, _T % 16, _D) for kind in "kv"}  # [64][128] bytes of a block


def scales(block):
    return np.ascontiguousarray(block[..., SCALES:SCALES + 8]).view(np.float32)


def pack(k, v):
    """k, v float64 [N, 64, 128]: N whole blocks, uint8 [N, 16512]."""
    out = np.zeros((k.shape[0], BLOCK_BYTES), np.uint8)
    for n in range(k.shape[0]):
        s = [need(x[n]) for x in (k, v)]
        for kind, x, f in zip("kv", (k, v), s):
            out[n, AT[kind]] = encode(x[n] / (f or 1.0))
        out[n, SCALES:SCALES + 8] = np.array(s, np.float32).view(np.uint8)
    return out


def unpack(blocks):
    """Blocks uint8 [N, 16512]: (K, V), float64 [N, 64, 128] each."""
    s = scales(blocks).astype(np.float64)
    with np.errstate(invalid="ignore"):
        return tuple(E4M3[blocks[:, AT[kind]]] * s[:, i, None, None] for i, kind in enumerate("kv"))


def append(store, k, v, pos, count, slot_blk=None):
    """store uint8 [U][nb][16512], k and v float64 [U][n][128]; writes in place.  Returns whether a position or a count
    was out of range, or no row held a block."""
    units, nb = store.shape[:2]
    flag = False
    for u in range(units):
        p, c = int(pos[u]), min(max(int(count[u]), 0), k.shape[1])
        flag |= c != int(count[u])
        for b in sorted({(p + j) // 64 for j in range(c)}):
            if slot_blk is None:
                row = b
            else:
                rows = np.nonzero(slot_blk[u] == b)[0] if b >= 0 else []
                row = int(rows[0]) if len(rows) else nb
            if not (b >= 0 and 0 <= row < nb):
                flag = True
                continue
            lo, hi = max(p, 64 * b), min(p + c, 64 * b + 64)
            block = store[u, row]
            for kind, x, at in zip("kv", (k, v), (SCALES, SCALES + 4)):
                new = x[u, lo - p:hi - p]
                had = float(block[at:at + 4].view(np.float32)[0]) if lo > 64 * b else 0.0
                m = math.frexp(had)[0] if math.isfinite(had) else 0.0
                had = had if m == 0.5 and 2.0 ** LEAST <= had <= 2.0 ** MOST else 0.0
                s = max(had, need(new))
                if had and s > had:
                    block[AT[kind]] = encode(E4M3[block[AT[kind]]] * (had / s))
                block[AT[kind][lo - 64 * b:hi - 64 * b]] = encode(new / (s or 1.0))
                block[at:at + 4] = np.array([s], np.float32).view(np.uint8)
    return flag


def attend(q, k, v, at, length, nq, scale):
    """One unit: q [R, 128] (row r is query token r % nq), k, v float64 [n, 64, 128] and their blocks' numbers at [n] (-1:
    none).  The result [R, 128] and the blocks' masses [n]; NaN where a value that a row sees is one."""
    out, mass = np.zeros(q.shape), np.zeros(len(at))
    token = np.asarray(at)[:, None] * 64 + np.arange(64)
    for r in range(q.shape[0]):
        see = (np.asarray(at)[:, None] >= 0) & (token < length - (nq - 1 - r % nq))
        if not see.any():
            continue
        with np.errstate(all="ignore"):
            z = k[see] @ q[r] * scale
            w = np.exp(z - z.max())
            w = w / w.sum()
            out[r] = w @ v[see]
        full = np.zeros(see.shape)
        full[see] = w
        mass += full.sum(1)
    return out, mass


def evict(acc, slot_blk, mass, lens, budget, sink, window, decay, next_block=None):
    """acc float32, slot_blk [U][slots]: (acc, slot_blk, next_slot, whether a next block found no row)."""
    acc, blk = acc.astype(np.float32).copy(), slot_blk.copy()
    units, slots = blk.shape
    row, flag = np.full(units, -1, np.int64), False
    for u in range(units):
        a = np.float32(decay) * acc[u]
        if mass is not None:
            a = a + mass[u]
        a = np.where((blk[u] >= 0) & ~np.isnan(a), a, np.float32(0))
        nxt = -1 if next_block is None else int(next_block[u])
        last = math.inf if lens is None else -(-max(int(lens[u]), 0) // 64) - window
        free = [s for s in range(slots) if blk[u, s] >= 0 and sink <= blk[u, s] < last and blk[u, s] != nxt]
        wants = nxt >= 0 and nxt not in blk[u]
        over = int((blk[u] >= 0).sum()) + wants - budget
        for s in sorted(free, key=lambda s: (a[s], -int(blk[u, s])))[:max(over, 0)]:
            blk[u, s], a[s] = -1, 0
        blk[u] = np.where(blk[u] < 0, -1, blk[u])
        if wants:
            empty = np.nonzero(blk[u] < 0)[0]
            if len(empty):
                row[u] = empty[0]
                blk[u, row[u]] = nxt
            else:
                flag = True
        elif nxt >= 0:
            row[u] = np.nonzero(blk[u] == nxt)[0][0]
        acc[u] = a
    return acc, blk, row, flag


PLAIN, LINEAR, BASE, PARTS = range(4)


def frequencies(rot, scaling=PLAIN, base=10000.0, factor=1.0, low=1.0, high=32.0, original=0.0):
    """Radians per position of each pair."""
    if scaling == BASE and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == LINEAR:
        f = f / factor
    if scaling == PARTS:
        g = np.clip((original * f / (2 * math.pi) - low) / (high - low), 0, 1)
        f = f * (g + (1 - g) / factor)
    return f


def rope(x, pos, f, interleaved, attention_factor=1.0, inverse=False):
    """x float64 [batch][heads][n][128], pos [batch]: rotated."""
    r, y = 2 * len(f), x.copy()
    one = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    two = one + (1 if interleaved else r // 2)
    for b in range(x.shape[0]):
        angle = (np.float64(pos[b]) + np.arange(x.shape[2]))[:, None] * f
        c, s = np.cos(angle), np.sin(angle) * (-1 if inverse else 1)
        y[b][..., one] = attention_factor * (x[b][..., one] * c - x[b][..., two] * s)
        y[b][..., two] = attention_factor * (x[b][..., two] * c + x[b][..., one] * s)
    return y
