"""Oracle of the 4-bit KV block store (include/nosa.h, nosa_quant_append): its definition in float64
NumPy, byte by byte, for the tests.  Shares no code with the kernels or the binding."""
from __future__ import annotations

import numpy as np

BLOCK_BYTES = 10240
TILE_BYTES = 2560


def quantise(x):
    """x [..., 128] float64: codes uint8 [..., 128], s and m float16 [..., 4]."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], 4, 32)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)  # NaN is handed on
        # extremes are bf16, so their float32 difference is what the definition divides
        m = lo.astype(np.float16)
        s = ((hi - lo).astype(np.float32).astype(np.float64) / 15).astype(np.float16)
        bad = ~(np.isfinite(m) & np.isfinite(s))
        m[bad] = np.nan
        s[bad] = np.nan
        n = np.rint((g - m.astype(np.float64)[..., None]) / s.astype(np.float64)[..., None])
        n = np.where(s[..., None] > 0, np.clip(n, 0, 15), 0)
    return n.astype(np.uint8).reshape(x.shape), s, m


def values(codes, s, m):
    """What codes [..., 128] with s, m [..., 4] stand for, float64."""
    wide = lambda a: np.repeat(a.astype(np.float64), 32, axis=-1)  # noqa: E731
    return codes.astype(np.float64) * wide(s) + wide(m)


def code_place(kind, i, d):
    """(byte within the tile, shift) of the code of dim d of the tile's token i; kind 'k' or 'v'."""
    if kind == "k":
        return 64 * i + 16 * ((d % 32) // 8) + 4 * (d // 32) + (d % 8) // 2, 4 * (d % 2)
    return (1024 + 512 * (i // 8) + 64 * ((d % 32) // 4) + 16 * ((i % 8) // 2) + 4 * (d // 32) + 2 * (i % 2)
            + (d % 4) // 2, 4 * (d % 2))


def scale_place(kind, which, i, gr):
    """Byte within the tile of group gr's s (which = 0) or m (1) of the tile's token i."""
    if kind == "k":
        return 2048 + 16 * i + 8 * which + 2 * gr
    return 2304 + 128 * which + 16 * (i // 2) + 4 * gr + 2 * (i % 2)


_I, _D = np.arange(16)[:, None], np.arange(128)[None, :]
_G = np.arange(4)[None, :]


def write_token(block, kind, row, codes, s, m):
    """Writes one token's row (0..63) into a block uint8 [10240]."""
    base, i = TILE_BYTES * (row // 16), row % 16
    byte, shift = code_place(kind, i, np.arange(128))
    for d in range(128):
        at = base + byte[d]
        block[at] = (int(block[at]) & ~(15 << shift[d]) & 255) | int(codes[d]) << shift[d]
    for gr in range(4):
        for which, a in ((0, s), (1, m)):
            at = base + scale_place(kind, which, i, gr)
            block[at:at + 2] = np.asarray([a[gr]], np.float16).view(np.uint8)


def append(store, k, v, pos, count):
    """store uint8 [U][nb][10240], k and v float64 [U][n][128]; writes in place.  Returns whether a
    position or a count was out of range."""
    units, nb = store.shape[:2]
    flag = False
    for u in range(units):
        c = min(max(int(count[u]), 0), k.shape[1])
        flag |= c != int(count[u])
        q = [quantise(x[u, :c]) for x in (k, v)]
        for j in range(c):
            p = int(pos[u]) + j
            if not 0 <= p < 64 * nb:
                flag = True
                continue
            for kind, (codes, s, m) in zip("kv", q):
                write_token(store[u, p // 64], kind, p % 64, codes[j], s[j], m[j])
    return flag


def pack(k, v):
    """k, v float64 [N, 64, 128]: N whole blocks, uint8 [N, 10240]."""
    out = np.zeros((k.shape[0], 4, TILE_BYTES), np.uint8)
    for kind, x in (("k", k), ("v", v)):
        codes, s, m = quantise(x)
        byte, shift = np.broadcast_arrays(*code_place(kind, _I, _D))
        c = (codes.reshape(-1, 4, 16, 128) << shift).astype(np.uint8)
        for low in (0, 1):  # each byte has an even and an odd dim
            out[:, :, byte[:, low::2]] |= c[..., low::2]
        for which, a in ((0, s), (1, m)):
            at = np.broadcast_arrays(scale_place(kind, which, _I, _G), np.zeros((16, 4)))[0].astype(int)
            b = np.ascontiguousarray(a.reshape(-1, 4, 16, 4)).view(np.uint8).reshape(-1, 4, 16, 4, 2)
            out[:, :, at] = b[..., 0]
            out[:, :, at + 1] = b[..., 1]
    return out.reshape(-1, BLOCK_BYTES)


def unpack(blocks):
    """Blocks uint8 [N, 10240]: K and V values and the groups' magnitudes: float64 [N, 64, 128] each, as
    (K, V, |n s| + |m| of K, of V)."""
    t = blocks.reshape(-1, 4, TILE_BYTES)
    got, size = [], []
    for kind in "kv":
        byte, shift = np.broadcast_arrays(*code_place(kind, _I, _D))
        codes = (t[:, :, byte] >> shift) & 15
        sm = []
        for which in (0, 1):
            at = np.broadcast_arrays(scale_place(kind, which, _I, _G), np.zeros((16, 4)))[0].astype(int)
            b = np.stack((t[:, :, at], t[:, :, at + 1]), -1)
            sm.append(np.repeat(np.ascontiguousarray(b).view(np.float16)[..., 0].astype(np.float64), 32, -1))
        got.append((codes * sm[0] + sm[1]).reshape(-1, 64, 128))
        size.append((codes * np.abs(sm[0]) + np.abs(sm[1])).reshape(-1, 64, 128))
    return got[0], got[1], size[0], size[1]


def attend(q, k, v, seen, scale):
    """q [R, 128], k and v [N, 128] float64, seen bool [R, N]: softmax attention of each row over the
    tokens it sees (zeros for none).  Values of tokens that a row does not see do not enter."""
    out = np.zeros(q.shape)
    for r in range(q.shape[0]):
        i = np.nonzero(seen[r])[0]
        if i.size:
            z = k[i] @ q[r] * scale
            with np.errstate(all="ignore"):
                p = np.exp(z - z.max())
                out[r] = p @ v[i] / p.sum()
    return out
