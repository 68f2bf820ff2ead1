"""Plain 64-bit implementations of the key/value cache and the tree attention, on the CPU, for the tests.

The cache is held here as f16 values per (sequence, slot); ``pack`` lays them out in pages and ``unpack`` reads
pages byte by byte, from the documented layout, without the library.
"""
import numpy as np

PAGE = 64


def q8_0(x):
    """fp32 [..., D] -> codes int8 [..., D], scales f16 [..., D/32]: d = amax/127, code = round_half_away(x/d)."""
    v = x.astype(np.float32).reshape(*x.shape[:-1], -1, 32)
    d = (np.abs(v).max(-1, keepdims=True) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(d == 0, np.float32(0), v / d).astype(np.float32)
    a = np.abs(q)
    fl = np.floor(a)
    code = np.where(a - fl >= 0.5, fl + 1, fl).clip(0, 127) * np.sign(q)
    return code.astype(np.int8).reshape(x.shape), d[..., 0].astype(np.float16)


def q8_0_values(code, d):
    v = code.reshape(*code.shape[:-1], -1, 32).astype(np.float32) * d[..., None].astype(np.float32)
    return v.astype(np.float16).reshape(code.shape)


def stored(x, ctype):
    """fp32 -> the f16 values that a cache of this type holds of it."""
    return x.astype(np.float16) if ctype == "f16" else q8_0_values(*q8_0(x))


def block_bytes(ctype, D):
    return PAGE * D * 4 if ctype == "f16" else PAGE * (2 * D + D // 8)


def _place(ctype, D, r, d):
    if ctype == "f16":
        return (d // 64) * PAGE * 128 + r * 128 + (((d % 64) // 8) ^ (r % 8)) * 16 + (d % 8) * 2
    swap = r % 8 if D == 128 else (r // 2) % 4
    return r * D + ((d // 16) ^ swap) * 16 + d % 16


def places(ctype, D):
    """(byte of every [row, element], V's offset, byte of every [row, scale] of K, V's scale offset)."""
    r, d = np.arange(PAGE)[:, None], np.arange(D)[None, :]
    if ctype == "f16":
        return _place(ctype, D, r, d), PAGE * D * 2, None, 0
    return (_place(ctype, D, r, d), PAGE * D, 2 * PAGE * D + (r * (D // 32) + np.arange(D // 32)[None, :]) * 2,
            PAGE * (D // 32) * 2)


def unpack(block, ctype, D):
    """One block's bytes -> K, V f16 [64, D]."""
    at, voff, sc, soff = places(ctype, D)
    half = block.view(np.float16)
    out = []
    for v in (0, 1):
        if ctype == "f16":
            out.append(half[(at + v * voff) // 2])
        else:
            code = (block[at + v * voff].astype(np.int16) - 128).astype(np.int8)
            out.append(q8_0_values(code, half[(sc + v * soff) // 2]))
    return out


def pack(K, V, ctype):
    """K, V fp32 [64, D] -> one block's bytes."""
    D = K.shape[1]
    at, voff, sc, soff = places(ctype, D)
    block = np.zeros(block_bytes(ctype, D), dtype=np.uint8)
    half = block.view(np.float16)
    for v, x in ((0, K), (1, V)):
        if ctype == "f16":
            half[(at + v * voff) // 2] = x.astype(np.float16)
        else:
            code, d = q8_0(x)
            block[at + v * voff] = (code.astype(np.int16) + 128).astype(np.uint8)
            half[(sc + v * soff) // 2] = d
    return block


def build(K, V, ctype, rng, spare=2, garbage=None):
    """K, V: lists (one per sequence) of fp32 [len, Hkv, D] -> (pages uint8 [n_pages, Hkv, block], table int32).

    Pages are handed out in random order; unused slots hold ``garbage`` (default: NaN scales or values)."""
    Hkv, D = K[0].shape[1:]
    need = [-(-max(1, k.shape[0]) // PAGE) for k in K]
    n = sum(need) + spare
    pages = np.zeros((n, Hkv, block_bytes(ctype, D)), dtype=np.uint8)
    order = rng.permutation(n)
    table = np.full((len(K), max(need) + 1), -7, dtype=np.int32)
    bad = np.float32(np.nan) if garbage is None else np.float32(garbage)
    at = 0
    for s, (k, v) in enumerate(zip(K, V)):
        for i in range(need[s]):
            p = order[at]
            at += 1
            table[s, i] = p
            for h in range(Hkv):
                kk, vv = np.full((PAGE, D), bad, np.float32), np.full((PAGE, D), bad, np.float32)
                part = k[i * PAGE:(i + 1) * PAGE, h]
                kk[:len(part)], vv[:len(part)] = part, v[i * PAGE:(i + 1) * PAGE, h]
                with np.errstate(invalid="ignore"):
                    pages[p, h] = pack(kk, vv, ctype)
    return pages, table


def norm_rope(x, w, eps, pos, inv_freq, interleaved):
    """x float64 [n, heads, D] -> normed (w or None) and rotated, float64."""
    x = x.astype(np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    if inv_freq is not None and len(inv_freq):
        h = len(inv_freq)
        t = pos.astype(np.float64)[:, None, None] * inv_freq.astype(np.float64)
        i = np.arange(h)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        y = x.copy()
        y[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
        y[..., b] = x[..., b] * np.cos(t) + x[..., a] * np.sin(t)
        x = y
    return x


def attention(q, K, V, ctx, mask, scale):
    """q f16 [T, Hq, D]; K, V f16 [ctx + T, Hkv, D]; mask: per node, an int of bits.

    Returns float64 out [T, Hq, D], A = sum p|v| / sum p of the same shape, and the largest sum |q||k| * |scale| over
    the seen keys [T, Hq, 1]: what the error bound of a 32-bit computation goes by."""
    T, Hq, D = q.shape
    G = Hq // K.shape[1]
    out, A, big = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq, 1))
    for i in range(T):
        see = list(range(ctx)) + [ctx + j for j in range(K.shape[0] - ctx) if (int(mask[i]) >> j) & 1]
        if not see:
            continue
        k, v = K[see].astype(np.float64), V[see].astype(np.float64)
        for h in range(Hq):
            qh = q[i, h].astype(np.float64)
            s = k[:, h // G] @ qh * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h], A[i, h] = p @ v[:, h // G], p @ np.abs(v[:, h // G])
            big[i, h] = (np.abs(k[:, h // G]) @ np.abs(qh)).max() * abs(scale)
    return out, A, big
