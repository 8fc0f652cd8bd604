"""Plain definitions, in 64 bits on the host, of the 4-bit format, the product, the layer from
4-bit tables, the table lookup and its gradient. Shares no code with the library."""
from __future__ import annotations

import numpy as np

import oracle

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BF16_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -24  # half a rounding step, relative to the value


def quantise(x: np.ndarray):
    """Codes [R, C] (one a byte) and scale bytes [R, C / 32] of x [R, C] (float64 values)."""
    R, C = x.shape
    b = x.reshape(R, C // 32, 32)
    codes = np.zeros(b.shape, np.uint8)
    scales = np.zeros(b.shape[:2], np.uint8)
    for r in range(R):
        for k in range(C // 32):
            blk = b[r, k]
            if not np.isfinite(blk).all():
                scales[r, k] = 255
                continue
            amax = np.abs(blk).max()
            e = 0
            if amax > 0:
                e = int(np.clip(int(np.frexp(amax)[1]) - 1 - 2, -127, 127)) + 127
            scales[r, k] = e
            y = blk / 2.0 ** (e - 127)
            # nearest magnitude; of two equally near, the one whose code is even
            dist = np.abs(np.abs(y)[:, None] - MAGNITUDES[None, :])
            near = dist == dist.min(axis=1, keepdims=True)
            even = near & (np.arange(8) % 2 == 0)[None, :]
            pick = np.where(even.any(axis=1), even.argmax(axis=1), near.argmax(axis=1))
            codes[r, k] = pick | (np.signbit(y).astype(np.uint8) << 3)
    return codes.reshape(R, C), scales


def pack(codes: np.ndarray) -> np.ndarray:
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty((packed.shape[0], packed.shape[1] * 2), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of codes [R, C] (one a byte) under scales [R, C / 32]."""
    m = MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return m * np.repeat(s, 32, axis=1)


def tile_bytes(scales: np.ndarray, fill=0) -> np.ndarray:
    """Row-major scales in 128 x 4 tiles, by the layout's formula."""
    R, B = scales.shape
    kt = -(-B // 4)
    out = np.full(-(-R // 128) * kt * 512, fill, np.uint8)
    for r in range(R):
        for b in range(kt * 4):
            at = (r // 128 * kt + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
            out[at] = scales[r, b] if b < B else 0
    return out


def random_mx4(rng, rows: int, cols: int, spread: int = 4):
    """Random codes (one a byte) and scale bytes around 1."""
    return (rng.integers(0, 16, (rows, cols), dtype=np.uint8),
            rng.integers(127 - spread, 127 + spread + 1, (rows, cols // 32), dtype=np.uint8))


def product_bound(a: np.ndarray, b: np.ndarray, half: float, want: np.ndarray) -> np.ndarray:
    """|error| of an fp32 sum of K exact products in any order, one rounding of the result:
    K - 1 additions, each off by at most a unit of 2^-23 (round to nearest halves that; the
    tensor cores may truncate) of a partial sum no larger than sum |a||b|; then half a step of
    the output type."""
    s = np.abs(a) @ np.abs(b).T
    acc = a.shape[1] * 2.0 ** -23 * s
    return acc + half * (np.abs(want) + acc)


def layer(cfg_v0, N, K, V, tokens, offsets, E0, E_vals, W_vals, histories=None, out_scale=1.0):
    """Eq. 2 and Eq. 3 on float64 tables; also the bound of the fp32 sums and the indices."""
    S = (N - 1) * K
    win = oracle.context_windows(N, tokens, offsets, histories=histories)
    idx = oracle.hash_indices(cfg_v0, N, K, V, win)
    G = np.concatenate([E_vals[s][idx[:, s]] for s in range(S)], axis=1)
    c = out_scale / (S + 1)
    y = G @ W_vals.T
    e0 = E0[np.asarray(tokens)]
    # the products' sums, the E_0 add, the scale (rounded to fp32) and its product: one 2^-24 each
    mag = np.abs(G) @ np.abs(W_vals).T
    acc = (G.shape[1] * 2.0 ** -23 * mag + 3 * F32_HALF * (mag + np.abs(e0))) * abs(c)
    return (e0 + y) * c, acc, idx


def lookup(values_: np.ndarray, ids: np.ndarray, scale: float, pad_id: int = -1) -> np.ndarray:
    out = values_[np.clip(ids, 0, None)] * np.float64(np.float32(scale))
    out[(ids == pad_id) & (pad_id >= 0)] = 0.0
    return out


def grad_rows(ids: np.ndarray, g: np.ndarray, scale: float, pad_id: int = -1):
    """Distinct ids ascending, their gradient rows, and the sums of magnitudes and counts."""
    keep = ~((ids == pad_id) & (pad_id >= 0))
    rows, where, count = np.unique(ids[keep], return_inverse=True, return_counts=True)
    s = np.float64(np.float32(scale))
    grads = np.zeros((len(rows), g.shape[1]))
    mags = np.zeros_like(grads)
    np.add.at(grads, where, g[keep])
    np.add.at(mags, where, np.abs(g[keep]))
    return rows, grads * s, mags * abs(s), count


def grad_bound(mags: np.ndarray, count: np.ndarray) -> np.ndarray:
    """count - 1 fp32 additions and the scale's product, each off by at most 2^-24 of the sum
    of magnitudes (second-order terms: under count * 2^-24 of that, covered by the + 1)."""
    return (count[:, None] + 1) * F32_HALF * mags
