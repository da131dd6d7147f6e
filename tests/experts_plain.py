"""The expert operators in plain numpy, 64 bits, from their definitions."""
import numpy as np

# half a unit in the last place, relative: 8, 11 and 24 significant bits
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def up(n, m):
    return -(-n // m) * m


def route(ids, experts, align):
    """(offsets, counts, row, slots of the rows 0..offsets[-1]-1), slot by slot."""
    flat = [int(v) for v in np.asarray(ids).reshape(-1)]
    members = [[i for i, v in enumerate(flat) if v == e] for e in range(experts)]
    offsets, slots, row = [0], [], [-1] * len(flat)
    for m in members:
        for j, i in enumerate(m):
            row[i] = offsets[-1] + j
        slots += m + [-1] * (up(len(m), align) - len(m))
        offsets.append(len(slots))
    return (np.array(offsets), np.array([len(m) for m in members]),
            np.array(row, dtype=np.int64).reshape(np.asarray(ids).shape), np.array(slots, dtype=np.int64))


def e4m3_values():
    """The value of each of the 256 bytes (NaN at 0x7F and 0xFF)."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        v[b] = np.nan if b & 127 == 127 else -x if b & 128 else x
    return v


E4M3 = e4m3_values()


def e4m3_bytes(x):
    """Nearest E4M3 byte of |x| <= 448 (ties to the even byte), 0x7F for NaN."""
    grid = E4M3[:127]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(grid, np.nan_to_num(a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, above = np.nan_to_num(a) - grid[lo], grid[hi] - np.nan_to_num(a)
    b = np.where(down < above, lo, np.where(above < down, hi, np.where(lo % 2 == 0, lo, hi)))
    b = np.where(grid[hi] == a, hi, b).astype(np.uint8)
    b = b | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), 0x7F, b).astype(np.uint8)


def scale_byte(top):
    """Of the least power of two s with top <= 448 s, at least 2^-126."""
    if top == 0:
        return 127
    b = 1
    while top > 448 * 2.0 ** (b - 127):
        b += 1
    return b


def cast_block(x):
    """(bytes, scale byte) of one block of any shape."""
    finite = np.isfinite(x)
    b = scale_byte(np.abs(np.where(finite, x, 0)).max(initial=0))
    return e4m3_bytes(np.where(finite, x, np.nan) / 2.0 ** (b - 127)), b


def cast(x, block_rows=1):
    """Blocks of block_rows x 128 of a 2-D matrix: (data bytes, scale bytes)
    as stored."""
    rows, cols = x.shape
    kb = up(cols, 128) // 128
    data = np.zeros((rows, kb * 128), np.uint8)
    scale = np.full((up(rows, block_rows) // block_rows, up(kb, 4)), 127, np.uint8)
    for r in range(0, rows, block_rows):
        for b in range(kb):
            q, s = cast_block(x[r:r + block_rows, b * 128:(b + 1) * 128])
            data[r:r + block_rows, b * 128:b * 128 + q.shape[1]] = q
            scale[r // block_rows, b] = s
    return data, scale


def values(data, scale, block_rows=1):
    """What stored blocks stand for."""
    s = 2.0 ** (scale[:, :data.shape[1] // 128].astype(np.float64) - 127)
    s = np.repeat(np.repeat(s, 128, 1), block_rows, 0)[:data.shape[0]]
    return E4M3[data] * s


def unit_bound(a, w):
    """How far the matrix unit's A W^T may be from exact, for A [rows, k] and
    W [n, k] as values of 8-bit blocks.  The unit adds the products of 8
    neighbouring k at a time, each cut toward zero to a multiple of 2^-13 of
    the group's largest power of two (measured: beside 2^16 in its group 2^3
    counts and 2^2 does not, whatever the signs; in another group 2^-7 does),
    and the groups in 32 bits.  So a group is off by less than 7 * 2^-13 of
    its largest product, and the K/8 sums by 2^-23 each of what they hold."""
    bound = np.zeros((a.shape[0], w.shape[0]))
    for k in range(0, a.shape[1], 8):
        p = np.abs(a[:, None, k:k + 8] * w[None, :, k:k + 8])
        bound += 7 * 2.0 ** -13 * p.max(-1)
    return bound + a.shape[1] / 8 * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)
