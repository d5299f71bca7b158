"""The rotation of rows and the cache held in 4 bits.

Test infrastructure only (see ``oracle/__init__``).

Reading: a code is a sign and one of eight magnitudes.  A number goes to the
nearest one of its unit's multiples, of two equally near to the one with the even
code; numbers beyond the last magnitude go to the last.  The unit of 32 channels of
a key is the least power of two (2^-127 at least) of which 7 are no less than the
largest magnitude; that of a value row is a sixth of its largest magnitude, in
float32 and then in 8 significant bits.  What is not finite makes its unit NaN.
"""

import math
from fractions import Fraction

import numpy as np

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def rotate(rows, positions, cos_sin, interleaved):
    """float64 rows [T, heads, dim], each turned by its position's angles."""
    x = np.array(rows, dtype=np.float64)
    rot = np.shape(cos_sin)[1]
    half = rot // 2
    out = x.copy()
    for t, p in enumerate(positions):
        if not 0 <= p < len(cos_sin):
            continue
        for i in range(half):
            c, s = float(cos_sin[p][i]), float(cos_sin[p][half + i])
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
            out[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            out[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return out


def code(x, unit):
    """The code of one finite number for a positive unit."""
    size = abs(Fraction(float(x))) / Fraction(float(unit))
    gaps = [abs(Fraction(m) - size) for m in MAGNITUDES]
    best = min(gaps)
    near = [i for i, g in enumerate(gaps) if g == best]
    pick = near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1]
    if size > 6:
        pick = 7
    return pick + (8 if math.copysign(1.0, x) < 0 else 0)


def key_unit(group):
    """The unit's byte (its exponent + 127; 255: NaN) of 32 channels."""
    if not np.isfinite(group).all():
        return 255
    top = Fraction(float(np.abs(group).max()))
    byte = 0
    while byte < 254 and top > 7 * Fraction(2) ** (byte - 127):
        byte += 1
    return byte


def value_unit(row):
    """The unit of a value row (a float32 number of 8 significant bits, NaN, or 0)."""
    if not np.isfinite(row).all():
        return np.float32(np.nan)
    sixth = np.float32(Fraction(float(np.abs(row).max())) / 6)
    # to 8 significant bits (never fewer than bfloat16's own smallest step), ties to even
    if sixth == 0:
        return sixth
    step = 2.0 ** (max(math.frexp(float(sixth))[1] - 8, -133))
    return np.float32(round(Fraction(float(sixth)) / Fraction(step)) * step)


def code_keys(row):
    """(codes [dim], bytes [dim / 32]) of a float32 key row."""
    row = np.asarray(row, dtype=np.float32)
    codes, units = [], []
    for g in range(0, len(row), 32):
        b = key_unit(row[g:g + 32])
        units.append(b)
        unit = Fraction(2) ** (b - 127)
        codes += [0 if b == 255 else code(x, float(unit)) for x in row[g:g + 32]]
    return codes, units


def code_values(row):
    """(codes [dim], unit) of a float32 value row."""
    row = np.asarray(row, dtype=np.float32)
    unit = value_unit(row)
    codes = [code(x, unit) if unit > 0 else 0 for x in row]
    return codes, unit


def unpack(packed):
    """float64 levels [.., 2 n] of packed codes [.., n]."""
    level = np.array(MAGNITUDES + tuple(-m for m in MAGNITUDES))
    packed = np.asarray(packed)
    both = np.stack([level[packed & 15], level[packed >> 4]], -1)
    return both.reshape(*packed.shape[:-1], 2 * packed.shape[-1])


def key_values(k_codes, k_scales):
    """float64 keys [.., dim] of packed codes and their bytes."""
    x = unpack(k_codes)
    b = np.asarray(k_scales)[..., :x.shape[-1] // 32].astype(np.float64)
    unit = np.where(b == 255, np.nan, np.exp2(b - 127))
    return x * np.repeat(unit, 32, -1)


def value_values(v_codes, v_scales):
    """float64 values [.., dim] of packed codes and their row scales."""
    return unpack(v_codes) * np.asarray(v_scales, dtype=np.float64)[..., None]
