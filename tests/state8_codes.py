"""What the 8-bit state of one tensor may be, given its moments in float64 and
how far a float64 evaluation of them may be off.

A scale comes from the block's maximum rounded to fp32, and a byte from the
moment times 448 / maximum. An interval around each moment therefore allows one
maximum, or two where a border between two fp32 values lies inside it, and for
each of them one byte, or two neighbours. Every scale and every byte is held to
that, in blocks whose scale is the other one too."""

import numpy as np

from oracle import state8 as S8


def step_slack(grad, m_codes, m_scale, v_codes, v_scale, hp, coef):
    """How far the float64 moments of a step may be off. m1 = b1*m + (1-b1)*g':
    the constants, the products and the sum are at most 8 roundings of either
    term; v1, a sum of two terms that are not negative, at most 8 of itself.
    The oracle and the kernel may each be off by so much: 16 together."""
    m, v = S8.decode(m_codes, m_scale, v_codes, v_scale)
    g = coef * np.asarray(grad, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        return (16 * 2.0 ** -53 * (np.abs(hp.beta1 * m) + np.abs((1 - hp.beta1) * g)),
                16 * 2.0 ** -53 * (hp.beta2 * v + (1 - hp.beta2) * g * g))


def tops(x, least, root):
    """fp32 maxima of the rows of a padded array, as scales are formed from them."""
    t = S8._top(x)
    t = np.sqrt(t) if root else t
    return np.maximum(t, np.float32(least))


def check(got, m1, v1, slack=None, what=""):
    """``got``: (m bytes, m scales, v bytes, v scales) of one tensor. ``slack``:
    (of m1, of v1), None where the moments are exact, as an import's are.
    Returns how many scales are not the ones of the moments themselves."""
    m1, v1 = np.asarray(m1, np.float64), np.asarray(v1, np.float64)
    n, other = m1.size, 0
    assert [x.size for x in got] == [n, -(-n // S8.BLOCK)] * 2, what
    for k, (x, least) in enumerate(((m1, S8.LEAST_MAX), (v1, S8.LEAST_ROOT))):
        name = f"{what}: {'mv'[k]}"
        codes, scales = got[2 * k], got[2 * k + 1]
        off = np.zeros(n) if slack is None else np.where(np.isfinite(x), slack[k], 0.0)
        if n == 0:
            continue
        with np.errstate(over="ignore", invalid="ignore"):
            size = np.abs(x) if k == 0 else x
            t = [tops(S8._blocks(y), least, k == 1) for y in (size, size - off, size + off)]
            allowed = [(y / np.float32(S8.E4M3_MAX)).astype(np.float32) for y in t]
            hit = [scales == a for a in allowed]
            assert (hit[0] | hit[1] | hit[2]).all(), f"{name} scales"
            other += int((~hit[0]).sum())
            top = np.where(hit[0], t[0], np.where(hit[1], t[1], t[2]))
            up = (np.float32(S8.E4M3_MAX) / top).astype(np.float64).repeat(S8.BLOCK)[:n]
            if k == 0:
                ok = [S8.e4m3_encode((x + s * off) * up) for s in (-1, 0, 1)]
            else:
                # a root and a product more than the kernel's comparison of squares: 4 roundings
                ok = []
                for s in (-1, 0, 1):
                    y = x + s * (off + 4 * 2.0 ** -53 * np.abs(x))
                    r = np.sqrt(y) * up
                    ok.append(S8.e4m3_encode(np.where(y > 0, np.maximum(r, 2.0 ** -9), r)))
        nan = codes & 0x7F == S8.NAN
        fits = np.zeros(n, bool)
        for c in ok:
            fits |= np.where(c & 0x7F == S8.NAN, nan, codes == c)
        assert fits.all(), f"{name} bytes at {np.flatnonzero(~fits)[:8]}: {codes[~fits][:8]}, {ok[1][~fits][:8]}"
    return other
