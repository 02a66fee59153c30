"""Decode attention over a 4-bit cache in 64 bits, with the error that the
kernel's roundings leave, per request, query head and group of 64 dims.

With w_t the softmax weights, a_t = s_t * code_t and m_t the two parts of a value,
an output is sum w_t a_t + sum w_t m_t, and the kernel rounds

 (1) each weight times scale, relative to a power of two that follows the largest
     of them of its head and group, to f16: half a step of 2^-10 of it, spread
     evenly, so a deviation of at most 2^-11 / sqrt(3) of w_t a_t; where it falls
     below 2^-14 of that power of two, which the kernel keeps at most the largest
     w_t s_t over 8, the rounding is absolute: 2^-28 of the largest, or all of it;
 (2) scores: the products of a 16-dim step, exact, meet in a binary32 accumulator
     that may truncate; eight such steps and the sums around them, 16 units of 2^-24
     of the sum of the parts' magnitudes, and 2^-22 of the exponential.  A code of an
     even (odd) dim enters as a subnormal f16, up to 2^10 (2^6) times which the adder
     may take for its magnitude: of 24 bits below the leading one of 2^10 (2^6) times
     a step's largest |q|, the last is 2^-13 (2^-17) of that |q| at most.  The 8 bits
     of a |q| reach below it only where it is less than 2^-6 (2^-10) of the largest,
     so each such dim with a code loses up to one unit of 2^-13 (2^-17) of the head's
     largest |q|, times the scale.  An error that is common to a request's tokens
     divides out, so w_t moves out by it times (value - out), independently;
 (3) the V product's accumulator, once per tile of 16 tokens, truncating: 2^-23 of
     the sum of w_t |a_t| a time, all in one direction at worst; and the minima's sum,
     to nearest: 2^-24 of its magnitude, times the root of the number of sums;
 (4) the output to bf16: half a step of 2^-7, spread evenly.

The norm of a group's error stays within 4 times the root of the sum of the
squares of the spread ones (a group's 64 dims share the weights' errors, so the
norm may be one weight's, at most sqrt(3) of its deviation), plus the norm of the
one-directional ones.
"""
import numpy as np

import _cache_reference as ref

U = 2.0 ** -24
GROUP = ref.GROUP


def attend(q_bits, pools, table, lens, sm_scale, window=0, sinks=0, sums=None):
    """(out, lse, bound of each group's error norm [B][Hq][D / 64], bound of lse's
    error).  sums: tiles of 16 tokens that one accumulator takes (default: all)."""
    NP, H, P, D = pools.shape
    B, Hq, _ = q_bits.shape
    G, K = Hq // H, D // GROUP
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    bound, lse_bound = np.zeros((B, Hq, K)), np.zeros((B, Hq))
    q = ref.bf16(q_bits).reshape(B, H, G, D)
    sm = float(np.float32(sm_scale))
    norms = lambda x: np.linalg.norm(x.reshape(G, K, GROUP), axis=-1)  # noqa: E731
    for b in range(B):
        t = ref.visible(int(lens[b]), window, sinks)
        pages = table[b, t // P]
        N = -(-t.size // 16) if sums is None else sums
        for h in range(H):
            k, ka, km = (x[:, h] for x in pools.rows("k", pages, t % P))
            v, va, vm = (x[:, h] for x in pools.rows("v", pages, t % P))
            qh = q[b, h]
            s = qh @ k.T * sm                                              # [G][T]
            e = np.exp(s - s.max(-1, keepdims=True))
            tot = e.sum(-1, keepdims=True)
            w = e / tot
            o = w @ v
            # (2): the sums' magnitudes, the minima times the groups' query sums
            qs = np.abs(qh.reshape(G, K, GROUP).sum(-1))
            size = abs(sm) * (np.abs(qh) @ np.abs(ka).T + qs @ np.abs(km[:, ::GROUP]).T)
            moved = 16 * U * (size + np.abs(s - s.max(-1, keepdims=True))) + 2.0 ** -22
            top = np.abs(qh).max(-1, keepdims=True)
            for parity, bits in ((0, 10), (1, 6)):
                aq = np.abs(qh[:, parity::2])
                small = (aq > 0) & (aq < 2.0 ** (bits - 16) * top)
                # (a dim's |a| is at most 15 scales: the scale of its group where it has a code)
                ks = np.repeat(np.abs(ref.bf16(pools.kp[pages, h, t % P])[..., 0]), GROUP // 2, -1)
                moved = moved + abs(sm) * 2.0 ** (bits - 23) * top * \
                    (small.astype(float) @ (ks * (ka[:, parity::2] != 0)).T)
            var = (w ** 2 @ va ** 2) * (2.0 ** -22 / 3)                     # (1)
            wm = (w * moved) ** 2
            var += wm @ v ** 2 - 2 * (wm @ v) * o + wm.sum(-1, keepdims=True) * o ** 2
            var += (2 * N) * (U * (w @ np.abs(vm))) ** 2                     # (3), minima
            var += (2.0 ** -8 * o) ** 2 / 3                                  # (4)
            one = 2 * U * N * (w @ np.abs(va))                               # (3), codes
            ps = np.abs(ref.bf16(pools.vp[pages, h, t % P])[..., 0])         # [T][K]
            for j in range(K):                                               # (1), small weights
                ws = w * ps[:, j]
                cut = np.minimum(ws, 2.0 ** -28 * ws.max(-1, keepdims=True))
                at = slice(j * GROUP, (j + 1) * GROUP)
                codes = np.divide(va[:, at], ps[:, j:j + 1], out=np.zeros_like(va[:, at]),
                                  where=ps[:, j:j + 1] > 0)
                one[:, at] += cut @ np.abs(codes)
            rows = slice(h * G, (h + 1) * G)
            out[b, rows], lse[b, rows] = o, (s.max(-1) + np.log(tot[:, 0]))
            bound[b, rows] = 4 * norms(np.sqrt(np.maximum(var, 0))) + norms(one)
            lse_bound[b, rows] = (w * moved).sum(-1) + np.sqrt(4 * N) * U + \
                4 * U * (np.abs(lse[b, rows]) + 1)
    return out, lse, bound, lse_bound


def check(got_out, got_lse, want, label=""):
    """Every group's error norm and every lse; returns the worst shares of the bounds."""
    out, lse, bound, lse_bound = want
    B, Hq, D = out.shape
    err = np.linalg.norm((got_out - out).reshape(B, Hq, D // GROUP, GROUP), axis=-1)
    share = err / np.maximum(bound, 1e-300)
    worst, lworst = share.max(), (np.abs(got_lse - lse) / lse_bound).max()
    assert np.isfinite(got_out).all() and np.isfinite(got_lse).all(), f"{label}: not finite"
    assert worst <= 1.0, f"{label}: {worst:.3g} of the bound at {np.unravel_index(share.argmax(), share.shape)}"
    assert lworst <= 1.0, f"{label}: lse {lworst:.3g} of its bound"
    return worst, lworst
