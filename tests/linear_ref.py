"""Linear attention with decays token by token in 64 bits, and how far 32-bit arithmetic may be from it.

S_t = e^g_t S_{t-1} + v_t k_t^T, o_t = scale S_t q_t, straight from the definition.

bound(): every term of an output (a product of a decay, q, k and v values, or of the start state) passes at most
  d roundings in a dot over d, 64 in a sum over a chunk's tokens, 8 in its decay factors (the rounding of an exponent x
  costs |x| 2^-24 of the term: see below), and for every later chunk 2 (the state times a decay, plus the chunk's sum) and
  the 64 of that chunk's sum only once; rounded up to (d + 136 + 3 chunks) steps of 2^-24 of the sum of the terms'
  magnitudes. A matrix instruction may cut instead of round a sum: twice that. The magnitudes are
  summed by the same recurrence with absolute values and with 0.9 g in place of g: |x| e^x <= 3.7 e^(0.9 x)
  covers the exponents' roundings."""

import numpy as np

STEP = 2.0 ** -24


def recurrence(q, k, v, g, S0, scale):
    """q, k [T, Hk, d], v [T, Hv, d], g [T, Hv], S0 [Hv, d, d] (d_v, d_k), float64 -> o [T, Hv, d], S."""
    T, Hk, d = q.shape
    Hv = v.shape[1]
    rep = Hv // Hk
    S = S0.copy()
    o = np.empty((T, Hv, d))
    for t in range(T):
        kt, qt = np.repeat(k[t], rep, 0), np.repeat(q[t], rep, 0)
        with np.errstate(invalid="ignore"):
            S = np.exp(g[t])[:, None, None] * S + v[t][:, :, None] * kt[:, None, :]
            o[t] = scale * np.einsum("hvk,hk->hv", S, qt)
    return o, S


def packed(q, k, v, g, S0, scale, cu):
    """recurrence() of every sequence of a pack; S0 [n, Hv, d, d]."""
    o, S = np.zeros((q.shape[0],) + v.shape[1:]), S0.copy()
    for i in range(len(cu) - 1):
        a, b = cu[i], cu[i + 1]
        if b > a:
            o[a:b], S[i] = recurrence(q[a:b], k[a:b], v[a:b], g[a:b], S0[i], scale)
    return o, S


def bound(q, k, v, g, S0, scale, cu, chunk=64):
    """Elementwise bounds (o, S) of the error of an fp32 computation."""
    o, S = packed(np.abs(q), np.abs(k), np.abs(v), 0.9 * g, np.abs(S0), abs(scale), cu)
    d = q.shape[-1]
    for i in range(len(cu) - 1):
        n = -(-(cu[i + 1] - cu[i]) // chunk)
        f = 2 * (d + 136 + 3 * n) * STEP
        o[cu[i]:cu[i + 1]] *= f
        S[i] *= f
    return o, S
