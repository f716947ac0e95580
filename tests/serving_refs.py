"""The short convolution, the selective scan and the pool compaction written out in fp64 (numpy), one
sequence and one token at a time, and the error bounds the tests hold the kernels to."""
import numpy as np

# half a step of each type, relative to the value
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def np64(t):
    return t.detach().to("cpu").double().numpy()


def conv(x, weight, bias, state, silu=True):
    """One sequence: x [T, C], weight [C, W], bias [C] or None, state [W-1, C] or None.  Returns (y, the last
    W-1 inputs, the sum of the absolute terms before the activation)."""
    T, C = x.shape
    W = weight.shape[1]
    u = np.concatenate([np.zeros((W - 1, C)) if state is None else state, x])
    z, mag = np.zeros((T, C)), np.zeros((T, C))
    if bias is not None:
        z, mag = z + bias, mag + np.abs(bias)
    for w in range(W):
        z = z + weight[:, w] * u[w:w + T]
        mag = mag + np.abs(weight[:, w] * u[w:w + T])
    with np.errstate(over="ignore"):
        y = z / (1.0 + np.exp(-z)) if silu else z
    return y, u[len(u) - (W - 1):], mag


def conv_bound(y, mag, dtype):
    """W <= 4 fp32 products and sums (each off by 2^-24 of the terms' magnitudes) through an activation of
    slope <= 1.1, its own error (bf16: about 2^-20 from the approximate exponential and division), the
    rounding of the output."""
    return HALF[dtype] * np.abs(y) + 1.1 * 8 * 2.0 ** -24 * mag + (2.0 ** -20 if dtype == "bf16" else 2.0 ** -21) * np.abs(y) + 1e-30


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def scan(x, dt, A, Bm, Cm, D=None, bias=None, S0=None):
    """One sequence: x [T, H, P], dt [T, H], Bm, Cm [T, G, N], S0 [H, N, P].  Returns (y, S_T) and the same
    recurrence on absolute values (what every term adds up to without cancellation)."""
    T, H, P = x.shape
    G, N = Bm.shape[1:]
    rep = H // G
    S = np.zeros((H, N, P)) if S0 is None else S0.astype(np.float64).copy()
    Sa = np.abs(S)
    y, ya = np.zeros((T, H, P)), np.zeros((T, H, P))
    for t in range(T):
        step = softplus(dt[t] + (0 if bias is None else bias))
        a = np.exp(step * A)
        Bt, Ct = np.repeat(Bm[t], rep, 0), np.repeat(Cm[t], rep, 0)
        up = Bt[:, :, None] * (step[:, None] * x[t])[:, None, :]
        S = a[:, None, None] * S + up
        Sa = a[:, None, None] * Sa + np.abs(up)
        y[t] = np.einsum("hnp,hn->hp", S, Ct)
        ya[t] = np.einsum("hnp,hn->hp", Sa, np.abs(Ct))
        if D is not None:
            y[t] += D[:, None] * x[t]
            ya[t] += np.abs(D[:, None] * x[t])
    return y, S, ya, Sa


def scan_bounds(y, ya, Sa, T, N, dtype, impl):
    """(bound of y, bound of S) element by element.

    fp32 arithmetic: a token's decay, time step and products are each off by a few 2^-24, and a term stays in
    the state for at most T tokens, so 8 T + N steps of 2^-24 of its magnitude cover it.  The tensor-core
    kernel reads the state and the decayed scores as bf16 operands (2^-8 of each term of y).  To the state it
    adds x w, w = s_j e^(..), as hi + lo: w is taken as two bf16 values (off by 2^-8 of the second, which is at
    most 2^-8 w), and lo, at most 2 * 2^-8 of the term, is rounded to bf16: (1 + 2) * 2^-16 of each term."""
    f32 = (8 * T + N + 64) * 2.0 ** -24
    by = HALF[dtype] * np.abs(y) + f32 * ya
    bS = f32 * Sa
    if impl == "tcgen05":
        by = by + 1.01 * 2.0 ** -8 * ya
        bS = bS + 3 * 2.0 ** -16 * Sa
    return by + 1e-30, bS + 1e-30


def compact(slots, done, n_slots):
    """(new table, {slot: where its contents go}) of kda_pool_compact."""
    live = [s for s, d in zip(slots, done) if s >= 0 and not d]
    L = len(live)
    holes = [s for s in range(L) if s not in set(live)]
    movers = sorted(s for s in live if s >= L)
    to = dict(zip(movers, holes))
    return [(to.get(s, s) if s >= 0 and not d else -1) for s, d in zip(slots, done)], to
