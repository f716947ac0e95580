"""The work that the serving operators beside the KDA recurrence are measured on.

Three operators, in the forms a serving engine calls them:

* the short causal convolution over channels, for prompts (batched or packed) and for single tokens
  with its states in a slot pool;
* the selective state space scan with a scalar decay per head, for prompts (batched or packed) and
  for single tokens with its states in a slot pool;
* copying, forking and compacting the slots of the state pools of several layers at once.

`run` computes them with elementary torch operations where `own` is false and with this repository's
entry points where it is true; `exact` is their definition in 64 bits, token by token.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 128          # tokens per chunk of the plain scan


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a short prompt's q, k and v (two heads of 64) in fp32: launch latency counts
        {"name": "conv_fp32_t256", "op": "conv", "dtype": "fp32", "B": 1, "T": 256, "C": 384, "W": 4},
        # q, k and v of 32 heads of 128 side by side, one prompt of 4096 tokens
        {"name": "conv_t4k_c12288", "op": "conv", "dtype": "bf16", "B": 1, "T": 4096, "C": 12288, "W": 4},
        # one of q, k, v of 96 heads of 128: prompts of 1 to 2048 tokens packed back to back
        {"name": "conv_packed_n16", "op": "conv_packed", "dtype": "bf16", "N": 16, "most": 2048, "C": 12288, "W": 4},
        # one token for each of 256 sequences: q, k and v of 96 heads of 128, states in 512 slots
        {"name": "conv_step_b256", "op": "conv_step", "dtype": "bf16", "B": 256, "C": 36864, "W": 4, "slots": 512},
        # the fp32 workload's shape: 256 tokens, two heads of 64
        {"name": "scan_fp32_t256", "op": "scan", "dtype": "fp32", "B": 1, "T": 256, "H": 2, "G": 1, "N": 64, "P": 64},
        # one prompt of 4096 tokens, 32 heads that share one B and C: fewer heads than the GPU has SMs
        {"name": "scan_t4k_h32", "op": "scan", "dtype": "bf16", "B": 1, "T": 4096, "H": 32, "G": 1, "N": 128, "P": 128},
        # four prompts of 8192 tokens, 96 heads: the training-length prefill
        {"name": "scan_b4_t8k_h96", "op": "scan", "dtype": "bf16", "B": 4, "T": 8192, "H": 96, "G": 8, "N": 128, "P": 128},
        # prompts of 1 to 2048 tokens packed back to back, heads of 64
        {"name": "scan_packed_n16", "op": "scan_packed", "dtype": "bf16", "N_seq": 16, "most": 2048, "H": 96, "G": 8,
         "N": 128, "P": 64},
        # one long context: 512 chunks carried in sequence
        {"name": "scan_t64k_h96", "op": "scan", "dtype": "bf16", "B": 1, "T": 65536, "H": 96, "G": 8, "N": 128, "P": 64},
        # one token for each of 256 sequences, states in 512 slots: the memory-bound step of decoding
        {"name": "scan_step_b256", "op": "scan_step", "dtype": "bf16", "B": 256, "H": 96, "G": 8, "N": 128, "P": 128,
         "slots": 512},
        # eight continuations of one prompt fork its states, four layers' scan and convolution pools
        {"name": "pool_fork_8", "op": "pool_copy", "layers": 4, "slots": 64, "H": 32, "N": 128, "P": 128, "C": 12288,
         "W": 4, "pairs": 8, "fork": True},
        # a third of 192 sequences ended: the others move to the front of eight layers' pools
        {"name": "pool_compact_192", "op": "pool_compact", "layers": 8, "slots": 256, "H": 32, "N": 128, "P": 128,
         "C": 12288, "W": 4, "B": 192},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _heads(rng, most):
    """A head count and a number of groups that divides it."""
    H = _log(rng, 1, most)
    return H, rng.choice([g for g in (1, 2, 4, 8) if H % g == 0])


def draw(rng):
    op = rng.choice(["conv", "conv", "conv_packed", "conv_step", "scan", "scan", "scan", "scan_packed", "scan_packed",
                     "scan_step", "pool_copy", "pool_compact"])
    W = rng.choice([2, 3, 4, 4])
    N, P = rng.choice([64, 128, 128]), rng.choice([64, 128])
    if op == "conv":
        T, C = _log(rng, 1, 8192), 8 * _log(rng, 8, 4608)
        B = _log(rng, 1, max(1, min(16, 16384 * 12288 // (T * C))))
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp32"]), "B": B, "T": T, "C": C, "W": W}
    if op == "conv_packed":
        return {"op": op, "dtype": "bf16", "N": _log(rng, 1, 16), "most": _log(rng, 1, 2048), "C": 8 * _log(rng, 8, 1536), "W": W}
    if op == "conv_step":
        B = _log(rng, 1, 256)
        return {"op": op, "dtype": rng.choice(["bf16", "fp32"]), "B": B, "C": 8 * _log(rng, 8, 4608), "W": W,
                "slots": B + rng.randrange(0, 257)}
    if op == "scan":
        if rng.random() < 0.25:
            H, G = _heads(rng, 16)
            return {"op": op, "dtype": "fp32", "B": _log(rng, 1, 4), "T": _log(rng, 1, 1024), "H": H, "G": G, "N": N, "P": P}
        H, G = _heads(rng, 96)
        T = _log(rng, 1, 16384)
        B = _log(rng, 1, max(1, min(8, 4 * 8192 * 96 // (T * H))))
        return {"op": op, "dtype": "bf16", "B": B, "T": T, "H": H, "G": G, "N": N, "P": P}
    if op == "scan_packed":
        H, G = _heads(rng, 96)
        return {"op": op, "dtype": "bf16", "N_seq": _log(rng, 1, 16), "most": _log(rng, 1, 2048), "H": H, "G": G, "N": N, "P": P}
    if op == "scan_step":
        H, G = _heads(rng, 96)
        B = _log(rng, 1, 256)
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp32"]), "B": B, "H": H, "G": G, "N": N, "P": P,
                "slots": B + rng.randrange(0, 257)}
    H, slots = _log(rng, 1, 32), rng.randrange(8, 257)
    pool = {"layers": _log(rng, 1, 8), "slots": slots, "H": H, "N": N, "P": P, "C": 8 * _log(rng, 8, 1536), "W": W}
    if op == "pool_copy":
        return {"op": op, **pool, "pairs": rng.randrange(1, slots // 2 + 1), "fork": rng.random() < 0.5}
    return {"op": op, **pool, "B": rng.randrange(1, slots + 1)}


# --------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dtype)


def _lengths(n, most):
    """n sequence lengths, uniform from 1 to `most`: the case's own, so that the packed batch has one size."""
    return np.random.RandomState(n * 65537 + most).randint(1, most + 1, n)


def _shuffled(n, most, seed):
    """The same lengths in an order of the seed's."""
    return np.random.RandomState(seed % (1 << 31)).permutation(_lengths(n, most))


def _offsets(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def _slots(B, slots, g):
    """B distinct slots out of a pool, in random order."""
    return torch.randperm(slots, generator=g, device="cuda")[:B].to(torch.int32)


def _decay_params(g, H):
    """Per head: the rate A < 0, the skip weight D and the time-step bias (softplus of it log-uniform on 1e-3..1e-1)."""
    A = torch.rand(H, generator=g, device="cuda").mul_(15.0).add_(1.0).neg_()
    D = torch.randn(H, generator=g, device="cuda").mul_(0.1).add_(1.0)
    step = torch.exp(torch.rand(H, generator=g, device="cuda").mul_(math.log(100.0)).add_(math.log(1e-3)))
    return A, D, step + torch.log(-torch.expm1(-step))


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    op = c["op"]
    s = {"case": c}
    if op.startswith("conv"):
        dt, C, W = DTYPES[c["dtype"]], c["C"], c["W"]
        s["weight"] = _normal(g, (C, W), dt, 1.0 / math.sqrt(W))
        s["bias"] = _normal(g, (C,), dt, 0.1)
        if op == "conv":
            s["x"] = _normal(g, (c["B"], c["T"], C), dt)
            s["state"] = _normal(g, (c["B"], W - 1, C), dt)
        elif op == "conv_packed":
            n = _shuffled(c["N"], c["most"], seed)
            s["cu"] = _offsets(n)
            s["x"] = _normal(g, (int(n.sum()), C), dt)
            s["state"] = _normal(g, (c["N"], W - 1, C), dt)
        else:
            s["x"] = _normal(g, (c["B"], C), dt)
            s["state"] = _normal(g, (c["slots"], W - 1, C), dt)
            s["slots"] = _slots(c["B"], c["slots"], g)
        return s
    if op.startswith("scan"):
        dt, H, G, N, P = DTYPES[c["dtype"]], c["H"], c["G"], c["N"], c["P"]
        s["A"], s["D"], s["dt_bias"] = _decay_params(g, H)
        if op == "scan":
            lead, states = (c["B"], c["T"]), c["B"]
        elif op == "scan_packed":
            n = _shuffled(c["N_seq"], c["most"], seed)
            s["cu"], s["most"] = _offsets(n), int(n.max())
            lead, states = (int(n.sum()),), c["N_seq"]
        else:
            lead, states = (c["B"],), c["slots"]
            s["slots"] = _slots(c["B"], c["slots"], g)
        s["x"] = _normal(g, lead + (H, P), dt)
        s["dt"] = _normal(g, lead + (H,), dt, 0.5)
        s["Bm"] = _normal(g, lead + (G, N), dt)
        s["Cm"] = _normal(g, lead + (G, N), dt, 1.0 / math.sqrt(N))
        s["S"] = _normal(g, (states, H, N, P), torch.float32, 0.5)
        return s
    s["pools"] = [_normal(g, (c["slots"], c["H"], c["N"], c["P"]), torch.float32) for _ in range(c["layers"])] + \
                 [_normal(g, (c["slots"], c["W"] - 1, c["C"]), torch.bfloat16) for _ in range(c["layers"])]
    if op == "pool_copy":
        some = _slots(c["slots"], c["slots"], g)
        s["dst"] = some[: c["pairs"]].contiguous()
        s["src"] = some[c["pairs"]: c["pairs"] + 1].expand(c["pairs"]).contiguous() if c["fork"] else some[-c["pairs"]:].contiguous()
    else:
        s["slots"] = _slots(c["B"], c["slots"], g)
        s["done"] = torch.rand(c["B"], generator=g, device="cuda") < 1 / 3
    return s


# ----------------------------------------------------------------------------- the operators, plain

def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _conv_windows(x, state, weight, bias):
    """x [.., T, C] after its last W-1 inputs state [.., W-1, C]: silu(sum_w weight[:, w] x[t - (W-1) + w] + bias)."""
    W = weight.shape[1]
    u = torch.cat([state, x], dim=-2)
    y = (u.float().unfold(-2, W, 1) * weight.float()).sum(-1) + bias.float()
    return _silu(y).to(x.dtype), u[..., u.shape[-2] - (W - 1):, :].contiguous()


def _conv_packed(x, state, weight, bias, cu):
    W = weight.shape[1]
    cu = cu.long()
    t = torch.arange(x.shape[0], device=x.device)
    n = torch.bucketize(t, cu[1:], right=True)
    taps = torch.arange(W, device=x.device) - (W - 1)

    def inputs(n, at):      # the inputs of sequence n at packed positions `at`, before its start from its state
        back = at - cu[n][:, None]
        return torch.where((back >= 0)[..., None], x[at.clamp(min=0)], state[n[:, None], (back + W - 1).clamp(0, W - 2)])

    y = (inputs(n, t[:, None] + taps).float() * weight.float().t()).sum(1) + bias.float()
    every = torch.arange(cu.shape[0] - 1, device=x.device)
    return _silu(y).to(x.dtype), inputs(every, cu[1:, None] + taps[: W - 1])


def _scan(x, step, A, Bm, Cm, D, S0):
    """x [B,T,H,P], step [B,T,H] (after the softplus; 0 leaves the state as it is), S0 [B,H,N,P], all fp32."""
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    Q = min(CHUNK, T)
    nc = -(-T // Q)
    grow = lambda v: torch.cat([v, v.new_zeros((B, nc * Q - T) + v.shape[2:])], 1).reshape((B, nc, Q) + v.shape[2:])  # noqa: E731
    xc, sc, Bc, Cc = grow(x), grow(step), grow(Bm), grow(Cm)
    # decays as differences of running sums: those in 64 bits, where 32 lose the small differences of large sums
    cum = (sc.double() * A.double()).cumsum(2).permute(0, 1, 3, 2)                       # [B,nc,H,Q]
    low = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    within = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~low, -math.inf)).float()
    scores = torch.einsum("bcign,bcjgn->bcgij", Cc, Bc)
    mixed = (scores[:, :, :, None] * within.reshape(B, nc, G, H // G, Q, Q)).reshape(B, nc, H, Q, Q)
    u = (xc * sc[..., None]).permute(0, 1, 3, 2, 4)                                      # [B,nc,H,Q,P]
    y = mixed @ u
    to_end = torch.exp(cum[..., -1:] - cum).float()
    Bh = Bc.permute(0, 1, 3, 4, 2)[:, :, :, None].expand(B, nc, G, H // G, N, Q).reshape(B, nc, H, N, Q)
    local = Bh @ (u * to_end[..., None])                                                 # [B,nc,H,N,P]
    # the state entering each chunk: S0 and the chunks before, decayed
    total = torch.cat([cum.new_zeros(B, 1, H), cum[..., -1].cumsum(1)], 1)               # [B,nc+1,H]
    low = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=x.device).tril()
    carry = torch.exp((total[:, :, None] - total[:, None]).masked_fill(~low[..., None], -math.inf)).float()
    sources = torch.cat([S0[:, None], local], 1)
    states = torch.einsum("bzsh,bshk->bzhk", carry, sources.reshape(B, nc + 1, H, N * P)).reshape(B, nc + 1, H, N, P)
    Ch = Cc.permute(0, 1, 3, 2, 4)[:, :, :, None].expand(B, nc, G, H // G, Q, N).reshape(B, nc, H, Q, N)
    y = y + (Ch @ states[:, :-1]) * torch.exp(cum).float()[..., None]
    y = y.permute(0, 1, 3, 2, 4).reshape(B, nc * Q, H, P)[:, :T]
    return y + D[:, None] * x, states[:, -1].contiguous()


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "conv":
        return _conv_windows(s["x"], s["state"], s["weight"], s["bias"])
    if op == "conv_packed":
        return _conv_packed(s["x"], s["state"], s["weight"], s["bias"], s["cu"])
    if op == "conv_step":
        at = s["slots"].long()
        y, new = _conv_windows(s["x"][:, None], s["state"][at], s["weight"], s["bias"])
        s["state"][at] = new
        return y[:, 0], s["state"]
    if op.startswith("scan"):
        x, A, D = s["x"].float(), s["A"], s["D"]
        step = _softplus(s["dt"].float() + s["dt_bias"])
        Bm, Cm = s["Bm"].float(), s["Cm"].float()
    if op == "scan":
        y, S = _scan(x, step, A, Bm, Cm, D, s["S"])
        return y.to(s["x"].dtype), S
    if op == "scan_packed":
        cu = s["cu"].long()
        at = cu[:-1, None] + torch.arange(s["most"], device=x.device)
        real = at < cu[1:, None]
        at = torch.where(real, at, 0)
        y, S = _scan(x[at] * real[..., None, None], step[at] * real[..., None], A, Bm[at] * real[..., None, None],
                     Cm[at] * real[..., None, None], D, s["S"])
        return y[real].to(s["x"].dtype), S
    if op == "scan_step":
        at = s["slots"].long()
        rep = c["H"] // c["G"]
        S = s["S"][at] * torch.exp(step * A)[..., None, None]
        S = S + Bm.repeat_interleave(rep, 1)[..., None] * (step[..., None] * x)[:, :, None]
        s["S"][at] = S
        y = (S * Cm.repeat_interleave(rep, 1)[..., None]).sum(2) + D[:, None] * x
        return y.to(s["x"].dtype), s["S"]
    if op == "pool_copy":
        src, dst = s["src"].long(), s["dst"].long()
        for p in s["pools"]:
            p[dst] = p[src]
        return s["pools"]
    # the live slots at or above the number of live sequences, in order, take the free slots below it, in order
    table, to = _compacted(s["slots"], s["done"], c["slots"])
    moved = torch.nonzero(to >= 0)[:, 0]
    for p in s["pools"]:
        p[to[moved]] = p[moved]
    return [table] + s["pools"]


def _compacted(slots, done, n):
    """The new slot table (ended sequences -1), and for each slot where its contents move (-1: they stay)."""
    live = (slots >= 0) & ~done
    used = torch.zeros(n, dtype=torch.bool, device=slots.device)
    used[slots[live].long()] = True
    at = torch.arange(n, device=slots.device)
    front = at < live.sum()
    holes, movers = at[front & ~used], at[~front & used]
    to = torch.full((n,), -1, dtype=torch.long, device=slots.device)
    to[movers] = holes
    there = to[slots.long().clamp(min=0)]
    return torch.where(live, torch.where(there >= 0, there.to(torch.int32), slots), -1).to(torch.int32), to


def _run_own(s):
    import linear_attention_recurrence_forward_b200 as kda
    op = s["case"]["op"]
    if op == "conv":
        return kda.kda_short_conv(s["x"], s["weight"], s["bias"], s["state"])
    if op == "conv_packed":
        return kda.kda_short_conv_varlen(s["x"], s["weight"], s["cu"], s["bias"], s["state"])
    if op == "conv_step":
        return kda.kda_short_conv_step_paged(s["x"], s["weight"], s["state"], s["slots"], s["bias"]), s["state"]
    if op == "scan":
        return kda.kda_ssm_forward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["dt_bias"], s["S"])
    if op == "scan_packed":
        return kda.kda_ssm_forward_varlen(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["cu"], s["D"], s["dt_bias"], s["S"])
    if op == "scan_step":
        return kda.kda_ssm_decode_step_paged(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["S"], s["slots"], s["D"],
                                             s["dt_bias"]), s["S"]
    if op == "pool_copy":
        kda.kda_pool_copy(s["pools"], s["src"], s["dst"])
        return s["pools"]
    return [kda.kda_pool_compact(s["pools"], s["slots"], s["done"])] + s["pools"]


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------------------------- their definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], s["case"]["op"]
    if op.startswith("conv"):
        return _exact_conv(s, c)
    if op.startswith("scan"):
        return _exact_scan(s, c)
    return None          # copies: nothing is computed


def _exact_conv(s, c):
    W, w, b = c["W"], s["weight"].double(), s["bias"].double()

    def one(x, before):                       # one sequence [T, C] after its last inputs [W-1, C]
        u = torch.cat([before, x]).double()
        acc = b.expand(x.shape[0], -1).clone()
        for k in range(W):
            acc += w[:, k] * u[k: k + x.shape[0]]
        return acc * torch.sigmoid(acc), u[u.shape[0] - (W - 1):]

    if op_is(c, "conv"):
        got = [one(s["x"][i], s["state"][i]) for i in range(c["B"])]
        return torch.stack([y for y, _ in got]), torch.stack([z for _, z in got])
    if op_is(c, "conv_packed"):
        ends = s["cu"].tolist()
        got = [one(s["x"][a:e], s["state"][i]) for i, (a, e) in enumerate(zip(ends, ends[1:]))]
        return torch.cat([y for y, _ in got]), torch.stack([z for _, z in got])
    state, ys = s["state"].double(), []
    for i, k in enumerate(s["slots"].tolist()):
        y, state[k] = one(s["x"][i: i + 1], s["state"][k])
        ys.append(y[0])
    return torch.stack(ys), state


def op_is(c, op):
    return c["op"] == op


def _exact_scan(s, c):
    """S <- exp(step A) S + B (step x)^T, y = S^T C + D x, one token after another."""
    H, rep = c["H"], c["H"] // c["G"]
    A, D, bias = s["A"].double(), s["D"].double(), s["dt_bias"].double()

    def tokens(x, dt, Bm, Cm, S):             # [b, T, ...] and the states [b, H, N, P], updated in place
        y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        for t in range(x.shape[1]):
            xt = x[:, t].double()
            v = dt[:, t].double() + bias
            step = torch.logaddexp(v, torch.zeros_like(v))
            S *= torch.exp(step * A)[..., None, None]
            Bt = Bm[:, t].double().repeat_interleave(rep, 1)
            Ct = Cm[:, t].double().repeat_interleave(rep, 1)
            S.view(-1, *S.shape[2:]).baddbmm_(Bt.reshape(-1, Bt.shape[-1], 1), (step[..., None] * xt).reshape(-1, 1, xt.shape[-1]))
            y[:, t] = torch.bmm(Ct.reshape(-1, 1, Ct.shape[-1]), S.view(-1, *S.shape[2:])).view(xt.shape) + D[:, None] * xt
        return y

    if op_is(c, "scan"):
        if c["T"] * c["B"] * H * c["N"] * c["P"] > 2e11:
            return None                       # over some twenty seconds
        S = s["S"].double()
        y = tokens(s["x"], s["dt"], s["Bm"], s["Cm"], S)
        return y, S
    if op_is(c, "scan_packed"):
        ends = s["cu"].tolist()
        S, ys = s["S"].double(), []
        for i, (a, e) in enumerate(zip(ends, ends[1:])):
            ys.append(tokens(s["x"][None, a:e], s["dt"][None, a:e], s["Bm"][None, a:e], s["Cm"][None, a:e], S[i: i + 1])[0])
        return torch.cat(ys), S
    at = s["slots"].long()
    S = s["S"][at].double()
    y = tokens(s["x"][:, None], s["dt"][:, None], s["Bm"][:, None], s["Cm"][:, None], S)
    whole = s["S"].double()
    whole[at] = S
    return y[:, 0], whole


# ----------------------------------------------------------------------------------------- work

def work(case):
    """Bytes: each input read once, each output written once.  Ended sequences by their mean."""
    c, op = dict(case), case["op"]
    if op.startswith("conv"):
        es, C, W = DTYPES[c["dtype"]].itemsize, c["C"], c["W"]
        tokens = {"conv": lambda: c["B"] * c["T"], "conv_packed": lambda: int(_lengths(c["N"], c["most"]).sum()), "conv_step": lambda: c["B"]}[op]()
        states = c["N"] if op == "conv_packed" else c["B"]
        return {"bytes": es * C * (2 * tokens + 2 * states * (W - 1) + W + 1), "flops": tokens * C * (2 * W + 5)}
    if op.startswith("scan"):
        es, H, G, N, P = DTYPES[c["dtype"]].itemsize, c["H"], c["G"], c["N"], c["P"]
        tokens = {"scan": lambda: c["B"] * c["T"], "scan_packed": lambda: int(_lengths(c["N_seq"], c["most"]).sum()), "scan_step": lambda: c["B"]}[op]()
        states = c["N_seq"] if op == "scan_packed" else c["B"]
        # the rank-one update and the read-out of an N x P state, a multiply and an add for each element
        return {"bytes": es * tokens * (2 * H * P + H + 2 * G * N) + 2 * 4.0 * states * H * N * P, "flops": 4.0 * tokens * H * N * P}
    slot = c["layers"] * (4 * c["H"] * c["N"] * c["P"] + 2 * (c["W"] - 1) * c["C"])
    if op == "pool_copy":
        return {"bytes": slot * (c["pairs"] + (1 if c["fork"] else c["pairs"])), "flops": 0}
    live = max(1.0, c["B"] * 2 / 3)
    return {"bytes": 2 * slot * max(0.1, live * (1 - live / c["slots"])), "flops": 0}
