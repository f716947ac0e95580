"""The selective scan: prompts (batched, packed), single tokens (plain, paged), against fp64."""
import numpy as np
import pytest
import torch

import linear_attention_recurrence_forward_b200 as kda
from linear_attention_recurrence_forward_b200 import STATUS
import serving_refs as ref
from serving_refs import np64

OK, INVALID, UNSUPPORTED, MISALIGNED = (STATUS[n] for n in
                                        ("KDA_OK", "KDA_ERR_INVALID_ARG", "KDA_ERR_UNSUPPORTED",
                                         "KDA_ERR_MISALIGNED"))
TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}
BASE, SZ = 0x7F0000000000, 1 << 33

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from linear_attention_recurrence_forward_b200 import build
    build.build()
    return kda.lib()


# ---------------------------------------------------------------------- refusals (CPU)

NAMES = ["x", "dt", "A", "Bm", "Cm", "D", "bias", "S0", "y", "ST", "ix", "ws"]
AT = {n: BASE + i * SZ for i, n in enumerate(NAMES)}


def call(L, form="batch", B=2, T=10, H=4, G=2, N=128, P=64, ldx=None, lddt=None, ldb=None, ldc=None, dtype=0, impl=0,
         n_slots=8, ws_bytes=1 << 32, **p):
    a = {**AT, **p}
    ld = (ldx or H * P, lddt or H, ldb or G * N, ldc or G * N)
    if form == "batch":
        return L.kda_ssm_forward(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["D"], a["bias"], a["S0"], a["y"], a["ST"],
                                 B, T, H, G, N, P, *ld, dtype, impl, a["ws"], ws_bytes, None)
    if form == "varlen":
        return L.kda_ssm_forward_varlen(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["ix"], a["D"], a["bias"], a["S0"],
                                        a["y"], a["ST"], B, T, H, G, N, P, *ld, dtype, impl, a["ws"], ws_bytes, None)
    if form == "step":
        return L.kda_ssm_decode_step(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["D"], a["bias"], a["ST"], a["y"],
                                     B, H, G, N, P, *ld, dtype, None)
    return L.kda_ssm_decode_step_paged(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["D"], a["bias"], a["ST"], n_slots,
                                       a["ix"], a["y"], B, H, G, N, P, *ld, dtype, None)


@pytest.mark.parametrize("form", ["batch", "varlen", "step", "paged"])
def test_refusals(L, form):
    f = lambda **k: call(L, form, **k)  # noqa: E731
    for k in (dict(B=0), dict(H=0), dict(G=0), dict(G=3), dict(ldx=64), dict(lddt=2), dict(ldb=64), dict(ldc=64),
              dict(x=None), dict(dt=None), dict(A=None), dict(Bm=None), dict(Cm=None), dict(y=None)):
        assert f(**k) == INVALID, k
    for k in (dict(N=32), dict(P=96), dict(N=256), dict(dtype=2)):
        assert f(**k) == UNSUPPORTED, k
    for k in (dict(x=AT["x"] + 8), dict(dt=AT["dt"] + 1), dict(A=AT["A"] + 2), dict(Bm=AT["Bm"] + 8), dict(Cm=AT["Cm"] + 2),
              dict(D=AT["D"] + 1), dict(bias=AT["bias"] + 2), dict(y=AT["y"] + 8), dict(ST=AT["ST"] + 4), dict(ldx=260),
              dict(ldb=260), dict(ldc=260)):
        assert f(**k) == MISALIGNED, k
    for n in ("x", "dt", "A", "Bm", "Cm", "D", "bias", "ST"):
        assert f(y=AT[n]) == INVALID, n                    # y on another argument
    for n in ("x", "Bm"):
        assert f(ST=AT[n] + 512) == INVALID, n
    if form in ("batch", "varlen"):
        assert f(T=-1) == INVALID
        assert f(impl=9) == INVALID
        assert f(ST=AT["S0"] + 4096) == INVALID            # partly over S0
        assert f(y=AT["S0"]) == INVALID
        assert f(dtype=1, impl=1) == UNSUPPORTED           # the tensor-core kernel is bf16 only
    if form in ("varlen", "paged"):
        assert f(ix=None) == INVALID
        assert f(ix=AT["ix"] + 2) == MISALIGNED
        assert f(ix=AT["y"]) == INVALID
    if form in ("step", "paged"):
        assert f(ST=None) == INVALID
    if form == "paged":
        assert f(n_slots=0) == INVALID


def test_binding_refuses_bad_tensors():
    x, dt, A, b = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 4), torch.zeros(4), torch.zeros(2, 5, 2, 64)
    with pytest.raises(ValueError):
        kda.kda_ssm_forward(x, dt, A, b, b)                                  # not on a GPU
    with pytest.raises(ValueError):
        kda.kda_ssm_forward(x.half(), dt.half(), A, b.half(), b.half())
    with pytest.raises(ValueError):
        kda.kda_ssm_forward(x, dt, A.double(), b, b)
    with pytest.raises(ValueError):
        kda.kda_ssm_forward(x.transpose(2, 3), dt, A, b, b)
    with pytest.raises(ValueError):
        kda.kda_ssm_forward(x, dt, A, b, b.bfloat16())


# ---------------------------------------------------------------------- GPU

def case(lead, H, G, N, P, dtype, seed=0, states=None, rate=16.0, step=None):
    """Inputs in the operators' distributions: rates -1..-rate, time steps 1e-3..1e-1 (or `step`)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda shape, s=1.0: torch.randn(shape, generator=g, device="cuda") * s  # noqa: E731
    A = -(1 + (rate - 1) * torch.rand(H, generator=g, device="cuda"))
    D = 1 + 0.1 * r((H,))
    s = step if step is not None else torch.exp(torch.rand(H, generator=g, device="cuda") * 4.6 - 6.9)
    bias = s + torch.log(-torch.expm1(-s)) if step is None else torch.full((H,), float(np.log(np.expm1(step))), device="cuda")
    x, dt = r(lead + (H, P)).to(TORCH[dtype]), r(lead + (H,), 0.5).to(TORCH[dtype])
    Bm, Cm = r(lead + (G, N)).to(TORCH[dtype]), r(lead + (G, N), N ** -0.5).to(TORCH[dtype])
    S0 = r((states if states is not None else lead[0], H, N, P), 0.5)
    return dict(x=x, dt=dt, A=A, Bm=Bm, Cm=Cm, D=D, dt_bias=bias, S0=S0)


def check(y, S, c, rows, n, dtype, impl, skip=True, start=True):
    """y [T, H, P] and S [H, N, P] of sequence n, tokens `rows` of the inputs, against fp64."""
    f = lambda k: np64(c[k][rows])  # noqa: E731
    T = y.shape[0]
    ry, rS, ya, Sa = ref.scan(f("x"), f("dt"), np64(c["A"]), f("Bm"), f("Cm"), np64(c["D"]) if skip else None,
                              np64(c["dt_bias"]) if skip else None, np64(c["S0"][n]) if start else None)
    by, bS = ref.scan_bounds(ry, ya, Sa, T, c["Bm"].shape[-1], dtype, impl)
    ey, eS = np.abs(np64(y) - ry), np.abs(np64(S) - rS)
    assert np.all(ey <= by), f"y {float((ey / by).max()):.3g} of its bound"
    assert np.all(eS <= bS), f"S {float((eS / bS).max()):.3g} of its bound"


IMPLS = [("fp32", "simt"), ("bf16", "simt"), ("bf16", "tcgen05")]


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("B,T,H,G,N,P", [(1, 1, 1, 1, 64, 64), (2, 7, 3, 1, 128, 64), (1, 64, 4, 2, 64, 128),
                                         (1, 127, 2, 2, 128, 128), (3, 128, 2, 1, 128, 128), (1, 129, 6, 2, 128, 64),
                                         (1, 300, 3, 3, 64, 64), (1, 700, 2, 1, 128, 128)])
def test_prompt(dtype, impl, B, T, H, G, N, P):
    c = case((B, T), H, G, N, P, dtype, seed=T)
    y, S = kda.kda_ssm_forward(**c, impl=impl)
    assert kda.kda_get_device_status() == 0
    for b in range(B):
        check(y[b], S[b], c, b, b, dtype, impl)


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("step,rate", [(2.0, 16.0), (1e-4, 1.5), (20.0, 2.0)])
def test_strong_and_weak_decay(dtype, impl, step, rate):
    """Time steps at which a token forgets everything before it, and at which hundreds of tokens stay."""
    c = case((1, 260), 3, 1, 128, 64, dtype, seed=3, step=step, rate=rate)
    y, S = kda.kda_ssm_forward(**c, impl=impl)
    check(y[0], S[0], c, 0, 0, dtype, impl)


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("T,H", [(260, 3), (1700, 1)])
def test_tokens_that_forget_everything(dtype, impl, T, H):
    """Time steps of a million here and there: the decay between the tokens after one does not come out of the
    difference of two sums of millions."""
    c = case((1, T), H, 1, 128, 64, dtype, seed=5)
    c["dt"][0, 3::37] = 1e6
    y, S = kda.kda_ssm_forward(**c, impl=impl)
    check(y[0], S[0], c, 0, 0, dtype, impl)


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
def test_optional_arguments_and_state_in_place(dtype, impl):
    c = case((2, 140), 4, 2, 128, 64, dtype, seed=5)
    y, S = kda.kda_ssm_forward(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], impl=impl)      # no D, no bias, S0 = 0
    for b in range(2):
        check(y[b], S[b], c, b, b, dtype, impl, skip=False, start=False)
    y1, S1 = kda.kda_ssm_forward(**c, impl=impl)
    held = c["S0"].clone()
    y2, S2 = kda.kda_ssm_forward(**{**c, "S0": held}, S_T=held, impl=impl)
    assert S2 is held and torch.equal(y1, y2) and torch.equal(S1, S2)
    y3, none = kda.kda_ssm_forward(**c, return_state=False, impl=impl)
    assert none is None and torch.equal(y1, y3)


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
def test_packed(dtype, impl):
    lengths, lead, tail = [1, 0, 127, 128, 129, 5, 0, 300, 2], 3, 4
    T, H, G, N, P = lead + sum(lengths) + tail, 4, 2, 128, 64
    c = case((T,), H, G, N, P, dtype, seed=9, states=len(lengths))
    for k in ("x", "dt", "Bm", "Cm"):                    # rows of no sequence reach nothing
        c[k][:lead] = float("nan")
        c[k][T - tail:] = float("inf")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]) + lead, dtype=torch.int32, device="cuda")
    y = torch.full((T, H, P), 7.0, dtype=TORCH[dtype], device="cuda")
    y, S = kda.kda_ssm_forward_varlen(**c, cu_seqlens=cu, y=y, impl=impl)
    assert kda.kda_get_device_status() == 0
    at = lead
    for n, k in enumerate(lengths):
        check(y[at:at + k], S[n], c, slice(at, at + k), n, dtype, impl)
        if k == 0:
            assert torch.equal(S[n], c["S0"][n])
        at += k
    assert bool((y[:lead] == 7).all()) and bool((y[T - tail:] == 7).all())


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("bad", [[0, 50, 130], [-2, 50, 100], [0, 70, 60]])
def test_invalid_offsets_are_reported_not_followed(dtype, impl, bad):
    c = case((100,), 2, 1, 128, 64, dtype, states=2)
    y = torch.full((100, 2, 64), 7.0, dtype=TORCH[dtype], device="cuda")
    y, S = kda.kda_ssm_forward_varlen(**c, cu_seqlens=torch.tensor(bad, dtype=torch.int32, device="cuda"), y=y, impl=impl)
    assert kda.kda_get_device_status() == INVALID
    assert torch.equal(S, c["S0"]) and bool((y == 7).all())


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
def test_slices_of_wider_rows(dtype, impl):
    """x, B, C and dt as slices of one projection's rows equal their contiguous copies, bit for bit."""
    B, T, H, G, N, P = 2, 200, 4, 2, 64, 64
    c = case((B, T), H, G, N, P, dtype, seed=4)
    wide = torch.zeros((B, T, H * P + 2 * G * N + 16), dtype=TORCH[dtype], device="cuda")
    parts, at = {}, 0
    for k, n in (("x", H * P), ("Bm", G * N), ("Cm", G * N), ("dt", H)):
        wide[..., at:at + n] = c[k].flatten(2)
        parts[k] = wide[..., at:at + n].unflatten(2, (c[k].shape[2:])) if k != "dt" else wide[..., at:at + n]
        at += n
    assert not parts["x"].is_contiguous()
    y, S = kda.kda_ssm_forward(**c, impl=impl)
    y2, S2 = kda.kda_ssm_forward(**{**c, **parts}, impl=impl)
    assert torch.equal(y, y2) and torch.equal(S, S2)


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
def test_no_tokens(dtype, impl):
    c = case((2, 0), 2, 1, 64, 64, dtype, states=2)
    y, S = kda.kda_ssm_forward(**c, impl=impl)
    assert y.shape == (2, 0, 2, 64) and torch.equal(S, c["S0"])
    _, S = kda.kda_ssm_forward(**{**c, "S0": None}, impl=impl)
    assert bool((S == 0).all())


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,H,G,N,P", [(1, 1, 1, 64, 64), (3, 6, 2, 128, 64), (2, 5, 5, 64, 128), (5, 4, 1, 128, 128)])
def test_steps(dtype, B, H, G, N, P):
    T = 4
    c = case((B, T), H, G, N, P, dtype, seed=B)
    S = c["S0"].clone()
    n_slots = B + 2
    slots = torch.randperm(n_slots, device="cuda")[:B].to(torch.int32)
    pool = torch.full((n_slots, H, N, P), 3.0, device="cuda")
    pool[slots.long()] = S
    ys = []
    for t in range(T):
        one = {k: c[k][:, t] for k in ("x", "dt", "Bm", "Cm")}
        y = kda.kda_ssm_decode_step(**one, A=c["A"], S=S, D=c["D"], dt_bias=c["dt_bias"])
        yp = kda.kda_ssm_decode_step_paged(**{k: v.contiguous() for k, v in one.items()}, A=c["A"], S_pool=pool, slots=slots,
                                           D=c["D"], dt_bias=c["dt_bias"])
        assert torch.equal(y, yp)
        ys.append(y)
    y = torch.stack(ys, 1)
    for b in range(B):
        check(y[b], S[b], c, b, b, dtype, "simt")
    assert torch.equal(pool[slots.long()], S) and kda.kda_get_device_status() == 0
    free = torch.ones(n_slots, dtype=torch.bool, device="cuda")
    free[slots.long()] = False
    assert bool((pool[free] == 3).all())


@gpu
def test_paged_step_skips_and_reports():
    c = case((3,), 2, 1, 64, 64, "bf16", states=4)
    pool, before = c.pop("S0"), None
    before = pool.clone()
    slots = torch.tensor([2, -1, 4], dtype=torch.int32, device="cuda")
    y = torch.full((3, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_ssm_decode_step_paged(**c, S_pool=pool, slots=slots, y=y)
    assert kda.kda_get_device_status() == INVALID
    assert bool((y[1:] == 7).all()) and not bool((y[0] == 7).all())
    assert torch.equal(pool[[0, 1, 3]], before[[0, 1, 3]])


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
def test_on_a_stream_and_in_a_graph(dtype, impl):
    c = case((1, 300), 2, 1, 128, 64, dtype, seed=8)
    y0, S0 = kda.kda_ssm_forward(**c, impl=impl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, S1 = kda.kda_ssm_forward(**c, impl=impl, stream=side)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(S0, S1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, Sg = kda.kda_ssm_forward(**c, impl=impl)
    for _ in range(2):
        yg.zero_()
        graph.replay()
        assert torch.equal(y0, yg) and torch.equal(S0, Sg)


LONG = [(1, 1700, 1, 1, 128, 128), (1, 2048, 3, 1, 64, 64), (2, 1281, 2, 1, 128, 64), (1, 4097, 2, 2, 64, 128)]


@pytest.mark.parametrize("B,T,H,G,N,P", LONG)
def test_long_prompts_of_few_heads_ask_for_a_workspace(L, B, T, H, G, N, P):
    need = kda.ssm_workspace_bytes(B, B * T, H, N, P)
    assert need >= 2 * B * H * N * P * 4 and need % 4 == 0
    assert kda.ssm_workspace_bytes(B, B * T, H, N, P, torch.float32) == 0
    assert kda.ssm_workspace_bytes(B, B * T, H, N, P, impl="simt") == 0
    assert kda.ssm_workspace_bytes(4, 4 * 8192, 96, 128, 128) == 0           # enough heads: no segments
    f = lambda **k: call(L, B=B, T=T, H=H, G=G, N=N, P=P, **k)  # noqa: E731
    assert f(ws=None) == INVALID and f(ws_bytes=need - 1) == INVALID
    assert f(ws=AT["ws"] + 8) == MISALIGNED
    assert f(ws=AT["ST"]) == INVALID and f(ws=AT["x"] + 64) == INVALID


@gpu
@pytest.mark.parametrize("B,T,H,G,N,P", LONG)
def test_segments(B, T, H, G, N, P):
    """Prompts cut into segments: against fp64, in place, and packed with shorter ones."""
    c = case((B, T), H, G, N, P, "bf16", seed=T, rate=1.5)
    y, S = kda.kda_ssm_forward(**c)
    assert kda.kda_get_device_status() == 0
    for b in range(B):
        check(y[b], S[b], c, b, b, "bf16", "tcgen05")
    held = c["S0"].clone()
    y2, S2 = kda.kda_ssm_forward(**{**c, "S0": held}, S_T=held)
    assert torch.equal(y, y2) and torch.equal(S, S2)
    ws = torch.full((kda.ssm_workspace_bytes(B, B * T, H, N, P),), 255, dtype=torch.uint8, device="cuda")   # NaN
    y3, S3 = kda.kda_ssm_forward(**c, workspace=ws)
    assert torch.equal(y, y3) and torch.equal(S, S3)


@gpu
def test_segments_in_graphs_and_beside_another_stream():
    """Both launches of a call captured and replayed, twice over in one graph, while another stream runs a call of
    its own: the second launch may start early, and must not read what the first has not written."""
    c = [case((1, 4096), 4, 1, 128, 128, "bf16", seed=s, rate=1.5) for s in (1, 2, 3)]
    want = [kda.kda_ssm_forward(**k) for k in c]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [kda.kda_ssm_forward(**k) for k in c[:2]]
    side = torch.cuda.Stream()
    for _ in range(5):
        for y, S in got:
            y.zero_()
            S.zero_()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        y3, S3 = kda.kda_ssm_forward(**c[2], stream=side)
        torch.cuda.synchronize()
        for (y, S), (yw, Sw) in zip(got + [(y3, S3)], want):
            assert torch.equal(y, yw) and torch.equal(S, Sw)
    assert kda.kda_get_device_status() == 0


@gpu
def test_segments_packed():
    lengths, lead, tail = [3000, 0, 129, 2500, 1500], 3, 5
    T, H, G, N, P = lead + sum(lengths) + tail, 2, 1, 128, 64
    c = case((T,), H, G, N, P, "bf16", seed=9, states=len(lengths), rate=1.5)
    assert kda.ssm_workspace_bytes(len(lengths), T, H, N, P) > 0
    for k in ("x", "dt", "Bm", "Cm"):
        c[k][:lead] = float("nan")
        c[k][T - tail:] = float("inf")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]) + lead, dtype=torch.int32, device="cuda")
    y = torch.full((T, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
    held = c["S0"].clone()
    y, S = kda.kda_ssm_forward_varlen(**{**c, "S0": held}, cu_seqlens=cu, y=y, S_T=held)
    assert kda.kda_get_device_status() == 0
    at = lead
    for n, k in enumerate(lengths):
        check(y[at:at + k], S[n], c, slice(at, at + k), n, "bf16", "tcgen05")
        at += k
    assert bool((y[:lead] == 7).all()) and bool((y[T - tail:] == 7).all())


@gpu
@pytest.mark.parametrize("P", [64, 128])
def test_many_short_prompts_beside_heavy_traffic(P):
    """Hundreds of calls over short packed prompts while another stream copies: loads and stores take long there, and
    no wait of the kernel may mistake one chunk's arrival for another's."""
    lengths = [1, 130, 257, 384, 511, 640, 90, 256] * 3
    T = sum(lengths)
    c = case((T,), 24, 2, 128, P, "bf16", seed=11, states=len(lengths))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    want = kda.kda_ssm_forward_varlen(**c, cu_seqlens=cu)
    a, b = (torch.empty(1 << 28, dtype=torch.uint8, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(300):
        if i % 4 == 0:
            with torch.cuda.stream(side):
                b.copy_(a)
        got = kda.kda_ssm_forward_varlen(**c, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
def test_a_wait_that_runs_out_is_reported():
    c = case((1, 300), 2, 1, 128, 64, "bf16", seed=8)
    want = kda.kda_ssm_forward(**c)
    kda.kda_debug_set_wait_fault(1, 20_000_000)
    try:
        kda.kda_ssm_forward(**c)
        assert kda.kda_get_device_status() == STATUS["KDA_ERR_TIMEOUT"]
    finally:
        kda.kda_debug_set_wait_fault(0)
    y, S = kda.kda_ssm_forward(**c)
    assert kda.kda_get_device_status() == 0 and torch.equal(y, want[0]) and torch.equal(S, want[1])


@gpu
def test_a_layer_as_it_is_served():
    """Convolution, scan, a fork of both states to three continuations, single tokens, compaction: each
    sequence's outputs equal one prompt over all its tokens."""
    T, more, H, G, N, P = 150, 6, 4, 2, 64, 64
    C, n_slots = H * P + 2 * G * N, 12
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w, b = (r(C, 4) * 0.5).bfloat16(), (r(C) * 0.1).bfloat16()
    A, D, bias = -1 - 3 * torch.rand(H, generator=g, device="cuda"), r(H), r(H) - 3
    prompt, tails = r(1, T, C).bfloat16(), r(3, more, C).bfloat16()
    dt_p, dt_t = r(1, T, H).bfloat16(), r(3, more, H).bfloat16()
    cut = lambda u: (u[..., :H * P].unflatten(-1, (H, P)), u[..., H * P:H * P + G * N].unflatten(-1, (G, N)),  # noqa: E731
                     u[..., H * P + G * N:].unflatten(-1, (G, N)))
    conv_pool = torch.zeros((n_slots, 3, C), dtype=torch.bfloat16, device="cuda")
    scan_pool = torch.zeros((n_slots, H, N, P), device="cuda")
    u, conv_pool[7:8] = kda.kda_short_conv(prompt, w, b)
    x, Bm, Cm = cut(u)
    _, scan_pool[7:8] = kda.kda_ssm_forward(x, dt_p, A, Bm, Cm, D, bias)
    ids = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kda.kda_pool_copy([conv_pool, scan_pool], ids(7, 7), ids(10, 3))
    slots = ids(7, 10, 3)
    got = []
    for t in range(more):
        if t == more // 2:
            slots = kda.kda_pool_compact([conv_pool, scan_pool], slots)
            assert sorted(slots.tolist()) == [0, 1, 2]
        u = kda.kda_short_conv_step_paged(tails[:, t], w, conv_pool, slots, b)
        x, Bm, Cm = cut(u)
        got.append(kda.kda_ssm_decode_step_paged(x, dt_t[:, t], A, Bm, Cm, scan_pool, slots, D, bias))
    got = torch.stack(got, 1)
    assert kda.kda_get_device_status() == 0
    for i in range(3):
        whole = torch.cat([prompt, tails[i:i + 1]], 1)
        u, _ = kda.kda_short_conv(whole, w, b)
        x, Bm, Cm = cut(u)
        ry, rS, ya, Sa = ref.scan(np64(x[0]), np64(torch.cat([dt_p, dt_t[i:i + 1]], 1)[0]), np64(A), np64(Bm[0]), np64(Cm[0]),
                                  np64(D), np64(bias))
        by, bS = ref.scan_bounds(ry, ya, Sa, T + more, N, "bf16", "tcgen05")
        assert np.all(np.abs(np64(got[i]) - ry[T:]) <= by[T:]), i
        assert np.all(np.abs(np64(scan_pool[int(slots[i])]) - rS) <= bS), i


@gpu
def test_convolution_feeds_the_kda_prefill():
    """q, k, v through the convolution, then the prefill with the fused prologue: parity with the oracle on
    the convolution's outputs, and the state carried over two parts of the prompt."""
    import oracle
    from helpers import max_rel_err
    B, T, H, d = 1, 130, 2, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    proj, w = r(B, T, 3 * H * d), (r(3 * H * d, 4) * 0.5)
    zg, zb = r(B, T, H, d), r(B, T, H)
    u, _ = kda.kda_short_conv(proj, w)
    q, k, v = (t.unflatten(-1, (H, d)).contiguous() for t in u.split(H * d, -1))
    o, S = kda.kda_forward_chunked_fused(q, k, v, zg, zb)
    o_ref, S_ref = oracle.forward_fused(q, k, v, zg, zb)
    assert max_rel_err(np64(o), o_ref) <= 2e-2 and max_rel_err(np64(S), S_ref) <= 2e-2


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("T,P", [(130, 64), (130, 128), (2048, 64), (2048, 128)])
def test_a_rate_of_nan_shows(dtype, impl, T, P):
    """A NaN in one head's A makes all of that head's outputs and its state NaN, in short prompts and in long ones
    that are cut into segments, and leaves the other heads as they were."""
    c = case((1, T), 3, 1, 128, P, dtype, seed=2)
    want, want_S = kda.kda_ssm_forward(**c, impl=impl)
    c["A"] = c["A"].clone()
    c["A"][1] = float("nan")
    y, S = kda.kda_ssm_forward(**c, impl=impl)
    assert bool(y[:, :, 1].isnan().all()) and bool(S[:, 1].isnan().all())
    assert torch.equal(y[:, :, ::2], want[:, :, ::2]) and torch.equal(S[:, ::2], want_S[:, ::2])


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("T", [1, 130, 256, 2050])
def test_a_rate_of_minus_infinity_forgets_everything(dtype, impl, T):
    """A = -infinity: every token starts from nothing.  The rows after the last token do not decay its state."""
    c = case((1, T), 3, 1, 128, 64, dtype, seed=4)
    c["A"][1] = -float("inf")
    y, S = kda.kda_ssm_forward(**c, impl=impl)
    assert kda.kda_get_device_status() == 0
    check(y[0], S[0], c, 0, 0, dtype, impl)


@gpu
@pytest.mark.parametrize("dtype,impl", IMPLS)
@pytest.mark.parametrize("offsets,status", [([0, 0, 0], OK), ([0, 5, 3], INVALID), ([0, 0, 1], INVALID), ([-1, 0, 0], INVALID)])
def test_packed_without_tokens(dtype, impl, offsets, status):
    """No tokens at all: the states pass through, and offsets that promise some are reported."""
    c = case((0,), 2, 1, 64, 128, dtype, states=2)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y, S = kda.kda_ssm_forward_varlen(**c, cu_seqlens=cu, impl=impl)
    assert kda.kda_get_device_status() == status
    assert y.shape == (0, 2, 128) and torch.equal(S, c["S0"])
    _, S = kda.kda_ssm_forward_varlen(**{**c, "S0": None}, cu_seqlens=cu, impl=impl)
    assert kda.kda_get_device_status() == status and bool((S == 0).all())
    held = c["S0"].clone()
    kda.kda_ssm_forward_varlen(**{**c, "S0": held}, cu_seqlens=cu, impl=impl, S_T=held)
    assert kda.kda_get_device_status() == status and torch.equal(held, c["S0"])
    kda.kda_ssm_forward_varlen(**c, cu_seqlens=cu, impl=impl, return_state=False)
    assert kda.kda_get_device_status() == status


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,P", [(64, 64), (128, 128)])
def test_no_skip_term_adds_nothing_to_infinities(dtype, N, P):
    """Without D there is no D x: an infinite x among positive B and C makes its column's outputs infinite from that
    token on, not 0 times infinity.  Token-serial kernel and single tokens."""
    c = case((1, 5), 2, 1, N, P, dtype, seed=6)
    del c["D"]
    for k in ("x", "Bm", "Cm", "S0"):
        c[k] = c[k].abs() + 0.125
    c["x"][0, 2, 1, 7] = float("inf")
    y, S = kda.kda_ssm_forward(**c, impl="simt")
    held = c["S0"].clone()
    steps = [kda.kda_ssm_decode_step(c["x"][:, t], c["dt"][:, t], c["A"], c["Bm"][:, t], c["Cm"][:, t], held, None, c["dt_bias"])
             for t in range(5)]
    for out, state in ((y, S), (torch.stack(steps, 1), held)):
        inf = torch.zeros(1, 5, 2, P, dtype=torch.bool, device="cuda")
        inf[0, 2:, 1, 7] = True
        assert torch.equal(out == float("inf"), inf) and bool(out[~inf].isfinite().all())
        assert bool((state[0, 1, :, 7] == float("inf")).all()) and int(state.isfinite().sum()) == state.numel() - N


@gpu
@pytest.mark.parametrize("T,H,P", [(4096, 2, 128), (1700, 1, 64)])
def test_a_wait_that_runs_out_in_a_segment_is_reported(T, H, P):
    """The launch over the segments' states ends by itself when one of its waits runs out (the launch after it has all
    its hand-offs), says so, and the next call is as if nothing had been."""
    c = case((1, T), H, 1, 128, P, "bf16", seed=8)
    assert kda.ssm_workspace_bytes(1, T, H, 128, P) > 0
    want = kda.kda_ssm_forward(**c)
    kda.kda_debug_set_wait_fault(1, 20_000_000)
    try:
        kda.kda_ssm_forward(**c)
        assert kda.kda_get_device_status() == STATUS["KDA_ERR_TIMEOUT"]
    finally:
        kda.kda_debug_set_wait_fault(0)
    for _ in range(3):
        y, S = kda.kda_ssm_forward(**c)
        assert kda.kda_get_device_status() == 0 and torch.equal(y, want[0]) and torch.equal(S, want[1])


@gpu
@pytest.mark.parametrize("B,T,H,G,N,P", LONG + [(1, 3000, 6, 2, 128, 64)])
def test_segments_with_what_is_optional(B, T, H, G, N, P):
    """Prompts cut into segments without S0, without D and dt_bias, without a wanted state, from slices of wider rows.
    The workspace starts as NaN: what is read of it was written."""
    c = case((B, T), H, G, N, P, "bf16", seed=T + 1, rate=1.5)
    need = kda.ssm_workspace_bytes(B, B * T, H, N, P)
    assert need > 0
    ws = lambda: torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # noqa: E731
    bare = {k: c[k] for k in ("x", "dt", "A", "Bm", "Cm")}
    y, S = kda.kda_ssm_forward(**bare, workspace=ws())
    assert kda.kda_get_device_status() == 0
    for b in range(B):
        check(y[b], S[b], c, b, b, "bf16", "tcgen05", skip=False, start=False)
    y1, none = kda.kda_ssm_forward(**bare, workspace=ws(), return_state=False)
    assert none is None and torch.equal(y, y1)
    want, want_S = kda.kda_ssm_forward(**c)
    y2, none = kda.kda_ssm_forward(**c, workspace=ws(), return_state=False)
    assert none is None and torch.equal(y2, want)
    wide = torch.full((B, T, H * P + 2 * G * N + H + 8 - H % 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    parts, at = {}, 0
    for k, n in (("x", H * P), ("Bm", G * N), ("Cm", G * N), ("dt", H)):
        wide[..., at:at + n] = c[k].flatten(2)
        parts[k] = wide[..., at:at + n].unflatten(2, c[k].shape[2:])
        at += n
    y3, S3 = kda.kda_ssm_forward(**{**c, **parts}, workspace=ws())
    assert torch.equal(y3, want) and torch.equal(S3, want_S)


@gpu
@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("lengths,H", [([1, 130, 257, 384, 511, 640, 90, 256] * 3, 24), ([3000, 0, 129, 2500, 1500], 2)])
def test_every_call_beside_heavy_traffic(P, lengths, H):
    """As above, each of a thousand calls compared on the device: short packed prompts, and prompts cut into segments."""
    T = sum(lengths)
    c = case((T,), H, 2, 128, P, "bf16", seed=11, states=len(lengths))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    y0, S0 = kda.kda_ssm_forward_varlen(**c, cu_seqlens=cu)
    a, b = (torch.empty(1 << 28, dtype=torch.uint8, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bad = torch.zeros((), dtype=torch.int32, device="cuda")
    y, S = torch.empty_like(y0), torch.empty_like(S0)
    for i in range(1000):
        if i % 4 == 0:
            with torch.cuda.stream(side):
                b.copy_(a)
        y.fill_(7.0)
        S.fill_(7.0)
        kda.kda_ssm_forward_varlen(**c, cu_seqlens=cu, y=y, S_T=S)
        bad += ((y != y0).any() | (S != S0).any()).int()
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0
    assert int(bad) == 0


@gpu
@pytest.mark.parametrize("N,P", [(64, 64), (128, 128)])
def test_a_long_memory_does_not_drift(N, P):
    """Decays of 0.999 a token, positive inputs: the roundings of a thousand remembered decays and updates do not add up
    to one side.  Each token rounds its decay (shared by the state's elements) and twice each element, by up to 2^-24
    of the value between one step and the next, 2^-24 / sqrt(12) in the mean square; sqrt(500) remembered tokens make
    3.8e-7 of the decays, six times that 2.3e-6, and the elements' own roundings average out.  Token-serial kernel
    and single tokens."""
    T, H = 4096, 2
    c = case((1, T), H, 1, N, P, "fp32", seed=12)
    for k in ("x", "Bm", "Cm", "S0"):
        c[k] = c[k].abs()
    c["A"].fill_(-0.02)
    c["dt"].mul_(0.2)
    c["dt_bias"].fill_(float(np.log(np.expm1(0.05))))
    step = torch.logaddexp(c["dt"][0].double() + c["dt_bias"].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    left = (step * c["A"].double()).cumsum(0)
    want = torch.einsum("tn,th,thp->hnp", c["Bm"][0, :, 0].double(), step * torch.exp(left[-1:] - left), c["x"][0].double()) \
        + torch.exp(left[-1])[:, None, None] * c["S0"][0].double()
    drift = lambda S: float(((S.double() - want) / want).mean().abs())  # noqa: E731
    _, S = kda.kda_ssm_forward(**c, impl="simt")
    assert drift(S[0]) <= 2.3e-6
    held = c["S0"].clone()
    for t in range(T):
        kda.kda_ssm_decode_step(c["x"][:, t], c["dt"][:, t], c["A"], c["Bm"][:, t], c["Cm"][:, t], held, c["D"], c["dt_bias"])
    assert drift(held[0]) <= 2.3e-6


@gpu
@pytest.mark.parametrize("B,H,P", [(4, 96, 64), (1, 2, 64), (1, 2, 128)])
def test_a_long_memory_of_the_tensor_core(B, H, P):
    """Without decay and from positive inputs the tensor core's sums lose at most 16 * 2^-23 of the state a chunk, the
    weights and weighted x at most 3 * 2^-16 of a term: in one run of chunks, and cut into segments."""
    T, N = 4096, 128
    c = case((B, T), H, 1, N, P, "bf16", seed=13)
    for k in ("x", "Bm", "S0"):
        c[k] = c[k].abs()
    c["A"].zero_()
    _, S = kda.kda_ssm_forward(**c, impl="tcgen05")
    step = torch.logaddexp(c["dt"][0, :, :2].double() + c["dt_bias"][:2].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    want = torch.einsum("tn,th,thp->hnp", c["Bm"][0, :, 0].double(), step, c["x"][0, :, :2].double()) + c["S0"][0, :2].double()
    assert bool(((S[0, :2].double() - want).abs() <= (T // 128 * 16 * 2.0 ** -23 + 3 * 2.0 ** -16 + 2.0 ** -20) * want).all())
