"""The short causal convolution: prompts (batched, packed), single tokens (plain, paged), against fp64."""
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
BASE, SZ = 0x7F0000000000, 1 << 32

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from linear_attention_recurrence_forward_b200 import build
    build.build()
    return kda.lib()


# ---------------------------------------------------------------------- refusals (CPU)

def ptrs():
    return dict(x=BASE, w=BASE + SZ, bias=BASE + 2 * SZ, st=BASE + 3 * SZ, y=BASE + 4 * SZ, so=BASE + 5 * SZ,
                cu=BASE + 6 * SZ)


def call(L, form="batch", B=2, T=10, C=128, W=4, ldx=None, ldy=None, act=1, dtype=0, n_slots=8, **p):
    a = {**ptrs(), **p}
    ldx, ldy = ldx or C, ldy or C
    if form == "batch":
        return L.kda_short_conv(a["x"], a["w"], a["bias"], a["st"], a["y"], a["so"], B, T, C, W, ldx, ldy, act, dtype, None)
    if form == "varlen":
        return L.kda_short_conv_varlen(a["x"], a["w"], a["bias"], a["cu"], a["st"], a["y"], a["so"], B, T, C, W, ldx, ldy,
                                       act, dtype, None)
    if form == "step":
        return L.kda_short_conv_step(a["x"], a["w"], a["bias"], a["st"], a["y"], B, C, W, ldx, ldy, act, dtype, None)
    return L.kda_short_conv_step_paged(a["x"], a["w"], a["bias"], a["st"], n_slots, a["cu"], a["y"], B, C, W, ldx, ldy,
                                       act, dtype, None)


@pytest.mark.parametrize("form", ["batch", "varlen", "step", "paged"])
def test_refusals(L, form):
    f = lambda **k: call(L, form, **k)  # noqa: E731
    for k in (dict(B=0), dict(B=-1), dict(C=0), dict(ldx=64), dict(ldy=64), dict(x=None), dict(w=None), dict(y=None)):
        assert f(**k) == INVALID, k
    for k in (dict(W=1), dict(W=5), dict(C=12), dict(dtype=2), dict(act=2)):
        assert f(**k) == UNSUPPORTED, k
    for k in (dict(x=BASE + 8), dict(w=BASE + SZ + 2), dict(bias=BASE + 2 * SZ + 4), dict(st=BASE + 3 * SZ + 8),
              dict(y=BASE + 4 * SZ + 8), dict(ldx=132), dict(ldy=132)):
        assert f(**k) == MISALIGNED, k
    assert f(y=BASE + 16) == INVALID                       # y inside x
    assert f(y=BASE + SZ) == INVALID                       # y on the weights
    assert f(y=BASE + 3 * SZ + 16) == INVALID              # y inside the state
    assert f(ldx=256, y=BASE + 256) == INVALID             # y between the rows of x
    if form in ("batch", "varlen"):
        assert f(T=-1) == INVALID
        assert f(so=BASE + 3 * SZ + 16) == INVALID         # the new state partly over the old one
        assert f(so=BASE + 4 * SZ) == INVALID              # the new state on y
        assert f(so=BASE + 5 * SZ + 8) == MISALIGNED
    if form == "varlen":
        assert f(cu=None) == INVALID
        assert f(cu=BASE + 6 * SZ + 2) == MISALIGNED
        assert f(cu=BASE + 4 * SZ) == INVALID              # offsets under y
    if form in ("step", "paged"):
        assert f(st=None) == INVALID
    if form == "paged":
        assert f(n_slots=0) == INVALID
        assert f(cu=None) == INVALID                       # the slot table
        assert f(cu=BASE + 3 * SZ) == INVALID              # the slot table inside the pool


@pytest.mark.parametrize("form", ["batch", "varlen", "step", "paged"])
def test_counts_near_32_bits_are_refused(L, form):
    """More than 2e9 tokens of a sequence, or sequences: sums with a strip or a group would pass 32 bits."""
    far = {k: BASE + i * (1 << 42) for i, k in enumerate(ptrs())}
    assert call(L, form, B=2 ** 31 - 2, T=0, C=8, **far) == INVALID
    if form in ("batch", "varlen"):
        assert call(L, form, B=1, T=2 ** 31 - 2, C=8, **far) == INVALID


def test_binding_refuses_bad_tensors():
    x, w = torch.zeros(2, 5, 64), torch.zeros(64, 4)
    with pytest.raises(ValueError):
        kda.kda_short_conv(x, w)                           # not on a GPU
    with pytest.raises(ValueError):
        kda.kda_short_conv(x.half(), w.half())             # dtype
    with pytest.raises(ValueError):
        kda.kda_short_conv(x, torch.zeros(32, 4))          # another channel count
    with pytest.raises(ValueError):
        kda.kda_short_conv(x, w, activation="relu")
    with pytest.raises(ValueError):
        kda.kda_short_conv(x.transpose(0, 1), w)           # rows that are not evenly spaced
    with pytest.raises(ValueError):
        kda.kda_short_conv(torch.zeros(2, 5, 128)[..., ::2], w)


# ---------------------------------------------------------------------- GPU

def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(TORCH[dtype])


def check(y, ref_y, mag, dtype):
    err = np.abs(np64(y) - ref_y)
    assert np.all(err <= ref.conv_bound(ref_y, mag, dtype)), float(err.max())


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,C,W", [(1, 1, 64, 4), (3, 2, 8, 4), (2, 3, 72, 4), (1, 4, 1032, 3), (2, 67, 1160, 4),
                                     (1, 300, 2048, 2), (5, 129, 384, 4), (1, 5000, 64, 3)])
def test_prompt(dtype, B, T, C, W):
    x, w = rand((B, T, C), dtype, 1), rand((C, W), dtype, 2, 0.5)
    b, st = rand((C,), dtype, 3, 0.3), rand((B, W - 1, C), dtype, 4)
    for bias, state, act in ((b, st, "silu"), (None, None, None)):
        y, so = kda.kda_short_conv(x, w, bias, state, activation=act)
        assert kda.kda_get_device_status() == 0
        for i in range(B):
            ry, rs, mag = ref.conv(np64(x[i]), np64(w), None if bias is None else np64(bias),
                                   None if state is None else np64(state[i]), act == "silu")
            check(y[i], ry, mag, dtype)
            assert np.array_equal(np64(so[i]), rs)         # the state is copied, not computed


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_packed(dtype, W):
    lengths, lead, tail, C = [1, 0, 2, 3, 4, 200, 0, 65, 1, 7, 64], 5, 3, 1096
    T = lead + sum(lengths) + tail
    x, w, b = rand((T, C), dtype, 1), rand((C, W), dtype, 2, 0.5), rand((C,), dtype, 3, 0.3)
    x[:lead] = float("nan")                                # rows of no sequence reach nothing
    x[T - tail:] = float("inf")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]) + lead, dtype=torch.int32, device="cuda")
    st = rand((len(lengths), W - 1, C), dtype, 4)
    before = st.clone()
    y = torch.full((T, C), 7.0, dtype=TORCH[dtype], device="cuda")
    y, so = kda.kda_short_conv_varlen(x, w, cu, b, st, y=y, state_out=st)        # the state in place
    assert so is st and kda.kda_get_device_status() == 0
    at = lead
    for n, k in enumerate(lengths):
        ry, rs, mag = ref.conv(np64(x[at:at + k]), np64(w), np64(b), np64(before[n]))
        check(y[at:at + k], ry, mag, dtype)
        assert np.array_equal(np64(so[n]), rs), n
        at += k
    assert bool((y[:lead] == 7).all()) and bool((y[T - tail:] == 7).all())


@gpu
def test_slices_of_wider_rows_and_split_prompts():
    """q, k, v slices of one projection, and a prompt in two parts carrying the state."""
    B, T, C = 2, 150, 128
    wide = rand((B, T, 3 * C + 8), "bf16", 1)
    w = rand((C, 4), "bf16", 2, 0.5)
    for i in range(3):
        x = wide[..., i * C:(i + 1) * C]
        y, so = kda.kda_short_conv(x, w)
        y2, so2 = kda.kda_short_conv(x.contiguous(), w)
        assert torch.equal(y, y2) and torch.equal(so, so2)
    x = wide[..., :C].contiguous()
    whole, end = kda.kda_short_conv(x, w)
    out = torch.zeros((B, T, 2 * C), dtype=torch.bfloat16, device="cuda")
    for b in range(B):      # one batch entry: any row spacing of its part
        y1, s1 = kda.kda_short_conv(x[b:b + 1, :70], w, y=out[b:b + 1, :70, C:])
        y2, s2 = kda.kda_short_conv(x[b:b + 1, 70:], w, None, s1, y=out[b:b + 1, 70:, C:])
        assert torch.equal(s2[0], end[b])
    assert torch.equal(out[..., C:], whole) and bool((out[..., :C] == 0).all())


@gpu
def test_empty_prompt_keeps_the_state():
    st = rand((2, 3, 64), "bf16", 1)
    x = torch.empty((2, 0, 64), dtype=torch.bfloat16, device="cuda")
    y, so = kda.kda_short_conv(x, rand((64, 4), "bf16", 2), None, st)
    assert y.shape == (2, 0, 64) and torch.equal(so, st)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    y, so = kda.kda_short_conv_varlen(x[0], rand((64, 4), "bf16", 2), cu, None, st)
    assert torch.equal(so, st) and kda.kda_get_device_status() == 0


@gpu
@pytest.mark.parametrize("bad", [[0, 50, 130], [-2, 50, 100], [0, 70, 60]])
def test_invalid_offsets_are_reported_not_followed(bad):
    x, w, st = rand((100, 64), "bf16", 1), rand((64, 4), "bf16", 2), rand((2, 3, 64), "bf16", 3)
    y = torch.full((100, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    y, so = kda.kda_short_conv_varlen(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), None, st, y=y)
    assert kda.kda_get_device_status() == INVALID
    assert torch.equal(so, st) and bool((y == 7).all())


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,C,W", [(1, 64, 4), (7, 1160, 4), (64, 4096, 3), (300, 72, 2)])
def test_steps_continue_a_prompt(dtype, B, C, W):
    """A prompt, then single tokens, equals the whole prompt: plain and paged, bit for bit."""
    T, more = 9, 5
    x, w, b = rand((B, T + more, C), dtype, 1), rand((C, W), dtype, 2, 0.5), rand((C,), dtype, 3, 0.3)
    whole, end = kda.kda_short_conv(x, w, b)
    _, st = kda.kda_short_conv(x[:, :T].contiguous(), w, b)
    n_slots = B + 3
    slots = torch.randperm(n_slots, device="cuda")[:B].to(torch.int32)
    pool = rand((n_slots, W - 1, C), dtype, 5)
    untouched = pool.clone()
    pool[slots.long()] = st
    for t in range(T, T + more):
        y = kda.kda_short_conv_step(x[:, t], w, st, b)
        yp = kda.kda_short_conv_step_paged(x[:, t].contiguous(), w, pool, slots, b)
        assert torch.equal(y, whole[:, t]) and torch.equal(yp, y)
    assert torch.equal(st, end) and torch.equal(pool[slots.long()], end)
    free = torch.ones(n_slots, dtype=torch.bool, device="cuda")
    free[slots.long()] = False
    assert torch.equal(pool[free], untouched[free]) and kda.kda_get_device_status() == 0


@gpu
def test_paged_step_skips_and_reports():
    pool, w = rand((4, 3, 64), "bf16", 1), rand((64, 4), "bf16", 2)
    before = pool.clone()
    slots = torch.tensor([2, -1, 4], dtype=torch.int32, device="cuda")
    y = torch.full((3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_short_conv_step_paged(rand((3, 64), "bf16", 3), w, pool, slots, y=y)
    assert kda.kda_get_device_status() == INVALID           # slot 4 of 4
    assert bool((y[1:] == 7).all()) and not bool((y[0] == 7).all())
    assert torch.equal(pool[[0, 1, 3]], before[[0, 1, 3]])


@gpu
def test_on_a_stream_and_in_a_graph():
    x, w, st = rand((2, 40, 256), "bf16", 1), rand((256, 4), "bf16", 2), rand((2, 3, 256), "bf16", 3)
    y0, s0 = kda.kda_short_conv(x, w, None, st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, s1 = kda.kda_short_conv(x, w, None, st, stream=side)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(s0, s1)
    graph = torch.cuda.CUDAGraph()
    live = st.clone()
    tok = x[:, 0].contiguous()
    with torch.cuda.graph(graph):
        yg = kda.kda_short_conv_step(tok, w, live)
    expect = st.clone()
    for t in range(3):
        tok.copy_(x[:, t])
        graph.replay()
        ye = kda.kda_short_conv_step(x[:, t], w, expect)
        assert torch.equal(yg, ye)
    assert torch.equal(live, expect)


@gpu
def test_extreme_values():
    """Large negative and positive inputs saturate the activation without NaN; infinities stay in their window."""
    w = torch.tensor([[0, 0, 0, 1.0]] * 8, device="cuda")
    x = torch.tensor([-1e4, 1e4, -88.0, 0.0, 3e38], device="cuda")[:, None].expand(5, 8).contiguous()[None]
    y, _ = kda.kda_short_conv(x, w)
    ry, _, mag = ref.conv(np64(x[0]), np64(w), None, None)
    check(y[0], ry, mag, "fp32")
    x = rand((1, 30, 64), "bf16", 1)
    x[0, 10] = float("inf")
    y, _ = kda.kda_short_conv(x, rand((64, 4), "bf16", 2))
    assert bool(torch.isfinite(y[0, :10].float()).all()) and bool(torch.isfinite(y[0, 14:].float()).all())


@gpu
@pytest.mark.parametrize("step", [False, True])
def test_fp32_activation_to_the_last_places(step):
    """SiLU of single values in fp32, relative to each value: the exponential (2^-22), its correction, a product,
    a sum and the last product (2^-24 each) and the reciprocal (2^-23) make 10 * 2^-24; below the normal numbers
    the exponential is off by up to 4 of the smallest steps, 2^-149, times the value."""
    v = torch.cat([torch.linspace(-104, 90, 40000, device="cuda"), torch.linspace(-1, 1, 9992, device="cuda"),
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e38, -3e38, -87.4, -88.8], device="cuda")])
    w = torch.zeros(8, 4, device="cuda")
    w[:, 3] = 1
    x = v.reshape(1, -1, 8)
    if step:
        y = kda.kda_short_conv_step(x[0], w, torch.zeros(x.shape[1], 3, 8, device="cuda"))
    else:
        y, _ = kda.kda_short_conv(x, w)
    z = np64(v)
    e = np.exp(-np.abs(z))
    ref_y = np.where(z < 0, z * e, z) / (1 + e)
    err = np.abs(np64(y).ravel() - ref_y)
    assert np.all(err <= 10 * 2.0 ** -24 * np.abs(ref_y) + 2.0 ** -147 * (1 + np.abs(z))), float((err / np.abs(ref_y + 1e-300)).max())
    assert bool(torch.isnan(kda.kda_short_conv(torch.full((1, 1, 8), float("nan"), device="cuda"), w)[0]).all())
    assert bool((kda.kda_short_conv(torch.full((1, 1, 8), float("inf"), device="cuda"), w)[0] == float("inf")).all())


@gpu
def test_slices_of_a_projection_feed_the_prefill_without_copies():
    """A call for each of q, k and v, slices of one projection: contiguous outputs that the KDA prefill takes as they
    are, equal to those of one call over all three, and states that carry the prompt on."""
    B, T, H, d = 2, 130, 2, 64
    C = H * d
    proj, w = rand((B, T, 3 * C), "bf16", 1), rand((3 * C, 4), "bf16", 2, 0.5)
    g, beta = -rand((B, T, H, d), "bf16", 3).abs(), rand((B, T, H), "bf16", 4).sigmoid()
    whole, end = kda.kda_short_conv(proj, w)
    parts = [kda.kda_short_conv(proj[..., i * C:(i + 1) * C], w[i * C:(i + 1) * C]) for i in range(3)]
    for i, (y, st) in enumerate(parts):
        assert y.is_contiguous() and torch.equal(y, whole[..., i * C:(i + 1) * C])
        assert torch.equal(st, end[..., i * C:(i + 1) * C])
    q, k, v = (y.view(B, T, H, d) for y, _ in parts)
    q, k = (torch.nn.functional.normalize(t.float(), dim=-1).bfloat16() for t in (q, k))
    o, S = kda.kda_forward_chunked(q, k, v, g, beta)
    assert kda.kda_get_device_status() == 0 and bool(o.isfinite().all()) and bool(S.isfinite().all())
