"""GPU parity of the layer operators against the float64 oracle, entry by entry.

Tolerances count roundings (half a step: bf16 2^-8, fp32 2^-24 of the value):
* rotary: two products and a sum in fp32 on sines and cosines good to 2^-22,
  then the output's rounding;
* linear attention: with A the same sums over absolute values, every term of an
  output passes at most one rounding to bf16 (its weight, or its state) besides
  the output's own, and fp32 sums of at most 256 terms a chunk; state updates
  carry two bf16 parts (2^-17; three, and nothing lost, where the state is
  returned) on the tensor cores, and one more fp32 rounding per chunk;
* norms: sums over a row in fp32 (a tree, counted as 64 roundings with the
  exponential and divisions), weight gradients over the rows in fp32.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_chunk_02_b200 import gdn
from oracle import layer_oracle as L

pytestmark = pytest.mark.gpu
U32, UBF, USTATE = 2.0 ** -24, 2.0 ** -8, 2.0 ** -17
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
half_step = lambda dtype: UBF if dtype == "bf16" else U32


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, want, tol, name):
    got = f64(got)
    assert got.shape == want.shape, name
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(np.abs(got - want)[bad].max()),
                           tuple(int(i[0]) for i in np.nonzero(bad)))


def rand(gen, *shape, dtype="f32", scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(DT[dtype]).cuda()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


@pytest.fixture(autouse=True)
def _status():
    yield
    torch.cuda.synchronize()
    assert gdn.gdn_get_status() == gdn.GDN_OK


# --------------------------------------------------------------------------- #
# rotary
# --------------------------------------------------------------------------- #
def rotary_tol(x, inv, m, inter, dtype):
    """Sum of the magnitudes of a pair's two terms, at most m (|a| + |b|)."""
    half = len(inv)
    mag = np.abs(x).copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        s = m * (np.abs(x[..., a]) + np.abs(x[..., b]))
        mag[..., a] = mag[..., b] = s
    return mag * (half_step(dtype) + 8 * 2.0 ** -23) * 1.01


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [128, 64, 16, 2, 10, 126])
def test_rotary(lib, dtype, inter, rot):
    B, Hq, Hk, T = 2, 5, 2, 19
    g = gen(rot)
    q, k = rand(g, B, Hq, T, 128, dtype=dtype), rand(g, B, Hk, T, 128, dtype=dtype)
    inv, m = gdn.gdn_rotary_frequencies(rot, scaling="yarn", factor=4.0, original_length=4096)
    pos = torch.randint(0, 1 << 20, (B, T), generator=g).cuda()
    for back in (False, True):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        gdn.gdn_rotary(q, k, pos, inv.cuda(), qo, ko, mscale=m, interleaved=inter, inverse=back)
        for x, y, name in ((q, qo, "q"), (k, ko, "k")):
            want = L.rotary(f64(x), f64(pos), f64(inv), m, inter, back)
            near(y, want, rotary_tol(f64(x), inv, m, inter, dtype), name)
        # in place, and the copied columns bit for bit
        qi, ki = q.clone(), k.clone()
        gdn.gdn_rotary(qi, ki, pos, inv.cuda(), qi, ki, mscale=m, interleaved=inter, inverse=back)
        assert torch.equal(qi, qo) and torch.equal(ki, ko)
        assert torch.equal(qo[..., rot:], q[..., rot:])


@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 0), (1, 1, 0, 3), (64, 1, 32, 16), (3, 17, 4, 4),
                                       (1, 4097, 9, 1)])
def test_rotary_strided_views_and_sizes(lib, B, T, Hq, Hk):
    """A fused projection's [B, T, heads, d] slices in, head-major out; far positions."""
    g = gen(T)
    fused = rand(g, B, T, Hq + Hk + 1, 128, dtype="bf16")
    keep = fused.clone()
    q = fused[:, :, :Hq].transpose(1, 2) if Hq else None
    k = fused[:, :, Hq:Hq + Hk].transpose(1, 2) if Hk else None
    inv, m = gdn.gdn_rotary_frequencies(128)
    pos = (torch.arange(T)[None] + torch.randint(0, 1 << 40, (B, 1), generator=g)).cuda()
    new = lambda x: None if x is None else torch.empty(x.shape, dtype=x.dtype, device="cuda")
    qo, ko = new(q), new(k)
    gdn.gdn_rotary(q, k, pos, inv.cuda(), qo, ko, mscale=m)
    # positions near 2^40: the angle's binary64 error is 2^-53 * 2^40 turns on top
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            want = L.rotary(f64(x), pos.cpu().numpy(), f64(inv), m)
            tol = rotary_tol(f64(x), inv, m, False, "bf16") + 2.0 ** -9 * np.abs(f64(x)).max()
            near(y, want, tol, "far")
    assert torch.equal(fused, keep)
    # the same in place on the fused buffer: nothing else moves
    gdn.gdn_rotary(q, k, pos, inv.cuda(), q, k, mscale=m)
    assert torch.equal(fused[:, :, Hq + Hk:], keep[:, :, Hq + Hk:])
    if q is not None:
        assert torch.equal(q, qo)


def test_rotary_copies_odd_values(lib):
    """Infinities and NaN outside the rotated columns stay where they are."""
    x = torch.zeros(1, 1, 3, 128, device="cuda")
    x[..., 64:] = float("inf")
    x[0, 0, 1, 100] = float("nan")
    inv, _ = gdn.gdn_rotary_frequencies(64)
    y = torch.empty_like(x)
    gdn.gdn_rotary(x, None, torch.arange(3, device="cuda")[None], inv.cuda(), y, None)
    assert torch.equal(y[..., 64:].nan_to_num(7.0), x[..., 64:].nan_to_num(7.0))
    assert (y[..., :64] == 0).all()


# --------------------------------------------------------------------------- #
# linear attention
# --------------------------------------------------------------------------- #
DECAYS = [-0.9, -0.05, -0.001, 0.0, -3.0, -0.3, -1e-5, -0.01]


def linear_case(seed, dtype, B, Hk, Hv, T, lens, carried):
    g = gen(seed)
    n = len(lens) if lens is not None else B
    c = dict(Q=rand(g, B, Hk, T, 128, dtype=dtype, scale=128 ** -0.5),
             K=rand(g, B, Hk, T, 128, dtype=dtype, scale=128 ** -0.5),
             V=rand(g, B, Hv, T, 128, dtype=dtype), dO=rand(g, B, Hv, T, 128, dtype=dtype),
             lg=torch.tensor((DECAYS * Hv)[:Hv]).cuda(), S0=None, dS=None, cu=None)
    if carried:
        c["S0"] = rand(g, n, Hv, 128, 128)
        c["dS"] = rand(g, n, Hv, 128, 128)
    if lens is not None:
        c["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    if lens is None:
        c["rows"] = [(b, 0, T) for b in range(B)]
    else:
        at = np.concatenate([[0], np.cumsum(lens)])
        c["rows"] = [(0, int(at[i]), lens[i]) for i in range(n)]
    return c


def oracle_linear(c, scale, absolute=False):
    """o, S over all sequences; of the absolute values if asked."""
    f = (lambda t: None if t is None else np.abs(f64(t))) if absolute else f64
    Q, K, V, S0 = (f(c[x]) for x in ("Q", "K", "V", "S0"))
    o, S = np.zeros(V.shape), np.zeros((len(c["rows"]), V.shape[1], 128, 128))
    for i, (b, a, n) in enumerate(c["rows"]):
        part = [x[b, :, a:a + n] for x in (Q, K, V)]
        o[b, :, a:a + n], S[i] = L.linear_forward(*part, f64(c["lg"]),
                                                  None if S0 is None else S0[i], scale)
    return o, S


def oracle_linear_grad(c, scale, absolute=False):
    f = (lambda t: None if t is None else np.abs(f64(t))) if absolute else f64
    Q, K, V, S0, dO, dS = (f(c[x]) for x in ("Q", "K", "V", "S0", "dO", "dS"))
    out = [np.zeros(Q.shape), np.zeros(K.shape), np.zeros(V.shape),
           np.zeros((len(c["rows"]), V.shape[1], 128, 128))]
    for i, (b, a, n) in enumerate(c["rows"]):
        q, k, v, do = (x[b, :, a:a + n] for x in (Q, K, V, dO))
        *g, e = L.linear_backward(q, k, v, f64(c["lg"]), None if S0 is None else S0[i], do,
                                  None if dS is None else dS[i], scale)
        for x, y in zip(out, g):
            x[b, :, a:a + n] = y
        out[3][i] = e
    return out


def out_tol(ref, mag, dtype, T):
    u = half_step(dtype)
    sums = (512 + T / 16) * U32
    return (u * np.abs(ref) + ((UBF + USTATE if dtype == "bf16" else 0.0) + sums) * mag) * 1.02 + 1e-30


def state_tol(mag, dtype, T):
    return ((USTATE if dtype == "bf16" else 0.0) + (512 + T / 16) * U32) * mag + 1e-30


def run_forward(c, scale, want_state=True):
    O = torch.full_like(c["V"], 77.0)
    S = torch.full((len(c["rows"]), c["V"].shape[1], 128, 128), 77.0, device="cuda") \
        if want_state else None
    n = gdn.gdn_linear_forward_workspace_bytes(c["K"], c["V"], c["cu"])
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")        # NaN everywhere
    gdn.gdn_linear_forward(c["Q"], c["K"], c["V"], c["lg"], c["S0"], O, S, ws, scale=scale,
                           cu_seqlens=c["cu"])
    return O, S


def run_backward(c, scale):
    outs = [torch.full_like(c[x], 77.0) for x in ("Q", "K", "V")]
    dS0 = torch.full((len(c["rows"]), c["V"].shape[1], 128, 128), 77.0, device="cuda")
    n = gdn.gdn_linear_backward_workspace_bytes(c["K"], c["V"], c["cu"])
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    gdn.gdn_linear_backward(c["Q"], c["K"], c["V"], c["lg"], c["S0"], c["dO"], c["dS"], *outs, dS0,
                            ws, scale=scale, cu_seqlens=c["cu"])
    return (*outs, dS0)


SHAPES = [                         # B, Hk, Hv, T, lens
    (1, 1, 1, 1, None), (2, 2, 2, 2, None), (1, 2, 4, 63, None), (1, 1, 2, 64, None),
    (1, 3, 3, 127, None), (2, 1, 1, 128, None), (1, 2, 2, 129, None), (1, 1, 3, 300, None),
    (1, 1, 8, 1025, None), (1, 1, 1, 1, [1]), (1, 1, 2, 40, [0, 1, 0, 33]),
    (1, 2, 4, 700, [128, 0, 129, 1, 127, 256]), (1, 1, 1, 1500, [5, 1400]),
    (1, 2, 2, 500, [0, 0, 0]), (1, 1, 2, 300, [1] * 70 + [3] * 20),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("carried", [False, True])
@pytest.mark.parametrize("B,Hk,Hv,T,lens", SHAPES)
def test_linear_forward(lib, dtype, carried, B, Hk, Hv, T, lens):
    c = linear_case(T, dtype, B, Hk, Hv, T, lens, carried)
    O, S = run_forward(c, 0.7)
    o, s = oracle_linear(c, 0.7)
    om, sm = oracle_linear(c, 0.7, absolute=True)
    used = T if lens is None else sum(lens)
    near(S, s, state_tol(sm, dtype, T), "S")
    near(O[:, :, :used], o[:, :, :used], out_tol(o, om, dtype, T)[:, :, :used], "O")
    assert (O[:, :, used:] == 77.0).all()              # rows of no sequence
    if not carried:
        O2, _ = run_forward(c, 0.7, want_state=False)
        assert torch.equal(O, O2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("carried", [False, True])
@pytest.mark.parametrize("B,Hk,Hv,T,lens", SHAPES)
def test_linear_backward(lib, dtype, carried, B, Hk, Hv, T, lens):
    c = linear_case(T + 1, dtype, B, Hk, Hv, T, lens, carried)
    got = run_backward(c, 0.7)
    want = oracle_linear_grad(c, 0.7)
    mag = oracle_linear_grad(c, 0.7, absolute=True)
    used = T if lens is None else sum(lens)
    near(got[3], want[3], state_tol(mag[3], dtype, T), "dS0")
    for x, y, m, name in zip(got, want[:3], mag, ("dQ", "dK", "dV")):
        near(x[:, :, :used], y[:, :, :used], out_tol(y, m, dtype, T)[:, :, :used], name)
        assert (x[:, :, used:] == 77.0).all(), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_long_is_cut_into_segments(lib, dtype):
    """Few heads over many rows: the call is cut, and its pieces fit together:
    the same rows as two calls with the state handed over."""
    T, cut = 6400, 3100
    c = linear_case(5, dtype, 1, 1, 2, T, None, True)
    assert gdn.gdn_linear_forward_workspace_bytes(c["K"], c["V"]) > 0
    O, S = run_forward(c, 1.0)
    o, s = oracle_linear(c, 1.0)
    om, sm = oracle_linear(c, 1.0, absolute=True)
    near(S, s, state_tol(sm, dtype, T), "S")
    near(O, o, out_tol(o, om, dtype, T), "O")
    got = run_backward(c, 1.0)
    want, mag = oracle_linear_grad(c, 1.0), oracle_linear_grad(c, 1.0, absolute=True)
    near(got[3], want[3], state_tol(mag[3], dtype, T), "dS0")
    for x, y, m, name in zip(got, want, mag, ("dQ", "dK", "dV")):
        near(x, y, out_tol(y, m, dtype, T), name)
    state = c["S0"]
    for a, b in ((0, cut), (cut, T)):
        part = {x: c[x][:, :, a:b].contiguous() for x in ("Q", "K", "V")}
        O1, state = run_forward(dict(c, **part, S0=state, rows=[(0, 0, b - a)]), 1.0)
        near(O1, o[:, :, a:b], out_tol(o, om, dtype, T)[:, :, a:b], "part")
    near(state, s, state_tol(sm, dtype, T), "state handed over")


def check_both_ways(c, dtype, T, forward=True, backward=True):
    if forward:
        O, S = run_forward(c, 0.7)
        o, s = oracle_linear(c, 0.7)
        om, sm = oracle_linear(c, 0.7, absolute=True)
        near(S, s, state_tol(sm, dtype, T), "S")
        near(O, o, out_tol(o, om, dtype, T), "O")
    if backward:
        got = run_backward(c, 0.7)
        want, mag = oracle_linear_grad(c, 0.7), oracle_linear_grad(c, 0.7, absolute=True)
        near(got[3], want[3], state_tol(mag[3], dtype, T), "dS0")
        for x, y, m, name in zip(got, want, mag, ("dQ", "dK", "dV")):
            near(x, y, out_tol(y, m, dtype, T), name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,backward", [(15, False), (5, True)])
def test_linear_some_are_cut(lib, dtype, B, backward):
    """Two lines more than one wave of 148 SMs takes: all but those stay whole."""
    Hk, Hv, T = 5, 10, 1300
    c = linear_case(7, dtype, B, Hk, Hv, T, None, True)
    size = (gdn.gdn_linear_backward_workspace_bytes if backward
            else gdn.gdn_linear_forward_workspace_bytes)(c["K"], c["V"])
    parts = 2 * (B * Hv * T * 128) * 4 if backward else 0          # of shared heads' gradients
    assert 0 < size - parts < B * Hv * 128 * 128 * 4
    check_both_ways(c, dtype, T, forward=not backward, backward=backward)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[2] * 40 + [1400, 0, 257], [130] * 3 + [9] * 33 + [900, 450, 260, 1],
                                  [0] * 35 + [1700],
                                  [1, 0, 2] * 400 + [300, 5] * 3 + [1200, 0, 130]])
def test_linear_packed_long_behind_short(lib, dtype, lens):
    c = linear_case(8, dtype, 1, 1, 2, sum(lens), lens, True)
    check_both_ways(c, dtype, sum(lens))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_no_rows_and_no_memory(lib, dtype):
    c = linear_case(6, dtype, 2, 1, 2, 0, None, True)
    _, S = run_forward(c, 1.0)
    assert torch.equal(S, c["S0"])
    assert torch.equal(run_backward(c, 1.0)[3], c["dS"])
    c = linear_case(7, dtype, 1, 1, 2, 200, None, False)
    c["lg"] = torch.tensor([float("-inf"), -200.0]).cuda()
    O, S = run_forward(c, 1.0)                          # o_t = v_t (k_t . q_t)
    o, s = oracle_linear(c, 1.0)
    om, sm = oracle_linear(c, 1.0, absolute=True)
    near(O, o, out_tol(o, om, dtype, 200), "O")
    near(S, s, state_tol(sm, dtype, 200), "S")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_rows_behind_and_between_do_not_leak(lib, dtype):
    """NaN and infinity in one packed sequence and behind the last leave the
    other sequences' results as they are."""
    lens = [70, 200, 130]
    c = linear_case(8, dtype, 1, 2, 2, 500, lens, True)
    good, goodS = run_forward(c, 1.0)
    grads = run_backward(c, 1.0)
    for x in ("Q", "K", "V", "dO"):
        c[x][:, :, 70:270:7] = float("nan")
        c[x][:, :, 75:270:7] = float("inf")
        c[x][:, :, 400:] = float("nan")
    O, S = run_forward(c, 1.0)
    for rows in (slice(0, 70), slice(270, 400)):
        assert torch.equal(O[:, :, rows], good[:, :, rows])
        for a, b in zip(run_backward(c, 1.0)[:3], grads):
            assert torch.equal(a[:, :, rows], b[:, :, rows])
    assert torch.equal(S[[0, 2]], goodS[[0, 2]])


@pytest.mark.parametrize("cu", [[0, 50, 40, 200], [0, 100, 300, 400], [-5, 20, 60, 100]])
def test_linear_bad_bounds_are_reported(lib, cu):
    c = linear_case(9, "bf16", 1, 1, 2, 300, [100, 100, 100], False)
    c["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
    run_forward(c, 1.0)
    assert gdn.gdn_get_status() == gdn.GDN_ERR_ARG
    run_backward(c, 1.0)
    assert gdn.gdn_get_status() == gdn.GDN_ERR_ARG


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_packed_rows_start_late(lib, dtype):
    """The first sequence need not start at row 0; the rows before it stay."""
    T, at = 400, [130, 131, 131, 300]
    c = linear_case(13, dtype, 1, 2, 4, T, [1, 0, 169], True)
    c["cu"] = torch.tensor(at, dtype=torch.int32).cuda()
    c["rows"] = [(0, 130, 1), (0, 131, 0), (0, 131, 169)]
    O, S = run_forward(c, 0.7)
    o, s = oracle_linear(c, 0.7)
    om, sm = oracle_linear(c, 0.7, absolute=True)
    near(S, s, state_tol(sm, dtype, T), "S")
    used = slice(130, 300)
    near(O[:, :, used], o[:, :, used], out_tol(o, om, dtype, T)[:, :, used], "O")
    got = run_backward(c, 0.7)
    want, mag = oracle_linear_grad(c, 0.7), oracle_linear_grad(c, 0.7, absolute=True)
    for x, y, m, name in zip(got, want[:3], mag, ("dQ", "dK", "dV")):
        near(x[:, :, used], y[:, :, used], out_tol(y, m, dtype, T)[:, :, used], name)
    for x in (O, *got[:3]):
        assert (x[:, :, :130] == 77.0).all() and (x[:, :, 300:] == 77.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_two_calls_at_once(lib, dtype):
    """Two streams, a workspace each: the bits of the calls one after the other."""
    cases = [linear_case(40 + i, dtype, 1, 1, 2, 2600, None, True) for i in range(2)]
    want = [(*run_forward(c, 1.0), *run_backward(c, 1.0)) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for c, st in zip(cases, streams):
        with torch.cuda.stream(st):
            got.append((*run_forward(c, 1.0), *run_backward(c, 1.0)))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# --------------------------------------------------------------------------- #
# single tokens
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hk,Hv,n", [(1, 1, 1, 1), (3, 2, 4, 5), (1, 8, 16, 4), (40, 2, 8, 1)])
def test_linear_decode(lib, dtype, B, Hk, Hv, n):
    g = gen(B + n)
    q = rand(g, B, Hk, n, 128, dtype=dtype, scale=128 ** -0.5)
    k = rand(g, B, Hk, n, 128, dtype=dtype, scale=128 ** -0.5)
    v = rand(g, B, Hv, n, 128, dtype=dtype)
    lg = torch.tensor((DECAYS * Hv)[:Hv]).cuda()
    pool = rand(g, B + 3, Hv, 128, 128)
    slots = torch.randperm(B + 3, generator=g)[:B].to(torch.int32)
    for at in (slots, None):
        S = pool.clone()
        O = torch.full_like(v, 77.0)
        gdn.gdn_linear_decode(q, k, v, lg, S, O, None if at is None else at.cuda(), scale=0.7)
        rows = range(B) if at is None else at.tolist()
        for b, s in enumerate(rows):
            args = (f64(q[b]), f64(k[b]), f64(v[b]), f64(lg))
            o, e = L.linear_forward(*args, f64(pool[s]), 0.7)
            om, em = L.linear_forward(*(np.abs(x) for x in args[:3]), args[3],
                                      np.abs(f64(pool[s])), 0.7)
            near(O[b], o, half_step(dtype) * np.abs(o) + 160 * U32 * om, "O")
            near(S[s], e, (4 * n + 4) * U32 * em, "S")
        rest = [i for i in range(B + 3) if i not in rows]
        assert torch.equal(S[rest], pool[rest])


def test_linear_decode_continues_a_prompt(lib):
    """A prompt's state, then its next tokens: as the longer prompt."""
    c = linear_case(11, "f32", 2, 1, 2, 140, None, False)
    o, s = oracle_linear(c, 1.0)
    om, sm = oracle_linear(c, 1.0, absolute=True)
    head = {x: c[x][:, :, :137].contiguous() for x in ("Q", "K", "V")}
    _, S = run_forward(dict(c, **head, rows=[(0, 0, 137), (1, 0, 137)]), 1.0)
    q, k, v = (c[x][:, :, 137:].contiguous() for x in ("Q", "K", "V"))
    O = torch.empty_like(v)
    gdn.gdn_linear_decode(q, k, v, c["lg"], S, O)
    near(O, o[:, :, 137:], out_tol(o, om, "f32", 140)[:, :, 137:], "O")
    near(S, s, state_tol(sm, "f32", 140), "S")


def test_linear_decode_slots_left_out_and_refused(lib):
    g = gen(12)
    x = rand(g, 6, 2, 1, 128)
    lg = torch.zeros(2).cuda()
    pool = rand(g, 4, 2, 128, 128)
    S, O = pool.clone(), torch.full_like(x, 77.0)
    gdn.gdn_linear_decode(x, x, x, lg, S, O, torch.tensor([2, -1, 0, -7, 1, -1],
                                                          dtype=torch.int32).cuda())
    assert gdn.gdn_get_status() == gdn.GDN_OK
    assert (O[[1, 3, 5]] == 77.0).all() and (O[[0, 2, 4]] != 77.0).any()
    assert torch.equal(S[3], pool[3])
    want, out = S.clone(), O.clone()
    # slot 4 is not there, slot 2 is named twice: those rows are left out and reported
    S, O = pool.clone(), torch.full_like(x, 77.0)
    gdn.gdn_linear_decode(x, x, x, lg, S, O, torch.tensor([2, 4, 0, 2, 1, 2 ** 31 - 1],
                                                          dtype=torch.int32).cuda())
    assert gdn.gdn_get_status() == gdn.GDN_ERR_ARG
    assert torch.equal(S, want) and torch.equal(O, out)


# --------------------------------------------------------------------------- #
# norms
# --------------------------------------------------------------------------- #
def norm_case(seed, dtype, B, T, H, d, parts, head_major=True):
    g = gen(seed)
    W = H * d
    y = rand(g, B, H, T, d, dtype=dtype).transpose(1, 2) if head_major \
        else rand(g, B, T, H, d, dtype=dtype)
    return dict(Y=y, Z=rand(g, B, T, W, dtype=dtype, scale=2.0) if "z" in parts else None,
                wo=rand(g, W) if "p" in parts else None,
                R=rand(g, B, T, W, dtype=dtype) if "r" in parts else None,
                wi=rand(g, W) if "n" in parts else None,
                dX=rand(g, B, T, W, dtype=dtype) if "x" in parts else None,
                dN=rand(g, B, T, W, dtype=dtype) if "n" in parts else None)


def flat(c):
    Y = c["Y"]
    B, T, H, d = Y.shape
    row = lambda t: None if t is None else f64(t).reshape(B * T, H * d)
    return (f64(Y).reshape(B * T, H, d), row(c["Z"]), f64(c["wo"]), row(c["R"]), f64(c["wi"]))


PARTS = ["zprnx", "zpx", "px", "zx", "pn", "rnx", "zprn", "nx"]
NORM_SHAPES = [(1, 1, 1, 8, True), (2, 3, 1, 128, True), (1, 5, 3, 128, True),
               (3, 2, 32, 128, False), (1, 67, 1, 264, True), (2, 9, 1, 2048, True),
               (1, 2, 1, 5000, True), (1, 2, 1, 16384, True), (1, 700, 16, 128, True)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("B,T,H,d,hm", NORM_SHAPES)
def test_block_norm(lib, dtype, act, parts, B, T, H, d, hm):
    c = norm_case(d + T, dtype, B, T, H, d, parts, hm)
    W = H * d
    empty = lambda: torch.empty(B, T, W, dtype=DT[dtype], device="cuda")
    X, N = empty(), empty() if "n" in parts else None
    gdn.gdn_block_norm(c["Y"], c["Z"], c["wo"], c["R"], c["wi"], X, N, scale=0.5, eps=1e-5,
                       act=act)
    y, z, wo, r, wi = flat(c)
    x, n = L.block_norm(y, z, wo, r, wi, 0.5, 1e-5, act)
    mag = np.abs(x) if r is None else np.abs(r) + np.abs(x - r)
    u = half_step(dtype)
    near(X.view(B * T, W), x, u * np.abs(x) + 64 * U32 * mag, "X")
    if n is not None:
        rms = np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        near(N.view(B * T, W), n, u * np.abs(n) + 128 * U32 * np.abs(wi) * (mag / rms + np.abs(x) / rms),
             "N")
        if r is not None:                              # the residual stream in place; X left out
            X2, N2 = c["R"].clone(), empty()
            gdn.gdn_block_norm(c["Y"], c["Z"], c["wo"], X2, c["wi"], X2, N2, scale=0.5, eps=1e-5,
                               act=act)
            assert torch.equal(X2, X) and torch.equal(N2, N)
        N2 = empty()
        gdn.gdn_block_norm(c["Y"], c["Z"], c["wo"], c["R"], c["wi"], None, N2, scale=0.5, eps=1e-5,
                           act=act)
        assert torch.equal(N2, N)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("B,T,H,d,hm", NORM_SHAPES)
def test_block_norm_backward(lib, dtype, act, parts, B, T, H, d, hm):
    c = norm_case(d + T + 1, dtype, B, T, H, d, parts, hm)
    W = H * d
    new = lambda t: None if t is None else torch.full_like(t, 77.0)
    dY = new(c["Y"])
    dZ, dR, dwo, dwi = new(c["Z"]), new(c["R"]), new(c["wo"]), new(c["wi"])
    n = gdn.gdn_block_norm_backward_workspace_bytes(c["Y"])
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    call = lambda *out: gdn.gdn_block_norm_backward(
        c["Y"], c["Z"], c["wo"], c["R"], c["wi"], c["dX"], c["dN"], *out, ws, scale=0.5, eps=1e-5,
        act=act)
    call(dY, dZ, dR, dwo, dwi)
    y, z, wo, r, wi = flat(c)
    row = lambda t: None if t is None else f64(t).reshape(B * T, W)
    gx, gn = row(c["dX"]), row(c["dN"])
    dy, dz, dr, gwo, gwi = L.block_norm_backward(y, z, wo, r, wi, gx, gn, 0.5, 1e-5, act)
    # magnitudes of the terms that the gradients are sums of
    x, _ = L.block_norm(y, z, wo, r, wi, 0.5, 1e-5, act)
    rx = np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
    mx = np.abs(x) if r is None else np.abs(r) + np.abs(x - r)
    mdx = np.zeros_like(x) if gx is None else np.abs(gx)
    if wi is not None:
        g = np.abs(gn * wi)
        mdx = mdx + g / rx + mx / rx * (g * mx).mean(-1, keepdims=True) / rx ** 2
    ry = np.sqrt((y * y).mean(-1, keepdims=True) + 1e-5) if wo is not None else np.ones(())
    yh = (np.abs(y) / ry).reshape(B * T, W)
    nn = yh * (1.0 if wo is None else np.abs(wo))
    a, da = (1.0, 0.0)
    if z is not None:
        s = 1.0 / (1.0 + np.exp(-z))
        a = np.abs(z * s) if act == "silu" else s
        da = s * (1.0 + np.abs(z) * (1.0 - s)) if act == "silu" else s * (1.0 - s)
    mdn = 0.5 * mdx * a
    u, k = half_step(dtype), 256 * U32
    if r is not None:
        near(dR.view(B * T, W), dr, u * np.abs(dr) + k * mdx, "dR")
    if z is not None:
        near(dZ.view(B * T, W), dz, u * np.abs(dz) + k * 0.5 * mdx * nn * da, "dZ")
    if wo is not None:
        near(dwo, gwo, (k + B * T * U32) * (mdn * yh).sum(0) + 1e-30, "dw_post")
        e = (mdn * np.abs(wo)).reshape(B * T, H, d)
        yy = yh.reshape(B * T, H, d)
        mdy = (e + yy * (e * yy).mean(-1, keepdims=True)) / ry
    else:
        mdy = mdn.reshape(B * T, H, d)
    near(dY.reshape(B * T, H, d), dy, u * np.abs(dy) + k * mdy, "dY")
    if wi is not None:
        near(dwi, gwi, (k + B * T * U32) * (np.abs(gn) * mx / rx).sum(0) + 1e-30, "dw_pre")
    if r is not None and gx is not None:               # dR over dX; the same order again
        keep = [t.clone() for t in (dY, dZ, dwo, dwi) if t is not None]
        c["dX"] = c["dX"].clone()
        call(dY, dZ, c["dX"], dwo, dwi)
        assert torch.equal(c["dX"], dR)
        assert all(torch.equal(a, b) for a, b in zip(keep, [t for t in (dY, dZ, dwo, dwi)
                                                            if t is not None]))


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_block_norm_gate_at_its_ends(lib, act):
    """Gates far out on both sides: one, or nothing, and slopes that vanish."""
    z = torch.tensor([-1e30, -200.0, -88.0, -60.0, 60.0, 88.0, 200.0, 1e30]).cuda()[None, None]
    y = torch.full((1, 1, 1, 8), 2.0, device="cuda")
    g, X = torch.ones_like(z), torch.empty_like(z)
    gdn.gdn_block_norm(y, z, None, None, None, X, None, act=act)
    want, _ = L.block_norm(f64(y)[0], f64(z)[0], None, None, None, act=act)
    assert np.allclose(f64(X)[0], want, rtol=1e-5, atol=1e-6)
    dY, dZ = torch.empty_like(y), torch.empty_like(z)
    gdn.gdn_block_norm_backward(y, z, None, None, None, g, None, dY, dZ, None, None, None, None,
                                act=act)
    dy, dz, *_ = L.block_norm_backward(f64(y)[0], f64(z)[0], None, None, None, f64(g)[0], None,
                                       act=act)
    assert np.allclose(f64(dY)[0, 0], dy, rtol=1e-5, atol=1e-6)
    assert np.allclose(f64(dZ)[0], dz, rtol=1e-5, atol=1e-6)
    z[...] = float("nan")
    gdn.gdn_block_norm(y, z, None, None, None, X, None, act=act)
    assert X.isnan().all()


def test_block_norm_without_rows(lib):
    Y = torch.empty(0, 4, 2, 128, device="cuda")
    w = torch.ones(256, device="cuda")
    dw = torch.full((256,), 77.0, device="cuda")
    none = torch.empty(0, 4, 256, device="cuda")
    gdn.gdn_block_norm(Y, None, w, None, None, none, None)
    gdn.gdn_block_norm_backward(Y, None, w, None, None, none, None, torch.empty_like(Y), None,
                                None, dw, None, None)
    assert (dw == 0).all()


# --------------------------------------------------------------------------- #
# together, on other streams, in graphs
# --------------------------------------------------------------------------- #
def layer(dtype, B, T, seed):
    """Inputs of one layer: a fused projection, a gate, a residual stream."""
    g = gen(seed)
    H, W = 4, 512
    c = dict(qkv=rand(g, B, T, 3 * H, 128, dtype=dtype, scale=128 ** -0.25),
             z=rand(g, B, T, W, dtype=dtype), r=rand(g, B, T, W, dtype=dtype),
             wo=rand(g, W, scale=0.1) + 1.0, wi=rand(g, W, scale=0.1) + 1.0,
             lg=torch.tensor([-0.5, -0.05, -0.01, -0.001]).cuda(),
             inv=gdn.gdn_rotary_frequencies(64)[0].cuda())
    return c, H, W


def layer_forward(c, H, W, first, S0, T0, T1):
    """Rows [T0, T1) of the layer: rotary, linear attention, gated norm and residual."""
    x = c["qkv"][:, T0:T1]
    B, T = x.shape[:2]
    q, k = (torch.empty(B, H, T, 128, dtype=x.dtype, device="cuda") for _ in range(2))
    pos = torch.arange(T0, T1, device="cuda").expand(B, T).contiguous() + first
    gdn.gdn_rotary(x[:, :, :H].transpose(1, 2), x[:, :, H:2 * H].transpose(1, 2), pos, c["inv"], q,
                   k)
    v = x[:, :, 2 * H:].transpose(1, 2).contiguous()
    O, S = torch.empty_like(v), torch.empty(B, H, 128, 128, device="cuda")
    if T == 1 and S0 is not None:
        S.copy_(S0)
        gdn.gdn_linear_decode(q, k, v, c["lg"], S, O)
    else:
        ws = torch.empty(gdn.gdn_linear_forward_workspace_bytes(k, v), dtype=torch.uint8,
                         device="cuda")
        gdn.gdn_linear_forward(q, k, v, c["lg"], S0, O, S, ws)
    X, N = (torch.empty(B, T, W, dtype=x.dtype, device="cuda") for _ in range(2))
    gdn.gdn_block_norm(O.transpose(1, 2), c["z"][:, T0:T1].contiguous(), c["wo"],
                       c["r"][:, T0:T1].contiguous(), c["wi"], X, N, scale=0.5, eps=1e-5)
    return X, N, S


def layer_oracle(c, H, W):
    x = f64(c["qkv"]).transpose(0, 2, 1, 3)
    B, _, T, _ = x.shape
    pos = np.arange(T)[None].repeat(B, 0)
    q, k = (L.rotary(a, pos, f64(c["inv"])) for a in (x[:, :H], x[:, H:2 * H]))
    o = np.stack([L.linear_forward(q[b], k[b], x[b, 2 * H:], f64(c["lg"]))[0] for b in range(B)])
    row = lambda t: f64(t).reshape(B * T, W)
    y = o.transpose(0, 2, 1, 3).reshape(B * T, H, 128)
    X, N = L.block_norm(y, row(c["z"]), f64(c["wo"]), row(c["r"]), f64(c["wi"]), 0.5, 1e-5)
    return X.reshape(B, T, W), N.reshape(B, T, W)


@pytest.mark.parametrize("dtype,tol", [("f32", 1e-5), ("bf16", 1e-2)])
def test_layer_prompt_then_tokens(lib, dtype, tol):
    """The run a serving program makes: a prompt, then token by token from its
    state, against the oracle's whole layer (relative Frobenius error, the
    suite's tolerances per type)."""
    B, T, P = 2, 135, 131
    c, H, W = layer(dtype, B, T, 21)
    X, N = layer_oracle(c, H, W)
    x, n, S = layer_forward(c, H, W, 0, None, 0, P)
    xs, ns = [x], [n]
    for t in range(P, T):
        x, n, S = layer_forward(c, H, W, 0, S, t, t + 1)
        xs.append(x)
        ns.append(n)
    for got, want in ((torch.cat(xs, 1), X), (torch.cat(ns, 1), N)):
        assert np.linalg.norm(f64(got) - want) <= tol * np.linalg.norm(want)


def test_layer_gradients_against_differences(lib):
    """The run's gradient (norm, attention, rotary backwards) against a
    central difference of the float64 oracle along a random direction."""
    B, T = 1, 150
    c, H, W = layer("f32", B, T, 22)
    g = gen(23)
    dX, dN = rand(g, B, T, W), rand(g, B, T, W)
    x = c["qkv"]
    q0, k0 = x[:, :, :H].transpose(1, 2), x[:, :, H:2 * H].transpose(1, 2)
    v = x[:, :, 2 * H:].transpose(1, 2).contiguous()
    q, k = (torch.empty(B, H, T, 128, device="cuda") for _ in range(2))
    pos = torch.arange(T, device="cuda")[None]
    gdn.gdn_rotary(q0, k0, pos, c["inv"], q, k)
    O = torch.empty_like(v)
    ws = torch.empty(max(gdn.gdn_linear_forward_workspace_bytes(k, v),
                         gdn.gdn_linear_backward_workspace_bytes(k, v)), dtype=torch.uint8,
                     device="cuda")
    gdn.gdn_linear_forward(q, k, v, c["lg"], None, O, None, ws)
    Y = O.transpose(1, 2)
    wn = torch.empty(gdn.gdn_block_norm_backward_workspace_bytes(Y), dtype=torch.uint8,
                     device="cuda")
    dO = torch.empty_like(O)
    dz, dr = torch.empty_like(c["z"]), torch.empty_like(c["r"])
    dwo, dwi = torch.empty_like(c["wo"]), torch.empty_like(c["wi"])
    gdn.gdn_block_norm_backward(Y, c["z"], c["wo"], c["r"], c["wi"], dX, dN, dO.transpose(1, 2),
                                dz, dr, dwo, dwi, wn, scale=0.5, eps=1e-5)
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    gdn.gdn_linear_backward(q, k, v, c["lg"], None, dO, None, dq, dk, dv, None, ws)
    dx = torch.empty_like(x)
    gdn.gdn_rotary(dq, dk, pos, c["inv"], dx[:, :, :H].transpose(1, 2),
                   dx[:, :, H:2 * H].transpose(1, 2), inverse=True)
    dx[:, :, 2 * H:] = dv.transpose(1, 2)
    got = dict(qkv=dx, z=dz, r=dr, wo=dwo, wi=dwi)
    gX, gN = f64(dX), f64(dN)
    h = 1e-6
    for name, grad in got.items():
        along = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        ends = []
        for s in (h, -h):
            moved = dict(c, **{name: c[name].double().cpu() + s * along})
            X, N = layer_oracle(moved, H, W)
            ends.append((X * gX).sum() + (N * gN).sum())
        slope = (ends[0] - ends[1]) / (2 * h)
        mine = float((grad.double().cpu() * along).sum())
        scale = float((grad.double().cpu() ** 2).sum() ** 0.5)
        assert abs(mine - slope) <= 1e-4 * scale, (name, mine, slope)


def test_layer_on_another_stream_and_in_a_graph(lib):
    """The same bits on a side stream, and captured and replayed on new inputs."""
    c, H, W = layer("bf16", 2, 200, 24)
    c2, _, _ = layer("bf16", 2, 200, 25)
    want, want2 = layer_forward(c, H, W, 0, None, 0, 200), layer_forward(c2, H, W, 0, None, 0, 200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer_forward(c, H, W, 0, None, 0, 200)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer_forward(c, H, W, 0, None, 0, 200)
    for x, w in ((c, want), (c2, want2)):
        for name in ("qkv", "z", "r", "wo", "wi"):
            c[name].copy_(x[name]) if x is not c else None
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_binding_checks_shapes_and_types(lib):
    c = linear_case(30, "bf16", 1, 1, 2, 64, None, False)
    O = torch.empty_like(c["V"])
    bad = [dict(Q=c["Q"][:, :, :32].contiguous()), dict(V=c["V"].float()),
           dict(lg=c["lg"].double()), dict(lg=c["lg"][:1]), dict(K=c["K"].cpu()),
           dict(V=c["V"].transpose(2, 3).contiguous().transpose(2, 3))]
    for change in bad:
        a = dict(c, **change)
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_linear_forward(a["Q"], a["K"], a["V"], a["lg"], None, O, None, None)
    with pytest.raises(ValueError):
        gdn.gdn_linear_forward(c["Q"], c["K"], c["V"], c["lg"], torch.zeros(2, 2, 128, 128).cuda(),
                               O, None, None)
    y = torch.zeros(1, 2, 1, 16, device="cuda")
    with pytest.raises(ValueError):
        gdn.gdn_block_norm(y, None, torch.ones(8).cuda(), None, None, torch.zeros(1, 2, 16).cuda(),
                           None)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_block_norm(y, None, None, None, None, None, None)


# --------------------------------------------------------------------------- #
# arguments at the alignment that the header asks for, and no more
# --------------------------------------------------------------------------- #
def shifted(t, by=16):
    """The same tensor on memory that starts ``by`` bytes past a 256-byte boundary."""
    raw = torch.full((t.nbytes + by,), 255, dtype=torch.uint8, device="cuda")
    assert raw.data_ptr() % 256 == 0
    return raw[by:].view(t.dtype).view(t.shape).copy_(t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hk,Hv,T,lens", [(1, 2, 4, 300, None), (2, 1, 1, 129, None),
                                            (1, 1, 2, 700, [128, 5, 129, 1, 400]),
                                            (1, 1, 2, 2600, None)])
def test_linear_at_16_byte_alignment(lib, dtype, B, Hk, Hv, T, lens):
    """Every tensor at 16 bytes past a multiple of 32: the bits of the aligned call."""
    c = linear_case(T + 2, dtype, B, Hk, Hv, T, lens, True)
    O, S = run_forward(c, 0.7)
    grads = run_backward(c, 0.7)
    m = {x: shifted(c[x]) for x in ("Q", "K", "V", "dO", "S0", "dS")}
    ws = [shifted(torch.full((f(c["K"], c["V"], c["cu"]),), 255, dtype=torch.uint8, device="cuda"))
          for f in (gdn.gdn_linear_forward_workspace_bytes, gdn.gdn_linear_backward_workspace_bytes)]
    O1, S1 = shifted(torch.full_like(O, 77.0)), shifted(torch.full_like(S, 77.0))
    gdn.gdn_linear_forward(m["Q"], m["K"], m["V"], c["lg"], m["S0"], O1, S1, ws[0], scale=0.7,
                           cu_seqlens=c["cu"])
    assert torch.equal(O1, O) and torch.equal(S1, S)
    out = [shifted(torch.full_like(t, 77.0)) for t in grads]
    gdn.gdn_linear_backward(m["Q"], m["K"], m["V"], c["lg"], m["S0"], m["dO"], m["dS"], *out, ws[1],
                            scale=0.7, cu_seqlens=c["cu"])
    assert all(torch.equal(a, b) for a, b in zip(out, grads))


# --------------------------------------------------------------------------- #
# gates at the types' lowest values
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_block_norm_gates_that_shut(lib, dtype, act):
    """Gates from -200 to the lowest value and minus infinity: nothing passes,
    forward or backward.  e^-200 is 1e-87; the gate is formed at -87, where both
    activations and their slopes are below 2e-36."""
    low = torch.finfo(DT[dtype]).min
    gates = [low, low / 2, -1e35, -1e30, -1e10, -200.0, -87.5, float("-inf")]
    z = torch.tensor(gates).to(DT[dtype]).cuda()[None, None]
    y = torch.full((1, 1, 1, 8), 3.0, dtype=DT[dtype], device="cuda")
    r = torch.tensor([1.0, -2.0, 0.5, 4.0, -1.0, 0.25, 8.0, 3.0]).to(DT[dtype]).cuda()[None, None]
    w = torch.full((8,), 2.0, device="cuda")
    X, N = torch.empty_like(z), torch.empty_like(z)
    gdn.gdn_block_norm(y, z, None, None, None, X, None, act=act)
    assert (X.float().abs() <= 3 * 2e-36).all(), X
    gdn.gdn_block_norm(y, z, w, r, w, X, N, act=act)
    assert torch.equal(X, r)
    g = torch.ones_like(z)
    dY, dZ, dR = torch.empty_like(y), torch.empty_like(z), torch.empty_like(z)
    gdn.gdn_block_norm_backward(y, z, None, None, None, g, None, dY, dZ, None, None, None, None,
                                act=act)
    assert (dY.float().abs() <= 2e-36).all() and (dZ.float().abs() <= 3 * 2e-36).all(), (dY, dZ)
    dw, dv = torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(gdn.gdn_block_norm_backward_workspace_bytes(y), dtype=torch.uint8, device="cuda")
    gdn.gdn_block_norm_backward(y, z, w, r, w, g, g, dY, dZ, dR, dw, dv, ws, act=act)
    # |dx| <= 1 + 2 / rms + ..: below 16 here, and n = 2
    for t, n in ((dY, 32), (dZ, 32), (dw, 16)):
        assert (t.float().abs() <= n * 2e-36).all(), t


# --------------------------------------------------------------------------- #
# decays that are not numbers
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,lens", [(1, None), (5, None), (150, None), (2600, None),
                                    (500, [3, 0, 128, 300])])
def test_linear_nan_decay_shows_in_its_head_alone(lib, dtype, T, lens):
    """A NaN log-decay: NaN wherever the recurrence has it (outputs and states;
    a last row's dK and dV meet no decay), other heads as without it."""
    c = linear_case(50, dtype, 1, 3, 3, T, lens, True)
    good = (*run_forward(c, 0.7), *run_backward(c, 0.7))
    c["lg"] = c["lg"].clone()
    c["lg"][1] = float("nan")
    got = (*run_forward(c, 0.7), *run_backward(c, 0.7))
    want = (*oracle_linear(c, 0.7), *oracle_linear_grad(c, 0.7))
    used = T if lens is None else sum(lens)
    for a, b, w in zip(got, good, want):
        rows = slice(None) if a.shape[2:] == (128, 128) and a.shape[0] == len(c["rows"]) else \
            slice(0, used)
        assert torch.equal(a[:, [0, 2]], b[:, [0, 2]])
        assert np.array_equal(np.isnan(f64(a[:, 1, rows])), np.isnan(w[:, 1, rows]))
    if T <= 5:
        O, S = torch.empty_like(c["V"]), c["S0"].clone()
        gdn.gdn_linear_decode(c["Q"], c["K"], c["V"], c["lg"], S, O, scale=0.7)
        assert O[:, 1].isnan().all() and S[:, 1].isnan().all()
        assert not O[:, [0, 2]].isnan().any() and not S[:, [0, 2]].isnan().any()


# --------------------------------------------------------------------------- #
# infinities and NaN at one row
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,lens,rows", [(6, None, (0, 3)), (200, None, (0, 63, 64, 127, 150, 199)),
                                         (2600, None, (5, 700, 1290, 2599)),
                                         (420, [100, 0, 257, 5], (99, 100, 230, 360))])
def test_linear_odd_values_reach_only_what_the_recurrence_has_them_in(lib, dtype, T, lens, rows):
    """One NaN or infinity in Q, K, V or dO: results are not finite exactly where
    the token-by-token formula's are not (a row never sees the rows on its other
    side), and the bits of the clean call elsewhere."""
    c = linear_case(60 + T, dtype, 1, 1, 1, T, lens, True)
    c["lg"] = torch.tensor([-0.01]).cuda()
    used = slice(0, T if lens is None else sum(lens))
    good = [t if t.shape[0] == len(c["rows"]) and t.shape[2:] == (128, 128) else t[:, :, used]
            for t in (*run_forward(c, 0.7), *run_backward(c, 0.7))]
    for at, name in zip(rows * 4, [x for x in ("V", "K", "Q", "dO") for _ in rows]):
        odd = dict(c, **{name: c[name].clone()})
        odd[name][0, 0, at, 37] = float("nan") if at % 2 else float("inf")
        got = (*run_forward(odd, 0.7), *run_backward(odd, 0.7))
        with np.errstate(invalid="ignore"):
            want = (*oracle_linear(odd, 0.7), *oracle_linear_grad(odd, 0.7))
        for a, b, w in zip(got, good, want):
            if a.shape != b.shape:
                a, w = a[:, :, used], w[:, :, used]
            fine = np.isfinite(w)
            assert np.array_equal(np.isfinite(f64(a)), fine), (name, at)
            assert torch.equal(a[torch.from_numpy(fine)], b[torch.from_numpy(fine)]), (name, at)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_padded_rows_may_hold_anything(lib, dtype):
    """A padded batch whose rows behind each prompt are NaN and infinity in V
    (keys zero there): the prompts' outputs have the clean batch's bits, prompts
    that are cut into segments and whole ones, and two such calls at once."""
    for B, H, T, used in ((2, 2, 300, (131, 260)), (1, 2, 2600, (1333,)), (40, 4, 260, None)):
        c = linear_case(70 + T, dtype, B, H, H, T, None, False)
        used = used or [(37 * b) % T + 1 for b in range(B)]
        for b, n in enumerate(used):
            c["K"][b, :, n:] = 0.0
        good, _ = run_forward(c, 0.7)
        for b, n in enumerate(used):
            c["V"][b, :, n:] = float("nan")
            c["V"][b, :, n + 3::5, ::3] = float("-inf")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            also, _ = run_forward(c, 0.7)
        got, _ = run_forward(c, 0.7)
        torch.cuda.synchronize()
        for b, n in enumerate(used):
            for o in (got, also):
                assert torch.equal(o[b, :, :n], good[b, :, :n]), (b, n)
                assert not o[b, :, n:].isfinite().any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hv", [2, 6])
@pytest.mark.parametrize("cu,fine", [([0, 100, 200, 420], (0, 1)), ([-8, 60, 160, 300], (1, 2)),
                                     ([0, 130, 90, 90], (0, 2)), ([0, 100, 600, 640], (0,))])
def test_linear_bad_bounds_leave_the_others(lib, dtype, Hv, cu, fine):
    """A sequence whose bounds break the rule is left out, wherever it stands:
    the others have their results, and all other rows stay as they were."""
    c = linear_case(14, dtype, 1, 2, Hv, 400, [1, 1, 1], True)
    c["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
    rows = [slice(cu[i], cu[i + 1]) for i in fine]
    O, S = run_forward(c, 0.7)
    got = run_backward(c, 0.7)
    assert gdn.gdn_get_status() == gdn.GDN_ERR_ARG
    seen = torch.zeros(400, dtype=torch.bool)
    for i, r in zip(fine, rows):
        part = {x: c[x][:, :, r].contiguous() for x in ("Q", "K", "V", "dO")}
        one = dict(c, **part, cu=torch.tensor([0, r.stop - r.start], dtype=torch.int32).cuda(),
                   S0=c["S0"][i:i + 1].contiguous(), dS=c["dS"][i:i + 1].contiguous(), rows=[0])
        for a, b in zip((O, *got[:3]), (run_forward(one, 0.7)[0], *run_backward(one, 0.7)[:3])):
            assert torch.equal(a[:, :, r], b)
        seen[r] = True
    for a in (O, *got[:3]):
        assert (a[:, :, ~seen] == 77.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hv", [148, 1])
def test_linear_slow_decay_over_many_steps(lib, dtype, Hv):
    """The state's decay over a step (a chunk of 64 or 128 rows, or a segment) is
    one number, whose rounding to a float would come back at every step: over s
    steps a mean of s 2^-26 of the state for the decays taken here, which round
    by 2^-25.4 and more.  What stays is a rounding at each of the state's updates
    (2^-24, uniform: / sqrt 3, in quadrature over steps) and the sums of 64 or
    128 products before it, counted as three more such roundings."""
    T, Hk = 16384, 1
    gd = torch.Generator(device="cuda")
    gd.manual_seed(71)
    rnd = lambda h: torch.randn(1, h, T, 128, generator=gd, device="cuda").to(DT[dtype])
    K, V = rnd(Hk), rnd(Hv)
    n = gdn.gdn_linear_forward_workspace_bytes(K, V)
    step = 64 if dtype == "f32" else 128
    if n:                                              # the length of a segment
        m = n // (Hv * 65536) + 1
        step = -(-(T // 128) // m) * 128
    assert (n > 0) == (Hv == 1)
    tries = -np.float32(1e-5) * (1 + np.arange(200, dtype=np.float32) / 128)
    lam = np.exp(tries.astype(np.float64) * step)
    off = np.abs(lam.astype(np.float32).astype(np.float64) / lam - 1)
    lg = torch.full((Hv,), float(tries[off.argmax()]), device="cuda")
    assert off.max() >= 2.0 ** -25.4
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    O, S = torch.empty_like(V), torch.empty(1, Hv, 128, 128, device="cuda")
    gdn.gdn_linear_forward(K, K, V, lg, None, O, S, ws, scale=128 ** -0.5)
    w = torch.exp(lg[0].double() * torch.arange(T - 1, -1, -1, device="cuda"))
    steps = T // min(step, 64 if dtype == "f32" else 128)
    tol = 4 * (steps / 3) ** 0.5 * U32
    for h in {0, Hv // 2, Hv - 1}:
        want = (V[0, h].double() * w[:, None]).T @ K[0, 0].double()
        err = float((S[0, h].double() - want).norm() / want.norm())
        assert err <= tol, (h, err, tol)


# --------------------------------------------------------------------------- #
# waits that run out
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("T,lens,kernel,block,backward", [
    (200, None, "outputs", 1, False), (1100, [900, 150, 50], "outputs", 0, False),
    (2600, None, "outputs", 3, False), (2600, None, "states", 2, False),
    (300, None, "outputs", 4, True), (2600, None, "states", 2, True),
])
def test_linear_expired_wait_reports_and_the_next_call_is_clean(lib, T, lens, kernel, block,
                                                                backward):
    """A tile that never comes: all of the block's roles give up within the
    bound, the status word says so, and the next call has the bits of one before."""
    c = linear_case(80, "bf16", 1, 2, 2, T, lens, True)
    run = (lambda: run_backward(c, 0.7)) if backward else (lambda: run_forward(c, 0.7))
    want = run()
    assert gdn.gdn_get_status() == gdn.GDN_OK
    gdn.gdn_debug_arm_linear_expiry(block, kernel, 5.0)
    run()
    assert gdn.gdn_get_status() == gdn.GDN_ERR_TIMEOUT
    assert "ran out" in gdn.gdn_last_error()
    got = run()
    assert gdn.gdn_get_status() == gdn.GDN_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# --------------------------------------------------------------------------- #
# outputs beside inputs in one buffer
# --------------------------------------------------------------------------- #
def test_views_of_one_buffer_that_share_no_memory(lib):
    """Layouts that interleave outputs and inputs in one allocation are taken, and
    overlapping views of the same buffers are refused with nothing written."""
    g = gen(90)
    B, T, H = 2, 37, 3
    inv = gdn.gdn_rotary_frequencies(64)[0].cuda()
    pos = torch.arange(T).expand(B, T).contiguous().cuda()
    x = rand(g, B, T, 4 * H, 128, dtype="bf16")        # q, k and room for both
    view = lambda i: x[:, :, i * H:(i + 1) * H].transpose(1, 2)
    want = [torch.empty(B, H, T, 128, dtype=x.dtype, device="cuda") for _ in range(2)]
    gdn.gdn_rotary(view(0), view(1), pos, inv, *want)
    gdn.gdn_rotary(view(0), view(1), pos, inv, view(2), view(3))
    assert torch.equal(view(2), want[0]) and torch.equal(view(3), want[1])
    y = torch.empty(B, H, 2 * T, 128, dtype=x.dtype, device="cuda")
    y[:, :, ::2] = view(0)                             # rows between the output's
    gdn.gdn_rotary(y[:, :, ::2], None, pos, inv, y[:, :, 1::2], None)
    assert torch.equal(y[:, :, 1::2], want[0])
    gdn.gdn_rotary(view(0), view(1), pos, inv, view(0), view(1))
    assert torch.equal(view(0), want[0]) and torch.equal(view(1), want[1])
    keep = x.clone()
    for qo, ko in ((x[:, :, 1:1 + H].transpose(1, 2), view(3)), (view(2), x[:, :, 5:8].transpose(1, 2)),
                   (view(2), view(1)[:, :, 1:])):
        q, k, p = (t[:, :, :ko.shape[2]] for t in (view(0), view(1), pos[:, None]))
        with pytest.raises(gdn.GdnError, match="shares memory"):
            gdn.gdn_rotary(q, k, p[:, 0].contiguous(), inv, qo[:, :, :ko.shape[2]], ko)
    assert torch.equal(x, keep)
    # a norm's output in the other half of its input's rows, then half a row too early
    buf = rand(g, 8, 2, 1, 256)
    X = torch.empty(8, 1, 256, device="cuda")
    w = rand(g, 256)
    gdn.gdn_block_norm(buf[:, :1], None, w, None, None, X, None)
    r = rand(g, 16, 1, 256)
    for out in (r[1:9], r[:8].view(-1)[128:-128].view(7, 1, 256)):
        n = out.shape[0]
        with pytest.raises(gdn.GdnError, match="shares memory"):
            gdn.gdn_block_norm(buf[:n, :1], None, w, r[:n], None, out, None)


# --------------------------------------------------------------------------- #
# errors in the 2-norm, where the bounds by element are wide
# --------------------------------------------------------------------------- #
# A bf16 output passes two independent roundings, its own and that of its terms
# (weights or state).  One spreads evenly over half a step, which is at most 2^-8
# of a value: 2^-8 / sqrt 3 in the 2-norm, two of them 0.0032.  A quarter more
# for the sampling.  A float32 output is a sum of at most 128 + 128 + 64 products
# in order: sqrt(320 / 3), about ten half steps in quadrature; 16 are allowed.
TOL2 = {"bf16": 1.25 * (2 / 3) ** 0.5 * UBF, "f32": 16 * U32}


def near2(got, want, dtype, rows, name):
    """By head and by 128 rows of a sequence, so that one lost boundary or one
    wrong tile shows however long the call is."""
    got = f64(got)
    for b, a, n in rows:
        for t in range(a, a + n, 128):
            x, w = (v[b, :, t:min(t + 128, a + n)] for v in (got, want))
            err = np.sqrt(((x - w) ** 2).sum((1, 2))) / np.sqrt((w ** 2).sum((1, 2)))
            assert (err <= TOL2[dtype]).all(), (name, b, t, err)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hk,Hv,T,lens", SHAPES + [(1, 3, 3, 6400, None), (50, 3, 3, 390, None),
                                                     (1, 3, 6, 3400, [3000, 260, 140])])
def test_linear_relative_error(lib, dtype, B, Hk, Hv, T, lens):
    c = linear_case(95 + T, dtype, B, Hk, Hv, T, lens, True)
    if Hk == 3:                                        # what a row adds is seen to the end
        c["lg"] = torch.tensor([-1e-3, -1e-5, 0.0, -1e-4, -1e-2, -2e-3][:Hv]).cuda()
    O, _ = run_forward(c, 0.7)
    near2(O, oracle_linear(c, 0.7)[0], dtype, c["rows"], "O")
    for x, y, name in zip(run_backward(c, 0.7), oracle_linear_grad(c, 0.7)[:3], ("dQ", "dK", "dV")):
        near2(x, y, dtype, c["rows"], name)


# --------------------------------------------------------------------------- #
# offsets past 32 bits
# --------------------------------------------------------------------------- #
def test_offsets_past_32_bits(lib):
    """More than 2^31 elements a tensor: the last rows and heads, and the last
    states of a pool, are those of a small call on them."""
    gd = torch.Generator(device="cuda")
    gd.manual_seed(97)
    rnd = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=gd, device="cuda", dtype=dt)
    # rotary and a norm: 17 million rows of 128
    T = (1 << 24) + 37
    x = rnd(1, 1, T, 128)
    pos = torch.arange(T, device="cuda")[None]
    inv = gdn.gdn_rotary_frequencies(128)[0].cuda()
    y, z = torch.empty_like(x), torch.empty(1, 1, 100, 128, dtype=x.dtype, device="cuda")
    gdn.gdn_rotary(x, None, pos, inv, y, None)
    gdn.gdn_rotary(x[:, :, -100:], None, pos[:, -100:].contiguous(), inv, z, None)
    assert torch.equal(y[:, :, -100:], z)
    w = rnd(128, dt=torch.float32)
    rows = lambda t: t[0, 0][None, :, None]            # [1, T, 1, 128]
    gdn.gdn_block_norm(rows(x), None, w, None, None, y[0], None)
    gdn.gdn_block_norm(rows(x[:, :, -100:]), None, w, None, None, z[0], None)
    assert torch.equal(y[0, :, -100:], z[0])
    del x, y
    # linear attention: 40 heads of 430000 rows
    H, T = 40, 430000
    K, V = rnd(1, 1, T, 128), rnd(1, H, T, 128)
    lg = torch.full((H,), -0.01, device="cuda")
    run = lambda v, o, g: gdn.gdn_linear_forward(
        K, K, v, g, None, o, None, torch.empty(gdn.gdn_linear_forward_workspace_bytes(K, v),
                                               dtype=torch.uint8, device="cuda"), scale=128 ** -0.5)
    O, last = torch.empty_like(V), torch.empty_like(V[:, :1])
    run(V, O, lg)
    run(V[:, -1:].contiguous(), last, lg[-1:])
    a, b = O[0, -1, -4096:].double(), last[0, 0, -4096:].double()
    assert (a - b).norm() <= 2 ** 0.5 * TOL2["bf16"] * b.norm()
    del V, O
    # a pool of 70000 states
    S = torch.zeros(70000, 1, 128, 128, device="cuda")
    q = rnd(2, 1, 1, 128, dt=torch.float32)
    S[[3, 69999]] = rnd(1, 128, 128, dt=torch.float32)
    o = torch.empty_like(q)
    at = torch.tensor([69999, 3], dtype=torch.int32, device="cuda")
    gdn.gdn_linear_decode(q[[0, 0]].contiguous(), q[[1, 1]].contiguous(), q[[0, 0]].contiguous(),
                          lg[:1], S, o, at)
    assert torch.equal(o[0], o[1]) and torch.equal(S[3], S[69999])
    assert int((S != 0).any(-1).any(-1).sum()) == 2


# --------------------------------------------------------------------------- #
# positions as far as binary64 has them
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_far_positions(lib, dtype, inter):
    """Angles of positions up to 2^53 against their exact remainders (60 digits):
    the errors of near positions, no more."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    tau = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    where = [0, 1, 12345, 10 ** 6, 2 ** 31 + 1, 10 ** 12, 2 ** 40 + 12345, 2 ** 52 + 1, 2 ** 53 - 1,
             -(10 ** 12), -7]
    T, half = len(where), 8
    g = gen(98)
    x = rand(g, 1, 1, T, 128, dtype=dtype)
    inv = torch.tensor([1.0, 0.75, 0.1, 3e-2, 1e-3, 1e-4, 3.3e-6, 1e-7])
    y = torch.empty_like(x)
    gdn.gdn_rotary(x, None, torch.tensor([where]).cuda(), inv.cuda(), y, None, interleaved=inter)
    left = np.array([[float(Decimal(p) * Decimal(float(f)) % tau) for f in inv] for p in where])
    want = f64(x)[0, 0].copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        c, s, xa, xb = np.cos(left[:, i]), np.sin(left[:, i]), f64(x)[0, 0, :, a], f64(x)[0, 0, :, b]
        want[:, a], want[:, b] = xa * c - xb * s, xa * s + xb * c
    near(y[0, 0], want, rotary_tol(f64(x)[0, 0], f64(inv), 1.0, inter, dtype), "far")


@pytest.mark.parametrize("how", ["one call", "calls of 8", "prompts of 8"])
def test_linear_slow_decay_over_many_tokens(lib, how):
    """16384 tokens one after the other: as over steps, one rounding per token to
    the state in quadrature, where a decay rounded to a float is off by the same
    2^-25.4 at each (1e-4 of the state in all)."""
    T, n = 16384, 16384 if how == "one call" else 8
    tries = -np.float32(1e-5) * (1 + np.arange(200, dtype=np.float32) / 128)
    lam = np.exp(tries.astype(np.float64))
    off = np.abs(lam.astype(np.float32).astype(np.float64) / lam - 1)
    assert off.max() >= 2.0 ** -25.4
    lg = torch.tensor([float(tries[off.argmax()])]).cuda()
    g = gen(99)
    dtype = "bf16" if how == "prompts of 8" else "f32"
    K, V = rand(g, 1, 1, T, 128, dtype=dtype), rand(g, 1, 1, T, 128, dtype=dtype)
    S, S2 = torch.zeros(1, 1, 128, 128, device="cuda"), torch.empty(1, 1, 128, 128, device="cuda")
    O = torch.empty_like(V[:, :, :n])
    for t in range(0, T, n):
        k, v = K[:, :, t:t + n], V[:, :, t:t + n]
        if how == "prompts of 8":
            gdn.gdn_linear_forward(k, k, v, lg, S, O, S2, None)
            S, S2 = S2, S
        else:
            gdn.gdn_linear_decode(k, k, v, lg, S, O)
    w = torch.exp(lg[0].double() * torch.arange(T - 1, -1, -1, device="cuda"))
    want = (V[0, 0].double() * w[:, None]).T @ K[0, 0].double()
    err = float((S[0, 0].double() - want).norm() / want.norm())
    assert err <= 2 * (T / 3) ** 0.5 * U32, err


# --------------------------------------------------------------------------- #
# gradients and tokens in a graph
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_and_tokens_captured_and_replayed(lib, dtype):
    """Linear backward of shared heads, packed and cut, a norm's gradients and a
    token step in one graph: on other inputs, and on inputs that hold NaN and
    infinities, the bits of the calls themselves."""
    def case(seed, odd=False):
        c = linear_case(seed, dtype, 1, 2, 4, 2900, [2600, 0, 5, 250], True)
        n = norm_case(seed, dtype, 2, 33, 4, 128, "zprnx")
        n["pool"], n["token"] = rand(gen(seed), 4, 4, 128, 128), rand(gen(seed), 2, 4, 1, 128, dtype=dtype)
        if odd:
            c["V"][0, 0, 700, 3], c["Q"][0, 1, 1900, 5] = float("nan"), float("inf")
            n["Z"][0, 3, 9] = torch.finfo(DT[dtype]).min
        return c, n

    def run(c, n):
        Y = n["Y"]
        new = lambda t: torch.full_like(t, 77.0)
        dY, dZ, dR, dwo, dwi = new(Y), new(n["Z"]), new(n["R"]), new(n["wo"]), new(n["wi"])
        ws = torch.empty(gdn.gdn_block_norm_backward_workspace_bytes(Y), dtype=torch.uint8,
                         device="cuda")
        gdn.gdn_block_norm_backward(Y, n["Z"], n["wo"], n["R"], n["wi"], n["dX"], n["dN"], dY, dZ, dR,
                                    dwo, dwi, ws)
        S, O = n["pool"].clone(), new(n["token"])
        gdn.gdn_linear_decode(n["token"], n["token"], n["token"], c["lg"], S, O, slots)
        return (*run_backward(c, 0.7), dY, dZ, dR, dwo, dwi, S, O)

    slots = torch.tensor([3, 1], dtype=torch.int32).cuda()
    sets = [case(110), case(111), case(112, odd=True)]
    want = [run(*s) for s in sets]
    c, n = case(110)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(c, n)
    for (c2, n2), w in zip(sets, want):
        for mine, other in ((c, c2), (n, n2)):
            for x in mine:
                if isinstance(mine[x], torch.Tensor):
                    mine[x].copy_(other[x])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, w):
            a, b = a.contiguous(), b.contiguous()
            assert torch.equal(a.isnan(), b.isnan())
            assert torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


# --------------------------------------------------------------------------- #
# behind the gated delta rule
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_block_norm_behind_the_gated_delta_rule(lib, dtype):
    """The head norm, gate and residual on what gdn_forward and gdn_decode leave,
    head-major as it lies: the oracle's values on the same outputs, the bits of a
    token-major copy."""
    from gated_deltanet_chunk_02_b200.inputs import Workload, make_decode_inputs, make_inputs
    H, T = 3, 128
    d = {k: v.cuda() for k, v in make_inputs(Workload(B=2, H=H, T=T, k=64, dtype=dtype), seed=5,
                                             with_q=True).items()}
    O = torch.empty_like(d["V"])
    Sf = torch.empty(2, H, 128, 128, device="cuda")
    ws = torch.empty(gdn.gdn_forward_workspace_bytes(d["K"], 64), dtype=torch.uint8, device="cuda")
    gdn.gdn_forward(d["Q"], d["K"], d["V"], d["beta"], d["g"], None, 3, 1, 8, 0, O, Sf, ws)
    t = {k: v.cuda() for k, v in make_decode_inputs(2, H, H, 1, dtype=dtype, seed=6).items()}
    o = torch.empty_like(t["V"])
    gdn.gdn_decode(t["Q"], t["K"], t["V"], t["beta"], t["loggate"], Sf, o)
    g = gen(120)
    wo, wi = rand(g, H * 128), rand(g, H * 128)
    for Y in (O.transpose(1, 2), o.transpose(1, 2)):
        B, n = Y.shape[:2]
        z, r = (rand(g, B, n, H * 128, dtype=dtype) for _ in range(2))
        out = []
        for y in (Y, Y.contiguous()):
            X, N = torch.empty_like(z), torch.empty_like(z)
            gdn.gdn_block_norm(y, z, wo, r, wi, X, N, scale=0.5, eps=1e-5)
            out.append((X, N))
        assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
        row = lambda a: f64(a).reshape(B * n, H * 128)
        x, want = L.block_norm(f64(Y).reshape(B * n, H, 128), row(z), f64(wo), row(r), f64(wi), 0.5,
                               1e-5)
        u, mag = half_step(dtype), np.abs(row(r)) + np.abs(x - row(r))
        rms = np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        near(X.view(B * n, -1), x, u * np.abs(x) + 64 * U32 * mag, "X")
        near(N.view(B * n, -1), want,
             u * np.abs(want) + 128 * U32 * np.abs(f64(wi)) * (mag / rms + np.abs(x) / rms), "N")
