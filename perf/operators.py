"""The layer operators around the chunk-wise kernels, as they are measured.

Cases of six calls that a linear-attention layer is made of: rotary positions
on queries and keys, linear attention with one decay per head (whole prompts,
packed prompts, their gradients, single tokens on a pool of states) and the
norms before and after a block with its gate and residual scale (and their
gradients).  ``run`` computes a case in its plain form, or, where ``own`` is
true, through the library's entry points.  Layouts are the library's: head
dimension 128, head-major ``[B, H, T, d]``, states ``[B, H, d_v, d_k]`` float32.
"""
import math

import torch

own = False

D = 128              # head dimension
CHUNK = 128          # chunk of the plain linear attention
EPS = 1e-6


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def listed():
    return [
        # a whole prompt of the long-context configuration, every head, long-context frequencies
        dict(name="rotary_prompt", op="rotary", dtype="bf16", B=1, Hq=16, Hk=16, T=65536, rot=128,
             layout="half", scaling="yarn", inverse=False, first=0),
        # one token of each request of a serving batch, far into its sequence, half the head
        dict(name="rotary_tokens", op="rotary", dtype="f32", B=64, Hq=32, Hk=16, T=1, rot=64,
             layout="interleaved", scaling="none", inverse=False, first=30000),
        # the long-context prompt: one sequence, few heads
        dict(name="linear_long", op="linear", dtype="bf16", B=1, Hk=16, Hv=16, T=65536, lens="",
             carried=False, decay="slow"),
        # prompts of different lengths packed behind one another, shared query and key heads,
        # states carried in; rows behind the last sequence
        dict(name="linear_packed", op="linear", dtype="bf16", B=1, Hk=16, Hv=32, T=8192,
             lens="1,700,0,2049,64,333,4096,17,900", carried=True, decay="spread"),
        # a training step's batch
        dict(name="linear_train", op="linear_grad", dtype="bf16", B=4, Hk=16, Hv=16, T=4096,
             lens="", carried=False, decay="spread"),
        # a short step in float32: odd lengths, shared heads, states carried in
        dict(name="linear_train_f32", op="linear_grad", dtype="f32", B=1, Hk=4, Hv=8, T=1000,
             lens="333,1,500,129", carried=True, decay="spread"),
        # a serving batch's next token, states in a pool
        dict(name="linear_tokens", op="linear_tokens", dtype="bf16", B=64, Hk=16, Hv=32, n=1,
             spare=8),
        # one request, a few drafted tokens at once
        dict(name="linear_draft", op="linear_tokens", dtype="f32", B=1, Hk=8, Hv=16, n=4, spare=0),
        # between two blocks of a training batch: post norm, gate, residual, next block's norm
        dict(name="norm_layer", op="norm", dtype="bf16", B=4, T=4096, H=1, d=2048, act="silu",
             post=True, gate=True, residual=True, pre=True),
        # the gated norm of each head behind a serving batch's token step
        dict(name="norm_heads", op="norm", dtype="bf16", B=64, T=1, H=32, d=128, act="silu",
             post=True, gate=True, residual=False, pre=False),
        dict(name="norm_layer_grad", op="norm_grad", dtype="bf16", B=4, T=4096, H=1, d=2048,
             act="silu", post=True, gate=True, residual=True, pre=True),
        # gradients of a head-wise norm in float32, odd length, gate by a logistic function
        dict(name="norm_heads_grad", op="norm_grad", dtype="f32", B=2, T=999, H=16, d=128,
             act="sigmoid", post=True, gate=True, residual=True, pre=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _lens(rng, total):
    """Lengths of packed sequences (zero and one among them) within ``total`` rows."""
    out, left = [], total
    for _ in range(rng.randint(1, 12)):
        n = rng.choice([0, 1, _log_int(rng, 1, max(1, total)), _log_int(rng, 1, max(1, total))])
        n = min(n, left)
        out.append(n)
        left -= n
    return ",".join(str(n) for n in out)


def draw(rng):
    op = rng.choice(["rotary", "linear", "linear", "linear_grad", "linear_grad", "linear_tokens",
                     "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rotary":
        Hk = rng.choice([1, 2, 3, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4])
        rows = (1 << 21 if dtype == "bf16" else 1 << 20) // (Hq + Hk)
        B = _log_int(rng, 1, 64)
        return dict(op=op, dtype=dtype, B=B, Hq=Hq, Hk=Hk, T=_log_int(rng, 1, max(1, rows // B)),
                    rot=rng.choice([128, 64, 32, 2 * rng.randint(1, 64)]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    inverse=rng.random() < 0.4, first=rng.choice([0, rng.randint(1, 1000000)]))
    if op in ("linear", "linear_grad"):
        Hk = rng.choice([1, 2, 4, 5, 16])
        Hv = Hk * rng.choice([1, 1, 2, 3])
        rows = (1 << 20 if op == "linear" else 1 << 18) >> (0 if dtype == "bf16" else 4)
        tokens = _log_int(rng, 1, max(1, min(65536, rows // Hv)))
        c = dict(op=op, dtype=dtype, Hk=Hk, Hv=Hv, carried=rng.random() < 0.5,
                 decay=rng.choice(["slow", "spread", "fast"]))
        if rng.random() < 0.5:
            return dict(c, B=1, T=tokens, lens=_lens(rng, tokens))
        B = rng.choice([1, 1, 2, 3, 4, 7])
        return dict(c, B=B, T=max(1, tokens // B), lens="")
    if op == "linear_tokens":
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hv = Hk * rng.choice([1, 2, 4])
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, max(1, 2048 // Hv)), Hk=Hk, Hv=Hv,
                    n=rng.choice([1, 1, 1, 2, 3, 5, 8]), spare=rng.choice([0, 1, 5]))
    if rng.random() < 0.5:
        H, d = _log_int(rng, 1, 64), D
    else:
        H, d = 1, 8 * _log_int(rng, 1, 1024)
    rows = _log_int(rng, 1, max(1, (1 << (25 if dtype == "bf16" else 24)) // (H * d)))
    rows = min(rows, 16384)
    B = rng.choice([1, 2, 3])
    c = dict(op=op, dtype=dtype, B=B, T=max(1, rows // B), H=H, d=d,
             act=rng.choice(["silu", "sigmoid"]), post=rng.random() < 0.8, gate=rng.random() < 0.7,
             residual=rng.random() < 0.7, pre=rng.random() < 0.7)
    if not (c["post"] or c["gate"] or c["pre"]):
        c["post"] = True
    return c


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case):
    return [int(x) for x in case["lens"].split(",")] if case["lens"] else []


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _frequencies(rot, scaling, base=10000.0, factor=8.0, original=8192):
    """Frequencies of the rotated pairs (float32) and the factor on cos and sin."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    m = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        turns = original * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
        m = 0.1 * math.log(factor) + 1.0
    return f.to(torch.float32), m


def _decays(case, gen, dev):
    """One log-decay per value head: shortest memory about 1.5, 20 or 30 tokens,
    longest about 100, 1000 or 30000, spread evenly in their logarithm."""
    H = case["Hv"]
    lo, hi = {"fast": (1.5, 100.0), "spread": (20.0, 1000.0), "slow": (30.0, 30000.0)}[case["decay"]]
    x = (torch.arange(H, dtype=torch.float64, device=dev) +
         torch.rand(H, generator=gen, device=dev, dtype=torch.float64)) / H
    memory = torch.exp(math.log(lo) + x * (math.log(hi) - math.log(lo)))
    return (-1.0 / memory).to(torch.float32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape, scale=1.0, dtype=None):
        x = torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)
        return x.mul_(scale).to(dtype or dt)

    st = {"case": dict(case)}
    op = case["op"]
    if op == "rotary":
        B, T = case["B"], case["T"]
        inv, m = _frequencies(case["rot"], case["scaling"])
        first = torch.zeros(B, 1, dtype=torch.int64, device=dev)
        if case["first"]:
            first = torch.randint(0, case["first"] + 1, (B, 1), generator=gen, device=dev)
        st.update(Q=normal(B, case["Hq"], T, D), K=normal(B, case["Hk"], T, D),
                  pos=first + torch.arange(T, device=dev), inv=inv.to(dev), m=m)
        st.update(Qo=torch.empty_like(st["Q"]), Ko=torch.empty_like(st["K"]))
    elif op in ("linear", "linear_grad"):
        B, T, Hk, Hv = case["B"], case["T"], case["Hk"], case["Hv"]
        lens = _lengths(case)
        nseq = len(lens) if lens else B
        st.update(Q=normal(B, Hk, T, D, scale=D ** -0.5), K=normal(B, Hk, T, D, scale=D ** -0.5),
                  V=normal(B, Hv, T, D), lg=_decays(case, gen, dev), cu=None, S0=None, lens=lens,
                  scale=1.0)
        if lens:
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        if case["carried"]:
            st["S0"] = normal(nseq, Hv, D, D, scale=0.5, dtype=torch.float32)
        if op == "linear":
            st.update(O=torch.zeros_like(st["V"]),
                      S=torch.empty(nseq, Hv, D, D, device=dev))
        else:
            st.update(dO=normal(B, Hv, T, D), dS=None, dQ=torch.zeros_like(st["Q"]),
                      dK=torch.zeros_like(st["K"]), dV=torch.zeros_like(st["V"]), dS0=None)
            if case["carried"]:
                st["dS"] = normal(nseq, Hv, D, D, scale=0.5, dtype=torch.float32)
                st["dS0"] = torch.empty(nseq, Hv, D, D, device=dev)
        if own:
            from gated_deltanet_chunk_02_b200 import gdn
            need = (gdn.gdn_linear_forward_workspace_bytes if op == "linear"
                    else gdn.gdn_linear_backward_workspace_bytes)
            st["ws"] = torch.empty(need(st["K"], st["V"], st["cu"]), dtype=torch.uint8, device=dev)
    elif op == "linear_tokens":
        B, n, Hk, Hv = case["B"], case["n"], case["Hk"], case["Hv"]
        slots = B + case["spare"]
        st.update(Q=normal(B, Hk, n, D, scale=D ** -0.5), K=normal(B, Hk, n, D, scale=D ** -0.5),
                  V=normal(B, Hv, n, D), lg=_decays(dict(case, decay="spread"), gen, dev),
                  S=normal(slots, Hv, D, D, scale=0.5, dtype=torch.float32),
                  slots=torch.randperm(slots, generator=gen, device=dev)[:B].to(torch.int32),
                  scale=1.0)
        st["O"] = torch.empty_like(st["V"])
    else:
        B, T, H, d = case["B"], case["T"], case["H"], case["d"]
        W = H * d
        st.update(Y=normal(B, H, T, d), Z=None, wo=None, R=None, wi=None, s=0.5)
        if case["gate"]:
            st["Z"] = normal(B, T, W)
        if case["post"]:
            st["wo"] = normal(W, scale=0.1, dtype=torch.float32).add_(1.0)
        if case["residual"]:
            st["R"] = normal(B, T, W, scale=2.0)
        if case["pre"]:
            st["wi"] = normal(W, scale=0.1, dtype=torch.float32).add_(1.0)
        empty = lambda: torch.empty(B, T, W, dtype=dt, device=dev)
        if op == "norm":
            st.update(X=empty(), N=empty() if case["pre"] else None)
        else:
            st.update(dX=normal(B, T, W), dN=normal(B, T, W) if case["pre"] else None,
                      dY=torch.empty_like(st["Y"]), dZ=empty() if case["gate"] else None,
                      dR=empty() if case["residual"] else None,
                      dwo=torch.empty(W, device=dev) if case["post"] else None,
                      dwi=torch.empty(W, device=dev) if case["pre"] else None)
            if own:
                from gated_deltanet_chunk_02_b200 import gdn
                st["ws"] = torch.empty(gdn.gdn_block_norm_backward_workspace_bytes(
                    st["Y"].transpose(1, 2)), dtype=torch.uint8, device=dev)
    return st


# --------------------------------------------------------------------------- #
# plain forms, in float32
# --------------------------------------------------------------------------- #
def _rotate(x, pos, inv, m, layout, inverse):
    rot = 2 * inv.numel()
    ang = pos.to(torch.float64)[:, None, :, None] * inv.to(torch.float64)
    c, s = (torch.cos(ang) * m).float(), (torch.sin(ang) * m).float()
    if inverse:
        s = -s
    y = x.float()
    r = y[..., :rot]
    if layout == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _powers(lg, n):
    """exp(lg * n) for the log-decays [H] and a vector of counts, float32 [H, len]."""
    return torch.exp(lg.double()[:, None] * n.double()[None, :]).float()


def _chunks(x, C):
    """[B, H, T, d] -> [B, H, nc, C, d] float32, zeros behind the last row."""
    B, H, T, d = x.shape
    nc = (T + C - 1) // C
    x = x.float()
    if nc * C != T:
        x = torch.cat([x, x.new_zeros(B, H, nc * C - T, d)], 2)
    return x.view(B, H, nc, C, d)


def _heads(x, Hv):
    return x if x.shape[1] == Hv else x.repeat_interleave(Hv // x.shape[1], 1)


def _start_states(k, v, w_end, a_chunk, S0):
    """States before each chunk and after the last: [B, H, nc + 1, d, d]."""
    U = torch.matmul((v * w_end[..., None]).transpose(-1, -2), k)
    B, H, nc = U.shape[:3]
    S = U.new_empty(B, H, nc + 1, D, D)
    S[:, :, 0] = 0.0 if S0 is None else S0
    for c in range(nc):
        S[:, :, c + 1] = a_chunk[:, c, None, None] * S[:, :, c] + U[:, :, c]
    return S


def _chunk_decays(lg, T, C, dev):
    nc = (T + C - 1) // C
    i = torch.arange(C, device=dev)
    n = torch.full((nc,), C, device=dev)
    n[-1] = T - (nc - 1) * C
    left = (n[:, None] - 1 - i[None, :]).clamp(min=0)
    w_end = _powers(lg, left.flatten()).view(-1, nc, C)          # to the chunk's end
    a_chunk = _powers(lg, n)                                     # across the chunk
    w_in = _powers(lg, i + 1)[:, None, :]                        # from its start
    m = _powers(lg, (i[:, None] - i[None, :]).clamp(min=0).flatten()).view(-1, 1, C, C)
    m = m * (i[:, None] >= i[None, :])
    return w_end, a_chunk, w_in, m


def _linear(q, k, v, lg, S0, scale):
    B, Hv, T, _ = v.shape
    w_end, a_chunk, w_in, m = _chunk_decays(lg, T, CHUNK, v.device)
    qc, kc, vc = (_chunks(_heads(x, Hv), CHUNK) for x in (q, k, v))
    S = _start_states(kc, vc, w_end, a_chunk, S0)
    o = torch.matmul(qc, S[:, :, :-1].transpose(-1, -2)) * w_in[..., None]
    o += torch.matmul(torch.matmul(qc, kc.transpose(-1, -2)) * m, vc)
    o = (o * scale).view(B, Hv, -1, D)[:, :, :T]
    return o.to(v.dtype), S[:, :, -1]


def _linear_grad(q, k, v, lg, S0, dO, dSf, scale):
    B, Hv, T, _ = v.shape
    Hk = k.shape[1]
    w_end, a_chunk, w_in, m = _chunk_decays(lg, T, CHUNK, v.device)
    qc, kc, vc, gc = (_chunks(_heads(x, Hv), CHUNK) for x in (q, k, v, dO))
    gc = gc * scale
    S = _start_states(kc, vc, w_end, a_chunk, S0)
    nc = qc.shape[2]
    G = torch.matmul((gc * w_in[..., None]).transpose(-1, -2), qc)
    E = torch.empty_like(S)                          # gradient of the state at each boundary
    E[:, :, nc] = 0.0 if dSf is None else dSf
    for c in range(nc - 1, -1, -1):
        E[:, :, c] = a_chunk[:, c, None, None] * E[:, :, c + 1] + G[:, :, c]
    p = torch.matmul(qc, kc.transpose(-1, -2)) * m
    dp = torch.matmul(gc, vc.transpose(-1, -2)) * m
    dq = torch.matmul(dp, kc) + torch.matmul(gc, S[:, :, :-1]) * w_in[..., None]
    dk = torch.matmul(dp.transpose(-1, -2), qc) + torch.matmul(vc, E[:, :, 1:]) * w_end[..., None]
    dv = torch.matmul(p.transpose(-1, -2), gc) + \
        torch.matmul(kc, E[:, :, 1:].transpose(-1, -2)) * w_end[..., None]

    def rows(x, H):
        x = x.view(B, Hv, -1, D)[:, :, :T]
        return x if H == Hv else x.view(B, H, Hv // H, T, D).sum(2)

    return rows(dq, Hk).to(q.dtype), rows(dk, Hk).to(k.dtype), rows(dv, Hv).to(v.dtype), E[:, :, 0]


def _sequences(st):
    """(first row, length, index) of each packed sequence that has rows."""
    at, out = 0, []
    for i, n in enumerate(st["lens"]):
        if n:
            out.append((at, n, i))
        at += n
    return out


def _run_linear(st):
    O, S = st["O"], st["S"]
    if not st["lens"]:
        o, s = _linear(st["Q"], st["K"], st["V"], st["lg"], st["S0"], st["scale"])
        O.copy_(o)
        S.copy_(s)
        return O, S
    S.zero_() if st["S0"] is None else S.copy_(st["S0"])
    for a, n, i in _sequences(st):
        part = [st[x][:, :, a:a + n] for x in ("Q", "K", "V")]
        o, s = _linear(*part, st["lg"], None if st["S0"] is None else st["S0"][i:i + 1],
                       st["scale"])
        O[:, :, a:a + n] = o
        S[i] = s[0]
    return O, S


def _run_linear_grad(st):
    outs = [st["dQ"], st["dK"], st["dV"]]
    if not st["lens"]:
        *g, e = _linear_grad(st["Q"], st["K"], st["V"], st["lg"], st["S0"], st["dO"], st["dS"],
                             st["scale"])
        for o, x in zip(outs, g):
            o.copy_(x)
        if st["dS0"] is not None:
            st["dS0"].copy_(e)
            outs.append(st["dS0"])
        return tuple(outs)
    if st["dS0"] is not None:
        st["dS0"].copy_(st["dS"])
    for a, n, i in _sequences(st):
        q, k, v, g = (st[x][:, :, a:a + n] for x in ("Q", "K", "V", "dO"))
        one = [None if st[x] is None else st[x][i:i + 1] for x in ("S0", "dS")]
        *gr, e = _linear_grad(q, k, v, st["lg"], one[0], g, one[1], st["scale"])
        for o, x in zip(outs, gr):
            o[:, :, a:a + n] = x
        if st["dS0"] is not None:
            st["dS0"][i] = e[0]
    return tuple(outs) if st["dS0"] is None else (*outs, st["dS0"])


def _run_linear_tokens(st):
    Hv = st["V"].shape[1]
    q, k = (_heads(st[x].float(), Hv) for x in ("Q", "K"))
    v = st["V"].float()
    at = st["slots"].long()
    S = st["S"][at]
    a = torch.exp(st["lg"])[None, :, None, None]
    for t in range(v.shape[2]):
        S = a * S + v[:, :, t, :, None] * k[:, :, t, None, :]
        st["O"][:, :, t] = (torch.matmul(S, q[:, :, t, :, None])[..., 0] * st["scale"])
    st["S"][at] = S
    return st["O"], st["S"]


def _norm_parts(st, wide):
    """The block norm's intermediates in the wide type."""
    c = st["case"]
    B, T, H, d = c["B"], c["T"], c["H"], c["d"]
    y = st["Y"].to(wide).transpose(1, 2)                          # [B, T, H, d]
    ry = 1.0 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) if c["post"] else None
    yh = y * ry if c["post"] else y
    n = yh.reshape(B, T, H * d)
    if c["post"]:
        n = n * st["wo"].to(wide)
    act = dact = None
    u = n
    if c["gate"]:
        z = st["Z"].to(wide)
        sg = 1.0 / (1.0 + torch.exp(-z))
        act = z * sg if c["act"] == "silu" else sg
        dact = sg * (1.0 + z * (1.0 - sg)) if c["act"] == "silu" else sg * (1.0 - sg)
        u = n * act
    x = u * st["s"]
    if c["residual"]:
        x = x + st["R"].to(wide)
    rx = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) if c["pre"] else None
    return ry, yh, n, act, dact, x, rx


def _norm(st, wide):
    *_, x, rx = _norm_parts(st, wide)
    return x, None if rx is None else x * rx * st["wi"].to(wide)


def _norm_grad(st, wide):
    c = st["case"]
    B, T, H, d = c["B"], c["T"], c["H"], c["d"]
    ry, yh, n, act, dact, x, rx = _norm_parts(st, wide)
    dx = st["dX"].to(wide)
    dwi = dwo = dz = None
    if c["pre"]:
        xh, dn = x * rx, st["dN"].to(wide)
        dwi = (dn * xh).sum((0, 1))
        g = dn * st["wi"].to(wide)
        dx = dx + rx * (g - xh * (g * xh).mean(-1, keepdim=True))
    dn = dx * st["s"]
    if c["gate"]:
        dz = dn * n * dact
        dn = dn * act
    if c["post"]:
        dwo = (dn * yh.reshape(B, T, H * d)).sum((0, 1))
        g = (dn * st["wo"].to(wide)).view(B, T, H, d)
        dy = ry * (g - yh * (g * yh).mean(-1, keepdim=True))
    else:
        dy = dn.view(B, T, H, d)
    return dy.transpose(1, 2), dz, dx if c["residual"] else None, dwo, dwi


def _plain(st):
    op = st["case"]["op"]
    if op == "rotary":
        c = st["case"]
        args = (st["pos"], st["inv"], st["m"], c["layout"], c["inverse"])
        return _rotate(st["Q"], *args), _rotate(st["K"], *args)
    if op == "linear":
        return _run_linear(st)
    if op == "linear_grad":
        return _run_linear_grad(st)
    if op == "linear_tokens":
        return _run_linear_tokens(st)
    dt = st["Y"].dtype
    if op == "norm":
        return tuple(x.to(dt) for x in _norm(st, torch.float32) if x is not None)
    dy, dz, dr, dwo, dwi = _norm_grad(st, torch.float32)
    return tuple(x for x in (dy.to(dt), None if dz is None else dz.to(dt),
                             None if dr is None else dr.to(dt), dwo, dwi) if x is not None)


# --------------------------------------------------------------------------- #
# the library's calls
# --------------------------------------------------------------------------- #
def _own(st):
    from gated_deltanet_chunk_02_b200 import gdn
    c = st["case"]
    op = c["op"]
    if op == "rotary":
        gdn.gdn_rotary(st["Q"], st["K"], st["pos"], st["inv"], st["Qo"], st["Ko"], mscale=st["m"],
                       interleaved=c["layout"] == "interleaved", inverse=c["inverse"])
        return st["Qo"], st["Ko"]
    if op == "linear":
        gdn.gdn_linear_forward(st["Q"], st["K"], st["V"], st["lg"], st["S0"], st["O"], st["S"],
                               st["ws"], scale=st["scale"], cu_seqlens=st["cu"])
        return st["O"], st["S"]
    if op == "linear_grad":
        gdn.gdn_linear_backward(st["Q"], st["K"], st["V"], st["lg"], st["S0"], st["dO"], st["dS"],
                                st["dQ"], st["dK"], st["dV"], st["dS0"], st["ws"],
                                scale=st["scale"], cu_seqlens=st["cu"])
        return tuple(st[x] for x in ("dQ", "dK", "dV", "dS0") if st[x] is not None)
    if op == "linear_tokens":
        gdn.gdn_linear_decode(st["Q"], st["K"], st["V"], st["lg"], st["S"], st["O"],
                              slots=st["slots"], scale=st["scale"])
        return st["O"], st["S"]
    Y = st["Y"].transpose(1, 2)
    if op == "norm":
        gdn.gdn_block_norm(Y, st["Z"], st["wo"], st["R"], st["wi"], st["X"], st["N"],
                           scale=st["s"], eps=EPS, act=c["act"])
        return tuple(x for x in (st["X"], st["N"]) if x is not None)
    gdn.gdn_block_norm_backward(Y, st["Z"], st["wo"], st["R"], st["wi"], st["dX"], st["dN"],
                                st["dY"].transpose(1, 2), st["dZ"], st["dR"], st["dwo"],
                                st["dwi"], st["ws"], scale=st["s"], eps=EPS, act=c["act"])
    return tuple(st[x] for x in ("dY", "dZ", "dR", "dwo", "dwi") if st[x] is not None)


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------- #
# what a pass cannot do without
# --------------------------------------------------------------------------- #
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "rotary":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * n * D * e + 8 * case["B"] * case["T"], "flops": 3 * n * case["rot"]}
    if op in ("linear", "linear_grad"):
        lens = _lengths(case)
        tokens = sum(lens) if lens else case["B"] * case["T"]
        nseq = len(lens) if lens else case["B"]
        q, v = tokens * case["Hk"] * D * e, tokens * case["Hv"] * D * e
        state = nseq * case["Hv"] * D * D * 4
        if op == "linear":
            return {"bytes": 2 * q + 2 * v + state * (2 if case["carried"] else 1),
                    "flops": 4 * tokens * case["Hv"] * D * D}
        return {"bytes": 4 * q + 3 * v + (3 * state if case["carried"] else 0),
                "flops": 10 * tokens * case["Hv"] * D * D}
    if op == "linear_tokens":
        rows = case["B"] * case["n"]
        return {"bytes": 2 * case["B"] * case["Hv"] * D * D * 4 +
                2 * rows * (case["Hk"] + case["Hv"]) * D * e,
                "flops": 5 * rows * case["Hv"] * D * D}
    n = case["B"] * case["T"] * case["H"] * case["d"]
    g, r, p = case["gate"], case["residual"], case["pre"]
    if op == "norm":
        return {"bytes": n * e * (2 + g + r + p), "flops": 12 * n}
    return {"bytes": n * e * (3 + 2 * g + 2 * r + p), "flops": 30 * n}


# --------------------------------------------------------------------------- #
# the definitions in 64 bits
# --------------------------------------------------------------------------- #
def _decayed_products(a, b, c, lg, reverse):
    """sum_j lambda^|i-j| (a_i . b_j) c_j over j <= i (j >= i if reverse), one
    sequence [H, n, d], blocks of rows against all the columns they meet."""
    H, n, _ = a.shape
    out = torch.empty_like(c)
    step = max(16, min(n, (1 << 26) // max(1, n)))
    for h in range(H):
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            j0, j1 = (i0, n) if reverse else (0, i1)
            dist = (torch.arange(i0, i1, device=a.device)[:, None] -
                    torch.arange(j0, j1, device=a.device)[None, :])
            if reverse:
                dist = -dist
            w = torch.where(dist >= 0, torch.exp(lg[h] * dist.clamp(min=0).double()), 0.0)
            out[h, i0:i1] = (w * (a[h, i0:i1] @ b[h, j0:j1].T)) @ c[h, j0:j1]
    return out


def _exact_linear(st, grad):
    Hk, Hv = st["K"].shape[1], st["V"].shape[1]
    B, T = st["V"].shape[0], st["V"].shape[2]
    lg = st["lg"].double()
    seqs = [(0, a, n, i) for a, n, i in _sequences(st)] if st["lens"] else \
        [(b, 0, T, b) for b in range(B)]
    zeros = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    state = lambda x: None if x is None else x.double()
    S0 = state(st["S0"])
    if grad:
        dSf = state(st["dS"])
        dQ, dK, dV = (torch.zeros(B, Hv, T, D, dtype=torch.float64, device=lg.device)
                      for _ in range(3))
        dS0 = None if dSf is None else dSf.clone()
    else:
        O = zeros(st["V"])
        S = zeros(st["S"]) if S0 is None else S0.clone()
    for b, a, n, i in seqs:
        q, k, v = (_heads(st[x][b:b + 1, :, a:a + n].double(), Hv)[0] for x in ("Q", "K", "V"))
        t = torch.arange(n, device=lg.device).double()
        w_in = torch.exp(lg[:, None] * (t + 1))[..., None]
        w_end = torch.exp(lg[:, None] * (n - 1 - t))[..., None]
        a_n = torch.exp(lg * n)[:, None, None]
        if not grad:
            o = _decayed_products(q, k, v, lg, False)
            s = (v * w_end).transpose(1, 2) @ k
            if S0 is not None:
                o += w_in * (q @ S0[i].transpose(1, 2))
                s += a_n * S0[i]
            O[b, :, a:a + n] = o * st["scale"]
            S[i] = s
            continue
        g = st["dO"][b, :, a:a + n].double() * st["scale"]
        dq = _decayed_products(g, v, k, lg, False)
        dk = _decayed_products(v, g, q, lg, True)
        dv = _decayed_products(k, q, g, lg, True)
        e = (g * w_in).transpose(1, 2) @ q
        if S0 is not None:
            dq += w_in * (g @ S0[i])
        if dSf is not None:
            dk += w_end * (v @ dSf[i])
            dv += w_end * (k @ dSf[i].transpose(1, 2))
            dS0[i] = e + a_n * dSf[i]
        for full, part in ((dQ, dq), (dK, dk), (dV, dv)):
            full[b, :, a:a + n] = part
    if not grad:
        return O, S
    share = lambda x: x if Hk == Hv else x.view(B, Hk, Hv // Hk, T, D).sum(2)
    out = (share(dQ), share(dK), dV)
    return out if dS0 is None else (*out, dS0)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        half = case["rot"] // 2
        ang = st["pos"].double()[:, None, :, None] * st["inv"].double()
        c, s = st["m"] * torch.cos(ang), st["m"] * torch.sin(ang)
        s = -s if case["inverse"] else s
        outs = []
        for x in (st["Q"], st["K"]):
            y = x.double()
            first = slice(0, half) if case["layout"] == "half" else slice(0, 2 * half, 2)
            second = slice(half, 2 * half) if case["layout"] == "half" else slice(1, 2 * half, 2)
            a, b = y[..., first].clone(), y[..., second].clone()
            y[..., first] = a * c - b * s
            y[..., second] = b * c + a * s
            outs.append(y)
        return tuple(outs)
    if op in ("linear", "linear_grad"):
        return _exact_linear(st, op == "linear_grad")
    if op == "linear_tokens":
        B, Hv, n, _ = st["V"].shape
        q, k = (_heads(st[x].double(), Hv) for x in ("Q", "K"))
        v, lg = st["V"].double(), st["lg"].double()
        S = st["S"].double()
        at = st["slots"].long()
        start = S[at]
        O = torch.empty_like(v)
        for t in range(n):
            o = torch.exp(lg * (t + 1))[None, :, None] * torch.einsum("bhvk,bhk->bhv", start,
                                                                      q[:, :, t])
            for j in range(t + 1):
                dot = (q[:, :, t] * k[:, :, j]).sum(-1, keepdim=True)
                o += torch.exp(lg * (t - j))[None, :, None] * dot * v[:, :, j]
            O[:, :, t] = o * st["scale"]
        w = torch.exp(lg[:, None] * (n - 1 - torch.arange(n, device=lg.device)))[None, :, :, None]
        S[at] = torch.exp(lg * n)[None, :, None, None] * start + \
            torch.einsum("bhnv,bhnk->bhvk", v * w, k)
        return O, S
    return _exact_norm(st, op == "norm_grad")


def _exact_norm(st, grad):
    """By automatic differentiation of the definition in 64 bits."""
    c = st["case"]
    B, T, H, d = c["B"], c["T"], c["H"], c["d"]
    leaf = {x: None if st[x] is None else st[x].double().requires_grad_(grad)
            for x in ("Y", "Z", "wo", "R", "wi")}
    with torch.set_grad_enabled(grad):
        n = leaf["Y"].permute(0, 2, 1, 3)
        if c["post"]:
            n = n / (n.square().mean(3, keepdim=True) + EPS).sqrt()
        n = n.reshape(B, T, H * d)
        if c["post"]:
            n = leaf["wo"] * n
        if c["gate"]:
            gate = torch.sigmoid(leaf["Z"])
            n = n * (gate * leaf["Z"] if c["act"] == "silu" else gate)
        x = st["s"] * n
        if c["residual"]:
            x = leaf["R"] + x
        h = None
        if c["pre"]:
            h = leaf["wi"] * x / (x.square().mean(2, keepdim=True) + EPS).sqrt()
        if not grad:
            return tuple(t for t in (x, h) if t is not None)
        loss = (x * st["dX"].double()).sum()
        if h is not None:
            loss = loss + (h * st["dN"].double()).sum()
        loss.backward()
    return tuple(leaf[x].grad for x in ("Y", "Z", "R", "wo", "wi") if leaf[x] is not None)
