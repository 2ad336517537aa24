"""What the layer's projections and its draft step are measured on.

Two operators, in the shapes a server of the gated delta-rule layer calls them with:

* ``linear``: out = act(x w^T + bias) + residual, the projections around the layer.
* ``draft`` / ``layer``: one step of speculative decoding. Each sequence first commits the
  accepted tokens of its previous draft to its recurrent state, then runs its new drafted tokens
  from there without advancing the state; what a later commit needs of them goes to a record.
  ``draft`` takes q, k, v and gates, ``layer`` the raw projections (causal convolution, SiLU, L2
  norm and gates in front, optional output gate behind).

A pass updates the state, the convolution state and the record in place, as a serving loop does.
"""
import math

import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_B = {"f32": 4, "bf16": 2, "f16": 2}
_EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def _lin(m, n, k, dtype="bf16", out="bf16", bias=False, act="none", res="none", pad=0, name=None):
    c = dict(op="linear", m=m, n=n, k=k, dtype=dtype, out=out, bias=bias, act=act, res=res,
             pad=pad)
    if name:
        c["name"] = name
    return c


def _draft(op, seqs, depth, lens, hk, hv, dk, dv, dtype, out, tiled=False, mixed=False,
           gate=False, name=None):
    c = dict(op=op, seqs=seqs, depth=depth, lens=lens, hk=hk, hv=hv, dk=dk, dv=dv, dtype=dtype,
             out=out, tiled=tiled, mixed=mixed, gate=gate)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the beta / alpha projection of one decode token: almost nothing but latency
        _lin(1, 64, 2048, out="f32", name="linear gates 1 token"),
        # the output projection of one decode token, added to the residual stream
        _lin(1, 2048, 4096, res="bf16", name="linear out 1 token"),
        # the q|k|v|z projection of a 64-sequence decode step: the weights' bytes
        _lin(64, 12288, 2048, name="linear in 64 tokens"),
        # an odd ragged batch with everything in the epilogue, x a column slice of a wider array
        _lin(333, 5003, 1160, dtype="f16", out="f16", bias=True, act="gelu", res="f32", pad=24,
             name="linear odd epilogue"),
        # the q|k|v projection of a 4096-token prompt
        _lin(4096, 8192, 2048, name="linear in 4096 tokens"),
        # the output projection of a chunk of 16384 prompt tokens
        _lin(16384, 2048, 4096, res="bf16", name="linear out 16384 tokens"),
        # one sequence that drafts 4 tokens: latency
        _draft("draft", 1, 4, "full", 16, 32, 128, 128, "f16", "bf16", name="draft 1 x 4"),
        # the 64-sequence decode batch, 4 drafted tokens each: the state's bytes
        _draft("draft", 64, 4, "full", 16, 32, 128, 128, "f16", "bf16", name="draft 64 x 4"),
        # the longest drafts, ragged, some sequences only committing, exact types, tiled heads
        _draft("draft", 64, 16, "ragged", 16, 32, 128, 128, "f32", "f32", tiled=True,
               name="draft 64 x 0..16"),
        # many sequences of a smaller layer with few heads, unequal head sizes
        _draft("draft", 96, 6, "ragged", 3, 12, 64, 32, "bf16", "f32", name="draft small heads"),
        # a small batch through the whole layer with its output gate
        _draft("layer", 8, 3, "full", 16, 32, 128, 128, "bf16", "bf16", gate=True,
               name="layer draft 8 x 3 gated"),
        # a large ragged batch through the whole layer, fused gate projection
        _draft("layer", 128, 8, "ragged", 16, 32, 128, 128, "bf16", "bf16", mixed=True,
               name="layer draft 128 x 0..8"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        while True:
            m = _log_int(rng, 1, 16384)
            n = _log_int(rng, 16, 12288)
            k = 8 * _log_int(rng, 8, 1024)
            if m * n * k <= 16384 * 2048 * 4096:
                break
        dtype = rng.choice(["bf16", "bf16", "f16"])
        return _lin(m, n, k, dtype=dtype, out=rng.choice([dtype, dtype, "f32"]),
                    bias=rng.random() < 0.4, act=rng.choice(["none", "none", "silu", "gelu",
                                                             "sigmoid"]),
                    res=rng.choice(["none", dtype, "f32"]), pad=8 * rng.randint(0, 4))
    while True:
        op = rng.choice(["draft", "draft", "layer"])
        seqs = _log_int(rng, 1, 128)
        depth = rng.randint(1, 16)
        hk = _log_int(rng, 1, 16)
        hv = hk * rng.choice([1, 2, 2, 4])
        dk = rng.choice([32, 64, 128, 128])
        dv = rng.choice([32, 64, 128, 128])
        if seqs * hv * dk * dv * (depth + 8) <= 128 * 32 * 128 * 128 * 16:
            break
    dtype = rng.choice(["f32", "bf16", "f16"] if op == "draft" else ["bf16", "bf16", "f32"])
    return _draft(op, seqs, depth, rng.choice(["full", "ragged"]), hk, hv, dk, dv, dtype,
                  rng.choice(["bf16", "f32"]), tiled=rng.random() < 0.3,
                  mixed=op == "layer" and rng.random() < 0.4,
                  gate=op == "layer" and rng.random() < 0.4)


def _lengths(c):
    """New tokens of each sequence (the previous draft had as many) and how many of the previous
    draft's tokens were accepted."""
    d = c["depth"]
    lens = [d if c["lens"] == "full" else (5 * i + d) % (d + 1) for i in range(c["seqs"])]
    return lens, [(3 * i + 1) % (lens[i] + 1) for i in range(c["seqs"])]


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        t = _T[c["dtype"]]
        wide = rn(m, k + c["pad"]).to(t)
        return dict(case=c, x=wide[:, c["pad"]:], w=(rn(n, k) * k ** -0.5).to(t),
                    bias=rn(n) * 0.5 if c["bias"] else None,
                    residual=None if c["res"] == "none" else rn(m, n).to(_T[c["res"]]),
                    out=torch.empty((m, n), dtype=_T[c["out"]], device="cuda"))
    B, D, hk, hv, dk, dv = (c[s] for s in ("seqs", "depth", "hk", "hv", "dk", "dv"))
    lens, acc = _lengths(c)
    ns = B + 2
    T = sum(lens)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    slots = torch.randperm(ns, generator=g, device="cuda")[:B].to(torch.int32)
    unit = lambda v: v / v.square().sum(-1, keepdim=True).add(_EPS).sqrt()  # noqa: E731
    slow = lambda *s: torch.exp(rn(*s) * 1.5 - 2.0)  # noqa: E731  decay rates, slow and fast
    n0 = torch.zeros(ns, dtype=torch.int32, device="cuda")
    n0[slots.long()] = i32(lens)
    # the key head of each value head
    heads = torch.arange(hv, device="cuda")
    heads = heads % hk if c["tiled"] else heads // (hv // hk)
    s = dict(case=c, lens=lens, heads=heads, cu=i32(cu), slots=slots, accepted=i32(acc),
             state=rn(ns, hv, dk, dv) * 0.05,
             rec_n=n0, rec_e=torch.exp(-slow(ns, hv, D)),
             rec_k=unit(rn(ns, hk, D, dk)), rec_u=rn(ns, hv, D, dv) * 0.5,
             o=torch.zeros((T, hv, dv), dtype=_T[c["out"]], device="cuda"))
    t = _T[c["dtype"]]
    if c["op"] == "draft":
        s.update(q=(unit(rn(T, hk, dk)) * dk ** -0.5).to(t), k=unit(rn(T, hk, dk)).to(t),
                 v=rn(T, hv, dv).to(t), g=-slow(T, hv), beta=torch.sigmoid(rn(T, hv)))
        return s
    C = 2 * hk * dk + hv * dv
    r = hv // hk
    s.update(x=rn(T, C).to(t), conv_w=rn(C, 4) * 0.5, conv_state=rn(ns, 3, C).to(t),
             rec_x=rn(ns, D, C).to(t), A_log=torch.log(torch.rand(hv, generator=g, device="cuda")
                                                       * 0.9 + 0.1),
             dt_bias=rn(hv), a=rn(T, hk, 2 * r) if c["mixed"] else rn(T, hv),
             b=None if c["mixed"] else rn(T, hv))
    if c["gate"]:
        s.update(z=rn(T, hv, dv).to(torch.bfloat16), norm_w=1.0 + 0.1 * rn(dv))
    return s


# --------------------------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "draft": _own_draft, "layer": _own_layer}[op](state)
    return {"linear": _plain_linear, "draft": _plain_draft, "layer": _plain_layer}[op](state)


def _own_linear(s):
    import gated_deltanet_linear_19_b200 as gdn
    return gdn.linear(s["x"], s["w"], bias=s["bias"], act=s["case"]["act"],
                      residual=s["residual"], out=s["out"])


def _own_dims(s, gdn):
    c = s["case"]
    layout = (gdn.GDN_GQA_TILED if c["tiled"] else 0) | (gdn.GDN_GATES_MIXED_BA if c["mixed"]
                                                         else 0)
    return gdn.Dims(s["state"].shape[0], c["hk"], c["hv"], c["dk"], c["dv"], 4, layout)


def _own_draft(s):
    import gated_deltanet_linear_19_b200 as gdn
    rec = gdn.DraftRecord(s["rec_n"], s["rec_e"], s["rec_k"], s["rec_u"])
    gdn.draft_step(_own_dims(s, gdn), s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"],
                   s["slots"], s["cu"], s["accepted"], rec, s["o"])
    return _outputs(s, s["o"])


def _own_layer(s):
    import gated_deltanet_linear_19_b200 as gdn
    rec = gdn.DraftRecord(s["rec_n"], s["rec_e"], s["rec_k"], s["rec_u"], s["rec_x"])
    gate = gdn.OutGate(s["z"], s["norm_w"], _EPS) if s["case"]["gate"] else None
    gdn.layer_draft(_own_dims(s, gdn), s["x"], s["conv_w"], s["conv_state"], s["cu"], s["slots"],
                    s["accepted"], s["a"], s["b"], s["A_log"], s["dt_bias"], s["state"], rec,
                    s["o"], eps=_EPS, gate=gate)
    return _outputs(s, s["o"])


def _outputs(s, o):
    keys = ("state", "rec_n", "rec_e", "rec_k", "rec_u") + (("conv_state", "rec_x")
                                                            if s["case"]["op"] == "layer" else ())
    return dict({k: s[k] for k in keys}, o=o)


# ------------------------------------------------------------------------------- plain forms
def _plain_linear(s):
    c = s["case"]
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif c["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * 0.5 ** 0.5))
    elif c["act"] == "sigmoid":
        y = 1.0 / (1.0 + torch.exp(-y))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(_T[c["out"]])


def _places(s):
    """[seqs, depth] packed row of every drafted token, and which of them exist."""
    D = s["case"]["depth"]
    j = torch.arange(D, device="cuda")
    cu = s["cu"].long()
    there = j[None] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None] + j[None], 0), there


def _plain_core(s, q, k, v, g, beta):
    """Commit and draft on padded [seqs, depth, ...] fp32 tensors."""
    new_k, q, k = k, q[:, :, s["heads"]], k[:, :, s["heads"]]
    c, slots = s["case"], s["slots"].long()
    D = c["depth"]
    at, there = _places(s)
    j = torch.arange(D, device="cuda")
    # commit: every accepted token's outer product, decayed by the accepted tokens after it
    took = j[None] < s["accepted"].long()[:, None]                       # [B, D]
    e = torch.where(took[:, None], s["rec_e"][slots], 1.0)               # [B, hv, D]
    suffix = torch.flip(torch.cumprod(torch.flip(e, (2,)), 2), (2,))     # prod of e_l, l >= j
    after = torch.cat([suffix[:, :, 1:], torch.ones_like(suffix[:, :, :1])], 2)
    ru = torch.where(took[:, None, :, None], s["rec_u"][slots], 0.0) * after[..., None]
    S = s["state"][slots] * suffix[:, :, 0, None, None] + \
        s["rec_k"][slots][:, s["heads"]].transpose(2, 3) @ ru
    s["state"][slots] = S
    # draft: the token recurrence on a copy of the state that is dropped
    en = torch.where(there[..., None], torch.exp(g), 1.0)
    bn = torch.where(there[..., None], beta, 0.0)
    o, us = [], []
    for t in range(D):
        S = S * en[:, t, :, None, None]
        u = bn[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(2))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        o.append((S * q[:, t, :, :, None]).sum(2))
        us.append(u)
    o, u = torch.stack(o, 1), torch.stack(us, 1)                         # [B, D, hv, dv]
    # the record's rows of this draft; rows behind its last token stay as they were
    put = lambda name, new, m: s[name].index_put_((slots,), torch.where(m, new, s[name][slots]))  # noqa: E731,E501
    put("rec_e", torch.exp(g).transpose(1, 2), there[:, None])
    put("rec_k", new_k.transpose(1, 2), there[:, None, :, None])
    put("rec_u", u.transpose(1, 2), there[:, None, :, None])
    s["rec_n"][slots] = s["cu"][1:] - s["cu"][:-1]
    return o[there]                                                      # packed [T, hv, dv]


def _plain_draft(s):
    at, _ = _places(s)
    f = lambda t: t.float()[at]  # noqa: E731
    o = _plain_core(s, f(s["q"]), f(s["k"]), f(s["v"]), f(s["g"]), f(s["beta"]))
    return _outputs(s, o.to(_T[s["case"]["out"]]))


def _plain_layer(s):
    c, slots = s["case"], s["slots"].long()
    hk, hv, dk, dv, D, B = c["hk"], c["hv"], c["dk"], c["dv"], c["depth"], c["seqs"]
    at, there = _places(s)
    # the convolution's window after the accepted tokens, then the new tokens
    old = torch.cat([s["conv_state"][slots], s["rec_x"][slots]], 1)
    pick = s["accepted"].long()[:, None] + torch.arange(3, device="cuda")[None]
    rows = torch.gather(old, 1, pick[:, :, None].expand(B, 3, old.shape[2]))
    s["conv_state"][slots] = rows
    x = s["x"][at]                                                       # [B, D, C]
    s["rec_x"][slots] = torch.where(there[..., None], x, s["rec_x"][slots])
    ext = torch.cat([rows, x], 1).float()
    y = sum(ext[:, j:j + D] * s["conv_w"][:, j] for j in range(4))
    y = y / (1.0 + torch.exp(-y))
    unit = lambda t: t / torch.sqrt(t.square().sum(-1, keepdim=True) + _EPS)  # noqa: E731
    q = unit(y[..., :hk * dk].reshape(B, D, hk, dk)) * dk ** -0.5
    k = unit(y[..., hk * dk:2 * hk * dk].reshape(B, D, hk, dk))
    v = y[..., 2 * hk * dk:].reshape(B, D, hv, dv)
    a, b = s["a"], s["b"]
    if c["mixed"]:
        r = hv // hk
        a, b = a[..., r:].reshape(-1, hv), a[..., :r].reshape(-1, hv)
    zz = a + s["dt_bias"]
    g = -torch.exp(s["A_log"]) * (torch.clamp(zz, min=0) + torch.log1p(torch.exp(-zz.abs())))
    beta = 1.0 / (1.0 + torch.exp(-b))
    o = _plain_core(s, q, k, v, g[at], beta[at])
    if c["gate"]:
        z = s["z"].float()
        o = o / torch.sqrt(o.square().mean(-1, keepdim=True) + _EPS) * s["norm_w"] * \
            (z / (1.0 + torch.exp(-z)))
    return _outputs(s, o.to(_T[c["out"]]))


# -------------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        b = (m * k + n * k) * _B[c["dtype"]] + m * n * _B[c["out"]]
        b += n * 4 if c["bias"] else 0
        b += m * n * _B[c["res"]] if c["res"] != "none" else 0
        return {"bytes": b, "flops": 2.0 * m * n * k}
    lens, acc = _lengths(c)
    hk, hv, dk, dv = c["hk"], c["hv"], c["dk"], c["dv"]
    S = hv * dk * dv
    row = 4 * (hk * dk + hv * dv + hv)  # a record's token: k, u, e
    b = flops = 0.0
    for t, a in zip(lens, acc):
        b += (4 * S if t or a else 0) + (4 * S if a else 0) + row * (t + a)
        flops += 2.0 * S * (2 * t + a)
    T = sum(lens)
    es = _B[c["dtype"]]
    C = 2 * hk * dk + hv * dv
    b += T * hv * dv * _B[c["out"]] + T * (C * es + 8 * hv)
    if c["op"] == "layer":
        # the window in and out, the recorded inputs out, those that enter the window in
        b += sum(C * es * ((6 if a else 3) + t + min(a, 3)) for t, a in zip(lens, acc))
        b += 16 * C + (T * hv * dv * 2 if c["gate"] else 0)
    return {"bytes": b, "flops": flops}


# ------------------------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "linear":
        y = torch.matmul(s["x"].double(), s["w"].double().T)
        if c["bias"]:
            y += s["bias"].double()
        if c["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif c["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif c["act"] == "sigmoid":
            y = torch.sigmoid(y)
        return y if s["residual"] is None else y + s["residual"].double()
    hk, hv, dk, dv = c["hk"], c["hv"], c["dk"], c["dv"]
    lens, acc = _lengths(c)
    slots = s["slots"].tolist()
    heads = s["heads"]
    out = {k: s[k].double() for k in ("state", "rec_e", "rec_k", "rec_u")}
    out["rec_n"] = s["rec_n"].clone()
    o = torch.zeros((sum(lens), hv, dv), dtype=torch.float64, device="cuda")
    if c["op"] == "layer":
        out["conv_state"], out["rec_x"] = s["conv_state"].double(), s["rec_x"].double()
    t0 = 0
    for n, slot in enumerate(slots):
        S = out["state"][slot]
        for j in range(acc[n]):  # the accepted tokens, one after another
            S = out["rec_e"][slot, :, j, None, None] * S + \
                torch.einsum("hd,hc->hdc", out["rec_k"][slot, heads, j],
                             out["rec_u"][slot, :, j])
        out["state"][slot] = S
        T, span = lens[n], slice(t0, t0 + lens[n])
        if c["op"] == "layer":
            X = s["x"][span].double()
            win = torch.cat([out["conv_state"][slot], out["rec_x"][slot][:acc[n]]])[-3:]
            out["conv_state"][slot] = win
            out["rec_x"][slot][:T] = X
            seen = torch.cat([win, X])
            w = s["conv_w"].double()
            u = torch.stack([(seen[i:i + 4] * w.T).sum(0) for i in range(T)]) if T else X
            u = u * torch.sigmoid(u)
            q, k, v = u.split([hk * dk, hk * dk, hv * dv], 1)
            q, k, v = q.view(T, hk, dk), k.view(T, hk, dk), v.view(T, hv, dv)
            q = q * (q.pow(2).sum(-1, keepdim=True) + _EPS).rsqrt() / math.sqrt(dk)
            k = k * (k.pow(2).sum(-1, keepdim=True) + _EPS).rsqrt()
            a = s["a"][span].double()
            if c["mixed"]:
                b, a = a.split([hv // hk, hv // hk], 2)
                a, b = a.reshape(T, hv), b.reshape(T, hv)
            else:
                b = s["b"][span].double()
            g = -s["A_log"].double().exp() * torch.logaddexp(a + s["dt_bias"].double(),
                                                             torch.zeros_like(a))
            beta = torch.sigmoid(b)
        else:
            q, k, v, g, beta = (s[m][span].double() for m in ("q", "k", "v", "g", "beta"))
        for i in range(T):  # the drafted tokens, by the definition
            ki, qi = k[i][heads], q[i][heads]
            S = g[i].exp()[:, None, None] * S
            u = beta[i][:, None] * (v[i] - torch.einsum("hdc,hd->hc", S, ki))
            S = S + torch.einsum("hd,hc->hdc", ki, u)
            o[t0 + i] = torch.einsum("hdc,hd->hc", S, qi)
            out["rec_e"][slot, :, i], out["rec_k"][slot, :, i] = g[i].exp(), k[i]
            out["rec_u"][slot, :, i] = u
        out["rec_n"][slot] = T
        t0 += T
    if c["gate"]:
        z = s["z"].double()
        o = o * (o.pow(2).mean(-1, keepdim=True) + _EPS).rsqrt() * s["norm_w"].double() * z * \
            torch.sigmoid(z)
    return dict(out, o=o)
