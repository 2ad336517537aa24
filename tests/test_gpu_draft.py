"""The draft step with rollback (gdn_draft_step, gdn_layer_draft) against the token recurrence in
64 bits: commit of the accepted tokens, outputs and records of the drafted ones, the convolution
window, and everything a skipped or absent sequence must leave alone.

Tolerances. The kernels compute in fp32: a value is a sum of at most d_k + 2 T products of earlier
values, each rounded to half a step (2^-24 relative), through at most T + 1 dependent tokens, so an
element is off by at most gamma = (T + 2) (d_k + 2 T + 16) 2^-24 times the same recurrence run on
absolute values (`bound`). An output in bf16 adds half its step, 2^-8 of the value. Errors of
random sign stay far below that bound, so the relative L2 error is held to 1e-5 as well (fp32).
The sums over d_k take each factor in two parts of 11 bits and leave out the product of both second
parts: a product is off by less than 2^-21 + 2^-22 + 2^-21 < 2^-19 of itself, 32 of gamma's steps,
and the matrix unit truncates its running sum d_k / 8 times, at most 2 steps each. gamma allows
(T + 2) (d_k + 16) steps for each dependent pass, more than the d_k / 4 + 32 that these take.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_19_b200 as gdn
from gated_deltanet_linear_19_b200 import Dims, OutGate, device_status
from gated_deltanet_linear_19_b200.layer import GDNLayer

pytestmark = pytest.mark.gpu

EPS = 1e-6


def head_map(d):
    h = np.arange(d.H_v)
    return h % d.H_k if d.layout & gdn.GDN_GQA_TILED else h // (d.H_v // d.H_k)


def f64(t):
    return t.detach().double().cpu().numpy()


class Model:
    """The operator on the host in 64 bits: state, record and window of every slot, and beside
    them the same numbers run on absolute values (the bound on rounding errors)."""

    def __init__(self, dims, depth, state, rec=None, conv=None):
        self.d, self.depth, self.hm = dims, depth, head_map(dims)
        self.S = f64(state)
        self.Sb = np.abs(self.S)
        s, hk, hv = dims.n_slots, dims.H_k, dims.H_v
        self.n = np.zeros(s, int)
        self.e = np.zeros((s, hv, depth))
        self.k = np.zeros((s, hk, depth, dims.d_k))
        self.u = np.zeros((s, hv, depth, dims.d_v))
        self.ub = np.zeros_like(self.u)
        if rec is not None:
            self.n, self.e = rec.n.cpu().numpy().astype(int), f64(rec.e)
            self.k, self.u = f64(rec.k), f64(rec.u)
            self.ub = np.abs(self.u)
        self.conv = None if conv is None else f64(conv)
        self.x = None if conv is None else np.zeros((s, depth, conv.shape[2]))

    def commit(self, slot, a, reset):
        if reset:
            self.S[slot] = 0
            self.Sb[slot] = 0
            if self.conv is not None:
                self.conv[slot] = 0
            a = 0
        for j in range(a):
            e, k = self.e[slot, :, j, None, None], self.k[slot, self.hm, j]
            self.S[slot] = e * self.S[slot] + k[:, :, None] * self.u[slot, :, j, None, :]
            self.Sb[slot] = e * self.Sb[slot] + np.abs(k)[:, :, None] * self.ub[slot, :, j, None, :]
        if a and self.conv is not None and self.conv.shape[1]:
            R = self.conv.shape[1]
            self.conv[slot] = np.concatenate([self.conv[slot], self.x[slot, :a]])[-R:]

    def draft(self, slot, q, k, v, g, beta):
        """Tokens of one sequence; returns o and its bound."""
        S, Sb = self.S[slot].copy(), self.Sb[slot].copy()
        o, ob = np.zeros(v.shape), np.zeros(v.shape)
        for i in range(len(g)):
            e, b = np.exp(g[i])[:, None, None], beta[i][:, None]
            kk, qq = k[i][self.hm], q[i][self.hm]
            S, Sb = e * S, e * Sb
            u = b * (v[i] - np.einsum("hdc,hd->hc", S, kk))
            ub = b * (np.abs(v[i]) + np.einsum("hdc,hd->hc", Sb, np.abs(kk)))
            S = S + kk[:, :, None] * u[:, None, :]
            Sb = Sb + np.abs(kk)[:, :, None] * ub[:, None, :]
            o[i] = np.einsum("hdc,hd->hc", S, qq)
            ob[i] = np.einsum("hdc,hd->hc", Sb, np.abs(qq))
            self.e[slot, :, i], self.k[slot, :, i] = np.exp(g[i]), k[i]
            self.u[slot, :, i], self.ub[slot, :, i] = u, ub
        self.n[slot] = len(g)
        return o, ob


def near(got, ref, bound, depth, d_k, what, bf16=False, rel=1e-5):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert np.isfinite(got).all(), what
    gamma = (depth + 2) * (d_k + 2 * depth + 16) * 2.0 ** -24
    room = gamma * bound + (2.0 ** -8 * np.abs(ref) if bf16 else 0.0) + 1e-30
    worst = float((np.abs(got - ref) / room).max()) if ref.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} of the bound"
    den = np.linalg.norm(ref)
    if den > 0:
        r = np.linalg.norm(got - ref) / den
        assert r < (2.0 ** -8 if bf16 else rel), f"{what}: rel {r:.2e}"


def inputs(dims, T, gen, dtype, out=torch.float32):
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k = rn(T, dims.H_k, dims.d_k), rn(T, dims.H_k, dims.d_k)
    q = q / q.norm(dim=-1, keepdim=True) * dims.d_k ** -0.5
    k = k / k.norm(dim=-1, keepdim=True)
    g = -torch.exp(rn(T, dims.H_v) * 1.5 - 2.0)
    beta = torch.sigmoid(rn(T, dims.H_v))
    c = lambda t: t.to(dtype).cuda()  # noqa: E731
    return (c(q), c(k), c(rn(T, dims.H_v, dims.d_v)), g.cuda(), beta.cuda(),
            torch.full((T, dims.H_v, dims.d_v), float("nan"), dtype=out, device="cuda"))


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run_steps(dims, depth, steps, dtype, out, seed, slots, reset_step=None):
    """Several draft steps in a row (lens, accepted of each), compared after each."""
    gen = torch.Generator().manual_seed(seed)
    state = (torch.randn((dims.n_slots, dims.H_v, dims.d_k, dims.d_v), generator=gen) * 0.1).cuda()
    rec = gdn.draft_record(dims, depth, device="cuda")
    for t in (rec.e, rec.k, rec.u):
        t.fill_(float("nan"))  # rows outside a record are never read
    m = Model(dims, depth, state)
    idle = [s for s in range(dims.n_slots) if s not in slots]
    before = state[idle].clone()
    for i, (lens, acc) in enumerate(steps):
        T = sum(lens)
        q, k, v, g, beta, o = inputs(dims, T, gen, dtype, out)
        reset = None
        if reset_step == i:
            reset = torch.tensor([j % 2 for j in range(len(slots))], dtype=torch.uint8).cuda()
        gdn.draft_step(dims, q, k, v, g, beta, state, i32(slots), cu_of(lens), i32(acc), rec, o,
                       reset=reset)
        assert device_status() == 0
        t0 = 0
        ref, bnd = np.zeros(tuple(o.shape)), np.zeros(tuple(o.shape))
        for n, slot in enumerate(slots):
            sl = slice(t0, t0 + lens[n])
            m.commit(slot, acc[n], reset is not None and bool(reset[n]))
            ref[sl], bnd[sl] = m.draft(slot, f64(q)[sl], f64(k)[sl], f64(v)[sl], f64(g)[sl],
                                       f64(beta)[sl])
            t0 += lens[n]
        args = (depth, dims.d_k)
        near(f64(o), ref, bnd, *args, f"o of step {i}", bf16=out == torch.bfloat16)
        near(f64(state)[slots], m.S[slots], m.Sb[slots], *args, f"state of step {i}")
        for n, slot in enumerate(slots):
            L = lens[n]
            assert int(rec.n[slot]) == L
            near(f64(rec.e)[slot, :, :L], m.e[slot, :, :L], m.e[slot, :, :L], *args, "record e")
            assert np.array_equal(f64(rec.k)[slot, :, :L], m.k[slot, :, :L])
            near(f64(rec.u)[slot, :, :L], m.u[slot, :, :L], m.ub[slot, :, :L], *args, "record u")
        assert torch.equal(state[idle], before)
        assert not rec.n[idle].any()
    return state, rec


@pytest.mark.parametrize("dtype,out", [(torch.float16, torch.bfloat16),
                                       (torch.float32, torch.float32),
                                       (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("depth", [1, 3, 4, 5, 8, 11, 16])
def test_steps_match_the_recurrence(depth, dtype, out):
    dims = Dims(n_slots=7, H_k=2, H_v=4, d_k=128, d_v=128)
    full = [depth] * 4
    mix = [depth, 0, 1, (depth + 1) // 2]
    steps = [(mix, [0, 0, 0, 0]), (full, [depth, 0, 1, 0]), (mix, [0, depth, depth // 2, depth]),
             ([0, 0, 1, 1], [depth, 0, 1, 0])]
    run_steps(dims, depth, steps, dtype, out, 100 + depth, [5, 0, 3, 6])


@pytest.mark.parametrize("hk,hv,dk,dv,layout", [
    (1, 1, 32, 32, 0), (3, 3, 64, 128, 0), (2, 6, 128, 64, gdn.GDN_GQA_TILED),
    (3, 12, 64, 32, 0), (1, 8, 32, 128, gdn.GDN_GQA_TILED), (5, 5, 128, 32, 0)])
def test_head_shapes(hk, hv, dk, dv, layout):
    dims = Dims(n_slots=4, H_k=hk, H_v=hv, d_k=dk, d_v=dv, layout=layout)
    steps = [([6, 2, 0], [0, 0, 0]), ([1, 7, 3], [4, 2, 0]), ([2, 2, 2], [1, 0, 3])]
    run_steps(dims, 7, steps, torch.float32, torch.float32, hk * 100 + dk, [2, 3, 0])


def test_reset_drops_the_record():
    dims = Dims(n_slots=4, H_k=2, H_v=2, d_k=128, d_v=128)
    steps = [([4, 4, 4], [0, 0, 0]), ([2, 0, 4], [3, 4, 1]), ([1, 2, 0], [2, 0, 4])]
    run_steps(dims, 4, steps, torch.float32, torch.float32, 9, [3, 1, 0], reset_step=1)


def test_gates_of_any_size():
    """exp(g) = 0 (g = -inf, -1e4), 1 (g = 0), tiny and ordinary decays side by side: nothing is
    lost to differences of sums of g."""
    dims = Dims(n_slots=2, H_k=1, H_v=2, d_k=64, d_v=64)
    gen = torch.Generator().manual_seed(5)
    state = torch.randn((2, 2, 64, 64), generator=gen).cuda()
    rec = gdn.draft_record(dims, 16)
    m = Model(dims, 16, state)
    vals = torch.tensor([0.0, -1e4, -1e-3, float("-inf"), -0.5, -88.0, -1e-7, -40.0])
    for step in range(2):
        q, k, v, g, beta, o = inputs(dims, 16, gen, torch.float32)
        g.copy_(vals[torch.randint(0, 8, (16, 2), generator=gen)])
        if step == 1:
            g[3:] = -0.01
        acc = 0 if step == 0 else 16
        gdn.draft_step(dims, q, k, v, g, beta, state, i32([1]), cu_of([16]), i32([acc]), rec, o)
        m.commit(1, acc, False)
        ref, bnd = m.draft(1, *(f64(t) for t in (q, k, v, g, beta)))
        near(f64(o), ref, bnd, 16, 64, "o")
        near(f64(state)[1], m.S[1], m.Sb[1], 16, 64, "state")
    assert device_status() == 0


def test_one_token_per_sequence_equals_decode():
    """cu_seqlens NULL; committing every token is the decode step."""
    dims = Dims(n_slots=3, H_k=2, H_v=4, d_k=128, d_v=128)
    gen = torch.Generator().manual_seed(11)
    state = (torch.randn((3, 4, 128, 128), generator=gen) * 0.1).cuda()
    ref_state = state.clone()
    rec = gdn.draft_record(dims, 2)
    slots = i32([2, 0])
    for step in range(4):
        q, k, v, g, beta, o = inputs(dims, 2, gen, torch.float32)
        ref = torch.empty_like(o)
        gdn.decode_step(dims, q, k, v, g, beta, ref_state, slots, ref)
        gdn.draft_step(dims, q, k, v, g, beta, state, slots, None,
                       None if step == 0 else i32([1, 1]), rec, o)
        near(f64(o), f64(ref), np.abs(f64(ref)) + 1.0, 4, 128, "o", rel=1e-6)
    none = torch.empty((0, 4, 128), device="cuda")
    gdn.draft_step(dims, none[:, :2], none[:, :2], none, none[:, :, 0].contiguous(),
                   none[:, :, 0].contiguous(), state, slots, i32([0, 0, 0]), i32([1, 1]), rec, none)
    assert device_status() == 0 and not rec.n.any()
    near(f64(state), f64(ref_state), np.abs(f64(ref_state)) + 1.0, 4, 128, "state", rel=1e-6)


# ------------------------------------------------------------------------------ the whole layer
def layer_inputs(dims, T, gen, xdt):
    r = dims.H_v // dims.H_k
    mixed = dims.layout & gdn.GDN_GATES_MIXED_BA
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    a = rn(T, dims.H_k, 2 * r) if mixed else rn(T, dims.H_v)
    b = None if mixed else rn(T, dims.H_v)
    return rn(T, dims.conv_dim).to(xdt).cuda(), a.cuda(), None if b is None else b.cuda()


def front64(dims, conv_w, A_log, dt_bias, win, x, a, b):
    """q, k, v, g, beta of a sequence's tokens behind the window, in 64 bits."""
    T, hk, hv, dk, dv = len(x), dims.H_k, dims.H_v, dims.d_k, dims.d_v
    y = x
    if dims.d_conv:
        seen = np.concatenate([win, x]) if dims.d_conv > 1 else x
        y = np.stack([(seen[i:i + dims.d_conv] * conv_w.T).sum(0) for i in range(T)]) if T else x
        y = y / (1 + np.exp(-y))
    q, k, v = np.split(y, [hk * dk, 2 * hk * dk], axis=1)
    q, k, v = q.reshape(T, hk, dk), k.reshape(T, hk, dk), v.reshape(T, hv, dv)
    q = q / np.sqrt((q ** 2).sum(-1, keepdims=True) + EPS) * dk ** -0.5
    k = k / np.sqrt((k ** 2).sum(-1, keepdims=True) + EPS)
    if b is None:
        r = hv // hk
        a, b = a[:, :, r:].reshape(T, hv), a[:, :, :r].reshape(T, hv)
    return q, k, v, -np.exp(A_log) * np.logaddexp(0, a + dt_bias), 1 / (1 + np.exp(-b))


@pytest.mark.parametrize("xdt,sdt,out", [(torch.bfloat16, torch.bfloat16, torch.bfloat16),
                                         (torch.float32, torch.float32, torch.float32),
                                         (torch.bfloat16, torch.float32, torch.float32)])
@pytest.mark.parametrize("hk,hv,dk,dv,d_conv,layout,gated", [
    (2, 4, 128, 128, 4, 0, True), (2, 4, 128, 128, 4, gdn.GDN_GATES_MIXED_BA, False),
    (1, 3, 64, 32, 3, gdn.GDN_GQA_TILED, True), (3, 3, 32, 128, 2, 0, False),
    (2, 2, 128, 64, 1, 0, False), (1, 2, 64, 64, 0, 0, True)])
def test_layer_draft(hk, hv, dk, dv, d_conv, layout, gated, xdt, sdt, out):
    dims = Dims(n_slots=5, H_k=hk, H_v=hv, d_k=dk, d_v=dv, d_conv=d_conv, layout=layout)
    depth, slots = 6, [4, 1, 2]
    gen = torch.Generator().manual_seed(dk + dv + d_conv)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    conv_w = rn(dims.conv_dim, d_conv) * 0.5 if d_conv else None
    layer = GDNLayer(dims, conv_w, rn(hv) - 1.0, rn(hv), eps=EPS, conv_dtype=sdt, o_dtype=out)
    layer.state.copy_(rn(*layer.state.shape) * 0.1)
    if layer.conv_state is not None:
        layer.conv_state.copy_(rn(*layer.conv_state.shape))
    rec = layer.draft_record(depth)
    m = Model(dims, depth, layer.state, conv=layer.conv_state)
    cw = None if conv_w is None else f64(conv_w)
    lens_acc = [([6, 1, 0], [0, 0, 0]), ([2, 5, 3], [2, 1, 0]), ([0, 3, 6], [1, 5, 2]),
                ([1, 0, 2], [0, 2, 6])]
    for step, (lens, acc) in enumerate(lens_acc):
        T = sum(lens)
        x, a, b = layer_inputs(dims, T, gen, xdt)
        z, nw = rn(T, hv, dv).to(torch.bfloat16).cuda(), (1 + 0.1 * rn(dv)).cuda()
        gate = OutGate(z, nw, EPS) if gated else None
        reset = None
        if step == 3:
            reset = torch.tensor([1, 0, 0], dtype=torch.uint8, device="cuda")
        o = layer.draft(x, a, b, cu_of(lens), i32(slots), i32(acc), rec, reset=reset, gate=gate)
        assert device_status() == 0
        t0 = 0
        ref, bnd = np.zeros((T, hv, dv)), np.zeros((T, hv, dv))
        for n, slot in enumerate(slots):
            sl = slice(t0, t0 + lens[n])
            m.commit(slot, acc[n], reset is not None and bool(reset[n]))
            win = m.conv[slot] if m.conv is not None else None
            xs = f64(x)[sl]
            f = front64(dims, cw, f64(layer.A_log), f64(layer.dt_bias), win, xs, f64(a)[sl],
                        None if b is None else f64(b)[sl])
            ref[sl], bnd[sl] = m.draft(slot, *f)
            if m.conv is not None:
                m.x[slot, :lens[n]] = f64(x[sl].to(sdt))
            t0 += lens[n]
        if gated:
            inv = 1 / np.sqrt((ref ** 2).mean(-1, keepdims=True) + EPS)
            zz = f64(z)
            w = f64(nw) * zz / (1 + np.exp(-zz))
            # d(o inv) <= inv (|do| + |o| inv^2 mean(|o| |do|)): bounded by the row's largest
            bnd = inv * (bnd + bnd.max(-1, keepdims=True)) * np.abs(w)
            ref = ref * inv * w
        # the front adds its own roundings (4 taps, exp, a norm over d_k): twice the steps
        near(f64(o), ref, 2 * bnd, depth, dk, f"o of step {step}", bf16=out == torch.bfloat16)
        near(f64(layer.state)[slots], m.S[slots], 2 * m.Sb[slots], depth, dk, "state")
        if m.conv is not None:
            assert np.array_equal(f64(layer.conv_state), m.conv)  # rolled bit for bit
            for n, slot in enumerate(slots):
                assert np.array_equal(f64(rec.x)[slot, :lens[n]], m.x[slot, :lens[n]])


def test_drafts_of_a_layer_follow_its_decode():
    """Speculative decoding and plain decoding of the same tokens: draft 4, keep 0 to 4 of them,
    over several rounds; the committed tokens' outputs, state and window are those of decode."""
    dims = Dims(n_slots=2, H_k=4, H_v=8, d_k=128, d_v=128)
    gen = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    w = (rn(dims.conv_dim, 4) * 0.5, rn(8) - 2.0, rn(8))
    plain, spec = (GDNLayer(dims, *w, o_dtype=torch.float32) for _ in range(2))
    rec = spec.draft_record(4)
    slots = i32([1])
    stream_x, stream_a, stream_b = layer_inputs(dims, 24, gen, torch.bfloat16)
    want = []
    for t in range(24):
        want.append(plain.decode(stream_x[t:t + 1], stream_a[t:t + 1], stream_b[t:t + 1],
                                 slots).clone())
        if t == 15:
            state16, conv16 = plain.state.clone(), plain.conv_state.clone()
    want = torch.cat(want)
    at, accepted = 0, 0
    for keep in [4, 0, 3, 1, 2, 4, 2]:  # 16 tokens
        n = 4
        wrong = layer_inputs(dims, n, gen, torch.bfloat16)  # tokens that will not be kept
        pick = lambda s, x: torch.cat([s[at:at + keep], x[keep:]]).contiguous()  # noqa: E731
        o = spec.draft(pick(stream_x, wrong[0]), pick(stream_a, wrong[1]), pick(stream_b, wrong[2]),
                       cu_of([n]), slots, i32([accepted]), rec)
        ref = f64(want[at:at + keep])
        near(f64(o)[:keep], ref, np.abs(ref) + 1.0, 16, 128, "o")
        at, accepted = at + keep, keep
    spec.commit_draft(slots, i32([accepted]), rec)
    assert device_status() == 0 and at == 16
    assert torch.equal(spec.conv_state[1], conv16[1])
    near(f64(spec.state[1]), f64(state16[1]), np.abs(f64(state16[1])) + 1.0, 16, 128, "state")
    assert not rec.n.any()


# ------------------------------------------------------------------------- refusals, odd calls
def small(n_slots=4, depth=4, seed=1):
    dims = Dims(n_slots=n_slots, H_k=1, H_v=2, d_k=64, d_v=64)
    gen = torch.Generator().manual_seed(seed)
    state = torch.randn((n_slots, 2, 64, 64), generator=gen).cuda()
    rec = gdn.draft_record(dims, depth)
    return dims, gen, state, rec


@pytest.mark.parametrize("what,status", [("long", -1), ("much", -1), ("negative", -1),
                                         ("slot", -2), ("twice", -2), ("cu", -1)])
def test_a_bad_sequence_is_skipped_whole(what, status):
    dims, gen, state, rec = small()
    q, k, v, g, beta, o = inputs(dims, 6, gen, torch.float32)
    gdn.draft_step(dims, q, k, v, g, beta, state, i32([0, 1, 2]), cu_of([2, 2, 2]), None, rec, o)
    assert device_status() == 0
    keep = [t.clone() for t in (state, rec.n, rec.e, rec.k, rec.u)]
    lens, slots, acc = [2, 2, 2], [0, 1, 2], [1, 1, 1]
    bad = 1
    if what == "long":
        lens = [1, 5, 1]
    elif what == "much":
        acc[1] = 3
    elif what == "negative":
        acc[1] = -1
    elif what == "slot":
        slots[1] = 4
    elif what == "twice":
        slots, bad = [0, 2, 2], 2
    q, k, v, g, beta, o = inputs(dims, 7, gen, torch.float32)
    cu = cu_of(lens)
    if what == "cu":
        cu = i32([0, 2, 99, 6])
        lens, bad = [2, 0, 0], 1  # sequence 2 starts beyond the tokens too
    gdn.draft_step(dims, q, k, v, g, beta, state, i32(slots), cu, i32(acc), rec, o)
    assert device_status() == status
    t0 = sum(lens[:bad])
    assert torch.isnan(o[t0:t0 + lens[bad]]).all()
    assert torch.isfinite(o[:lens[0]]).all()
    gone = {"twice": [1, 3], "slot": [1, 3], "cu": [1, 2, 3]}.get(what, [1, 3])
    for new, old in zip((state, rec.n, rec.e, rec.k, rec.u), keep):
        assert torch.equal(new[gone], old[gone])
    assert not torch.equal(state[0], keep[0][0])


def test_gated_layer_leaves_a_skipped_sequence_alone():
    dims = Dims(n_slots=3, H_k=1, H_v=2, d_k=64, d_v=64)
    layer = GDNLayer(dims, torch.randn(dims.conv_dim, 4), torch.zeros(2), torch.zeros(2))
    rec = layer.draft_record(3)
    x, a, b = layer_inputs(dims, 6, torch.Generator().manual_seed(1), torch.bfloat16)
    gate = OutGate(torch.randn((6, 2, 64), device="cuda"), torch.ones(64, device="cuda"))
    out = torch.full((6, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    layer.draft(x, a, b, cu_of([2, 2, 2]), i32([0, 9, 2]), i32([0, 0, 0]), rec, gate=gate, out=out)
    assert device_status() == -2
    assert (out[2:4] == 7.0).all() and not (out[:2] == 7.0).all() and not (out[4:] == 7.0).all()


def test_python_refusals():
    dims, gen, state, rec = small()
    q, k, v, g, beta, o = inputs(dims, 2, gen, torch.float32)
    ok = dict(slot_ids=i32([0]), cu_seqlens=cu_of([2]), accepted=i32([0]), record=rec)

    def call(**over):
        a = {**ok, **over}
        gdn.draft_step(dims, q, k, v, g, beta, state, a["slot_ids"], a["cu_seqlens"],
                       a["accepted"], a["record"], o, workspace=over.get("workspace"))

    call()
    for bad in (dict(slot_ids=ok["slot_ids"].long()), dict(cu_seqlens=cu_of([1, 1])),
                dict(accepted=i32([0, 0])), dict(accepted=ok["accepted"].long()),
                dict(record=gdn.draft_record(Dims(3, 1, 2, 64, 64), 4)),
                dict(record=gdn.DraftRecord(rec.n, rec.e, rec.k, rec.u.double())),
                dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call(**bad)
    args = dict(q=q, k=k, v=v, g=g, beta=beta, state=state, o=o)
    for name, t in (("q", q[:, :, :32].contiguous()), ("k", k[:1]), ("k", k.half()), ("v", v[:1]),
                    ("v", v.double()), ("g", g[:1]), ("g", g.half()), ("beta", beta.cpu()),
                    ("state", state[:3]), ("state", state.half()), ("o", o[:1]), ("o", o.cpu()),
                    ("q", q.transpose(0, 1)), ("o", None)):
        w = {**args, name: t}
        with pytest.raises(ValueError):
            gdn.draft_step(dims, w["q"], w["k"], w["v"], w["g"], w["beta"], w["state"],
                           ok["slot_ids"], ok["cu_seqlens"], None, rec, w["o"])
    with pytest.raises(gdn.GdnError) as e:
        call(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == gdn._lib.GDN_EWORKSPACE
    with pytest.raises(gdn.GdnError) as e:
        gdn.draft_step(dims, q, k, v, g, beta, state, ok["slot_ids"], ok["cu_seqlens"], None,
                       gdn.draft_record(dims, 17), o)
    assert e.value.status == gdn._lib.GDN_EINVAL
    assert device_status() == 0


def test_graph_replay_and_side_stream():
    """A captured step replayed on changing inputs, and two steps on two streams with workspaces of
    their own, give what the eager calls on one stream give."""
    dims, gen, state, rec = small(n_slots=8, depth=5)
    lens, slots, acc = [5, 3], i32([6, 2]), i32([2, 3])
    q, k, v, g, beta, o = inputs(dims, 8, gen, torch.float16, torch.bfloat16)
    ws = torch.empty(gdn.draft_workspace_size(dims, 8, 2, 5), dtype=torch.uint8, device="cuda")
    cu = cu_of(lens)

    def step(st, rc, out, s=None, w=ws, sl=slots):
        gdn.draft_step(dims, q, k, v, g, beta, st, sl, cu, acc, rc, out, workspace=w, stream=s)

    clone = lambda r: gdn.DraftRecord(r.n.clone(), r.e.clone(), r.k.clone(), r.u.clone())  # noqa: E731
    # the record of a first draft, so that the accepted counts are valid
    gdn.draft_step(dims, q, k, v, g, beta, state, slots, cu, None, rec, o, workspace=ws)
    s1, r1, o1 = state.clone(), clone(rec), torch.empty_like(o)
    s2, r2, o2 = state.clone(), clone(rec), torch.empty_like(o)
    keep_s, keep_r = state.clone(), clone(rec)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s2, r2, o2)
    torch.cuda.current_stream().wait_stream(side)
    s2.copy_(keep_s)
    for x, y in ((r2.n, keep_r.n), (r2.e, keep_r.e), (r2.k, keep_r.k), (r2.u, keep_r.u)):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s2, r2, o2)
    for _ in range(3):
        step(s1, r1, o1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, o2) and torch.equal(s1, s2) and torch.equal(r1.u, r2.u)
        q.copy_(q.flip(0))
        v.mul_(0.5)
    # two streams, other slots, own workspaces
    s3, r3, o3, o4 = keep_s.clone(), clone(keep_r), torch.empty_like(o), torch.empty_like(o)
    other = i32([1, 5])
    r3.n[other.long()] = keep_r.n[slots.long()]
    r3.e[other.long()], r3.k[other.long()] = r3.e[slots.long()], r3.k[slots.long()]
    r3.u[other.long()], s3[other.long()] = r3.u[slots.long()], s3[slots.long()]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    w2 = torch.empty_like(ws)
    step(s3, r3, o3, a, ws)
    step(s3, r3, o4, b, w2, other)
    torch.cuda.synchronize()
    assert torch.equal(o3, o4) and torch.equal(s3[slots.long()], s3[other.long()])
    assert device_status() == 0


def test_offsets_beyond_32_bits():
    """A pool of more than 2^31 state values and record bytes: its last slot works like the first
    of a small pool."""
    big = Dims(n_slots=4200, H_k=16, H_v=32, d_k=128, d_v=128)
    one = Dims(n_slots=1, H_k=16, H_v=32, d_k=128, d_v=128)
    gen = torch.Generator().manual_seed(2)
    q, k, v, g, beta, o = inputs(big, 3, gen, torch.float16, torch.bfloat16)
    s0 = torch.randn((1, 32, 128, 128), generator=gen).cuda()
    state = torch.empty((4200, 32, 128, 128), device="cuda")
    state[4199] = s0[0]
    rec, rec0, o0 = gdn.draft_record(big, 16), gdn.draft_record(one, 16), torch.empty_like(o)
    for acc in ([0], [2]):
        gdn.draft_step(big, q, k, v, g, beta, state, i32([4199]), cu_of([3]), i32(acc), rec, o)
        gdn.draft_step(one, q, k, v, g, beta, s0, i32([0]), cu_of([3]), i32(acc), rec0, o0)
    assert device_status() == 0
    assert torch.equal(o, o0) and torch.equal(state[4199], s0[0])
    assert torch.equal(rec.u[4199], rec0.u[0]) and torch.equal(rec.k[4199], rec0.k[0])


def test_results_do_not_depend_on_the_batch():
    dims = Dims(n_slots=40, H_k=2, H_v=4, d_k=128, d_v=128)
    gen = torch.Generator().manual_seed(8)
    state = torch.randn((40, 4, 128, 128), generator=gen).cuda()
    alone, rec, rec1 = state.clone(), gdn.draft_record(dims, 4), gdn.draft_record(dims, 4)
    q, k, v, g, beta, o = inputs(dims, 160, gen, torch.float16, torch.bfloat16)
    o1 = torch.empty_like(o[:4])
    slots = torch.randperm(40, generator=gen).int().cuda()
    for acc in (0, 3):
        gdn.draft_step(dims, q, k, v, g, beta, state, slots, cu_of([4] * 40), i32([acc] * 40), rec, o)
        s = slots[17:18].contiguous()
        sl = slice(68, 72)
        gdn.draft_step(dims, q[sl], k[sl], v[sl], g[sl], beta[sl], alone, s, cu_of([4]), i32([acc]),
                       rec1, o1)
        assert torch.equal(o1, o[sl]) and torch.equal(alone[s.long()], state[s.long()])
    assert device_status() == 0


@pytest.mark.parametrize("depth", [4, 7, 16])
def test_many_sequences_equal_single_calls(depth):
    """More tiles than blocks, ragged drafts with commits only, nothing at all, resets and skipped
    sequences among them: every sequence gives the bits of a call of its own."""
    dims = Dims(n_slots=220, H_k=2, H_v=6, d_k=128, d_v=128)
    gen = torch.Generator().manual_seed(depth)
    n = 200  # x 6 heads x 2 column tiles
    state = torch.randn((220, 6, 128, 128), generator=gen).cuda()
    alone = state.clone()
    slots = torch.randperm(220, generator=gen)[:n].int().cuda()
    slots[50], slots[120] = -1, slots[3]  # out of range, taken already: both are skipped
    recs = [gdn.draft_record(dims, depth) for _ in range(2)]
    lens0 = [depth] * n
    q, k, v, g, beta, o = inputs(dims, sum(lens0), gen, torch.float16)
    gdn.draft_step(dims, q, k, v, g, beta, state, slots, cu_of(lens0), None, recs[0], o)
    assert device_status() == -2
    for x, y in ((recs[1].n, recs[0].n), (recs[1].e, recs[0].e), (recs[1].k, recs[0].k),
                 (recs[1].u, recs[0].u)):
        x.copy_(y)
    lens = [(7 * i) % (depth + 1) for i in range(n)]
    acc = [(5 * i) % (depth + 1) if i % 3 else 0 for i in range(n)]
    reset = torch.tensor([i % 11 == 4 for i in range(n)], dtype=torch.uint8).cuda()
    q, k, v, g, beta, o = inputs(dims, sum(lens), gen, torch.float16)
    gdn.draft_step(dims, q, k, v, g, beta, state, slots, cu_of(lens), i32(acc), recs[0], o,
                   reset=reset)
    assert device_status() == -2
    o1, t0 = torch.full_like(o, float("nan")), 0
    for i in range(n):
        sl = slice(t0, t0 + lens[i])
        t0 += lens[i]
        if i in (50, 120):
            assert torch.isnan(o[sl]).all()
            continue
        one = [t[sl].clone() for t in (q, k, v, g, beta, o1)]  # slices need not be 16-byte aligned
        gdn.draft_step(dims, *one[:5], alone, slots[i:i + 1].clone(), cu_of([lens[i]]),
                       i32([acc[i]]), recs[1], one[5], reset=reset[i:i + 1].clone())
        o1[sl] = one[5]
    assert device_status() == 0
    assert torch.equal(o.nan_to_num(7.0), o1.nan_to_num(7.0)) and torch.equal(state, alone)
    for x, y in ((recs[1].n, recs[0].n), (recs[1].e, recs[0].e), (recs[1].k, recs[0].k),
                 (recs[1].u, recs[0].u)):
        assert torch.equal(x, y)


def test_scales_of_state_and_keys():
    """States of 1e-12 to 1e12 and keys far from unit length: the parts of the column sums lose
    nothing to the values' size."""
    dims = Dims(n_slots=4, H_k=1, H_v=1, d_k=128, d_v=64)
    gen = torch.Generator().manual_seed(21)
    scale = torch.tensor([1e-12, 1.0, 1e6, 1e12])[:, None, None, None]
    state = (torch.randn((4, 1, 128, 64), generator=gen) * scale).cuda()
    rec = gdn.draft_record(dims, 3)
    m = Model(dims, 3, state)
    q, k, v, g, beta, o = inputs(dims, 12, gen, torch.float32)
    k.mul_(torch.logspace(-3, 0, 12).cuda()[:, None, None])
    gdn.draft_step(dims, q, k, v, g, beta, state, i32([0, 1, 2, 3]), cu_of([3] * 4), None, rec, o)
    assert device_status() == 0
    for n in range(4):
        sl = slice(3 * n, 3 * n + 3)
        ref, bnd = m.draft(n, *(f64(t)[sl] for t in (q, k, v, g, beta)))
        near(f64(o)[sl], ref, bnd, 3, 128, f"o at {n}")
        near(f64(rec.u)[n, :, :3], m.u[n, :, :3], m.ub[n, :, :3], 3, 128, f"u at {n}")


def test_layer_refusals():
    dims = Dims(n_slots=2, H_k=1, H_v=2, d_k=64, d_v=64)
    layer = GDNLayer(dims, torch.randn(dims.conv_dim, 4), torch.zeros(2), torch.zeros(2))
    rec = layer.draft_record(3)
    x, a, b = layer_inputs(dims, 2, torch.Generator().manual_seed(1), torch.bfloat16)
    gate = OutGate(torch.zeros((2, 2, 64), device="cuda"), torch.ones(64, device="cuda"))

    def call(x=x, a=a, b=b, rec=rec, gate=gate, cu=cu_of([2])):
        layer.draft(x, a, b, cu, i32([0]), i32([0]), rec, gate=gate)

    call()
    for bad in (dict(x=x[:, :-4].contiguous()), dict(a=a[:1]), dict(b=b.half()),
                dict(rec=gdn.DraftRecord(rec.n, rec.e, rec.k, rec.u)),
                dict(rec=gdn.DraftRecord(rec.n, rec.e, rec.k, rec.u, rec.x.float())),
                dict(gate=OutGate(gate.z[:1], gate.norm_w)),
                dict(gate=OutGate(gate.z, gate.norm_w[:32])), dict(cu=cu_of([1, 1]))):
        with pytest.raises(ValueError):
            call(**bad)
    assert device_status() == 0


def test_a_stream_of_its_own_without_a_workspace():
    """The workspace made for a call on another stream is that stream's: the current stream may
    take memory and write it meanwhile."""
    dims, gen, state, rec = small(n_slots=8, depth=5)
    q, k, v, g, beta, o = inputs(dims, 8, gen, torch.float16)
    slots, cu = i32([6, 2]), cu_of([5, 3])
    want_o = torch.empty_like(o)
    gdn.draft_step(dims, q, k, v, g, beta, state, slots, cu, None, rec, want_o)
    want = rec.u.clone()
    side = torch.cuda.Stream()
    for _ in range(20):
        rec.u.zero_()
        side.wait_stream(torch.cuda.current_stream())
        gdn.draft_step(dims, q, k, v, g, beta, state, slots, cu, None, rec, o, stream=side)
        torch.full((gdn.draft_workspace_size(dims, 8, 2, 5),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, want_o) and torch.equal(rec.u, want)
    assert device_status() == 0


@pytest.mark.parametrize("depth", [4, 8, 16])
def test_nan_and_infinity_stay_behind_their_token(depth):
    """A token that is not finite leaves the tokens before it, the other sequences and the
    committed state as they were; committing only what lies before it is clean."""
    dims = Dims(n_slots=3, H_k=1, H_v=2, d_k=64, d_v=64)
    gen = torch.Generator().manual_seed(depth)
    state = torch.randn((3, 2, 64, 64), generator=gen).cuda()
    rec = gdn.draft_record(dims, depth)
    q, k, v, g, beta, o = inputs(dims, 2 * depth, gen, torch.float32)
    args = (i32([0, 2]), cu_of([depth, depth]))
    s0, r0 = state.clone(), gdn.draft_record(dims, depth)
    want = torch.empty_like(o)
    gdn.draft_step(dims, q, k, v, g, beta, s0, *args, None, r0, want)
    for at in range(1, depth):
        for t, value in ((k, float("nan")), (v, float("inf")), (q, float("nan"))):
            bad = t.clone()
            bad[at] = value
            x = {id(q): q, id(k): k, id(v): v}
            x[id(t)] = bad
            gdn.draft_step(dims, x[id(q)], x[id(k)], x[id(v)], g, beta, state, *args, None, rec, o)
            assert torch.equal(o[:at], want[:at]) and torch.equal(o[depth:], want[depth:])
            assert not torch.isfinite(o[at]).all()
            assert torch.equal(rec.u[0, :, :at], r0.u[0, :, :at]) and torch.equal(rec.u[2], r0.u[2])
            assert torch.equal(state, s0)
    none = [t[:0] for t in (q, k, v, g, beta)]
    for st, r in ((state, rec), (s0, r0)):
        gdn.draft_step(dims, *none, st, i32([0, 2]), cu_of([0, 0]), i32([depth - 1, depth]), r,
                       o[:0].clone())
    assert torch.equal(state, s0) and device_status() == 0
