"""GDNBlock: the projections (gdn_linear) around the layer's decode, prefill and draft steps, run
together from hidden states to hidden states, against the same formulas in 64 bits.

Tolerances. The block rounds to bf16 (half a step, h = 2^-8) three times on the way: x, z and o.
To first order an output is off by the sum of what each rounding moves it, and errors of random
sign add in squares: relative to the norm of the block's own contribution (the output without the
residual), x enters through q, k and v (each normalised or linear, slopes of SiLU up to 1.1) and
through all earlier tokens' state, z and o once each, and the output is rounded once more. With up
to 4 h for x and h for each of the others in the L2 norm this is at most 7 h = 0.027; the gates and
the state are fp32.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_19_b200 as gdn
from gated_deltanet_linear_19_b200 import Dims, device_status
from gated_deltanet_linear_19_b200.layer import GDNBlock, GDNLayer

pytestmark = pytest.mark.gpu

EPS = 1e-6
REL = 7 * 2.0 ** -8


def make(dims, hidden, seed):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    layer = GDNLayer(dims, rn(dims.conv_dim, 4) * 0.5, rn(dims.H_v) - 2.0, rn(dims.H_v), eps=EPS)
    w = [(rn(n, hidden) * hidden ** -0.5).bfloat16()
         for n in (dims.conv_dim, dims.H_v * dims.d_v, 2 * dims.H_v)]
    out = (rn(hidden, dims.H_v * dims.d_v) * (dims.H_v * dims.d_v) ** -0.5).bfloat16()
    return GDNBlock(layer, *w, 1 + 0.1 * rn(dims.d_v), out, norm_eps=EPS), gen


class Plain:
    """One sequence of the block, token by token in 64 bits."""

    def __init__(self, block):
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        self.d, layer = block.layer.dims, block.layer
        d = self.d
        self.wx, self.wz, self.wg, self.wo = (f(w) for w in (block.w_x, block.w_z, block.w_gates,
                                                             block.w_out))
        self.nw, self.cw, self.al, self.dt = (f(t) for t in (block.norm_w, layer.conv_w,
                                                             layer.A_log, layer.dt_bias))
        self.S = np.zeros((d.H_v, d.d_k, d.d_v))
        self.win = np.zeros((3, d.conv_dim))
        h = np.arange(d.H_v)
        self.hm = h % d.H_k if d.layout & gdn.GDN_GQA_TILED else h // (d.H_v // d.H_k)

    def token(self, hidden):
        d, sg = self.d, lambda t: 1 / (1 + np.exp(-t))
        self.win = np.concatenate([self.win, (self.wx @ hidden)[None]])
        y = (self.win * self.cw.T).sum(0)
        self.win = self.win[1:]
        y = y * sg(y)
        q, k, v = np.split(y, [d.H_k * d.d_k, 2 * d.H_k * d.d_k])
        q, k, v = q.reshape(-1, d.d_k), k.reshape(-1, d.d_k), v.reshape(-1, d.d_v)
        unit = lambda t: t / np.sqrt((t * t).sum(-1, keepdims=True) + EPS)  # noqa: E731
        q, k = unit(q)[self.hm] * d.d_k ** -0.5, unit(k)[self.hm]
        g = self.wg @ hidden
        if d.layout & gdn.GDN_GATES_MIXED_BA:
            b, a = np.split(g.reshape(d.H_k, 2, -1), 2, axis=1)
            a, b = a.reshape(-1), b.reshape(-1)
        else:
            a, b = np.split(g, 2)
        e = np.exp(-np.exp(self.al) * np.logaddexp(0, a + self.dt))
        S = e[:, None, None] * self.S
        u = sg(b)[:, None] * (v - np.einsum("hdc,hd->hc", S, k))
        self.S = S + k[:, :, None] * u[:, None, :]
        o = np.einsum("hdc,hd->hc", self.S, q)
        z = (self.wz @ hidden).reshape(d.H_v, d.d_v)
        o = o / np.sqrt((o * o).mean(-1, keepdims=True) + EPS) * self.nw * z * sg(z)
        return self.wo @ o.reshape(-1)


def near(got, want, what):
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert np.isfinite(got).all(), what
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel < REL, f"{what}: {rel:.4f}"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("hk,hv,dk,dv,layout,hidden", [
    (2, 4, 128, 128, 0, 256), (2, 4, 128, 128, gdn.GDN_GATES_MIXED_BA, 136),
    (1, 3, 64, 32, gdn.GDN_GQA_TILED, 72)])
def test_prompt_then_drafts_then_decode(hk, hv, dk, dv, layout, hidden):
    """Two sequences: prompts, speculative steps that keep some of their tokens, a commit, plain
    decode steps; every kept token's output is that of the recurrence over the kept tokens."""
    dims = Dims(n_slots=3, H_k=hk, H_v=hv, d_k=dk, d_v=dv, layout=layout)
    block, gen = make(dims, hidden, 100 + dk + layout)
    plain = [Plain(block), Plain(block)]
    hid = lambda t: torch.randn((t, hidden), generator=gen).bfloat16().cuda()  # noqa: E731
    slots = i32([2, 0])
    want = lambda n, h: np.stack([plain[n].token(t) for t in h.double().cpu().numpy()])  # noqa: E731

    h = hid(70 + 5)
    y = block.prefill(h, i32([0, 70, 75]), slots)
    near(y, np.concatenate([want(0, h[:70]), want(1, h[70:])]), "prompt")

    rec = block.layer.draft_record(4)
    accepted = [0, 0]
    for step, keep in enumerate([(4, 1), (0, 2), (2, 0), (3, 2)]):
        lens = [4, 3]
        h, res = hid(7), hid(7)
        y = block.draft(h, i32([0, 4, 7]), slots, i32(accepted), rec, residual=res)
        y = y.double() - res.double()
        for n, at in enumerate((0, 4)):
            k = keep[n]
            if k:  # the others' outputs belong to a continuation that is dropped
                got = want(n, h[at:at + k])
                # the residual's own rounding: half a step of values up to 4
                ref = got / np.linalg.norm(got)
                d = (y[at:at + k].cpu().numpy() - got) / np.linalg.norm(got)
                room = REL + 2.0 ** -8 * float(res.double().norm()) / np.linalg.norm(got)
                assert np.linalg.norm(d) < room and np.isfinite(ref).all(), f"draft {step}"
        assert lens[0] >= keep[0] and lens[1] >= keep[1]
        accepted = list(keep)
    block.layer.commit_draft(slots, i32(accepted), rec)
    for step in range(3):
        h = hid(2)
        y = block.decode(h, slots)
        near(y, np.concatenate([want(0, h[:1]), want(1, h[1:])]), f"decode {step}")
    assert device_status() == 0


def test_residual_stream_in_place_and_replay():
    """out = residual, eager against a captured step that is replayed, on the same states."""
    dims = Dims(n_slots=4, H_k=2, H_v=4, d_k=128, d_v=128)
    block, gen = make(dims, 256, 5)
    hid = torch.randn((6, 256), generator=gen).bfloat16().cuda()
    stream = torch.randn((6, 256), generator=gen).bfloat16().cuda()
    slots, cu, acc = i32([1, 3]), i32([0, 3, 6]), i32([2, 1])
    rec = block.layer.draft_record(3)
    block.draft(hid, cu, slots, None, rec)
    keep = [t.clone() for t in (block.layer.state, block.layer.conv_state, rec.n, rec.e, rec.k,
                                rec.u, rec.x)]

    def restore():
        for t, k in zip((block.layer.state, block.layer.conv_state, rec.n, rec.e, rec.k, rec.u,
                         rec.x), keep):
            t.copy_(k)

    eager = stream.clone()
    out = block.draft(hid, cu, slots, acc, rec, residual=eager, out=eager)
    assert out.data_ptr() == eager.data_ptr() and not torch.equal(eager, stream)
    after = block.layer.state.clone()
    restore()
    buf = stream.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.draft(hid, cu, slots, acc, rec, residual=buf, out=buf)
    # a larger call in between takes a larger workspace: the graph's own stays
    many = torch.randn((12, 256), generator=gen).bfloat16().cuda()
    block.draft(many, i32([0, 3, 6, 9, 12]), i32([0, 1, 2, 3]), None, block.layer.draft_record(3))
    restore()
    buf.copy_(stream)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(buf, eager) and torch.equal(block.layer.state, after)
    assert device_status() == 0


def test_refusals():
    dims = Dims(n_slots=2, H_k=1, H_v=2, d_k=64, d_v=64)
    block, _ = make(dims, 64, 1)
    w = (block.w_x, block.w_z, block.w_gates, block.norm_w, block.w_out)
    for i in (0, 1, 2, 4):
        bad = list(w)
        bad[i] = w[i][:-1]
        with pytest.raises(ValueError):
            GDNBlock(block.layer, *bad)
        bad[i] = w[i].half()
        with pytest.raises(ValueError):
            GDNBlock(block.layer, *bad)
    with pytest.raises(ValueError):
        GDNBlock(block.layer, *w[:3], w[3][:-1], w[4])
    h = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        block.decode(h[:, :56], i32([0]))
    with pytest.raises(ValueError):
        block.decode(h, i32([0]), residual=torch.zeros((2, 64), device="cuda"))
    assert device_status() == 0
