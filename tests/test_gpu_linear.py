"""The matrix product with bias, activation and residual in its epilogue (gdn_linear) against the
same formula in 64 bits.

Tolerances. Products of two 16-bit numbers are exact in fp32. Adding K of them, 16 per tensor-core
instruction, rounds or truncates at most twice per instruction and once more per joined partial
sum, each by at most one step (2^-23) of a running sum that A = sum_k |x w| bounds: an element is
off by at most (K / 8 + 16) 2^-23 (A + |bias|) before the activation. The activations' slopes are at
most 1.13 and their own evaluation is good to a few steps (8 2^-23 of the value). The output adds
half its step: 2^-24 (fp32), 2^-8 (bf16), 2^-11 (fp16) of the value.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_19_b200 as gdn
from gated_deltanet_linear_19_b200 import _lib, device_status, linear

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def reference(x, w, bias=None, act="none", residual=None):
    x, w = x.double(), w.double()
    y, a = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        y, a = y + bias.double(), a + bias.double().abs()
    if act == "silu":
        y = y * torch.sigmoid(y)
    elif act == "gelu":
        y = y * torch.special.ndtr(y)
    elif act == "sigmoid":
        y = torch.sigmoid(y)
    return (y, a) if residual is None else (y + residual.double(), a + residual.double().abs())


def check(out, ref, a, k, what=""):
    out = out.double()
    assert torch.isfinite(out).all(), what
    room = 1.13 * (k / 8 + 16) * 2.0 ** -23 * a + 8 * 2.0 ** -23 * ref.abs() + \
        HALF_OF[what.split()[0]] * ref.abs() + 2.0 ** -25
    worst = float(((out - ref).abs() / room).max()) if ref.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} of the bound"


HALF_OF = {str(t): v for t, v in HALF.items()}


def rows(m, n, gen, dtype, pad=0, scale=1.0):
    """[m, n] with a row stride of n + pad elements."""
    wide = (torch.randn((m, n + pad), generator=gen) * scale).to(dtype).cuda()
    return wide[:, :n]


# rows, columns and K on both sides of every tile edge (16, 32, 64, 128, 256 tokens; 128 columns;
# 64 K elements), the smallest and odd ones
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 32, 33, 64, 65, 100, 128, 129, 255, 256, 257, 513,
                               1000])
@pytest.mark.parametrize("n,k", [(1, 8), (64, 2048), (127, 72), (128, 64), (257, 1160),
                                 (1000, 4096)])
def test_sizes(m, n, k):
    gen = torch.Generator().manual_seed(m * 7919 + n * 31 + k)
    dtype = [torch.bfloat16, torch.float16][(m + n) % 2]
    out = [torch.float32, dtype][(m + n // 2) % 2]
    x, w = rows(m, k, gen, dtype), rows(n, k, gen, dtype, scale=k ** -0.5)
    y = linear(x, w, out_dtype=out)
    assert device_status() == 0 and y.dtype == out
    check(y, *reference(x, w), k, f"{out} {m}x{n}x{k}")


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("res", [None, torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
def test_epilogues(act, res, out):
    for m, n, k in ((3, 200, 136), (70, 129, 520), (300, 515, 264), (1500, 768, 128)):
        gen = torch.Generator().manual_seed(m)
        dtype = torch.float16 if out == torch.float16 else torch.bfloat16
        x, w = rows(m, k, gen, dtype, pad=8), rows(n, k, gen, dtype, pad=16, scale=k ** -0.5)
        bias = torch.randn(n, generator=gen).cuda()
        r = None if res is None else rows(m, n, gen, res, pad=3)
        wide = torch.full((m, n + 5), 9.0, dtype=out, device="cuda")
        y = linear(x, w, bias=bias, act=act, residual=r, out=wide[:, :n])
        assert y.data_ptr() == wide.data_ptr()
        check(y, *reference(x, w, bias, act, r), k, f"{out} {act} {res} {m}")
        assert (wide[:, n:] == 9.0).all()  # nothing beyond the row
    assert device_status() == 0


@pytest.mark.parametrize("m", [1, 40, 300, 2000])
def test_residual_in_place_and_rows_beyond(m):
    """out = residual, as a residual stream is updated; rows behind the last token stay."""
    gen = torch.Generator().manual_seed(m)
    x, w = rows(m, 512, gen, torch.bfloat16), rows(256, 512, gen, torch.bfloat16, scale=0.05)
    buf = torch.randn((m + 3, 256), generator=gen).to(torch.bfloat16).cuda()
    before = buf.clone()
    linear(x, w, residual=buf[:m], out=buf[:m])
    ref, a = reference(x, w, residual=before[:m])
    check(buf[:m], ref, a, 512, "torch.bfloat16 in place")
    assert torch.equal(buf[m:], before[m:])
    assert device_status() == 0


def test_nan_and_infinity_stay_in_their_rows_and_columns():
    for m in (5, 300):
        gen = torch.Generator().manual_seed(1)
        x, w = rows(m, 256, gen, torch.bfloat16), rows(200, 256, gen, torch.bfloat16)
        good = linear(x, w, out_dtype=torch.float32)
        x, w = x.clone(), w.clone()
        x[2, 7] = float("nan")
        x[4, 100] = float("inf")
        w[131, 3] = float("nan")
        y = linear(x, w, out_dtype=torch.float32)
        assert torch.isnan(y[2]).all() and torch.isnan(y[:, 131]).all()
        assert not torch.isfinite(y[4]).any()
        keep = torch.ones_like(y, dtype=torch.bool)
        keep[2], keep[4], keep[:, 131] = False, False, False
        assert torch.equal(y[keep], good[keep])
    # saturating activations
    x = torch.full((1, 8), 1e3, dtype=torch.bfloat16, device="cuda")
    w = torch.stack([torch.full((8,), s * 1e3) for s in (1.0, -1.0)]).to(torch.bfloat16).cuda()
    for act, want in (("silu", (8e6, 0.0)), ("gelu", (8e6, 0.0)), ("sigmoid", (1.0, 0.0))):
        y = linear(x, w, act=act, out_dtype=torch.float32)[0]
        assert abs(float(y[0]) / want[0] - 1) < 1e-2 and abs(float(y[1])) == want[1]


def test_same_bits_every_time_and_alone_or_in_a_batch():
    """No atomics: a call repeats its bits; a token's result at the same tile shape does not depend
    on its neighbours."""
    gen = torch.Generator().manual_seed(4)
    x, w = rows(16, 4096, gen, torch.bfloat16), rows(2048, 4096, gen, torch.bfloat16)
    y = linear(x, w, out_dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(linear(x, w, out_dtype=torch.float32), y)
    assert torch.equal(linear(x[3:4], w, out_dtype=torch.float32), y[3:4])


@pytest.mark.parametrize("m,n", [(1, 2048), (1, 12288), (50, 20000), (100, 12288), (200, 4096),
                                 (900, 5003), (2048, 2048)])
def test_long_sums_keep_fp32(m, n):
    """The matrix unit cuts its running sum off, so one accumulator's relative error grows with K in
    proportion. Partial sums of 256 elements, added rounded, do not: each keeps the relative error
    that it has alone, so the whole has that of K = 256, a quarter more for the draw of the inputs,
    and roundings: log2 of the partial sums' number, each by 2^-24 at most in the L2 norm of values
    whose running sum stays below the final one's size, 8 of them for K up to 65536."""
    def error(k):
        gen = torch.Generator().manual_seed(k)
        x, w = rows(m, k, gen, torch.bfloat16), rows(n, k, gen, torch.bfloat16, scale=k ** -0.5)
        ref = reference(x, w)[0]
        return float((linear(x, w, out_dtype=torch.float32).double() - ref).norm() / ref.norm())

    short = max(error(256), error(512))
    for k in (1024, 2048, 4104, 8192):
        e = error(k)
        assert e <= 1.25 * short + 8 * 2.0 ** -24, f"K = {k}: {e:.2e}, K = 256: {short:.2e}"
    assert device_status() == 0


def test_streams_graph_and_chains():
    """Chained products (each reading what the one before wrote), eager, on a side stream and
    replayed from a graph."""
    gen = torch.Generator().manual_seed(6)
    for m in (1, 64, 700):
        w = [rows(512, 512, gen, torch.bfloat16, scale=512 ** -0.5) for _ in range(4)]
        x = rows(m, 512, gen, torch.bfloat16)
        bufs = [torch.empty((m, 512), dtype=torch.bfloat16, device="cuda") for _ in range(4)]

        def chain():
            h = x
            for i in range(4):
                h = linear(h, w[i], act="silu", residual=h, out=bufs[i])

        chain()
        want = [b.clone() for b in bufs]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for b in bufs:
                b.zero_()
            chain()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(bufs, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain()
        for _ in range(2):
            for b in bufs:
                b.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(bufs, want))
        x.copy_(-x)
        graph.replay()
        replayed = [b.clone() for b in bufs]
        chain()
        assert all(torch.equal(a, b) for a, b in zip(bufs, replayed))
    assert device_status() == 0


def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((32, 64), dtype=torch.bfloat16, device="cuda")
    assert linear(x[:0], w).shape == (0, 32)
    bad = [dict(x=x.half()), dict(x=x[:, :32]), dict(w=w.cpu()),
           dict(x=torch.zeros((64, 4), dtype=torch.bfloat16, device="cuda").t()),
           dict(out=torch.zeros((4, 31), device="cuda")), dict(bias=torch.zeros(32)),
           dict(bias=torch.zeros(32, dtype=torch.bfloat16, device="cuda")),
           dict(residual=torch.zeros((3, 32), device="cuda")),
           dict(out=torch.zeros((4, 32), device="cuda"), out_dtype=torch.bfloat16)]
    for b in bad:
        a = dict(x=x, w=w)
        a.update(b)
        with pytest.raises(ValueError):
            linear(a.pop("x"), a.pop("w"), **a)
    with pytest.raises(KeyError):
        linear(x, w, act="relu6")

    def status(x, w, **kw):
        with pytest.raises(gdn.GdnError) as e:
            linear(x, w, **kw)
        return e.value.status

    wide = torch.zeros((4, 77), dtype=torch.bfloat16, device="cuda")
    assert status(wide[:, :64], w) == _lib.GDN_EINVAL                      # row stride 77
    assert status(torch.zeros((4, 80), dtype=torch.bfloat16, device="cuda")[:, 1:65],
                  w) == _lib.GDN_EALIGN
    assert status(x[:, :60], w[:, :60]) == _lib.GDN_EINVAL                 # K % 8
    assert status(x.float(), w.float()) == _lib.GDN_EINVAL
    assert status(x[:1].expand(4, 64), w) == _lib.GDN_EINVAL               # row stride 0
    assert status(x, w, residual=torch.zeros((1, 32), device="cuda").expand(4, 32)) == \
        _lib.GDN_EINVAL
    assert device_status() == 0


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in x and in out: the last rows are those of a small call."""
    m, k, n = 2 ** 20 + 40, 2048, 2049
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(5)
    w = rows(n, k, gen, torch.bfloat16, scale=k ** -0.5)
    x[-300:] = rows(300, k, gen, torch.bfloat16)
    out = linear(x, w)
    check(out[-300:], *reference(x[-300:], w), k, "torch.bfloat16 last rows")
    assert not out[: m - 300].any()
    assert device_status() == 0
