"""Packed causal attention against the formula in 64 bits (GPU).

Tolerances: a probability and a score gradient are rounded once to bf16 for their
product (relative 2^-8 at most), an output once more; sums, statistics and exponentials
are 32-bit, whose share is bounded by 2^-13 of the sums of magnitudes (a score of d
products is off by at most (d + 2) 2^-24 of its magnitudes, which moves p by that much
in nats: below 6e-5 for N(0, 1) operands of 128 dims).
"""
import math

import pytest
import torch

from nf4_layer_streamed_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
R = 2.0 ** -8   # a rounding to bf16
F = 2.0 ** -13  # what 32-bit arithmetic adds, relative to sums of magnitudes

LENGTHS = [[1], [2, 1], [127], [128], [129], [1, 1, 1, 1], [0, 5, 0, 257, 1, 0], [640, 33, 255, 128], [16] * 40]
HEADS = [(9, 3, 64), (4, 1, 128), (2, 2, 128), (8, 1, 64), (3, 1, 128)]


def make(lengths, n_q, n_kv, d, seed=0, extra_rows=0):
    """q, k, v as column slices of one buffer whose rows behind the last sequence are NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed + sum(lengths) + n_q * d)
    total = sum(lengths)
    buf = torch.full((total + extra_rows, (n_q + 2 * n_kv) * d), math.nan, dtype=torch.bfloat16, device=DEV)
    buf[:total] = torch.randn(total, buf.shape[1], generator=g, device=DEV).to(torch.bfloat16)
    do = torch.randn(total, n_q * d, generator=g, device=DEV).to(torch.bfloat16)
    return buf[:, :n_q * d], buf[:, n_q * d:(n_q + n_kv) * d], buf[:, (n_q + n_kv) * d:], do


def reference(lengths, q, k, v, n_q, n_kv, d, scale):
    """(o, lse, bound of o) in float64."""
    o, lse, tol, a = [], [], [], 0
    for n in lengths:
        qh, kh, vh = heads64(q, k, v, a, n, n_q, n_kv, d)
        s = (qh @ kh.transpose(1, 2) * scale).masked_fill(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), -math.inf)
        p = torch.softmax(s, 2)
        out = p @ vh
        o.append(out.transpose(0, 1).flatten(1))
        lse.append(torch.logsumexp(s, 2))
        tol.append((((R + F) * (p @ vh.abs())) + R * out.abs()).transpose(0, 1).flatten(1))
        a += n
    return torch.cat(o), torch.cat(lse, 1), torch.cat(tol)


def heads64(q, k, v, a, n, n_q, n_kv, d):
    qh = q[a:a + n].double().reshape(n, n_q, d).transpose(0, 1)
    kh, vh = (x[a:a + n].double().reshape(n, n_kv, d).transpose(0, 1).repeat_interleave(n_q // n_kv, 0) for x in (k, v))
    return qh, kh, vh


def reference_grad(lengths, q, k, v, o, do, lse, n_q, n_kv, d, scale):
    """Gradients and their bounds in float64, from the given o and lse."""
    out, a = [], 0
    for n in lengths:
        qh, kh, vh = heads64(q, k, v, a, n, n_q, n_kv, d)
        oh, dh, _ = heads64(o, do, do, a, n, n_q, n_q, d)
        s = (qh @ kh.transpose(1, 2) * scale).masked_fill(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), -math.inf)
        p = torch.exp(s - lse[:, a:a + n, None].double())
        ds = p * (dh @ vh.transpose(1, 2) - (dh * oh).sum(2, keepdim=True))
        mag = p * (dh.abs() @ vh.abs().transpose(1, 2) + (dh * oh).abs().sum(2, keepdim=True))

        def shared(x):  # the query heads that share a key head
            return x.reshape(n_kv, n_q // n_kv, n, d).sum(1)
        dq, tq = scale * ds @ kh, scale * (R * ds.abs() + F * mag) @ kh.abs()
        dk, tk = shared(scale * ds.transpose(1, 2) @ qh), shared(scale * (R * ds.abs() + F * mag).transpose(1, 2) @ qh.abs())
        dv, tv = shared(p.transpose(1, 2) @ dh), shared((R + F) * p.transpose(1, 2) @ dh.abs())
        out.append([x.transpose(0, 1).flatten(1) for x in (dq, dk, dv, tq + R * dq.abs(), tk + R * dk.abs(), tv + R * dv.abs())])
        a += n
    return [torch.cat(x) for x in zip(*out)]


def within(got, want, tol, what):
    off = (got.double() - want).abs() - tol
    assert torch.isfinite(got).all() and off.max().item() <= 1e-7, (what, off.max().item())


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda n: "-".join(map(str, n[:7])))
def test_forward_and_gradients(lengths, heads):
    n_q, n_kv, d = heads
    q, k, v, do = make(lengths, n_q, n_kv, d, extra_rows=70)
    pack = api.PackedRows(lengths)
    scale = d ** -0.5
    o, lse = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d)
    want, wl, tol = reference(lengths, q, k, v, n_q, n_kv, d, scale)
    within(o, want, tol, "o")
    within(lse, wl, 6e-5 + 2.0 ** -22 * wl.abs(), "lse")
    got = api.packed_attention_bwd(pack, q, k, v, o, do, lse, n_q, n_kv, d)
    ref = reference_grad(lengths, q, k, v, o, do, lse, n_q, n_kv, d, scale)
    for name, g, w, t in zip(("dq", "dk", "dv"), got, ref[:3], ref[3:]):
        within(g, w, t, name)


def test_many_short_sequences_and_a_long_one():
    lengths = [1] * 700 + [2500] + [3] * 300
    n_q, n_kv, d = 4, 2, 64
    q, k, v, do = make(lengths, n_q, n_kv, d)
    pack = api.PackedRows(lengths)
    o, lse = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d)
    ones = [1] * 700
    torch.testing.assert_close(o[:700].reshape(700, n_kv, 2, d), v[:700].reshape(700, n_kv, 1, d).expand(-1, -1, 2, -1),
                               rtol=0, atol=0)  # one token: p = 1
    want, wl, tol = reference(lengths[700:], q[700:], k[700:], v[700:], n_q, n_kv, d, d ** -0.5)
    within(o[700:], want, tol, "o")
    within(lse[:, 700:], wl, 6e-5 + 2.0 ** -22 * wl.abs(), "lse")
    dq, dk, dv = api.packed_attention_bwd(pack, q, k, v, o, do, lse, n_q, n_kv, d)
    ref = reference_grad(ones + lengths[700:], q, k, v, o, do, lse, n_q, n_kv, d, d ** -0.5)
    for name, g, w, t in zip(("dq", "dk", "dv"), (dq, dk, dv), ref[:3], ref[3:]):
        within(g, w, t, name)


@pytest.mark.parametrize("heads", [(6, 2, 128), (5, 1, 64), (10, 5, 128)], ids=str)
def test_gradients_of_many_sequences(heads):
    """So many key tiles that each is one block's work, where a few are two blocks'."""
    n_q, n_kv, d = heads
    lengths = [129, 1, 200] * 24
    q, k, v, do = make(lengths, n_q, n_kv, d, extra_rows=3)
    pack = api.PackedRows(lengths)
    o, lse = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d)
    total = sum(lengths)
    buf = torch.full((total + 3, (n_q + 2 * n_kv) * d), 7.0, dtype=torch.bfloat16, device=DEV)
    outs = (buf[:, :n_q * d], buf[:, n_q * d:(n_q + n_kv) * d], buf[:, (n_q + n_kv) * d:])
    got = api.packed_attention_bwd(pack, q, k, v, o, do, lse, n_q, n_kv, d, out=outs)
    ref = reference_grad(lengths, q, k, v, o, do, lse, n_q, n_kv, d, d ** -0.5)
    for name, g, w, t in zip(("dq", "dk", "dv"), got, ref[:3], ref[3:]):
        within(g[:total], w, t, name)
    assert (buf[total:] == 7.0).all()
    g0 = buf.clone()
    rows = torch.ones(total + 3, dtype=torch.bool, device=DEV)
    rows[130:330] = False  # the third sequence, whose rows the tiles of the second one reach
    q1, k1, v1, do1 = (x.clone() for x in (q, k, v, do))
    for x in (q1, k1, v1, do1):
        x[130:330] = math.nan
    o1, l1 = api.packed_attention_fwd(pack, q1, k1, v1, n_q, n_kv, d)
    api.packed_attention_bwd(pack, q1, k1, v1, o1, do1, l1, n_q, n_kv, d, out=outs)
    assert torch.equal(buf[rows], g0[rows])
    # the same bits again, eagerly and from two captured calls in flight at once
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    got = [api.packed_attention_bwd(pack, q, k, v, o, do, lse, n_q, n_kv, d)]
    for g in graphs:
        with torch.cuda.graph(g):
            got.append(api.packed_attention_bwd(pack, q, k, v, o, do, lse, n_q, n_kv, d))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for grads in got:
        assert torch.equal(torch.cat(grads, 1), g0[:total])
    assert api.device_error()[0] == 0


@pytest.mark.parametrize("factor", [0.01, 30.0])
def test_flat_and_sharp_rows(factor):
    """Scores all alike, and scores of hundreds of nats that grow along the keys (the
    running maximum moves at almost every tile)."""
    lengths, n_q, n_kv, d = [700, 260], 2, 1, 64
    q, k, v, do = make(lengths, n_q, n_kv, d, seed=3)
    q, v = q.contiguous(), v.contiguous()
    ramp = torch.linspace(0.1, 1.0, sum(lengths), device=DEV)[:, None]
    q = (q.float().abs() * factor).to(torch.bfloat16)
    k = (k.float().abs() * ramp).to(torch.bfloat16)
    pack = api.PackedRows(lengths)
    o, lse = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d)
    want, wl, tol = reference(lengths, q, k, v, n_q, n_kv, d, d ** -0.5)
    # a score is off by (d + 2) 2^-24 of its magnitude, here up to hundreds of nats
    shift = (d + 2) * 2.0 ** -24 * wl.abs().max().item()
    within(o, want, tol * (1 + shift / R), "o")
    within(lse, wl, 6e-5 + shift + 2.0 ** -22 * wl.abs(), "lse")


def test_scale_argument_and_gradient_against_differences():
    lengths, n_q, n_kv, d, scale = [5, 131], 2, 1, 64, 0.3
    q, k, v, do = make(lengths, n_q, n_kv, d, seed=9)
    pack = api.PackedRows(lengths)
    o, lse = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d, scale=scale)
    grads = api.packed_attention_bwd(pack, q, k, v, o, do, lse, n_q, n_kv, d, scale=scale)
    x = [t.double().contiguous() for t in (q, k, v)]

    def loss(x):
        return (reference(lengths, *x, n_q, n_kv, d, scale)[0] * do.double()).sum().item()
    g = torch.Generator(device=DEV).manual_seed(1)
    for i in range(3):
        step = torch.randn(x[i].shape, generator=g, device=DEV, dtype=torch.float64)
        step /= step.norm()
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 1e-4 * step, x[i] - 1e-4 * step
        diff = (loss(up) - loss(down)) / 2e-4
        got = (grads[i].double() * step).sum().item()
        # o is rounded to bf16 before delta: every element of the gradient is off by about R of its size
        assert abs(got - diff) <= 4 * R * grads[i].double().norm().item() * 1.0, (i, got, diff)


def test_scores_below_the_range():
    """Keys of the type's lowest value, whose scores are -inf in fp32: they have no part in rows that
    see others too, also where they fill whole tiles."""
    lengths, n_q, n_kv, d, n = [300, 20], 4, 2, 64, 140
    q, k, v, do = make(lengths, n_q, n_kv, d)
    q, k = q.abs(), k.clone()
    k[:n] = torch.finfo(torch.bfloat16).min
    pack = api.PackedRows(lengths)
    o, lse = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d)
    assert (lse[:, :n] == -math.inf).all() and o[:n].isnan().all()
    qh, kh, vh = (x[n:300].double().reshape(300 - n, h, d).transpose(0, 1) for x, h in ((q, n_q), (k, n_kv), (v, n_kv)))
    kh, vh = kh.repeat_interleave(2, 0), vh.repeat_interleave(2, 0)
    s = (qh @ kh.transpose(1, 2) * d ** -0.5).masked_fill(torch.ones(300 - n, 300 - n, dtype=torch.bool, device=DEV).triu(1), -math.inf)
    p = torch.softmax(s, 2)
    want, mag = ((p @ x).transpose(0, 1).flatten(1) for x in (vh, vh.abs()))
    within(o[n:300], want, R * want.abs() + (R + F) * mag, "o")
    within(lse[:, n:300], torch.logsumexp(s, 2), 6e-5 + 2.0 ** -22 * torch.logsumexp(s, 2).abs(), "lse")
    alone, alone_lse = api.packed_attention_fwd(api.PackedRows([20]), q[300:], k[300:], v[300:], n_q, n_kv, d)
    assert torch.equal(o[300:320], alone) and torch.equal(lse[:, 300:], alone_lse)


def test_other_sequences_and_rows_behind_are_left_alone():
    lengths, n_q, n_kv, d = [200, 77, 130], 4, 2, 128
    q, k, v, do = make(lengths, n_q, n_kv, d, extra_rows=9)
    q, k, v = q.clone(), k.clone(), v.clone()
    pack = api.PackedRows(lengths)
    o0, l0 = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d)
    g0 = api.packed_attention_bwd(pack, q, k, v, o0, do, l0, n_q, n_kv, d)
    rows = torch.ones(sum(lengths), dtype=torch.bool, device=DEV)
    rows[200:277] = False
    for bad in (math.nan, math.inf, torch.finfo(torch.bfloat16).min):
        q1, k1, v1, do1 = (t.clone() for t in (q, k, v, do))
        for t in (q1, k1, v1, do1):
            t[200:277] = bad
        out = torch.full((sum(lengths) + 9, n_q * d), 7.0, dtype=torch.bfloat16, device=DEV)
        o1, l1 = api.packed_attention_fwd(pack, q1, k1, v1, n_q, n_kv, d, out=out)
        assert torch.equal(o1[:407][rows], o0[rows]) and torch.equal(l1[:, rows], l0[:, rows])
        assert (out[407:] == 7.0).all()
        o1 = torch.where(rows[:, None], o0, torch.full_like(o0, bad))
        l1 = torch.where(rows, l0, torch.full_like(l0, bad))
        buf = torch.full((sum(lengths) + 9, (n_q + 2 * n_kv) * d), 7.0, dtype=torch.bfloat16, device=DEV)
        outs = (buf[:, :n_q * d], buf[:, n_q * d:(n_q + n_kv) * d], buf[:, (n_q + n_kv) * d:])
        g1 = api.packed_attention_bwd(pack, q1, k1, v1, o1, do1, l1, n_q, n_kv, d, out=outs)
        for a, b in zip(g1, g0):
            assert torch.equal(a[:407][rows], b[rows])
        assert (buf[407:] == 7.0).all()


def test_no_rows():
    pack = api.PackedRows([0, 0])
    z = torch.zeros(4, 128, dtype=torch.bfloat16, device=DEV)
    o, lse = api.packed_attention_fwd(pack, z, z, z, 2, 2, 64)
    assert o.shape == (0, 128) and lse.shape == (2, 0)
    g = api.packed_attention_bwd(pack, z, z, z, o, o, lse, 2, 2, 64)
    assert all(x.shape == (0, 128) for x in g)


def test_deterministic_on_another_stream_and_in_a_graph():
    lengths, n_q, n_kv, d = [300, 1, 129, 514], 8, 2, 128
    q, k, v, do = make(lengths, n_q, n_kv, d)
    pack = api.PackedRows(lengths)

    def both(stream=None):
        o, lse = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d, stream=stream)
        return (o, lse) + api.packed_attention_bwd(pack, q, k, v, o, do, lse, n_q, n_kv, d, stream=stream)
    want = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both())
        graphs.append(g)
    # two captured steps in flight at once do not share a workspace
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    assert api.device_error()[0] == 0


def test_row_offsets_beyond_32_bits():
    """Rows 2^16 elements apart: the last ones start more than 2^31 elements into the buffer."""
    n_q, n_kv, d, ld = 2, 1, 64, 1 << 16
    lengths = [32760, 200, 1]
    total = sum(lengths)
    buf = torch.empty(total, ld, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    w = (n_q + 2 * n_kv) * d
    at = (0, ld // 2, ld - w)  # q, k, v spread over the row
    buf[:, :n_q * d] = torch.randn(total, n_q * d, generator=g, device=DEV).to(torch.bfloat16)
    for a in at[1:]:
        buf[:, a:a + n_kv * d] = torch.randn(total, n_kv * d, generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = buf[:, :n_q * d], buf[:, at[1]:at[1] + n_kv * d], buf[:, at[2]:at[2] + n_kv * d]
    pack = api.PackedRows(lengths)
    o, lse = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d, out=buf[:, 4096:4096 + n_q * d])
    tail = slice(32760, total)
    want, wl, tol = reference(lengths[1:], q[tail], k[tail], v[tail], n_q, n_kv, d, d ** -0.5)
    within(o[tail], want, tol, "o")
    do = torch.randn(total, n_q * d, generator=g, device=DEV).to(torch.bfloat16)
    outs = (buf[:, 8192:8192 + n_q * d], buf[:, 12288:12288 + n_kv * d], buf[:, 16384:16384 + n_kv * d])
    api.packed_attention_bwd(pack, q, k, v, o, do, lse, n_q, n_kv, d, out=outs)
    ref = reference_grad(lengths[1:], q[tail], k[tail], v[tail], o[tail], do[tail], lse[:, tail], n_q, n_kv, d, d ** -0.5)
    for name, x, w, t in zip(("dq", "dk", "dv"), outs, ref[:3], ref[3:]):
        within(x[tail], w, t, name)


@pytest.mark.parametrize("lengths,heads,scale", [
    ([300, 129, 1], (4, 1, 64), 0.3), ([300, 129, 1], (4, 1, 64), 0.03), ([512], (8, 2, 128), 0.13),
    ([129, 1, 200] * 24, (6, 2, 128), 0.13), ([129, 1, 200] * 24, (5, 1, 64), 0.3), ([257], (2, 2, 128), 0.02)], ids=str)
def test_scale_of_every_output(lengths, heads, scale):
    """Scales that are not 1 / sqrt(head_dim), element by element, where a key tile is two blocks' work and where
    it is one's.  A score is off by (d + 2) 2^-24 scale sum |q||k|: for N(0, 1) operands the sum is below
    1.5 x 0.64 d (d = 64) and 1.3 x 0.64 d (d = 128), so 7.2e-5 nats at 0.3 and 64 dims, 1.1e-4 at 0.13 and 128:
    within 2^-13, the share F that the bounds count."""
    n_q, n_kv, d = heads
    q, k, v, do = make(lengths, n_q, n_kv, d, seed=11)
    pack = api.PackedRows(lengths)
    o, lse = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d, scale=scale)
    want, wl, tol = reference(lengths, q, k, v, n_q, n_kv, d, scale)
    within(o, want, tol, "o")
    within(lse, wl, F + 2.0 ** -22 * wl.abs(), "lse")
    got = api.packed_attention_bwd(pack, q, k, v, o, do, lse, n_q, n_kv, d, scale=scale)
    ref = reference_grad(lengths, q, k, v, o, do, lse, n_q, n_kv, d, scale)
    for name, g, w, t in zip(("dq", "dk", "dv"), got, ref[:3], ref[3:]):
        within(g, w, t, name)
        # the bounds tell the scale: half of these gradients, or their opposite, lies outside them
        assert ((0.5 * w).abs() > t).any() and (w.abs() > t).any()


@pytest.mark.parametrize("copies", [1, 40])
def test_gradients_of_scores_below_the_range(copies):
    """Keys whose scores are -inf in fp32, single ones and a whole tile, in rows that see others too: the
    probabilities there are 0, and so is their share of every gradient."""
    lengths, n_q, n_kv, d = [300, 20] * copies, 4, 2, 64
    q, k, v, do = make(lengths, n_q, n_kv, d, seed=12)
    q, k = q.abs(), k.clone()
    low = torch.zeros(sum(lengths), dtype=torch.bool, device=DEV)
    for a in range(0, sum(lengths), 320):
        low[a + 5] = low[a + 310] = True
        low[a + 128:a + 256] = True
    k[low] = torch.finfo(torch.bfloat16).min
    pack = api.PackedRows(lengths)
    o, lse = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d)
    want, wl, tol = reference(lengths, q, k, v, n_q, n_kv, d, d ** -0.5)
    within(o, want, tol, "o")
    within(lse, wl, 6e-5 + 2.0 ** -22 * wl.abs(), "lse")
    dq, dk, dv = api.packed_attention_bwd(pack, q, k, v, o, do, lse, n_q, n_kv, d)
    ref = reference_grad(lengths, q, k, v, o, do, lse, n_q, n_kv, d, d ** -0.5)
    for name, g, w, t in zip(("dq", "dk", "dv"), (dq, dk, dv), ref[:3], ref[3:]):
        within(g, w, t, name)
    assert (dk[low] == 0).all() and (dv[low] == 0).all()


def test_gradients_of_rows_that_see_only_scores_below_the_range():
    """Rows that see nothing above -inf are NaN, in the forward and in their gradients; the rows and keys behind them
    and the next sequence are as if they were not there."""
    lengths, n_q, n_kv, d, n = [300, 20], 4, 2, 64, 140
    q, k, v, do = make(lengths, n_q, n_kv, d)
    q, k = q.abs(), k.clone()
    k[:n] = torch.finfo(torch.bfloat16).min
    pack = api.PackedRows(lengths)
    o, lse = api.packed_attention_fwd(pack, q, k, v, n_q, n_kv, d)
    got = api.packed_attention_bwd(pack, q, k, v, o, do, lse, n_q, n_kv, d)
    assert got[0][:n].isnan().all()
    cut = [x[n:] for x in (q, k, v, o, do)]
    ref = reference_grad([300 - n, 20], *cut, lse[:, n:], n_q, n_kv, d, d ** -0.5)
    for name, g, w, t in zip(("dq", "dk", "dv"), got, ref[:3], ref[3:]):
        within(g[n:], w, t, name)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [20, 36, 100])
def test_finite_scores_of_any_size(d, power):
    """Scores of up to 2^114 of either sign, exact in fp32 (a whole number times a power of 2 in every dim): the keys of
    a row's largest score share the probability and the others have none."""
    lengths, n_q, n_kv = [300, 1, 77], 4, 2
    n = sum(lengths)
    g = torch.Generator(device=DEV).manual_seed(power + d)
    c = torch.randint(-100, 101, (n, n_kv), generator=g, device=DEV)
    c[:40] = -c[:40].abs() - 1                            # rows that see nothing but scores far below 0
    q = torch.full((n, n_q * d), 2.0 ** (power // 2), dtype=torch.bfloat16, device=DEV)
    k = (c.double() * 2.0 ** (power - power // 2)).to(torch.bfloat16).repeat_interleave(d, 1)
    v = torch.randn(n, n_kv * d, generator=g, device=DEV).to(torch.bfloat16)
    o, lse = api.packed_attention_fwd(api.PackedRows(lengths), q, k, v, n_q, n_kv, d)
    want, wl, tol = reference(lengths, q, k, v, n_q, n_kv, d, d ** -0.5)
    within(o, want, tol, "o")
    # fp32: the scale and its product, the product with ln 2 and the result are rounded
    assert ((lse.double() - wl).abs() <= 2.0 ** -21 * wl.abs() + 6e-5).all()


def test_scores_that_grow_far_along_the_keys():
    """The maximum goes from ordinary scores to ones of 2^50 and on, tile by tile, and elsewhere falls from there."""
    n, n_q, n_kv, d = 640, 2, 1, 64
    g = torch.Generator(device=DEV).manual_seed(3)
    tile = torch.arange(n, device=DEV) // 128
    v = torch.randn(2 * n, n_kv * d, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.ones(2 * n, n_q * d, dtype=torch.bfloat16, device=DEV)
    size = 2.0 ** torch.tensor([-3.0, 4.0, 11.0, 50.0, 60.0], device=DEV)
    c = torch.randint(1, 101, (2, n), generator=g, device=DEV)
    k = torch.cat((size[tile] * c[0], size.flip(0)[tile] * c[1]))[:, None].expand(-1, d).to(torch.bfloat16)
    o, lse = api.packed_attention_fwd(api.PackedRows([n, n]), q, k, v, n_q, n_kv, d)
    want, wl, tol = reference([n, n], q, k, v, n_q, n_kv, d, d ** -0.5)
    within(o, want, tol, "o")
    assert ((lse.double() - wl).abs() <= 2.0 ** -21 * wl.abs() + 6e-5).all()
