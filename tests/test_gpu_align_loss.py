"""Preference and policy losses against their formulas in 64 bits (GPU).

Tolerances: an exponential is off by at most |x - max| 2^-23 + 2^-22 of itself; those that
carry the sum lie within 24 nats of the maximum (the rest adds less than e^-24 V < 1e-5 of
... their own error), so a sum of them is off by less than 24 2^-23 + 2^-22 = 3.1e-6, and
its 32-bit additions (at most 64 in a chain) by 64 2^-24 = 3.8e-6: LP = 7e-6 nats on a
log probability.  The gradient is rounded once to bf16 (2^-8)."""
import math

import pytest
import torch
import torch.nn.functional as F

from nf4_layer_streamed_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
LP = 7e-6
R = 2.0 ** -8


def make(rows, vocab, seed=0, ld=None, offset=0, std=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed + rows + vocab)
    ld = vocab + offset if ld is None else ld
    buf = torch.full((rows, ld), math.nan, dtype=torch.bfloat16, device=DEV)
    x = buf[:, offset:offset + vocab]
    x.copy_((torch.randn(rows, vocab, generator=g, device=DEV) * std).to(torch.bfloat16))
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV).to(torch.int32)
    t[::5] = -1
    if rows > 3:
        t[1], t[2], t[3] = vocab, 0, vocab - 1      # outside the vocabulary; its first and last token
    return x, t, g


def logp64(x, t, vocab):
    has = (t >= 0) & (t < vocab)
    lp = torch.log_softmax(x.double(), 1).gather(1, t.clamp(0, vocab - 1).long()[:, None])[:, 0]
    return torch.where(has, lp, torch.zeros_like(lp)), has


def grad64(x, t, has, c):
    g = -torch.softmax(x.double(), 1)
    g.scatter_add_(1, t.clamp(0, x.shape[1] - 1).long()[:, None], torch.ones(len(t), 1, dtype=torch.float64, device=DEV))
    return torch.where(has[:, None], g * c[:, None], torch.zeros_like(g))


def check_grad(got, x, t, has, c, dc):
    """dc: how far the coefficient of each row may be off."""
    assert (got[~has] == 0).all()
    got, x, t, c, dc, has = got[has], x[has], t[has], c[has], dc[has], has[has]
    want = grad64(x, t, has, c)
    p = torch.softmax(x.double(), 1)
    hot = torch.zeros_like(p).scatter_(1, t.clamp(0, x.shape[1] - 1).long()[:, None], 1.0)
    # p is off by the error of its exponent, |x - max - log sum| 2^-23 nats and 2^-22, and by LP from the sum
    rel = (-p.clamp(min=1e-300).log()).clamp(max=100) * 2.0 ** -23 + 2.0 ** -22 + LP
    tol = R * want.abs() + c.abs()[:, None] * p * rel + dc[:, None] * (p + hot) + 1e-38
    off = ((got.double() - want).abs() / tol).max().item()
    assert off <= 1.0


VOCABS = [1, 7, 64, 1000, 49152, 50257, 128256, 262147]


@pytest.mark.parametrize("kind,eps", [("sigmoid", 0.0), ("sigmoid", 0.1), ("hinge", 0.0), ("squared", 0.0)])
@pytest.mark.parametrize("vocab", VOCABS)
def test_preference(vocab, kind, eps):
    lengths = [5, 17, 1, 0, 40, 12]
    n = sum(lengths)
    x, t, g = make(n, vocab, offset=vocab % 3)
    pack = api.PackedRows(lengths)
    beta = 0.1
    lp, has = logp64(x, t, vocab)
    lp.requires_grad_(True)
    total = torch.stack([lp[pack.cu[i]:pack.cu[i + 1]].sum() for i in range(6)])
    ref = (total.detach() + 5.0 * torch.randn(6, generator=g, device=DEV, dtype=torch.float64)).float()
    gap = (total[0::2] - total[1::2]) - (ref[0::2].double() - ref[1::2].double())
    h = beta * gap
    if kind == "sigmoid":
        loss = -((1 - eps) * F.logsigmoid(h) + eps * F.logsigmoid(-h)).mean()
    elif kind == "hinge":
        loss = torch.relu(1 - h).mean()
    else:
        loss = ((gap - 1 / (2 * beta)) ** 2).mean()
    loss.backward()
    f = api.preference_loss_fwd(pack, x, t, ref, beta, kind=kind, label_smoothing=eps)
    assert ((f.logp.double() - lp).abs() <= LP + 2.0 ** -24 * lp.abs()).all()
    seq_err = LP * torch.tensor(lengths, device=DEV) + 2.0 ** -24 * total.abs()
    assert ((f.seq_logp.double() - total).abs() <= seq_err).all()
    gap_err = LP * torch.tensor([22.0, 1.0, 52.0], device=DEV, dtype=torch.float64)
    assert ((f.margin.double() - h).abs() <= beta * gap_err + 2.0 ** -22 * h.abs()).all()
    slope = 1.0 if kind != "squared" else (2 * (gap - 1 / (2 * beta)).abs().max().item() + 1e-3) / beta
    assert abs(f.loss.item() - loss.item()) <= slope * beta * gap_err.max().item() + 2.0 ** -22 * abs(loss.item())
    second = {"sigmoid": beta * beta / 4, "hinge": 0.0, "squared": 2.0}[kind]  # bound of the loss's second derivative
    dc = (second * gap_err / 3).repeat_interleave(2)[pack.seq.long()] + 2.0 ** -22 * lp.grad.abs()
    d = api.preference_loss_bwd(pack, x, t, f)
    check_grad(d, x, t, has, lp.grad, dc)
    half = api.preference_loss_bwd(pack, x, t, f, grad_scale=0.5)
    assert torch.equal(half.float(), d.float() * 0.5) or half.float().abs().min() < 1e-37
    inplace = x.clone() if vocab % 3 == 0 else torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=DEV).copy_(x)
    api.preference_loss_bwd(pack, inplace, t, f, out=inplace)
    assert torch.equal(inplace, d)


@pytest.mark.parametrize("kind", ["hinge", "squared"])
def test_smoothing_is_the_sigmoid_losss(kind):
    lengths = [5, 7, 2, 1]
    x, t, g = make(sum(lengths), 999, seed=4)
    pack, ref = api.PackedRows(lengths), torch.randn(4, generator=g, device=DEV)
    outs = []
    for eps in (0.0, 0.1):
        f = api.preference_loss_fwd(pack, x, t, ref, 0.1, kind=kind, label_smoothing=eps)
        outs.append((f.loss, f.margin, f.coef, api.preference_loss_bwd(pack, x, t, f)))
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and outs[0][2].abs().max() > 0


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("kl", [0.0, 0.05])
def test_policy(vocab, kl):
    policy(61, vocab, kl, vocab + 9, 1)


@pytest.mark.parametrize("vocab", [24575, 49152, 106496, 110003])
def test_policy_of_many_long_rows(vocab):
    """More rows than blocks fit on the GPU at once, of lengths that take each kind of block."""
    policy(701, vocab, 0.05, vocab + 8 + -vocab % 8, 0)


def policy(n, vocab, kl, ld, offset):
    x, t, g = make(n, vocab, seed=1, ld=ld, offset=offset)
    lp, has = logp64(x, t, vocab)
    r = lambda s: torch.randn(n, generator=g, device=DEV) * s  # noqa: E731
    old, ref, adv = (lp.detach() + 0.3 * r(1.0)).float(), (lp.detach() + r(0.5)).float(), r(1.0)
    w = torch.rand(n, generator=g, device=DEV) / n
    low, high = 0.2, 0.28
    # rows where the clip decides within the error of r are moved off the border
    ratio = (lp - old.double()).exp()
    near = ((ratio - (1 - low)).abs() < 1e-4) | ((ratio - (1 + high)).abs() < 1e-4)
    old[near] += 0.01
    lp.requires_grad_(True)
    ratio = (lp - old.double()).exp()
    best = torch.minimum(ratio * adv.double(), ratio.clamp(1 - low, 1 + high) * adv.double())
    gap = ref.double() - lp
    each = torch.where(has, w.double() * (kl * (gap.exp() - gap - 1) - best), 0.0)
    each.sum().backward()
    args = (x, t, old, ref if kl else None, adv, w, low, high, kl)
    loss, logp, d = api.policy_loss(*args)
    err = w.double() * ((LP + 2.0 ** -21) * (ratio * adv.double()).abs() + kl * ((gap.exp() - 1).abs() * LP + 2.0 ** -21 * (gap.exp() + gap.abs())))
    assert ((logp.double() - lp).abs() <= LP + 2.0 ** -24 * lp.abs()).all()
    assert abs(loss.item() - each.sum().item()) <= err[has].sum().item() + 2.0 ** -23 * abs(each.sum().item())
    dc = w.double() * ((LP + 2.0 ** -21) * (ratio * adv.double()).abs() + kl * (gap.exp() * LP + 2.0 ** -21 * (gap.exp() + 1)))
    check_grad(d, x, t, has, lp.grad, dc.detach())
    again = api.policy_loss(*args)
    assert torch.equal(again[0], loss) and torch.equal(again[2], d)
    only = api.policy_loss(*args, grad=False)
    assert only[2] is None and torch.equal(only[0], loss) and torch.equal(only[1], logp)
    api.policy_loss(*args, out=x)                        # in place
    assert torch.equal(x, d)


def test_policy_gradient_against_differences():
    n, vocab = 6, 40
    x, t, g = make(n, vocab, seed=4)
    t[:] = torch.arange(n, device=DEV)
    lp, _ = logp64(x, t, vocab)
    old, ref = (lp + 0.05).float(), (lp - 0.2).float()
    adv, w = torch.linspace(-1, 1, n, device=DEV), torch.full((n,), 1.0 / n, device=DEV)
    d = api.policy_loss(x, t, old, ref, adv, w, 0.2, 0.2, 0.1)[2].double()

    def loss(y):
        p = torch.log_softmax(y, 1).gather(1, t.long()[:, None])[:, 0]
        r, gap = (p - old.double()).exp(), ref.double() - p
        return (w * (0.1 * (gap.exp() - gap - 1) - torch.minimum(r * adv, r.clamp(0.8, 1.2) * adv))).sum().item()
    for i in range(n):
        for j in (i, 7, 39):
            y = x.double()
            y[i, j] += 1e-5
            up = loss(y)
            y[i, j] -= 2e-5
            diff = (up - loss(y)) / 2e-5
            assert abs(d[i, j].item() - diff) <= R * abs(diff) + 1e-8


def test_masked_tokens_lowest_values_and_non_finite_rows():
    vocab, lengths = 1003, [4, 4]
    x, t, _ = make(8, vocab)
    t[:] = torch.tensor([3, 4, 5, 6, -1, 8, 9, -1], device=DEV)
    low = torch.finfo(torch.bfloat16).min
    x[0, 10:] = -math.inf               # masked tokens
    x[1, :] = low                       # nothing but the lowest value: uniform
    x[2, 20:] = low
    x[3, :] = -math.inf
    x[3, 6] = 2.0                       # one token left: probability 1
    x[4] = math.nan                     # a row without a target
    x[7] = math.inf
    pack = api.PackedRows(lengths)
    ref = torch.zeros(2, device=DEV)
    f = api.preference_loss_fwd(pack, x, t, ref, 0.1)
    lp, has = logp64(x, t, vocab)
    assert ((f.logp.double() - lp).abs() <= LP + 2.0 ** -24 * lp.abs()).all()
    assert f.logp[3] == 0.0 and abs(f.logp[1].item() + math.log(vocab)) < 2e-6
    d = api.preference_loss_bwd(pack, x, t, f)
    assert torch.isfinite(d).all() and (d[4] == 0).all() and (d[7] == 0).all()
    c = f.coef.double()[pack.seq.long()]
    check_grad(d, x, t, has, c, 2.0 ** -22 * c.abs())
    # a row that is not finite spoils its own gradient and its pair's, not another pair's
    lengths2 = [4, 4, 4, 4]
    x2, t2 = torch.cat((x, x)), torch.cat((t, t))
    x2[0, 5] = math.nan
    pack2 = api.PackedRows(lengths2)
    f2 = api.preference_loss_fwd(pack2, x2, t2, torch.zeros(4, device=DEV), 0.1)
    assert torch.isnan(f2.loss) and torch.isnan(f2.margin[0]) and torch.equal(f2.margin[1:], f.margin)
    d2 = api.preference_loss_bwd(pack2, x2, t2, f2)
    assert torch.equal(d2[8:].float(), d.float() * 0.5)


def test_extreme_margins_and_ratios():
    vocab = 100
    x, t, _ = make(2, vocab)
    t[:] = 1
    pack = api.PackedRows([1, 1])
    lp, _ = logp64(x, t, vocab)
    for far in (1e4, -1e4, 1e30):
        ref = torch.stack((lp[0] - far, lp[1])).float()
        f = api.preference_loss_fwd(pack, x, t, ref, 0.1)
        h = 0.1 * ((lp[0] - lp[1]) - (ref[0].double() - ref[1].double()))
        assert abs(f.loss.item() + F.logsigmoid(h).item()) <= 1e-5 * abs(h.item())
        assert torch.isfinite(api.preference_loss_bwd(pack, x, t, f)).all()
    old = (lp - torch.tensor([500.0, -500.0], device=DEV)).float()   # r overflows to inf, and to 0
    one = torch.ones(2, device=DEV)
    loss, _, d = api.policy_loss(x, t, old, None, one, one, 0.2, 0.2)
    assert loss.item() == pytest.approx(-1.2) and (d == 0).all()      # clipped; 0 x its gradient
    loss, _, d = api.policy_loss(x, t, old, None, one * 0, one, 0.2, 0.2)
    assert loss.item() == 0.0 and (d == 0).all()


def test_rows_behind_and_no_rows():
    x, t, _ = make(9, 333)
    t = t[:7].contiguous()
    pack = api.PackedRows([3, 4])
    f = api.preference_loss_fwd(pack, x, t, torch.zeros(2, device=DEV), 0.1)
    out = torch.full((9, 333), 7.0, dtype=torch.bfloat16, device=DEV)
    api.preference_loss_bwd(pack, x, t, f, out=out)
    assert (out[7:] == 7.0).all() and (out[:7].float().abs() < 1).all()
    r = torch.ones(7, device=DEV)
    out.fill_(7.0)
    api.policy_loss(x, t, r, None, r, r, 0.2, 0.2, out=out)
    assert (out[7:] == 7.0).all()
    empty = api.PackedRows([0, 0])
    f = api.preference_loss_fwd(empty, x[:0], t[:0], torch.tensor([1.0, 3.0], device=DEV), 0.5)
    assert f.loss.item() == pytest.approx(math.log1p(math.exp(-1.0)), rel=1e-6) and f.margin.item() == 1.0
    assert api.preference_loss_bwd(empty, x[:0], t[:0], f).shape == (0, 333)
    loss, logp, d = api.policy_loss(x[:0], t[:0], r[:0], None, r[:0], r[:0], 0.2, 0.2)
    assert loss.item() == 0.0 and logp.shape == (0,) and d.shape == (0, 333)


def test_streams_and_graphs():
    x, t, _ = make(40, 5000)
    pack = api.PackedRows([9, 11, 13, 7])
    ref, r = torch.zeros(4, device=DEV), torch.ones(40, device=DEV)

    def both(stream=None):
        f = api.preference_loss_fwd(pack, x, t, ref, 0.1, stream=stream)
        return (f.loss, f.logp, api.preference_loss_bwd(pack, x, t, f, stream=stream)) + \
            api.policy_loss(x, t, r, r, r, r, 0.2, 0.2, 0.1, stream=stream)
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
    x.copy_(x.flip(1))
    want = both()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_row_offsets_beyond_32_bits():
    rows, vocab, ld = 34000, 1000, 1 << 17     # the last rows start over 2^32 elements into the buffer
    buf = torch.empty(rows, ld, dtype=torch.bfloat16, device=DEV)
    x = buf[:, 8:8 + vocab]
    g = torch.Generator(device=DEV).manual_seed(1)
    x.copy_(torch.randn(rows, vocab, generator=g, device=DEV).to(torch.bfloat16))
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV).to(torch.int32)
    pack = api.PackedRows([17000, 17000])
    tail = slice(rows - 50, rows)
    keep = x[tail].clone()
    lp, has = logp64(keep, t[tail], vocab)
    f = api.preference_loss_fwd(pack, x, t, torch.zeros(2, device=DEV), 1e-4)
    assert ((f.logp[tail].double() - lp).abs() <= LP + 2.0 ** -24 * lp.abs()).all()
    api.preference_loss_bwd(pack, x, t, f, out=x)
    c = f.coef.double()[1].expand(50)
    check_grad(x[tail], keep, t[tail], has, c, 2.0 ** -22 * c.abs())


@pytest.mark.parametrize("vocab", [1003, 49152, 128256])
@pytest.mark.parametrize("kl", [0.0, 0.05])
def test_policy_rows_that_are_not_finite(vocab, kl):
    """NaN and +inf in a row's logits, or a NaN advantage, make the row's gradient NaN, not zero."""
    x, t, g = make(8, vocab, seed=6)
    t[:] = torch.tensor([3, 4, 5, 6, 7, 8, -1, 9], device=DEV)
    lp, _ = logp64(x, t, vocab)
    old, ref, adv, w = (lp + 0.1).float(), (lp - 0.2).float(), torch.linspace(-1, 1, 8, device=DEV), torch.full((8,), 0.125, device=DEV)
    args = (old, ref if kl else None)
    _, logp0, d0 = api.policy_loss(x, t, *args, adv, w, 0.2, 0.2, kl)
    bad, adv1 = x.clone(), adv.clone()
    bad[1, 50] = math.nan
    bad[2, 60] = math.inf
    bad[3, 6] = math.nan                # the target's
    bad[6] = math.nan                   # a row without a target
    adv1[4] = math.nan
    for inplace in (False, True):
        loss, logp, d = api.policy_loss(bad, t, *args, adv1, w, 0.2, 0.2, kl, out=bad if inplace else None)
        assert torch.isnan(loss).all()
        assert torch.isnan(logp[1:4]).all() and torch.equal(logp[[0, 4, 5, 7]], logp0[[0, 4, 5, 7]])
        assert torch.isnan(d[1:5]).all()
        assert (d[6] == 0).all() and torch.equal(d[[0, 5, 7]], d0[[0, 5, 7]])


@pytest.mark.parametrize("eps", [0.0, 0.1])
def test_pairs_with_a_sequence_of_probability_zero(eps):
    """A target whose logit is -inf: the margin is infinite.  Where the rejected sequence has it, the pair's loss is
    0 without smoothing (not 0 x inf) and its gradient 0; where the preferred one has it, the loss is infinite."""
    vocab, lengths, beta = 1003, [3, 4, 2, 5], 0.1
    x, t, _ = make(14, vocab, seed=8)
    t[:] = torch.arange(20, 34, device=DEV)
    ref = torch.zeros(4, device=DEV)
    pack = api.PackedRows(lengths)
    f0 = api.preference_loss_fwd(pack, x, t, ref, beta, label_smoothing=eps)
    d0 = api.preference_loss_bwd(pack, x, t, f0)
    h = f0.margin[1].double()
    other = -((1 - eps) * F.logsigmoid(h) + eps * F.logsigmoid(-h)).item()
    for row, infinite in ((4, math.inf), (1, -math.inf)):
        y = x.clone()
        y[row, t[row].long()] = -math.inf
        f = api.preference_loss_fwd(pack, y, t, ref, beta, label_smoothing=eps)
        assert f.margin[0].item() == infinite and torch.equal(f.margin[1:], f0.margin[1:])
        # slope of the pair's loss: beta (eps sigmoid(h) - (1 - eps) sigmoid(-h)), halved by the mean
        c = beta * (eps if infinite > 0 else -(1 - eps)) / 2
        assert f.coef[0].item() == pytest.approx(c, rel=2.0 ** -22, abs=0) and f.coef[1].item() == -f.coef[0].item()
        if infinite > 0 and eps == 0.0:
            assert f.loss.item() == pytest.approx(other / 2, rel=2.0 ** -23 * (1 + abs(h.item())))  # h is rounded to fp32
        else:
            assert f.loss.item() == math.inf
        d = api.preference_loss_bwd(pack, y, t, f)
        assert torch.isfinite(d).all() and torch.equal(d[7:], d0[7:])
        if c == 0.0:
            assert (d[:7] == 0).all()
        has = torch.ones(7, dtype=torch.bool, device=DEV)
        coef = torch.tensor([c] * 3 + [-c] * 4, dtype=torch.float64, device=DEV)
        check_grad(d[:7], y[:7], t[:7], has, coef, 2.0 ** -22 * coef.abs())


def check_half(half, d, vocab):
    """Halving is exact in bf16, but for values at the end of its range."""
    big = d.float().abs() > 1e-30
    assert torch.equal(half.float()[big], 0.5 * d.float()[big])
    assert (half.float()[~big].abs() <= 1e-30).all()
    assert big.any() or vocab == 1


@pytest.mark.parametrize("vocab", VOCABS)
def test_grad_scale_scales_every_element(vocab):
    lengths = [5, 17, 1, 0, 40, 12]
    n = sum(lengths)
    x, t, g = make(n, vocab, seed=7, offset=vocab % 3)
    pack = api.PackedRows(lengths)
    r = torch.randn(n, generator=g, device=DEV)
    f = api.preference_loss_fwd(pack, x, t, torch.randn(6, generator=g, device=DEV), 0.1)
    check_half(api.preference_loss_bwd(pack, x, t, f, grad_scale=0.5), api.preference_loss_bwd(pack, x, t, f), vocab)
    args = (x, t, f.logp, f.logp + 0.1 * r, r, torch.full((n,), 0.1, device=DEV), 0.2, 0.2, 0.05)
    loss, logp, d = api.policy_loss(*args)
    half_loss, half_logp, half = api.policy_loss(*args, grad_scale=0.5)
    check_half(half, d, vocab)
    assert torch.equal(half_loss, loss) and torch.equal(half_logp, logp)


def test_captured_behind_other_kinds_of_work():
    """Launches that may begin early, captured behind a memset, a copy, a join of two streams, and first of all."""
    vocab, lengths = 5000, [9, 11, 13, 7]
    x, t, _ = make(40, vocab, seed=2)
    pack, none = api.PackedRows(lengths), api.PackedRows([0, 0])
    ref, r = torch.zeros(4, device=DEV), torch.ones(40, device=DEV)
    f = api.preference_loss_fwd(pack, x, t, ref, 0.1)
    want = api.preference_loss_bwd(pack, x, t, f)
    out, y, side = torch.empty_like(x), x.clone(), torch.cuda.Stream()
    gap = torch.tensor([1.0, 3.0], device=DEV)
    torch.cuda.synchronize()

    def memset():
        out.zero_()

    def copy():
        y.copy_(x)

    def join():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out.fill_(1.0)
        y.copy_(x)
        torch.cuda.current_stream().wait_stream(side)

    def nothing():
        pass
    for before in (memset, copy, join, nothing):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            before()
            api.preference_loss_bwd(pack, y, t, f, out=out)
            y2 = y.clone()
            empty = api.preference_loss_fwd(none, x[:0], t[:0], gap, 0.5)
            before()
            loss = api.policy_loss(x[:0], t[:0], r[:0], None, r[:0], r[:0], 0.2, 0.2)[0]
            full = api.policy_loss(y2, t, r, None, r, r, 0.2, 0.2)
            api.preference_loss_bwd(pack, y, t, f, out=out)
        for _ in range(2):
            y.zero_() if before in (copy, join) else None
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), before.__name__
            assert empty.loss.item() == pytest.approx(math.log1p(math.exp(-1.0)), rel=1e-6) and loss.item() == 0.0
            assert torch.isfinite(full[0]).all()
