"""Rotary positions against the formula in 64 bits (GPU).

Tolerance: one rounding to bf16 (2^-8 relative), and 32-bit sine, cosine and products
(each off by less than 2^-20 absolute) on the two members of the pair."""
import math

import pytest
import torch

from nf4_layer_streamed_b200 import api
from tests.test_rope_table import BANDED, YARN, frequencies

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rotate(x, heads, d, rot, inter, pos, freqs, m, sign):
    """(rotated, sum of magnitudes of what each output adds up) in float64."""
    ang = pos.double()[:, None] * torch.from_numpy(freqs).to(DEV)
    c, s = (ang.cos() * m)[:, None], (sign * ang.sin() * m)[:, None]
    x = x.double().reshape(-1, heads, d)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, mag = x.clone(), torch.zeros_like(x)
    ya, yb, t = a * c - b * s, b * c + a * s, (a.abs() + b.abs()) * m
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = ya, yb
        mag[..., 0:rot:2] = mag[..., 1:rot:2] = t
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ya, yb
        mag[..., :rot // 2] = mag[..., rot // 2:rot] = t
    return y.flatten(1), mag.flatten(1)


def check(got, x, heads, d, rot, inter, pos, freqs, m, sign):
    want, mag = rotate(x, heads, d, rot, inter, pos, freqs, m, sign)
    assert ((got.double() - want).abs() - 2.0 ** -8 * want.abs() - 2.0 ** -19 * mag).max().item() <= 0.0


@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("rows,n_q,n_kv,d,rot,scaling", [
    (1, 9, 3, 64, 64, None), (255, 9, 3, 64, 32, {"kind": "linear", "factor": 4.0}), (33, 32, 8, 128, 128, BANDED),
    (1000, 5, 1, 128, 64, YARN), (7, 1, 1, 16, 16, None), (20000, 2, 1, 96, 48, None), (3, 3, 3, 512, 272, YARN)])
def test_rotation_both_ways(rows, n_q, n_kv, d, rot, scaling, inter):
    g = torch.Generator(device=DEV).manual_seed(rows + d)
    buf = torch.randn(rows, (n_q + 2 * n_kv) * d + 8, generator=g, device=DEV).to(torch.bfloat16)
    q, k = buf[:, :n_q * d], buf[:, n_q * d:(n_q + n_kv) * d]
    pos = torch.randint(-1000, 1 << 20, (rows,), generator=g, device=DEV).to(torch.int32)
    freqs, m = frequencies(rot, 500000.0, scaling)
    rope = api.Rope(d, 500000.0, rot_dim=rot, interleaved=inter, scaling=scaling)
    for inverse in (False, True):
        qo, ko = api.rope_apply(rope, pos, q, k, n_q, n_kv, inverse=inverse)
        sign = -1.0 if inverse else 1.0
        check(qo, q, n_q, d, rot, inter, pos, freqs, m, sign)
        check(ko, k, n_kv, d, rot, inter, pos, freqs, m, sign)
    # in place, and the neighbouring columns stay
    keep = buf.clone()
    api.rope_apply(rope, pos, q, k, n_q, n_kv, inverse=True, out=(q, k))
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(buf[:, (n_q + n_kv) * d:], keep[:, (n_q + n_kv) * d:])


def test_far_and_negative_positions_and_rows_behind():
    n_q, n_kv, d = 4, 2, 64
    pos = torch.tensor([0, 1, -1, 2**31 - 1, -2**31, 10**9, 131071], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(9, n_q * d, generator=g, device=DEV).to(torch.bfloat16)
    k = torch.randn(9, n_kv * d, generator=g, device=DEV).to(torch.bfloat16)
    rope = api.Rope(d, 10000.0)
    freqs, m = frequencies(d, 10000.0, None)
    out = (torch.full_like(q, 7.0), torch.full_like(k, 7.0))
    api.rope_apply(rope, pos, q, k, n_q, n_kv, out=out)
    # the float64 reference itself is off by 2^31 2^-53 radians at the farthest positions
    check(out[0][:7], q[:7], n_q, d, d, False, pos, freqs, m, 1.0)
    check(out[1][:7], k[:7], n_kv, d, d, False, pos, freqs, m, 1.0)
    assert torch.equal(out[0][0], q[0]) and (out[0][7:] == 7.0).all() and (out[1][7:] == 7.0).all()
    none = api.rope_apply(rope, pos[:0], q, k, n_q, n_kv)
    assert none[0].shape == (0, n_q * d)


def test_gradient_is_the_transpose():
    """<R x, y> = <x, R^T y> for the bf16 outputs, to the roundings of both sides."""
    rows, n_q, n_kv, d = 64, 2, 2, 128
    g = torch.Generator(device=DEV).manual_seed(2)
    x, y = (torch.randn(rows, n_q * d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    pos = torch.arange(rows, dtype=torch.int32, device=DEV) + 70000
    for inter in (False, True):
        rope = api.Rope(d, 500000.0, rot_dim=96, interleaved=inter, scaling=YARN)
        fx = api.rope_apply(rope, pos, x, x, n_q, n_kv)[0].double()
        ty = api.rope_apply(rope, pos, y, y, n_q, n_kv, inverse=True)[0].double()
        a, b = (fx * y.double()).sum(1), (x.double() * ty).sum(1)
        bound = 2.0 ** -8 * ((fx * y.double()).abs().sum(1) + (x.double() * ty).abs().sum(1))
        assert ((a - b).abs() <= bound * 1.01).all()


def test_stream_and_graph():
    rows, n_q, n_kv, d = 300, 8, 2, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn(rows, n_q * d, generator=g, device=DEV).to(torch.bfloat16)
    k = torch.randn(rows, n_kv * d, generator=g, device=DEV).to(torch.bfloat16)
    pos = torch.arange(rows, dtype=torch.int32, device=DEV)
    rope = api.Rope(d, 10000.0)
    want = api.rope_apply(rope, pos, q, k, n_q, n_kv)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = api.rope_apply(rope, pos, q, k, n_q, n_kv, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.rope_apply(rope, pos, q, k, n_q, n_kv)
    q.copy_(q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], api.rope_apply(rope, pos, q, k, n_q, n_kv)[0])
