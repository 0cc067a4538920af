"""A run of the packed operators together (GPU): rotary positions, attention, a head and
the preference loss, forward and backward, and the policy loss on the same logits, against
the whole chain in 64 bits without roundings.

Tolerance: every tensor between the operators is rounded to bf16 (2^-8 at most, 2^-9.8 in
the mean square), at most a dozen of them in a row on a gradient's way: 2e-2 of the
largest value, the bound that the layer's chain is held to."""
import math

import pytest
import torch

from nf4_layer_streamed_b200 import api
from tests.helpers import TOL, close
from tests.test_rope_table import BANDED, frequencies

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rotated(x, heads, d, pos, freqs):
    ang = pos.double()[:, None] * torch.from_numpy(freqs).to(DEV)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    x = x.reshape(-1, heads, d)
    a, b = x[..., :d // 2], x[..., d // 2:]
    return torch.cat((a * c - b * s, b * c + a * s), -1).flatten(1)


@pytest.mark.parametrize("n_q,n_kv,d,vocab", [(9, 3, 64, 4096), (8, 2, 128, 2048)])
def test_preference_step_over_packed_rows(n_q, n_kv, d, vocab):
    lengths = [150, 131, 64, 200, 17, 1]
    pack = api.PackedRows(lengths)
    n, qd, kvd = pack.total, n_q * d, n_kv * d
    g = torch.Generator(device=DEV).manual_seed(d)
    qkv = torch.randn(n, qd + 2 * kvd, generator=g, device=DEV).to(torch.bfloat16)
    head = (torch.randn(vocab, qd, generator=g, device=DEV) * 0.1).to(torch.bfloat16)
    targets = torch.randint(0, vocab, (n,), generator=g, device=DEV).to(torch.int32)
    targets[pack.cu[1:].long() - 1] = -1
    ref = torch.randn(6, generator=g, device=DEV)
    rope = api.Rope(d, 10000.0, scaling=BANDED)

    # the framework's calls
    q, k, v = qkv[:, :qd], qkv[:, qd:qd + kvd], qkv[:, qd + kvd:]
    rq, rk = api.rope_apply(rope, pack.positions, q, k, n_q, n_kv)
    o, lse = api.packed_attention_fwd(pack, rq, rk, v, n_q, n_kv, d)
    logits = api.gemm_bf16(o, head)
    f = api.preference_loss_fwd(pack, logits, targets, ref, 0.1)
    dlogits = api.preference_loss_bwd(pack, logits, targets, f)
    do = api.gemm_bf16(dlogits, head, b_trans=True)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = dqkv[:, :qd], dqkv[:, qd:qd + kvd], dqkv[:, qd + kvd:]
    api.packed_attention_bwd(pack, rq, rk, v, o, do, lse, n_q, n_kv, d, out=(dq, dk, dv))
    api.rope_apply(rope, pack.positions, dq, dk, n_q, n_kv, inverse=True, out=(dq, dk))

    # the chain in 64 bits
    x = qkv.double().requires_grad_(True)
    freqs, _ = frequencies(d, 10000.0, BANDED)
    xq, xk = rotated(x[:, :qd], n_q, d, pack.positions, freqs), rotated(x[:, qd:qd + kvd], n_kv, d, pack.positions, freqs)
    parts, a = [], 0
    for m in lengths:
        hq = xq[a:a + m].reshape(m, n_q, d).transpose(0, 1)
        hk, hv = (t[a:a + m].reshape(m, n_kv, d).transpose(0, 1).repeat_interleave(n_q // n_kv, 0)
                  for t in (xk, x[:, qd + kvd:]))
        s = (hq @ hk.transpose(1, 2) / math.sqrt(d)).masked_fill(torch.ones(m, m, dtype=torch.bool, device=DEV).triu(1),
                                                                  -math.inf)
        parts.append((torch.softmax(s, 2) @ hv).transpose(0, 1).flatten(1))
        a += m
    out = torch.cat(parts)
    z = out @ head.double().T
    lp = torch.log_softmax(z, 1).gather(1, targets.clamp(min=0).long()[:, None])[:, 0] * (targets >= 0)
    total = torch.stack([lp[pack.cu[i]:pack.cu[i + 1]].sum() for i in range(6)])
    r = ref.double()
    margin = 0.1 * ((total[0::2] - total[1::2]) - (r[0::2] - r[1::2]))
    loss = -torch.nn.functional.logsigmoid(margin).mean()
    loss.backward()
    close(o, out.detach().cpu().numpy(), TOL, "o")
    close(logits, z.detach().cpu().numpy(), TOL, "logits")
    assert abs(f.loss.item() - loss.item()) <= TOL * loss.item()
    for name, b, e in (("dq", 0, qd), ("dk", qd, qd + kvd), ("dv", qd + kvd, qd + 2 * kvd)):
        close(dqkv[:, b:e], x.grad[:, b:e].cpu().numpy(), TOL, name)

    # the policy loss over the same rows, its old model being this one
    w = torch.full((n,), 1.0 / n, device=DEV)
    adv = torch.randn(n, generator=g, device=DEV)
    pl, logp, pd = api.policy_loss(logits, targets, f.logp, None, adv, w, 0.2, 0.2)
    assert torch.equal(logp, f.logp)
    want = -(w * adv)[targets >= 0].double().sum().item()      # r = 1
    assert abs(pl.item() - want) <= 1e-5 * (w * adv.abs()).sum().item()
    zl = logits.double().requires_grad_(True)
    plp = torch.log_softmax(zl, 1).gather(1, targets.clamp(min=0).long()[:, None])[:, 0]
    (-(w * adv).double() * plp * (targets >= 0)).sum().backward()
    close(pd, zl.grad.cpu().numpy(), TOL, "policy gradient")


def test_captured_preference_step():
    """The run above as one graph: replayed on new inputs it gives the bits of the eager calls."""
    n_q, n_kv, d, vocab = 8, 2, 128, 2048
    lengths = [150, 131, 64, 200, 17, 1]
    pack = api.PackedRows(lengths)
    n, qd, kvd = pack.total, n_q * d, n_kv * d
    g = torch.Generator(device=DEV).manual_seed(2)
    qkv = torch.randn(n, qd + 2 * kvd, generator=g, device=DEV).to(torch.bfloat16)
    head = (torch.randn(vocab, qd, generator=g, device=DEV) * 0.1).to(torch.bfloat16)
    targets = torch.randint(0, vocab, (n,), generator=g, device=DEV).to(torch.int32)
    targets[pack.cu[1:].long() - 1] = -1
    ref, adv = torch.randn(6, generator=g, device=DEV), torch.randn(n, generator=g, device=DEV)
    w = torch.full((n,), 1.0 / n, device=DEV)
    rope = api.Rope(d, 10000.0, scaling=BANDED)

    def step():
        rq, rk = api.rope_apply(rope, pack.positions, qkv[:, :qd], qkv[:, qd:qd + kvd], n_q, n_kv)
        v = qkv[:, qd + kvd:]
        o, lse = api.packed_attention_fwd(pack, rq, rk, v, n_q, n_kv, d)
        logits = api.gemm_bf16(o, head)
        f = api.preference_loss_fwd(pack, logits, targets, ref, 0.1)
        dlogits = api.preference_loss_bwd(pack, logits, targets, f)
        do = api.gemm_bf16(dlogits, head, b_trans=True)
        dq, dk, dv = api.packed_attention_bwd(pack, rq, rk, v, o, do, lse, n_q, n_kv, d)
        dq, dk = api.rope_apply(rope, pack.positions, dq, dk, n_q, n_kv, inverse=True)
        return (f.loss, f.margin, f.logp, dq, dk, dv) + api.policy_loss(logits, targets, f.logp, None, adv, w, 0.2, 0.2)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(2):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device=DEV))
        want = [x.clone() for x in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)) and want[3].abs().max() > 0
    assert api.device_error()[0] == 0
