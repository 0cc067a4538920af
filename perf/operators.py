"""The operators of training on packed sequences, as a user's program calls them, beside
their plain forms: causal grouped-query attention over sequences of different lengths
that lie one behind the other (forward, and the gradients), rotary positions that start
again at every sequence (with frequencies scaled for long contexts, in both layouts, and
the transposed rotation of the backward pass), the preference loss over pairs of
sequences and the clipped policy loss with its KL term, each with the gradient of the
logits.

Where ``own`` is false, run() computes the plain form in elementary torch operations;
where it is true, it makes the framework's calls.
"""
import math

import torch

own = False
DEV = "cuda"

# (n_q, n_kv, head_dim, rope theta, vocab): the SmolLM2-shaped, Llama-8B-shaped and
# 32B-class layers of this repository's workloads.
SHAPES = {
    "smollm2": (9, 3, 64, 10000.0, 49152),
    "llama8b": (32, 8, 128, 500000.0, 128256),
    "32b": (40, 8, 128, 500000.0, 128256),
}

_ATTN_8B_BATCH = [512, 301, 129, 511, 77, 500, 17, 1]          # one 4 x 512 step's rows, packed
_ATTN_8B_LONG = [8192, 4111, 2048, 1333, 700, 14, 1]           # long documents with short ones between
_BWD_8B_LONG = [8192, 2047, 1200, 600, 129, 77, 1]
_SMALL = [37, 90, 128, 1]                                      # four short samples


def _lens(lengths):
    return ",".join(str(n) for n in lengths)


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def listed():
    return [
        # the smallest call: a handful of short samples on the smallest model; latency counts
        {"name": "attn_fwd_small", "op": "attn_fwd", "shape": "smollm2", "lengths": _lens(_SMALL)},
        # one layer of an ordinary fine-tuning step: 2048 rows of samples of all lengths
        {"name": "attn_fwd_8b", "op": "attn_fwd", "shape": "llama8b", "lengths": _lens(_ATTN_8B_BATCH)},
        # long-context training: an 8k document beside shorter ones
        {"name": "attn_fwd_8b_long", "op": "attn_fwd", "shape": "llama8b", "lengths": _lens(_ATTN_8B_LONG)},
        # the gradients of the same three kinds of batch
        {"name": "attn_bwd_small", "op": "attn_bwd", "shape": "smollm2", "lengths": _lens(_SMALL)},
        {"name": "attn_bwd_8b", "op": "attn_bwd", "shape": "llama8b", "lengths": _lens(_ATTN_8B_BATCH)},
        {"name": "attn_bwd_8b_long", "op": "attn_bwd", "shape": "llama8b", "lengths": _lens(_BWD_8B_LONG)},
        # rotation of the queries and keys of a small step: rotate-half pairs, no scaling
        {"name": "rope_fwd_small", "op": "rope_fwd", "shape": "smollm2", "lengths": _lens(_SMALL), "rot_dim": 64,
         "interleaved": False, "scaling": "none", "offset": 0},
        # the transposed rotation (backward pass) of a long batch: neighbouring pairs, half of each
        # head, frequencies scaled for contexts far beyond the trained one
        {"name": "rope_bwd_8b_long", "op": "rope_bwd", "shape": "llama8b", "lengths": _lens(_ATTN_8B_LONG),
         "rot_dim": 64, "interleaved": True, "scaling": "yarn", "offset": 100000},
        # two short preference pairs on the small vocabulary
        {"name": "pref_small", "op": "pref", "vocab": 49152, "lengths": "37,41,64,50", "kind": "sigmoid",
         "smoothing": 0.0, "beta": 0.1},
        # a full preference step of the large vocabulary: four pairs, 2048 rows
        {"name": "pref_8b", "op": "pref", "vocab": 128256, "lengths": "301,277,512,140,222,260,77,259",
         "kind": "sigmoid", "smoothing": 0.1, "beta": 0.1},
        # a short rollout on the small vocabulary
        {"name": "policy_small", "op": "policy", "vocab": 49152, "rows": 96, "masked": 0.25, "clip_low": 0.2,
         "clip_high": 0.2, "kl": 0.02},
        # a policy step on the large vocabulary, a third of the rows being prompt
        {"name": "policy_8b", "op": "policy", "vocab": 128256, "rows": 1999, "masked": 0.33, "clip_low": 0.2,
         "clip_high": 0.28, "kl": 0.05},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_lengths(rng, rows, longest):
    """Sequences of log-uniform length until `rows` rows are full (the last one ragged)."""
    out, left = [], rows
    while left > 0 and len(out) < 64:
        n = min(left, _log_int(rng, 1, longest))
        out.append(n)
        left -= n
    return out


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_bwd", "rope_fwd", "rope_bwd", "pref", "policy"])
    if op in ("attn_fwd", "attn_bwd"):
        shape = rng.choice(["smollm2", "llama8b", "32b"])
        lengths, most = None, sum(n * n for n in _ATTN_8B_LONG if n > 2048) * SHAPES["llama8b"][0] * 128
        if op == "attn_bwd":
            most = sum(n * n for n in _BWD_8B_LONG) * SHAPES["llama8b"][0] * 128
        while lengths is None or sum(n * n for n in lengths) * SHAPES[shape][0] * SHAPES[shape][2] > most:
            lengths = _draw_lengths(rng, _log_int(rng, 64, 16384), 8192)
        return {"op": op, "shape": shape, "lengths": _lens(lengths)}
    if op in ("rope_fwd", "rope_bwd"):
        shape = rng.choice(["smollm2", "llama8b"])
        d = SHAPES[shape][2]
        return {"op": op, "shape": shape, "lengths": _lens(_draw_lengths(rng, _log_int(rng, 64, 16384), 8192)),
                "rot_dim": rng.choice([d, d // 2]), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "banded", "yarn"]), "offset": rng.choice([0, 0, 5000, 500000])}
    vocab = rng.choice([49152, 128256, 32000, 50257, _log_int(rng, 2000, 128256)])
    rows = _log_int(rng, 32, min(4096, 2048 * 128256 // vocab))
    if op == "pref":
        pairs = rng.randint(1, max(1, min(8, rows // 4)))
        cuts = sorted(rng.sample(range(1, rows), 2 * pairs - 1))
        lengths = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
        return {"op": op, "vocab": vocab, "lengths": _lens(lengths), "kind": rng.choice(["sigmoid", "hinge", "squared"]),
                "smoothing": rng.choice([0.0, 0.1]), "beta": rng.choice([0.05, 0.1, 0.3])}
    return {"op": op, "vocab": vocab, "rows": min(rows, 1999), "masked": round(rng.uniform(0.0, 0.6), 2),
            "clip_low": 0.2, "clip_high": rng.choice([0.2, 0.28]), "kl": rng.choice([0.0, 0.02, 0.1])}


# ------------------------------------------------------------------------------ frequencies

def _scaling(case):
    """The scaling of the rotary frequencies that the case names."""
    return {"none": None,
            "linear": {"kind": "linear", "factor": 4.0},
            "banded": {"kind": "banded", "factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192},
            "yarn": {"kind": "yarn", "factor": 16.0, "beta_fast": 32.0, "beta_slow": 1.0, "original": 8192},
            }[case["scaling"]]


def _frequencies(rot_dim, theta, scaling):
    """Angle per position of each pair (float64, on the host), and the factor on cos and sin."""
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    inv = theta ** (-2.0 * i / rot_dim)
    if scaling is None:
        return inv, 1.0
    f = scaling["factor"]
    if scaling["kind"] == "linear":
        return inv / f, 1.0
    orig = scaling["original"]
    if scaling["kind"] == "banded":
        turns = orig * inv / (2 * math.pi)  # turns over the original context
        keep = ((turns - scaling["low"]) / (scaling["high"] - scaling["low"])).clamp(0.0, 1.0)
        return inv * keep + inv / f * (1 - keep), 1.0

    def pair_of(turns):  # the pair that turns that often over the original context
        return rot_dim * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(theta))

    low = max(math.floor(pair_of(scaling["beta_fast"])), 0)
    high = min(math.ceil(pair_of(scaling["beta_slow"])), rot_dim - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0


# ------------------------------------------------------------------------------ inputs

def _pack_state(lengths):
    s = {"lengths": lengths}
    if own:
        from nf4_layer_streamed_b200 import api
        s["pack"] = api.PackedRows(lengths, device=DEV)  # a program plans a batch once for all of its layers
    return s


def _qkv(g, total, n_q, n_kv, d):
    """Queries, keys and values side by side, as the fused projection leaves them."""
    qkv = torch.randn(total, (n_q + 2 * n_kv) * d, generator=g, device=DEV).to(torch.bfloat16)
    return qkv[:, :n_q * d], qkv[:, n_q * d:(n_q + n_kv) * d], qkv[:, (n_q + n_kv) * d:]


def _logits(g, rows, vocab, targets):
    """A trained model's logits: most tokens far down, the target often near the top."""
    x = torch.randn(rows, vocab, generator=g, device=DEV) * 2.0
    lift = 6.0 + 3.0 * torch.randn(rows, generator=g, device=DEV)
    x[torch.arange(rows, device=DEV), targets.clamp(min=0).long()] += lift
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    if op in ("attn_fwd", "attn_bwd", "rope_fwd", "rope_bwd"):
        n_q, n_kv, d, theta, _ = SHAPES[case["shape"]]
        s = _pack_state(_lengths(case))
        total = sum(s["lengths"])
        q, k, v = _qkv(g, total, n_q, n_kv, d)
        s.update(op=op, n_q=n_q, n_kv=n_kv, d=d, q=q, k=k, v=v)
        if op == "attn_bwd":
            s["o"], s["lse"] = _attention_plain(s)
            s["do"] = torch.randn(total, n_q * d, generator=g, device=DEV).to(torch.bfloat16)
        if op in ("rope_fwd", "rope_bwd"):
            # every sequence starts at its own place in a longer document
            start = torch.randint(0, case["offset"] + 1, (len(s["lengths"]),), generator=g, device=DEV).tolist()
            s["positions"] = torch.cat([torch.arange(a, a + n, dtype=torch.int32) for a, n in
                                        zip(start, s["lengths"])]).to(DEV)
            s["freqs"], s["mscale"] = _frequencies(case["rot_dim"], theta, _scaling(case))
            s["freqs"] = s["freqs"].to(DEV)
            s.update(rot_dim=case["rot_dim"], interleaved=case["interleaved"])
            if own:
                from nf4_layer_streamed_b200 import api
                s["rope"] = api.Rope(d, theta, rot_dim=case["rot_dim"], interleaved=case["interleaved"],
                                     scaling=_scaling(case), device=DEV)
        return s
    if op == "pref":
        s = _pack_state(_lengths(case))
        rows = sum(s["lengths"])
        targets = torch.randint(0, case["vocab"], (rows,), generator=g, device=DEV).to(torch.int32)
        # no loss on the prompt (the first quarter of a sequence) and on a sequence's last row
        seq = torch.repeat_interleave(torch.arange(len(s["lengths"])), torch.tensor(s["lengths"])).to(DEV)
        first = torch.cumsum(torch.tensor([0] + s["lengths"]), 0)[:-1].to(DEV)[seq]
        length = torch.tensor(s["lengths"], device=DEV)[seq]
        at = torch.arange(rows, device=DEV) - first
        targets[(at < length // 4) | (at == length - 1)] = -1
        logits = _logits(g, rows, case["vocab"], targets)
        s.update(op=op, logits=logits, targets=targets, seq=seq, kind=case["kind"], smoothing=case["smoothing"],
                 beta=case["beta"])
        # the reference model's sums: the frozen base answers like the adapted model, some nats apart
        logp = _token_logp(logits, targets)[0]
        drift = 6.0 * torch.randn(len(s["lengths"]), generator=g, device=DEV, dtype=torch.float64)
        s["ref_logp"] = (_by_sequence(logp, seq, len(s["lengths"])) + drift).float()
        return s
    rows = case["rows"]
    targets = torch.randint(0, case["vocab"], (rows,), generator=g, device=DEV).to(torch.int32)
    targets[torch.rand(rows, generator=g, device=DEV) < case["masked"]] = -1
    targets[0] = 1
    logits = _logits(g, rows, case["vocab"], targets)
    logp = _token_logp(logits, targets)[0]
    s = {"op": op, "logits": logits, "targets": targets, "clip_low": case["clip_low"], "clip_high": case["clip_high"],
         "kl": case["kl"]}
    s["old_logp"] = (logp + 0.2 * torch.randn(rows, generator=g, device=DEV)).float()
    s["ref_logp"] = (logp + 0.3 * torch.randn(rows, generator=g, device=DEV)).float()
    s["advantages"] = torch.randn(rows, generator=g, device=DEV)
    s["weights"] = (targets >= 0).float() / (targets >= 0).sum()  # the mean over the rows with a target
    return s


# ------------------------------------------------------------------------------ plain forms

def _heads(x, a, n, h, d):
    return x[a:a + n].float().reshape(n, h, d).transpose(0, 1)


def _attention_plain(s):
    """o = softmax(q k^T / sqrt(d), causal, within each sequence) v, and the log-sum-exp."""
    n_q, n_kv, d = s["n_q"], s["n_kv"], s["d"]
    o, lse, a = [], [], 0
    for n in s["lengths"]:
        q, k, v = _heads(s["q"], a, n, n_q, d), _heads(s["k"], a, n, n_kv, d), _heads(s["v"], a, n, n_kv, d)
        k, v = k.repeat_interleave(n_q // n_kv, 0), v.repeat_interleave(n_q // n_kv, 0)
        t = (q @ k.transpose(1, 2)) / math.sqrt(d)
        t.masked_fill_(torch.ones(n, n, dtype=torch.bool, device=t.device).triu(1), -math.inf)
        m = t.amax(2, keepdim=True)
        t.sub_(m).exp_()
        z = t.sum(2, keepdim=True)
        o.append(((t @ v) / z).transpose(0, 1).reshape(n, n_q * d).to(torch.bfloat16))
        lse.append((m + z.log())[..., 0])
        a += n
    return torch.cat(o), torch.cat(lse, 1)


def _attention_grad_plain(s):
    """dv = p^T do, ds = p (do v^T - rowsum(do o)) / sqrt(d), dq = ds k, dk = ds^T q."""
    n_q, n_kv, d = s["n_q"], s["n_kv"], s["d"]
    dq, dk, dv, a = [], [], [], 0
    for n in s["lengths"]:
        q, k, v = _heads(s["q"], a, n, n_q, d), _heads(s["k"], a, n, n_kv, d), _heads(s["v"], a, n, n_kv, d)
        o, do = _heads(s["o"], a, n, n_q, d), _heads(s["do"], a, n, n_q, d)
        k, v = k.repeat_interleave(n_q // n_kv, 0), v.repeat_interleave(n_q // n_kv, 0)
        p = (q @ k.transpose(1, 2)) / math.sqrt(d)
        p.masked_fill_(torch.ones(n, n, dtype=torch.bool, device=p.device).triu(1), -math.inf)
        p.sub_(s["lse"][:, a:a + n, None]).exp_()
        gv = (p.transpose(1, 2) @ do).reshape(n_kv, -1, n, d).sum(1)
        ds = do @ v.transpose(1, 2)
        ds.sub_((do * o).sum(2, keepdim=True)).mul_(p).div_(math.sqrt(d))
        gk = (ds.transpose(1, 2) @ q).reshape(n_kv, -1, n, d).sum(1)
        dq.append((ds @ k).transpose(0, 1).reshape(n, -1).to(torch.bfloat16))
        dk.append(gk.transpose(0, 1).reshape(n, -1).to(torch.bfloat16))
        dv.append(gv.transpose(0, 1).reshape(n, -1).to(torch.bfloat16))
        a += n
    return torch.cat(dq), torch.cat(dk), torch.cat(dv)


def _rotate_plain(s, x, heads, sign):
    angle = s["positions"].double()[:, None] * s["freqs"][None, :]
    c = (angle.cos() * s["mscale"]).float()[:, None, :]
    sn = (angle.sin() * (sign * s["mscale"])).float()[:, None, :]
    x = x.float().reshape(x.shape[0], heads, s["d"])
    rot, rest = x[..., :s["rot_dim"]], x[..., s["rot_dim"]:]
    if s["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        y = torch.stack((a * c - b * sn, b * c + a * sn), -1).flatten(2)
    else:
        a, b = rot[..., :s["rot_dim"] // 2], rot[..., s["rot_dim"] // 2:]
        y = torch.cat((a * c - b * sn, b * c + a * sn), -1)
    return torch.cat((y, rest), -1).reshape(x.shape[0], -1).to(torch.bfloat16)


def _token_logp(logits, targets):
    """(log probability of each row's target in float64, 0 without one; row maximum; sum)."""
    x = logits.float()
    m = x.amax(1)
    z = (x - m[:, None]).exp_().sum(1, dtype=torch.float64)
    t = x.gather(1, targets.clamp(min=0).long()[:, None])[:, 0]
    lp = t.double() - m.double() - z.log()
    return torch.where(targets >= 0, lp, torch.zeros_like(lp)), m, z


def _by_sequence(logp, seq, n):
    return torch.zeros(n, dtype=torch.float64, device=logp.device).index_add_(0, seq, logp)


def _logits_grad_plain(logits, targets, m, z, coef):
    """coef (onehot - softmax) per row, zero in rows without a target."""
    coef = torch.where(targets >= 0, coef, torch.zeros_like(coef)).float()
    g = (logits.float() - m[:, None]).exp_().mul_((-coef / z.float())[:, None])
    g.scatter_add_(1, targets.clamp(min=0).long()[:, None], coef[:, None])
    return g.to(torch.bfloat16)


def _preference_plain(s):
    logp, m, z = _token_logp(s["logits"], s["targets"])
    n, beta, eps = len(s["lengths"]), s["beta"], s["smoothing"]
    total = _by_sequence(logp, s["seq"], n)
    gap = (total[0::2] - total[1::2]) - (s["ref_logp"][0::2].double() - s["ref_logp"][1::2].double())
    if s["kind"] == "sigmoid":
        h = beta * gap
        loss = (1 - eps) * torch.log1p(torch.exp(-h)) + eps * torch.log1p(torch.exp(h))
        slope = beta * (eps / (1 + torch.exp(-h)) - (1 - eps) / (1 + torch.exp(h)))
    elif s["kind"] == "hinge":
        loss = (1 - beta * gap).clamp(min=0)
        slope = torch.where(beta * gap < 1, -beta, 0.0).double()
    else:
        loss = (gap - 1 / (2 * beta)) ** 2
        slope = 2 * (gap - 1 / (2 * beta))
    coef = torch.stack((slope, -slope), 1).reshape(-1) / (n // 2)
    dlogits = _logits_grad_plain(s["logits"], s["targets"], m, z, coef[s["seq"]])
    return loss.mean().reshape(1).float(), total.float(), (beta * gap).float(), logp.float(), dlogits


def _policy_plain(s):
    logp, m, z = _token_logp(s["logits"], s["targets"])
    adv, w = s["advantages"].double(), s["weights"].double()
    r = torch.exp(logp - s["old_logp"].double())
    free, held = r * adv, r.clamp(1 - s["clip_low"], 1 + s["clip_high"]) * adv
    d = s["ref_logp"].double() - logp
    has = s["targets"] >= 0
    row = w * (s["kl"] * (d.exp() - d - 1) - torch.minimum(free, held))
    coef = w * (s["kl"] * (1 - d.exp()) - torch.where(free <= held, free, torch.zeros_like(free)))
    dlogits = _logits_grad_plain(s["logits"], s["targets"], m, z, coef)
    return torch.where(has, row, torch.zeros_like(row)).sum().reshape(1).float(), logp.float(), dlogits


def run(state):
    s = state
    op = s["op"]
    if own:
        from nf4_layer_streamed_b200 import api
        if op == "attn_fwd":
            return api.packed_attention_fwd(s["pack"], s["q"], s["k"], s["v"], s["n_q"], s["n_kv"], s["d"])
        if op == "attn_bwd":
            return api.packed_attention_bwd(s["pack"], s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["n_q"],
                                            s["n_kv"], s["d"])
        if op in ("rope_fwd", "rope_bwd"):
            return api.rope_apply(s["rope"], s["positions"], s["q"], s["k"], s["n_q"], s["n_kv"],
                                  inverse=op == "rope_bwd")
        if op == "pref":
            fwd = api.preference_loss_fwd(s["pack"], s["logits"], s["targets"], s["ref_logp"], s["beta"],
                                          kind=s["kind"], label_smoothing=s["smoothing"])
            dlogits = api.preference_loss_bwd(s["pack"], s["logits"], s["targets"], fwd)
            return fwd.loss, fwd.seq_logp, fwd.margin, fwd.logp, dlogits
        return api.policy_loss(s["logits"], s["targets"], s["old_logp"], s["ref_logp"], s["advantages"], s["weights"],
                               s["clip_low"], s["clip_high"], s["kl"])
    if op == "attn_fwd":
        return _attention_plain(s)
    if op == "attn_bwd":
        return _attention_grad_plain(s)
    if op in ("rope_fwd", "rope_bwd"):
        sign = 1.0 if op == "rope_fwd" else -1.0
        return _rotate_plain(s, s["q"], s["n_q"], sign), _rotate_plain(s, s["k"], s["n_kv"], sign)
    return _preference_plain(s) if op == "pref" else _policy_plain(s)


# ------------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op in ("attn_fwd", "attn_bwd", "rope_fwd", "rope_bwd"):
        n_q, n_kv, d, _, _ = SHAPES[case["shape"]]
        lengths = _lengths(case)
        total = sum(lengths)
        qb, kb = total * n_q * d * 2, total * n_kv * d * 2
        pairs = sum(n * (n + 1) // 2 for n in lengths)  # unmasked (query, key) pairs
        if op == "attn_fwd":  # q, k, v, o, lse; two products
            return {"bytes": 2 * qb + 2 * kb + 4 * n_q * total, "flops": 4 * d * n_q * pairs}
        if op == "attn_bwd":  # q, k, v, o, do, lse, dq, dk, dv; five products
            return {"bytes": 4 * qb + 4 * kb + 4 * n_q * total, "flops": 10 * d * n_q * pairs}
        return {"bytes": 2 * (qb + kb) + 4 * total, "flops": 3 * total * (n_q + n_kv) * case["rot_dim"]}
    if op == "pref":
        lengths = _lengths(case)
        have = sum(max(0, n - n // 4 - 1) for n in lengths)  # rows with a target: read, and their gradient written
        return {"bytes": 2 * case["vocab"] * (have + sum(lengths)) + 12 * sum(lengths), "flops": 8 * have * case["vocab"]}
    rows = case["rows"]
    have = rows * (1 - case["masked"])
    return {"bytes": int(2 * case["vocab"] * (have + rows)) + 24 * rows, "flops": int(8 * have * case["vocab"])}


# ------------------------------------------------------------------------------ 64 bits

def _exact_attention(s, grad):
    """Head by head in float64, the gradients by autograd of the definition."""
    n_q, n_kv, d = s["n_q"], s["n_kv"], s["d"]
    total = sum(s["lengths"])
    x = {n: s[n].double() for n in ("q", "k", "v")}
    o, lse = torch.zeros_like(x["q"]), torch.zeros(n_q, total, dtype=torch.float64, device=DEV)
    gr = {n: torch.zeros_like(t) for n, t in x.items()}
    for h in range(n_q):
        qs, ks = slice(h * d, (h + 1) * d), slice(h // (n_q // n_kv) * d, (h // (n_q // n_kv) + 1) * d)
        a = 0
        for n in s["lengths"]:
            rows = slice(a, a + n)
            q, k, v = (x[c][rows, w].clone().requires_grad_(grad) for c, w in (("q", qs), ("k", ks), ("v", ks)))
            score = torch.einsum("id,jd->ij", q, k) * d ** -0.5
            i = torch.arange(n, device=DEV)
            score = torch.where(i[:, None] >= i[None, :], score, torch.tensor(-math.inf, device=DEV, dtype=torch.float64))
            out = torch.softmax(score, 1) @ v
            if grad:
                out.backward(s["do"][rows, qs].double())
                gr["q"][rows, qs] += q.grad
                gr["k"][rows, ks] += k.grad
                gr["v"][rows, ks] += v.grad
            else:
                o[rows, qs], lse[h, rows] = out, torch.logsumexp(score, 1)
            a += n
    return (gr["q"], gr["k"], gr["v"]) if grad else (o, lse)


def _exact_rotation(case, s, sign):
    """The pairs as complex numbers, turned by e^(i angle)."""
    theta, d, r = SHAPES[case["shape"]][3], s["d"], case["rot_dim"]
    freqs, scale = _frequencies(r, theta, _scaling(case))
    turn = torch.polar(torch.full((sum(s["lengths"]), r // 2), scale, dtype=torch.float64),
                       sign * torch.outer(s["positions"].cpu().double(), freqs)).to(DEV)
    out = []
    for x, heads in ((s["q"], s["n_q"]), (s["k"], s["n_kv"])):
        y = x.double().reshape(-1, heads, d).clone()
        for h in range(heads):
            i = torch.arange(r // 2, device=DEV)
            re, im = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
            z = torch.complex(y[:, h, re], y[:, h, im]) * turn
            y[:, h, re], y[:, h, im] = z.real, z.imag
        out.append(y.reshape(-1, heads * d))
    return tuple(out)


def _exact_rows(s, rows_at_once=128):
    """log softmax of each row's target in float64."""
    t = s["targets"].long()
    lp = torch.zeros(t.numel(), dtype=torch.float64, device=DEV)
    for a in range(0, t.numel(), rows_at_once):
        b = slice(a, a + rows_at_once)
        x = torch.log_softmax(s["logits"][b].double(), 1)
        lp[b] = x[torch.arange(x.shape[0], device=DEV), t[b].clamp(min=0)]
    return lp * (t >= 0)


def _exact_logits_grad(s, dlogp, rows_at_once=128):
    t = s["targets"].long()
    out = torch.zeros(s["logits"].shape, dtype=torch.float64, device=DEV)
    for a in range(0, t.numel(), rows_at_once):
        for_rows = torch.arange(a, min(a + rows_at_once, t.numel()), device=DEV)
        for_rows = for_rows[t[for_rows] >= 0]
        p = -torch.softmax(s["logits"][for_rows].double(), 1)
        p[torch.arange(len(for_rows), device=DEV), t[for_rows]] += 1
        out[for_rows] = p * dlogp[for_rows, None]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("attn_fwd", "attn_bwd"):
        return _exact_attention(s, op == "attn_bwd")
    if op in ("rope_fwd", "rope_bwd"):
        return _exact_rotation(case, s, 1.0 if op == "rope_fwd" else -1.0)
    logp = _exact_rows(s).requires_grad_(True)
    if op == "pref":
        n = len(s["lengths"])
        total = torch.stack([logp[s["seq"] == i].sum() for i in range(n)])
        ratio = total - s["ref_logp"].double()
        margin = s["beta"] * (ratio[0::2] - ratio[1::2])
        if s["kind"] == "sigmoid":
            ls = torch.nn.functional.logsigmoid
            loss = -((1 - s["smoothing"]) * ls(margin) + s["smoothing"] * ls(-margin)).mean()
        elif s["kind"] == "hinge":
            loss = torch.relu(1 - margin).mean()
        else:
            loss = (margin / s["beta"] - 0.5 / s["beta"]).square().mean()
        loss.backward()
        return (loss.detach().reshape(1), total.detach(), margin.detach(), logp.detach(),
                _exact_logits_grad(s, logp.grad))
    ratio = (logp - s["old_logp"].double()).exp()
    adv = s["advantages"].double()
    best = torch.minimum(ratio * adv, torch.clamp(ratio, 1 - s["clip_low"], 1 + s["clip_high"]) * adv)
    gap = s["ref_logp"].double() - logp
    each = s["weights"].double() * (s["kl"] * (torch.expm1(gap) - gap) - best)
    loss = each[s["targets"] >= 0].sum()
    loss.backward()
    return loss.detach().reshape(1), logp.detach(), _exact_logits_grad(s, logp.grad)
