"""Refusals of the preference and policy losses (host only)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from nf4_layer_streamed_b200 import api, binding as B


def _args():
    pack = api.PackedRows([3, 4], device="cpu")
    return pack, torch.zeros(7, 50, dtype=torch.bfloat16), torch.zeros(7, dtype=torch.int32), torch.zeros(2)


def test_preference_refuses():
    pack, x, t, ref = _args()
    with pytest.raises(TypeError, match="pack"):
        api.preference_loss_fwd(None, x, t, ref, 0.1)
    with pytest.raises(ValueError, match="pairs"):
        api.preference_loss_fwd(api.PackedRows([3, 3, 1], device="cpu"), x, t, torch.zeros(3), 0.1)
    with pytest.raises(ValueError, match="kind"):
        api.preference_loss_fwd(pack, x, t, ref, 0.1, kind="cubic")
    with pytest.raises(ValueError, match="logits"):
        api.preference_loss_fwd(pack, x.float(), t, ref, 0.1)
    with pytest.raises(ValueError, match="logits"):
        api.preference_loss_fwd(pack, x[:6], t, ref, 0.1)
    with pytest.raises(ValueError, match="strides"):
        api.preference_loss_fwd(pack, torch.zeros(50, 7, dtype=torch.bfloat16).t(), t, ref, 0.1)
    with pytest.raises(ValueError, match="targets"):
        api.preference_loss_fwd(pack, x, t.long(), ref, 0.1)
    with pytest.raises(ValueError, match="ref_logp"):
        api.preference_loss_fwd(pack, x, t, ref.double(), 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        api.preference_loss_fwd(pack, x, t, ref, 0.1)
    f = api.PreferenceForward(*(torch.zeros(n) for n in (1, 2, 1, 7, 2, 28)))
    with pytest.raises(TypeError, match="fwd"):
        api.preference_loss_bwd(pack, x, t, ref)
    with pytest.raises(ValueError, match="columns"):
        api.preference_loss_bwd(pack, x, t, f, out=torch.zeros(7, 49, dtype=torch.bfloat16))
    big = torch.zeros(9, 50, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlaps"):
        api.preference_loss_bwd(pack, big[:7], t, f, out=big[1:8])
    with pytest.raises(ValueError, match="CUDA"):
        api.preference_loss_bwd(pack, x, t, f, out=x)            # in place
    other = api.PreferenceForward(*(torch.zeros(n) for n in (1, 2, 1, 7, 2, 24)))
    with pytest.raises(ValueError, match="row_stats"):           # of another batch
        api.preference_loss_bwd(pack, x, t, other)


def test_policy_refuses():
    _, x, t, _ = _args()
    r = torch.zeros(7)
    with pytest.raises(ValueError, match="ref_logp"):
        api.policy_loss(x, t, r, r[:6], r, r, 0.2, 0.2, 0.1)
    with pytest.raises(TypeError, match="ref_logp"):
        api.policy_loss(x, t, r, None, r, r, 0.2, 0.2, 0.1)
    with pytest.raises(ValueError, match="out"):
        api.policy_loss(x, t, r, r, r, r, 0.2, 0.2, grad=False, out=x)
    with pytest.raises(ValueError, match="CUDA"):
        api.policy_loss(x, t, r, None, r, r, 0.2, 0.2)


def test_c_calls_check_their_arguments_on_the_host():
    n = np.array([3, 4], np.int32)
    pack = B.Pack()
    B.call("nf4ls_pack_layout", n.ctypes.data, 2, ctypes.byref(pack))
    pack.plan_dev = 256
    cfg = B.PreferenceCfg(0, 0.1, 0.0)
    x = B.Logits(256, 50, 50, 256)
    out = B.PreferenceOut(*[256] * 6)

    def fwd(ref=256):
        return B.call_status("nf4ls_preference_fwd", ctypes.byref(pack), ctypes.byref(cfg), ctypes.byref(x), ref,
                             ctypes.byref(out), None)

    def bwd(d=512, ld=50):
        return B.call_status("nf4ls_preference_bwd", ctypes.byref(pack), ctypes.byref(x), ctypes.byref(out), 1.0, d, ld,
                             None)

    def each(obj, cases, *calls):
        for field, bad, want in cases:
            keep = getattr(obj, field)
            setattr(obj, field, bad)
            for c in calls:
                assert c() == want, (field, bad, B.last_error())
            setattr(obj, field, keep)
    each(cfg, [("kind", 3, -1), ("beta", 0.0, -1), ("beta", math.nan, -1), ("label_smoothing", 0.5, -1),
               ("label_smoothing", -0.1, -1)], fwd)
    cfg.kind = 1  # smoothing is checked whether or not the kind uses it
    each(cfg, [("label_smoothing", 0.5, -1)], fwd)
    cfg.kind = 0
    each(x, [("vocab", 0, -2), ("ld", 49, -2), ("logits_dev", 0, -1), ("logits_dev", 255, -3),
             ("targets_dev", 258, -3)], fwd, bwd)
    each(out, [("row_stats", 264, -3), ("row_stats", 0, -1), ("coef", 0, -1)], fwd, bwd)
    each(out, [("loss", 0, -1), ("margin", 0, -1), ("logp", 0, -1), ("seq_logp", 0, -1)], fwd)
    assert fwd(ref=None) == -1
    assert bwd(d=None) == -1 and bwd(ld=49) == -2 and bwd(d=511) == -3 and bwd(d=256, ld=64) == -1
    pack.n_seqs = 1
    assert fwd() == -2
    p = B.PolicyCfg(0.2, 0.2, 0.1, 1.0)
    rows = B.PolicyRows(256, 256, 256, 256)

    def pol(n=7, loss=256):
        return B.call_status("nf4ls_policy_loss", ctypes.byref(p), n, ctypes.byref(x), ctypes.byref(rows), loss, 256,
                             256, 512, 50, None)
    each(p, [("clip_low", -0.1, -1), ("clip_low", 1.5, -1), ("clip_high", math.inf, -1), ("kl_coef", -1.0, -1),
             ("grad_scale", math.nan, -1)], pol)
    each(rows, [("old_logp", 0, -1), ("ref_logp", 0, -1), ("weights", 0, -1)], pol)
    each(x, [("vocab", 0, -2), ("ld", 49, -2), ("targets_dev", 0, -1)], pol)
    assert pol(n=-1) == -1 and pol(loss=None) == -1
