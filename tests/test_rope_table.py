"""Rotary frequency tables against the published formulas, and refusals (host only)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from nf4_layer_streamed_b200 import api, binding as B

BANDED = {"kind": "banded", "factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192}
YARN = {"kind": "yarn", "factor": 16.0, "beta_fast": 32.0, "beta_slow": 1.0, "original": 4096}


def frequencies(rot, theta, scaling):
    inv = theta ** (-2.0 * np.arange(rot // 2) / rot)
    if scaling is None:
        return inv, 1.0
    f = scaling["factor"]
    if scaling["kind"] == "linear":
        return inv / f, 1.0
    if scaling["kind"] == "banded":  # by wavelength, as it was published
        wave = 2 * math.pi / inv
        smooth = (scaling["original"] / wave - scaling["low"]) / (scaling["high"] - scaling["low"])
        mid = (1 - smooth) * inv / f + smooth * inv
        return np.where(wave < scaling["original"] / scaling["high"], inv,
                        np.where(wave > scaling["original"] / scaling["low"], inv / f, mid)), 1.0

    def dim(n):
        return rot * math.log(scaling["original"] / (n * 2 * math.pi)) / (2 * math.log(theta))
    lo, hi = max(math.floor(dim(scaling["beta_fast"])), 0), min(math.ceil(dim(scaling["beta_slow"])), rot - 1)
    ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0, 1)
    return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1


@pytest.mark.parametrize("scaling", [None, {"kind": "linear", "factor": 4.0}, BANDED, YARN],
                         ids=lambda s: s["kind"] if s else "none")
@pytest.mark.parametrize("rot,theta", [(64, 10000.0), (128, 500000.0), (16, 10000.0)])
def test_table(rot, theta, scaling):
    r = api.Rope(128, theta, rot_dim=rot, scaling=scaling, device="cpu")
    want, m = frequencies(rot, theta, scaling)
    got = r.turns_host.astype(np.float64) * 2.0 ** -64 * 2 * math.pi
    # the table's own step of 2^-64 turns, and float64 roundings of both sides
    assert np.all(np.abs(got - want) <= 2 * math.pi * 2.0 ** -64 + 1e-14 * want)
    assert abs(r.mscale - m) <= 2.0 ** -23 * m


def test_refusals():
    for kw in (dict(head_dim=24), dict(head_dim=528), dict(rot_dim=144), dict(rot_dim=8), dict(theta=1.0),
               dict(theta=math.inf), dict(scaling={"kind": "linear", "factor": 0.5}),
               dict(scaling=dict(BANDED, low=4.0)), dict(scaling=dict(YARN, original=0)),
               dict(scaling=dict(YARN, factor=math.nan))):
        args = dict(head_dim=128, theta=10000.0, device="cpu")
        args.update(kw)
        with pytest.raises(B.NF4LSError):
            api.Rope(**args)
    for bad in ({"kind": "cubic", "factor": 2.0}, {"kind": "linear"}, {"kind": "yarn", "factor": 2.0},
                {"kind": "linear", "factor": 2.0, "original": 5}):
        with pytest.raises(ValueError, match="scaling"):
            api.Rope(128, 10000.0, scaling=bad, device="cpu")
    r = api.Rope(64, 10000.0, device="cpu")
    pos = torch.zeros(6, dtype=torch.int32)
    q, k = torch.zeros(6, 256, dtype=torch.bfloat16), torch.zeros(6, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="rope"):
        api.rope_apply(None, pos, q, k, 4, 2)
    with pytest.raises(ValueError, match="positions"):
        api.rope_apply(r, pos.long(), q, k, 4, 2)
    with pytest.raises(ValueError, match="heads"):
        api.rope_apply(r, pos, q, k, 4, 0)
    with pytest.raises(ValueError, match="k: expected"):
        api.rope_apply(r, pos, q, k, 4, 4)
    with pytest.raises(ValueError, match="q: expected"):
        api.rope_apply(r, pos, q[:5], k, 4, 2)
    buf = torch.zeros(6, 520, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlaps"):
        api.rope_apply(r, pos, buf[:, :256], buf[:, 256:384], 4, 2, out=(buf[:, 8:264], buf[:, 384:512]))
    with pytest.raises(ValueError, match="overlaps"):
        api.rope_apply(r, pos, buf[:, :256], buf[:, 256:384], 4, 2, out=(buf[:, 256:512], buf[:, :128]))
    with pytest.raises(ValueError, match="CUDA"):            # in place is no overlap
        api.rope_apply(r, pos, buf[:, :256], buf[:, 256:384], 4, 2, out=(buf[:, :256], buf[:, 256:384]))


def test_c_call_checks_its_arguments_on_the_host():
    cfg = B.RopeCfg(64, 64, 0, 0, 10000.0, 1.0, 0.0, 0.0, 0.0)
    t = B.RopeRows(256, 256, 256, 256, 256, 256, 6, 4, 2, 256, 128, 256, 128, 0, 1.0)

    def call():
        return B.call_status("nf4ls_rope_apply", ctypes.byref(cfg), ctypes.byref(t), None)
    for field, bad, want in (("rows", -1, -2), ("n_q", 2000, -2), ("turns_dev", 0, -1), ("turns_dev", 264, -3),
                             ("positions_dev", 0, -1), ("q", 0, -1), ("k_out", 8, -3), ("ld_q", 255, -2),
                             ("ld_k", 132, -2), ("ld_q_out", 248, -2), ("rows", 1 << 30, -2)):
        keep = getattr(t, field)
        setattr(t, field, bad)
        assert call() == want, field
        setattr(t, field, keep)
    t.n_q = t.n_kv = 0
    assert call() == -2
    cfg.rot_dim = 72
    assert call() == -2


def test_c_call_refuses_in_place_with_another_row_stride():
    cfg = B.RopeCfg(64, 32, 0, 0, 10000.0, 1.0, 0.0, 0.0, 0.0)
    for side in ("q", "k"):
        t = B.RopeRows(256, 256, 256, 512, 1024, 2048, 6, 4, 2, 256, 128, 256, 128, 0, 1.0)
        setattr(t, side + "_out", getattr(t, side))
        setattr(t, f"ld_{side}_out", 320)
        assert B.call_status("nf4ls_rope_apply", ctypes.byref(cfg), ctypes.byref(t), None) == -1
        assert f"{side} in place" in B.last_error()
