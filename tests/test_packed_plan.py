"""The plan of a packed batch and the refusals of the packed calls (host only)."""
import ctypes

import numpy as np
import pytest
import torch

from nf4_layer_streamed_b200 import api, binding as B


def _tiles(p, off):
    n = p.pack.n_tiles
    return p.plan[off:off + 16 * n].view(torch.int32).view(n, 4).tolist()


@pytest.mark.parametrize("lengths", [[1], [0], [0, 0, 0], [128], [129, 127], [3, 0, 300, 128, 1, 0], [1] * 500,
                                     [4097, 1, 640]])
def test_plan_lists_every_row_and_tile_once(lengths):
    p = api.PackedRows(lengths, device="cpu")
    first = np.concatenate([[0], np.cumsum(lengths)])
    assert (p.total, p.n_seqs, p.max_len) == (first[-1], len(lengths), max(lengths))
    assert p.cu.tolist() == first.tolist()
    assert p.positions.tolist() == [i for n in lengths for i in range(n)]
    assert p.seq.tolist() == [s for s, n in enumerate(lengths) for _ in range(n)]
    want, index = [], 0
    for s, n in enumerate(lengths):
        for t in range((n + 127) // 128):
            want.append([int(first[s]), n, t, index])
            index += 1
    q, k = _tiles(p, p.pack.off_query_tiles), _tiles(p, p.pack.off_key_tiles)
    assert sorted(q) == sorted(want) and sorted(k) == sorted(want)
    assert p.pack.n_blocks == sum(t + 1 for _, _, t, _ in q)
    work_q = [t for _, _, t, _ in q]
    work_k = [(n + 127) // 128 - t for _, n, t, _ in k]
    assert work_q == sorted(work_q, reverse=True) and work_k == sorted(work_k, reverse=True)


def test_plan_refusals():
    for bad in ([], [[1, 2]], [-1], [1, -5], [1 << 29]):
        with pytest.raises(ValueError):
            api.PackedRows(bad, device="cpu")
    with pytest.raises(B.NF4LSError, match="more than"):
        api.PackedRows([1 << 28, 1], device="cpu")
    n = np.array([5, 7], np.int32)
    pack = B.Pack()
    assert B.call_status("nf4ls_pack_layout", None, 2, ctypes.byref(pack)) == -1
    assert B.call_status("nf4ls_pack_layout", n.ctypes.data, 0, ctypes.byref(pack)) == -1
    assert B.call_status("nf4ls_pack_layout", n.ctypes.data, (1 << 20) + 1, ctypes.byref(pack)) == -1
    B.call("nf4ls_pack_layout", n.ctypes.data, 2, ctypes.byref(pack))
    buf = np.zeros(pack.plan_bytes, np.uint8)
    assert B.call_status("nf4ls_pack_fill", n.ctypes.data, ctypes.byref(pack), buf.ctypes.data, buf.size - 1) == -1
    other = np.array([5, 8], np.int32)
    assert B.call_status("nf4ls_pack_fill", other.ctypes.data, ctypes.byref(pack), buf.ctypes.data, buf.size) == -1
    assert not buf.any()


def _attention_args(n_q=4, n_kv=2, d=64, rows=12, dtype=torch.bfloat16):
    z = lambda w: torch.zeros(rows, w, dtype=dtype)  # noqa: E731
    return api.PackedRows([5, 7], device="cpu"), z(n_q * d), z(n_kv * d), z(n_kv * d)


def test_attention_refuses_what_the_kernels_would_misread():
    pack, q, k, v = _attention_args()
    with pytest.raises(TypeError, match="pack"):
        api.packed_attention_fwd([5, 7], q, k, v, 4, 2, 64)
    with pytest.raises(ValueError, match="head_dim"):
        api.packed_attention_fwd(pack, q, k, v, 4, 2, 96)
    with pytest.raises(ValueError, match="multiple"):
        api.packed_attention_fwd(pack, q, k, v, 4, 3, 64)
    with pytest.raises(ValueError, match="scale"):
        api.packed_attention_fwd(pack, q, k, v, 4, 2, 64, scale=0.0)
    with pytest.raises(ValueError, match="q: expected"):
        api.packed_attention_fwd(pack, q.float(), k, v, 4, 2, 64)
    with pytest.raises(ValueError, match="q: expected"):
        api.packed_attention_fwd(pack, q[:11], k, v, 4, 2, 64)       # fewer rows than the pack
    with pytest.raises(ValueError, match="k: expected"):
        api.packed_attention_fwd(pack, q, k[:, :64], v, 4, 2, 64)
    with pytest.raises(ValueError, match="strides"):
        api.packed_attention_fwd(pack, torch.zeros(12, 260, dtype=torch.bfloat16)[:, :256], k, v, 4, 2, 64)
    with pytest.raises(ValueError, match="strides"):
        api.packed_attention_fwd(pack, torch.zeros(256, 12, dtype=torch.bfloat16).t(), k, v, 4, 2, 64)
    with pytest.raises(ValueError, match="aligned"):
        api.packed_attention_fwd(pack, torch.zeros(12, 264, dtype=torch.bfloat16)[:, 4:260], k, v, 4, 2, 64)
    with pytest.raises(ValueError, match="overlaps"):
        api.packed_attention_fwd(pack, q, k, v, 4, 2, 64, out=q)
    with pytest.raises(ValueError, match="CUDA"):
        api.packed_attention_fwd(pack, q, k, v, 4, 2, 64)
    lse = torch.zeros(4, 12)
    with pytest.raises(ValueError, match="lse"):
        api.packed_attention_bwd(pack, q, k, v, q, q, lse[:, :11], 4, 2, 64)
    buf = torch.zeros(12, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlaps"):
        api.packed_attention_bwd(pack, q, k, v, q, q, lse, 4, 2, 64,
                                 out=(buf[:, :256], buf[:, 248:376], buf[:, 384:512]))
    with pytest.raises(ValueError, match="CUDA"):      # column slices of one buffer do not overlap
        api.packed_attention_bwd(pack, q, k, v, q, q, lse, 4, 2, 64,
                                 out=(buf[:, :256], buf[:, 256:384], buf[:, 384:512]))


def test_attention_c_calls_check_their_arguments_on_the_host():
    n = np.array([5, 7], np.int32)
    pack = B.Pack()
    B.call("nf4ls_pack_layout", n.ctypes.data, 2, ctypes.byref(pack))
    heads = B.PackedHeads(4, 2, 64, 0.125)
    t = B.PackedAttention(256, 256, 256, 256, 256, 256, 256, 256, 256, 256, 128, 128, 256, 256, 256, 128, 128)

    def fwd():
        return B.call_status("nf4ls_packed_attention_fwd", ctypes.byref(pack), ctypes.byref(heads), ctypes.byref(t), None)

    def bwd(ws=256, nbytes=1 << 30):
        return B.call_status("nf4ls_packed_attention_bwd", ctypes.byref(pack), ctypes.byref(heads), ctypes.byref(t),
                             ws, nbytes, None)
    assert fwd() == -1 and "plan" in B.last_error()
    pack.plan_dev = 264
    assert fwd() == -3
    pack.plan_dev = 256
    assert bwd(nbytes=4 * 2 * 2 * 128 * 4 - 1) == -1 and "workspace" in B.last_error()
    assert bwd(ws=264) == -3
    for field, bad, want in (("n_q", 5, -2), ("n_kv", 0, -2), ("head_dim", 80, -2), ("scale", -1.0, -1),
                             ("scale", float("nan"), -1)):
        keep = getattr(heads, field)
        setattr(heads, field, bad)
        assert fwd() == want and bwd() == want, field
        setattr(heads, field, keep)
    for field, bad, want in (("q", 0, -1), ("k", 264, -3), ("ld_q", 255, -2), ("ld_v", 132, -2), ("o", 8, -3),
                             ("ld_o", 128, -2), ("lse", 0, -1)):
        keep = getattr(t, field)
        setattr(t, field, bad)
        assert fwd() == want and bwd() == want, field
        setattr(t, field, keep)
    for field, bad, want in (("d_o", 0, -1), ("dk", 8, -3), ("ld_dq", 128, -2)):
        keep = getattr(t, field)
        setattr(t, field, bad)
        assert bwd() == want, field
        setattr(t, field, keep)
    pack.n_tiles = 13                                           # not what the layout gave
    assert fwd() == -1
    assert B.call_status("nf4ls_packed_attention_fwd", None, ctypes.byref(heads), ctypes.byref(t), None) == -1


def test_argument_structs_are_laid_out_like_the_bindings():
    for packed, struct in ((api._ATTENTION, B.PackedAttention), (api._ROPE_ROWS, B.RopeRows),
                           (api._LOGITS, B.Logits), (api._PREF_OUT, B.PreferenceOut), (api._POLICY_CFG, B.PolicyCfg),
                           (api._POLICY_ROWS, B.PolicyRows), (api._PREF_CFG, B.PreferenceCfg)):
        assert packed.size == ctypes.sizeof(struct)
        n = len(struct._fields_)
        values = [float(i + 1) if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(struct._fields_)]
        got = struct.from_buffer_copy(packed.pack(*values))
        assert [getattr(got, name) for name, _ in struct._fields_] == values and n == len(values)


def test_head_configuration_is_taken_by_value():
    """A 0-dim tensor that changes in place is read anew at every call (refused here when its value is)."""
    pack, q, k, v = _attention_args()
    scale, n_kv = torch.tensor(0.5), torch.tensor(2)
    for call in (lambda: api.packed_attention_fwd(pack, q, k, v, 4, n_kv, 64, scale=scale),
                 lambda: api.packed_attention_bwd(pack, q, k, v, q, q, torch.zeros(4, 12), 4, n_kv, 64, scale=scale)):
        scale.fill_(0.5), n_kv.fill_(2)
        with pytest.raises(ValueError, match="CUDA"):      # every other argument is good
            call()
        scale.fill_(-1.0)
        with pytest.raises(ValueError, match="scale -1.0"):
            call()
        scale.fill_(0.5), n_kv.fill_(3)
        with pytest.raises(ValueError, match="not a multiple of 3"):
            call()


@pytest.mark.parametrize("shape", [(12, 4), (48,), (1, 4, 12), (2, 24)])
def test_gradients_refuse_statistics_of_another_layout(shape):
    """lse is [n_q, total]: the same number of values in another order would be misread."""
    pack, q, k, v = _attention_args()
    with pytest.raises(ValueError, match="lse: expected"):
        api.packed_attention_bwd(pack, q, k, v, q, q, torch.zeros(shape), 4, 2, 64)


def test_lengths_are_whole_numbers():
    for bad in ([1.5], [3, 2.999], np.array([4.0, np.nan]), torch.tensor([0.5, 8.0])):
        with pytest.raises(ValueError, match="whole"):
            api.PackedRows(bad, device="cpu")
    for good in ([3, 2], (3.0, 2.0), np.array([3, 2], np.int16), torch.tensor([3, 2])):
        assert api.PackedRows(good, device="cpu").cu.tolist() == [0, 3, 5]
    for far in ([2.0 ** 70, 1.0], [float("inf")], np.array([2 ** 64 - 1], np.uint64)):
        with pytest.raises(ValueError, match="outside"):
            api.PackedRows(far, device="cpu")


def test_overlap_is_found_across_storages():
    """A view that came back through dlpack shares memory, though its storage starts elsewhere."""
    pack, q, k, v = _attention_args()
    buf = torch.zeros(12, 512, dtype=torch.bfloat16)
    alias = torch.from_dlpack(buf[:, 128:384])
    with pytest.raises(ValueError, match="overlaps"):
        api.packed_attention_fwd(pack, buf[:, :256], k, v, 4, 2, 64, out=alias)
    with pytest.raises(ValueError, match="CUDA"):          # its neighbours' columns are no overlap
        api.packed_attention_fwd(pack, q, buf[:, :128], buf[:, 384:], 4, 2, 64, out=alias)
    rows = torch.zeros(20, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlaps"):
        api.packed_attention_fwd(pack, rows[:12], k, v, 4, 2, 64, out=torch.from_dlpack(rows[8:]))
