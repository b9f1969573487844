"""The training calls refuse bad arguments on the host, before any device
work (no GPU needed)."""
import ctypes

import pytest
import torch

import block_sparse_attention_losa_b200 as losa

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: the checks fail first
OUT = [ctypes.c_void_p(0x100000 * i) for i in (1, 2, 3)]


def _spec(n_axes=3, grid=(3, 5, 7), dim=(16, 24, 24), start=(0, 0, 0), scale=(1.0, 1.0, 1.0),
          theta=1e4, n_text=2, pairing=0):
    return losa.RopeSpec(n_axes, (ctypes.c_int * 3)(*grid), (ctypes.c_int * 3)(*dim),
                         (ctypes.c_int * 3)(*start), (ctypes.c_double * 3)(*scale), theta,
                         n_text, pairing)


def _strides(B, L, H, d):
    return [L * H * d, H * d, d] * 3


def _rope(unpack, spec={}, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, in_dt=0, B=2, H=3, L=107, L_pad=128, d=64, pos=None,
             qo=OUT[0], ko=OUT[1], vo=OUT[2], out_dt=0)
    a.update(kw)
    st = a.get("strides", _strides(2, 107, 3, 64))
    st = None if st is None else (ctypes.c_int64 * 9)(*st)
    sp = None if spec is None else ctypes.byref(_spec(**spec))
    lib = losa.lib()
    if unpack:
        return lib.losa_rope_unpack(a["q"], a["k"], a["v"], a["in_dt"], a["B"], a["H"], a["L"],
                                    a["L_pad"], a["d"], sp, a["pos"], a["qo"], a["ko"], a["vo"],
                                    a["out_dt"], st, None)
    return lib.losa_rope_pack(a["q"], a["k"], a["v"], a["in_dt"], st, a["B"], a["H"], a["L"],
                              a["L_pad"], a["d"], sp, a["pos"], a["qo"], a["ko"], a["vo"],
                              a["out_dt"], None)


BAD = [
    dict(q=None), dict(qo=None), dict(vo=None), dict(q=None, k=None, v=None),
    dict(q=None, k=None, v=None, qo=None, ko=None, vo=None), dict(in_dt=2), dict(out_dt=-1),
    dict(B=0), dict(H=0), dict(L=0), dict(L=129), dict(L_pad=300), dict(d=96), dict(B=300, H=300),
    dict(strides=None), dict(q=ctypes.c_void_p(0x10001)), dict(ko=ctypes.c_void_p(0x10001)),
    dict(in_dt=1, k=ctypes.c_void_p(0x10002)), dict(strides=[-1, 192, 64] * 3),
    dict(strides=[20544, 1 << 50, 64] * 3), dict(spec=None), dict(spec=dict(n_axes=0)),
    dict(spec=dict(n_axes=4)), dict(spec=dict(grid=(3, 5, 8))), dict(spec=dict(grid=(-3, -5, 7))),
    dict(spec=dict(grid=(1 << 30, 1 << 30, 1 << 30))), dict(spec=dict(dim=(16, 24, 26))),
    dict(spec=dict(dim=(16, 23, 24))), dict(spec=dict(dim=(0, 24, 24))),
    dict(spec=dict(theta=0.0)), dict(spec=dict(theta=float("inf"))),
    dict(spec=dict(theta=float("nan"))), dict(spec=dict(scale=(1.0, float("nan"), 1.0))),
    dict(spec=dict(n_text=-1)), dict(spec=dict(n_text=108)), dict(spec=dict(pairing=2)),
    dict(pos=FAKE, spec=dict(n_text=108)), dict(pos=ctypes.c_void_p(0x10002)),
    dict(qo=FAKE), dict(vo=FAKE), dict(qo=OUT[2]), dict(ko=OUT[0]), dict(vo=OUT[1]),
    dict(spec=dict(theta=1e-320, scale=(1.0, 1e10, 1.0))), dict(spec=dict(scale=(1e305, 1.0, 1.0))),
]


@pytest.mark.parametrize("unpack", [False, True])
@pytest.mark.parametrize("bad", BAD)
def test_rope_refuses_bad_arguments(unpack, bad):
    assert _rope(unpack, **bad) == -1


@pytest.mark.parametrize("strides", [[0, 192, 64], [20544, 0, 64], [20544, 192, 0],
                                     [20544, 192, 32], [20480, 192, 64], [64, 128, 64 * 214 - 1]])
def test_unpack_refuses_outputs_that_overlap_themselves(strides):
    assert _rope(True, strides=strides * 3) == -1


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on a GPU")
@pytest.mark.parametrize("unpack", [False, True])
@pytest.mark.parametrize("good", [
    {}, dict(k=None, ko=None), dict(v=None, vo=None, in_dt=1), dict(L=1, L_pad=1, spec=dict(
        grid=(1, 1, 1), n_text=0), strides=_strides(2, 1, 3, 64)),
    dict(L=128, spec=dict(n_text=23), strides=_strides(2, 128, 3, 64)),
    dict(spec=dict(n_axes=1, grid=(105, 9, 9), dim=(64, 1, 1))),
    # Head-major, and the views of a fused projection.
    dict(strides=[3 * 107 * 64, 64, 107 * 64] * 3), dict(strides=[107 * 576, 576, 64] * 3),
    # One batch: its stride is not used.
    dict(B=1, strides=[0, 192, 64] * 3),
])
def test_rope_accepts_up_to_the_device_check(unpack, good):
    assert _rope(unpack, **good) == -6


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on a GPU")
def test_pack_reads_broadcast_inputs_and_positions():
    assert _rope(False, strides=[0, 0, 0] * 3) == -6
    assert _rope(False, pos=FAKE, spec=dict(grid=(9, 9, 9))) == -6


def test_backward_refuses_null_pattern_and_pointers():
    lib = losa.lib()
    args = [FAKE, FAKE, FAKE, 0, FAKE, 1, FAKE, FAKE, 0, 64, 100, 0.1, None, FAKE, FAKE, FAKE, 0,
            FAKE, 1 << 20, None]
    assert lib.losa_sparse_attn_bwd(*args) == -1
    assert lib.losa_sparse_attn_bwd_workspace(None, 0, 0, 64) == -1
    assert lib.losa_pattern_prepare_bwd(None, None) == -1
    assert lib.losa_pattern_export_bwd(None, None, None, None, None, None) == -1


def test_rope_class_refuses_bad_axes():
    for kw in (dict(grid=(2, 3), dims=(32, 16, 16)), dict(grid=(2, 3, 4, 5), dims=(2, 2, 2, 2)),
               dict(grid=(), dims=()), dict(grid=(4,), dims=(64,), pairing="odd"),
               dict(grid=(4,), dims=(64,), start=(1, 2)), dict(grid=(4,), dims=(64,), scale=()),
               dict(grid=(2 ** 31,), dims=(64,))):
        with pytest.raises(ValueError):
            losa.Rope(**kw)


def test_binding_refuses_host_tensors_and_shapes():
    rope = losa.Rope((2, 3, 4), (16, 24, 24))
    x = torch.zeros(1, 24, 2, 64)
    with pytest.raises(ValueError):
        losa.rope_pack(x, x, x, 32, rope)
    with pytest.raises(ValueError):
        losa.rope_unpack(None, None, None, 24, rope)
    with pytest.raises(ValueError):
        losa.sparse_attn_bwd(x, x, x, x, x, x, 24, None)
