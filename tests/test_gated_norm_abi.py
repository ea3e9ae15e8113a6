"""Host-side argument checks of the gated scan's and the group norm's C entries: no GPU is needed, and a refused
call launches nothing."""
import ctypes

import pytest

from state_space_model_02_gb300 import build as cuda_build
from state_space_model_02_gb300 import ssd

GOOD = ctypes.c_void_p(0x100000)
OK_ELEM = ctypes.c_void_p(0x100002)   # aligned to a bf16 value only
ODD = ctypes.c_void_p(0x100001)


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return ssd.load_library()


def gated(**kw):
    base = dict(batch=2, seqlen=64, dim=96, x_stride=0, gate_stride=0, io_dtype=ssd.SSD_BF16, kind=2, complement=0, flags=0)
    base.update(kw)
    return ctypes.byref(ssd.GatedShape(**base))


def norm(**kw):
    base = dict(batch=2, seqlen=64, channels=96, ngroups=4, x_stride=0, z_stride=0, eps=1e-5, io_dtype=ssd.SSD_BF16,
                act=2, flags=0)
    base.update(kw)
    return ctypes.byref(ssd.NormShape(**base))


BAD_GATED = [(dict(batch=0), 1), (dict(seqlen=0), 1), (dict(dim=0), 1), (dict(io_dtype=7), 1), (dict(kind=3), 1),
             (dict(kind=-1), 1), (dict(complement=2), 1), (dict(flags=1), 1), (dict(x_stride=95), 1),
             (dict(gate_stride=-1), 1), (dict(batch=65536), 2), (dict(dim=(1 << 20) + 1), 2), (dict(seqlen=1 << 45), 2)]


@pytest.mark.parametrize("bad,rc", BAD_GATED)
def test_gated_shapes(lib, bad, rc):
    s = gated(**bad)
    assert lib.ssd_gated_workspace_bytes(s) == 0 and lib.ssd_gated_bwd_workspace_bytes(s) == 0
    assert lib.ssd_gated_scan(s, *([GOOD] * 7), 1 << 40, None) == rc and lib.ssd_last_error()
    assert lib.ssd_gated_scan_bwd(s, *([GOOD] * 9), 1 << 40, None) == rc
    assert lib.ssd_gated_decode(s, *([GOOD] * 5), None) == rc


def test_gated_pointers(lib):
    assert lib.ssd_gated_scan(None, *([GOOD] * 7), 1 << 40, None) == 1
    # which arguments are required, and which alignment each has
    for call, count, required, elem in ((lib.ssd_gated_scan, 6, (0, 1, 3), (0, 1)),
                                        (lib.ssd_gated_scan_bwd, 8, (0, 1, 2, 3, 5, 6), (0, 1)),
                                        (lib.ssd_gated_decode, 5, (0, 1, 2, 3, 4), (0, 1))):
        rest = () if call is lib.ssd_gated_decode else (GOOD, 1 << 40)
        for k in range(count):
            args = [GOOD] * count
            if k in required:
                args[k] = None
                assert call(gated(), *args, *rest, None) == 1, (call.__name__, k)
            args[k] = ODD if k in elem else OK_ELEM
            assert call(gated(), *args, *rest, None) == 3, (call.__name__, k)
            if k in elem:
                args[k] = OK_ELEM
                assert call(gated(io_dtype=ssd.SSD_F32), *args, *rest, None) == 3


def test_gated_workspace(lib):
    s = gated(batch=1, seqlen=1 << 20)   # two columns: the sequence is cut into segments
    for query, call, count in ((lib.ssd_gated_workspace_bytes, lib.ssd_gated_scan, 6),
                               (lib.ssd_gated_bwd_workspace_bytes, lib.ssd_gated_scan_bwd, 8)):
        n = query(s)
        assert n > 0
        assert call(s, *([GOOD] * count), None, n, None) == 6 and b"workspace" in lib.ssd_last_error()
        assert call(s, *([GOOD] * count), GOOD, n - 1, None) == 6
        assert call(s, *([GOOD] * count), ctypes.c_void_p(0x100010), n, None) == 3
    assert lib.ssd_gated_workspace_bytes(gated(batch=8, seqlen=8192, dim=5120)) == 0


BAD_NORM = [(dict(batch=0), 1), (dict(seqlen=0), 1), (dict(channels=0), 1), (dict(ngroups=0), 1), (dict(ngroups=5), 1),
            (dict(io_dtype=2), 1), (dict(act=4), 1), (dict(act=-1), 1), (dict(flags=2), 1), (dict(eps=-1.0), 1),
            (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(x_stride=95), 1), (dict(z_stride=5), 1),
            (dict(channels=1 << 21), 2), (dict(seqlen=1 << 45), 2), (dict(batch=1 << 30), 2)]


@pytest.mark.parametrize("bad,rc", BAD_NORM)
def test_norm_shapes(lib, bad, rc):
    s = norm(**bad)
    assert lib.ssd_norm_workspace_bytes(s) == 0 and lib.ssd_norm_bwd_workspace_bytes(s) == 0
    assert lib.ssd_group_norm(s, *([GOOD] * 8), 1 << 40, None) == rc and lib.ssd_last_error()
    assert lib.ssd_group_norm_bwd(s, *([GOOD] * 12), 1 << 40, None) == rc


def test_norm_pointers(lib):
    assert lib.ssd_group_norm(None, *([GOOD] * 8), 1 << 40, None) == 1
    for call, count, required, elem in ((lib.ssd_group_norm, 7, (0, 1, 4), (0, 1)),
                                        (lib.ssd_group_norm_bwd, 11, (0, 1, 4, 5, 6, 7, 8), (0, 1))):
        for k in range(count):
            args = [GOOD] * (count + 1)
            if k in required:
                args[k] = None
                assert call(norm(), *args, 1 << 40, None) == 1, (call.__name__, k)
            args[k] = ODD if k in elem else OK_ELEM
            assert call(norm(), *args, 1 << 40, None) == 3, (call.__name__, k)
    # z is asked for by the gates alone, the mean not by the root mean square
    args = [GOOD] * 8
    args[0] = ODD
    args[1] = None
    assert lib.ssd_group_norm(norm(act=1), *args, 1 << 40, None) == 3


def test_norm_workspace(lib):
    s = norm(batch=2, seqlen=1 << 20, channels=4096, ngroups=8)
    for query, call, count in ((lib.ssd_norm_workspace_bytes, lib.ssd_group_norm, 7),
                               (lib.ssd_norm_bwd_workspace_bytes, lib.ssd_group_norm_bwd, 11)):
        n = query(s)
        if n == 0:
            continue
        assert call(s, *([GOOD] * count), None, n, None) == 6 and b"workspace" in lib.ssd_last_error()
        assert call(s, *([GOOD] * count), GOOD, n - 1, None) == 6
        assert call(s, *([GOOD] * count), ctypes.c_void_p(0x100010), n, None) == 3
