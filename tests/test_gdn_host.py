"""Host side of the gated delta rule's calls (no GPU): exports, sizes, refusals, NVTX ranges.

A refused call returns before it touches the device, so made-up addresses are safe here."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SHAPE = wl.LayerShape(nheads=8, head_dim=128, d_state=128, n_groups=4)
P = 1 << 20  # an aligned address nothing reads


@pytest.fixture(scope="module")
def lib():
    bld.build()
    return bd.lib()


STEP = ["desc", "pool", "stride", "slots", "ids", "scratch", "batch", "ntok", "xbc", "dt", "beta", "A", "bias", "sp",
        "sg", "l2", "scale", "y", "err", "stream"]
STEP_OK = dict(pool=P, stride=8 * 128 * 128, slots=16, ids=P, scratch=None, batch=2, ntok=1, xbc=P, dt=P, beta=P, A=P,
               bias=None, sp=1, sg=1, l2=1, scale=1.0, y=P, err=None, stream=None)
INT8 = ["desc", "store", "entries", "ids", "batch", "xbc", "dt", "beta", "A", "bias", "sp", "sg", "l2", "scale", "y",
        "err", "stream"]
INT8_OK = dict(store=P, entries=4, ids=P, batch=2, xbc=P, dt=P, beta=P, A=P, bias=None, sp=1, sg=1, l2=1, scale=1.0,
               y=P, err=None, stream=None)
SCAN = ["desc", "pool", "stride", "slots", "cu", "nseq", "T", "ids", "init", "ckpt", "max_ckpt", "interval", "v", "k",
        "q", "dt", "beta", "A", "bias", "sp", "sg", "l2", "scale", "y", "ws", "ws_bytes", "err", "stream"]
SCAN_OK = dict(pool=P, stride=8 * 128 * 128, slots=16, cu=P, nseq=2, T=100, ids=P, init=None, ckpt=None, max_ckpt=0,
               interval=0, v=P, k=P, q=P, dt=P, beta=P, A=P, bias=None, sp=1, sg=1, l2=1, scale=1.0, y=P, ws=P,
               ws_bytes=1 << 40, err=None, stream=None)


def _call(lib, name, order, good, desc, **change):
    args = dict(good, desc=ctypes.byref(desc) if desc is not None else None, **change)
    return getattr(lib, name)(*[args[n] for n in order])


CASES = {"gdn_state_update": (STEP, STEP_OK), "gdn_state_update_int8": (INT8, INT8_OK), "gdn_chunk_scan": (SCAN, SCAN_OK)}
REFUSED = [
    *[(n, a, None, bd.MAMBA_EINVAL) for n in CASES for a in ("ids", "A")],
    *[("gdn_state_update", a, None, bd.MAMBA_EINVAL) for a in ("pool", "xbc", "dt", "beta", "y")],
    *[("gdn_state_update_int8", a, None, bd.MAMBA_EINVAL) for a in ("store", "xbc", "dt", "beta", "y")],
    *[("gdn_chunk_scan", a, None, bd.MAMBA_EINVAL) for a in ("pool", "cu", "v", "k", "q", "dt", "beta", "y", "ws")],
    ("gdn_state_update", "batch", -1, bd.MAMBA_EINVAL), ("gdn_state_update", "batch", 65536, bd.MAMBA_EINVAL),
    ("gdn_state_update", "ntok", 0, bd.MAMBA_EINVAL), ("gdn_state_update", "ntok", 9, bd.MAMBA_EINVAL),
    ("gdn_state_update", "stride", 8 * 128 * 128 - 8, bd.MAMBA_EINVAL), ("gdn_state_update", "slots", 0, bd.MAMBA_EINVAL),
    ("gdn_state_update", "pool", P + 8, bd.MAMBA_EALIGN), ("gdn_state_update", "xbc", P + 2, bd.MAMBA_EALIGN),
    ("gdn_state_update", "y", P + 1, bd.MAMBA_EALIGN), ("gdn_state_update", "stride", 8 * 128 * 128 + 4, bd.MAMBA_EALIGN),
    ("gdn_state_update_int8", "batch", 65536, bd.MAMBA_EINVAL), ("gdn_state_update_int8", "entries", 0, bd.MAMBA_EINVAL),
    ("gdn_state_update_int8", "store", P + 8, bd.MAMBA_EALIGN), ("gdn_state_update_int8", "xbc", P + 8, bd.MAMBA_EALIGN),
    ("gdn_chunk_scan", "nseq", -1, bd.MAMBA_EINVAL), ("gdn_chunk_scan", "nseq", 65536, bd.MAMBA_EINVAL),
    ("gdn_chunk_scan", "T", -1, bd.MAMBA_EINVAL), ("gdn_chunk_scan", "stride", 100, bd.MAMBA_EINVAL),
    ("gdn_chunk_scan", "ws_bytes", 100, bd.MAMBA_ENOSPACE), ("gdn_chunk_scan", "ws", P + 8, bd.MAMBA_EALIGN),
    *[("gdn_chunk_scan", a, P + 8, bd.MAMBA_EALIGN) for a in ("pool", "v", "k", "q", "y")],
]


@pytest.mark.parametrize("name,arg,value,status", REFUSED)
def test_a_bad_argument_is_refused(lib, name, arg, value, status):
    order, good = CASES[name]
    assert _call(lib, name, order, good, bd.layer_desc(SHAPE), **{arg: value}) == status


@pytest.mark.parametrize("interval,max_ckpt", [(0, 2), (-64, 2), (100, 2), (64, 0)])
def test_bad_checkpoint_arguments_are_refused(lib, interval, max_ckpt):
    assert _call(lib, "gdn_chunk_scan", SCAN, SCAN_OK, bd.layer_desc(SHAPE), ckpt=P, interval=interval,
                 max_ckpt=max_ckpt) == bd.MAMBA_EINVAL


@pytest.mark.parametrize("name", CASES)
def test_bad_layers_are_refused(lib, name):
    order, good = CASES[name]
    assert _call(lib, name, order, good, None) == bd.MAMBA_EINVAL
    ragged = wl.LayerShape(nheads=8, head_dim=128, d_state=128, n_groups=3)
    assert _call(lib, name, order, good, bd.layer_desc(ragged)) == bd.MAMBA_EINVAL
    odd = wl.LayerShape(nheads=4, head_dim=96, d_state=128, n_groups=4)
    assert _call(lib, name, order, good, bd.layer_desc(odd)) == bd.MAMBA_EUNSUPPORTED


@pytest.mark.parametrize("name,arg", [("gdn_state_update", "batch"), ("gdn_state_update_int8", "batch"),
                                      ("gdn_chunk_scan", "nseq")])
def test_a_call_of_no_rows_is_ok_and_touches_nothing(lib, name, arg):
    order, good = CASES[name]
    none = {k: None for k in ("pool", "store", "ids", "xbc", "cu", "v", "y") if k in good}
    assert _call(lib, name, order, good, bd.layer_desc(SHAPE), **{arg: 0}, **none) == bd.MAMBA_OK


def test_workspace_sizes(lib):
    d = bd.layer_desc(SHAPE)
    assert bd.gdn_chunk_scan_workspace_bytes(d, -1, 1) == 0 == bd.gdn_chunk_scan_workspace_bytes(d, 1, -1)
    sizes = [bd.gdn_chunk_scan_workspace_bytes(d, t, n) for t, n in ((0, 1), (1000, 1), (1000, 9), (100000, 9))]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_the_header_declares_what_the_binding_has(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mamba_state.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*\w+\s+(gdn_\w+)\s*\(", text, flags=re.M))
    assert names == {n for n in bd.SIGNATURES if n.startswith("gdn_")} and len(names) == 4
    for n in names:
        assert hasattr(lib, n)


def test_each_call_opens_and_closes_its_nvtx_range(lib, tmp_path):
    if os.environ.get("MAMBA_NVTX", "1") == "0":
        pytest.skip("library built without NVTX ranges")
    probe = str(tmp_path / "libnvtx_probe.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-Wall", os.path.join(HERE, "nvtx_probe.c"), "-o", probe], check=True)
    script = (f"import ctypes\nlib = ctypes.CDLL({bld.LIB!r})\n"
              f"for n in {list(CASES)!r}:\n    assert getattr(lib, n)(*[ctypes.c_void_p(0)] * 32) < 0\n"
              f"p = ctypes.CDLL({probe!r})\np.nvtx_probe_log.restype = ctypes.c_char_p\nprint(p.nvtx_probe_log().decode())")
    r = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, NVTX_INJECTION64_PATH=probe))
    assert r.returncode == 0, r.stderr
    assert [x for x in r.stdout.splitlines() if x] == [e for n in CASES for e in ("+" + n, "-")]
