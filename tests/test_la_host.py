"""Host side of linear attention's calls and of the batch plan (no GPU): exports, sizes, refusals, NVTX ranges.

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
HP, GN = 8 * 128, 4 * 128


@pytest.fixture(scope="module")
def lib():
    bld.build()
    return bd.lib()


STEP = ["desc", "pool", "stride", "slots", "ids", "scratch", "batch", "ntok", "xbc", "decay", "norm", "kw", "qw", "eps", "pos", "freq",
        "rot", "inter", "scale", "y", "err", "stream"]
STEP_OK = dict(pool=P, stride=HP * 128, slots=16, ids=P, scratch=None, batch=2, ntok=1, xbc=P, decay=P, norm=1, kw=P, qw=None, eps=1e-6,
               pos=P, freq=P, rot=64, inter=0, scale=1.0, y=P, err=None, stream=None)
PREP = ["desc", "k", "ks", "q", "qs", "tokens", "norm", "kw", "qw", "eps", "pos", "freq", "rot", "inter", "ko", "kos", "qo", "qos", "stream"]
PREP_OK = dict(k=P, ks=HP + 2 * GN, q=P, qs=GN, tokens=3, norm=1, kw=None, qw=None, eps=1e-6, pos=P, freq=P, rot=128, inter=0, ko=2 * P,
               kos=GN, qo=2 * P, qos=GN, stream=None)
SCAN = ["desc", "pool", "stride", "slots", "cu", "nseq", "T", "ids", "init", "ckpt", "max_ckpt", "interval", "v", "vs", "k", "ks", "q",
        "qs", "decay", "scale", "y", "ws", "ws_bytes", "err", "stream"]
SCAN_OK = dict(pool=P, stride=HP * 128, slots=16, cu=P, nseq=2, T=100, ids=P, init=None, ckpt=None, max_ckpt=0, interval=0, v=P, vs=HP,
               k=P, ks=GN, q=P, qs=GN, decay=P, scale=1.0, y=P, ws=P, ws_bytes=1 << 40, err=None, stream=None)
PLAN = ["new", "past", "rows", "table", "tstride", "cols", "block", "slots", "max_tokens", "max_ckpt", "cu", "ids", "init", "src", "dst",
        "ckpt", "pos", "tok", "err", "stream"]
PLAN_OK = dict(new=P, past=P, rows=2, table=P, tstride=4, cols=4, block=64, slots=9, max_tokens=10, max_ckpt=2, cu=P, ids=P, init=None,
               src=None, dst=None, ckpt=P, pos=None, tok=None, err=None, stream=None)
CASES = {"la_state_update": (STEP, STEP_OK), "la_qk_norm_rope": (PREP, PREP_OK), "la_chunk_scan": (SCAN, SCAN_OK)}


def _call(lib, name, desc=None, **change):
    order, good = CASES.get(name) or (PLAN, PLAN_OK)
    args = dict(good, desc=ctypes.byref(desc) if desc is not None else None, **change)
    return getattr(lib, name)(*[args[n] for n in order])


E, U, A = bd.MAMBA_EINVAL, bd.MAMBA_EUNSUPPORTED, bd.MAMBA_EALIGN
REFUSED = [
    *[("la_state_update", {a: None}, E) for a in ("pool", "ids", "xbc", "decay", "y", "pos", "freq")],
    *[("la_state_update", {"batch": b}, E) for b in (-1, 65536)], *[("la_state_update", {"ntok": n}, E) for n in (0, 9)],
    ("la_state_update", {"stride": HP * 128 - 8}, E), ("la_state_update", {"slots": 0}, E), ("la_state_update", {"rot": -16}, E),
    ("la_state_update", {"eps": -1.0}, E), ("la_state_update", {"eps": float("nan")}, E),
    ("la_state_update", {"rot": 144}, U), ("la_state_update", {"rot": 24}, U),
    ("la_state_update", {"pool": P + 8}, A), ("la_state_update", {"xbc": P + 2}, A), ("la_state_update", {"y": P + 1}, A),
    ("la_state_update", {"stride": HP * 128 + 4}, A),
    *[("la_qk_norm_rope", {a: None}, E) for a in ("k", "q", "ko", "qo", "pos", "freq")],
    ("la_qk_norm_rope", {"tokens": -1}, E), *[("la_qk_norm_rope", {a: GN - 8}, E) for a in ("ks", "qs", "kos", "qos")],
    ("la_qk_norm_rope", {"ko": P}, E), ("la_qk_norm_rope", {"qo": P, "qos": GN + 8}, E),  # in place, but rows at another distance
    ("la_qk_norm_rope", {"rot": 130}, U), *[("la_qk_norm_rope", {a: GN + 4}, A) for a in ("qs", "kos", "qos")],
    *[("la_qk_norm_rope", {a: 3 * P + 8}, A) for a in ("k", "q", "ko", "qo")],
    *[("la_chunk_scan", {a: None}, E) for a in ("pool", "cu", "ids", "decay", "ws", "v", "k", "q", "y")],
    *[("la_chunk_scan", {"nseq": n}, E) for n in (-1, 65536)], ("la_chunk_scan", {"T": -1}, E), ("la_chunk_scan", {"stride": 100}, E),
    ("la_chunk_scan", {"vs": HP - 8}, E), ("la_chunk_scan", {"ks": GN - 8}, E), ("la_chunk_scan", {"qs": GN - 8}, E),
    *[("la_chunk_scan", {"ckpt": P, "interval": i, "max_ckpt": m}, E) for i, m in ((0, 2), (-128, 2), (64, 2), (128, 0))],
    ("la_chunk_scan", {"ws_bytes": 100}, bd.MAMBA_ENOSPACE),
    *[("la_chunk_scan", {a: P + 8}, A) for a in ("pool", "v", "k", "q", "y", "ws")],
    *[("la_chunk_scan", {a: n}, A) for a, n in (("vs", HP + 4), ("ks", GN + 4), ("qs", GN + 4), ("stride", HP * 128 + 4))],
    *[("mamba_batch_plan", {a: None}, E) for a in ("new", "past", "table", "cu", "ids")],
    *[("mamba_batch_plan", {"rows": r}, E) for r in (-1, 65536)], ("mamba_batch_plan", {"max_tokens": -1}, E),
    ("mamba_batch_plan", {"block": -1}, E), ("mamba_batch_plan", {"slots": 0}, E), ("mamba_batch_plan", {"cols": 0}, E),
    ("mamba_batch_plan", {"tstride": 3}, E), ("mamba_batch_plan", {"src": P}, E), ("mamba_batch_plan", {"dst": P}, E),
    ("mamba_batch_plan", {"max_ckpt": 0}, E),
]


@pytest.mark.parametrize("name,change,status", REFUSED, ids=lambda x: str(x))
def test_a_bad_argument_is_refused(lib, name, change, status):
    assert _call(lib, name, bd.layer_desc(SHAPE), **change) == status


@pytest.mark.parametrize("name", CASES)
def test_bad_layers_are_refused(lib, name):
    assert _call(lib, name) == E
    ragged = wl.LayerShape(nheads=8, head_dim=128, d_state=128, n_groups=3)
    assert _call(lib, name, bd.layer_desc(ragged)) == E
    odd = wl.LayerShape(nheads=4, head_dim=128, d_state=96, n_groups=4)
    wide = dict(rot=96) if name == "la_qk_norm_rope" else {}
    assert _call(lib, name, bd.layer_desc(odd), **wide) == U


@pytest.mark.parametrize("name,change", [("la_state_update", dict(batch=0, pool=None, ids=None, xbc=None, y=None)),
                                         ("la_qk_norm_rope", dict(tokens=0, k=None, q=None)), ("la_chunk_scan", dict(nseq=0, pool=None, v=None))])
def test_a_call_of_no_rows_is_ok_and_touches_nothing(lib, name, change):
    assert _call(lib, name, bd.layer_desc(SHAPE), **change) == bd.MAMBA_OK


def test_workspace_sizes(lib):
    d = bd.layer_desc(SHAPE)
    assert bd.la_chunk_scan_workspace_bytes(d, -1, 1) == 0 == bd.la_chunk_scan_workspace_bytes(d, 1, -1)
    assert 0 < bd.la_chunk_scan_workspace_bytes(d, 0, 1) <= 4096
    # one long prompt is cut into as many segments as make a block an SM: 19 of 8 heads, a state and the initial one each
    one = bd.la_chunk_scan_workspace_bytes(d, 100000, 1)
    assert 19 * 8 * 128 * 128 * 4 <= one <= 24 * 8 * 128 * 128 * 4
    # enough sequences need no cutting, and no states in the workspace
    assert bd.la_chunk_scan_workspace_bytes(d, 100000, 20) <= 4096
    assert bd.la_chunk_scan_workspace_bytes(d, 100000, 65535) <= 32 * 65535 + 4096


def test_the_header_declares_what_the_binding_has(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mamba_state.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*\w+\s+(la_\w+|mamba_batch_plan)\s*\(", text, flags=re.M))
    assert names == {n for n in bd.SIGNATURES if n.startswith("la_") or n == "mamba_batch_plan"} and len(names) == 5
    for n in names:
        assert hasattr(lib, n)


def test_each_call_opens_and_closes_its_nvtx_range(lib, tmp_path):
    if os.environ.get("MAMBA_NVTX", "1") == "0":
        pytest.skip("library built without NVTX ranges")
    probe = str(tmp_path / "libnvtx_probe.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-Wall", os.path.join(HERE, "nvtx_probe.c"), "-o", probe], check=True)
    calls = [*CASES, "mamba_batch_plan"]
    script = (f"import ctypes\nlib = ctypes.CDLL({bld.LIB!r})\n"
              f"for n in {calls!r}:\n    assert getattr(lib, n)(*[ctypes.c_void_p(0)] * 32) < 0\n"
              f"p = ctypes.CDLL({probe!r})\np.nvtx_probe_log.restype = ctypes.c_char_p\nprint(p.nvtx_probe_log().decode())")
    r = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, NVTX_INJECTION64_PATH=probe))
    assert r.returncode == 0, r.stderr
    assert [x for x in r.stdout.splitlines() if x] == [e for n in calls for e in ("+" + n, "-")]


def test_the_workspace_of_no_sequences(tmp_path):
    """Of any layer, in a process of its own, which a division by no blocks would end."""
    script = (f"import sys\nsys.path.insert(0, {ROOT!r})\nfrom recurrent_state_update_gb300 import binding as bd, workloads as wl\n"
              "for heads in (1, 76, 152, 153, 160, 1000):\n"
              "    d = bd.layer_desc(wl.LayerShape(nheads=heads, head_dim=64, d_state=128, n_groups=1))\n"
              "    for tokens in (0, 1, 100, 1 << 20):\n"
              "        assert 0 < bd.la_chunk_scan_workspace_bytes(d, tokens, 0) <= 4096\n")
    r = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])


def test_more_tokens_than_their_counters_hold_are_refused(lib):
    """Loops step 16 or 128 tokens past the last one and sequences of more than a whole segment are not expected, so that the most
    tokens are 2^31 - 128.  (The workspace given here is too small, which is checked after that.)"""
    d, most = bd.layer_desc(SHAPE), 2 ** 31 - 128
    assert bd.la_chunk_scan_workspace_bytes(d, most, 1) > 0
    assert _call(lib, "la_chunk_scan", d, T=most, ws_bytes=0) == bd.MAMBA_ENOSPACE
    for tokens in (most + 1, 2 ** 31 - 1):
        assert bd.la_chunk_scan_workspace_bytes(d, tokens, 1) == 0
        assert _call(lib, "la_chunk_scan", d, T=tokens, ws_bytes=0) == E


@pytest.mark.parametrize("field,value", [("conv_kernel", 0), ("conv_kernel", 99), ("num_spec", -1), ("conv_dtype", 7),
                                         ("conv_dtype", bd.MAMBA_F32), ("dt_dtype", -1)])
def test_fields_of_the_convolution_and_the_steps_are_not_looked_at(lib, field, value):
    """These layers have neither.  Each call gets as far as an argument that it refuses with another status."""
    d, plain = bd.layer_desc(SHAPE), bd.layer_desc(SHAPE)
    setattr(d, field, value)
    assert bd.la_chunk_scan_workspace_bytes(d, 5000, 2) == bd.la_chunk_scan_workspace_bytes(plain, 5000, 2) > 0
    assert _call(lib, "la_state_update", d, y=P + 1) == A
    assert _call(lib, "la_chunk_scan", d, ws_bytes=0) == bd.MAMBA_ENOSPACE
    assert _call(lib, "la_qk_norm_rope", d, k=3 * P + 8) == A
    assert _call(lib, "la_state_update", d, batch=0) == _call(lib, "la_chunk_scan", d, nseq=0) == _call(lib, "la_qk_norm_rope", d, tokens=0) == 0


@pytest.mark.parametrize("field", ["state_dtype", "act_dtype", "nheads", "head_dim", "d_state", "n_groups"])
def test_the_other_fields_are(lib, field):
    d = bd.layer_desc(SHAPE)
    setattr(d, field, -1)
    for name in CASES:
        assert _call(lib, name, d) == E
    assert bd.la_chunk_scan_workspace_bytes(d, 5000, 2) == 0


@pytest.mark.parametrize("heads,head_dim,d_state", [(1, 64, 64), (8, 128, 128), (32, 128, 128), (40, 64, 128), (12, 32, 64)])
def test_a_workspace_of_the_most_tokens_serves_fewer(lib, heads, head_dim, d_state):
    """A program asks once, for the most tokens of a batch."""
    d = bd.layer_desc(wl.LayerShape(nheads=heads, head_dim=head_dim, d_state=d_state, n_groups=1), state=wl.F32)
    row = heads * (head_dim + 2 * d_state)
    for nseq in (1, 2, 5, 30):
        sizes = [bd.la_chunk_scan_workspace_bytes(d, t, nseq) for t in range(0, 120000, 37)]
        assert sizes == sorted(sizes)
        for t in (1, 511, 513, 2433, 19457, 77777):  # refused for its keys' address, not for its workspace
            assert _call(lib, "la_chunk_scan", d, T=t, nseq=nseq, vs=row, ks=row, qs=row, k=P + 8, stride=heads * head_dim * d_state,
                         ws_bytes=max(bd.la_chunk_scan_workspace_bytes(d, u, nseq) for u in range(t, t + 2000, 100))) == A
