"""Host-side tests of libseqops.so: exports, validation and the binding's checks.  No GPU needed and
no kernel launched: calls that must be refused run in a child process that sees no GPU, so that even a
validation bug could not turn a stand-in pointer into a launch."""

import ctypes
import json
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sequence_ops.h")

sq = pytest.importorskip("causal_conv1d_verify_amd._seqops")
from causal_conv1d_verify_amd import _lib as base  # noqa: E402

EINVAL, ENOTSUP = base.CV_EINVAL, base.CV_ENOTSUP
STRUCTS = (("sq_scan_shape_t", sq.SqScanShape), ("sq_scan_data_t", sq.SqScanData),
           ("sq_scan_info_t", sq.SqScanInfo), ("sq_rotary_shape_t", sq.SqRotaryShape),
           ("sq_accept_shape_t", sq.SqAcceptShape))


def _lib():
    if not os.path.exists(sq.LIB_PATH):
        pytest.skip("libseqops.so not built (run __graft_entry__.build())")
    return sq.load()


def test_header_binding_and_library_agree():
    lib = _lib()
    text = open(HEADER).read()
    declared = set(re.findall(r"^\s*CV_API\s+(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, re.M))
    assert declared == set(sq.EXPORTS)
    res = subprocess.run(["nm", "-D", "--defined-only", sq.LIB_PATH], capture_output=True, text=True, check=True)
    assert set(re.findall(r"\bT (\w+)$", res.stdout, re.M)) == declared
    assert lib.seqops_abi_version() == int(re.search(r"#define SEQUENCE_OPS_ABI_VERSION (\d+)", text).group(1))


def test_struct_layouts(tmp_path):
    """The ctypes structures have the C structures' sizes and offsets."""
    src = tmp_path / "layout.c"
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "sequence_ops.h"', "int main(void) {"]
    for name, cls in STRUCTS:
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    src.write_text("\n".join(lines) + "return 0;}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", f"-I{ROOT}/include", str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    got = dict(line.rsplit(" ", 1) for line in out.splitlines())
    for name, cls in STRUCTS:
        assert int(got[name]) == ctypes.sizeof(cls)
        for f in cls._fields_:
            assert int(got[f"{name}.{f[0]}"]) == getattr(cls, f[0]).offset


_CHILD = r"""
import ctypes, json, sys
sys.path.insert(0, sys.argv[1])
from causal_conv1d_verify_amd import _lib as B, _seqops as L
lib = L.load()
A = 0x10000
res = {}
def note(name, rc):
    res[name] = [rc, lib.seqops_last_error().decode()]

def shape(**kw):
    d = dict(n_seq=4, T=8, d=64, d_state=16, x_dtype=B.CV_BF16, state_dtype=B.CV_F32, n_slots=4, softplus=1,
             x_seq_stride=512, x_tok_stride=64, dt_seq_stride=512, dt_tok_stride=64, z_seq_stride=512, z_tok_stride=64,
             b_seq_stride=128, b_tok_stride=16, c_seq_stride=128, c_tok_stride=16, out_seq_stride=512, out_tok_stride=64,
             state_slot_stride=1024)
    d.update(kw)
    return L.SqScanShape(**d)
def data(**kw):
    d = {f[0]: A for f in L.SqScanData._fields_}
    d.update(kw)
    return L.SqScanData(**d)
def prefill(name, s, p=None, state=A, slot=A, cu=A, init=A, out=A, ws=A, size=1 << 40):
    note("prefill:" + name, lib.selscan_prefill(s, p or data(), state, slot, cu, init, out, ws, size, None))
def update(name, s, p=None, state=A, slot=A, out=A):
    note("update:" + name, lib.selscan_update(s, p or data(), state, slot, out, None))
def verify(name, s, p=None, state=A, slot=A, out=A):
    note("verify:" + name, lib.selscan_verify(s, p or data(), state, slot, out, None))
def commit(name, s, p=None, state=A, slot=A, num=A):
    note("commit:" + name, lib.selscan_commit(s, p or data(), state, slot, num, None))
ALL = (prefill, update, verify, commit)
bad = dict(n_seq=dict(n_seq=-1), T=dict(T=0), d0=dict(d=0), N0=dict(d_state=0), d_odd=dict(d=60), N_odd=dict(d_state=12),
           N_big=dict(d_state=72), softplus=dict(softplus=2), x_type=dict(x_dtype=7), s_type=dict(state_dtype=-1),
           pair=dict(x_dtype=B.CV_F32, state_dtype=B.CV_BF16), n_slots=dict(n_slots=-1), x_negative=dict(x_tok_stride=-8),
           b_negative=dict(b_tok_stride=-1), dt_unaligned=dict(dt_tok_stride=68), slot_short=dict(state_slot_stride=512),
           slot_unaligned=dict(state_slot_stride=1026))
for name, kw in bad.items():
    for f in ALL:
        f(name, shape(**kw))
    note("workspace:" + name, lib.selscan_prefill_workspace(shape(**kw)))
    note("describe:" + name, lib.selscan_describe(1, shape(**kw), ctypes.byref(L.SqScanInfo())))
for name, kw in dict(z_unaligned=dict(z_tok_stride=68), out_unaligned=dict(out_tok_stride=68), out_toks=dict(out_tok_stride=56),
                     c_negative=dict(c_tok_stride=-2)).items():
    for f in (prefill, update, verify):
        f(name, shape(**kw))
update("out_rows", shape(out_seq_stride=64)); verify("out_rows", shape(out_seq_stride=64))
for f in (update, verify, commit):
    f("T33", shape(T=33))
for name in ("x", "dt", "z", "b", "c", "out"):
    prefill("far_" + name, shape(T=100, **{name + "_tok_stride": 1 << 30}))
for f in ALL:
    for p in ("x", "dt", "A", "B"):
        f("null_" + p, shape(), data(**{p: None}))
    for p in ("x", "dt", "A", "dt_bias"):
        f("off_" + p, shape(), data(**{p: A + 8}))
    f("off_B", shape(), data(B=A + 1))
    f("null_state", shape(), state=None)
    f("off_state", shape(), state=A + 8)
    f("off_slot", shape(), slot=A + 2)
    f("short_slots", shape(n_slots=3), slot=None)
    f("empty", shape(n_seq=0))
    if f is not commit:
        f("null_C", shape(), data(C=None))
        f("off_z", shape(), data(z=A + 4)); f("off_D", shape(), data(D=A + 4)); f("off_C", shape(), data(C=A + 1))
        f("null_out", shape(), out=None); f("off_out", shape(), out=A + 8)
prefill("tokens", shape(tokens=-1)); prefill("null_cu", shape(), cu=None); prefill("off_init", shape(), init=A + 1)
commit("off_num", shape(), num=A + 1)
long = shape(n_seq=1, T=4096, tokens=4096)
need = lib.selscan_prefill_workspace(long)
res["need"] = need
if need > 0:
    prefill("ws_small", long, size=need - 1); prefill("ws_null", long, ws=None); prefill("ws_off", long, ws=A + 8)
note("describe:null", lib.selscan_describe(0, shape(), None)); note("describe:call", lib.selscan_describe(4, shape(), ctypes.byref(L.SqScanInfo())))
for name in ("prefill", "update", "verify", "commit"):
    fn = getattr(lib, "selscan_" + name)
    n = len(fn.argtypes)
    note(name + ":null_shape", fn(*([None] * (n - 2)), *([0, None] if name == "prefill" else [None, None])))
    a = [shape(), None] + [A] * (n - 3) + [None]
    if name == "prefill":
        a[-2] = 1 << 40
    note(name + ":null_data", fn(*a))

def rshape(**kw):
    d = dict(tokens=4, q_heads=2, k_heads=2, dim=64, rot=32, eps=1e-6, x_dtype=B.CV_BF16, interleaved=0, wide_positions=1)
    for n in ("q", "k", "q_out", "k_out"):
        d[n + "_tok_stride"], d[n + "_head_stride"] = 128, 64
    d.update(kw)
    return L.SqRotaryShape(**d)
def rotary(name, s, q=A, k=A, qw=A, kw=A, pos=A, freq=A, qo=A, ko=A):
    note("rotary:" + name, lib.norm_rotary(s, q, k, qw, kw, pos, freq, qo, ko, None))
for name, kw in dict(tokens=dict(tokens=-1), q_heads=dict(q_heads=0), k_heads=dict(k_heads=-1), dim0=dict(dim=0), rot=dict(rot=-16),
                     rot_over=dict(rot=80), dim_odd=dict(dim=72, rot=0), dim_big=dict(dim=272, rot=16), rot_odd=dict(rot=24),
                     many_heads=dict(q_heads=1 << 21), eps=dict(eps=-1.0), eps_nan=dict(eps=float("nan")), x_type=dict(x_dtype=3),
                     q_negative=dict(q_tok_stride=-8), k_unaligned=dict(k_head_stride=68), out_unaligned=dict(q_out_tok_stride=132),
                     out_heads=dict(q_out_head_stride=56), k_out_toks=dict(k_out_tok_stride=64)).items():
    rotary(name, rshape(**kw))
for p in ("q", "k", "pos", "freq", "qo", "ko"):
    rotary("null_" + p, rshape(), **{p: None})
for p in ("q", "k", "qw", "kw", "qo", "ko"):
    rotary("off_" + p, rshape(), **{p: A + 8})
rotary("off_pos", rshape(), pos=A + 4); rotary("off_freq", rshape(), freq=A + 2)
rotary("null_shape", None)
rotary("empty", rshape(tokens=0), *[None] * 8)

def ashape(**kw):
    d = dict(n_seq=4, T=8, vocab=1000, p_dtype=B.CV_F32, tokens_stride=8, parent_stride=8, uniform_stride=8, path_stride=8,
             target_seq_stride=8000, target_tok_stride=1000, draft_seq_stride=7000, draft_tok_stride=1000)
    d.update(kw)
    return L.SqAcceptShape(**d)
def accept(name, s, tokens=A, parent=None, target=A, draft=A, uniform=A, slot=A, num=A, nxt=A, last=A, path=A, ws=A, size=1 << 40):
    note("accept:" + name, lib.accept_drafts(s, tokens, parent, target, draft, uniform, slot, num, nxt, last, path, ws, size, None))
for name, kw in dict(n_seq=dict(n_seq=-1), T=dict(T=0), vocab=dict(vocab=0), T33=dict(T=33), vocab_big=dict(vocab=(1 << 24) + 1),
                     p_type=dict(p_dtype=5), tokens_negative=dict(tokens_stride=-1), target_negative=dict(target_tok_stride=-4),
                     path_rows=dict(path_stride=7)).items():
    accept(name, ashape(**kw))
    if name not in ("path_rows",):
        note("accept_workspace:" + name, lib.accept_drafts_workspace(ashape(**kw)))
accept("draft_negative", ashape(draft_seq_stride=-1))
accept("tree_pair", ashape(), parent=A)
accept("parent_negative", ashape(parent_stride=-1), parent=A, draft=None)
for p in ("tokens", "target", "uniform", "num", "nxt", "ws"):
    accept("null_" + p, ashape(), **{p: None})
for p in ("tokens", "target", "draft", "uniform", "slot", "num", "nxt", "last", "path"):
    accept("off_" + p, ashape(), **{p: A + 2})
accept("off_parent", ashape(), parent=A + 2, draft=None)
accept("off_ws", ashape(), ws=A + 8)
accept("ws_small", ashape(), size=lib.accept_drafts_workspace(ashape()) - 1)
accept("null_shape", None)
accept("empty", ashape(n_seq=0))
print(json.dumps(res))
"""


@pytest.fixture(scope="module")
def refusals():
    _lib()
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    run = subprocess.run([sys.executable, "-c", _CHILD, ROOT], capture_output=True, text=True, env=env, timeout=300)
    assert run.returncode == 0, run.stderr[-3000:]
    return json.loads(run.stdout.strip().splitlines()[-1])


def test_bad_calls_are_refused(refusals):
    assert refusals.pop("need") > 0
    unsupported = {"d_odd", "N_odd", "N_big", "pair", "T33", "dim_odd", "dim_big", "rot_odd", "many_heads", "vocab_big",
                   "tree_pair", "ws_off"}
    for name, (rc, detail) in refusals.items():
        short = name.split(":")[1]
        if short == "empty":
            assert rc == 0, (name, rc, detail)
            continue
        want = ENOTSUP if short in unsupported or short.startswith(("off_", "far_")) or "unaligned" in short else EINVAL
        assert rc == want, (name, rc, detail)
        assert detail, name
    assert len(refusals) > 230


def test_descriptions():
    """Which kernel and how many launches a call gets."""
    lib = _lib()

    def info(call, **kw):
        d = dict(n_seq=4, T=8, d=8192, d_state=16, x_dtype=base.CV_BF16, state_dtype=base.CV_F32, n_slots=4, softplus=1,
                 state_slot_stride=8192 * 16)
        d.update(kw)
        for n in ("x", "dt", "z", "out"):
            d[n + "_tok_stride"], d[n + "_seq_stride"] = d["d"], d["d"] * d["T"]
        d["state_slot_stride"] = d["d"] * d["d_state"]
        got = sq.SqScanInfo()
        rc = lib.selscan_describe(call, sq.SqScanShape(**d), ctypes.byref(got))
        assert rc == 0, lib.seqops_last_error()
        return got

    def far(call, **kw):
        """The channels of a workgroup where some tokens are too far apart for 32-bit offsets."""
        d = dict(n_seq=1, T=8, d=64, d_state=16, x_dtype=base.CV_BF16, state_dtype=base.CV_F32, n_slots=1, softplus=1,
                 x_tok_stride=64, dt_tok_stride=64, z_tok_stride=64, out_tok_stride=64, b_tok_stride=16, c_tok_stride=16)
        d.update(kw)
        got = sq.SqScanInfo()
        assert lib.selscan_describe(call, sq.SqScanShape(**d), ctypes.byref(got)) == 0
        return got.channels

    assert far(sq.SQ_SCAN_VERIFY) == 64
    for name in ("x", "dt", "z", "b", "out"):
        near = (2 ** 30 - 1 - 64) // 3 // 8 * 8    # elements of bf16
        assert far(sq.SQ_SCAN_VERIFY, **{name + "_tok_stride": near}) == 64
        assert far(sq.SQ_SCAN_VERIFY, **{name + "_tok_stride": near + 8}) == 256
    assert far(sq.SQ_SCAN_UPDATE, c_tok_stride=2 ** 26) == 64 and far(sq.SQ_SCAN_UPDATE, c_tok_stride=2 ** 27) == 256
    one = info(sq.SQ_SCAN_UPDATE, T=1)
    assert (one.launches, one.channels, one.workgroups) == (1, 256, 4 * 32)
    assert info(sq.SQ_SCAN_VERIFY).channels == 64 and info(sq.SQ_SCAN_COMMIT).channels == 256
    assert info(sq.SQ_SCAN_VERIFY, T=7).channels == 256
    assert info(sq.SQ_SCAN_VERIFY, T=4, d_state=64).channels == 64
    assert info(sq.SQ_SCAN_VERIFY, T=32, d_state=8).channels == 256
    batch = info(sq.SQ_SCAN_PREFILL, n_seq=8, n_slots=8, T=2048, tokens=8 * 2048)
    assert (batch.launches, batch.workspace_bytes, batch.segment_tokens) == (1, 0, 0)
    long = info(sq.SQ_SCAN_PREFILL, n_seq=1, T=16384, d=4096, tokens=16384)
    assert long.launches == 2 and long.workspace_bytes > 0 and 64 <= long.segment_tokens <= 1024
    assert info(sq.SQ_SCAN_PREFILL, n_seq=0).launches == 0


def test_binding_checks_shapes_before_the_library():
    """What the binding itself refuses, on CPU tensors (whose device is refused first)."""
    torch = pytest.importorskip("torch")
    import causal_conv1d_verify_amd as cv

    _lib()
    x, B, A, state = torch.zeros(2, 3, 64), torch.zeros(2, 3, 16), torch.zeros(64, 16), torch.zeros(2, 64, 16)
    i32 = torch.zeros(2, dtype=torch.int32)
    calls = [lambda: cv.selective_scan_update(x, x, A, B, B, state, x), lambda: cv.selective_scan_verify(x, x, A, B, B, state, x),
             lambda: cv.selective_scan_commit(x, x, A, B, state),
             lambda: cv.selective_scan_prefill(x[0], x[0], A, B[0], B[0], state, x[0], i32, max_len=3),
             lambda: cv.qk_norm_rotary(x, None, None, None, x, None),
             lambda: cv.accept_drafts(i32[:, None], x[:, :1], torch.zeros(2, 1), i32, i32)]
    for call in calls:
        with pytest.raises(ValueError, match="same GPU"):
            call()
    for name in ("selective_scan_prefill", "selective_scan_update", "selective_scan_verify", "selective_scan_commit",
                 "qk_norm_rotary", "accept_drafts"):
        assert callable(getattr(cv, name)) and name in cv.__all__


@pytest.fixture
def m(monkeypatch):
    """The binding without its device check and its stream."""
    pytest.importorskip("torch")
    from causal_conv1d_verify_amd import sequence_ops

    _lib()
    monkeypatch.setattr(sequence_ops, "_same_gpu", lambda first, *others: first.device)
    monkeypatch.setattr(sequence_ops, "_on_stream", lambda stream, dev: 0)

    def workspace(need, given, handle, dev):
        import torch

        given = torch.empty(need, dtype=torch.uint8) if given is None else given
        if not given.is_contiguous():
            raise ValueError("workspace must be contiguous")
        return given, given.numel()

    monkeypatch.setattr(sequence_ops, "_workspace", workspace)
    return sequence_ops


def test_scan_binding_refusals(m):
    import torch

    z = torch.zeros
    good = dict(x=z(2, 3, 64), dt=z(2, 3, 64), A=z(64, 16), B=z(2, 3, 16), C=z(2, 3, 16), state=z(5, 64, 16), out=z(2, 3, 64))
    i32 = torch.zeros(2, dtype=torch.int32)
    m._scan_args("update", *good.values(), z=good["x"], D=z(64), dt_bias=z(64), slot_idx=i32)
    for bad in (dict(x=z(2, 4, 64)), dict(x=z(2, 192)), dict(dt=z(2, 3, 32)), dict(B=z(2, 4, 16)), dict(C=z(2, 3, 8)),
                dict(out=z(2, 3, 72)), dict(A=z(16, 64)), dict(A=z(16, 64).t()), dict(A=z(64, 16).double()),
                dict(state=z(5, 16, 64)), dict(state=z(5, 16, 64).transpose(1, 2)), dict(x=z(2, 3, 128)[..., ::2]),
                dict(B=z(2, 3, 32)[..., ::2]), dict(z=z(2, 3, 32)), dict(D=z(32)), dict(D=z(64).double()), dict(dt_bias=z(128)[::2]),
                dict(slot_idx=i32[:1]), dict(slot_idx=i32.long()), dict(num_tokens=z(2))):
        a = dict(good)
        kw = {n: bad.pop(n) for n in list(bad) if n not in a}
        a.update(bad)
        with pytest.raises(ValueError):
            m._scan_args("update", *a.values(), **kw)
    for bad in (dict(x=good["x"].bfloat16()), dict(C=good["C"].bfloat16()), dict(out=good["x"].bfloat16()),
                dict(state=good["state"].half())):
        a = dict(good)
        a.update(bad)
        with pytest.raises(TypeError):
            m._scan_args("update", *a.values())
    cu = torch.tensor([0, 3, 3], dtype=torch.int32)
    packed = [t[0] if n in ("x", "dt", "B", "C", "out") else t for n, t in good.items()]
    m._scan_args("prefill", *packed, cu_seqlens=cu, max_len=3)
    for kw in (dict(cu_seqlens=cu.long(), max_len=3), dict(cu_seqlens=cu[:0], max_len=3), dict(cu_seqlens=cu, max_len=2 ** 31),
               dict(cu_seqlens=cu, max_len=3, has_initial_state=i32[:1]), dict(cu_seqlens=cu[None], max_len=3)):
        with pytest.raises(ValueError):
            m._scan_args("prefill", *packed, **kw)
    with pytest.raises(ValueError):
        m._scan_args("prefill", *good.values(), cu_seqlens=cu, max_len=3)
    with pytest.raises(m.SeqOpsError):
        m._scan_args("prefill", *[t[..., :60] if t.shape[-1] == 64 else t[..., :60, :].contiguous() if t.shape[-2] == 64 else t
                                  for t in packed], cu_seqlens=cu, max_len=3)


def test_describe_makes_no_workspace(m, monkeypatch):
    import torch

    x, B = torch.zeros(3000, 64, dtype=torch.bfloat16), torch.zeros(3000, 16, dtype=torch.bfloat16)
    args = (x, x, torch.zeros(64, 16), B, B, torch.zeros(1, 64, 16), torch.zeros_like(x))
    cu = torch.tensor([0, 3000], dtype=torch.int32)
    made, empty = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(a) or empty(*a, **kw))
    for call in (lambda: m.selective_scan_describe("prefill", *args, cu, max_len=3000),
                 lambda: m.selective_scan_describe("prefill", *args, cu_seqlens=cu, max_len=3000)):
        info = call()
        assert info.launches == 2 and info.workspace_bytes > 0 and not made
    few = [t[None, :5] if t.shape[0] == 3000 else t for t in args]
    assert m.selective_scan_describe("verify", *few).launches == 1
    assert m.selective_scan_describe("commit", *few[:4], few[5]).launches == 1
    with pytest.raises(KeyError):
        m.selective_scan_describe("forward", *few)


def test_rotary_binding_refusals(m):
    import torch

    z = torch.zeros
    q, k, pos, freq = z(5, 4, 64), z(5, 2, 64), torch.zeros(5, dtype=torch.int64), z(16)
    good = dict(q=q, k=k, positions=pos, inv_freq=freq, q_out=q, k_out=k)
    m._rotary_args(*good.values(), q_weight=z(64), k_weight=z(64))
    m._rotary_args(q, None, pos.int(), freq, q, None)
    m._rotary_args(q, k, None, None, q, k)
    for bad in (dict(q_out=z(5, 4, 32)), dict(k=z(4, 2, 64)), dict(k=z(5, 2, 32)), dict(k_out=z(5, 3, 64)), dict(k=None),
                dict(k_out=None), dict(positions=None), dict(inv_freq=None), dict(positions=pos.float()), dict(positions=pos[:4]),
                dict(inv_freq=z(33)), dict(inv_freq=z(16).double()), dict(inv_freq=z(32)[::2]), dict(q=z(5, 4, 128)[..., ::2]),
                dict(q=z(5, 256), q_out=z(5, 256)), dict(q_weight=z(32)), dict(k_weight=z(128)[::2]),
                dict(k=None, k_out=None, k_weight=z(64))):
        a = dict(good)
        kw = {n: bad.pop(n) for n in list(bad) if n not in a}
        a.update(bad)
        with pytest.raises(ValueError):
            m._rotary_args(*a.values(), **kw)
    for bad in (dict(k=k.bfloat16()), dict(q_out=q.bfloat16()), dict(q_weight=z(64).bfloat16())):
        a = dict(good)
        kw = {n: bad.pop(n) for n in list(bad) if n not in a}
        a.update(bad)
        with pytest.raises(TypeError):
            m._rotary_args(*a.values(), **kw)


def test_accept_binding_refusals(m):
    import torch

    z = torch.zeros
    i = torch.zeros(3, 4, dtype=torch.int32)
    good = dict(tokens=i, target=z(3, 4, 50), uniform=z(3, 4), num_tokens=i[:, 0].contiguous(), next_token=i[:, 0].contiguous())
    m._accept_args(*good.values(), draft=z(3, 3, 50), path=i, window_index=i[:, 0].contiguous(), slot_idx=i[:, 0].contiguous())
    m._accept_args(*good.values(), parent=i)
    one = dict(tokens=i[:, :1], target=z(3, 1, 50), uniform=z(3, 1), num_tokens=good["num_tokens"], next_token=good["next_token"])
    m._accept_args(*one.values(), draft=z(3, 0, 50))
    for bad in (dict(tokens=i.long()), dict(tokens=i[:, :3]), dict(tokens=i.t().contiguous().t()), dict(target=z(3, 200)),
                dict(target=z(3, 4, 100)[..., ::2]), dict(uniform=z(3, 3)), dict(uniform=z(3, 4).double()),
                dict(num_tokens=i[:, 0]), dict(next_token=z(3)), dict(draft=z(3, 4, 50)), dict(draft=z(3, 3, 100)[..., ::2]),
                dict(parent=i, draft=z(3, 3, 50)), dict(parent=i[:2]), dict(path=i.long()), dict(window_index=i[0]),
                dict(slot_idx=i[:, 0])):
        a = dict(good)
        kw = {n: bad.pop(n) for n in list(bad) if n not in a}
        a.update(bad)
        with pytest.raises(ValueError):
            m._accept_args(*a.values(), **kw)
    with pytest.raises(TypeError):
        m._accept_args(*good.values(), draft=z(3, 3, 50).bfloat16())
    with pytest.raises(TypeError):
        m._accept_args(*{**good, "target": z(3, 4, 50).half()}.values())


def test_the_call_module_leaves_other_arguments_alone():
    """CPU tensors, no tensors, wrong counts: None, and no exception of the module's own."""
    torch = pytest.importorskip("torch")
    _lib()
    if not os.path.exists(os.path.join(os.path.dirname(sq.LIB_PATH), "_sqcall.so")):
        pytest.skip("_sqcall.so not built (run __graft_entry__.build())")
    from causal_conv1d_verify_amd import _sqcall as c

    x, B = torch.zeros(2, 3, 64), torch.zeros(2, 3, 16)
    i = torch.zeros(2, 3, dtype=torch.int32)
    for kind in (0, 1, 2, 3, 9):
        assert c.scan(kind, x, x, B, B, B, B, x, None, 3, None, None, None, True, None, None, None, None) is None
    assert c.scan(0, x[0], x[0], B, B[0], B[0], B, x[0], i[0], "3", x, None, None, True, None, None, None, None) is None
    assert c.scan(1, None, 3, "A", B, B, B, x, None, None, None, None, None, 1, None, None, None, None) is None
    assert c.scan() is None and c.rotary(x) is None and c.accept(x) is None
    assert c.rotary(x, None, None, None, x, None, None, None, 1e-6, False) is None
    assert c.rotary(x, x, i[0], None, x, None, "w", None, "eps", 0) is None
    assert c.accept(i, x, x, i[0], i[0], None, None, None, None, None, None) is None
    assert c.accept(i, "t", x, None, i[0], None, None, None, None, None, None) is None
