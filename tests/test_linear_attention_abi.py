"""Host-side tests of liblinattn.so: exports, validation and the binding's checks.  No GPU
needed and no kernel launched: calls that must be refused run in a child process that sees no
GPU, so that even a validation bug could not turn a stand-in pointer into a launch."""

import ctypes
import json
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "linear_attention.h")

la = pytest.importorskip("causal_conv1d_verify_amd._linattn")
from causal_conv1d_verify_amd import _lib as base  # noqa: E402

EINVAL, ENOTSUP = base.CV_EINVAL, base.CV_ENOTSUP


def _lib():
    if not os.path.exists(la.LIB_PATH):
        pytest.skip("liblinattn.so not built (run __graft_entry__.build())")
    return la.load()


def test_header_binding_and_library_agree():
    lib = _lib()
    text = open(HEADER).read()
    declared = set(re.findall(r"^\s*CV_API\s+(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, re.M))
    assert declared == set(la.EXPORTS)
    res = subprocess.run(["nm", "-D", "--defined-only", la.LIB_PATH], capture_output=True,
                         text=True, check=True)
    assert set(re.findall(r"\bT (\w+)$", res.stdout, re.M)) == declared
    want = int(re.search(r"#define LINEAR_ATTENTION_ABI_VERSION (\d+)", text).group(1))
    assert lib.linattn_abi_version() == want


def test_struct_layouts(tmp_path):
    """The ctypes structures have the C structures' sizes and offsets."""
    src = tmp_path / "layout.c"
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "linear_attention.h"',
             "int main(void) {"]
    for name, cls in (("la_shape_t", la.LaShape), ("la_norm_shape_t", la.LaNormShape)):
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    src.write_text("\n".join(lines) + "return 0;}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", f"-I{ROOT}/include", str(src), "-o", exe],
                   check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    got = dict(line.rsplit(" ", 1) for line in out.splitlines())
    for name, cls in (("la_shape_t", la.LaShape), ("la_norm_shape_t", la.LaNormShape)):
        assert int(got[name]) == ctypes.sizeof(cls)
        for f in cls._fields_:
            assert int(got[f"{name}.{f[0]}"]) == getattr(cls, f[0]).offset


_CHILD = r"""
import ctypes, json, sys
sys.path.insert(0, sys.argv[1])
from causal_conv1d_verify_amd import _lib as B, _linattn as L
lib = L.load()
A, H = 0x10000, 64
res = {}
def shape(**kw):
    d = dict(n_seq=4, T=8, q_heads=2, v_heads=4, dk=64, dv=32, scale=0.125, x_dtype=B.CV_BF16,
             state_dtype=B.CV_F32, n_slots=4,
             q_seq_stride=8 * 512, q_tok_stride=512, q_head_stride=64,
             k_seq_stride=8 * 512, k_tok_stride=512, k_head_stride=64,
             v_seq_stride=8 * 512, v_tok_stride=512, v_head_stride=32,
             out_seq_stride=8 * 128, out_tok_stride=128, out_head_stride=32,
             g_seq_stride=32, g_tok_stride=4, state_slot_stride=4 * 64 * 32)
    d.update(kw)
    return L.LaShape(**d)
def note(name, rc):
    res[name] = [rc, lib.linattn_last_error().decode()]
def update(name, s, q=A, k=A, v=A, g=A, state=A, slot=A, out=A):
    note("update:" + name, lib.linattn_update(s, q, k, v, g, state, slot, out, None))
def verify(name, s, q=A, k=A, v=A, g=A, state=A, slot=A, out=A):
    note("verify:" + name, lib.linattn_verify(s, q, k, v, g, state, slot, out, None))
def commit(name, s, k=A, v=A, g=A, state=A, slot=A, num=A):
    note("commit:" + name, lib.linattn_commit(s, k, v, g, state, slot, num, None))
def prefill(name, s, q=A, k=A, v=A, g=A, state=A, slot=A, cu=A, init=A, out=A, ws=A, size=1 << 40):
    note("prefill:" + name, lib.linattn_prefill(s, q, k, v, g, state, slot, cu, init, out, ws, size, None))
bad = dict(
    n_seq=dict(n_seq=-1), T=dict(T=0), q_heads=dict(q_heads=0), groups=dict(q_heads=3),
    v_heads=dict(v_heads=0), dk0=dict(dk=0), dv0=dict(dv=-8), dk_odd=dict(dk=60), dv_odd=dict(dv=12),
    dk_big=dict(dk=264), dv_big=dict(dv=264), x_type=dict(x_dtype=7), s_type=dict(state_dtype=-1),
    pair=dict(x_dtype=B.CV_F32, state_dtype=B.CV_BF16), n_slots=dict(n_slots=-1),
    k_negative=dict(k_tok_stride=-8), v_unaligned=dict(v_head_stride=36), k_unaligned=dict(k_tok_stride=516),
    slot_short=dict(state_slot_stride=64), slot_unaligned=dict(state_slot_stride=4 * 64 * 32 + 2),
    g_negative=dict(g_tok_stride=-1))
for name, kw in bad.items():
    update(name, shape(**kw)); verify(name, shape(**kw)); commit(name, shape(**kw)); prefill(name, shape(**kw))
    note("workspace:" + name, lib.linattn_prefill_workspace(shape(**kw)))
outs = dict(scale=dict(scale=float("nan")), q_unaligned=dict(q_tok_stride=12), out_unaligned=dict(out_tok_stride=132),
            out_heads=dict(out_head_stride=24), out_toks=dict(out_tok_stride=96))
for name, kw in outs.items():
    update(name, shape(**kw)); verify(name, shape(**kw)); prefill(name, shape(**kw))
update("out_rows", shape(out_seq_stride=128)); verify("out_rows", shape(out_seq_stride=128))
for f in (update, verify, commit):
    f("T33", shape(T=33))
    f("slots_short", shape(n_slots=3), slot=None)
    f("empty", shape(n_seq=0))
    for p in ("k", "v", "state"):
        f("null_" + p, shape(), **{p: None}); f("off_" + p, shape(), **{p: A + 8})
    f("off_g", shape(), g=A + 2); f("off_slot", shape(), slot=A + 1)
for f in (update, verify, prefill):
    for p in ("q", "out"):
        f("null_" + p, shape(), **{p: None}); f("off_" + p, shape(), **{p: A + 4})
commit("off_num", shape(), num=A + 2)
prefill("null_cu", shape(), cu=None); prefill("off_init", shape(), init=A + 1)
prefill("slots_short", shape(n_slots=3), slot=None); prefill("empty", shape(n_seq=0))
long = shape(T=100000, n_seq=1, q_heads=1, v_heads=1)
need = lib.linattn_prefill_workspace(long)
res["need"] = need
if need > 0:
    prefill("ws_small", long, size=need - 1)
    prefill("ws_null", long, ws=None)
    prefill("ws_off", long, ws=A + 8)
for name in ("update", "verify", "commit", "prefill"):
    fn = getattr(lib, "linattn_" + name)
    note(name + ":null_shape", fn(*[None] * len(fn.argtypes[:-2]), *([0, None] if name == "prefill" else [None, None])))

def nshape(**kw):
    d = dict(rows=4, heads=2, dim=64, eps=1e-6, scale=1.0, x_dtype=B.CV_BF16, res_dtype=B.CV_BF16,
             activation=0, gate_first=0, y_row_stride=128, y_head_stride=64, gate_row_stride=128,
             gate_head_stride=64, out_row_stride=128, out_head_stride=64, res_row_stride=64,
             res_out_row_stride=64)
    d.update(kw)
    return L.LaNormShape(**d)
def gated(name, s, y=A, z=A, w=A, out=A):
    note("gated:" + name, lib.norm_gated(s, y, z, w, out, None))
def residual(name, s, y=A, pw=A, z=A, r=A, ro=A, w=A, out=A):
    note("residual:" + name, lib.norm_residual(s, y, pw, z, r, ro, w, out, None))
both = dict(rows=dict(rows=-1), dim0=dict(dim=0), dim_odd=dict(dim=60), dim_big=dict(dim=16392),
            eps=dict(eps=-1.0), eps_inf=dict(eps=float("inf")), eps_nan=dict(eps=float("nan")),
            x_type=dict(x_dtype=9), y_negative=dict(y_row_stride=-128), y_unaligned=dict(y_row_stride=132),
            gate_unaligned=dict(gate_row_stride=4), out_unaligned=dict(out_row_stride=132),
            out_rows=dict(out_row_stride=56))
for name, kw in both.items():
    gated(name, nshape(**kw)); residual(name, nshape(**{**dict(heads=1), **kw}))
gated("heads", nshape(heads=0)); gated("act", nshape(activation=2)); gated("dim_2056", nshape(dim=2056))
gated("out_heads", nshape(out_head_stride=56)); gated("empty", nshape(rows=0), None, None, None, None)
for p in ("y", "w", "out"):
    gated("null_" + p, nshape(), **{p: None}); gated("off_" + p, nshape(), **{p: A + 8})
gated("off_z", nshape(), z=A + 4)
one = dict(heads=1)
residual("heads", nshape(heads=2)); residual("scale", nshape(heads=1, scale=float("inf")))
residual("r_type", nshape(heads=1, res_dtype=5))
residual("pair", nshape(heads=1, x_dtype=B.CV_F32))
residual("r_unaligned", nshape(heads=1, res_row_stride=68)); residual("ro_rows", nshape(heads=1, res_out_row_stride=56))
for p in ("y", "r", "ro", "w"):
    residual("null_" + p, nshape(**one), **{p: None})
for p in ("y", "pw", "z", "r", "ro", "w", "out"):
    residual("off_" + p, nshape(**one), **{p: A + 8})
residual("empty", nshape(heads=1, rows=0), *[None] * 7)
print(json.dumps(res))
"""


@pytest.fixture(scope="module")
def refusals():
    _lib()
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    run = subprocess.run([sys.executable, "-c", _CHILD, ROOT], capture_output=True, text=True,
                         env=env, timeout=300)
    assert run.returncode == 0, run.stderr[-3000:]
    return json.loads(run.stdout.strip().splitlines()[-1])


def test_bad_calls_are_refused(refusals):
    need = refusals.pop("need")
    assert need >= 0
    unsupported = {"dk_odd", "dv_odd", "dk_big", "dv_big", "pair", "T33", "dim_odd", "dim_big",
                   "dim_2056"}
    for name, (rc, detail) in refusals.items():
        short = name.split(":")[1]
        if short == "empty":
            assert rc == 0, (name, rc, detail)
            continue
        want = ENOTSUP if short in unsupported or short.startswith("off_") or "unaligned" in short \
            or short == "ws_off" else EINVAL
        assert rc == want, (name, rc, detail)
        assert detail, name
    assert len(refusals) > 170


def test_binding_checks_shapes_before_the_library():
    """What the binding itself refuses, on CPU tensors (whose device is refused last)."""
    torch = pytest.importorskip("torch")
    import causal_conv1d_verify_amd as cv

    _lib()
    t = torch.zeros(2, 3, 4, 64)
    state = torch.zeros(2, 4, 64, 64)
    with pytest.raises(ValueError, match="same GPU"):
        cv.linear_attn_update(t, t, t, None, state, t)
    with pytest.raises(ValueError, match="same GPU"):
        cv.gated_norm(t[0], t[0], torch.zeros(64), t[0])
    with pytest.raises(ValueError, match="same GPU"):
        cv.residual_norm(t[0, 0], t[0, 0], torch.zeros(64), t[0, 0])
    for name in ("linear_attn_prefill", "linear_attn_update", "linear_attn_verify",
                 "linear_attn_commit", "gated_norm", "residual_norm"):
        assert callable(getattr(cv, name)) and name in cv.__all__


def test_binding_refusals(monkeypatch):
    """The binding's shape, type and stride checks (device check and launch taken out)."""
    torch = pytest.importorskip("torch")
    from causal_conv1d_verify_amd import linear_attention as m

    _lib()
    monkeypatch.setattr(m, "_same_gpu", lambda first, *others: first.device)
    monkeypatch.setattr(m, "_on_stream", lambda stream, dev: 0)
    z = torch.zeros
    q, v, state = z(2, 3, 2, 64), z(2, 3, 4, 32), z(5, 4, 64, 32)
    g = z(2, 3, 4)
    out = z(2, 3, 4, 32)
    m._attn_args("update", q, q, v, g, state, out)
    m._attn_args("update", q, q, v, g[0, 0], state, out)
    i32 = torch.zeros(2, dtype=torch.int32)
    for bad in (dict(k=z(2, 4, 2, 64)), dict(k=z(2, 3, 128)), dict(q=z(2, 3, 4, 64)),
                dict(out=z(2, 3, 4, 40)), dict(state=z(5, 4, 32, 64)),
                dict(state=z(5, 4, 32, 64).transpose(2, 3)), dict(g=z(2, 3, 2)),
                dict(g=z(2, 3, 4, dtype=torch.float64)), dict(g=z(3, 4)),
                dict(g=z(2, 3, 8)[..., ::2]), dict(v=z(2, 3, 4, 64)[..., ::2]),
                dict(slot_idx=i32[:1]), dict(slot_idx=i32.long()), dict(num_tokens=z(2))):
        a = dict(q=q, k=q, v=v, g=g, state=state, out=out)
        kw = {n: bad.pop(n) for n in list(bad) if n not in a}
        a.update(bad)
        with pytest.raises(ValueError):
            m._attn_args("update", *a.values(), **kw)
    for bad in (dict(q=q.bfloat16()), dict(out=out.bfloat16()), dict(state=state.half())):
        a = dict(q=q, k=q, v=v, g=g, state=state, out=out)
        a.update(bad)
        with pytest.raises(TypeError):
            m._attn_args("update", *a.values())
    cu = torch.tensor([0, 3, 3], dtype=torch.int32)
    p = dict(cu_seqlens=cu, max_len=3)
    m._attn_args("prefill", q[0], q[0], v[0], g[0], state, out[0], **p)
    with pytest.raises(ValueError):
        m._attn_args("prefill", q, q, v, g, state, out, **p)
    with pytest.raises(ValueError):
        m._attn_args("prefill", q[0], q[0], v[0], g[0], state, out[0], cu_seqlens=cu.long(), max_len=3)
    y, w = z(4, 64), z(64)
    m._gated_args(y, y, w, y)
    for args, kw in (((y, z(4, 32), w, y), {}), ((y, y, z(32), y), {}), ((y, y, w, z(3, 64)), {}),
                     ((y, y, w, y), dict(activation="gelu")), ((z(64), None, w, z(64)), {}),
                     ((z(4, 128)[:, ::2], y, w, y), {})):
        with pytest.raises(ValueError):
            m._gated_args(*args, **kw)
    m._residual_args(y, y, w, y, gate=w)
    for args, kw in (((y, z(3, 64), w, y), {}), ((y, y, None, y), {}), ((y, y, w, None), {}),
                     ((y, y, w, y), dict(gate=z(32))), ((y, y, w, y), dict(post_weight=z(32))),
                     ((y, y, w, z(4, 128)[:, ::2]), {})):
        with pytest.raises(ValueError):
            m._residual_args(*args, **kw)
    with pytest.raises(TypeError):
        m._residual_args(y, y, w, y, residual_out=y.bfloat16())
