"""Refusals of the adapter and balance calls (CPU): every call here fails host-side validation, or has nothing to
do, before any CUDA call."""

import ctypes

import pytest

from grouped_nf4_expert_b200 import build as e4b_build
from grouped_nf4_expert_b200 import e4b

INVALID, UNSUPPORTED, SMALL = e4b.E4B_ERR_INVALID_ARG, e4b.E4B_ERR_UNSUPPORTED, e4b.E4B_ERR_WORKSPACE_TOO_SMALL
ref = ctypes.byref


@pytest.fixture(scope="module")
def so():
    e4b_build.build()
    return e4b.lib()


@pytest.fixture()
def p():
    buf = (ctypes.c_uint8 * 1040)()  # host memory standing in for device pointers: only addresses are looked at
    base = (ctypes.addressof(buf) + 15) & ~15
    yield [base + 16 * i for i in range(64)]
    del buf


@pytest.mark.parametrize("field,value,status", [
    ("K", 0, UNSUPPORTED), ("K", 96, UNSUPPORTED), ("K", 1 << 21, UNSUPPORTED), ("N", 0, UNSUPPORTED),
    ("N", 12, UNSUPPORTED), ("N", -8, UNSUPPORTED), ("n_adapters", 0, UNSUPPORTED), ("n_adapters", 1025, UNSUPPORTED),
    ("r", 4, UNSUPPORTED), ("r", 12, UNSUPPORTED), ("r", 72, UNSUPPORTED), ("blocksize", 32, UNSUPPORTED),
])
def test_projection_dims(so, field, value, status):
    d = e4b.ProjDimsC(128, 72, 3, 8, 64)
    out = e4b.ProjSizes()
    assert so.e4b_proj_get_sizes(ref(d), 10, ref(out)) == 0
    setattr(d, field, value)
    assert so.e4b_proj_get_sizes(ref(d), 10, ref(out)) == status


def test_projection_sizes(so):
    d = e4b.ProjDimsC(128, 72, 3, 8, 64)
    out = e4b.ProjSizes()
    assert so.e4b_proj_get_sizes(ref(d), -1, ref(out)) == INVALID
    assert so.e4b_proj_get_sizes(ref(d), (1 << 24) + 1, ref(out)) == UNSUPPORTED
    assert so.e4b_proj_get_sizes(ref(d), 10, None) == INVALID
    assert so.e4b_proj_get_sizes(None, 10, ref(out)) == INVALID
    assert so.e4b_proj_get_sizes(ref(d), 1000, ref(out)) == 0
    assert out.rows_cap == 1280 and out.rows_cap % 256 == 0  # 1000 + 31 * 4, rounded up
    assert so.e4b_proj_get_sizes(ref(d), 0, ref(out)) == 0 and out.rows_cap == 0


def test_projection_calls(so, p):
    d = e4b.ProjDimsC(128, 72, 3, 8, 64)
    sz = e4b.ProjSizes()
    assert so.e4b_proj_get_sizes(ref(d), 10, ref(sz)) == 0
    base, ad = e4b.Nf4Matrix(p[0], p[1]), e4b.AdapterFactors(p[2], p[3], p[4])
    gr = e4b.AdapterGroups(p[5], p[6], p[7])
    ids, x, y, ws, lp = p[8], p[9], p[10], p[11], p[12]
    big, wsb = sz.serve_workspace_bytes, sz.workspace_bytes
    serve, group = so.e4b_multi_lora_serve_fwd, so.e4b_adapter_group
    assert serve(ref(d), 10, ids, x, ref(base), ref(ad), y, ws, big - 1, None) == SMALL
    assert serve(ref(d), 10, ids, x, ref(base), ref(ad), y, ws + 4, big, None) == INVALID
    assert serve(ref(d), 10, None, x, ref(base), ref(ad), y, ws, big, None) == INVALID
    assert serve(ref(d), 10, ids + 2, x, ref(base), ref(ad), y, ws, big, None) == INVALID
    assert serve(ref(d), 10, ids, x + 8, ref(base), ref(ad), y, ws, big, None) == INVALID
    assert serve(ref(d), 10, ids, x, ref(base), ref(ad), None, ws, big, None) == INVALID
    assert serve(ref(d), 10, ids, x, None, ref(ad), y, ws, big, None) == INVALID
    assert serve(ref(d), 10, ids, x, ref(e4b.Nf4Matrix(p[0], None)), ref(ad), y, ws, big, None) == INVALID
    assert serve(ref(d), 10, ids, x, ref(base), ref(e4b.AdapterFactors(p[2], p[3], None)), y, ws, big, None) == INVALID
    assert group(ref(d), 10, ids, ref(e4b.AdapterGroups(p[5], p[6], None)), None) == INVALID
    assert group(ref(d), 10, None, ref(gr), None) == INVALID
    fwd, dgrad, wgrad = so.e4b_multi_lora_fwd, so.e4b_multi_lora_dgrad, so.e4b_multi_lora_wgrad
    for call in (fwd, dgrad):
        assert call(ref(d), 10, ref(gr), x, ref(base), ref(ad), lp, y, ws, wsb - 1, None) == SMALL
        assert call(ref(d), 10, None, x, ref(base), ref(ad), lp, y, ws, wsb, None) == INVALID
        assert call(ref(d), 10, ref(gr), x, ref(base), ref(ad), None, y, ws, wsb, None) == INVALID
        assert call(ref(d), 10, ref(gr), None, ref(base), ref(ad), lp, y, ws, wsb, None) == INVALID
        assert call(ref(d), 0, None, None, None, None, None, None, None, 0, None) == 0
    assert wgrad(ref(d), 10, ref(gr), x, y, lp, None, p[13], p[14], ws, wsb, None) == INVALID
    assert wgrad(ref(d), 10, ref(gr), x, y, lp, lp, None, p[14], ws, wsb, None) == INVALID
    assert wgrad(ref(d), 10, ref(gr), x, y, lp, lp, p[13], p[14], ws, 8, None) == SMALL
    assert serve(ref(d), 0, None, None, None, None, None, None, 0, None) == 0
    assert group(ref(d), 0, None, None, None) == 0


@pytest.mark.parametrize("field,value,status", [
    ("E", 0, UNSUPPORTED), ("E", 1025, UNSUPPORTED), ("top_k", 0, UNSUPPORTED), ("top_k", 9, UNSUPPORTED),
    ("S", 0, UNSUPPORTED), ("S", (1 << 20) + 1, UNSUPPORTED), ("balance_coef", float("inf"), INVALID),
    ("z_coef", float("nan"), INVALID),
])
def test_balance_dims(so, field, value, status):
    d = e4b.BalanceDims(8, 2, 3, 0.1, 0.2)
    n = e4b.c_sz(0)
    assert so.e4b_balance_get_sizes(ref(d), 10, ref(n)) == 0 and n.value > 0
    setattr(d, field, value)
    assert so.e4b_balance_get_sizes(ref(d), 10, ref(n)) == status


def test_balance_calls(so, p):
    d = e4b.BalanceDims(8, 2, 3, 0.1, 0.2)
    n = e4b.c_sz(0)
    assert so.e4b_balance_get_sizes(ref(d), 10, ref(n)) == 0
    assert so.e4b_balance_get_sizes(ref(d), -1, ref(n)) == INVALID
    assert so.e4b_balance_get_sizes(ref(d), 10, None) == INVALID
    st = e4b.BalanceStats(*p[0:4])
    logits, ids, seq, mask, loss, ws, dl = p[4:11]
    fwd, bwd = so.e4b_balance_fwd, so.e4b_balance_bwd
    assert fwd(ref(d), 10, logits, ids, None, mask, ref(st), loss, ws, n.value, None) == INVALID  # S != 1
    assert fwd(ref(d), 10, logits, ids, seq + 2, mask, ref(st), loss, ws, n.value, None) == INVALID
    assert fwd(ref(d), 10, logits, None, seq, mask, ref(st), loss, ws, n.value, None) == INVALID
    assert fwd(ref(d), 10, logits + 4, ids, seq, mask, ref(st), loss, ws, n.value, None) == INVALID
    assert fwd(ref(d), 10, logits, ids, seq, mask, None, loss, ws, n.value, None) == INVALID
    assert fwd(ref(d), 10, logits, ids, seq, mask, ref(st), None, ws, n.value, None) == INVALID
    assert fwd(ref(d), 10, logits, ids, seq, mask, ref(st), loss, ws, n.value - 1, None) == SMALL
    assert fwd(ref(d), 10, logits, ids, seq, mask, ref(st), loss, None, n.value, None) == INVALID
    assert bwd(ref(d), 10, logits, None, mask, ref(st), None, 0, dl, None) == INVALID
    assert bwd(ref(d), 10, logits, seq, mask, ref(st), None, 0, None, None) == INVALID
    assert bwd(ref(d), 10, logits, seq, mask, ref(st), dl + 2, 0, dl, None) == INVALID
    assert bwd(ref(d), 10, logits, seq, mask, ref(e4b.BalanceStats(p[0], p[1], None, p[3])), None, 0, dl,
               None) == INVALID
    assert bwd(ref(d), 0, None, None, None, None, None, 0, None, None) == 0


def _header():
    import re
    return re.sub(r"/\*.*?\*/", "", open(e4b.OPERATORS_HEADER).read(), flags=re.S)


def test_binding_matches_the_header(so):
    import re
    text = _header()
    protos = re.findall(r"^\s*e4b_status\s+(e4b_\w+)\s*\(([^;{]*?)\)\s*;", text, flags=re.M | re.S)
    assert len(protos) == 9
    for name, args in protos:
        assert hasattr(so, name)
        assert len(e4b._SIGNATURES[name][1]) == args.count(",") + 1, name
    structs = {}
    for body, name in re.findall(r"typedef\s+struct\s*\{(.*?)\}\s*(\w+)\s*;", text, flags=re.S):
        fields = []
        for decl in filter(None, (d.strip() for d in body.split(";"))):
            fields += [re.findall(r"\w+", part)[-1] for part in decl.split(",")]
        structs[name] = fields
    pairs = {"e4b_proj_dims": e4b.ProjDimsC, "e4b_nf4_matrix": e4b.Nf4Matrix,
             "e4b_adapter_factors": e4b.AdapterFactors, "e4b_adapter_groups": e4b.AdapterGroups,
             "e4b_proj_sizes": e4b.ProjSizes, "e4b_balance_dims": e4b.BalanceDims,
             "e4b_balance_stats": e4b.BalanceStats}
    assert set(structs) == set(pairs)
    for cname, cls in pairs.items():
        assert [f[0] for f in cls._fields_] == structs[cname], cname


def test_header_is_c(tmp_path):
    import os
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "e4b_operators.h"\nint main(void) { return E4B_MAX_ADAPTERS == 1024 ? 0 : 1; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(e4b.OPERATORS_HEADER), "-c", str(src),
                    "-o", str(tmp_path / "t.o")], check=True)
