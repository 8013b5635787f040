"""The linear layer, the grouped products, the router and the weighted sum without a GPU: the
ctypes mirrors match the C structs, and every refusal comes from the host before any launch."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "inkattn.h")
BASE = 1 << 40       # addresses that no call here dereferences, far apart


@pytest.fixture(scope="module")
def ia():
    from relative_bias_hybrid_gb300 import build
    build.build()
    import relative_bias_hybrid_gb300.inkattn as ia
    ia.lib()
    return ia


def _at(i):
    return BASE + (i << 36)


def _linear(ia, **kw):
    p = ia.LinearParams()
    p.struct_size = ctypes.sizeof(ia.LinearParams)
    p.N_tok, p.K, p.F = 64, 128, 96
    p.x, p.w, p.bias, p.residual, p.out, p.dev_status = (_at(i) for i in range(6))
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _grouped(ia, **kw):
    p = ia.GroupedLinearParams()
    p.struct_size = ctypes.sizeof(ia.GroupedLinearParams)
    p.E, p.M, p.N_x, p.K, p.F = 8, 64, 20, 128, 96
    p.x, p.w, p.bias, p.expert_offsets, p.row_token, p.out, p.dev_status = (_at(i) for i in range(7))
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _route(ia, **kw):
    p = ia.RouteParams()
    p.struct_size = ctypes.sizeof(ia.RouteParams)
    p.N_tok, p.E, p.n_shared, p.top_k, p.scale = 5000, 256, 2, 6, 1.0
    p.logits, p.topk_ids, p.weights, p.expert_offsets, p.row_token, p.token_rows = (_at(i) for i in range(6))
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _combine(ia, **kw):
    p = ia.ExpertCombineParams()
    p.struct_size = ctypes.sizeof(ia.ExpertCombineParams)
    p.N_tok, p.M, p.F, p.top_k, p.n_shared = 64, 128, 256, 2, 1
    p.y, p.shared, p.weights, p.token_rows, p.out, p.dev_status = (_at(i) for i in range(6))
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def test_ctypes_structs_match_c_layout(ia, tmp_path):
    structs = {"inkattn_linear_params": ia.LinearParams, "inkattn_grouped_linear_params": ia.GroupedLinearParams,
               "inkattn_route_params": ia.RouteParams, "inkattn_expert_combine_params": ia.ExpertCombineParams}
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void){"]
    for cname, py in structs.items():
        lines.append(f'printf("{cname} sizeof %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    lines.append("return 0;}")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c11", str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        cname, field, value = line.split()
        py = structs[cname]
        assert (ctypes.sizeof(py) if field == "sizeof" else getattr(py, field).offset) == int(value), line


def test_linear_refusals(ia):
    bad = [dict(struct_size=8), dict(N_tok=-1), dict(K=0), dict(K=12), dict(K=(1 << 20) + 8), dict(F=0),
           dict(F=(1 << 20) + 1), dict(act=5), dict(act=-1), dict(out_dtype=2), dict(x=None), dict(w=None),
           dict(out=None), dict(x=_at(0) + 8), dict(w=_at(1) + 2), dict(out=_at(4) + 4), dict(residual=_at(3) + 8),
           dict(bias=_at(2) + 2), dict(dev_status=_at(5) + 1),
           dict(out=_at(0) + 16), dict(out=_at(1) + 1600), dict(out=_at(2)),        # over x, w, bias
           dict(out=_at(3) + 16),                                                    # over part of the residual
           dict(out=_at(3), out_dtype=ia.INKATTN_DTYPE_F32)]                         # in place, another type
    for kw in bad:
        assert ia.inkattn_linear(_linear(ia, **kw), stream=0, raise_on_error=False) == ia.INKATTN_ERR_INVALID_ARG, kw
    assert ia.lib().inkattn_linear(None, None) == ia.INKATTN_ERR_INVALID_ARG


def test_grouped_linear_refusals(ia):
    bad = [dict(struct_size=8), dict(E=0), dict(E=1025), dict(M=-1), dict(N_x=-1), dict(N_x=0), dict(K=4),
           dict(F=0), dict(act=9), dict(out_dtype=-1), dict(expert_offsets=None), dict(expert_offsets=_at(3) + 2),
           dict(row_token=_at(4) + 1), dict(row_token=None),                         # 20 rows of x for 64 rows
           dict(x=None), dict(w=None), dict(out=None), dict(x=_at(0) + 4), dict(out=_at(5) + 8),
           dict(out=_at(0)), dict(out=_at(1) + 4096), dict(out=_at(3)), dict(out=_at(4) + 16)]
    for kw in bad:
        st = ia.inkattn_grouped_linear(_grouped(ia, **kw), stream=0, raise_on_error=False)
        assert st == ia.INKATTN_ERR_INVALID_ARG, kw
    assert ia.lib().inkattn_grouped_linear(None, None) == ia.INKATTN_ERR_INVALID_ARG


def test_route_refusals_and_workspace(ia):
    bad = [dict(struct_size=8), dict(N_tok=-1), dict(E=0), dict(E=1025), dict(n_shared=-1), dict(n_shared=17),
           dict(top_k=0), dict(top_k=17), dict(E=4, top_k=5), dict(score=2), dict(scale=float("inf")),
           dict(scale=float("nan")), dict(N_tok=1 << 28, top_k=2), dict(logits=None), dict(topk_ids=None),
           dict(weights=None), dict(expert_offsets=None), dict(row_token=None), dict(token_rows=None),
           dict(logits=_at(0) + 2), dict(weights=_at(2) + 1), dict(topk_ids=_at(0) + 64), dict(row_token=_at(5))]
    ws = ctypes.c_void_p(_at(9))
    for kw in bad:
        p = _route(ia, **kw)
        assert ia.inkattn_route_workspace_bytes(p) == 0, kw
        assert ia.lib().inkattn_route(ctypes.byref(p), ws, 1 << 30, None) == ia.INKATTN_ERR_INVALID_ARG, kw
    p = _route(ia)
    need = ia.inkattn_route_workspace_bytes(p)
    assert 0 < need <= 152 * 256 * 4
    for ptr, n in ((None, need), (ctypes.c_void_p(_at(9)), need - 1), (ctypes.c_void_p(_at(9) + 8), need)):
        assert ia.lib().inkattn_route(ctypes.byref(p), ptr, n, None) == ia.INKATTN_ERR_INVALID_ARG
    assert ia.inkattn_route_workspace_bytes(_route(ia, N_tok=288)) == 0


def test_route_workspace_overlaps_no_array(ia):
    p = _route(ia)
    need = ia.inkattn_route_workspace_bytes(p)
    for i in range(6):
        assert ia.lib().inkattn_route(ctypes.byref(p), ctypes.c_void_p(_at(i)), need, None) == ia.INKATTN_ERR_INVALID_ARG
    assert ia.lib().inkattn_route(ctypes.byref(p), ctypes.c_void_p(_at(4) + 5000 * 6 * 4 - 16), need, None) == \
        ia.INKATTN_ERR_INVALID_ARG
    # one beside them passes this check and meets the next, which wants a device
    assert ia.lib().inkattn_route(ctypes.byref(p), ctypes.c_void_p(_at(9)), need, None) != ia.INKATTN_OK


def test_expert_combine_refusals(ia):
    bad = [dict(struct_size=8), dict(N_tok=-1), dict(M=-1), dict(F=0), dict(F=12), dict(F=(1 << 20) + 8),
           dict(top_k=0), dict(top_k=17), dict(n_shared=-1), dict(n_shared=17), dict(y=None), dict(shared=None),
           dict(weights=None), dict(token_rows=None), dict(out=None), dict(y=_at(0) + 8), dict(shared=_at(1) + 2),
           dict(out=_at(4) + 4), dict(weights=_at(2) + 2), dict(token_rows=_at(3) + 1), dict(dev_status=_at(5) + 2),
           dict(out=_at(0)), dict(out=_at(1) + 32), dict(out=_at(2)), dict(out=_at(3)),
           dict(N_tok=2 ** 31 - 1, F=1 << 20)]
    for kw in bad:
        st = ia.inkattn_expert_combine(_combine(ia, **kw), stream=0, raise_on_error=False)
        assert st == ia.INKATTN_ERR_INVALID_ARG, kw


def test_binding_refusals(ia):
    """Shapes, types and strides that a params struct cannot express."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    x, w, out = torch.zeros(4, 16, dtype=bf), torch.zeros(8, 16, dtype=bf), torch.zeros(4, 8, dtype=bf)
    ia.linear_params(x=x, w=w, out=out)
    for kw in (dict(w=torch.zeros(9, 16, dtype=bf)), dict(w=torch.zeros(8, 24, dtype=bf)),
               dict(act="swiglu"), dict(bias=torch.zeros(7)), dict(residual=torch.zeros(4, 9, dtype=bf)),
               dict(x=torch.zeros(16, 4, dtype=bf).t()), dict(out=torch.zeros(5, 8, dtype=bf))):
        with pytest.raises(ValueError):
            ia.linear_params(**{**dict(x=x, w=w, out=out), **kw})
    for kw in (dict(x=x.float()), dict(out=out.half()), dict(bias=torch.zeros(8, dtype=bf))):
        with pytest.raises(TypeError):
            ia.linear_params(**{**dict(x=x, w=w, out=out), **kw})
    with pytest.raises(ValueError):
        ia.linear_params(x=x, w=w.to("meta"), out=out)
    with pytest.raises(KeyError):
        ia.linear_params(x=x, w=w, out=out, act="tanh")
    good = dict(x=x, w=torch.zeros(3, 8, 16, dtype=bf), expert_offsets=torch.zeros(4, dtype=i32),
                row_token=torch.zeros(6, dtype=i32), out=torch.zeros(6, 8, dtype=bf))
    ia.grouped_linear_params(**good)
    for kw in (dict(expert_offsets=torch.zeros(3, dtype=i32)), dict(row_token=torch.zeros(5, dtype=i32)),
               dict(bias=torch.zeros(3, 7)), dict(act="swiglu")):
        with pytest.raises(ValueError):
            ia.grouped_linear_params(**{**good, **kw})
    with pytest.raises(TypeError):
        ia.grouped_linear_params(**{**good, "expert_offsets": torch.zeros(4, dtype=torch.int64)})
    r = dict(logits=torch.zeros(4, 10), topk_ids=torch.zeros(4, 2, dtype=i32), weights=torch.zeros(4, 4),
             expert_offsets=torch.zeros(9, dtype=i32), row_token=torch.zeros(8, dtype=i32),
             token_rows=torch.zeros(4, 2, dtype=i32), n_shared=2)
    ia.route_params(**r)
    for kw in (dict(n_shared=1), dict(weights=torch.zeros(4, 2)), dict(row_token=torch.zeros(4, dtype=i32)),
               dict(token_rows=torch.zeros(4, 3, dtype=i32))):
        with pytest.raises(ValueError):
            ia.route_params(**{**r, **kw})
    c = dict(y=torch.zeros(8, 16, dtype=bf), weights=torch.zeros(4, 3), token_rows=torch.zeros(4, 2, dtype=i32),
             shared=torch.zeros(1, 4, 16, dtype=bf), out=torch.zeros(4, 16, dtype=bf))
    ia.expert_combine_params(**c)
    for kw in (dict(shared=None), dict(weights=torch.zeros(4, 2)), dict(out=torch.zeros(4, 8, dtype=bf))):
        with pytest.raises(ValueError):
            ia.expert_combine_params(**{**c, **kw})


def test_params_keep_their_tensors(ia):
    """A params struct holds addresses; the tensors behind them live as long as it does."""
    import gc
    import weakref
    bias = torch.zeros(8)
    seen = weakref.ref(bias)
    p = ia.linear_params(x=torch.zeros(4, 16, dtype=torch.bfloat16), w=torch.zeros(8, 16, dtype=torch.bfloat16),
                         out=torch.zeros(4, 8, dtype=torch.bfloat16), bias=bias)
    address = bias.data_ptr()
    del bias
    gc.collect()
    assert p.bias == address and seen() is not None
    del p
    gc.collect()
    assert seen() is None
