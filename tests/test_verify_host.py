"""The calls at a verification step's end without a GPU: struct layouts, refusals of the library and of the
binding, and the 4-bit cache's checks."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "inkattn.h")
FAKE = 1 << 20            # non-null and aligned: these calls never dereference it


@pytest.fixture(scope="module")
def ia():
    from relative_bias_hybrid_gb300 import build
    build.build()
    import relative_bias_hybrid_gb300.inkattn as ia
    ia.lib()
    return ia


def test_ctypes_structs_match_c_layout(ia, tmp_path):
    structs = {"inkattn_token_probs_params": ia.TokenProbsParams, "inkattn_verify_drafts_params": ia.VerifyDraftsParams,
               "inkattn_conv_rows": ia.ConvRows, "inkattn_conv_rollback_params": ia.ConvRollbackParams}
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void){"]
    for cname, py in structs.items():
        lines.append(f'printf("{cname} sizeof %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f[0]} %zu\\n", offsetof({cname}, {f[0]}));' for f in py._fields_]
    lines.append(f'printf("max states %d\\n", INKATTN_ROLLBACK_MAX_STATES - {ia.ROLLBACK_MAX_STATES}); return 0;}}')
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c11", str(src), "-o", str(tmp_path / "layout")], check=True)
    for line in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.splitlines():
        cname, field, value = line.split()
        if cname == "max":
            assert int(value) == 0
        elif field == "sizeof":
            assert ctypes.sizeof(structs[cname]) == int(value), cname
        else:
            assert getattr(structs[cname], field).offset == int(value), (cname, field)


def _far(i):
    return FAKE + (i << 32)      # arrays that do not overlap


def _fill(p, fields, changes):
    p.struct_size = ctypes.sizeof(p)
    for k, v in {**fields, **changes}.items():
        setattr(p, k, v)
    return p


def _probs(ia, **kw):
    return _fill(ia.TokenProbsParams(), dict(N_tok=4, V=100, logits_dtype=1, logits_stride=100, probs_stride=100,
                                             logits=_far(0), probs=_far(1), temperature=_far(2), dev_status=_far(3)), kw)


def _verify(ia, **kw):
    names = ("target_p", "draft_p", "token_ids", "cu_seqlens_q", "u_accept", "u_sample", "n_new", "out_tokens", "dev_status")
    return _fill(ia.VerifyDraftsParams(), dict(B=2, N_tok=6, V=100, target_stride=100, draft_stride=100,
                                               **{n: _far(i) for i, n in enumerate(names)}), kw)


def _rollback(ia, state=None, **kw):
    names = ("cu_seqlens_q", "state_slot", "n_keep", "dev_status")
    p = _fill(ia.ConvRollbackParams(), dict(B=2, N_tok=6, num_state_slots=4, n_states=2,
                                            **{n: _far(i) for i, n in enumerate(names)}), kw)
    for s in range(2):
        c = p.states[s]
        c.C, c.x_stride, c.x, c.state_before, c.state_after = 64, 64, _far(10 + s), _far(20 + s), _far(30 + s)
    for k, v in (state or {}).items():
        setattr(p.states[1], k, v)
    return p


@pytest.mark.parametrize("kw", [
    dict(struct_size=8), dict(N_tok=-1), dict(N_tok=(1 << 24) + 1), dict(V=0), dict(V=(1 << 20) + 1), dict(logits_stride=99),
    dict(probs_stride=99), dict(logits_stride=(1 << 32) + 1), dict(logits_dtype=2), dict(logits=None), dict(probs=None),
    dict(logits=FAKE + 2), dict(probs=_far(1) + 2), dict(temperature=_far(2) + 1), dict(dev_status=_far(3) + 2),
    dict(probs=_far(0) + 16),                                   # in part over the logits
    dict(probs=_far(0), probs_stride=104),                      # over them with another stride
    dict(probs=_far(0), logits_dtype=0),                        # over bf16 logits
    dict(temperature=_far(1) + 8), dict(dev_status=_far(1) + 8)])
def test_token_probs_refusals(ia, kw):
    assert ia.inkattn_token_probs(_probs(ia, **kw), stream=0, raise_on_error=False) == ia.INKATTN_ERR_INVALID_ARG
    assert ia.lib().inkattn_token_probs(None, None) == ia.INKATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(struct_size=8), dict(B=0), dict(B=(1 << 20) + 1), dict(N_tok=-1), dict(N_tok=(1 << 24) + 1), dict(V=0),
    dict(V=(1 << 20) + 1), dict(target_stride=99), dict(draft_stride=99), dict(target_p=None), dict(token_ids=None),
    dict(cu_seqlens_q=None), dict(u_accept=None), dict(u_sample=None), dict(n_new=None), dict(out_tokens=None),
    dict(target_p=FAKE + 2), dict(out_tokens=_far(7) + 2), dict(draft_p=_far(1) + 1),
    dict(out_tokens=_far(2)), dict(n_new=_far(7) + 20), dict(n_new=_far(0) + 400), dict(out_tokens=_far(1) + 2396),
    dict(dev_status=_far(6)), dict(dev_status=_far(3) + 4)])
def test_verify_drafts_refusals(ia, kw):
    assert ia.inkattn_verify_drafts(_verify(ia, **kw), stream=0, raise_on_error=False) == ia.INKATTN_ERR_INVALID_ARG
    assert ia.lib().inkattn_verify_drafts(None, None) == ia.INKATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(struct_size=8), dict(B=0), dict(B=65536), dict(N_tok=-1), dict(num_state_slots=0), dict(n_states=0),
    dict(n_states=9), dict(cu_seqlens_q=None), dict(state_slot=None), dict(n_keep=None), dict(n_keep=_far(2) + 2),
    dict(state=dict(C=60)), dict(state=dict(C=0)), dict(state=dict(C=72)), dict(state=dict(x_stride=68)), dict(state=dict(x=None)),
    dict(state=dict(x=_far(11) + 8)), dict(state=dict(state_before=None)), dict(state=dict(state_after=_far(31) + 8)),
    dict(state=dict(state_after=_far(21) + 16)),                # in part over its own state before
    dict(state=dict(state_after=_far(30))), dict(state=dict(state_after=_far(20))), dict(state=dict(state_after=_far(10))),
    dict(state=dict(state_after=_far(2))), dict(dev_status=_far(31))])
def test_conv_rollback_refusals(ia, kw):
    assert ia.inkattn_conv_rollback(_rollback(ia, **kw), stream=0, raise_on_error=False) == ia.INKATTN_ERR_INVALID_ARG
    assert ia.lib().inkattn_conv_rollback(None, None) == ia.INKATTN_ERR_INVALID_ARG


def test_valid_params_get_past_the_checks(ia):
    """Made without a GPU, or with arrays that are not on it, a valid call fails later than its checks."""
    calls = [(ia.inkattn_token_probs, _probs(ia)), (ia.inkattn_token_probs, _probs(ia, probs=_far(0))),
             (ia.inkattn_verify_drafts, _verify(ia)), (ia.inkattn_verify_drafts, _verify(ia, draft_p=None, draft_stride=0)),
             (ia.inkattn_conv_rollback, _rollback(ia)),
             (ia.inkattn_conv_rollback, _rollback(ia, state=dict(state_after=_far(21))))]
    for call, p in calls:
        status = call(p, stream=0, raise_on_error=False)
        if not torch.cuda.is_available():
            assert status in (ia.INKATTN_ERR_CUDA, ia.INKATTN_ERR_UNSUPPORTED)


def test_binding_checks_shapes_types_and_rows(ia):
    f, i = torch.float32, torch.int32
    z = torch.zeros
    with pytest.raises(ValueError):
        ia.token_probs_params(logits=z(4, 10), probs=z(4, 11))
    with pytest.raises(TypeError):
        ia.token_probs_params(logits=z(4, 10, dtype=torch.float16), probs=z(4, 10))
    with pytest.raises(ValueError):
        ia.token_probs_params(logits=z(10, 4).t(), probs=z(4, 10))
    with pytest.raises(ValueError):
        ia.token_probs_params(logits=z(1, 10).expand(4, 10), probs=z(4, 10))
    p = ia.token_probs_params(logits=z(4, 16)[:, :10], probs=z(4, 12)[:, :10], temperature=z(4))
    assert (p.N_tok, p.V, p.logits_stride, p.probs_stride) == (4, 10, 16, 12)
    ok = dict(target_p=z(3, 10), token_ids=z(3, dtype=i), cu_seqlens_q=z(2, dtype=i), u_accept=z(3), u_sample=z(1),
              n_new=z(1, dtype=i), out_tokens=z(3, dtype=i))
    assert ia.verify_drafts_params(**ok).draft_p is None
    for bad in (dict(draft_p=z(3, 9)), dict(u_accept=z(2)), dict(n_new=z(2, dtype=i)), dict(out_tokens=z(4, dtype=i))):
        with pytest.raises(ValueError):
            ia.verify_drafts_params(**{**ok, **bad})
    with pytest.raises(TypeError):
        ia.verify_drafts_params(**{**ok, "token_ids": z(3, dtype=torch.int64)})
    b = torch.bfloat16
    one = dict(x=[z(3, 16, dtype=b)], state_before=[z(2, 3, 16, dtype=b)], state_after=[z(2, 3, 16, dtype=b)],
               n_keep=z(1, dtype=i), cu_seqlens_q=z(2, dtype=i), state_slot=z(1, dtype=i))
    assert ia.conv_rollback_params(**one).states[0].x_stride == 16
    wide = ia.conv_rollback_params(**{**one, "x": [z(3, 48, dtype=b)[:, 16:32]]})
    assert wide.states[0].x_stride == 48 and wide.states[0].C == 16
    for bad in (dict(x=[]), dict(x=[z(3, 8, dtype=b)]), dict(state_after=[z(2, 2, 16, dtype=b)]), dict(n_keep=z(2, dtype=i))):
        with pytest.raises(ValueError):
            ia.conv_rollback_params(**{**one, **bad})


def _attn(ia, **kw):
    names = ("q", "r", "P", "k_cache", "v_cache", "k_scale", "v_scale", "cu_seqlens_q", "seqlen_k", "block_table", "out")
    return _fill(ia.AttnParams(), dict(B=2, N_tok=2, max_seqlen_q=1, max_seqlen_k=64, Hq=8, Hkv=1, head_dim=128, block_size=64,
                                       num_blocks=4, max_blocks_per_seq=1, d_r=32, rel_extent=16, kv_dtype=ia.INKATTN_KV_I4,
                                       **{n: _far(i) for i, n in enumerate(names)}), kw)


def test_four_bit_caches_are_refused_where_they_are_not_read(ia):
    none = dict(stream=0, raise_on_error=False)
    assert ia.inkattn_prefill(_attn(ia), **none) == ia.INKATTN_ERR_UNSUPPORTED
    assert ia.inkattn_prefill_e4m3(_attn(ia), None, **none) == ia.INKATTN_ERR_INVALID_ARG
    for kv in (ia.INKATTN_KV_BF16, ia.INKATTN_KV_E4M3):
        assert ia.inkattn_prefill_i4(_attn(ia, kv_dtype=kv), None, **none) == ia.INKATTN_ERR_INVALID_ARG
    size = ia.inkattn_prefill_workspace_bytes(_attn(ia))
    assert size == 2 * (2 * 64 * 128 * 2) + 256
    assert ia.inkattn_prefill_i4(_attn(ia), None, **none) == ia.INKATTN_ERR_INVALID_ARG      # no workspace
    for bad in (dict(k_scale=None), dict(v_scale=None), dict(k_scale=_far(5) + 4), dict(kv_dtype=3), dict(kv_dtype=5)):
        for call in (ia.inkattn_decode, ia.inkattn_combine):
            assert call(_attn(ia, **bad), 1, None, **none) == ia.INKATTN_ERR_INVALID_ARG


def test_binding_tells_the_caches_apart_by_their_rows(ia):
    u8, i = torch.uint8, torch.int32

    def params(k, v, ks, vs):
        return ia.attn_params(q=torch.zeros((1, 4, 128), dtype=torch.bfloat16), k_cache=k, v_cache=v, k_scale=ks, v_scale=vs,
                              cu_seqlens_q=torch.zeros(2, dtype=i), seqlen_k=torch.zeros(1, dtype=i),
                              block_table=torch.zeros((1, 1), dtype=i), out=torch.zeros((1, 4, 128)), max_seqlen_q=1,
                              max_seqlen_k=1)
    k4, s4 = torch.zeros((3, 2, 64, 64), dtype=u8), torch.zeros((3, 2, 64, 4), dtype=u8)
    assert params(k4, k4.clone(), s4, s4.clone()).kv_dtype == ia.INKATTN_KV_I4
    k8, s8 = torch.zeros((3, 2, 64, 128), dtype=u8), torch.zeros((3, 2, 64))
    assert params(k8, k8.clone(), s8, s8.clone()).kv_dtype == ia.INKATTN_KV_E4M3
    with pytest.raises(ValueError):
        params(k4, k4.clone(), s4[:2], s4.clone())
    with pytest.raises(ValueError):
        params(k4, k8, s4, s4.clone())
    with pytest.raises(TypeError):
        params(k4, k4.clone(), s4.float(), s4.clone())
