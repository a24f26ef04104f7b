"""The key/value-cache entry points reject bad arguments on the host before
any launch, their argument structs have the header's layout, and the binding
rejects what it can see.  No GPU needed."""
import ctypes
import os
import subprocess

import pytest

from nvfp4_block_scaled_02_amd import _native as N

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x100000  # aligned non-null address that is never dereferenced
INV, UNS = N.ERR_INVALID, N.ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


def _cache(**kw):
    a = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, k_amax=FAKE, v_amax=FAKE,
             num_pages=10, kv_heads=2, page_size=16, head_dim=128, global_fp8_max=256.0)
    a.update(kw)
    return N.KVCacheArgs(**a)


BAD_CACHES = [
    (dict(k_codes=None), INV), (dict(k_scales=None), INV), (dict(v_codes=None), INV),
    (dict(v_scales=FAKE + 8), INV), (dict(k_codes=FAKE + 4), INV), (dict(k_amax=None), INV),
    (dict(v_amax=FAKE + 2), INV), (dict(num_pages=0), INV), (dict(num_pages=-1), INV),
    (dict(num_pages=1 << 31), INV), (dict(kv_heads=0), INV), (dict(kv_heads=1025), INV),
    (dict(page_size=0), INV), (dict(page_size=24), INV), (dict(page_size=4), INV),
    (dict(page_size=2048), INV), (dict(page_size=-16), INV), (dict(global_fp8_max=0.0), INV),
    (dict(global_fp8_max=NAN), INV), (dict(global_fp8_max=INF), INV), (dict(head_dim=0), INV),
    (dict(head_dim=120), INV), (dict(num_pages=(1 << 31) - 1, kv_heads=1024, page_size=1024), INV),
    (dict(head_dim=32), UNS), (dict(head_dim=96), UNS), (dict(head_dim=320), UNS),
]

PLAN = dict(ctx_lens=FAKE, new_lens=FAKE, batch=3, block_table=FAKE, table_width=8,
            free_pages=FAKE, free_count=FAKE, num_pages=10, page_size=16, tokens=5, cu_new=FAKE,
            seq_lens=FAKE, positions=FAKE, slots=FAKE, free_count_out=FAKE, refused=FAKE)


@pytest.mark.parametrize("kw", [
    dict(ctx_lens=None), dict(new_lens=None), dict(seq_lens=None), dict(block_table=None),
    dict(positions=None), dict(slots=None), dict(free_pages=None), dict(free_count=None),
    dict(cu_new=None), dict(free_count_out=None), dict(refused=None), dict(batch=-1),
    dict(tokens=-1), dict(table_width=-1), dict(batch=1 << 31), dict(tokens=1 << 31),
    dict(table_width=1 << 31), dict(num_pages=0), dict(num_pages=1 << 31), dict(page_size=4),
    dict(page_size=48), dict(page_size=2048), dict(page_size=0), dict(slots=FAKE + 4),
    dict(ctx_lens=FAKE + 1), dict(refused=FAKE + 2), dict(batch=1 << 30, table_width=1 << 30),
])
def test_plan_rejects(kw):
    assert N.lib().nvfp4_kv_plan(N.KVPlanArgs(**{**PLAN, **kw}), None) == INV


def test_null_argument_structs():
    l = N.lib()
    assert l.nvfp4_kv_plan(None, None) == INV
    assert l.nvfp4_qk_norm_rope(None, None) == INV
    assert l.nvfp4_qk_norm_rope_bwd(None, FAKE, 256, FAKE, 256, None, None, None, None) == INV
    assert l.nvfp4_kv_append(None, None) == INV
    assert l.nvfp4_kv_read(None, FAKE, 1, FAKE, FAKE, None) == INV
    assert l.nvfp4_kv_attention(None, None) == INV
    assert l.nvfp4_kv_attention_workspace_bytes(None) == 0


QK = dict(q=FAKE, k=FAKE, tokens=4, q_heads=8, k_heads=2, head_dim=128, q_stride=1024,
          k_stride=256, positions=FAKE, cos=FAKE, sin=FAKE, max_pos=64, rot_dim=128, pairs=0,
          q_weight=FAKE, k_weight=FAKE, eps=1e-6, q_out=FAKE, k_out=FAKE, q_out_stride=1024,
          k_out_stride=256)
BAD_QK = [
    (dict(q=None), INV), (dict(k=None), INV), (dict(q_out=None), INV), (dict(q=FAKE + 4), INV),
    (dict(tokens=-1), INV), (dict(q_heads=-1), INV), (dict(q_heads=0, k_heads=0), INV),
    (dict(q_heads=1025, q_stride=1 << 20), INV), (dict(head_dim=0), INV), (dict(head_dim=100), INV),
    (dict(q_stride=1020), INV), (dict(k_stride=0), INV), (dict(q_stride=1026), INV),
    (dict(q_out_stride=512), INV), (dict(q_out_stride=-1024), INV), (dict(positions=None), INV),
    (dict(cos=None), INV), (dict(sin=FAKE + 4), INV), (dict(max_pos=0), INV), (dict(rot_dim=-32), INV),
    (dict(rot_dim=160), INV), (dict(pairs=2), INV), (dict(pairs=-1), INV), (dict(eps=-1.0), INV),
    (dict(eps=NAN), INV), (dict(eps=INF), INV), (dict(q_weight=FAKE + 2), INV),
    (dict(tokens=1 << 40), INV), (dict(rot_dim=48), UNS), (dict(head_dim=112, rot_dim=0), UNS),
    (dict(head_dim=288, q_stride=8 * 288, k_stride=576, q_out_stride=8 * 288, k_out_stride=576), UNS),
]


@pytest.mark.parametrize("kw,want", BAD_QK + [(dict(k_out=None), INV), (dict(k_out_stride=128), INV)])
def test_norm_rope_rejects(kw, want):
    assert N.lib().nvfp4_qk_norm_rope(N.QKArgs(**{**QK, **kw}), None) == want


def test_norm_rope_empty_is_ok():
    l = N.lib()
    assert l.nvfp4_qk_norm_rope(N.QKArgs(**{**QK, "tokens": 0, "q": None, "k": None}), None) == N.OK


def _bwd(qk=None, **kw):
    a = dict(gq=FAKE, gqs=1024, gk=FAKE, gks=256, dqw=FAKE, dkw=FAKE, ws=FAKE)
    a.update(kw)
    return N.lib().nvfp4_qk_norm_rope_bwd(N.QKArgs(**{**QK, **(qk or {})}), a["gq"], a["gqs"],
                                          a["gk"], a["gks"], a["dqw"], a["dkw"], a["ws"], None)


@pytest.mark.parametrize("kw", [
    dict(gq=None), dict(gk=None), dict(gq=FAKE + 4), dict(gqs=1020), dict(gks=128), dict(dqw=None),
    dict(dkw=None), dict(dqw=FAKE + 2), dict(ws=None), dict(ws=FAKE + 8),
])
def test_norm_rope_bwd_rejects(kw):
    assert _bwd(**kw) == INV


def test_norm_rope_bwd_weight_gradients_follow_the_weights():
    assert _bwd(dict(q_weight=None)) == INV and _bwd(dict(k_weight=None)) == INV
    assert _bwd(dict(q_weight=None, k_weight=None, tokens=0), dqw=None, dkw=None, ws=None) == N.OK
    for kw, want in BAD_QK:
        assert _bwd(kw, gqs=4096, gks=4096) == want, kw
    l = N.lib()
    assert l.nvfp4_qk_norm_rope_bwd_workspace_bytes(0) == 0
    assert l.nvfp4_qk_norm_rope_bwd_workspace_bytes(128) > 0


def _append(qk=None, cache=None, **kw):
    a = dict(v=FAKE, v_stride=256, slots=FAKE, select=1)
    a.update(kw)
    return N.lib().nvfp4_kv_append(N.KVAppendArgs(qk=N.QKArgs(**{**QK, **(qk or {})}),
                                                  cache=_cache(**(cache or {})), **a), None)


@pytest.mark.parametrize("kw,want", [
    (dict(v=None), INV), (dict(v=FAKE + 4), INV), (dict(v_stride=128), INV), (dict(v_stride=258), INV),
    (dict(slots=None), INV), (dict(slots=FAKE + 4), INV), (dict(select=5), INV), (dict(select=-1), INV),
    (dict(select=2), UNS), (dict(select=3), UNS), (dict(select=4), UNS),
])
def test_append_rejects(kw, want):
    assert _append(**kw) == want


def test_append_rejects_what_its_parts_reject():
    for kw, want in BAD_CACHES:
        if "head_dim" not in kw:
            assert _append(cache=kw) == want, kw
    for kw, want in BAD_QK:
        if "head_dim" not in kw and not set(kw) & {"k_out", "k_out_stride"}:
            assert _append(qk=kw) == want, kw
    assert _append(cache=dict(head_dim=64)) == INV  # not the keys' width
    assert _append(cache=dict(kv_heads=4)) == INV
    assert _append(qk=dict(tokens=0)) == N.OK


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_read_and_attention_reject_bad_caches(kw, want):
    l, c = N.lib(), _cache(**kw)
    assert l.nvfp4_kv_read(c, FAKE, 1, FAKE, FAKE, None) == want
    q_heads = 2 * max(1, kw.get("kv_heads", 2))
    assert _attn(cache=kw, q_heads=min(q_heads, 1024), q_stride=1 << 20) == want


def test_read_rejects():
    l, c = N.lib(), _cache()
    assert l.nvfp4_kv_read(c, None, 1, FAKE, FAKE, None) == INV
    assert l.nvfp4_kv_read(c, FAKE + 4, 1, FAKE, FAKE, None) == INV
    assert l.nvfp4_kv_read(c, FAKE, -1, FAKE, FAKE, None) == INV
    assert l.nvfp4_kv_read(c, FAKE, 1 << 42, FAKE, FAKE, None) == INV
    assert l.nvfp4_kv_read(c, FAKE, 1, None, None, None) == INV
    assert l.nvfp4_kv_read(c, FAKE, 1, FAKE + 4, None, None) == INV
    assert l.nvfp4_kv_read(c, None, 0, FAKE, None, None) == N.OK


def _attn_args(cache=None, **kw):
    a = dict(q=FAKE, tokens=6, q_stride=1024, q_heads=8, block_table=FAKE, batch=3, table_width=8,
             seq_lens=FAKE, cu_q=FAKE, max_seq_len=128, scale=0.1, causal=1, window=0, out=FAKE,
             lse=None, workspace=FAKE)
    a.update(kw)
    return N.KVAttentionArgs(cache=_cache(**(cache or {})), **a)


def _attn(cache=None, **kw):
    return N.lib().nvfp4_kv_attention(_attn_args(cache, **kw), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(q=FAKE + 8), dict(out=FAKE + 8), dict(lse=FAKE + 2),
    dict(cu_q=FAKE + 2), dict(cu_q=None), dict(tokens=-1), dict(batch=-1), dict(table_width=-1),
    dict(max_seq_len=-1), dict(window=-1), dict(tokens=1 << 31), dict(batch=1 << 31),
    dict(table_width=1 << 31), dict(max_seq_len=1 << 31), dict(q_heads=0), dict(q_heads=7),
    dict(q_heads=1026, q_stride=1 << 20), dict(q_stride=512), dict(q_stride=1028), dict(scale=NAN),
    dict(scale=INF), dict(seq_lens=None), dict(block_table=None), dict(workspace=FAKE + 8),
    dict(batch=1 << 30, table_width=1 << 30), dict(q_heads=-8),
])
def test_attention_rejects(kw):
    assert _attn(**kw) == INV


def test_attention_counters_are_aligned_and_change_no_size():
    assert _attn(counters=FAKE + 8) == INV
    for kw in (dict(tokens=3, cu_q=None), dict(tokens=3), dict(tokens=6)):
        a, b = (_attn_args(max_seq_len=100000, counters=c, **kw) for c in (None, FAKE))
        assert N.lib().nvfp4_kv_attention_workspace_bytes(a) == N.lib().nvfp4_kv_attention_workspace_bytes(b) > 0


def test_attention_positions_stay_in_32_bits():
    assert _attn(table_width=(1 << 26) + 1) == UNS


def test_attention_empty_is_ok_and_workspace_is_required():
    assert _attn(tokens=0, q=None, out=None, workspace=None) == N.OK
    l = N.lib()
    args = _attn_args(tokens=3, cu_q=None, max_seq_len=100000)
    if l.nvfp4_kv_attention_workspace_bytes(args):
        args.workspace = None
        assert l.nvfp4_kv_attention(args, None) == INV


@pytest.mark.parametrize("c_name,struct", [
    ("nvfp4_kv_cache", N.KVCacheArgs), ("nvfp4_kv_plan_args", N.KVPlanArgs),
    ("nvfp4_qk_args", N.QKArgs), ("nvfp4_kv_append_args", N.KVAppendArgs),
    ("nvfp4_kv_attention_args", N.KVAttentionArgs)])
def test_struct_layouts_match_the_header(tmp_path, c_name, struct):
    src = tmp_path / "layout.c"
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "nvfp4.h"', "int main(void) {"]
    lines += [f'  printf("%zu\\n", offsetof({c_name}, {f}));' for f, _ in struct._fields_]
    lines += [f'  printf("%zu\\n", sizeof({c_name}));',
              "  return 0;", "}"]
    src.write_text("\n".join(lines) + "\n")
    exe = tmp_path / "layout"
    r = subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", f"-I{ROOT}/include",
                        "-I/opt/rocm/include", str(src), "-o", str(exe)], capture_output=True, text=True)
    if r.returncode != 0:
        pytest.skip(f"cannot build a host program against the HIP headers: {r.stderr[:200]}")
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [getattr(struct, f).offset for f, _ in struct._fields_] + [ctypes.sizeof(struct)]


def test_binding_rejects_host_tensors():
    torch = pytest.importorskip("torch")
    import nvfp4_block_scaled_02_amd as nv
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        nv.qk_norm_rope(x, x)
    with pytest.raises(ValueError, match="GPU"):
        nv.kv_plan(i, i, i.view(4, 1), i, i[:1], page_size=16, num_pages=4, tokens=4)
    with pytest.raises(ValueError, match="q, k or both"):
        nv.qk_norm_rope(None, None)
    with pytest.raises(ValueError, match="pairs"):
        nv.qk_norm_rope(x, x, pairs="other")
    with pytest.raises(ValueError, match="GPU"):
        nv.kv_cache(4, 2, 16, 64, torch.ones(2), torch.ones(2))
