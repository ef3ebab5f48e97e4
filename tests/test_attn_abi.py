"""Refusals of the attention layer's entry points, on the CPU: no call here reaches a kernel (each fails validation or
has nothing to do)."""
import pytest

import linear_attention_sequence_gated_amd as gdn
from linear_attention_sequence_gated_amd import gdn as raw

A = 0x10000  # a 16-byte aligned fake address; validation rejects before any use


def tables(**kw):
    args = dict(seq_lens=A, new_lens=A, block_table=A, free_blocks=A, slot_map=A, cu_seqlens=A, lens_after=A, used=A,
                R=4, width=8, n_free=10, block_tokens=16, num_blocks=64, T=100, stream=None)
    args.update(kw)
    return gdn.gdn_block_tables(**args)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), raw.GDN_ERR_SHAPE), (dict(width=-1), raw.GDN_ERR_SHAPE), (dict(n_free=-1), raw.GDN_ERR_SHAPE),
    (dict(T=-1), raw.GDN_ERR_SHAPE), (dict(num_blocks=-1), raw.GDN_ERR_SHAPE), (dict(block_tokens=0), raw.GDN_ERR_SHAPE),
    (dict(R=1 << 20), raw.GDN_ERR_SHAPE), (dict(num_blocks=1 << 27), raw.GDN_ERR_SHAPE),
    (dict(width=1 << 27), raw.GDN_ERR_SHAPE), (dict(block_tokens=48), raw.GDN_ERR_UNSUPPORTED),
    (dict(block_tokens=8), raw.GDN_ERR_UNSUPPORTED), (dict(block_tokens=256), raw.GDN_ERR_UNSUPPORTED),
    *((dict([(n, None)]), raw.GDN_ERR_NULL) for n in ("seq_lens", "new_lens", "block_table", "free_blocks", "slot_map",
                                                      "cu_seqlens", "lens_after", "used")),
    *((dict([(n, A + 4)]), raw.GDN_ERR_ALIGN) for n in ("seq_lens", "new_lens", "block_table", "free_blocks", "slot_map",
                                                        "cu_seqlens", "lens_after", "used")),
])
def test_tables_argument_errors(kw, status):
    assert tables(**kw) == status


def test_tables_largest_slot_map():
    """Slots are counted in 32 bits, some way past the last: the longest maps are refused, whatever fits below them."""
    assert tables(T=2 ** 31 - 1) == raw.GDN_ERR_SHAPE and tables(T=2 ** 31 - 4096) == raw.GDN_ERR_SHAPE
    assert tables(T=2 ** 31 - 4097, slot_map=None) == raw.GDN_ERR_NULL  # past the check of sizes


def append(**kw):
    args = dict(k=A, v=A, slot_map=A, k_cache=A, v_cache=A, k_scale=A, v_scale=A, k_stride=256, v_stride=256, T=10,
                Hkv=4, D=64, block_tokens=16, num_blocks=64, dtype=gdn.GDN_BF16, cache_format=gdn.GDN_CACHE_I8, stream=None)
    args.update(kw)
    return gdn.gdn_cache_append(**args)


CACHE_ERRORS = [
    (dict(dtype=7), raw.GDN_ERR_DTYPE), (dict(dtype=gdn.GDN_F32), raw.GDN_ERR_UNSUPPORTED),
    (dict(dtype=gdn.GDN_C64), raw.GDN_ERR_UNSUPPORTED), (dict(cache_format=2), raw.GDN_ERR_DTYPE),
    (dict(cache_format=-1), raw.GDN_ERR_DTYPE), (dict(Hkv=0), raw.GDN_ERR_SHAPE), (dict(D=0), raw.GDN_ERR_SHAPE),
    (dict(num_blocks=-1), raw.GDN_ERR_SHAPE), (dict(num_blocks=1 << 27), raw.GDN_ERR_SHAPE),
    (dict(block_tokens=0), raw.GDN_ERR_SHAPE), (dict(block_tokens=24), raw.GDN_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", CACHE_ERRORS + [
    (dict(T=-1), raw.GDN_ERR_SHAPE), (dict(T=1 << 26), raw.GDN_ERR_SHAPE), (dict(D=96, k_stride=384, v_stride=384), raw.GDN_ERR_UNSUPPORTED),
    (dict(k_stride=255), raw.GDN_ERR_SHAPE), (dict(v_stride=248), raw.GDN_ERR_SHAPE), (dict(k_stride=260), raw.GDN_ERR_SHAPE),
    (dict(k_stride=-256), raw.GDN_ERR_SHAPE),
    *((dict([(n, None)]), raw.GDN_ERR_NULL) for n in ("k", "v", "slot_map", "k_cache", "v_cache", "k_scale", "v_scale")),
    *((dict([(n, A + 8)]), raw.GDN_ERR_ALIGN) for n in ("k", "v", "slot_map", "k_cache", "v_cache", "k_scale", "v_scale")),
])
def test_append_argument_errors(kw, status):
    assert append(**kw) == status


def test_append_of_nothing_is_noop():
    none = dict(k=None, v=None, slot_map=None, k_cache=None, v_cache=None, k_scale=None, v_scale=None)
    assert append(T=0, **none) == raw.GDN_OK
    assert append(num_blocks=0, **none) == raw.GDN_OK


def decode(**kw):
    args = dict(q=A, k_cache=A, v_cache=A, k_scale=A, v_scale=A, block_table=A, seq_lens=A, out=A, lse=A, scale=0.125,
                q_stride=512, R=3, Hq=8, Hkv=4, D=64, block_tokens=16, num_blocks=64, width=72, dtype=gdn.GDN_BF16,
                cache_format=gdn.GDN_CACHE_I8, workspace=A, workspace_bytes=1 << 40, stream=None)
    args.update(kw)
    return gdn.gdn_attn_decode(**args)


@pytest.mark.parametrize("kw,status", CACHE_ERRORS + [
    (dict(R=-1), raw.GDN_ERR_SHAPE), (dict(R=1 << 20), raw.GDN_ERR_SHAPE), (dict(width=-1), raw.GDN_ERR_SHAPE),
    (dict(width=1 << 27), raw.GDN_ERR_SHAPE), (dict(Hq=6), raw.GDN_ERR_SHAPE), (dict(Hq=0), raw.GDN_ERR_SHAPE),
    (dict(R=1 << 19, Hq=64, q_stride=4096), raw.GDN_ERR_SHAPE), (dict(R=1 << 18, width=1 << 26), raw.GDN_ERR_SHAPE),
    (dict(D=32), raw.GDN_ERR_UNSUPPORTED), (dict(q_stride=504), raw.GDN_ERR_SHAPE), (dict(q_stride=516), raw.GDN_ERR_SHAPE),
    *((dict([(n, None)]), raw.GDN_ERR_NULL) for n in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table",
                                                      "seq_lens", "out")),
    *((dict([(n, A + 8)]), raw.GDN_ERR_ALIGN) for n in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table",
                                                        "seq_lens", "out", "lse", "workspace")),
    (dict(workspace=None), raw.GDN_ERR_WORKSPACE), (dict(workspace_bytes=0), raw.GDN_ERR_WORKSPACE),
])
def test_decode_argument_errors(kw, status):
    assert decode(**kw) == status


def test_decode_workspace():
    need = gdn.gdn_attn_decode_workspace_bytes(3, 8, 4, 64, 16, 72)  # 9 units of 128 tokens and one ahead of them x 3 x 4, two shares each
    assert need == 2 * 120 * 2 * 66 * 4
    assert decode(workspace_bytes=need - 1) == raw.GDN_ERR_WORKSPACE
    assert gdn.gdn_attn_decode_workspace_bytes(3, 8, 3, 64, 16, 72) == 0  # unsupported arguments
    assert gdn.gdn_attn_decode_workspace_bytes(3, 8, 4, 64, 16, 9) == 0  # short: nothing to join
    assert decode(R=0, q=None, seq_lens=None, out=None) == raw.GDN_OK


def test_decode_forms_follow_groups_and_widths():
    """The longest table, in units of 128 tokens, that one workgroup to a request and key head takes: it grows with
    their number while each has a CU, whatever the head size, and again with how many wait for one."""
    for D in (64, 128):
        def whole(groups):
            units = 0
            while gdn.gdn_attn_decode_workspace_bytes(groups, 1, 1, D, 128, units + 1) == 0:
                units += 1
            return units
        few = [whole(g) for g in range(1, 257)]
        assert few == sorted(few) and few[0] == 8 and max(b - a for a, b in zip(few, few[1:])) == 1
        many = [whole(g) for g in range(257, 1200, 7)]
        assert many == sorted(many) and many[-1] == 64 and max(b - a for a, b in zip(many, many[1:])) == 1


def test_decode_longest_tables():
    """A length on the device may be anything and is cut to the table's width; tokens are counted in 32 bits, some way
    past that, so the widest tables are refused."""
    for bt in (16, 128):
        for w in ((2 ** 31 - 1) // bt, (2 ** 31 - 4096) // bt):
            assert decode(R=1, block_tokens=bt, width=w) == raw.GDN_ERR_SHAPE
            assert gdn.gdn_attn_decode_workspace_bytes(1, 8, 4, 64, bt, w) == 0
        w = (2 ** 31 - 4096) // bt - 1
        assert decode(R=1, block_tokens=bt, width=w, workspace=None) == raw.GDN_ERR_WORKSPACE  # past the check of sizes


def prompt(**kw):
    args = dict(q=A, k=A, v=A, cu_seqlens=A, out=A, lse=A, scale=0.125, q_stride=512, k_stride=256, v_stride=256, T=100,
                R=3, Hq=8, Hkv=4, D=64, dtype=gdn.GDN_BF16, zero_rest=0, stream=None)
    args.update(kw)
    return gdn.gdn_attn_prompt(**args)


PROMPT_ERRORS = [
    (dict(dtype=3), raw.GDN_ERR_DTYPE), (dict(dtype=gdn.GDN_F32), raw.GDN_ERR_UNSUPPORTED),
    (dict(T=-1), raw.GDN_ERR_SHAPE), (dict(R=-1), raw.GDN_ERR_SHAPE), (dict(R=1 << 20), raw.GDN_ERR_SHAPE),
    (dict(T=1 << 25), raw.GDN_ERR_SHAPE), (dict(Hq=6), raw.GDN_ERR_SHAPE), (dict(Hkv=0), raw.GDN_ERR_SHAPE),
    (dict(Hq=-8, Hkv=-4), raw.GDN_ERR_SHAPE), (dict(D=0), raw.GDN_ERR_SHAPE), (dict(D=256), raw.GDN_ERR_UNSUPPORTED),
    (dict(q_stride=256), raw.GDN_ERR_SHAPE), (dict(k_stride=252), raw.GDN_ERR_SHAPE), (dict(v_stride=260), raw.GDN_ERR_SHAPE),
    (dict(k_stride=1 << 24), raw.GDN_ERR_SHAPE),
]


@pytest.mark.parametrize("kw,status", PROMPT_ERRORS + [
    *((dict([(n, None)]), raw.GDN_ERR_NULL) for n in ("q", "k", "v", "cu_seqlens", "out", "lse")),
    *((dict([(n, A + 8)]), raw.GDN_ERR_ALIGN) for n in ("q", "k", "v", "cu_seqlens", "out", "lse")),
])
def test_prompt_argument_errors(kw, status):
    assert prompt(**kw) == status


def test_prompt_of_nothing_is_noop():
    none = dict(q=None, k=None, v=None, cu_seqlens=None, out=None, lse=None)
    assert prompt(T=0, **none) == raw.GDN_OK


# lse and delta [8, 100], and the sums of two shares of the query heads of a key head [2, 2, 100, 4, 64]
BWD_NEED = 2 * 100 * 8 * 4 + 2 * 2 * 100 * 4 * 64 * 4


def prompt_bwd(**kw):
    args = dict(q=A, k=A, v=A, out=A, lse=A, grad_out=A, cu_seqlens=A, grad_q=A, grad_k=A, grad_v=A, scale=0.125,
                q_stride=512, k_stride=256, v_stride=256, grad_out_stride=512, grad_q_stride=512, grad_k_stride=256,
                grad_v_stride=256, T=100, R=3, Hq=8, Hkv=4, D=64, dtype=gdn.GDN_BF16, zero_rest=0,
                workspace=A, workspace_bytes=1 << 40, stream=None)
    args.update(kw)
    return gdn.gdn_attn_prompt_bwd(**args)


@pytest.mark.parametrize("kw,status", PROMPT_ERRORS + [
    *((dict([(n + "_stride", 508)]), raw.GDN_ERR_SHAPE) for n in ("grad_out", "grad_q")),
    *((dict([(n + "_stride", 248)]), raw.GDN_ERR_SHAPE) for n in ("grad_k", "grad_v")),
    *((dict([(n, None)]), raw.GDN_ERR_NULL) for n in ("q", "k", "v", "out", "lse", "grad_out", "cu_seqlens", "grad_q",
                                                      "grad_k", "grad_v")),
    *((dict([(n, A + 8)]), raw.GDN_ERR_ALIGN) for n in ("q", "k", "v", "out", "lse", "grad_out", "cu_seqlens", "grad_q",
                                                        "grad_k", "grad_v", "workspace")),
    (dict(workspace=None), raw.GDN_ERR_WORKSPACE), (dict(workspace_bytes=BWD_NEED - 1), raw.GDN_ERR_WORKSPACE),
])
def test_prompt_bwd_argument_errors(kw, status):
    assert prompt_bwd(**kw) == status


def test_prompt_bwd_workspace():
    assert gdn.gdn_attn_prompt_bwd_workspace_bytes(100, 8, 4, 64) == BWD_NEED
    # a key head per query head, or tiles enough for one workgroup each: no shares
    assert gdn.gdn_attn_prompt_bwd_workspace_bytes(100, 8, 8, 64) == 2 * 100 * 8 * 4
    assert gdn.gdn_attn_prompt_bwd_workspace_bytes(1 << 20, 8, 4, 64) == 2 * (1 << 20) * 8 * 4
    assert gdn.gdn_attn_prompt_bwd_workspace_bytes(100, 8, 3, 64) == 0
    none = {n: None for n in ("q", "k", "v", "out", "lse", "grad_out", "cu_seqlens", "grad_q", "grad_k", "grad_v", "workspace")}
    assert prompt_bwd(T=0, **none) == raw.GDN_OK


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf"), 1e39])
@pytest.mark.parametrize("call", [decode, prompt, prompt_bwd])
def test_scales_that_are_no_numbers(call, scale):
    assert call(scale=scale) == raw.GDN_ERR_SHAPE
    assert call(scale=-0.125, q=None) == raw.GDN_ERR_NULL  # past the check


def test_cache_helpers_refuse_on_cpu():
    torch = pytest.importorskip("torch")
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.block_tables(i, i, i.view(2, 2), i, 16, 4, 4)
    x, c, s = torch.zeros(4, 1, 64, dtype=torch.bfloat16), torch.zeros(2, 1, 16, 64, dtype=torch.int8), torch.zeros(2, 1)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.cache_append(x, x, i, c, c, s, s)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.attn_decode(x, c, c, s, s, i.view(4, 1), i)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.attn_prompt(x, x, x, i)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.attn_prompt_bwd(x, x, x, x, s, x, i)
