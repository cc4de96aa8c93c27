"""The serving operators on the CPU: every refusal (checked before anything is
launched), the page sizes, the structures against the header, and the 64-bit
reference that the GPU tests use against hand-derived values.  No GPU needed."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import serve_ref as ref


@pytest.fixture(scope="module")
def df11():
    from entropy_decoding_b200 import build
    build.build()
    from entropy_decoding_b200 import df11 as mod
    return mod


STRUCTS = {"df11_kv_extend_args": "KvExtendArgs", "df11_rope_side": "RopeSide", "df11_qk_norm_rope_args": "QkNormRopeArgs",
           "df11_kv4_cache": "Kv4Cache", "df11_kv4_attention_args": "Kv4AttentionArgs"}
CONSTANTS = {"DF11_FP32": "DF11_FP32", "DF11_DEV_ERR_PAGES": "DEV_ERR_PAGES"}


def test_structures_and_constants_match_the_header(df11, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "df11.h"', "int main(void) {"]
    for c, py in STRUCTS.items():
        for field, _ in getattr(df11, py)._fields_:
            lines.append(f'printf("{c} {field} %zu %zu\\n", offsetof({c}, {field}), sizeof((({c} *)0)->{field}));')
        lines.append(f'printf("{c} sizeof %zu 0\\n", sizeof({c}));')
    for c in CONSTANTS:
        lines.append(f'printf("const {c} %llu 0\\n", (unsigned long long)({c}));')
    src, exe = tmp_path / "abi.c", tmp_path / "abi"
    src.write_text("\n".join(lines + ["return 0; }"]) + "\n")
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", os.path.dirname(df11.HEADER_PATH), str(src), "-o",
                    str(exe)], check=True)
    view = {}
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        a, b, x, y = line.split()
        view[a, b] = (int(x), int(y))
    for c, py in STRUCTS.items():
        cls = getattr(df11, py)
        for field, ctype in cls._fields_:
            assert view[c, field] == (getattr(cls, field).offset, ctypes.sizeof(ctype)), (c, field)
        assert ctypes.sizeof(cls) == view[c, "sizeof"][0]
    for c, py in CONSTANTS.items():
        assert view["const", c][0] == getattr(df11, py)


def test_packed_arguments_are_the_structures(df11):
    """The bytes that the calls pass are those of the structure with the same fields."""
    def numbers(cls, i=3):
        out = []
        for _, t in cls._fields_:
            out += numbers(t, i + 7) if issubclass(t, ctypes.Structure) else [0.5 * i if t is ctypes.c_float else i << 20]
            i += 1
        return out

    def build(cls, values):
        return cls(*[build(t, values) if issubclass(t, ctypes.Structure) else values.pop(0) for _, t in cls._fields_])

    for cls, pack in ((df11.KvExtendArgs, df11._extend_args), (df11.QkNormRopeArgs, df11._rope_args),
                      (df11.Kv4AttentionArgs, df11._attention_args)):
        values = numbers(cls)
        assert pack(*values) == bytes(build(cls, list(values)))


def refused(df11, status, fn, *args, **kw):
    with pytest.raises(df11.Df11Error) as e:
        fn(*args, **kw)
    assert e.value.status == status, (e.value.status, args, kw)


def test_page_bytes(df11):
    for page in (16, 32, 64, 128):
        for d in (64, 128):
            assert df11.df11_kv4_page_bytes(page, 8, d) == page * 8 * 2 * (d // 2 + d // 16)
    for bad in ((8, 8, 128), (48, 8, 128), (256, 8, 128), (16, 0, 128), (16, -1, 128), (16, 1025, 128), (16, 8, 96),
                (16, 8, 256), (0, 8, 128)):
        assert df11.df11_kv4_page_bytes(*bad) == 0


A = 1 << 20  # a 16-byte aligned address; nothing reads it


def test_extend_refusals(df11):
    good = dict(kv_lens_ptr=A, new_lens_ptr=A, n_reqs=2, free_pages_ptr=A, n_free_ptr=A, block_table_ptr=A, max_pages=4,
                page_size=16, kv_lens_out_ptr=A, q_start_ptr=A, slots_ptr=A, positions_ptr=A, max_tokens=8,
                n_free_out_ptr=A)
    bad = [dict(n_reqs=-1), dict(max_pages=-1), dict(max_tokens=-1), dict(page_size=0), dict(page_size=8),
           dict(page_size=24), dict(page_size=256), dict(page_size=-16)]
    bad += [{k: 0} for k in good if k.endswith("_ptr")]
    bad += [{k: A + 2} for k in good if k.endswith("_ptr")] + [dict(slots_ptr=A + 4)]
    for b in bad:
        refused(df11, df11.DF11_EINVAL, df11.df11_kv_extend, **{**good, **b})


def test_extend_refuses_what_it_cannot_count(df11):
    """The kernel counts requests in 31 bits, 512 at a time."""
    args = dict(kv_lens_ptr=A, new_lens_ptr=A, free_pages_ptr=A, n_free_ptr=A, block_table_ptr=A, max_pages=4,
                page_size=16, kv_lens_out_ptr=A, q_start_ptr=A, slots_ptr=A, positions_ptr=A, max_tokens=8,
                n_free_out_ptr=A)
    for n in (2 ** 31 - 512, 2 ** 31 - 1):
        refused(df11, df11.DF11_EUNSUPPORTED, df11.df11_kv_extend, n_reqs=n, **args)


def test_rope_refusals(df11):
    side = (A, 512, A, A, 512, 4)
    good = dict(q=side, k=(A, 512, 0, A, 128, 1), n_tokens=3, head_dim=128, positions_ptr=A, inv_freq_ptr=A, rot_dim=128)
    E, U = df11.DF11_EINVAL, df11.DF11_EUNSUPPORTED

    def q(i, v):
        s = list(side)
        s[i] = v
        return dict(q=tuple(s))

    bad = [(E, q(0, 0)), (E, q(0, A + 8)), (E, q(1, 511)), (E, q(1, 510)), (E, q(1, 514)), (E, q(2, A + 2)), (E, q(3, 0)),
           (E, q(3, A + 2)), (E, q(4, 511)), (E, q(4, 516)), (E, q(5, -1)), (E, q(5, 5)), (E, q(1, 1 << 41)),
           (E, dict(n_tokens=-1)), (U, dict(head_dim=96)), (U, dict(head_dim=0)), (U, dict(head_dim=512)),
           (E, dict(rot_dim=-8)), (E, dict(rot_dim=136)), (E, dict(rot_dim=4)), (E, dict(positions_ptr=0)),
           (E, dict(positions_ptr=A + 2)), (E, dict(inv_freq_ptr=0)), (E, dict(inv_freq_ptr=A + 4)),
           (E, dict(interleaved=2)), (E, dict(eps=-1e-6)), (E, dict(eps=float("nan"))), (E, dict(eps=float("inf")))]
    for status, b in bad:
        refused(df11, status, df11.df11_qk_norm_rope, **{**good, **b})
    # nothing to do: no launch, no error
    df11.df11_qk_norm_rope(**{**good, "n_tokens": 0})
    df11.df11_qk_norm_rope(None, None, 3, 128, A, A, 128)


def test_rope_in_place_refusals(df11):
    """In place, a row is written where it was read: neither at another stride nor in another type."""
    good = dict(q=(A, 512, A, A, 512, 4), k=None, n_tokens=3, head_dim=128, positions_ptr=A, inv_freq_ptr=A, rot_dim=128,
                dtype="bf16")
    for b in [dict(q=(A, 512, A, A, 520, 4)), dict(q=(A, 520, 0, A, 512, 4)), dict(q=None, k=(A, 128, A, A, 136, 1)),
              dict(dtype="fp32"), dict(dtype="fp32", n_tokens=1)]:
        refused(df11, df11.DF11_EINVAL, df11.df11_qk_norm_rope, **{**good, **b})


def test_none_is_null(df11):
    """None for a pointer is a NULL pointer, in each place: refused by the library where one is needed, else taken."""
    E = df11.DF11_EINVAL
    extend = [A, A, 2, A, A, A, 4, 16, A, A, A, A, 8, A]
    for i in (0, 1, 3, 4, 5, 8, 9, 10, 11, 13):
        refused(df11, E, df11.df11_kv_extend, *extend[:i], None, *extend[i + 1:])
    side = (A, 512, None, A, 512, 4)
    for q in ((None, *side[1:]), (*side[:3], None, *side[4:])):
        refused(df11, E, df11.df11_qk_norm_rope, q, None, 3, 128, A, A, 128)
    refused(df11, E, df11.df11_qk_norm_rope, side, None, 3, 128, None, A, 128)
    refused(df11, E, df11.df11_qk_norm_rope, side, None, 3, 128, A, None, 128)
    df11.df11_qk_norm_rope(side, None, 0, 128, None, None, 0)
    c = cache(df11)
    attend = dict(q_ptr=A, q_token_stride=512, o_ptr=A, o_token_stride=512, n_q_heads=4, q_start_ptr=A, kv_lens_ptr=A,
                  block_table_ptr=A, n_reqs=2, max_pages=4, n_tokens=5, max_q_len=3, scale=0.1, workspace_ptr=A,
                  workspace_bytes=1 << 40)
    for name in ("q_ptr", "o_ptr", "q_start_ptr", "kv_lens_ptr", "block_table_ptr", "workspace_ptr"):
        refused(df11, E, df11.df11_kv4_attention, c, **{**attend, name: None})
    for name in ("k_ptr", "v_ptr", "slots_ptr"):
        refused(df11, E, df11.df11_kv4_append, c, **{**dict(k_ptr=A, k_token_stride=256, v_ptr=A, v_token_stride=256,
                                                            slots_ptr=A, n_tokens=3), name: None})
    refused(df11, E, df11.df11_kv4_gather, c, None, 3, A, A)
    # what is no pointer, or a count that is none, stays an error of its own
    for wrong in (["x", *extend[1:]], [*extend[:2], None, *extend[3:]]):
        with pytest.raises(Exception) as e:
            df11.df11_kv_extend(*wrong)
        assert not isinstance(e.value, df11.Df11Error)


def bad_caches(df11):
    ok = dict(pages=A, n_pages=4, page_size=16, n_heads=2, head_dim=128, k_scale=1.0, v_scale=1.0)
    E, U = df11.DF11_EINVAL, df11.DF11_EUNSUPPORTED
    nan, inf = float("nan"), float("inf")
    yield from ((st, df11.Kv4Cache(**{**ok, **b})) for st, b in [
        (E, dict(pages=0)), (E, dict(pages=A + 8)), (E, dict(n_pages=0)), (E, dict(n_pages=1 << 31)),
        (U, dict(page_size=8)), (U, dict(page_size=0)), (U, dict(page_size=17)), (E, dict(n_heads=0)),
        (E, dict(n_heads=1025)), (U, dict(head_dim=80)), (U, dict(head_dim=256)), (E, dict(k_scale=0.0)),
        (E, dict(k_scale=-1.0)), (E, dict(k_scale=nan)), (E, dict(k_scale=inf)), (E, dict(v_scale=0.0)),
        (E, dict(v_scale=nan)), (E, dict(v_scale=inf))])


def cache(df11, **kw):
    return df11.Kv4Cache(**{**dict(pages=A, n_pages=4, page_size=16, n_heads=2, head_dim=128, k_scale=1.0, v_scale=1.0),
                            **kw})


def test_append_and_gather_refusals(df11):
    for status, c in bad_caches(df11):
        refused(df11, status, df11.df11_kv4_append, c, A, 256, A, 256, A, 3)
        refused(df11, status, df11.df11_kv4_gather, c, A, 3, A, A)
    c, E = cache(df11), df11.DF11_EINVAL
    good = dict(k_ptr=A, k_token_stride=256, v_ptr=A, v_token_stride=264, slots_ptr=A, n_tokens=3)
    for b in [dict(k_ptr=0), dict(k_ptr=A + 8), dict(k_token_stride=255), dict(k_token_stride=248),
              dict(k_token_stride=260), dict(v_ptr=0), dict(v_ptr=A + 2), dict(v_token_stride=128),
              dict(v_token_stride=258), dict(slots_ptr=0), dict(slots_ptr=A + 4), dict(n_tokens=-1)]:
        refused(df11, E, df11.df11_kv4_append, c, **{**good, **b})
    df11.df11_kv4_append(c, **{**good, "n_tokens": 0})
    for b in [dict(slots_ptr=0), dict(slots_ptr=A + 4), dict(n_tokens=-1), dict(k_out_ptr=A + 8), dict(v_out_ptr=A + 4)]:
        refused(df11, E, df11.df11_kv4_gather, c, **{**dict(slots_ptr=A, n_tokens=3, k_out_ptr=A, v_out_ptr=A), **b})
    df11.df11_kv4_gather(c, A, 0, A, A)
    df11.df11_kv4_gather(c, A, 3, 0, 0)
    # a dtype of the weights is not one of the activations
    st = df11._lib.df11_kv4_append(c, A, 256, A, 256, A, 3, df11.DF11_FP8_E4M3, None, None)
    assert st == E
    assert df11._lib.df11_kv4_gather(c, A, 3, A, A, 7, None, None) == E


def test_attention_refusals(df11):
    good = dict(q_ptr=A, q_token_stride=512, o_ptr=A, o_token_stride=512, n_q_heads=4, q_start_ptr=A, kv_lens_ptr=A,
                block_table_ptr=A, n_reqs=2, max_pages=4, n_tokens=5, max_q_len=3, scale=0.1, workspace_ptr=A,
                workspace_bytes=1 << 40)
    for status, c in bad_caches(df11):
        refused(df11, status, df11.df11_kv4_attention, c, **good)
    c, E = cache(df11), df11.DF11_EINVAL
    for b in [dict(q_ptr=0), dict(q_ptr=A + 8), dict(q_token_stride=511), dict(q_token_stride=516), dict(o_ptr=0),
              dict(o_ptr=A + 4), dict(o_token_stride=256), dict(n_q_heads=0), dict(n_q_heads=3), dict(n_q_heads=-2),
              dict(n_q_heads=1 << 17), dict(q_start_ptr=0), dict(q_start_ptr=A + 2), dict(kv_lens_ptr=0),
              dict(block_table_ptr=0), dict(block_table_ptr=A + 1), dict(n_reqs=-1), dict(max_pages=-1),
              dict(n_tokens=-1), dict(max_q_len=-1), dict(scale=float("nan")), dict(scale=float("inf")),
              dict(workspace_ptr=0), dict(workspace_ptr=A + 8), dict(causal=2), dict(window=-1),
              dict(causal=False, window=5), dict(lse_ptr=A + 2)]:
        refused(df11, E, df11.df11_kv4_attention, c, **{**good, **b})
    for b in [dict(n_reqs=0), dict(n_tokens=0), dict(max_q_len=0)]:  # nothing to do
        df11.df11_kv4_attention(c, **{**good, **b})
    for b in [(0, 2, 5, 3), (3, 2, 5, 3), (4, -1, 5, 3), (4, 2, -1, 3), (4, 2, 5, -1)]:
        assert df11.df11_kv4_attention_workspace_bytes(c, *b) == 0
    # past 31 bits: 2 ** 30 tokens of 4 heads; 2 ** 16 requests x 2 heads x 8 tiles of rows x (2 ** 13 * 16 / 64 + 16)
    # chunks; 2 ** 28 x 2 x 1 x (1 + 16)
    for b in [dict(n_tokens=1 << 30), dict(n_reqs=1 << 16, max_q_len=32, max_pages=1 << 13),
              dict(n_reqs=1 << 28, max_pages=0)]:
        refused(df11, df11.DF11_EUNSUPPORTED, df11.df11_kv4_attention, c, **{**good, **b})


def test_attention_refuses_scales_past_fp32(df11):
    """The scores' factor is the product of two scales, each finite: where that is not, 0 times it would be NaN."""
    good = dict(q_ptr=A, q_token_stride=512, o_ptr=A, o_token_stride=512, n_q_heads=4, q_start_ptr=A, kv_lens_ptr=A,
                block_table_ptr=A, n_reqs=2, max_pages=4, n_tokens=5, max_q_len=3, workspace_ptr=A, workspace_bytes=1 << 40)
    for k, scale in ((1e30, 1e10), (1e30, -1e10), (1.0, 3e38), (3e38, 1.0), (1e38, 3.0)):
        refused(df11, df11.DF11_EINVAL, df11.df11_kv4_attention, cache(df11, k_scale=k), scale=scale, **good)
    for k, scale in ((1e30, 1e7), (2e38, -1.0), (1e38, 1e-38), (1e-30, 1e-30)):  # nothing to do, but no error either
        df11.df11_kv4_attention(cache(df11, k_scale=k), scale=scale, **{**good, "n_tokens": 0})


# ------------------------------------------------------------------ the reference itself

def test_reference_quantizer_by_hand():
    # max 6: scale 1, the levels themselves; 2.5 lies between 2 and 3: to the even code 2; 5 to 4; 0.25 to 0; -0.75 to -1
    x = np.zeros(16, np.float32)
    x[:8] = [6, 2.5, 5, 0.25, -0.75, 1.25, 1.75, -3.5]
    codes, sb, val = ref.quantize(x, 1.0)
    assert sb.tolist() == [0x38]  # 1.0 in E4M3
    assert val[:8].tolist() == [6, 2, 4, 0, -1, 1, 2, -4]
    assert codes[:8].tolist() == [7, 4, 6, 0, 10, 2, 4, 14]
    # 448 * 6 saturates; an infinity does as well and leaves the others at its scale; a NaN is +6
    x[:4] = [np.inf, 448, -1e30, np.nan]
    _, sb, val = ref.quantize(x, 1.0)
    assert sb.tolist() == [126] and val[:4].tolist() == [2688, 448, -2688, 2688]
    assert (ref.quantize(np.full(16, 2.0 ** -14, np.float32), 1.0)[2] == 0).all()  # scale below E4M3's range
    assert (ref.quantize(np.full(16, 2.0 ** -14, np.float32), 2.0 ** -10)[2] != 0).all()


def test_reference_e4m3_grid():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.E4M3)


def test_reference_cache_layout_by_hand():
    c = ref.Cache(2, 16, 1, 64, 1.0, 1.0)
    k = np.zeros((1, 1, 64), np.float32)
    k[0, 0, 17] = 6.0  # block 1, element 1: byte 8, high nibble
    v = np.zeros((1, 1, 64), np.float32)
    v[0, 0, 35] = -1.5 * 2  # block 2, element 3: byte 1 of the piece, high nibble; scale 0.5: level -6
    c.write([16 + 6], k, v)
    b = c.bytes[1, 0]
    assert not c.bytes[0].any()
    assert b[6 * 32 + 8] == 0x70 and b[16 * 32 + 6 * 4 + 1] == 0x38
    vc = 16 * 32 + 16 * 4
    assert b[vc + ((1 * 4 + 2) * 4 + 2) * 8 + 1] == 0xF0
    assert b[vc + 16 * 32 + 2 * 16 + 6] == 0x30
    assert np.count_nonzero(b) == 4


def test_reference_attention_closed_forms():
    q = torch.zeros(3, 2, 64, dtype=torch.float64)
    v = torch.randn(5, 1, 64, dtype=torch.float64)
    o, lse, *_ = ref.attention(q, torch.randn(5, 1, 64, dtype=torch.float64), v, True, 0, 1.0)
    for i in range(3):  # equal scores: the mean of the keys seen
        assert torch.allclose(o[i, 1], v[:3 + i, 0].mean(0)) and abs(lse[i, 0] - np.log(3 + i)) < 1e-12
    o, lse, *_ = ref.attention(q, torch.randn(2, 1, 64, dtype=torch.float64), v[:2], True, 0, 1.0)
    assert (o[0] == 0).all() and torch.isinf(lse[0]).all() and torch.equal(o[1, 0], v[0, 0])
    o, lse, *_ = ref.attention(q, torch.randn(5, 1, 64, dtype=torch.float64), v, True, 1, 1.0)
    assert torch.equal(o[2, 0], v[4, 0]) and torch.equal(o[0, 1], v[2, 0])


def test_reference_extend_by_hand():
    # request 0 holds 15 of 16 tokens of page 9 and adds 2: page 4 (the top of the stack) starts with the second
    t, kv, qs, slots, pos, nf = ref.extend([15, 0], [2, 1], [7, 2, 4], 3, [[9, -1], [-1, -1]], 16, 5)
    assert t == [[9, 4], [2, -1]] and kv == [17, 1] and qs == [0, 2, 3] and nf == 1
    assert slots == [9 * 16 + 15, 4 * 16, 2 * 16, -1, -1] and pos == [15, 16, 0, 0, 0]
