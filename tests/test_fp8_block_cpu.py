"""Host-side checks of the block-scaled E4M3 cache's entry points, no GPU needed,
and the 64-bit quantiser of the tests against torch's E4M3 rounding."""
import numpy as np
import pytest
import torch

import fp8_block_ref as ref
import gqa_attention_gb300 as g

FAKE = 0x10000  # never dereferenced: every case below fails a host check first
BAD, UNSUP = g.GQA_ERR_INVALID_ARG, g.GQA_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gqa_attention_gb300 import build

    build.build()
    g.load()


def _append(paged, **kw):
    a = dict(k_new=FAKE, v_new=FAKE, new_stride=256, n_new=None, seq_lens=FAKE, B=1, T=4, S_max=64,
             H_kv=2, d=128, block=16, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, table=FAKE, pages=4,
             page_size=16, max_blocks=4)
    a.update(kw)
    if paged:
        return g.gqa_kv_append_paged_fp8_block(
            a["k_new"], a["v_new"], a["new_stride"], a["n_new"], a["table"], a["seq_lens"], a["B"],
            a["T"], a["pages"], a["page_size"], a["max_blocks"], a["H_kv"], a["d"], a["block"],
            a["k"], a["v"], a["ks"], a["vs"], stream=0)
    return g.gqa_kv_append_fp8_block(a["k_new"], a["v_new"], a["new_stride"], a["n_new"],
                                     a["seq_lens"], a["B"], a["T"], a["S_max"], a["H_kv"], a["d"],
                                     a["block"], a["k"], a["v"], a["ks"], a["vs"], stream=0)


def _read(paged, **kw):
    a = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, table=FAKE, seq_lens=FAKE, B=1, S_max=64, pages=4,
             page_size=16, max_blocks=4, H_kv=2, d=128, block=16, start=0, S_out=64, ko=FAKE,
             vo=FAKE)
    a.update(kw)
    if paged:
        return g.gqa_kv_read_paged_fp8_block(
            a["k"], a["v"], a["ks"], a["vs"], a["table"], a["seq_lens"], a["B"], a["pages"],
            a["page_size"], a["max_blocks"], a["H_kv"], a["d"], a["block"], a["start"], a["S_out"],
            a["ko"], a["vo"], stream=0)
    return g.gqa_kv_read_fp8_block(a["k"], a["v"], a["ks"], a["vs"], a["seq_lens"], a["B"],
                                   a["S_max"], a["H_kv"], a["d"], a["block"], a["start"],
                                   a["S_out"], a["ko"], a["vo"], stream=0)


def _decode(paged, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, table=FAKE, seq_lens=FAKE, B=1, T_q=1,
             S_max=64, pages=4, page_size=16, max_blocks=4, H_q=8, H_kv=2, d=128, block=16,
             scale=0.1, n_split=1, ws=None, out=FAKE, lse=FAKE)
    a.update(kw)
    if paged:
        return g.gqa_attn_decode_paged_fp8_block(
            a["q"], a["k"], a["v"], a["ks"], a["vs"], a["table"], a["seq_lens"], a["B"], a["T_q"],
            a["pages"], a["page_size"], a["max_blocks"], a["H_q"], a["H_kv"], a["d"], a["block"],
            a["scale"], a["n_split"], a["ws"], a["out"], a["lse"], stream=0)
    return g.gqa_attn_decode_fp8_block(a["q"], a["k"], a["v"], a["ks"], a["vs"], a["seq_lens"],
                                       a["B"], a["T_q"], a["S_max"], a["H_q"], a["H_kv"], a["d"],
                                       a["block"], a["scale"], a["n_split"], a["ws"], a["out"],
                                       a["lse"], stream=0)


COMMON = [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(ks=None), BAD), (dict(vs=None), BAD),
    (dict(seq_lens=None), BAD), (dict(B=0), BAD), (dict(B=65536), BAD), (dict(H_kv=0), BAD),
    (dict(k=FAKE + 8), BAD), (dict(ks=FAKE + 2), BAD), (dict(seq_lens=FAKE + 1), BAD),
    (dict(d=96), UNSUP), (dict(d=256), UNSUP), (dict(block=8), UNSUP), (dict(block=48), UNSUP),
    (dict(block=256), UNSUP), (dict(block=0), UNSUP),
]
CONTIGUOUS = [(dict(S_max=0), BAD), (dict(S_max=2 ** 30, B=2), BAD)]
PAGED = [
    (dict(table=None), BAD), (dict(table=FAKE + 2), BAD), (dict(pages=0), BAD),
    (dict(max_blocks=0), BAD), (dict(page_size=0), BAD), (dict(page_size=8), UNSUP),
    (dict(page_size=48), UNSUP), (dict(block=32), BAD),  # a block longer than its page
    (dict(page_size=1 << 20, max_blocks=1 << 11), BAD), (dict(page_size=1 << 20, pages=1 << 11), BAD),
]


@pytest.mark.parametrize("call", [_append, _read, _decode])
@pytest.mark.parametrize("paged", [False, True])
def test_shared_refusals(call, paged):
    for kw, status in COMMON + (PAGED if paged else CONTIGUOUS):
        assert call(paged, **kw) == status, (kw, paged)


@pytest.mark.parametrize("paged", [False, True])
def test_append_refusals(paged):
    for kw in (dict(k_new=None), dict(v_new=None), dict(T=0), dict(new_stride=255),
               dict(new_stride=248), dict(new_stride=260), dict(k_new=FAKE + 8),
               dict(n_new=FAKE + 2)):
        assert _append(paged, **kw) == BAD, kw


@pytest.mark.parametrize("paged", [False, True])
def test_read_refusals(paged):
    for kw in (dict(ko=None), dict(vo=None), dict(start=-1), dict(S_out=0), dict(ko=FAKE + 8),
               dict(start=2 ** 31 - 2, S_out=4)):
        assert _read(paged, **kw) == BAD, kw


@pytest.mark.parametrize("paged", [False, True])
def test_decode_refusals(paged):
    for kw, status in [
        (dict(q=None), BAD), (dict(out=None), BAD), (dict(lse=None), BAD), (dict(n_split=0), BAD),
        (dict(n_split=3), BAD), (dict(n_split=3, ws=FAKE + 16), BAD), (dict(H_q=9), BAD),
        (dict(T_q=0), BAD), (dict(T_q=65), BAD), (dict(H_q=34), UNSUP), (dict(T_q=17), UNSUP),
        (dict(scale=float("nan")), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
        (dict(q=FAKE + 8), BAD), (dict(out=FAKE + 8), BAD),
    ]:
        assert _decode(paged, **kw) == status, kw
    if not paged:
        assert _decode(False, T_q=5, S_max=4) == BAD


def test_default_splits_cover_the_cache():
    for B, T_q, H, S in [(1, 1, 8, 32768), (1, 8, 8, 32768), (1, 1, 2, 1024), (64, 1, 4, 4001),
                         (8, 1, 8, 131072)]:
        n = g.gqa_attn_decode_fp8_block_default_splits(B, T_q, 8 * H, H, S)
        assert -(-S // 8192) <= n <= max(1, -(-S // 256))
    assert g.gqa_attn_decode_fp8_block_default_splits(1, 1, 9, 8, 4096) == 1
    assert g.gqa_attn_decode_fp8_block_default_splits(0, 1, 8, 8, 4096) == 1


def test_helpers_refuse_cpu_tensors_and_wrong_layouts():
    k8, v8, ks, vs = g.kv_cache_fp8_block(2, 40, 3, 64, 16, device="cpu")
    assert ks.shape == (2, 3, 3) and k8.dtype == torch.uint8
    lens = torch.ones(2, dtype=torch.int32)
    x = torch.zeros(2, 1, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(g.GQAError):  # not on a CUDA device
        g.kv_append_fp8_block(x, x, k8, v8, ks, vs, lens, 16)
    with pytest.raises(g.GQAError):  # scales of another block size
        g.kv_read_fp8_block(k8, v8, ks, vs, lens, 32)
    with pytest.raises(g.GQAError):  # codes that are not dense
        g.decode_fp8_block(x[:, 0], k8[:, ::2], v8[:, ::2], ks, vs, lens, 16)


def test_reference_rounding_against_torch():
    gen = np.random.default_rng(0)
    x = np.concatenate([gen.standard_normal(4000) * 2.0 ** gen.integers(-12, 10, 4000), ref._POS,
                        (ref._POS[1:] + ref._POS[:-1]) / 2, [0.0, 449.0, 1e9]])
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.round_e4m3(x.astype(np.float64)), want)
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, ref.E4M3, equal_nan=True)


@pytest.mark.parametrize("amax", [0.0, 1e-38, 2.0 ** -100 * 448, 1.75, 1.7578125, 448.0, 449.0, 3e38])
def test_reference_scale_is_the_smallest(amax):
    s = ref.block_scale(amax)
    assert amax / s <= 448 and (s == 2.0 ** -100 or amax / (s / 2) > 448)
