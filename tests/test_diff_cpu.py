"""Host-side checks of the rotated append and of differential attention, no GPU needed: every
refusal before a launch, the split counts, and the tests' 64-bit forms against closed forms."""
import numpy as np
import pytest
import torch

import diff_ref as ref
import gqa_attention_gb300 as g

FAKE = 0x10000  # never dereferenced: every case below fails a host check first
BAD, UNSUP = g.GQA_ERR_INVALID_ARG, g.GQA_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gqa_attention_gb300 import build

    build.build()
    g.load()


def _append(paged, fp8, **kw):
    a = dict(q=FAKE, k_new=FAKE, v_new=FAKE, q_stride=1024, kv_stride=1024, freqs=FAKE, rot=128,
             inter=0, n_new=None, pos=None, table=FAKE, lens=FAKE, B=2, T=4, S_max=64, pages=8,
             page_size=16, max_blocks=4, H_q=8, H_kv=2, d=128, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE,
             q_out=FAKE)
    a.update(kw)
    head = (a["q"], a["k_new"], a["v_new"], a["q_stride"], a["kv_stride"], a["freqs"], a["rot"],
            a["inter"], a["n_new"], a["pos"])
    shape = (a["pages"], a["page_size"], a["max_blocks"]) if paged else (a["S_max"],)
    tail = (a["H_q"], a["H_kv"], a["d"], a["k"], a["v"])
    if fp8:
        tail += (a["ks"], a["vs"])
    call = {(0, 0): g.gqa_kv_append, (1, 0): g.gqa_kv_append_paged, (0, 1): g.gqa_kv_append_fp8,
            (1, 1): g.gqa_kv_append_paged_fp8}[int(paged), int(fp8)]
    return call(*head, *((a["table"],) if paged else ()), a["lens"], a["B"], a["T"], *shape, *tail,
                a["q_out"], stream=0)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_append_refusals(paged, fp8):
    for kw, status in [
        (dict(k_new=None), BAD), (dict(v_new=None), BAD), (dict(lens=None), BAD),
        (dict(k=None), BAD), (dict(v=None), BAD), (dict(q=None), BAD), (dict(q_out=None), BAD),
        (dict(B=0), BAD), (dict(T=0), BAD), (dict(H_kv=0), BAD), (dict(H_q=0), BAD),
        (dict(H_kv=65536), BAD), (dict(H_q=65536, q_stride=1 << 30), BAD),
        (dict(d=96), UNSUP), (dict(d=8), UNSUP), (dict(d=256), UNSUP),
        (dict(rot=-16), BAD), (dict(rot=144), BAD), (dict(rot=8), UNSUP), (dict(rot=100), UNSUP),
        (dict(freqs=None), BAD), (dict(freqs=FAKE + 2), BAD), (dict(inter=2), BAD),
        (dict(kv_stride=255), BAD), (dict(kv_stride=248), BAD), (dict(kv_stride=260), BAD),
        (dict(q_stride=1016), BAD), (dict(q_stride=1028), BAD), (dict(kv_stride=-1024), BAD),
        (dict(q=FAKE + 8), BAD), (dict(q_out=FAKE + 8), BAD), (dict(k_new=FAKE + 8), BAD),
        (dict(v_new=FAKE + 8), BAD), (dict(k=FAKE + 8), BAD), (dict(v=FAKE + 8), BAD),
        (dict(lens=FAKE + 2), BAD), (dict(n_new=FAKE + 2), BAD), (dict(pos=FAKE + 1), BAD),
        (dict(B=1 << 20, T=1 << 12, S_max=1), BAD),
    ]:
        assert _append(paged, fp8, **kw) == status, kw
    if fp8:
        for kw in (dict(ks=None), dict(vs=None), dict(ks=FAKE + 2), dict(vs=FAKE + 2)):
            assert _append(paged, fp8, **kw) == BAD, kw
    if not paged:
        for kw in (dict(S_max=0), dict(S_max=-4), dict(S_max=0x7fff0001, B=1), dict(S_max=0x40000000)):
            assert _append(False, fp8, **kw) == BAD, kw


PAGED = [(dict(table=None), BAD), (dict(table=FAKE + 2), BAD), (dict(pages=0), BAD),
         (dict(max_blocks=0), BAD), (dict(page_size=0), BAD), (dict(page_size=8), UNSUP),
         (dict(page_size=48), UNSUP), (dict(page_size=1 << 20, max_blocks=1 << 11), BAD),
         (dict(page_size=1 << 20, pages=1 << 11), BAD)]


def _decode(paged, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, lam=FAKE, sb=0, st=0, sh=0, B=1, T_q=1,
             S_max=64, pages=4, page_size=16, max_blocks=4, H=8, H_kv=2, d=128, split=0, scale=0.1,
             w=None, eps=-1.0, mul=1.0, n_split=1, ws=None, out=FAKE, lse=FAKE)
    a.update(kw)
    lam = (a["lam"], a["sb"], a["st"], a["sh"], a["B"], a["T_q"])
    tail = (a["H"], a["H_kv"], a["d"], a["split"], a["scale"], a["w"], a["eps"], a["mul"],
            a["n_split"], a["ws"], a["out"], a["lse"])
    if paged:
        return g.gqa_attn_decode_paged_diff(a["q"], a["k"], a["v"], a["table"], a["lens"], *lam,
                                            a["pages"], a["page_size"], a["max_blocks"], *tail,
                                            stream=0)
    return g.gqa_attn_decode_diff(a["q"], a["k"], a["v"], a["lens"], *lam, a["S_max"], *tail,
                                  stream=0)


def _prefill(_, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, lens=FAKE, lam=FAKE, sb=0, st=0, sh=0, B=1, T_q=16, S_max=64,
             H=8, H_kv=2, d=128, split=0, scale=0.1, window=-1, w=None, eps=-1.0, mul=1.0, n_part=1,
             ws=None, out=FAKE, lse=FAKE)
    a.update(kw)
    return g.gqa_attn_prefill_diff(a["q"], a["k"], a["v"], a["lens"], a["lam"], a["sb"], a["st"],
                                   a["sh"], a["B"], a["T_q"], a["S_max"], a["H"], a["H_kv"], a["d"],
                                   a["split"], a["scale"], a["window"], a["w"], a["eps"], a["mul"],
                                   a["n_part"], a["ws"], a["out"], a["lse"], stream=0)


COMMON = [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(lam=None), BAD),
    (dict(out=None), BAD), (dict(lse=None), BAD), (dict(lam=FAKE + 2), BAD), (dict(sb=-1), BAD),
    (dict(st=-1), BAD), (dict(sh=-1), BAD), (dict(H=0), BAD), (dict(H=7), BAD), (dict(H_kv=0), BAD),
    (dict(H=32768, H_kv=32768), BAD), (dict(d=96), UNSUP), (dict(d=16), UNSUP), (dict(split=2), BAD),
    (dict(split=-1), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(mul=float("nan")), BAD), (dict(mul=float("inf")), BAD), (dict(w=FAKE), BAD),
    (dict(w=FAKE + 2, eps=1e-5), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(B=0), BAD), (dict(B=65536), BAD), (dict(T_q=0), BAD),
    (dict(T_q=65), BAD), (dict(q=FAKE + 8), BAD), (dict(k=FAKE + 8), BAD), (dict(out=FAKE + 8), BAD),
    (dict(lens=FAKE + 2), BAD), (dict(lse=FAKE + 2), BAD),
]


@pytest.mark.parametrize("call,paged", [(_decode, False), (_decode, True), (_prefill, False)])
def test_attention_refusals(call, paged):
    for kw, status in COMMON + (PAGED if paged else []):
        assert call(paged, **kw) == status, kw


@pytest.mark.parametrize("paged", [False, True])
def test_decode_refusals(paged):
    for kw, status in [
        (dict(lens=None), BAD), (dict(n_split=0), BAD), (dict(n_split=3), BAD),
        (dict(n_split=3, ws=FAKE + 16), BAD), (dict(n_split=65536, ws=FAKE), BAD),
        (dict(H=18), UNSUP), (dict(T_q=9), UNSUP), (dict(lse=FAKE + 4), BAD),
    ]:
        assert _decode(paged, **kw) == status, kw
    if not paged:
        assert _decode(False, T_q=5, S_max=4) == BAD
        assert _decode(False, S_max=0) == BAD
        assert _decode(False, S_max=0x40000000, B=2) == BAD


def test_prefill_refusals():
    for kw in (dict(n_part=0), dict(n_part=9), dict(n_part=2), dict(n_part=2, ws=FAKE + 16),
               dict(T_q=32, S_max=16), dict(S_max=0), dict(B=1 << 10, T_q=1 << 20, S_max=1 << 20)):
        assert _prefill(None, **kw) == BAD, kw


def test_default_splits():
    for B, T, H, Hk, S in [(1, 1, 32, 8, 32768), (8, 1, 32, 8, 65536), (1, 1, 4, 2, 1024),
                           (4, 4, 32, 8, 16384), (64, 1, 8, 4, 4001)]:
        n = g.gqa_attn_decode_diff_default_splits(B, T, H, Hk, S, 128)
        assert -(-S // 8192) <= n <= max(1, -(-S // 128))
    assert g.gqa_attn_decode_diff_default_splits(1, 1, 9, 8, 4096, 128) == 1
    assert g.gqa_attn_decode_diff_default_splits(0, 1, 8, 8, 4096, 128) == 1
    assert g.gqa_attn_decode_diff_default_splits(1, 0, 8, 8, 4096, 128) == 1


def test_default_parts():
    # (no GPU here: the SM count falls back to a default)
    assert g.gqa_attn_prefill_diff_default_parts(3, 333, 2903, 8, 2, 1000) == 1
    assert g.gqa_attn_prefill_diff_default_parts(1, 128, 32768, 8, 2, -1) == 8
    assert g.gqa_attn_prefill_diff_default_parts(1, 4096, 4096, 8, 2, -1) == 1
    for bad in ((0, 128, 32768, 8, 2, -1), (1, 0, 32768, 8, 2, -1), (1, 128, 0, 8, 2, -1),
                (1, 128, 32768, 7, 2, -1), (1, 128, 32768, 8, 0, -1), (1, 128, 32768, 1 << 30, 2, -1)):
        assert g.gqa_attn_prefill_diff_default_parts(*bad) == 1


def test_defaults_of_the_largest_arguments():
    M = 2 ** 31 - 1
    for T in (1, 8, M):
        for S in (1, 1 << 20, M):
            for d in (32, 64, 128):
                for B, H, Hk in ((M, M, M), (1, M, M), (M, 1, 1), (1, M, 1), (1 << 30, 1 << 30, 1 << 30),
                                 (1 << 20, 1 << 22, 1 << 22), (1, 1, 1)):
                    n = g.gqa_attn_decode_diff_default_splits(B, T, H, Hk, S, d)
                    assert 1 <= n <= max(2 * 152, -(-S // 128))
                    for w in (-M - 1, -1, 0, M):
                        assert 1 <= g.gqa_attn_prefill_diff_default_parts(B, T, S, H, Hk, w) <= 8
    assert g.gqa_attn_prefill_diff_default_parts(M, M, M, 32767, 1, -1) == 1


def test_helpers_refuse_cpu_tensors():
    k = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    lens, lam = torch.ones(1, dtype=torch.int32), torch.ones(1)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(g.GQAError):
        g.kv_append(k[:, :1], k[:, :1], k, k, lens)
    with pytest.raises(g.GQAError):
        g.decode_diff(q, k, k, lens, lam)
    with pytest.raises(g.GQAError):
        g.prefill_diff(q[:, None], k, k, lam)
    with pytest.raises(g.GQAError):
        g.decode_diff(None, k, k, lens, lam)


def test_default_splits_of_long_sequences_are_taken_by_the_call():
    # (d = 16, of no kernel, is looked at after the splits)
    for S in (1 << 29, 536862720, 536862721, 1 << 30, 0x7fff0000):
        for T, H, d in ((1, 1, 64), (8, 4, 64), (8, 4, 128)):
            for B in (1, 3, 100):
                n = g.gqa_attn_decode_diff_default_splits(B, T, H, 1, S, d)
                assert 1 <= n <= 65535
                tile = 128 if d == 128 and T * 2 * H > 16 else 64
                chunk = -(-(-(-S // n)) // tile) * tile
                assert n * chunk < 2 ** 31
                if B * S <= 0x7fff0000:
                    assert _decode(False, B=B, T_q=T, H=H, H_kv=1, S_max=S, d=16, n_split=n,
                                   ws=FAKE) == UNSUP


@pytest.mark.parametrize("T,H_of,d", [(1, 4, 128), (4, 4, 128), (8, 4, 64), (1, 1, 32), (2, 8, 128)])
def test_default_splits_share_out_long_sequences(T, H_of, d):
    # A split has at most 8192 tokens, or one sequence's splits fill the SMs, or several sequences'
    # (those that are cut by their lengths, and the many that are not: eight CTAs to an SM).  On
    # mma.sync 32 rows are a CTA.
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 148
    rows = 2 * T * H_of
    groups = 1 if d == 128 or rows <= 16 else -(-rows // 32)
    for Hk in (1, 2, 3, 4, 5, 8):
        for B in range(1, 129):
            for S in (8192, 8193, 16384, 65536, 1 << 20):
                n = g.gqa_attn_decode_diff_default_splits(B, T, H_of * Hk, Hk, S, d)
                fills = (2 * n * Hk > sms if B == 1 else (n + 1) * B * Hk > 8 * sms
                         or (B <= 96 and n * B * Hk * groups >= sms))
                assert n * 8192 >= S or fills, (Hk, B, S, n)


# -------------------------------------------------------- the 64-bit forms --
def test_turning_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    freqs = np.float32(10000.0 ** (-np.arange(8) / 8))
    q, k = rng.standard_normal((2, 1, 1, 20))
    dots = []
    for a, b in ((3, 1), (1002, 1000), (70002, 70000)):
        for inter in (False, True):
            x, _ = ref.turn(q, [a], freqs, inter)
            y, _ = ref.turn(k, [b], freqs, inter)
            assert abs((x ** 2).sum() - (q ** 2).sum()) < 1e-9
            assert np.array_equal(x[..., 16:], q[..., 16:])
            dots.append(((x * y).sum(), inter))
    for inter in (False, True):
        d = [v for v, i in dots if i == inter]
        assert max(d) - min(d) < 1e-9
    # a quarter turn, by hand: frequency pi / 2 at position 1 takes (1, 0) to (0, 1)
    x, _ = ref.turn(np.array([[[1.0, 0.0]]]), [1], [np.pi / 2], True)
    assert np.allclose(x, [[[0.0, 1.0]]])
    x, _ = ref.turn(np.array([[[1.0, 0.0]]]), [-1], [np.pi / 2], False)
    assert np.allclose(x, [[[0.0, -1.0]]])


def test_attention_closed_forms():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((6, 1, 4))
    lam = np.full((6, 1), 0.25)
    # zero queries: both maps are the mean of what is seen
    o, lse, _, _ = ref.attention(np.zeros((6, 2, 4)), rng.standard_normal((6, 1, 4)), v, lam, 0.5,
                                 False)
    mean = np.cumsum(v[:, 0], 0) / np.arange(1, 7)[:, None]
    assert np.allclose(o[:, 0], 0.75 * mean) and np.allclose(lse[:, 0], np.log(np.arange(1, 7)))
    # a window of one sees the token itself; the norm leaves a root mean square of one
    o, _, _, _ = ref.attention(np.zeros((6, 2, 4)), np.zeros((6, 1, 4)), v, lam, 0.5, False, window=0,
                               norm_eps=0.0, out_scale=2.0)
    assert np.allclose((o ** 2).mean(-1), 4.0)
    assert np.allclose(o[:, 0] / v[:, 0], 2.0 / np.sqrt((v[:, 0] ** 2).mean(-1, keepdims=True)))
    # split keys are shared keys of rows padded with zeros
    q, k = rng.standard_normal((3, 2, 8)), rng.standard_normal((6, 1, 8))
    v = rng.standard_normal((6, 1, 8))
    wide = np.zeros((3, 4, 8))
    wide[:, 0::2, :4], wide[:, 1::2, 4:] = q[..., :4], q[..., 4:]
    lam = rng.random((3, 2))
    a = ref.attention(q, k, v, lam, 0.3, True)
    b = ref.attention(wide, k, v, lam, 0.3, False)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])
