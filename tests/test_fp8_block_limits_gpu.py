"""The block-scaled E4M3 cache at the limits of what its calls accept: scales that are NaN,
negative or near the type's largest, heads that share a tile in batches of long capacity, and
weights far below the largest."""
import math

import numpy as np
import pytest
import torch

import fp8_block_ref as ref
import gqa_attention_gb300 as g
from test_fp8_block_gpu import Cache, check_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_attention_gb300 import build

    build.build()
    g.load()
    yield
    assert g.gqa_last_device_error() == g.GQA_OK


# ------------------------------------------------------- scales behind the mask --
@pytest.mark.parametrize("name,bad", [("v", math.nan), ("v", -1.0), ("v", -math.inf), ("k", math.nan)])
@pytest.mark.parametrize("d,H,G,T_q,n_split", [(128, 2, 4, 2, 1), (128, 2, 8, 8, 3), (64, 1, 1, 64, 1),
                                               (32, 4, 2, 5, 200), (128, 1, 16, 4, 2)])
@pytest.mark.parametrize("ctx,page", [(17, 0), (129, 16), (163, 0), (401, 32)])
def test_bad_scales_reach_the_rows_that_see_their_tokens(name, bad, d, H, G, T_q, n_split, ctx, page):
    """A NaN scale, or a negative one of the values, on a block of one head that begins behind
    the first query's last token: NaN for the queries that see the block, and no others."""
    T_q = min(T_q, ctx)
    c = Cache(2, ctx, H, d, 16, page, seed=d + T_q + ctx)
    k, v = c.rows(ctx)
    c.append(k, v, [ctx, ctx])
    q = torch.randn(2, T_q, H * G, d, generator=c.gen).to(torch.bfloat16)
    t = (ctx - 1) // 16 * 16  # of sequence 1, head H - 1
    unit, at = (int(c.table[1, t // page]), t % page // 16) if page else (1, t // 16)
    (c.vs if name == "v" else c.ks)[unit, at, H - 1] = bad
    c.scale[name][1, t // 16, H - 1] = math.nan
    hit = torch.zeros(2, T_q, H * G, dtype=torch.bool)
    hit[1, max(0, t - (ctx - T_q)):, (H - 1) * G:] = True
    out, lse = g.decode_fp8_block(q.to(DEV), *c.args(), c.lens(), 16, n_split=n_split,
                                  block_table=c.table)
    assert torch.equal(lse.isnan().cpu(), hit)
    assert torch.equal(out.isnan().cpu(), hit[..., None].expand(-1, -1, -1, d))
    o, l, to, tl = c.expect(q, 1 / math.sqrt(d))
    ok = ~hit.numpy()
    assert (np.abs(out.double().cpu().numpy() - o) <= to)[ok].all()
    assert (np.abs(lse.double().cpu().numpy() - l) <= tl)[ok].all()


# ------------------------------------------------------------ the largest scales --
@pytest.mark.parametrize("exps", [(127.0, 126.5, 120.0, 127.9), (127.5,) * 4])
@pytest.mark.parametrize("T_q,G", [(1, 8), (2, 16)])
def test_value_scales_up_to_the_largest(exps, T_q, G):
    """Value scales up to 2^127.9 whose products with the codes, at most 1, are within bf16."""
    c = Cache(1, 256, 1, 64, 64, 0, seed=T_q)
    k, v = c.rows(256)
    c.append(k, v, [256])
    codes = torch.randint(0, 0x39, c.v8.shape, generator=c.gen, dtype=torch.uint8)
    codes |= torch.randint(0, 2, c.v8.shape, generator=c.gen, dtype=torch.uint8) << 7
    c.v8.copy_(codes)
    c.val["v"] = ref.E4M3[codes.numpy()]
    c.vs.copy_(torch.tensor([2.0 ** e for e in exps]).view(1, 4, 1))
    c.scale["v"] = c.vs.double().cpu().numpy()
    q = torch.randn(1, T_q, G, 64, generator=c.gen).to(torch.bfloat16)
    o, l, to, tl = c.expect(q, 1 / 8)
    # scores are held together with logarithms of up to 135, whose half step in fp32 is 2^-17:
    # a key's own, the reference's and the sum's
    more = 3 * 2.0 ** -17
    mag = [ref.attention(q[0].double().numpy(), c.val["k"][0], c.scale["k"][0], np.abs(c.val["v"][0]),
                         c.scale["v"][0], 256, 64, 1 / 8)[0]]
    to = to + 2 * more * np.stack(mag)
    for n_split in (1, 2):
        out, lse = g.decode_fp8_block(q.to(DEV), *c.args(), c.lens(), 64, n_split=n_split)
        assert (np.abs(lse.double().cpu().numpy() - l) <= tl + more).all()
        assert (np.abs(out.double().cpu().numpy() - o) <= to).all()


@pytest.mark.parametrize("exps", [(-100.0, -6.0, -5.0), (-6.0, -math.inf, -math.inf, -7.0),
                                  (20.0, -50.0), (-100.0, -100.0, -100.0, -100.0, 0.0)])
@pytest.mark.parametrize("T_q,G", [(1, 8), (2, 8), (2, 16), (8, 8)])
@pytest.mark.parametrize("block", [16, 64, 128])
def test_value_scales_far_apart(exps, T_q, G, block):
    """Blocks of no, or the smallest, values and others, next to one another, in the tiles of
    another stream or in another split: all count alike in the sum of weights."""
    S = 1100
    c = Cache(1, S, 1, 64, block, 0, seed=T_q + block)
    k, v = c.rows(S)
    c.append(k, v, [S])
    codes = torch.randint(0, 0x39, c.v8.shape, generator=c.gen, dtype=torch.uint8)
    codes |= torch.randint(0, 2, c.v8.shape, generator=c.gen, dtype=torch.uint8) << 7
    c.v8.copy_(codes)
    c.val["v"] = ref.E4M3[codes.numpy()]
    nb = c.vs.shape[1]
    c.vs.copy_(torch.tensor([2.0 ** exps[i % len(exps)] for i in range(nb)]).view(1, nb, 1))
    c.scale["v"] = c.vs.double().cpu().numpy()
    q = torch.randn(1, T_q, G, 64, generator=c.gen).to(torch.bfloat16)
    o, l, to, tl = c.expect(q, 1 / 8)
    # logarithms of up to 115 in fp32: half a step of 2^-18 for a key's own, the reference's
    # and the sum's; weights left out are below 2^(100 - 126) of the largest, 1100 of them
    more = 3 * 2.0 ** -18 + 1100 * 2.0 ** -26
    mag = ref.attention(q[0].double().numpy(), c.val["k"][0], c.scale["k"][0], np.abs(c.val["v"][0]),
                        c.scale["v"][0], S, block, 1 / 8)[0]
    for n_split in (1, 2, 3, 9):
        out, lse = g.decode_fp8_block(q.to(DEV), *c.args(), c.lens(), block, n_split=n_split)
        assert (np.abs(lse.double().cpu().numpy() - l) <= tl + more).all(), n_split
        assert (np.abs(out.double().cpu().numpy() - o) <= to + 2 * more * mag).all(), n_split


# ---------------------------------------------------- appending under odd scales --
@pytest.mark.parametrize("old", [-5.0, -0.001, math.nan, 0.0, -0.0])
def test_append_under_a_negative_or_nan_scale(old):
    """A block keeps the larger of its present scale's magnitude and the new one, and its older
    values: a negative scale moves its sign into the codes, a NaN one makes NaN codes."""
    c = Cache(1, 64, 2, 64, 32, 0, seed=7)
    k, v = c.rows(40)
    c.append(k, v, [40])
    c.ks[0, 1, 1] = old
    held = float(c.ks[0, 1, 1])
    before = c.gather()["k"][0][0, 32:40, 1].copy()
    k, v = c.rows(12)
    x = k[0, :, 1].double().numpy()
    # (the reference holds what the call is to leave: the rest of the cache by its own rule)
    c.append(k, v, [12])
    fresh = ref.block_scale(np.abs(x).max())
    s = max(abs(held), fresh) if held == held else fresh
    c.scale["k"][0, 1, 1] = s
    c.val["k"][0, 32:40, 1] = ref.round_e4m3(before * (held / s))
    got = c.gather()["k"]
    assert got[1][0, 1, 1] == s
    assert np.array_equal(got[0][0, 32:40, 1], c.val["k"][0, 32:40, 1], equal_nan=True)
    # x / s in fp32 (2^-24) may tip a tie: one step of the code at most
    want = ref.round_e4m3(x / s)
    assert (np.abs(got[0][0, 40:52, 1] - want) <= np.maximum(2.0 ** -3 * np.abs(want), 2.0 ** -9)).all()
    c.val["k"][0, 40:52, 1] = got[0][0, 40:52, 1]
    c.check()


# ------------------------------------------------- packed heads of long capacity --
@pytest.mark.parametrize("T_q,G,page", [(1, 8, 0), (1, 16, 0), (2, 5, 64), (1, 8, 128)])
def test_heads_that_share_a_tile_in_batches_of_long_capacity(T_q, G, page):
    """Four heads of d = 32 in a CTA, whose rows together are enough for splits that are cut by the
    lengths: short sequences in a cache of long capacity, other lengths beside the same ones, bad
    lengths among them."""
    B, H, S = 24, 8, 19456
    c = Cache(B, 700, H, 32, 64, page, seed=G)
    k, v = c.rows(700)
    lens = [700, T_q, 129] + [700 - 5 * i for i in range(B - 3)]
    c.append(k, v, lens)
    if page:  # a table of long capacity: what lies past the lengths is never read
        table = torch.full((B, S // page), -1, dtype=torch.int32, device=DEV)
        table[:, :c.table.shape[1]] = c.table
        c.table = table
    else:
        wide = g.kv_cache_fp8_block(B, S, H, 32, 64, DEV)
        for new, old in zip(wide, c.args()):
            new[:, :old.shape[1]] = old
        c.k8, c.v8, c.ks, c.vs = wide
    assert g.gqa_attn_decode_fp8_block_default_splits(B, T_q, H * G, H, S) > 1
    q = torch.randn(B, T_q, H * G, 32, generator=c.gen).to(torch.bfloat16)
    check_decode(c, T_q, G, None, q=q)
    check_decode(c, T_q, G, 30, q=q)
    out, lse = check_decode(c, T_q, G, 7, q=q)
    qd = q.to(DEV) if T_q > 1 else q[:, 0].contiguous().to(DEV)
    others = c.lens()
    others[3:] = torch.arange(B - 3, dtype=torch.int32, device=DEV) % 40 + T_q
    out2, lse2 = g.decode_fp8_block(qd, *c.args(), others, 64, n_split=7,
                                    block_table=c.table)
    # the same sums in another cut: two results within the tolerances of check_decode
    o, l, to, tl = c.expect(q, 1 / math.sqrt(32))

    def same(out2, lse2):
        assert (np.abs(out2[:3].double().cpu().numpy().reshape(o[:3].shape) - o[:3]) <= to[:3]).all()
        assert (np.abs(lse2[:3].double().cpu().numpy().reshape(l[:3].shape) - l[:3]) <= tl[:3]).all()

    same(out2, lse2)
    others[5], others[6] = S + 1, T_q - 1
    out2, lse2 = g.decode_fp8_block(qd, *c.args(), others, 64, n_split=7,
                                    block_table=c.table)
    assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
    assert bool(out2[5:7].isnan().all()) and bool(lse2[5:7].isnan().all())
    same(out2, lse2)
    assert bool(out2[7:].isfinite().all())
