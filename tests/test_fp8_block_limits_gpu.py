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


# ------------------------------------------------------ weights far below the largest --
def _behind_a_sink(S, T_q, G, B, share, mean, at=0, seed=0):
    """Codes, scales and queries such that token `at` has a value of zero and all but `share`
    of every row's weight, the rest lying log-normally (0.7) over the other tokens, whose
    values have the given mean."""
    gen = torch.Generator().manual_seed(seed)
    H, d = 1, 128
    cache = g.kv_cache_fp8_block(B, S, H, d, 64, DEV)
    k8, v8, ks, vs = cache
    x = (0.7 * torch.randn(S, generator=gen)).double()
    x[at] = -math.inf
    x[at] = float(torch.logsumexp(x, 0)) + math.log((1 - share) / share)
    # in two elements of the key, E4M3 each: x = a + b / 16
    a = torch.from_numpy(ref.round_e4m3(x.numpy()))
    b = torch.from_numpy(ref.round_e4m3(16 * (x - a).numpy()))
    k = torch.zeros(S, d, dtype=torch.float64)
    k[:, 0], k[:, 1] = a, b
    v = torch.randn(S, d, generator=gen).double() + mean
    v = torch.from_numpy(ref.round_e4m3(v.numpy()))
    v[at] = 0
    k8[:, :, 0] = k.float().to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    v8[:, :, 0] = v.float().to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    ks.fill_(1.0), vs.fill_(1.0)
    q = torch.zeros(B, T_q, H * G, d, dtype=torch.bfloat16)
    q[..., 0], q[..., 1] = 1.0, 1 / 16
    p = torch.exp(a + b / 16)
    z = p.cumsum(0)[-T_q:, None]  # of query t: the tokens up to its own
    o = (p[:, None] * v).cumsum(0)[-T_q:] / z
    mag = (p[:, None] * v.abs()).cumsum(0)[-T_q:] / z
    tile = slice(at // 128 * 128, at // 128 * 128 + 128)
    own = (p[tile, None] * v[tile].abs()).sum(0) / z
    return cache, q.to(DEV), *(y.numpy() for y in (o, torch.log(z[:, 0]), mag, own))


SINKS = [(32768, 1, 8, 1, None), (32768, 8, 8, 1, None), (8192, 8, 8, 1, 1), (32768, 8, 8, 3, 3),
         (8192, 4, 4, 2, None), (4096, 2, 16, 1, 1), (1024, 1, 4, 1, 1)]


@pytest.mark.parametrize("S,T_q,G,B,n_split", SINKS)
@pytest.mark.parametrize("at", [0, 700])
def test_a_tail_behind_a_sink_keeps_its_weight(S, T_q, G, B, n_split, at):
    """A token with a value of zero and all but 2^-12 of the weight; values of mean 1. The tail's
    weights are held to 2^-9 of themselves outside the sink's tile."""
    cache, q, o, l, mag, own = _behind_a_sink(S, T_q, G, B, 2.0 ** -12, 1.0, at)
    lens = torch.full((B,), S, dtype=torch.int32, device=DEV)
    out, lse = g.decode_fp8_block(q, *cache, lens, 64, scale=1.0, n_split=n_split)
    # O to 2^-8 (bf16), weights to 2^-9, or 2^-14 of their tile's largest, which is under 8 times
    # the mean; the sink's tile may lose its own tail. Scores are below 32: 2^-18 in all.
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -17) * mag + own
    do = np.abs(out.double().cpu().numpy() - o[None, :, None])
    assert (do <= tol[None, :, None]).all(), float((do / tol[None, :, None]).max())
    assert (np.abs(lse.double().cpu().numpy() - l[None, :, None]) <= 2.0 ** -16).all()


@pytest.mark.parametrize("S,T_q,G,B,n_split", SINKS)
@pytest.mark.parametrize("share", [0.03, 0.01])
def test_a_tail_of_mean_zero_behind_a_sink(S, T_q, G, B, n_split, share):
    """The same with 3% and 1% left and values of mean 0, whose sum is as small as the errors of
    its terms add up to."""
    cache, q, o, *_ = _behind_a_sink(S, T_q, G, B, share, 0.0)
    lens = torch.full((B,), S, dtype=torch.int32, device=DEV)
    out, _ = g.decode_fp8_block(q, *cache, lens, 64, scale=1.0, n_split=n_split)
    err = np.linalg.norm(out.double().cpu().numpy() - o[None, :, None], axis=-1)
    rel = err / np.linalg.norm(o, axis=-1)[None, :, None]
    # The sink's tile: its weights are rounded in steps of 2^-14 where the sink's is 2^7, a
    # deviation of 2^-14 / sqrt(12) each against weights of 2^7 share / (1 - share) / S on
    # average, whose squares are e^0.49 of the average's; 128 of S tokens have it.
    # Everything else: O to 2^-8, weights to less. Half as much again, for the scatter of a
    # sum of 128 terms.
    dev = 2.0 ** -14 / math.sqrt(12) * S * (1 - share) / (share * 2.0 ** 7)
    dev *= math.sqrt(128 / S / math.exp(0.49))
    assert rel.max() <= 1.5 * math.hypot(dev, 2.0 ** -8), (float(rel.max()), dev)


@pytest.mark.parametrize("e", [-100, -61, -60, 0])
@pytest.mark.parametrize("S,T_q,G,B,n_split", SINKS)
def test_a_sink_over_value_scales_of_every_size(S, T_q, G, B, n_split, e):
    """The sum of weights, which is held over the value scales, stays within fp32 whether or not
    references fall."""
    cache, q, o, l, mag, own = _behind_a_sink(S, T_q, G, B, 2.0 ** -20, 1.0)
    cache[3].fill_(2.0 ** e)
    lens = torch.full((B,), S, dtype=torch.int32, device=DEV)
    out, lse = g.decode_fp8_block(q, *cache, lens, 64, scale=1.0, n_split=n_split)
    # logarithms of up to 135: half a step of 2^-17 for a key's own, the reference's, the sum's
    assert (np.abs(lse.double().cpu().numpy() - l[None, :, None]) <= 2.0 ** -16 + 3 * 2.0 ** -17).all()
    assert bool(out.isfinite().all())
    assert (np.abs(out.double().cpu().numpy()) <= 1.1 * mag[None, :, None] * 2.0 ** e).all()


# ----------------------------------------------------------------- refusals of a chunk --
def test_chunk_refuses_outputs_of_another_shape():
    c = Cache(2, 64, 2, 64, 16, 0, seed=3)
    k, v = c.rows(40)
    c.append(k, v, [40, 33])
    q = torch.randn(2, 5, 8, 64, generator=c.gen).to(torch.bfloat16).to(DEV)
    out = torch.empty(2, 5, 8, 64, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(2, 8, 5, device=DEV)
    for bad in (dict(out=out[:1]), dict(out=out[:, :4]), dict(out=out.float()), dict(out=out.cpu()),
                dict(out=out.transpose(1, 2)), dict(lse=lse[:, :, :4]), dict(lse=lse.half()),
                dict(lse=torch.empty(2, 5, 8, device=DEV))):
        with pytest.raises(g.GQAError):
            g.prefill_chunk_fp8_block(q, *c.args(), c.lens(), 16, **bad)
    want = g.prefill_chunk_fp8_block(q, *c.args(), c.lens(), 16)
    got = g.prefill_chunk_fp8_block(q, *c.args(), c.lens(), 16, out=out, lse=lse)
    assert got[0] is out and torch.equal(out, want[0]) and torch.equal(lse, want[1])
