"""The block-scaled E4M3 cache where it can go wrong: NaN in masked places, heads that
share a tile, scales the caller wrote, pools past 32-bit offsets, memory around the
buffers, streams of the caller's, two sequences on one page, batches cut by their lengths,
and the bounds-checking build against the default build."""
import math

import numpy as np
import pytest
import torch

import fp8_block_ref as ref
import gqa_attention_gb300 as g
from gqa_attention_gb300 import _binding
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


# -------------------------------------------------------- NaN behind the mask --
@pytest.mark.parametrize("d,H,G,T_q,n_split", [(128, 2, 4, 2, 1), (128, 1, 1, 8, 1), (64, 2, 8, 8, 3),
                                               (128, 2, 1, 64, 2), (32, 4, 2, 5, 200),
                                               (128, 1, 5, 6, 1)])
@pytest.mark.parametrize("ctx", [300, 128, 131, 64])
@pytest.mark.parametrize("page", [0, 16])
def test_nan_values_stay_behind_the_mask(d, H, G, T_q, n_split, ctx, page):
    """NaN among the last tokens' keys and values reaches the queries that see those tokens,
    in the element it stands in (values) or the whole row (keys), and nothing else."""
    c = Cache(2, ctx, H, d, 16, page, seed=d + T_q + ctx)
    k, v = c.rows(ctx)
    lens = [ctx, max(T_q, ctx - 7)]
    q = torch.randn(2, T_q, H * G, d, generator=c.gen).to(torch.bfloat16)
    bad_o = torch.zeros(2, T_q, H * G, d, dtype=torch.bool)
    bad_l = torch.zeros(2, T_q, H * G, dtype=torch.bool)
    hits = {0: [(lens[0] - 1, H - 1, d - 1), (lens[0] - T_q + 1, 0, 17)], 1: [(lens[1] - 1, 0, 0)]}
    for b, list_ in hits.items():
        for t, h, e in list_:
            v[b, t, h, e] = float("nan")
            first = t - (lens[b] - T_q)  # the first query that sees token t
            bad_o[b, first:, h * G:(h + 1) * G, e] = True
    t = lens[0] - T_q // 2 - 1
    k[0, t, 0, 3] = float("inf")
    bad_o[0, t - (lens[0] - T_q):, :G] = True
    bad_l[0, t - (lens[0] - T_q):, :G] = True
    c.append(k, v, lens)
    out, lse = g.decode_fp8_block(q.to(DEV), *c.args(), c.lens(), 16, n_split=n_split,
                                  block_table=c.table)
    assert torch.equal(out.isnan().cpu(), bad_o) and torch.equal(lse.isnan().cpu(), bad_l)
    # everything else is what it is with zeros in their place
    kk, vv = (np.nan_to_num(c.val[n]) for n in "kv")
    for b in range(2):
        o, l, to, tl = ref.attention(q[b].double().numpy(), kk[b], c.scale["k"][b], vv[b],
                                     c.scale["v"][b], lens[b], 16, 1 / math.sqrt(d))
        do = np.abs(out[b].double().cpu().numpy() - o)
        dl = np.abs(lse[b].double().cpu().numpy() - l)
        assert (do <= to)[~bad_o[b].numpy()].all() and (dl <= tl)[~bad_l[b].numpy()].all()


# ------------------------------------------------ heads of d = 32 that share a tile --
@pytest.mark.parametrize("H", [4, 8, 12])
@pytest.mark.parametrize("T_q,G", [(1, 8), (1, 16), (2, 5), (7, 2), (1, 11), (3, 6)])
@pytest.mark.parametrize("block,page", [(16, 0), (64, 128), (128, 0), (32, 32)])
def test_heads_that_share_a_tile(H, T_q, G, block, page):
    c = Cache(2, 700, H, 32, block, page, seed=H + T_q + G + block)
    k, v = c.rows(700)
    c.append(k, v, [700, 129 + T_q])
    check_decode(c, T_q, G, 100, what=f"H={H} T_q={T_q} G={G}")


# -------------------------------------------------------------- scales of the caller's --
def test_append_under_scales_that_are_no_powers_of_two():
    """A present scale that the caller wrote is kept where it is the larger one (codes are
    e4m3(x / s)), and replaced, with the older codes rounded again, where it is not."""
    c = Cache(1, 64, 2, 64, 32, 0, seed=5)
    k, v = c.rows(40)
    c.append(k, v, [40])
    for name, s in (("k", c.ks), ("v", c.vs)):
        s[0, 1] = torch.tensor([3.7, 0.0003], device=DEV)
        c.scale[name][0, 1] = s[0, 1].double().cpu().numpy()
    k, v = c.rows(20)
    c.append(k, v, [20])
    got = c.gather()
    for name in "kv":
        val, scale = got[name]
        assert np.array_equal(scale[0], c.scale[name][0])
        # x / s in fp32 (2^-24) before its rounding to four bits may tip a tie: one step
        # of the code (2^-3 of it, or the subnormal step 2^-9) at most, and rarely
        off = np.abs(val[0, :60] - c.val[name][0, :60])
        assert (off <= np.maximum(2.0 ** -3 * np.abs(c.val[name][0, :60]), 2.0 ** -9)).all()
        assert (off > 0).mean() < 1e-2


# ------------------------------------------------------- pools past 32-bit offsets --
def test_pool_with_offsets_past_32_bits():
    """Pages at the end of a pool of more than 2^32 codes, and at its start."""
    page, H, d, block = 128, 8, 128, 64
    units = 2 ** 32 // (page * H * d) + 9
    k8, v8, ks, vs = g.kv_cache_fp8_block(units, page, H, d, block, DEV)
    c = Cache(2, 5 * page, H, d, block, page, seed=6)
    table = torch.tensor([[units - 1, 0, units - 5, 3, units - 2],
                          [units - 3, units - 4, 1, units - 6, units - 7]], dtype=torch.int32)
    used = table.flatten().long().to(DEV)
    for t in (k8, v8):
        t[used] = 0x7F
    for t in (ks, vs):
        t[used] = float("nan")
    c.k8, c.v8, c.ks, c.vs, c.table = k8, v8, ks, vs, table.to(DEV)
    k, v = c.rows(600)
    c.append(k, v, [600, 431])
    c.gather = lambda: {n: (ref.E4M3[x[used].cpu().numpy()].reshape(2, 5 * page, H, d),
                            s[used].double().cpu().numpy().reshape(2, -1, H))
                        for n, x, s in (("k", k8, ks), ("v", v8, vs))}
    c.check()
    ko, vo = g.kv_read_fp8_block(*c.args(), c.lens(), block, 0, None, None, c.table)
    for name, o in (("k", ko), ("v", vo)):
        s = c.scale[name][0][np.arange(600) // block][..., None]
        assert np.array_equal(o[0, :600].double().cpu().numpy(), c.val[name][0, :600] * s)
    for T_q, n_split in ((1, 1), (1, 3), (4, 2)):
        check_decode(c, T_q, 4, n_split)


def test_last_sequence_of_a_long_contiguous_cache():
    B, S, H, d, block = 3, 600_000, 16, 128, 128  # 3.7e9 codes
    k8, v8, ks, vs = g.kv_cache_fp8_block(B, S, H, d, block, DEV)
    gen = torch.Generator().manual_seed(8)
    k = torch.randn(B, 3, H, d, generator=gen).to(torch.bfloat16)
    v = torch.randn(B, 3, H, d, generator=gen).to(torch.bfloat16)
    lens = torch.tensor([0, 130, 3], dtype=torch.int32)
    n_new = torch.tensor([0, 2, 3], dtype=torch.int32)
    for t in (k8, v8):
        t[1, :128] = 0
    for t in (ks, vs):
        t[1, 0] = 1.0
    kd, vd, ld, nd = (x.to(DEV) for x in (k, v, lens, n_new))
    g.kv_append_fp8_block(kd, vd, k8, v8, ks, vs, ld, block, n_new=nd)
    ko, vo = (torch.zeros(B, 3, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g.kv_read_fp8_block(k8, v8, ks, vs, ld, block, 0, ko, vo)
    val, scale = np.zeros((S, H, d))[:3], np.zeros((1, H))
    ref.append(k[2].double().numpy(), val, scale, 0, block)
    assert np.array_equal(ko[2].double().cpu().numpy(), val * scale[0][:, None])
    assert bool((ko[0] == 0).all())
    assert g.gqa_last_device_error() == g.GQA_OK


# ------------------------------------------------------------ memory around buffers --
def _guarded(shape, dtype, margin=4096):
    """A tensor inside a larger buffer of the byte 0xA5, and a check that the rest is intact."""
    n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
    raw = torch.full((margin + -(-n // 256) * 256 + margin,), 0xA5, dtype=torch.uint8, device=DEV)

    def intact():
        return bool((raw[:margin] == 0xA5).all()) and bool((raw[margin + n:] == 0xA5).all())

    return raw[margin:margin + n].view(dtype).view(shape), intact


@pytest.mark.parametrize("d,T_q,G,n_split", [(128, 1, 8, 1), (128, 8, 8, 3), (64, 3, 5, 2),
                                             (32, 1, 7, 150), (128, 1, 16, 4)])
@pytest.mark.parametrize("page", [0, 32])
def test_nothing_is_written_around_the_buffers(d, T_q, G, n_split, page):
    B, S, H, block = 2, 333, 4, 32
    c = Cache(B, S, H, d, block, page, seed=d + T_q)
    checks = []
    for name in ("k8", "v8", "ks", "vs"):
        old = getattr(c, name)
        new, intact = _guarded(old.shape, old.dtype)
        new.copy_(old)
        setattr(c, name, new)
        checks.append(intact)
    k, v = c.rows(S - 1)
    c.append(k, v, [S - 1, 200])
    k, v = c.rows(1, gain=9.0)
    c.append(k, v, [1, 1], pad=8)
    c.check()
    outs = {}
    for name, shape, dt in (("ko", (B, 150, H, d), torch.bfloat16), ("vo", (B, 150, H, d), torch.bfloat16),
                            ("out", (B, T_q, H * G, d), torch.bfloat16),
                            ("lse", (B, T_q, H * G), torch.float32),
                            ("ws", (g.gqa_attn_decode_workspace_bytes(B * T_q, H * G, d, n_split),),
                             torch.uint8)):
        outs[name], intact = _guarded(shape, dt)
        checks.append(intact)
    g.kv_read_fp8_block(*c.args(), c.lens(), block, 101, outs["ko"], outs["vo"], c.table)
    q = torch.randn(B, T_q, H * G, d, generator=c.gen).to(torch.bfloat16)
    g.decode_fp8_block(q.to(DEV), *c.args(), c.lens(), block, n_split=n_split, workspace=outs["ws"],
                       out=outs["out"], lse=outs["lse"], block_table=c.table)
    torch.cuda.synchronize()
    assert all(f() for f in checks)
    o, l, to, tl = c.expect(q, 1 / math.sqrt(d))
    assert (np.abs(outs["out"].double().cpu().numpy() - o) <= to).all()
    assert (np.abs(outs["lse"].double().cpu().numpy() - l) <= tl).all()
    # rows of tokens past the second sequence's end are what they were
    assert bool((outs["ko"][1, 201 - 101:].view(torch.uint8) == 0xA5).all())


# -------------------------------------------------------------------- calls together --
def test_sequences_that_share_a_prefix_page():
    """Two sequences whose first pages are the same ones, decoded in one batch."""
    c = Cache(2, 256, 2, 128, 32, 64, seed=9)
    k, v = c.rows(256)
    k[1, :128], v[1, :128] = k[0, :128], v[0, :128]
    c.append(k, v, [256, 200])
    c.table[1, :2] = c.table[0, :2]
    check_decode(c, 1, 8, 1)
    check_decode(c, 4, 8, 2)


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_results_on_a_stream_of_the_callers(kind):
    """Every result of the helpers is allocated on the stream that is given, so that what the
    current stream does with its own memory at the time does not reach it."""
    c = Cache(2, 900, 2, 128, 16, 0, seed=10)
    k, v = c.rows(900)
    c.append(k, v, [900, 500])
    lens = c.lens()
    q = torch.randn(2, 16, 128, generator=c.gen).to(torch.bfloat16).to(DEV)
    q2 = torch.randn(2, 20, 16, 128, generator=c.gen).to(torch.bfloat16).to(DEV)
    want = (*g.decode_fp8_block(q, *c.args(), lens, 16), *g.kv_read_fp8_block(*c.args(), lens, 16),
            *g.prefill_chunk_fp8_block(q2, *c.args(), lens, 16))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = side if kind == "stream" else side.cuda_stream
    busy = torch.ones(1 << 24, device=DEV)
    for _ in range(4):
        for _ in range(20):
            busy.mul_(1.0)
        fill = [torch.full((2, 900, 2, 128), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
        del fill
        got = (*g.decode_fp8_block(q, *c.args(), lens, 16, stream=s),
               *g.kv_read_fp8_block(*c.args(), lens, 16, stream=s),
               *g.prefill_chunk_fp8_block(q2, *c.args(), lens, 16, stream=s))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


# ------------------------------------------------------- splits cut by the lengths --
@pytest.mark.parametrize("T_q,G", [(4, 8), (8, 8), (17, 1), (3, 7)])
@pytest.mark.parametrize("page", [0, 128])
def test_splits_cut_by_the_lengths(T_q, G, page):
    """Ragged batches of many query rows: one long sequence and short ones, equal ones, all of
    the shortest length, a bad length among good ones, with room for few or many splits."""
    B, H, d, S = 6, 2, 64, 26000  # 12 of 152 SMs' groups, 204 tiles
    c = Cache(B, S, H, d, 128, page, seed=T_q + G)
    k, v = c.rows(9000)
    c.append(k, v, [9000, T_q, 128, 4000, 127 + T_q, 1000])
    for n_split in (2, 5, 24, None):
        out, lse = check_decode(c, T_q, G, n_split, what=f"{n_split}")
    q = torch.randn(B, T_q, H * G, d, generator=c.gen).to(torch.bfloat16).to(DEV)

    def run(lens, n_split=None):
        return g.decode_fp8_block(q, *c.args(), torch.tensor(lens, dtype=torch.int32, device=DEV), 128,
                                  n_split=n_split, block_table=c.table)

    good = run(c.len)
    for bad in (S + 200, T_q - 1, -1):
        out, lse = run([c.len[0], bad, *c.len[2:]])
        assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
        assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
        for x, y in ((out, good[0]), (lse, good[1])):
            # the others: the same sums in another cut, each within (2^-8 + 2^-9) of values
            # below 1.3, whose difference is below 2^-6
            rest = [0, 2, 3, 4, 5]
            assert bool(((x[rest] - y[rest]).abs().float() <= 2.0 ** -6).all())
    again = run(c.len)
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
    for lens in ([T_q] * B, [9000, T_q, T_q, 4000, T_q, 640], [min(n, 64 + 40 * T_q) for n in c.len]):
        c.len = [max(T_q, min(n, m)) for n, m in zip(lens, (9000, T_q, 128, 4000, 127 + T_q, 1000))]
        for n_split in (3, None):
            check_decode(c, T_q, G, n_split, q=q.cpu(), what=f"{c.len}")


def test_splits_cut_by_the_lengths_over_small_pages():
    c = Cache(4, 20000, 4, 64, 16, 16, seed=72)
    k, v = c.rows(3000)
    c.append(k, v, [3000, 900, 5, 129])
    for T_q, G in ((5, 4), (5, 10)):
        check_decode(c, T_q, G, None)


def test_splits_cut_by_the_lengths_follow_a_captured_step():
    """The cut is made on the device: a captured call replayed with other lengths."""
    B, H, d, S, T_q, G = 4, 4, 32, 20000, 5, 4  # 16 groups of heads, 157 tiles
    c = Cache(B, S, H, d, 64, 0, seed=71)
    k, v = c.rows(6000)
    c.append(k, v, [6000, 3000, 700, T_q])
    q = torch.randn(B, T_q, H * G, d, generator=c.gen).to(torch.bfloat16)
    qd, lens = q.to(DEV), c.lens()
    out, lse = g.decode_fp8_block(qd, *c.args(), lens, 64)
    ws = g.decode_workspace(B * T_q, H * G, d, 16)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        g.decode_fp8_block(qd, *c.args(), lens, 64, n_split=16, workspace=ws, out=out, lse=lse)
    for new in ([6000, 3000, 700, T_q], [T_q, 3000, 64, T_q], [5999, 129, 128, T_q]):
        c.len = new
        lens.copy_(c.lens())
        graph.replay()
        torch.cuda.synchronize()
        o, l, to, tl = c.expect(q, 1 / math.sqrt(d))
        assert (np.abs(out.double().cpu().numpy() - o) <= to).all()
        assert (np.abs(lse.double().cpu().numpy() - l) <= tl).all()


# -------------------------------------------------------- the bounds-checking build --
@pytest.fixture(scope="module")
def checking(tmp_path_factory):
    from gqa_attention_gb300 import build

    d = tmp_path_factory.mktemp("bounds")
    path = build.build(extra_flags=["-DGQA_DEBUG_BOUNDS=1"],
                       lib_path=str(d / "libgqa_attn_bounds.so"), build_dir=str(d / "obj"))
    saved, _binding._lib = _binding._lib, None
    try:
        lib = _binding.load(path)
    finally:
        _binding._lib = saved
    yield lib
    _binding._lib = saved


@pytest.mark.parametrize("d,H,G,T_q,n_split", [(128, 2, 8, 1, 1), (128, 2, 8, 8, 3), (64, 3, 5, 3, 2),
                                               (32, 4, 8, 1, 200), (128, 1, 16, 1, None),
                                               (128, 2, 8, 4, 2)])
@pytest.mark.parametrize("block,page", [(16, 0), (16, 16), (64, 128), (128, 0)])
def test_bounds_checking_build_agrees(checking, d, H, G, T_q, n_split, block, page):
    def run(lib):
        saved, _binding._lib = _binding._lib, lib
        try:
            c = Cache(3, 500, H, d, block, page, seed=d + G)
            k, v = c.rows(499)
            c.append(k, v, [499, T_q, 129 + T_q], pad=8)
            k, v = c.rows(1, gain=5.0)
            c.append(k, v, [1, 1, 0])
            q = torch.randn(3, T_q, H * G, d, generator=c.gen).to(torch.bfloat16).to(DEV)
            bad = c.lens()
            bad[1] = 501
            outs = [*c.args(), *g.kv_read_fp8_block(*c.args(), c.lens(), block, 3, None, None, c.table),
                    *g.decode_fp8_block(q, *c.args(), c.lens(), block, n_split=n_split,
                                        block_table=c.table)]
            assert g.gqa_last_device_error() == g.GQA_OK
            if not page:
                outs += g.decode_fp8_block(q, *c.args(), bad, block, n_split=n_split)
                outs += g.kv_read_fp8_block(*c.args(), bad, block)
                assert g.gqa_last_device_error() == g.GQA_ERR_INVALID_ARG
            return outs
        finally:
            _binding._lib = saved

    for x, y in zip(run(g.load()), run(checking)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
