"""The rotated append and differential attention in a library that checks every computed global
store (-DGQA_DEBUG_BOUNDS=1): no store outside the buffers, outputs equal to the default build's
bit for bit; and nothing written around outputs and caches that lie inside larger buffers."""
import pytest
import torch

import gqa_attention_gb300 as g
from test_debug_bounds_gpu import _compare, libs  # noqa: F401  (the fixture builds the library)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rnd(*s):
    return torch.randn(*s, device=DEV).to(torch.bfloat16)


def table_for(B, nb, units):
    return torch.randperm(units, device=DEV)[: B * nb].view(B, nb).to(torch.int32)


@pytest.mark.parametrize("d,H,Hk,T,page,n_split", [
    (32, 4, 2, 1, 0, 1), (64, 8, 2, 1, 16, 3), (128, 16, 2, 1, 64, None), (64, 6, 1, 5, 16, 2),
    (128, 8, 1, 4, 0, 1), (128, 8, 1, 4, 64, 5), (32, 2, 1, 13, 0, None), (128, 3, 3, 1, 0, 40),
])
@pytest.mark.parametrize("split", [False, True])
def test_decode_stays_in_bounds(libs, d, H, Hk, T, page, n_split, split):  # noqa: F811
    def run():
        lens = torch.tensor([T, 900, 77], dtype=torch.int32, device=DEV)
        if page:
            nb = -(-900 // page)
            table = table_for(3, nb, 3 * nb + 1)
            k, v = (rnd(3 * nb + 1, page, Hk, d) for _ in "kv")
        else:
            table, (k, v) = None, (rnd(3, 900, Hk, d) for _ in "kv")
        q = rnd(3, T, H if split else 2 * H, d)
        lam = torch.rand(3, T, H, device=DEV)
        return g.decode_diff(q, k, v, lens, lam, split_keys=split, norm_eps=1e-5, n_split=n_split,
                             block_table=table)

    _compare(libs, run)


def test_cut_batches_stay_in_bounds(libs):  # noqa: F811
    for d, T, H in ((128, 4, 8), (64, 3, 6), (128, 1, 4)):
        def run():
            lens = torch.tensor([9000, T, 300, 64], dtype=torch.int32, device=DEV)
            table = torch.zeros(4, 3200, dtype=torch.int32, device=DEV)
            table[:, :141] = table_for(4, 141, 564)
            k, v = (rnd(564, 64, 1, d) for _ in "kv")
            return g.decode_diff(rnd(4, T, 2 * H, d), k, v, lens, torch.rand(4, T, H, device=DEV),
                                 block_table=table)

        _compare(libs, run)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("split", [False, True])
def test_prefill_stays_in_bounds(libs, d, split):  # noqa: F811
    for S, T, n_part, window in ((300, 300, 1, -1), (700, 45, 3, -1), (700, 150, 1, 90)):
        def run():
            lens = None if T == S else torch.tensor([700, T], dtype=torch.int32, device=DEV)
            return g.prefill_diff(rnd(2, T, 4 if split else 8, d), rnd(2, S, 2, d), rnd(2, S, 2, d),
                                  torch.rand(2, T, 4, device=DEV), lens, split_keys=split,
                                  norm_eps=1e-5, window=window, n_part=n_part)

        _compare(libs, run)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_stays_in_bounds(libs, fp8):  # noqa: F811
    for B, T, Hq, Hk, d, page in ((3, 1, 8, 2, 128, 16), (2, 333, 5, 5, 64, 0), (1, 7, 3, 20, 128, 64),
                                  (1, 3000, 8, 8, 128, 0)):
        def run():
            S = T + 30
            per, units = (page, B * -(-S // page)) if page else (-(-S // 4) * 4, B)
            k, v = (torch.zeros(units, per, Hk, d, device=DEV,
                                dtype=torch.uint8 if fp8 else torch.bfloat16) for _ in "kv")
            more = {}
            if fp8:
                more = {n: torch.zeros(units, per, device=DEV) for n in ("k_scale", "v_scale")}
            if page:
                more["block_table"] = table_for(B, -(-S // page), units)
            lens = torch.tensor([T + 7 * b for b in range(B)], dtype=torch.int32, device=DEV)
            out = g.kv_append(rnd(B, T, Hk, d), rnd(B, T, Hk, d), k, v, lens,
                              freqs=torch.rand(d // 2, device=DEV), q=rnd(B, T, Hq, d), **more)
            # (codes as 16-bit words for the comparison of bits)
            as16 = [x.view(torch.bfloat16) if fp8 else x for x in (k, v)]
            return [out, *as16] + ([more["k_scale"], more["v_scale"]] if fp8 else [])

        _compare(libs, run)


def guarded(shape, dtype):
    """A dense tensor inside a larger buffer of canaries; and the check of those."""
    n = 1
    for s in shape:
        n *= s
    size = torch.empty(0, dtype=dtype).element_size()
    pad = 4096 // size
    whole = torch.full(((n + 2 * pad) * size,), 0x5A, dtype=torch.uint8, device=DEV)
    inner = whole.view(dtype)[pad:pad + n].view(shape)

    def intact():
        return bool((whole[:pad * size] == 0x5A).all() and (whole[(pad + n) * size:] == 0x5A).all())

    return inner, intact


def test_nothing_is_written_around_outputs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    checks = []

    def buf(shape, dtype=torch.bfloat16):
        x, ok = guarded(shape, dtype)
        checks.append(ok)
        return x

    for d, T, H, Hk, n in ((64, 1, 5, 5, 1), (128, 3, 8, 1, 2), (32, 7, 4, 2, 3), (128, 1, 8, 1, None)):
        k, v = rnd(3, 500, Hk, d), rnd(3, 500, Hk, d)
        lens = torch.tensor([500, T, 129], dtype=torch.int32, device=DEV)
        lam = torch.rand(3, T, H, device=DEV)
        g.decode_diff(rnd(3, T, 2 * H, d), k, v, lens, lam, n_split=n, norm_eps=1e-5,
                      out=buf((3, T, H, d)), lse=buf((3, T, 2 * H), torch.float32),
                      workspace=buf((g.gqa_attn_decode_workspace_bytes(3 * T, 2 * H, d, n or 1),),
                                    torch.uint8) if n and n > 1 else None)
        g.prefill_diff(rnd(3, T, 2 * H, d), k, v, lam, lens, out=buf((3, T, H, d)),
                       lse=buf((3, 2 * H, T), torch.float32))
    for fp8 in (False, True):
        more = dict(k_scale=buf((2, 44), torch.float32), v_scale=buf((2, 44), torch.float32)) \
            if fp8 else {}
        kind = torch.uint8 if fp8 else torch.bfloat16
        lens = torch.tensor([44, 30], dtype=torch.int32, device=DEV)
        g.kv_append(rnd(2, 30, 3, 64), rnd(2, 30, 3, 64), buf((2, 44, 3, 64), kind),
                    buf((2, 44, 3, 64), kind), lens, q=rnd(2, 30, 7, 64), q_out=buf((2, 30, 7, 64)),
                    freqs=torch.rand(32, device=DEV), **more)
    torch.cuda.synchronize()
    assert g.gqa_last_device_error() == g.GQA_OK
    assert all(ok() for ok in checks)
