"""Differential attention on the GPU at the limits of its arguments: the longest sequences, key rows
that are not finite, default splits of large batches."""
import pytest
import torch

import diff_ref as ref
import gqa_attention_gb300 as g
from test_diff_gpu import Case

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


def test_cut_batch_of_the_longest_sequences():
    """Two sequences of up to 2^31 - 2^16 tokens in pages of 65536, all but the last of each the
    same page: its keys are far from every query, and only the last 130 tokens have a weight.  The
    last piece of the longer one ends past 2^31, were it a whole one."""
    page, H, T, d, n = 65536, 8, 2, 128, 130
    lens = [0x7fff0000, 0x60000000]
    c = Case([n, n], T, H, 1, d, lam="token", seed=1)
    c.q[..., 0] = c.q[..., 0].abs() + 1
    k = torch.zeros(3, page, 1, d, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    k[..., 0] = -30000.0  # (a score below -2600: its weight is 0 in fp32)
    for b in range(2):
        k[1 + b, -n:], v[1 + b, -n:] = c.k[b], c.v[b]
    table = torch.zeros(2, lens[0] // page, dtype=torch.int32, device=DEV)
    for b, L in enumerate(lens):
        table[b, L // page - 1] = 1 + b
    want = c.expect()
    for n_split in (None, 152):
        out, lse = g.decode_diff(c.q.to(DEV), k, v, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                 c.lam.to(DEV), block_table=table, n_split=n_split)
        c.compare(out, lse, want, n_split)


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("T,H,Hk,d,n_split", [
    (1, 3, 3, 64, 1), (1, 8, 2, 128, 2), (2, 8, 1, 128, 1), (3, 5, 1, 32, 3), (8, 4, 1, 64, 1),
    (8, 8, 2, 128, 2), (5, 3, 1, 128, 1),
])
@pytest.mark.parametrize("prefill", [False, True])
def test_split_keys_see_their_own_half_of_a_key(T, H, Hk, d, n_split, prefill):
    """NaN or an infinity in one half of a key row reaches that half's map alone; where its score
    is minus infinity, it is as a key of no weight."""
    half = d // 2
    for u in (0, 1):
        c = Case([70, 200], T, H, Hk, d, True, S=200, seed=d + T + u)
        at = u * half + 3
        c.q[..., at] = -1.0 - c.q[..., at].abs()
        run = (lambda: c.prefill(n_part=n_split)) if prefill else (lambda: c.decode(n_split=n_split))

        def maps(x):  # lse, [B, T, H, map]
            x = x.transpose(1, 2) if prefill else x
            return x.reshape(2, T, H, 2)

        c.k[:, 5, :, at] = 1e5  # a score below -3000 in map u: its weight is 0 in fp32
        out, lse = run()
        assert torch.isfinite(out.float()).all()
        c.k[:, 5, :, at] = float("inf")
        far, far_lse = run()
        assert same(far, out) and torch.equal(far_lse, lse)
        c.k[:, 5, :, u * half:(u + 1) * half] = float("nan")
        bad, bad_lse = run()
        assert bad.isnan().all() and maps(bad_lse)[..., u].isnan().all()
        assert torch.equal(maps(bad_lse)[..., 1 - u], maps(lse)[..., 1 - u])
        torch.cuda.synchronize()
        assert g.gqa_last_device_error() == g.GQA_OK


@pytest.mark.parametrize("d,T", [(64, 1), (128, 2)])
def test_default_splits_of_the_widest_table(d, T):
    # short sequences behind a table of 2^31 - 2^16 tokens: nearly all of the default splits are empty
    page, H = 65536, 8
    c = Case([700], T, H, 1, d, lam="head", seed=d)
    k = torch.full((2, page, 1, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    k[1, :700], v[1, :700] = c.k[0], c.v[0]
    table = torch.full((1, 32767), -1, dtype=torch.int32, device=DEV)
    table[0, 0] = 1
    q, lam = c.q.to(DEV), c.lam.to(DEV)
    out, lse = g.decode_diff(q, k, v, c.dev_lens(), lam, block_table=table)
    c.compare(out, lse, c.expect())
