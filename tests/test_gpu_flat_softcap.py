"""Softcaps so small that every score comes out as nothing: attention is the mean of the
values seen, the log of its sums that of their number, and weights are shared alike."""
import pytest
import torch

import gqa_attention_cu_gb300 as pva
from paged_cases import DT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, HKV = 8, 2
CAPS = [1e-9, 1e-12, -1e-20, 1e-37, 1e-44]
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def near(got, ref, size, n, dtype):
    """A rounding of the output, one of 2^-24 a key in the sum, and 2^-20 of exponentials."""
    tol = HALF[dtype] * ref.abs() + ((n + 16) * 2.0 ** -24 + 2.0 ** -20) * size
    assert ((got.cpu().double() - ref).abs() <= tol).all()


def mean_of(v, n):
    """[Hkv, rows, d] -> [H, d], and of the sizes."""
    v = v[:, :n].double().repeat_interleave(H // HKV, 0)
    return v.mean(1), v.abs().mean(1)


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("by", [0.0, 1.0])  # all scores zero, or some
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("bf16", 256), ("f16", 96), ("f32", 80)])
def test_packed(dtype, d, by, cap):
    """Prompts and single rows, with and without the library's own workspace."""
    td, lens = DT[dtype], [130, 1, 1]
    kv = [200, 300, 7]
    q = (by * randn(sum(lens), H, d)).to(td)
    k, v = randn(sum(kv), HKV, d, seed=1).to(td), randn(sum(kv), HKV, d, seed=2).to(td)
    cu = [torch.tensor([0, *torch.tensor(x).cumsum(0).tolist()], dtype=torch.int32, device=DEV) for x in (lens, kv)]
    for call in (pva.pva_forward, pva.pva_forward_noalloc):
        out = torch.full_like(q, float("nan"), device=DEV)
        call(q.to(DEV), k.to(DEV), v.to(DEV), *cu, out, 3, H, HKV, d, d, softcap=cap, is_causal=1)
        torch.cuda.synchronize()
        assert pva.pva_get_status() == 0
        row, first = 0, 0
        for nq, n in zip(lens, kv):
            for t in range(nq):
                near(out[row], *mean_of(v[first:first + n].transpose(0, 1), n - nq + t + 1), n, dtype)
                row += 1
            first += n


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("by", [0.0, 1.0])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("bf16", 256), ("f32", 80)])
@pytest.mark.parametrize("T", [1, 3])
def test_caches(T, dtype, d, by, cap):
    """A tree step, rows behind a prefix, and the weights of the rows."""
    td, past, m = DT[dtype], 150, 90
    n = past + T
    q = (by * randn(1, T, H, d)).to(td)
    k, v = randn(2, HKV, 256, d, seed=1).to(td), randn(2, HKV, 256, d, seed=2).to(td)
    new = [c[:1, :, past:n].transpose(1, 2).contiguous().to(DEV) for c in (k, v)]
    own = [c[:1].clone().to(DEV) for c in (k, v)]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    out = torch.full_like(q, float("nan"), device=DEV)
    pva.pva_gqa_tree(q.to(DEV), *new, *own, i32(past), out, H, HKV, softcap=cap)
    assert pva.pva_get_status() == 0
    for t in range(T):
        near(out[0, t], *mean_of(v[0], past + t + 1), n, dtype)
    lse = torch.empty(1, T, H, device=DEV)
    pva.pva_gqa_prefix(q.to(DEV), k.to(DEV), v.to(DEV), i32(n), i32(m), out, H, HKV, lse=lse, softcap=cap)
    assert pva.pva_get_status() == 0
    for t in range(T):
        near(out[0, t], *mean_of(torch.cat([v[1, :, :m], v[0]], 1), m + past + t + 1), m + n, dtype)
        assert (lse[0, t].cpu().double() - torch.tensor(float(m + past + t + 1)).double().log()).abs().max() <= 2.0 ** -18
    share = torch.zeros(n, dtype=torch.float64)
    for t in range(T):
        share[:past + t + 1] += H // HKV / (past + t + 1)
    for sums in (None, torch.tensor([past + t + 1.0 for t in range(T)], device=DEV).log()[None, :, None].expand(1, T, H).contiguous()):
        w = torch.full((1, HKV, n), float("nan"), device=DEV)
        pva.pva_kvcache_weights(q.to(DEV), own[0], i32(n), w, H, lse=sums, softcap=cap)
        assert pva.pva_get_status() == 0
        assert ((w[0].cpu().double() - share).abs() <= 2.0 ** -18 * share).all()
