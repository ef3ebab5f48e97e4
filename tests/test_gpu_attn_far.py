"""The attention layer where offsets pass 32 bits: rows at the largest distance, caches of more than 4 GiB."""
import numpy as np
import pytest

from gpu_util import note, torch_dev
from test_gpu_attn_cache import ints
from test_gpu_attn_prompt import check_forward, offsets
from test_gpu_attn_prompt_bwd import check

pytestmark = pytest.mark.gpu
FAR = 2 ** 24 - 8


def rows(torch, rng, T, heads, D, fill=True):
    """Parts [T, n, D] of rows that are FAR elements apart."""
    buf = torch.empty((T - 1) * FAR + sum(heads) * D, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((T, sum(heads), D), (FAR, D, 1))
    if fill:
        x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32)).cuda())
    return x.split(heads, 1)


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_rows_far_apart(D):
    """300 rows: 10 GB between the first and the last."""
    torch = torch_dev()
    q, k, v, do = rows(torch, np.random.default_rng(D), 300, [4, 2, 2, 4], D)
    note(f"far prompt D{D}")
    check_forward(torch, q, k, v, offsets([170, 130]))
    into = rows(torch, None, 300, [4, 2, 2], D, fill=False)
    check(torch, q, k, v, offsets([170, 130]), do=do, into=list(into))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_cache_past_4_gib(kind):
    """Blocks all over caches of 4.9 GB each, rows 2^26 bytes apart: the bits that small ones give."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    H, BT, D, NB = 16, 64, 128, 37000
    rng = np.random.default_rng(5)
    dt = torch.int8 if kind == "int8" else torch.float8_e4m3fn
    T = 200
    k, v = (torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2))
    buf = torch.empty((T - 1) * 2 ** 25 + 2 * H * D, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((T, 2 * H, D), (2 ** 25, D, 1))
    far[:, :H], far[:, H:] = k, v
    q = torch.from_numpy(rng.standard_normal((2, H, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    lens = ints(torch, [130, 70])
    results = []
    for nb, ids, kv in ((6, [3, 0, 5, 1, 2], (k, v)), (NB, [NB - 1, 17, 33001, 35000, 32768], (far[:, :H], far[:, H:]))):
        cache = [torch.zeros(nb, H, BT, D, dtype=torch.int8, device="cuda").view(dt) for _ in range(2)]
        scales = [torch.zeros(nb, H, device="cuda") for _ in range(2)]
        slots = np.concatenate([ids[i] * BT + np.arange(n) for i, n in enumerate((64, 64, 2, 64, 6))])
        note(f"far cache {kind} {nb} blocks")
        gdn.cache_append(*kv, ints(torch, slots), *cache, *scales)
        out, lse = gdn.attn_decode(q, *cache, *scales, ints(torch, [ids[:3], ids[3:] + [-1]]), lens)
        results.append([c[ids].view(torch.int8) for c in cache] + [s[ids] for s in scales] + [out, lse])
        torch.cuda.synchronize()
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert bool((results[0][4] != 0).any())
