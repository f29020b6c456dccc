"""How far sv_prefix_attention is from 64 bits as a whole: the relative 2-norm of
its outputs, which an element's bound (a sum of the worst of every key) cannot hold
behind long prefixes.

With v rounded to the type, a number is off by up to half a step; of the reference
itself rounding leaves `own`.  What comes before it, in 32 bits: a score's D products
and its scale, roundings of independent sign, sqrt(D) 2^-24 of some |q| |k| scale <= 8
here; the base-2 exponential 2^-22; a sum of n weights sqrt(n) 2^-24.  With up to 128
query rows of a KV head a weight keeps two parts of the type, half^2 of itself.  All of
them independent from key to key, so relative to `spread` as to a weight; near the
middle between two numbers they count twice.  With more rows a weight is rounded once:
half / sqrt(3) of it in the mean square, of weights times values `spread`."""
import math

import pytest
import torch

import test_gpu_prefix_attention as prefix

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_library()


def norms(out, q, kv, pt, pl, t, n):
    """Relative 2-norms: of the output's error, of rounding the reference, of the
    weighted values taken apart (`spread`)."""
    B, Hq, D = q.shape
    page, Hkv = kv.shape[2], kv.shape[3]
    W = B // len(pl)
    err = own = spread = size = 0.0
    for b in range(B):
        rows = []
        for table, length in ((pt[b // W], int(pl[b // W])), (t[b], int(n[b]))):
            j = torch.arange(length)
            rows.append(kv[:, table[j // page].long(), j % page])
        k, v = torch.cat(rows, 1).to(DEV).double()
        x = torch.einsum("hgd,jhd->hgj", q[b].to(DEV).double().view(Hkv, -1, D), k) / math.sqrt(D)
        w = torch.softmax(x, -1)
        want = torch.einsum("hgj,jhd->hgd", w, v).reshape(Hq, D)
        err += float((out[b].double() - want).square().sum())
        own += float((want.to(q.dtype).double() - want).square().sum())
        spread += float(torch.einsum("hgj,jhd->hgd", w.square(), v.square()).sum())
        size += float(want.square().sum())
    return tuple(math.sqrt(s / size) for s in (err, own, spread))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("plens,lens,Hq,Hkv,page", [
    ([300], [0, 20, 3], 8, 2, 16),
    ([20011], [17, 0, 300, 1], 16, 2, 64),              # over the whole card
    ([700, 129], [5] * 32, 16, 2, 20),                  # 128 rows, tiles of whole pages
    ([900], [30] * 4, 32, 2, 1),                        # 64 rows, copied slot by slot
    ([1500], [9] * 16, 18, 2, 33),                      # 144 rows: two tiles, one ragged
    ([20011], [40] * 24, 32, 2, 64),                    # 384 rows: three tiles
])
def test_relative_error(plens, lens, Hq, Hkv, page, D, dtype):
    q, kv, pt, pl, t, n = prefix.make(plens, lens, Hq, Hkv, D, page, dtype, seed=D, sigma=0.5)
    kv = kv.nan_to_num(0.0)                             # (0 in slots that are not visible)
    out = sv.prefix_attention(*(x.to(DEV) for x in (q, kv, pt, pl, t, n)))
    torch.cuda.synchronize()
    err, own, spread = norms(out, q, kv, pt, pl, t, n)
    half = torch.finfo(dtype).eps / 2
    slots = max(plens) + max(lens)
    before = half ** 2 + 2.0 ** -24 * (8 * math.sqrt(D) + 4 + math.sqrt(slots))
    one_part = len(lens) // len(plens) * Hq // Hkv > 128
    bound = math.hypot(own, half / math.sqrt(3) * spread if one_part else 0.0) + 2 * before * max(1.0, spread)
    assert err <= bound, (err, own, spread, bound)
