"""The workspaces of the paged attention and the eviction: the bytes the query
names are enough, none of them is read before the call has written it, and none
beside them is written.  A workspace of exactly that size lies in the middle of
a larger buffer; buffer and workspace hold a pattern before the first call, and
what the call before left before the others, whose sequences are shorter."""
import numpy as np
import pytest
import torch

import plain_serving as plain
import test_gpu_kv_evict as evict
import test_gpu_paged_attention as paged

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")
DEV = "cuda:0"
EDGE = 1 << 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_library()


class Guarded:
    def __init__(self, nbytes, fill):
        self.all = torch.full((nbytes + 2 * EDGE,), fill, dtype=torch.uint8, device=DEV)
        self.fill, self.ws = fill, self.all[EDGE:EDGE + nbytes]

    def check_edges(self):
        assert (self.all[:EDGE] == self.fill).all() and (self.all[EDGE + self.ws.numel():] == self.fill).all()


def _shorter(lens):
    return [n // 3 for n in lens], [min(n, i % 3) for i, n in enumerate(lens)]


@pytest.mark.parametrize("fill", [0xFF, 0x00])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,page", [
    ([100, 3], 4, 2, 16),                                # each sequence whole: no room for two units
    ([9001], 6, 1, 16),                                  # one sequence
    ([9001], 40, 2, 20),                                 # and three groups of query heads
    ([3000, 700, 1], 8, 2, 16),                          # cut one by one
    ([3000, 0, 513] + [700] * 57, 4, 2, 16),             # equal shares
    ([5000] + [40] * 99, 17, 1, 20),
    ([1500] + [9] * 699, 2, 1, 16),                      # found by a map
])
def test_paged_attention(lens, Hq, Hkv, page, weights, fill):
    D, dtype = 64, torch.bfloat16
    per = -(-max(lens) // page) + 1
    guard = Guarded(sv.sv_paged_attention_workspace(len(lens), Hq, Hkv, D, page, per, weights=weights), fill)
    for seed, ns in enumerate((lens,) + _shorter(lens)):
        case = paged.make(ns, Hq, Hkv, D, page, dtype, seed, extra_pages=per - max(1, -(-max(ns) // page)))
        assert case[2].shape[1] == per
        paged.check(*case, weights=weights, workspace=guard.ws)
        guard.check_edges()


@pytest.mark.parametrize("fill", [0xFF, 0x00])
@pytest.mark.parametrize("L,lens,Hkv,budget,sinks,recent", [
    (1, [1000, 77, 5], 2, 60, 3, 11),                    # a few CTAs choose the same
    (1, [12345], 2, 5000, 0, 0),                         # and each a part
    (1, [30, 12345], 2, 12000, 4, 11996),                # nothing to choose
    (2, [701, 260] + [90] * 18, 4, 60, 3, 11),           # small CTAs
])
def test_kv_evict(L, lens, Hkv, budget, sinks, recent, fill):
    guard = Guarded(sv.sv_kv_evict_workspace(L, len(lens), Hkv, budget), fill)
    for seed, ns in enumerate((lens,) + _shorter(lens)):
        kv, table, n, w = evict.make(L, ns, Hkv, 8, 16, seed=seed)
        want = plain.kv_evict(evict.as_bytes(kv), table.numpy(), n.numpy(), w.numpy(), budget, sinks, recent)
        k, ws, kept, new, st = evict.run(kv, table, n, w, budget, sinks, recent, workspace=guard.ws)
        assert not st.any() and np.array_equal(kept, want[2]) and np.array_equal(new, want[3])
        assert np.array_equal(evict.as_bytes(k), want[0]) and np.array_equal(ws, want[1])
        guard.check_edges()
