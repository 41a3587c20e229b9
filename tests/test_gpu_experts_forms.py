"""Dispatch calls on both sides of the border between their two forms: pairs up
to 4096 and past them, few experts and many, wide rows (which side each is on,
tests/test_dispatch_form.py)."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import test_gpu_experts as base
from tests.gpu_util import to_dev

pytestmark = pytest.mark.gpu

SIZES = [  # T, k, E, kind, H
    (512, 8, 40, "own", 256), (64, 64, 70, "any", 128), (241, 17, 20, "any", 256),   # 4096 and 4097 pairs
    (4096, 1, 1, "one", 128), (4096, 1, 2, "any", 128), (4097, 1, 3, "any", 128), (900, 1, 1, "own", 1024),
    (3, 2, 4096, "any", 256), (64, 8, 4096, "own", 256), (512, 8, 4096, "any", 128), (1000, 1, 4096, "any", 256),
    (130, 2, 300, "any", 4224),
]


@pytest.mark.parametrize("T,k,E,kind,H", SIZES)
def test_copies(T, k, E, kind, H):
    base.test_dispatch_copies_rows_and_clears_padding(T, k, E, kind, H)


@pytest.mark.parametrize("kind_of", ["fp8", "e8m0", "int8"])
@pytest.mark.parametrize("T,k,E,kind,H", SIZES)
def test_codes(T, k, E, kind, H, kind_of):
    base.test_dispatch_quantizes_like_the_token_quantizers(T, k, E, kind, H, kind_of)


@pytest.mark.parametrize("T,k,E", [(512, 8, 256), (4096, 1, 2), (64, 8, 4096)])
def test_replayed_beside_eager_calls(T, k, E):
    """Either form from a captured graph, three times, with other calls between."""
    rng = np.random.default_rng(T)
    x, ids = base.bf16(rng.standard_normal((T, 384))), to_dev(base.choices(rng, T, k, E, "own"))
    calls = [lambda: dg.dg_moe_dispatch(x, ids, E), lambda: dg.dg_moe_dispatch_int8(x, ids, E)]
    for call in calls:
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        here = want[-3][want[-3] >= 0].long()
        for _ in range(3):
            for t in got:
                t.fill_(3)
            graph.replay()
            call()
            torch.cuda.synchronize()
            same = [torch.equal(a, b) for a, b in zip(got[-3:], want[-3:])]
            same += [torch.equal(a[here], b[here]) for a, b in zip(got[:-3], want[:-3])]
            assert all(same)
