"""The 16-bit paged cache at the edges of its types and tiles."""
import math

import pytest
import torch

import offloaded_kv_decode_gb300 as clo
import paged_ref as ref
from test_paged16_cache_gpu import rand, random_bounds, select

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- selection

@pytest.mark.parametrize("why", ["scale", "score", "block"])
@pytest.mark.parametrize("n_first,n_last,n_sel", [(1, 2, 8), (0, 1, 1), (3, 5, 8), (2, 0, 9)])
def test_first_and_last_blocks_come_before_those_without_a_score(n_first, n_last, n_sel, why):
    """More blocks of keys that are not finite, of scores beyond fp32 and of bad table entries
    than a request selects: its first and last ones, the one being filled among them, stay."""
    nb, Hkv, odd = 40, 2, range(4, 37)
    bounds = random_bounds(nb + 8, Hkv, 12)
    q = rand(2, 4, ref.D, dtype=torch.bfloat16, seed=13)
    table = torch.randperm(nb + 8, generator=torch.Generator().manual_seed(14))[:nb].to(torch.int32).repeat(2, 1)
    ids = table[0, 4:37].long()
    if why == "scale":
        bounds[ids] = ref.pack_records(torch.zeros(len(ids), Hkv, 2, ref.D, dtype=torch.int64), torch.full((len(ids), Hkv), math.inf))
    elif why == "score":  # the largest key where the query's code is positive, the smallest where it is negative
        codes = torch.stack([torch.full((ref.D,), 127), torch.full((ref.D,), -127)]).expand(len(ids), Hkv, 2, ref.D)
        bounds[ids] = ref.pack_records(codes, torch.full((len(ids), Hkv), 1e36))
    else:
        table[0, 4:37] = -1
    sel, err = select(q, bounds.cuda(), table.cuda(), [nb * 16 - 3, 20], n_sel, n_first, n_last)
    assert err == (clo.FLAG_BAD_INDEX if why == "block" else 0)
    keep = list(range(n_first)) + list(range(nb - n_last, nb))
    want = sorted(keep + list(odd)[:n_sel - len(keep)])
    for h in range(Hkv):
        assert sel[0, h].tolist() == want
        assert sel[1, h].tolist() == ([0, 1] + [-1] * n_sel)[:n_sel] if n_sel > 1 else [1]
