"""Edges of the calls over the paged latent cache that the plain cases do not
reach: many pieces of work in one share, calls cut between their launches, values
without a finite weight, the largest counts. References and tolerances are those
of test_cache_attention.py.
"""
import numpy as np
import pytest
import torch

from test_cache_attention import SM, check_rows, dsa, randn, sees  # noqa: F401
from test_gpu_parity import no_device_error

pytestmark = pytest.mark.gpu


def packed_cache(lens, seed):
    """A paged cache of many sequences, blocks in a random order (no Python loop)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = torch.as_tensor(lens)
    nb = (lens + 63) // 64
    nblk = int(nb.sum()) + 1
    used = torch.arange(max(1, int(nb.max()))).unsqueeze(0) < nb.unsqueeze(1)
    table = torch.full(used.shape, -1, dtype=torch.int32)
    table[used] = torch.randperm(nblk, generator=g, device="cuda").cpu().to(torch.int32)[:int(nb.sum())]
    return dict(kv_pool=randn(g, nblk, 64, 576), block_table=table.cuda(),
                seq_len=lens.to(torch.int32).cuda(), g=g)


def seq_rows(c, b):
    n = int(c["seq_len"][b])
    t = c["block_table"][b, : (n + 63) // 64].long()
    return c["kv_pool"][t].reshape(-1, 576)[:n].double().cpu().numpy()


# ------------------------------------------------- many pieces in one share

@pytest.mark.parametrize("B,nq,H,most,window", [(3000, 1, 128, 500, 0), (3000, 2, 65, 300, 100),
                                                (20000, 1, 16, 130, 0)])
def test_decode_of_thousands_of_short_sequences(dsa, B, nq, H, most, window):  # noqa: F811
    """Shares of forty sequences and more, found by a scan over all of them."""
    lens = [(37 * i + i // 7) % most for i in range(B)]
    c = packed_cache(lens, B + nq)
    q = randn(c["g"], B, nq, H, 576)
    cache = (c["kv_pool"], c["block_table"], c["seq_len"])
    if window:
        out, lse = dsa.window_mla_decode_paged(q, *cache, 3, window, SM)
    else:
        out, lse = dsa.split_mla_decode_paged(q, *cache, SM)
    no_device_error(dsa)
    for b in range(0, B, B // 75):
        n = lens[b]
        see = np.stack([sees(n - nq + j, n, 3, window) for j in range(nq)]).repeat(H, 0)
        check_rows(out[b].view(-1, 512), lse[b].view(-1), q[b].view(-1, 576), seq_rows(c, b), see)
