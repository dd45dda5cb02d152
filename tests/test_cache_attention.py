"""Attention over ranges of the latent cache (split decode, sliding window with
sinks), the totals of attention weight and eviction by them, on the GPU, against
plain 64-bit forms.

Tolerances, from the arithmetic (u = 2^-24, gamma_n = n u / (1 - n u)):
  * a logit is an fp32 sum of 576 products of bf16 values, which are exact in
    fp32, so it is off by dz <= sm_scale gamma_580 |q| max|k| (a few roundings of
    the scaling are in the 580); lse_atol() gives what that does to lse;
  * an output element sums p_s v_s with p_s = exp(z_s - lse) rounded once to bf16
    (2^-8) and off by dz, the exponential (2^-20) and the normaliser's error, and is
    rounded once to bf16 itself: |d| <= (2^-8 + 2 rel) sum_s p_s |v_s| + 2^-8 |out|;
  * a total adds p's that are off by dz, the exponential and the rounding of lse to
    fp32 in log2 units, in an fp32 sum of nq H terms.
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_parity import _gamma, lse_atol, no_device_error

pytestmark = pytest.mark.gpu

SM = 1.0 / 24.0
U = 2.0 ** -24
BF = 2.0 ** -8            # half a step of bf16, relative
BAD = -6                  # DSA_ERR_DEVICE_BOUNDS


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_long_02_b200 as d
    return d


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def make_cache(lens, seed=0, extra_blocks=3, max_blocks=None, poison=True):
    """A paged cache whose blocks lie in a random order; rows behind a sequence's
    last token, unused blocks and unused table entries hold what must not matter."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = [(n + 63) // 64 for n in lens]
    nblk = sum(nb) + extra_blocks
    mb = max_blocks or max(1, max(nb))
    perm = torch.randperm(nblk, generator=g, device="cuda").cpu().to(torch.int32)
    table = torch.full((len(lens), mb), 0x7F000000 if poison else -1, dtype=torch.int32)
    kv = randn(g, nblk, 64, 576)
    off = 0
    used = torch.zeros(nblk, 64, dtype=torch.bool)
    for b, n in enumerate(lens):
        table[b, : nb[b]] = perm[off: off + nb[b]]
        off += nb[b]
        for i in range(nb[b]):
            used[int(table[b, i]), : max(0, min(64, n - 64 * i))] = True
    if poison:
        junk = torch.tensor([math.nan, math.inf, -math.inf]).repeat(192).to(torch.bfloat16).cuda()
        kv[~used.cuda()] = junk
    return dict(kv_pool=kv, block_table=table.cuda(),
                seq_len=torch.tensor(lens, dtype=torch.int32).cuda(), g=g)


def rows_of(c, b, n):
    t = c["block_table"][b, : (n + 63) // 64].long().cpu()
    return c["kv_pool"].cpu()[t].reshape(-1, 576)[:n].double().numpy()


def plain(q, k, see):
    """q [r, 576], k [n, 576] float64, see [r, n] -> out, lse, sum p|v|, p."""
    z = np.where(see, SM * (q @ k.T), -np.inf) if k.shape[0] else np.full(see.shape, -np.inf)
    m = z.max(1, keepdims=True, initial=-np.inf)
    safe = np.where(np.isfinite(m), m, 0.0)
    e = np.where(see, np.exp(z - safe), 0.0)
    l = e.sum(1, keepdims=True)
    p = np.divide(e, l, out=np.zeros_like(e), where=l > 0)
    with np.errstate(divide="ignore"):
        lse = (safe + np.log(l))[:, 0]
    return p @ k[:, :512], lse, p @ np.abs(k[:, :512]), p


def sees(pos, n, sinks, window):
    s = np.arange(n)
    see = s <= pos
    if window:
        see &= (s > pos - window) | (s < sinks)
    return see


def check_rows(out, lse, q, k, see):
    """One sequence's rows: out [r, 512] and lse [r] of the library against plain()."""
    q = q.double().cpu().numpy()
    ref, ref_lse, absum, _ = plain(q, k, see)
    n = max(1, k.shape[0])
    kn = np.linalg.norm(k, axis=1).max(initial=0.0)
    tol_lse = lse_atol(q, float(kn), SM, ref_lse, n)
    got, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    none = ~see.any(1)
    assert (got[none] == 0).all() and (l[none] == -np.inf).all()
    assert np.isfinite(got).all()
    some = ~none
    off = np.abs(l[some] - ref_lse[some])
    assert (off <= tol_lse[some]).all(), off.max()
    rel = 2 * tol_lse[:, None] + 2.0 ** -18
    tol = (BF + rel) * absum + BF * np.abs(ref) * (1 + BF) + 1e-30
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.abs(got - ref)[bad][:4], tol[bad][:4], np.argwhere(bad)[:4])


def check_decode(dsa, lens, nq, H, sinks, window, seed=0, q_scale=1.0, **kw):
    c = make_cache(lens, seed, **kw)
    q = (randn(c["g"], len(lens), nq, H, 576) * q_scale).contiguous()
    if window:
        out, lse = dsa.window_mla_decode_paged(q, c["kv_pool"], c["block_table"], c["seq_len"],
                                               sinks, window, SM)
    else:
        out, lse = dsa.split_mla_decode_paged(q, c["kv_pool"], c["block_table"], c["seq_len"], SM)
    no_device_error(dsa)
    for b, n in enumerate(lens):
        k = rows_of(c, b, n)
        see = np.stack([sees(n - nq + j, n, sinks, window) for j in range(nq)]).repeat(H, 0)
        check_rows(out[b].view(-1, 512), lse[b].view(-1), q[b].view(-1, 576), k, see)
    return c, q, out, lse


# ------------------------------------------------------------- split decode

LENS = [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 513, 1000]


@pytest.mark.parametrize("nq,H", [(1, 128), (1, 1), (2, 128), (3, 8), (4, 16), (5, 31), (2, 65),
                                  (1, 64), (9, 127)])
def test_split_decode(dsa, nq, H):
    check_decode(dsa, LENS, nq, H, 0, 0, seed=nq * 131 + H)


@pytest.mark.parametrize("n", [1, 64, 129, 640, 4097, 20001])
def test_split_decode_one_sequence(dsa, n):
    check_decode(dsa, [n], 1, 128, 0, 0, seed=n)


def test_split_decode_many_short_sequences(dsa):
    check_decode(dsa, [(7 * i) % 131 for i in range(400)], 1, 4, 0, 0, seed=3)


def test_split_decode_very_uneven_lengths(dsa):
    check_decode(dsa, [30000, 1, 0, 70, 9000, 3, 64], 2, 16, 0, 0, seed=4)


def test_split_decode_table_wider_than_needed(dsa):
    check_decode(dsa, [100, 5, 700], 1, 8, 0, 0, seed=5, max_blocks=300)


@pytest.mark.parametrize("q_scale", [8.0, 60.0])
def test_split_decode_large_and_rising_logits(dsa, q_scale):
    """Peaked rows whose running maximum is replaced many times on the way."""
    lens = [2500, 333]
    c = make_cache(lens, 6)
    for b, n in enumerate(lens):
        t = c["block_table"][b].long()
        for i in range((n + 63) // 64):
            c["kv_pool"][t[i]] = (c["kv_pool"][t[i]].float() * (0.1 + 0.05 * i)).to(torch.bfloat16)
    q = (randn(c["g"], 2, 1, 128, 576) * q_scale).contiguous()
    out, lse = dsa.split_mla_decode_paged(q, c["kv_pool"], c["block_table"], c["seq_len"], SM)
    no_device_error(dsa)
    for b, n in enumerate(lens):
        check_rows(out[b].view(-1, 512), lse[b].view(-1), q[b].view(-1, 576), rows_of(c, b, n),
                   np.ones((128, n), bool))


def test_split_decode_matches_the_dense_kernel(dsa):
    c = make_cache([777, 2100], 7, poison=False)
    q = randn(c["g"], 2, 2, 128, 576)
    args = (q, c["kv_pool"], c["block_table"], c["seq_len"], SM)
    a, la = dsa.split_mla_decode_paged(*args)
    b, lb = dsa.dense_causal_mla_decode_paged(*args)
    no_device_error(dsa)
    assert (a.float() - b.float()).abs().max() <= 2e-2
    assert (la - lb).abs().max() <= 2e-3


def test_split_decode_bad_pages_and_lengths_are_recorded(dsa):
    lens = [300, 300, 300]
    c = make_cache(lens, 8, poison=False)
    q = randn(c["g"], 3, 1, 16, 576)
    args = (q, c["kv_pool"], c["block_table"], c["seq_len"])
    table = c["block_table"].cpu()
    for bad in (-1, c["kv_pool"].shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 2] = bad
        out, lse = dsa.split_mla_decode_paged(q, c["kv_pool"], t.cuda(), c["seq_len"], SM)
        assert dsa.get_device_error() == BAD
        for b in range(3):
            see = np.ones((16, 300), bool)
            if b == 1:
                see[:, 128:192] = False
            check_rows(out[b].view(-1, 512), lse[b].view(-1), q[b].view(-1, 576),
                       rows_of(c, b, 300), see)
    for n in (-5, 64 * table.shape[1] + 1, 2 ** 31 - 1):
        s = torch.tensor([300, n, 300], dtype=torch.int32).cuda()
        out, lse = dsa.split_mla_decode_paged(q, c["kv_pool"], c["block_table"], s, SM)
        assert dsa.get_device_error() == BAD
        k = rows_of(c, 1, 320) if n > 0 else np.zeros((0, 576))
        check_rows(out[1].view(-1, 512), lse[1].view(-1), q[1].view(-1, 576), k,
                   np.ones((16, k.shape[0]), bool))
    no_device_error(dsa)


def test_split_decode_past_32_bit_offsets(dsa):
    """Blocks whose rows lie past 2^31 elements (and 2^32 bytes) of the pool."""
    nblk = 60000
    kv = torch.empty(nblk, 64, 576, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    table = torch.tensor([[nblk - 1, 3, nblk - 2, 58255]], dtype=torch.int32)
    kv[table[0].long().cuda()] = randn(g, 4, 64, 576)
    q = randn(g, 1, 1, 32, 576)
    n = torch.tensor([250], dtype=torch.int32).cuda()
    c = dict(kv_pool=kv[table[0].long().cuda()], block_table=torch.arange(4).view(1, 4).cuda())
    for sinks, window in ((0, 0), (3, 70)):
        if window:
            out, lse = dsa.window_mla_decode_paged(q, kv, table.cuda(), n, sinks, window, SM)
        else:
            out, lse = dsa.split_mla_decode_paged(q, kv, table.cuda(), n, SM)
        no_device_error(dsa)
        check_rows(out.view(-1, 512), lse.view(-1), q.view(-1, 576), rows_of(c, 0, 250),
                   sees(249, 250, sinks, window)[None].repeat(32, 0))


def test_streams_graph_and_workspace(dsa):
    """The calls of a decode step captured into a graph and replayed on new data,
    and run on a stream of their own, with a caller's workspace."""
    lens = [500, 77, 1300]
    c = make_cache(lens, 10, poison=False)
    q = randn(c["g"], 3, 1, 128, 576)
    ws = torch.full((max(256, dsa.split_mla_decode_workspace_size(3, 1, c["block_table"].shape[1],
                                                                  128)),), 255,
                    dtype=torch.uint8, device="cuda")
    out = torch.empty(3, 1, 128, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 1, 128, device="cuda")
    mass = torch.zeros(3, c["block_table"].shape[1] * 64, device="cuda")
    cache = (c["kv_pool"], c["block_table"], c["seq_len"])

    def step(stream=None):
        dsa.split_mla_decode_paged(q, *cache, SM, out=out, lse=lse, workspace=ws, stream=stream)
        dsa.attention_mass_paged(q, *cache, lse, SM, mass, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    first = out.clone(), lse.clone(), mass.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    mass.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (out, lse, mass)):
        assert torch.equal(a, b)
    q.copy_(randn(c["g"], 3, 1, 128, 576))
    ws.fill_(77)
    graph.replay()
    no_device_error(dsa)
    for b, n in enumerate(lens):
        check_rows(out[b].view(-1, 512), lse[b].view(-1), q[b].view(-1, 576), rows_of(c, b, n),
                   np.ones((128, n), bool))


# ------------------------------------------------------- window with sinks

@pytest.mark.parametrize("sinks,window", [(0, 1), (0, 64), (4, 63), (64, 65), (65, 128), (200, 17),
                                          (1, 300), (5, 2 ** 31 - 1), (2 ** 31 - 1, 1)])
@pytest.mark.parametrize("nq,H", [(1, 128), (3, 8), (2, 65)])
def test_window_decode(dsa, sinks, window, nq, H):
    check_decode(dsa, [0, 1, 2, 64, 65, 130, 700, 1001], nq, H, sinks, window, seed=window % 1000)


def test_window_decode_reads_only_visible_blocks(dsa):
    """Blocks behind the window may have any table entry: nothing is recorded."""
    lens = [1000, 640]
    c = make_cache(lens, 11, poison=False)
    q = randn(c["g"], 2, 1, 32, 576)
    ref = dsa.window_mla_decode_paged(q, c["kv_pool"], c["block_table"], c["seq_len"], 3, 100, SM)
    t = c["block_table"].clone()
    t[0, 1:14] = -7
    t[1, 1:8] = 2 ** 31 - 1
    got = dsa.window_mla_decode_paged(q, c["kv_pool"], t, c["seq_len"], 3, 100, SM)
    no_device_error(dsa)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


@pytest.mark.parametrize("T,S,q_pos0,H,sinks,window", [
    (1, 1, 0, 128, 0, 1), (65, 65, 0, 128, 4, 32), (130, 400, 270, 8, 0, 129),
    (37, 37, 0, 5, 2, 1000), (200, 300, 100, 16, 70, 64), (33, 33, 0, 1, 1, 7),
    (3, 5000, 4997, 128, 4, 4096), (150, 150, 0, 64, 128, 1), (77, 100, 60, 128, 0, 20),
    (20, 50, 200, 16, 0, 100), (20, 50, 200, 16, 3, 100), (260, 260, 0, 127, 4, 130)])
def test_window_prefill(dsa, T, S, q_pos0, H, sinks, window):
    """Odd sizes, chunks at an offset, rows past the cache that see few keys or none."""
    g = torch.Generator(device="cuda").manual_seed(T + S)
    q, kv = randn(g, T, H, 576), randn(g, S, 576)
    last = q_pos0 + T - 1
    if last + 1 < S:
        kv[last + 1:] = math.nan                       # keys of later chunks
    out, lse = dsa.window_mla(q, kv, sinks, window, SM, q_pos0=q_pos0)
    no_device_error(dsa)
    n = min(S, last + 1)
    k = kv[:n].double().cpu().numpy()
    see = np.stack([sees(q_pos0 + t, n, sinks, window) for t in range(T)]).repeat(H, 0)
    check_rows(out.view(-1, 512), lse.view(-1), q.view(-1, 576), k, see)


@pytest.mark.parametrize("H", [8, 128])
def test_window_prefill_later_keys_do_not_matter(dsa, H):
    """A NaN or infinite row reaches only the queries that see it."""
    g = torch.Generator(device="cuda").manual_seed(12)
    T, w, s = 150, 40, 2
    q, kv = randn(g, T, H, 576), randn(g, T, 576)
    ref, ref_lse = dsa.window_mla(q, kv, s, w, SM)
    bad = kv.clone()
    bad[70] = math.nan
    bad[71, :512] = math.inf
    bad[71, 100:512:2] = -math.inf
    out, lse = dsa.window_mla(q, bad, s, w, SM)
    no_device_error(dsa)
    clean = [t for t in range(T) if not (70 <= t < 71 + w)]
    assert torch.equal(out[clean], ref[clean]) and torch.equal(lse[clean], ref_lse[clean])
    assert torch.isnan(out[70:70 + w].float()).all()


def test_window_prefill_equals_index_sets(dsa):
    """The same window through dsa_window_indices and the sparse MLA."""
    g = torch.Generator(device="cuda").manual_seed(13)
    T, H, w = 300, 128, 96
    q, kv = randn(g, T, H, 576), randn(g, T, 576)
    out, lse = dsa.window_mla(q, kv, 0, w, SM)
    idx = dsa.window_indices(T, T, w, w)
    ref, ref_lse = dsa.sparse_mla(q, kv, idx, SM)
    no_device_error(dsa)
    assert (out.float() - ref.float()).abs().max() <= 2e-2
    assert (lse - ref_lse).abs().max() <= 2e-3


def test_window_prefill_long_and_dense(dsa):
    """A window over the whole prefix is dense causal attention; many rows, few heads."""
    g = torch.Generator(device="cuda").manual_seed(14)
    T, H = 3001, 8
    q, kv = randn(g, T, H, 576), randn(g, T, 576)
    out, lse = dsa.window_mla(q, kv, 0, T, SM)
    no_device_error(dsa)
    k = kv.double().cpu().numpy()
    for t in (0, 1, 15, 16, 63, 64, 1000, 2047, 2999, 3000):
        see = sees(t, T, 0, 0)[None].repeat(H, 0)
        check_rows(out[t], lse[t], q[t], k, see)


# --------------------------------------------------------- attention totals

def check_mass(dsa, c, lens, q, lse, mass0, mass):
    B, nq, H = q.shape[:3]
    got = mass.double().cpu().numpy()
    old = mass0.double().cpu().numpy()
    for b, n in enumerate(lens):
        k = rows_of(c, b, n)
        qb = q[b].reshape(-1, 576).double().cpu().numpy()
        z = SM * (qb @ k.T)
        see = np.stack([sees(n - nq + j, n, 0, 0) for j in range(nq)]).repeat(H, 0)
        lb = lse[b].reshape(-1, 1).double().cpu().numpy()
        live = see & np.isfinite(lb)
        p = np.where(live, np.exp(np.where(live, z - lb, 0.0)), 0.0)
        w = p.sum(0)
        keep = np.where(np.arange(n) < n - nq, old[b, :n], 0.0)
        kn = np.linalg.norm(k, axis=1).max(initial=0.0)
        dz = SM * _gamma(580) * np.linalg.norm(qb, axis=1, keepdims=True) * kn
        rel = 2 * dz + 2.0 ** -20 + 4 * U * np.where(np.isfinite(lb), np.abs(lb), 0) \
            + 4 * U * np.abs(SM * np.linalg.norm(qb, axis=1, keepdims=True) * kn)
        tol = (p * rel).sum(0) + _gamma(nq * H + 8) * w + 2 * U * (keep + w)
        bad = np.abs(got[b, :n] - (keep + w)) > tol
        assert not bad.any(), (np.abs(got[b, :n] - keep - w)[bad][:4], tol[bad][:4],
                               np.argwhere(bad)[:4])
        assert np.array_equal(got[b, n:], old[b, n:], equal_nan=True)


@pytest.mark.parametrize("nq,H", [(1, 128), (1, 1), (2, 128), (3, 8), (4, 16), (2, 65), (5, 31)])
def test_attention_mass(dsa, nq, H):
    lens = LENS
    c = make_cache(lens, 20 + nq)
    q = randn(c["g"], len(lens), nq, H, 576)
    cache = (c["kv_pool"], c["block_table"], c["seq_len"])
    _, lse = dsa.split_mla_decode_paged(q, *cache, SM)
    ld = c["block_table"].shape[1] * 64 + 4
    mass0 = torch.rand(len(lens), ld, generator=c["g"], device="cuda")
    for b, n in enumerate(lens):
        mass0[b, max(0, n - nq):] = math.nan           # no totals yet
    mass = mass0.clone()
    dsa.attention_mass_paged(q, *cache, lse, SM, mass)
    no_device_error(dsa)
    check_mass(dsa, c, lens, q, lse, mass0, mass)
    again = mass0.clone()
    dsa.attention_mass_paged(q, *cache, lse, SM, again)
    assert torch.equal(again.view(torch.int32), mass.view(torch.int32))
    # every query gives a weight of one in all
    for b, n in enumerate(lens):
        if n > nq:
            total = (mass[b, :n] - torch.where(torch.arange(n, device="cuda") < n - nq,
                                               mass0[b, :n], 0.0)).double().sum().item()
            assert abs(total - nq * H) <= 1e-3 * nq * H


def test_attention_mass_long(dsa):
    lens = [9000, 40, 20500]
    c = make_cache(lens, 30)
    q = randn(c["g"], 3, 2, 128, 576)
    cache = (c["kv_pool"], c["block_table"], c["seq_len"])
    _, lse = dsa.split_mla_decode_paged(q, *cache, SM)
    mass0 = torch.rand(3, c["block_table"].shape[1] * 64, generator=c["g"], device="cuda")
    mass = mass0.clone()
    dsa.attention_mass_paged(q, *cache, lse, SM, mass)
    no_device_error(dsa)
    check_mass(dsa, c, lens, q, lse, mass0, mass)


def test_attention_mass_ignores_queries_without_a_normaliser(dsa):
    lens = [130]
    c = make_cache(lens, 31)
    q = randn(c["g"], 1, 2, 8, 576)
    cache = (c["kv_pool"], c["block_table"], c["seq_len"])
    _, lse = dsa.split_mla_decode_paged(q, *cache, SM)
    lse[0, 0] = -math.inf
    mass0 = torch.zeros(1, 192, device="cuda")
    mass = mass0.clone()
    dsa.attention_mass_paged(q, *cache, lse, SM, mass)
    no_device_error(dsa)
    check_mass(dsa, c, lens, q, lse, mass0, mass)


def test_attention_mass_bad_pages(dsa):
    lens = [300]
    c = make_cache(lens, 32, poison=False)
    q = randn(c["g"], 1, 1, 16, 576)
    cache = [c["kv_pool"], c["block_table"], c["seq_len"]]
    _, lse = dsa.split_mla_decode_paged(q, *cache, SM)
    mass0 = torch.rand(1, 320, generator=c["g"], device="cuda")
    ref, got = mass0.clone(), mass0.clone()
    dsa.attention_mass_paged(q, *cache, lse, SM, ref)
    cache[1] = cache[1].clone()
    cache[1][0, 1] = 2 ** 30
    dsa.attention_mass_paged(q, *cache, lse, SM, got)
    assert dsa.get_device_error() == BAD
    assert torch.equal(got[0, 64:128], mass0[0, 64:128])
    keep = torch.ones(320, dtype=torch.bool)
    keep[64:128] = False
    assert torch.equal(got[0, keep.cuda()], ref[0, keep.cuda()])


# ------------------------------------------------------------------ eviction

def kept_slots(mass, n, budget, sinks, recent):
    if n <= budget:
        return list(range(n))
    rank = lambda i: -math.inf if math.isnan(mass[i]) else mass[i]      # noqa: E731
    mid = sorted(range(sinks, n - recent), key=lambda i: (-rank(i), i))
    nan = [i for i in mid if math.isnan(mass[i])]
    mid = [i for i in mid if not math.isnan(mass[i])] + nan             # NaN below -inf
    return list(range(sinks)) + sorted(mid[: budget - sinks - recent]) + list(range(n - recent, n))


def check_evict(dsa, lens, budget, sinks, recent, values, seed=0, alias=False, index=True, ld_extra=0):
    c = make_cache(lens, seed, poison=False)
    g, nblk = c["g"], c["kv_pool"].shape[0]
    B, ld = len(lens), c["block_table"].shape[1] * 64 + ld_extra
    mass = values(g, B, ld)
    k8 = torch.randint(0, 256, (nblk, 64, 128), generator=g, device="cuda", dtype=torch.uint8)
    ks = torch.rand(nblk, 64, generator=g, device="cuda")
    before = [c["kv_pool"].view(torch.int16).clone(), k8.clone(), ks.clone()]
    m0, len0 = mass.clone(), c["seq_len"].clone()
    kw = dict(k8_pool=k8, k_scale_pool=ks) if index else {}
    if alias:
        kw.update(seq_len_out=c["seq_len"], mass_out=mass)
    else:
        kw.update(mass_out=torch.full((B, ld + 8), -3.0, device="cuda"))
    idx, new, mout = dsa.cache_evict_paged(c["kv_pool"], c["block_table"], c["seq_len"], mass,
                                           budget, sinks, recent, **kw)
    no_device_error(dsa)
    want = [t.clone() for t in before]
    want_mass = m0.clone() if alias else torch.full((B, ld + 8), -3.0, device="cuda")
    rows = m0.cpu().tolist()
    for b, n in enumerate(lens):
        kept = kept_slots(rows[b], n, budget, sinks, recent)
        assert int(new[b]) == len(kept)
        assert idx[b].tolist() == kept + [-1] * (budget - len(kept)), b
        src = torch.tensor(kept, dtype=torch.long, device="cuda")
        dst = torch.arange(len(kept), device="cuda")
        t = c["block_table"][b].long()
        at = lambda s: t[s // 64] * 64 + s % 64                          # noqa: E731
        for w, o in zip(want if index else want[:1], before):
            w.view(nblk * 64, -1)[at(dst)] = o.view(nblk * 64, -1)[at(src)]
        want_mass[b, : len(kept)] = m0[b, src]
    got = [c["kv_pool"].view(torch.int16), k8, ks]
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(mout.view(torch.int32), want_mass.view(torch.int32))
    if not alias:
        assert torch.equal(c["seq_len"], len0) and torch.equal(mass.view(torch.int32),
                                                               m0.view(torch.int32))
    return c


def heavy(g, B, ld):
    return torch.exp(2 * torch.randn(B, ld, generator=g, device="cuda"))


def tied(g, B, ld):
    return torch.randint(0, 3, (B, ld), generator=g, device="cuda").float()


def odd(g, B, ld):
    v = torch.randn(B, ld, generator=g, device="cuda")
    r = torch.rand(B, ld, generator=g, device="cuda")
    for lo, x in ((0.0, math.nan), (0.1, math.inf), (0.2, -math.inf), (0.3, 0.0), (0.4, -0.0),
                  (0.5, 1e-42)):
        v[(r >= lo) & (r < lo + 0.1)] = x
    return v


EV_LENS = [0, 1, 63, 64, 65, 200, 201, 500, 1003, 2500]


@pytest.mark.parametrize("values", [heavy, tied, odd])
@pytest.mark.parametrize("budget,sinks,recent", [(200, 4, 60), (1, 0, 0), (1, 1, 0), (1, 0, 1),
                                                 (64, 0, 64), (64, 64, 0), (130, 65, 65),
                                                 (999, 3, 0), (77, 0, 13), (4000, 4, 100)])
def test_evict(dsa, values, budget, sinks, recent):
    check_evict(dsa, EV_LENS, budget, sinks, recent, values, seed=budget)


@pytest.mark.parametrize("alias,index", [(True, True), (True, False), (False, False)])
def test_evict_in_place_and_without_the_indexer_cache(dsa, alias, index):
    check_evict(dsa, EV_LENS, 190, 2, 30, odd, seed=41, alias=alias, index=index, ld_extra=12)


def test_evict_long(dsa):
    check_evict(dsa, [70001, 128 * 64, 33000], 16001, 4, 1000, heavy, seed=42, alias=True)
    check_evict(dsa, [40000], 39999, 0, 0, heavy, seed=43, alias=True)       # one token goes
    check_evict(dsa, [40000], 39000, 39000, 0, heavy, seed=44)               # nothing moves
    check_evict(dsa, [40000], 39000, 0, 39000, heavy, seed=45)               # all move alike
    check_evict(dsa, [3000] * 150, 700, 4, 100, tied, seed=46)


@pytest.mark.parametrize("B", [2, 5, 12, 31, 33, 75, 160])
def test_evict_batches(dsa, B):
    """Each way rows are split: column slices, clusters of eight to one."""
    lens = [(37 + 211 * b) % 1900 for b in range(B)]
    check_evict(dsa, lens, 417, 5, 61, tied if B % 2 else heavy, seed=48 + B, alias=B > 30)


def test_evict_bad_pages_and_lengths(dsa):
    c = make_cache([500, 500], 47, poison=False)
    mass = torch.rand(2, 512, generator=c["g"], device="cuda")
    before = c["kv_pool"].clone()
    t = c["block_table"].clone()
    t[0, 5] = -1
    t[0, 6] = 2 ** 31 - 1
    idx, new, _ = dsa.cache_evict_paged(c["kv_pool"], t, c["seq_len"], mass, 100, 0, 100)
    assert dsa.get_device_error() == BAD
    src, dst = torch.arange(400, 500), torch.arange(100)
    ok = (src // 64 < 5) | (src // 64 > 6)
    for b in range(2):
        tb = c["block_table"][b].long().cpu()
        want = before.view(-1, 576).cpu().clone()
        s, d = (src[ok], dst[ok]) if b == 0 else (src, dst)
        got = c["kv_pool"].view(-1, 576).cpu()
        assert torch.equal(got[tb[d // 64] * 64 + d % 64], want[tb[s // 64] * 64 + s % 64])
    s = torch.tensor([9999, -3], dtype=torch.int32).cuda()
    idx, new, _ = dsa.cache_evict_paged(c["kv_pool"], c["block_table"], s, mass, 600, 0, 0)
    assert dsa.get_device_error() == BAD
    assert new.tolist() == [512, 0] and idx[0, :512].tolist() == list(range(512))
    assert (idx[0, 512:] == -1).all() and (idx[1] == -1).all()
    no_device_error(dsa)


# ------------------------------------------------------------- all together

def test_decode_totals_eviction_decode(dsa):
    """Decode steps whose totals decide an eviction, then a decode over what is left:
    attention over exactly the kept tokens."""
    lens = [700, 150, 1200]
    c = make_cache(lens, 50, poison=False)
    cache = (c["kv_pool"], c["block_table"], c["seq_len"])
    mass = torch.full((3, c["block_table"].shape[1] * 64), math.nan, device="cuda")
    q_all = randn(c["g"], 3, 40, 16, 576)               # 40 tokens at once start every total ...
    _, lse = dsa.split_mla_decode_paged(q_all, *cache, SM)
    mass[:, :] = 0.0
    dsa.attention_mass_paged(q_all, *cache, lse, SM, mass)
    q = randn(c["g"], 3, 1, 16, 576)                    # ... and one more token adds to them
    _, lse = dsa.split_mla_decode_paged(q, *cache, SM)
    dsa.attention_mass_paged(q, *cache, lse, SM, mass)
    no_device_error(dsa)
    rows = [rows_of(c, b, n) for b, n in enumerate(lens)]
    totals = mass.cpu().tolist()
    idx, new, mass = dsa.cache_evict_paged(*cache, mass, 300, 4, 64, seq_len_out=c["seq_len"],
                                           mass_out=mass)
    q2 = randn(c["g"], 3, 1, 16, 576)
    out, lse2 = dsa.split_mla_decode_paged(q2, *cache, SM)
    wout, wlse = dsa.window_mla_decode_paged(q2, *cache, 4, 100, SM)
    no_device_error(dsa)
    for b, n in enumerate(lens):
        kept = kept_slots(totals[b], n, 300, 4, 64)
        k = rows[b][kept]
        m = len(kept)
        assert int(c["seq_len"][b]) == m
        check_rows(out[b].view(-1, 512), lse2[b].view(-1), q2[b].view(-1, 576), k,
                   np.ones((16, m), bool))
        check_rows(wout[b].view(-1, 512), wlse[b].view(-1), q2[b].view(-1, 576), k,
                   sees(m - 1, m, 4, 100)[None].repeat(16, 0))


# ------------------------------------------------ streams, faults, workspaces

def test_window_decode_hidden_keys_do_not_matter(dsa):
    """Keys no query sees hold NaN and infinities, inside blocks that are read."""
    for nq, H, sinks, window in ((1, 128, 3, 70), (2, 128, 70, 5), (3, 8, 0, 130), (4, 31, 1, 1)):
        lens = [1000, 777, 130, 65, 3]
        c = make_cache(lens, 60 + nq)
        for b, n in enumerate(lens):
            see = np.stack([sees(n - nq + j, n, sinks, window) for j in range(nq)]).any(0)
            for s in np.nonzero(~see)[0]:
                row = c["kv_pool"][int(c["block_table"][b, s // 64]), s % 64]
                row[:] = (math.nan, math.inf, -math.inf)[s % 3]
        q = randn(c["g"], len(lens), nq, H, 576)
        out, lse = dsa.window_mla_decode_paged(q, c["kv_pool"], c["block_table"], c["seq_len"],
                                               sinks, window, SM)
        no_device_error(dsa)
        for b, n in enumerate(lens):
            k = rows_of(c, b, n)
            see = np.stack([sees(n - nq + j, n, sinks, window) for j in range(nq)])
            k[~see.any(0)] = 0.0
            check_rows(out[b].view(-1, 512), lse[b].view(-1), q[b].view(-1, 576), k,
                       see.repeat(H, 0))


def test_a_timeout_is_reported_and_nothing_runs_until_it_is_read(dsa):
    """The bounded waits run out (a barrier that nothing arrives at), the call comes
    back, later kernels leave everything as it is, and the next clean call is right."""
    lens = [500, 90]
    c = make_cache(lens, 70, poison=False)
    q = randn(c["g"], 2, 1, 128, 576)
    cache = (c["kv_pool"], c["block_table"], c["seq_len"])
    mass = torch.rand(2, 512, generator=c["g"], device="cuda")
    lse0 = torch.zeros(2, 1, 128, device="cuda")
    kv0, mass0 = c["kv_pool"].clone(), mass.clone()
    no_device_error(dsa)
    dsa.debug_stall(dsa.DEBUG_STALL_MLA)
    try:
        dsa.split_mla_decode_paged(q, *cache, SM)
        dsa.attention_mass_paged(q, *cache, lse0, SM, mass)
        idx = torch.full((2, 64), -9, dtype=torch.int32, device="cuda")
        lens_out = torch.full((2,), -9, dtype=torch.int32, device="cuda")
        dsa.cache_evict_paged(*cache, mass, 64, 0, 8, idx=idx, seq_len_out=lens_out, mass_out=mass)
        st = dsa.get_device_error()
    finally:
        dsa.debug_stall(0)
    assert st == -5, dsa.STATUS.get(st, st)
    assert torch.equal(mass, mass0) and torch.equal(c["kv_pool"], kv0)
    assert (idx == -9).all() and (lens_out == -9).all()
    out, lse = dsa.split_mla_decode_paged(q, *cache, SM)
    no_device_error(dsa)
    for b, n in enumerate(lens):
        check_rows(out[b].view(-1, 512), lse[b].view(-1), q[b].view(-1, 576), rows_of(c, b, n),
                   np.ones((128, n), bool))


def test_two_calls_at_once(dsa):
    """Different problems on two streams, each with a workspace of its own, many times
    over; and a stream given without a workspace or outputs."""
    g = torch.Generator(device="cuda").manual_seed(80)
    c = make_cache([3000, 17, 900], 81, poison=False)
    qa = randn(g, 3, 2, 128, 576)
    qb, kvb = randn(g, 500, 16, 576), randn(g, 500, 576)
    cache = (c["kv_pool"], c["block_table"], c["seq_len"])
    ra = dsa.split_mla_decode_paged(qa, *cache, SM)
    rb = dsa.window_mla(qb, kvb, 4, 100, SM)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append((dsa.split_mla_decode_paged(qa, *cache, SM, stream=s1),
                    dsa.window_mla(qb, kvb, 4, 100, SM, stream=s2)))
    torch.cuda.synchronize()
    no_device_error(dsa)
    for a, b in got:
        assert torch.equal(a[0], ra[0]) and torch.equal(a[1], ra[1])
        assert torch.equal(b[0], rb[0]) and torch.equal(b[1], rb[1])


def test_workspace_ends_where_it_says(dsa):
    for B, nq, H, lens in ((1, 1, 128, [5000]), (3, 2, 31, [700, 3, 1500])):
        c = make_cache(lens, 90 + B, poison=False)
        q = randn(c["g"], B, nq, H, 576)
        mb = c["block_table"].shape[1]
        need = dsa.split_mla_decode_workspace_size(B, nq, mb, H)
        buf = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
        cache = (c["kv_pool"], c["block_table"], c["seq_len"])
        a = dsa.split_mla_decode_paged(q, *cache, SM, workspace=buf[:need])
        assert (buf[need:] == 171).all()
        b = dsa.split_mla_decode_paged(q, *cache, SM)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        with pytest.raises(dsa.DSAError):
            dsa.split_mla_decode_paged(q, *cache, SM, workspace=buf[:need - 1])
    no_device_error(dsa)


def test_counts_past_32_bits_are_refused(dsa):
    q = torch.zeros(2, 4, 576, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(2, 64, 576, dtype=torch.bfloat16, device="cuda")
    bt = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    sl = torch.ones(1, dtype=torch.int32, device="cuda")
    mass = torch.zeros(1, 64, device="cuda")
    big = 2**32 + 1
    for call in (lambda: dsa.window_mla(q, pool[0], 1, big, SM),
                 lambda: dsa.window_mla(q, pool[0], big, 8, SM),
                 lambda: dsa.window_mla(q, pool[0], 1, 8, SM, q_pos0=big),
                 lambda: dsa.window_mla_decode_paged(q[:1, None], pool, bt, sl, 1, big, SM),
                 lambda: dsa.window_mla_decode_paged(q[:1, None], pool, bt, sl, big, 1, SM),
                 lambda: dsa.cache_evict_paged(pool, bt, sl, mass, big, 0, 0),
                 lambda: dsa.cache_evict_paged(pool, bt, sl, mass, 8, big, 0),
                 lambda: dsa.cache_evict_paged(pool, bt, sl, mass, 8, 0, big)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_outputs_on_any_16_byte_boundary(dsa):
    """Outputs and inputs that start 16 bytes into an allocation."""
    g = torch.Generator(device="cuda").manual_seed(95)

    def off(*shape):
        n = math.prod(shape)
        return torch.zeros(n + 8, dtype=torch.bfloat16, device="cuda")[8:].view(*shape)

    T, H, S = 200, 128, 200
    q, kv, out = off(T, H, 576), off(S, 576), off(T, H, 512)
    q.copy_(randn(g, T, H, 576))
    kv.copy_(randn(g, S, 576))
    ref, ref_lse = dsa.window_mla(q.clone(), kv.clone(), 1, 90, SM)
    got, lse = dsa.window_mla(q, kv, 1, 90, SM, out=out)
    no_device_error(dsa)
    assert got.data_ptr() == out.data_ptr() and out.data_ptr() % 32 == 16
    assert torch.equal(got, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("T,H,window", [(300, 128, 200), (75, 128, 2000), (149, 128, 65),
                                        (1200, 16, 500), (20000, 1, 9)])
def test_window_prefill_shares(dsa, T, H, window):
    """Row tiles cut over several shares and whole ones, one share holding many."""
    g = torch.Generator(device="cuda").manual_seed(T)
    p0 = 3000 if T < 100 else 0
    q, kv = randn(g, T, H, 576), randn(g, p0 + T, 576)
    out, lse = dsa.window_mla(q, kv, 2, window, SM, q_pos0=p0)
    no_device_error(dsa)
    k = kv.double().cpu().numpy()
    for t in sorted({0, 1, T // 3, T // 2, T - 2, T - 1}):
        see = sees(p0 + t, p0 + T, 2, window)
        cols = np.nonzero(see)[0]
        check_rows(out[t], lse[t], q[t], k[cols], np.ones((H, len(cols)), bool))


def test_nothing_to_do(dsa):
    """Empty batches and prompts, and batches of empty sequences."""
    kv = torch.zeros(2, 64, 576, dtype=torch.bfloat16, device="cuda")
    q0 = torch.zeros(0, 1, 8, 576, dtype=torch.bfloat16, device="cuda")
    t0 = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    l0 = torch.zeros(0, dtype=torch.int32, device="cuda")
    out, lse = dsa.split_mla_decode_paged(q0, kv, t0, l0, SM)
    assert out.shape == (0, 1, 8, 512) and lse.shape == (0, 1, 8)
    dsa.window_mla(q0[:, 0], kv[0], 0, 4, SM)
    dsa.attention_mass_paged(q0, kv, t0, l0, lse, SM, torch.zeros(0, 128, device="cuda"))
    dsa.cache_evict_paged(kv, t0, l0, torch.zeros(0, 128, device="cuda"), 5, 0, 0)
    q = torch.ones(90, 2, 8, 576, dtype=torch.bfloat16, device="cuda")
    t = torch.full((90, 2), -1, dtype=torch.int32, device="cuda")
    n = torch.zeros(90, dtype=torch.int32, device="cuda")
    out, lse = dsa.split_mla_decode_paged(q, kv, t, n, SM)
    assert (out == 0).all() and (lse == -math.inf).all()
    mass = torch.full((90, 128), 3.0, device="cuda")
    dsa.attention_mass_paged(q, kv, t, n, lse, SM, mass)
    idx, new, _ = dsa.cache_evict_paged(kv, t, n, mass, 5, 1, 1)
    assert (mass == 3).all() and (idx == -1).all() and (new == 0).all()
    no_device_error(dsa)
