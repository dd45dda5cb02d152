"""Edges of the calls over the paged latent cache that the plain cases do not
reach: many pieces of work in one share, calls cut between their launches, values
without a finite weight, the largest counts. References and tolerances are those
of test_cache_attention.py.
"""
import numpy as np
import pytest
import torch

from test_cache_attention import (SM, check_evict, check_rows, dsa, odd, plain, randn,  # noqa: F401
                                  sees)
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
    perm = torch.randperm(nblk, generator=g, device="cuda").cpu().to(torch.int32)
    table[used] = perm[:int(nb.sum())]
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


@pytest.mark.parametrize("T,H,sinks,window,ragged", [
    (2500, 128, 4, 70, 0),        # equal shares or whole row tiles: 34 of them a cluster
    (2501, 65, 0, 130, 300),      # the same, the first rows with less and less to see
    (16500, 65, 3, 40, 0),        # too many row tiles to scan: whole ones, no workspace
    (16385, 128, 0, 9, 0)])
def test_window_prefill_of_thousands_of_row_tiles(dsa, T, H, sinks, window, ragged):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(T + H)
    S = T - ragged                                      # rows past the cache see less
    q, kv = randn(g, T, H, 576), randn(g, S, 576)
    assert (dsa.window_mla_workspace_size(T, S, H, 0, sinks, window) == 0) == (T > 16384)
    out, lse = dsa.window_mla(q, kv, sinks, window, SM)
    no_device_error(dsa)
    k = kv.double().cpu().numpy()
    # 16 rows of every 90 and the last: pieces of all places and turns of the shares' rings
    for t0 in [*range(0, T - 16, 90), T - 16]:
        lo = max(0, min(S, t0 - window + 1))
        hi = min(S, t0 + 16)
        cols = np.unique(np.concatenate([np.arange(min(sinks, S)), np.arange(lo, hi)]))
        see = np.stack([sees(t, S, sinks, window)[cols] for t in range(t0, t0 + 16)]).repeat(H, 0)
        check_rows(out[t0:t0 + 16].reshape(-1, 512), lse[t0:t0 + 16].reshape(-1),
                   q[t0:t0 + 16].reshape(-1, 576), k[cols], see)


# ------------------------------------- a call cut between its two launches

class Halves:
    """A captured call of two launches that can be replayed one launch at a time."""

    def __init__(self, call):
        from cuda.bindings import driver
        self.drv = driver
        call()                                          # what is set up once, outside the capture
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(self.graph):
            call()
        raw = driver.CUgraph(self.graph.raw_cuda_graph())
        n = self._do(driver.cuGraphGetNodes(raw))[1]
        nodes = self._do(driver.cuGraphGetNodes(raw, n))[0]
        root = self._do(driver.cuGraphGetRootNodes(raw, 1))[0][0]
        assert n == 2
        self.nodes = sorted(nodes, key=lambda k: int(k) != int(root))
        self.exe = self._do(driver.cuGraphInstantiate(raw, 0))[0]

    def _do(self, result):
        assert result[0] == self.drv.CUresult.CUDA_SUCCESS, result[0]
        return result[1:]

    def run(self, half):
        for i, node in enumerate(self.nodes):
            self._do(self.drv.cuGraphNodeSetEnabled(self.exe, node, int(i == half)))
        self._do(self.drv.cuGraphLaunch(self.exe, torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()

    def close(self):
        self._do(self.drv.cuGraphExecDestroy(self.exe))
        self.graph.reset()


def leave_a_timeout(dsa):  # noqa: F811
    """A pending timeout: a bounded wait (1 s) that nothing arrives at runs out."""
    kv = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 1, 8, 576, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    dsa.debug_stall(dsa.DEBUG_STALL_MLA)
    try:
        dsa.split_mla_decode_paged(q, kv, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), one,
                                   SM)
        torch.cuda.synchronize()
    finally:
        dsa.debug_stall(0)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B", [1, 40])
def test_an_eviction_is_done_as_a_whole_or_not_at_all(dsa, B, in_place):  # noqa: F811
    """Between the selection and the move another stream's caller clears the timeout
    that the selection met, or another stream's kernel records one."""
    lens, budget = [900 - 7 * (b % 9) for b in range(B)], 300
    c = packed_cache(lens, 60 + B)
    mass = torch.rand(B, c["block_table"].shape[1] * 64, generator=c["g"], device="cuda")
    idx = torch.empty(B, budget, dtype=torch.int32, device="cuda")
    new = c["seq_len"] if in_place else torch.empty_like(c["seq_len"])
    mout = mass if in_place else torch.empty_like(mass)
    state = [c["kv_pool"], c["seq_len"], mass, idx, new, mout]

    def call():
        dsa.cache_evict_paged(c["kv_pool"], c["block_table"], c["seq_len"], mass, budget, 4, 50,
                              idx=idx, seq_len_out=new, mass_out=mout)

    idx.zero_(), new.copy_(c["seq_len"]), mout.copy_(mass)
    start = [t.clone() for t in state]
    halves = Halves(call)
    done = [t.clone() for t in state]                   # what one whole call makes of it
    for t, s in zip(state, start):
        t.copy_(s)
    # outputs that look like those of an earlier call
    idx.copy_(torch.arange(budget, device="cuda").expand(B, -1) * 2)
    if not in_place:
        new.fill_(budget)
    held = [t.clone() for t in state]
    no_device_error(dsa)
    leave_a_timeout(dsa)
    halves.run(0)
    assert dsa.get_device_error() == -5                 # read, and cleared, by somebody else
    halves.run(1)
    no_device_error(dsa)
    for t, h in zip(state, held):
        assert torch.equal(t, h)
    halves.run(0)
    leave_a_timeout(dsa)
    halves.run(1)
    assert dsa.get_device_error() == -5
    for t, d in zip(state, done):
        assert torch.equal(t, d)
    halves.close()


# ----------------------------------------------------------- largest counts

def test_evict_with_a_budget_of_no_limit(dsa):  # noqa: F811
    """The largest budget the interface takes: all is kept, and its row of slots ends
    where it should."""
    c = packed_cache([700], 90)
    mass = torch.rand(1, 704, generator=c["g"], device="cuda")
    kv, budget = c["kv_pool"].clone(), 2 ** 31 - 1
    buf = torch.zeros(budget + 65, dtype=torch.int32, device="cuda")
    idx = buf[32:32 + budget].view(1, budget)
    _, new, mout = dsa.cache_evict_paged(c["kv_pool"], c["block_table"], c["seq_len"], mass, budget,
                                         4, 100, idx=idx)
    no_device_error(dsa)
    assert new.tolist() == [700] and torch.equal(c["kv_pool"], kv)
    assert torch.equal(mout[:, :700], mass[:, :700])
    assert idx[0, :700].tolist() == list(range(700))
    for part in idx[0, 700:].split(1 << 28):
        assert int(part.max()) == -1 and int(part.min()) == -1
    assert not buf[:32].any() and not buf[32 + budget:].any()


def test_a_split_call_is_joined_whatever_the_error_word_says(dsa):  # noqa: F811
    """Between the shares and their join another stream's kernel records a timeout, or
    its caller clears the one that the shares met."""
    lens = [9000, 40, 3001]
    c = packed_cache(lens, 95)
    q = randn(c["g"], 3, 1, 128, 576)
    out = torch.empty(3, 1, 128, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 1, 128, device="cuda")
    ws = torch.full((dsa.split_mla_decode_workspace_size(3, 1, c["block_table"].shape[1], 128),),
                    255, dtype=torch.uint8, device="cuda")
    halves = Halves(lambda: dsa.split_mla_decode_paged(q, c["kv_pool"], c["block_table"],
                                                       c["seq_len"], SM, out=out, lse=lse,
                                                       workspace=ws))
    ref = out.clone(), lse.clone()
    no_device_error(dsa)
    out.fill_(7), lse.fill_(7), ws.fill_(255)
    halves.run(0)
    leave_a_timeout(dsa)
    halves.run(1)
    assert dsa.get_device_error() == -5
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    out.fill_(7), lse.fill_(7), ws.fill_(255)
    leave_a_timeout(dsa)
    halves.run(0)
    assert dsa.get_device_error() == -5
    halves.run(1)
    no_device_error(dsa)
    assert (out == 7).all() and (lse == 7).all()
    halves.close()


# ------------------------------------------- infinite values that rows do see

def check_infinite_rows(out, lse, q, k, see):
    """Rows over keys of which some are infinite in single dims. A logit of +inf or NaN
    makes the row NaN; one of -inf has no weight, and 0 times the key's infinite value
    makes that dim of the row NaN, and no other."""
    with np.errstate(invalid="ignore"):
        z = q.double().cpu().numpy() @ k.T
    whole = (see & ~(z < np.inf)).any(1)
    part = ~whole
    assert torch.isnan(out[torch.from_numpy(whole).to(out.device)].float()).all()
    assert not torch.isfinite(lse[torch.from_numpy(whole).to(out.device)]).any()
    inf = np.isinf(k)
    dims = (see.astype(np.float32) @ inf[:, :512].astype(np.float32) > 0)[part]
    rows = torch.from_numpy(np.nonzero(part)[0]).to(out.device)
    got = out[rows].clone()
    want = torch.from_numpy(dims).to(out.device)
    assert torch.equal(torch.isnan(got.float()), want)
    finite = see[part] & np.isfinite(z[part])
    k0 = np.where(inf, 0.0, k)
    ref = plain(q[rows].double().cpu().numpy(), k0, finite)[0]
    got[want] = torch.from_numpy(ref).to(out.device)[want].to(got.dtype)
    check_rows(got, lse[rows], q[rows], k0, finite)
    return int(whole.sum()), int(dims.any(1).sum())


@pytest.mark.parametrize("H,sinks,window", [(8, 0, 40), (128, 3, 40), (65, 70, 200), (1, 2, 1000)])
def test_window_prefill_over_single_infinite_values(dsa, H, sinks, window):  # noqa: F811
    """Keys seen by all rows of a tile, by some, and by none, in rows of whole units and
    of cut ones; in dims of both halves, the rope dims, several dims and several keys."""
    g = torch.Generator(device="cuda").manual_seed(70 + H)
    T = 190
    q, kv = randn(g, T, H, 576), randn(g, T, 576)
    # queries on one side of the infinities, so that a third of them meets -inf alone
    spots = [(0, 5, 1), (2, 300, -1), (63, 511, 1), (64, 0, 1), (64, 256, 1), (100, 255, -1),
             (101, 570, 1), (130, 17, 1), (131, 17, -1), (189, 448, 1)]
    for s, d, sign in spots:
        kv[s, d] = sign * float("inf")
        side = (torch.arange(T, device="cuda") % 3 == 0).view(T, 1)
        q[:, :, d] = torch.where(side, q[:, :, d], q[:, :, d].abs() * -sign)
    q[:, :, 17] = randn(g, T, H)
    out, lse = dsa.window_mla(q, kv, sinks, window, SM)
    no_device_error(dsa)
    k = kv.double().cpu().numpy()
    see = np.stack([sees(t, T, sinks, window) for t in range(T)]).repeat(H, 0)
    whole, some = check_infinite_rows(out.view(-1, 512), lse.view(-1), q.view(-1, 576), k, see)
    assert whole > T * H // 8 and some > T * H // 8


@pytest.mark.parametrize("nq,H,lens", [(3, 8, [700, 65]), (2, 128, [9000, 130]), (4, 32, [20001])])
def test_split_decode_over_single_infinite_values(dsa, nq, H, lens):  # noqa: F811
    """The same in a paged cache, in sequences whose parts are joined."""
    c = packed_cache(lens, 80 + nq)
    q = randn(c["g"], len(lens), nq, H, 576)
    for b, n in enumerate(lens):
        for s, d in ((n - 1, 3), (n - 2, 400), (n - nq, 77), (n // 2, 130), (5, 511)):
            c["kv_pool"][int(c["block_table"][b, s // 64]), s % 64, d] = float("inf")
            q[b, :, ::2, d] = -q[b, :, ::2, d].abs()
    out, lse = dsa.split_mla_decode_paged(q, c["kv_pool"], c["block_table"], c["seq_len"], SM)
    no_device_error(dsa)
    for b, n in enumerate(lens):
        see = np.stack([sees(n - nq + j, n, 0, 0) for j in range(nq)]).repeat(H, 0)
        whole, some = check_infinite_rows(out[b].view(-1, 512), lse[b].view(-1),
                                          q[b].view(-1, 576), seq_rows(c, b), see)
        assert whole > 0 and some >= nq * H // 2


def test_row_tiles_that_take_over_a_second(dsa):  # noqa: F811
    """75 sequences of a hundred million tokens that share four blocks, so that roles
    wait for the end of a row tile longer than the limit of a wait that makes no
    progress. Queries of 0 see all keys alike: a weight's sum is exact (multiples of 64
    below 2^30). A value's sum is one of n / 16 steps of the tensor core, which holds it
    in fp32 and may cut where it does not round: off by 2^-23 a step, 0.75 in all."""
    blocks = 100_000_000 // 64 // 4 * 4
    B, n = 75, blocks * 64
    v = 2.0 ** (torch.arange(576, device="cuda") % 3)
    kv = v.to(torch.bfloat16).expand(4, 64, 576).contiguous()
    table = torch.arange(4, dtype=torch.int32, device="cuda").repeat(B, blocks // 4)
    q = torch.zeros(B, 1, 1, 576, dtype=torch.bfloat16, device="cuda")
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    no_device_error(dsa)
    out, lse = dsa.split_mla_decode_paged(q, kv, table, lens, SM)
    no_device_error(dsa)
    assert ((out.float() - v[:512]).abs() <= n / 16 * 2.0 ** -23 * v[:512]).all()
    assert (lse.double() - np.log(n)).abs().max() <= 8 * 2.0 ** -24 * np.log(n)


# ------------------------------------------------- sums over millions of keys

def check_long_rows(out, lse, q, k, times):
    """Rows over keys k [n, 576] that each occur `times` often, in 64 bits on the GPU.

    A value's sum is added up by the tensor core in runs of 131072 keys, 16 keys a step
    that may cut where it does not round: 8192 2^-23 = 2^-10 of sum p |v|. The runs and
    the weights are added up in fp32, a term for 128 keys. The rest as in check_rows."""
    n = float(times.sum())
    q, k = q.double(), k.double()
    z = SM * (q @ k.T) + times.double().log()
    ref_lse = torch.logsumexp(z, 1, keepdim=True)
    p = (z - ref_lse).exp()
    ref, absum = p @ k[:, :512], p @ k[:, :512].abs()
    dz = SM * 580 * 2.0 ** -24 * q.norm(dim=1, keepdim=True) * k.norm(dim=1).max()
    run = (n / 128 + 128) * 2.0 ** -24
    tol_lse = 2 * dz + 2 * run + 2.0 ** -20 * (1 + ref_lse.abs())
    off = (lse.double().view(-1, 1) - ref_lse).abs()
    assert (off <= tol_lse).all(), (off.max(), tol_lse.min())
    tol = (2.0 ** -8 + 2 * tol_lse + 2.0 ** -18 + 2.0 ** -10 + run) * absum + 2.0 ** -8 * ref.abs()
    bad = (out.double() - ref).abs() > tol
    assert not bad.any(), ((out.double() - ref).abs()[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("B,late", [(75, 0), (75, 2048), (3, 64), (148, 0)])
def test_split_decode_of_millions_of_tokens(dsa, B, late):  # noqa: F811
    """Four million tokens a sequence out of few blocks, values all positive: row tiles in
    one share and cut ones. The last `late` blocks draw e^6.25 times the weight, so that
    the reference maximum of what was summed before them moves."""
    g = torch.Generator(device="cuda").manual_seed(B + late)
    blocks, H = 65536, 2
    kv = torch.rand(32, 64, 576, generator=g, device="cuda").to(torch.bfloat16)
    kv[16:, :, :512] += 2
    kv[:, :, 575] = 0
    kv[16:, :, 575] = 6.25
    q = randn(g, B, 1, H, 576)
    q[..., :512] *= 0.1                                 # the values' size says little
    q[..., 575] = 24
    early = torch.arange(blocks - late, dtype=torch.int32, device="cuda") % 16
    row = torch.cat([early, 16 + torch.arange(late, dtype=torch.int32, device="cuda") % 16])
    lens = torch.full((B,), blocks * 64, dtype=torch.int32, device="cuda")
    out, lse = dsa.split_mla_decode_paged(q, kv, row.repeat(B, 1), lens, SM)
    no_device_error(dsa)
    times = torch.bincount(row, minlength=32).repeat_interleave(64)
    k = kv.view(-1, 576)[times > 0]
    check_long_rows(out.view(-1, 512), lse.view(-1), q.view(-1, 576), k, times[times > 0])


def test_window_prefill_of_whole_row_tiles_over_long_prefixes(dsa):  # noqa: F811
    """Too many row tiles to scan, each longer than a run of the tensor core's sums: the
    call needs a workspace, which ends where it says."""
    g = torch.Generator(device="cuda").manual_seed(99)
    T, H, p0 = 16385, 65, 150000
    S = p0 + T
    kv = torch.rand(S, 576, generator=g, device="cuda").to(torch.bfloat16)
    q = randn(g, T, H, 576)
    need = dsa.window_mla_workspace_size(T, S, H, p0, 0, S)
    assert need > 0 and dsa.window_mla_workspace_size(T, S, H, p0, 4, 130000) == 0
    ws = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    out, lse = dsa.window_mla(q, kv, 0, S, SM, q_pos0=p0, workspace=ws[:need])
    no_device_error(dsa)
    assert (ws[need:] == 171).all()
    for t in (0, 73, 74, 9000, T - 1):
        k = kv[:p0 + t + 1]
        check_long_rows(out[t], lse[t], q[t], k, torch.ones(len(k), device="cuda"))


@pytest.mark.parametrize("lens,budget", [([400_000], 100_003), ([41_500] + [100] * 80, 20_001)])
def test_evict_of_more_totals_than_shared_memory_holds(dsa, lens, budget):  # noqa: F811
    """Totals that the selection reads from memory on each pass: past eight CTAs' places,
    and past one CTA's where the batch leaves a sequence no more."""
    check_evict(dsa, lens, budget, 4, 1000, odd, seed=len(lens), alias=True)
