"""Refusals of the range attention, attention totals and eviction entry points:
bad arguments are turned down on the host, with no GPU."""
import ctypes

import pytest
import torch

from test_abi import dsa  # noqa: F401  (the fixture that builds and loads the library)

FAKE = ctypes.c_void_p(1 << 20)       # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)
BIG = 1 << 40
F = ctypes.c_float


def split(L, q=FAKE, kv=FAKE, bt=FAKE, sl=FAKE, B=2, nq=1, mb=4, nblk=8, H=128, sm=0.1, out=FAKE,
          lse=None, ws=FAKE, nbytes=BIG):
    return L.dsa_split_mla_decode_paged(q, kv, bt, sl, B, nq, mb, nblk, H, F(sm), out, lse, ws,
                                        nbytes, None)


def wdecode(L, q=FAKE, kv=FAKE, bt=FAKE, sl=FAKE, B=2, nq=1, mb=4, nblk=8, H=128, sinks=4,
            window=8, sm=0.1, out=FAKE, lse=None, ws=FAKE, nbytes=BIG):
    return L.dsa_window_mla_decode_paged(q, kv, bt, sl, B, nq, mb, nblk, H, sinks, window, F(sm),
                                         out, lse, ws, nbytes, None)


def window(L, q=FAKE, kv=FAKE, T=4, S=4, H=8, p0=0, sinks=0, window=4, sm=0.1, out=FAKE, lse=None,
           ws=FAKE, nbytes=BIG):
    return L.dsa_window_mla(q, kv, T, S, H, p0, sinks, window, F(sm), out, lse, ws, nbytes, None)


def mass(L, q=FAKE, kv=FAKE, bt=FAKE, sl=FAKE, lse=FAKE, B=2, nq=1, mb=4, nblk=8, H=128, sm=0.1,
         m=FAKE, ld=256):
    return L.dsa_attention_mass_paged(q, kv, bt, sl, lse, B, nq, mb, nblk, H, F(sm), m, ld, None)


def evict(L, kv=FAKE, k8=None, ks=None, bt=FAKE, sl=FAKE, m=FAKE, ld=256, B=2, mb=4, nblk=8,
          budget=100, sinks=4, recent=16, idx=FAKE, slo=FAKE, mo=None, ldo=256):
    return L.dsa_cache_evict_paged(kv, k8, ks, bt, sl, m, ld, B, mb, nblk, budget, sinks, recent,
                                   idx, slo, mo, ldo, None)


DECODE_BAD = [dict(q=None), dict(kv=None), dict(bt=None), dict(sl=None), dict(out=None),
              dict(q=ODD), dict(kv=ODD), dict(out=ODD), dict(B=-1), dict(nq=0), dict(mb=0),
              dict(nblk=0), dict(sm=0.0), dict(sm=-1.0), dict(sm=float("nan")), dict(mb=1 << 25),
              dict(nblk=1 << 26), dict(B=1 << 20, nq=1 << 10)]


@pytest.mark.parametrize("bad", DECODE_BAD)
def test_split_decode_refuses(dsa, bad):  # noqa: F811
    assert split(dsa.lib(), **bad) == -1


@pytest.mark.parametrize("bad", DECODE_BAD + [dict(sinks=-1), dict(window=0), dict(window=-3)])
def test_window_decode_refuses(dsa, bad):  # noqa: F811
    assert wdecode(dsa.lib(), **bad) == -1


@pytest.mark.parametrize("bad", [dict(q=None), dict(kv=None), dict(out=None), dict(q=ODD),
                                 dict(kv=ODD), dict(out=ODD), dict(T=-1), dict(S=0), dict(p0=-1),
                                 dict(sinks=-1), dict(window=0), dict(sm=0.0), dict(S=(1 << 30) + 1),
                                 dict(p0=2 ** 31 - 4), dict(T=1 << 28, H=128)])
def test_window_prefill_refuses(dsa, bad):  # noqa: F811
    assert window(dsa.lib(), **bad) == -1


@pytest.mark.parametrize("bad", DECODE_BAD[:4] + DECODE_BAD[5:7] + DECODE_BAD[8:]
                         + [dict(lse=None), dict(m=None), dict(ld=255)])
def test_attention_mass_refuses(dsa, bad):  # noqa: F811
    assert mass(dsa.lib(), **bad) == -1


@pytest.mark.parametrize("bad", [dict(kv=None), dict(bt=None), dict(sl=None), dict(m=None),
                                 dict(idx=None), dict(slo=None), dict(kv=ODD), dict(k8=ODD),
                                 dict(B=-1), dict(mb=0), dict(nblk=0), dict(budget=0),
                                 dict(sinks=-1), dict(recent=-1), dict(sinks=60, recent=41),
                                 dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(ld=255),
                                 dict(mo=FAKE, ldo=260), dict(mo=ctypes.c_void_p(1 << 21), ldo=99),
                                 dict(mb=1 << 25, ld=1 << 40)])
def test_evict_refuses(dsa, bad):  # noqa: F811
    assert evict(dsa.lib(), **bad) == -1


def test_unsupported_and_empty(dsa):  # noqa: F811
    L = dsa.lib()
    for H in (0, 129, -1):
        assert split(L, H=H) == -2 and wdecode(L, H=H) == -2 and window(L, H=H) == -2
        assert mass(L, H=H) == -2
    assert evict(L, B=65536) == -2
    # an empty batch or prompt is a no-op, whatever its pointers
    assert split(L, B=0, q=None, out=None, ws=None, nbytes=0) == 0
    assert wdecode(L, B=0, q=None, out=None, ws=None, nbytes=0) == 0
    assert window(L, T=0, q=None, out=None) == 0
    assert mass(L, B=0, q=None) == 0 and evict(L, B=0, idx=None) == 0


def test_workspace_is_checked(dsa):  # noqa: F811
    L = dsa.lib()
    need = L.dsa_split_mla_decode_workspace_size(2, 1, 4, 128)
    if need:
        for f in (split, wdecode):
            assert f(L, ws=None, nbytes=0) == -3 and f(L, nbytes=need - 1) == -3
            assert f(L, ws=ODD, nbytes=need) == -3
    need = L.dsa_window_mla_workspace_size(4, 4096, 8, 4092, 0, 4096)
    if need:
        assert window(L, S=4096, p0=4092, window=4096, ws=None, nbytes=0) == -3
        assert window(L, S=4096, p0=4092, window=4096, nbytes=need - 1) == -3
    for bad in ((0, 1, 4, 8), (1, 0, 4, 8), (1, 1, 0, 8), (1, 1, 4, 0), (1, 1, 4, 129)):
        assert L.dsa_split_mla_decode_workspace_size(*bad) == 0
    assert L.dsa_window_mla_workspace_size(0, 4, 8, 0, 0, 4) == 0


def test_binding_refuses_tensors_that_do_not_fit(dsa):  # noqa: F811
    kv = torch.zeros(2, 64, 576, dtype=torch.bfloat16)
    q = torch.zeros(1, 1, 8, 576, dtype=torch.bfloat16)
    bt, sl = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):                     # host tensors
        dsa.split_mla_decode_paged(q, kv, bt, sl, 0.1)
    with pytest.raises(ValueError):
        dsa.window_mla(q[0], kv[0], 0, 4, 0.1)
    with pytest.raises(ValueError):
        dsa.cache_evict_paged(kv, bt, sl, torch.zeros(1, 128), 10, 0, 0)


@pytest.mark.parametrize("arg", [3, 4, 5])
@pytest.mark.parametrize("value", [2**31, 2**32 + 1, -2**32])
def test_counts_past_32_bits_are_refused(arg, value):
    from sparse_attention_long_02_b200 import window_mla_workspace_size

    args = [4, 100, 128, 0, 1, 64]
    window_mla_workspace_size(*args)
    args[arg] = value
    with pytest.raises(ValueError, match="32 bits"):
        window_mla_workspace_size(*args)
