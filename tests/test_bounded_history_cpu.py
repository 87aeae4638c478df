"""CPU checks of the bounded-history operators: the oracle's own definitions against identities and hand
values, and the C ABI's refusals (no call here reaches a device)."""
import ctypes
import math
import os

import numpy as np
import pytest

from oracle import ispa_oracle as orc

P = 0x10000
NAN = float("nan")


@pytest.fixture(scope="module")
def ispa():
    from kv_cache_compression_tma_b200 import build, ispa as mod
    if not os.path.exists(mod.LIB_PATH):
        build.build()
    return mod


def g(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


# ------------------------------------------------------------------------------------------ oracle
def test_mass_of_all_keys_sums_to_one_per_query():
    """Over the whole key set the weights of a row sum to 1, so the masses of a head sum to n_q."""
    q, kl, kh = g(5, 2, 8, seed=1), g(6, 2, 8, seed=2), g(9, 2, 8, seed=3)
    z = lambda k: np.stack([np.log(np.exp(q[:, h] @ k[:, h].T / math.sqrt(8)).sum(1)) for h in range(2)])
    ll, lh = z(kl), z(kh)
    m = [orc.attn_mass(q, k, ll, lh, np.zeros((2, len(k)))) for k in (kl, kh)]
    assert np.allclose(m[0].sum(1) + m[1].sum(1), 5.0, atol=1e-12)
    twice = orc.attn_mass(q, kh, ll, lh, m[1], decay=0.5)
    assert np.allclose(twice, 1.5 * m[1])
    dead = orc.attn_mass(q, kh, np.full_like(ll, -np.inf), None, m[1])
    assert np.array_equal(dead, m[1])
    b = np.zeros((2, 9))
    b[0, 4] = -np.inf
    kh[4, 0] = NAN
    masked = orc.attn_mass(q, kh, ll, lh, np.zeros((2, 9)), bias=b)
    assert masked[0, 4] == 0 and np.isfinite(masked).all()


def test_insert_hand_values():
    # capacity 4, full: masses 3 1 2 0; new 1.5 0.5 5: drop the three lowest (0, 0.5, 1)
    src = orc.cache_insert([[3, 1, 2, 0]], [[0, 1, 2, 3]], [[1.5, 0.5, 5]], 4, 4, 0, 100)
    assert src.tolist() == [[0, 4, 2, 6]]
    # ties keep the earlier candidate; a protected position outranks any mass; NaN leaves first
    src = orc.cache_insert([[1, 1, NAN, 9]], [[0, 1, 2, 3]], [[1, 1]], 4, 4, 0, 5)
    assert src.tolist() == [[0, 1, 5, 3]]
    # room left: plain append, nothing moves
    src = orc.cache_insert([[1, 0]], [[0, 1]], [[0, 0]], 2, 8, 0, 100)
    assert src.tolist() == [[0, 1, 2, 3]]
    # room for part of them: the evicted slot first, then the unused one
    src = orc.cache_insert([[5, 0]], [[0, 1]], [[7, 6]], 2, 3, 0, 100)
    assert src.tolist() == [[0, 2, 3]]


def test_selecting_every_block_is_full_attention():
    q, ks, kl, kh = g(7, 2, 16, seed=4), g(3, 2, 16, seed=5), g(5, 2, 16, seed=6), g(10, 2, 16, seed=7)
    vs, vl, vh = g(3, 2, 16, seed=8), g(5, 2, 16, seed=9), g(10, 2, 16, seed=10)
    idx = orc.block_select(q, orc.block_means(kh, 4), 5, 2)
    assert idx.shape == (2, 4, 5) and np.array_equal(idx[0, 0], [0, 1, 2, -1, -1])
    s = orc.block_sparse(q, ks, vs, kl, vl, kh, vh, idx, 4, 2)
    d = orc.dual_stream(q, ks, vs, kl, vl, kh, vh)
    for w in ("O_loc", "O_full", "lse_loc", "lse_hist", "lse_full"):
        assert np.allclose(s[w], d[w], atol=1e-12), w
    none = orc.block_sparse(q, ks, vs, kl, vl, kh, vh, -np.ones((2, 7, 1)), 4, 1)
    assert np.array_equal(none["O_full"], none["O_loc"]) and np.isneginf(none["lse_hist"]).all()


def test_select_ties_and_nan():
    means = np.ones((4, 1, 2))
    means[2] = 3
    assert orc.block_select(np.ones((1, 1, 2)), means, 2, 1).tolist() == [[[0, 2]]]
    means[0] = NAN
    assert orc.block_select(np.ones((1, 1, 2)), means, 3, 1).tolist() == [[[1, 2, 3]]]


# ------------------------------------------------------------------------------------------ refusals
def mass_args(**kw):
    a = dict(dtype=0, H=2, hd=64, q=P, n_q=8, ld_q=128, k=P, n_k=16, ld_k=128, ll=P, lh=P, bias=P, ld_bias=16, scale=0.0,
             decay=1.0, flags=0, mass=P, out=P, ld_mass=16, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=3), 1), (dict(H=0), 1), (dict(hd=48), 2), (dict(hd=32), 2), (dict(hd=0), 2), (dict(n_q=-1), 1),
    (dict(n_k=-1), 1), (dict(n_k=1 << 31), 1), (dict(ld_q=127), 1), (dict(ld_k=64), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(q=P + 1), 1), (dict(dtype=1, k=P + 2), 1), (dict(ll=None), 1), (dict(ll=P + 2), 1), (dict(lh=P + 1), 1),
    (dict(ld_bias=15), 1), (dict(bias=P + 2), 1), (dict(scale=-1.0), 1), (dict(scale=NAN), 1), (dict(decay=-0.5), 1),
    (dict(decay=float("inf")), 1), (dict(decay=NAN), 1), (dict(flags=2), 1), (dict(mass=None), 1), (dict(out=None), 1),
    (dict(out=P + 2), 1), (dict(ld_mass=15), 1), (dict(n_k=0, k=None, mass=None, out=None), 0),
])
def test_mass_refusals(ispa, kw, expect):
    n0 = ispa.launch_count()
    assert ispa.lib().ispa_attn_mass(*mass_args(**kw)) == expect
    assert ispa.launch_count() == n0


def insert_args(**kw):
    a = dict(dtype=0, H=2, hd=64, k=P, v=P, ld_cache=128, capacity=16, n=16, mass=P, pos=P, ld_state=16, k_new=P, v_new=P,
             n_new=4, ld_new=128, mass_new=P, ld_mass_new=4, pos_new=16, below=0, frm=100, mass_out=P, pos_out=P, ld_out=16,
             stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), 1), (dict(H=0), 1), (dict(hd=48), 2), (dict(k=None), 1), (dict(v=None), 1), (dict(k=P + 1), 1),
    (dict(ld_cache=64), 1), (dict(capacity=15), 1), (dict(capacity=1 << 30), 1), (dict(n=-1), 1), (dict(mass=None), 1),
    (dict(pos=None), 1), (dict(mass=P + 2), 1), (dict(ld_state=15), 1), (dict(k_new=None), 1), (dict(v_new=P + 1), 1),
    (dict(n_new=-1), 1), (dict(ld_new=64), 1), (dict(mass_new=P + 1), 1), (dict(ld_mass_new=3), 1), (dict(pos_new=-1), 1),
    (dict(pos_new=2 ** 31 - 3), 1), (dict(mass_out=None), 1), (dict(pos_out=None), 1), (dict(ld_out=15), 1),
    (dict(ld_out=20), 1), (dict(n_new=65537, ld_mass_new=65537), 2),
    (dict(capacity=0, n=0, k=None, v=None, mass=None), 0), (dict(n=0, n_new=0, capacity=8, k_new=None), 0),
])
def test_insert_refusals(ispa, kw, expect):
    n0 = ispa.launch_count()
    assert ispa.lib().ispa_cache_insert(*insert_args(**kw)) == expect
    assert ispa.launch_count() == n0


def test_block_means_and_select_refusals(ispa):
    m, s = ispa.lib().ispa_block_means, ispa.lib().ispa_block_select
    # (dtype, H, hd, k, n_k, ld_k, block, first, means, ld_means, stream)
    assert m(9, 2, 64, P, 100, 128, 64, 0, P, 128, None) == 1
    assert m(0, 0, 64, P, 100, 128, 64, 0, P, 128, None) == 1
    assert m(0, 2, 40, P, 100, 128, 64, 0, P, 128, None) == 2
    assert m(0, 2, 64, P, -1, 128, 64, 0, P, 128, None) == 1
    assert m(0, 2, 64, P, 100, 127, 64, 0, P, 128, None) == 1
    assert m(0, 2, 64, P, 100, 128, 0, 0, P, 128, None) == 1
    assert m(0, 2, 64, P, 100, 128, 64, -1, P, 128, None) == 1
    assert m(0, 2, 64, P, 100, 128, 64, 0, None, 128, None) == 1
    assert m(0, 2, 64, P + 1, 100, 128, 64, 0, P, 128, None) == 1
    assert m(0, 2, 64, P, 100, 128, 64, 0, P + 2, 128, None) == 1
    assert m(0, 2, 64, P, 100, 128, 64, 0, P, 100, None) == 1
    assert m(0, 2, 64, None, 100, 128, 64, 2, None, 128, None) == 0  # no block from `first` on
    assert m(0, 2, 64, None, 0, 128, 64, 0, None, 128, None) == 0
    # (dtype, H, hd, q, n_q, ld_q, q_block, means, n_blocks, ld_means, n_sel, idx, stream)
    assert s(9, 2, 64, P, 8, 128, 1, P, 4, 128, 2, P, None) == 1
    assert s(0, 2, 40, P, 8, 128, 1, P, 4, 128, 2, P, None) == 2
    assert s(0, 2, 64, P, -8, 128, 1, P, 4, 128, 2, P, None) == 1
    assert s(0, 2, 64, P, 8, 100, 1, P, 4, 128, 2, P, None) == 1
    assert s(0, 2, 64, P, 8, 128, 0, P, 4, 128, 2, P, None) == 1
    assert s(0, 2, 64, P, 8, 128, 1, None, 4, 128, 2, P, None) == 1
    assert s(0, 2, 64, P, 8, 128, 1, P, 16385, 128, 2, P, None) == 2
    assert s(0, 2, 64, P, 8, 128, 1, P, 4, 100, 2, P, None) == 1
    assert s(0, 2, 64, P, 8, 128, 1, P, 4, 128, 0, P, None) == 1
    assert s(0, 2, 64, P, 8, 128, 1, P, 4, 128, 2, None, None) == 1
    assert s(0, 2, 64, P + 1, 8, 128, 1, P, 4, 128, 2, P, None) == 1
    assert s(0, 2, 64, P, 8, 128, 1, P, 4, 128, 2, P + 2, None) == 1
    assert s(0, 2, 64, None, 0, 128, 1, None, 4, 128, 2, None, None) == 0


def attn_args(ispa, **kw):
    a = ispa.AttnArgs()
    a.dtype, a.n_heads, a.head_dim, a.flags, a.n_q = 0, 2, 64, 0, 8
    for i in range(3):
        a.n_kv[i], a.ld_k[i], a.ld_v[i] = 8, 128, 128
        a.k[i] = a.v[i] = P
    a.q, a.ld_q, a.ld_o = P, 128, 128
    a.o_loc = a.o_full = a.lse_loc = a.lse_hist = P
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_packed_attention_arguments_are_the_structure(ispa):
    """Every field of the packed form lands where the structure has it."""
    from kv_cache_compression_tma_b200 import ispa as mod
    a, n, values = ispa.AttnArgs(), 0, []
    for name, kind in a._fields_:
        for i in range(getattr(kind, "_length_", 1)):
            n += 1
            values.append(n * 0.5 if kind is ctypes.c_float else n)
            if hasattr(kind, "_length_"):
                getattr(a, name)[i] = values[-1]
            else:
                setattr(a, name, values[-1])
    assert mod._ATTN_ARGS.pack(*values) == bytes(a)


def test_block_sparse_refusals(ispa):
    f = ispa.lib().ispa_block_sparse_attn
    call = lambda idx=P, n_sel=2, block=64, q_block=1, **kw: f(ctypes.byref(attn_args(ispa, **kw)), idx, n_sel, block, q_block, None)
    n0 = ispa.launch_count()
    assert f(None, P, 2, 64, 1, None) == 1
    assert call(dtype=5) == 1 and call(head_dim=48) == 2 and call(flags=2) == 1 and call(ld_q=64) == 1
    assert call(n_sel=-1) == 1 and call(idx=None) == 1 and call(idx=P + 2) == 1
    assert call(block=0) == 1 and call(block=65537) == 1 and call(q_block=0) == 1
    assert call(q_block=64) == 2 and call(q_block=100) == 2      # neither single rows nor whole tiles
    a = attn_args(ispa)
    a.kv_bias[2], a.ld_bias[2] = P, 8
    assert f(ctypes.byref(a), P, 2, 64, 1, None) == 2            # no biased segments
    a = attn_args(ispa)
    a.n_kv[0] = a.n_kv[1] = 0
    assert f(ctypes.byref(a), P, 2, 64, 1, None) == 1            # empty local branch
    assert call(n_q=0) == 0
    assert ispa.launch_count() == n0


# ------------------------------------------------------------------------------------------ the binding
def test_sizes_past_the_abis_integers_are_refused(monkeypatch):
    """ctypes drops the high bits of an integer: a block of 2^32 + 1 tokens would pass the binding's shape
    checks and reach the library as one of 1.  On host tensors with the library faked: no call gets through."""
    import torch
    from kv_cache_compression_tma_b200 import ispa

    class Library:
        def __getattr__(self, name):
            return lambda *a: pytest.fail(f"{name} was called")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # what get_device() says of a host tensor
    monkeypatch.setattr(ispa, "lib", Library)
    monkeypatch.setattr(ispa, "_stream", lambda stream: 0)
    k, means = torch.zeros((8, 2, 64)), torch.zeros((8, 2, 64))
    mass, pos = torch.zeros((2, 8)), torch.zeros((2, 8), dtype=torch.int32)
    idx = torch.zeros((2, 1, 1), dtype=torch.int32)
    wrap = 2 ** 32 + 1
    insert = lambda pos_new=8, **kw: ispa.cache_insert(k, k, mass, pos, 8, k, k, None, pos_new, **kw)
    sparse = lambda **kw: ispa.block_sparse_attn(k, k, k, k, k, k, k, idx, **kw)
    bad = [lambda: ispa.block_means(k, means, wrap), lambda: ispa.block_means(k, means, 4, first=2 ** 64),
           lambda: ispa.block_means(k, means, 4, first=-1), lambda: ispa.block_select(k, means, 1, q_block=wrap),
           lambda: ispa.block_select(k, means, wrap, out=idx.expand(2, 8, 1)), lambda: sparse(block=wrap, q_block=8),
           lambda: sparse(block=4, q_block=wrap), lambda: insert(keep_from=2 ** 31), lambda: insert(keep_from=2 ** 32),
           lambda: insert(keep_below=2 ** 31), lambda: insert(keep_below=-2 ** 31 - 1), lambda: insert(pos_new=wrap)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    cache = ispa.MassCache(2, 64, 8, dtype=torch.float32, device="cpu")
    cache.seen = 2 ** 31
    for kw in ({}, {"recent": 4}):
        with pytest.raises(ValueError):
            cache.insert(k, k, **kw)
    assert cache.seen == 2 ** 31 and cache.n == 0


def test_block_sparse_outputs_must_differ(ispa):
    """Two outputs in one array: the tensor-core kernel keeps part of one in the other's place meanwhile."""
    f = ispa.lib().ispa_block_sparse_attn
    for same in ({}, dict(o_full=2 * P, d_out=P), dict(o_full=2 * P, d_out=2 * P)):
        for q_block in (1, 128):
            assert f(ctypes.byref(attn_args(ispa, **same)), P, 2, 64, q_block, None) == 1
