"""Bounded-history operators where values are not finite, shares are small or buffers change hands; the
tolerances are those of test_gpu_bounded_history.py unless a test derives another."""
import numpy as np
import pytest

from oracle import ispa_oracle as orc
from gpu_helpers import ATTN_TOL, host, rel
from test_gpu_bounded_history import F32_TOL, MASS_TOL, ROW_TOL, check_sparse, dt, lse_of, sparse_case, tensor

pytestmark = pytest.mark.gpu

MASS_CALLS = [("bf16", 128, 2), ("bf16", 64, 20), ("bf16", 128, 200), ("bf16", 64, 300), ("fp32", 32, 5), ("fp32", 128, 40)]


def mass_of(q, k, ll, lh, **kw):
    """The call's weights and the oracle's, [H, n_k]."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    H, n_k = q.shape[1], k.shape[0]
    got = ispa.attn_mass(q, k, ll, lh, torch.zeros((H, n_k), device="cuda"), **kw)
    assert ispa.get_device_status() == ispa.ISPA_OK
    with np.errstate(all="ignore"):
        return host(got), orc.attn_mass(host(q), host(k), host(ll), None if lh is None else host(lh), np.zeros((H, n_k)))


# ------------------------------------------------------------------------------------------ weights
@pytest.mark.parametrize("dtype,hd,n_q", MASS_CALLS)
@pytest.mark.parametrize("hist", ["none", "empty", "finite"])
def test_mass_keeps_a_nan_log_sum_exp(cuda_ok, dtype, hd, n_q, hist):
    """A row whose lse_loc is NaN makes every weight of its head NaN, whatever the history's lse is; the other
    head does not see it."""
    import torch
    q, k = tensor((n_q, 2, hd), 1, dt(dtype), 2.0), tensor((150, 2, hd), 2, dt(dtype))
    ll = lse_of(q, k) + 0.5
    lh = {"none": None, "empty": torch.full_like(ll, -float("inf")), "finite": ll - 1.0}[hist]
    ll[0, n_q // 2] = float("nan")
    got, want = mass_of(q, k, ll, lh)
    assert np.isnan(want[0]).all() and np.isnan(got[0]).all()
    assert np.max(np.abs(got[1] - want[1]) / want[1]) <= MASS_TOL


@pytest.mark.parametrize("dtype,hd,n_q", MASS_CALLS)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_mass_of_rows_without_keys_whose_scores_are_not_finite(cuda_ok, dtype, hd, n_q, value):
    """A row whose log-sum-exp is -inf adds nothing, whatever its query holds."""
    import torch
    q, k = tensor((n_q, 2, hd), 3, dt(dtype), 2.0), tensor((150, 2, hd), 4, dt(dtype))
    ll = lse_of(q, k)
    dead = [0, n_q // 2, n_q - 1] if n_q > 2 else [1]
    ll[:, dead] = -float("inf")
    q[dead] = value
    got, want = mass_of(q, k, ll, torch.full_like(ll, -float("inf")))
    assert np.max(np.abs(got - want) / want) <= MASS_TOL


@pytest.mark.parametrize("n_q", [8, 200])
def test_mass_of_weights_past_the_largest_number(cuda_ok, n_q):
    """Log-sum-exps that do not cover the key (those of attention over selected blocks, say): a weight may
    pass 1, and past fp32 it is infinite, whichever query it comes from.  Weights up to e^80 stay exact:
    |logit| + |L| <= 100 in the exponent is 100 2^-24 = 6e-6 of MASS_TOL."""
    import torch
    q, k = tensor((n_q, 1, 128), 5, torch.bfloat16, 2.0), tensor((150, 1, 128), 6, torch.bfloat16)
    bias = torch.zeros((1, 150), device="cuda")
    bias[:, 3] = -float("inf")
    for i in range(8):
        ll = torch.full((1, n_q), 9.0, device="cuda")
        ll[:, i] = -200.0
        got, _ = mass_of(q, k, ll, None, kv_bias=bias)
        assert got[0, 3] == 0 and np.isposinf(np.delete(got[0], 3)).all(), i
        ll[:, i] = -65.0
        got, want = mass_of(q, k, ll, None)
        assert np.max(np.abs(got - want) / want) <= MASS_TOL, i


# ------------------------------------------------------------------------------------------ sparse attention
@pytest.mark.parametrize("dtype,hd,n_q,q_block", [("bf16", 64, 2, 1), ("bf16", 128, 2, 1), ("bf16", 128, 3, 128), ("bf16", 64, 200, 128),
                                                  ("bf16", 128, 200, 128), ("fp32", 64, 3, 2)])
@pytest.mark.parametrize("last", [1, 2, 4, 9])
def test_sparse_infinite_values_stay_infinite(cuda_ok, dtype, hd, n_q, q_block, last):
    """An infinity in the `last`-th value row from the end of the local keys (5, 16 + 13 of them) or of the
    history gives that infinity in its column, wherever the key lies in its tile."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    for n_loc in (5, 29):
        if last > n_loc:
            continue
        t, _ = sparse_case(dtype, 2, hd, n_q, q_block, 0, n_loc, 75, 64, 2, 80)
        idx = torch.tensor([0, 1], dtype=torch.int32, device="cuda").repeat(2, -(-n_q // q_block), 1)
        t["v_loc"][-last, :, 3] = float("inf")
        t["v_hist"][-last, :, 7] = -float("inf")
        out = ispa.block_sparse_attn(*t.values(), idx, block=64, q_block=q_block)
        with np.errstate(all="ignore"):
            ref = orc.block_sparse(*(host(x) for x in t.values()), idx.cpu().numpy(), 64, q_block)
        tol = F32_TOL if dtype == "fp32" else ROW_TOL if n_q < 100 else ATTN_TOL
        for got, want, w in ((out["o_loc"], ref["O_loc"], "o_loc"), (out["o_full"], ref["O_full"], "o_full")):
            got, want = host(got).reshape(want.shape), want
            inf = np.isinf(want)
            assert inf[..., 3].all() and inf[..., 7].any() == (w == "o_full")
            assert np.array_equal(got[inf], want[inf]) and rel(got[~inf], want[~inf]) <= tol[w], (w, n_loc)


def small_share(dtype, H, hd, n_q, q_block, n_loc, seed, scale=1.0):
    """A case whose history weighs next to nothing: queries of positive elements (about 2.6 each) against history
    keys moved by -0.8, so that the scores lie 2.6 * 0.8 * sqrt(hd) lower."""
    import torch
    t, _ = sparse_case(dtype, H, hd, n_q, q_block, 6, n_loc, 200, 64, 3, seed)
    t["q"].copy_(t["q"].abs() + 1)
    t["k_hist"].sub_(0.8)
    for name in ("v_sink", "v_loc"):
        t[name].mul_(scale)
    return t, torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda").repeat(H, -(-n_q // q_block), 1)


@pytest.mark.parametrize("dtype,hd,n_q,q_block", [("fp32", 64, 3, 1), ("fp32", 128, 5, 4), ("bf16", 64, 2, 1), ("bf16", 128, 3, 128),
                                                  ("bf16", 64, 200, 128), ("bf16", 128, 200, 128)])
def test_sparse_difference_of_a_small_share(cuda_ok, dtype, hd, n_q, q_block):
    """D = O_full - O_loc keeps its relative accuracy where the history's share (here about 1e-7 and less) is
    below the rounding of O_full."""
    t, idx = small_share(dtype, 2, hd, n_q, q_block, 90, 81)
    out = check_sparse(t, idx, 64, q_block, F32_TOL if dtype == "fp32" else ROW_TOL if n_q < 100 else ATTN_TOL)
    assert np.abs(host(out["d"])).max() < 1e-4


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -128])
def test_sparse_local_output_is_held_in_32_bits(cuda_ok, hd, scale):
    """Under a history that weighs nothing O_full is O_loc: the local output that the tensor-core kernel sets
    aside while it walks the history comes back as it was, so both round alike (subnormal ones too)."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    t, idx = small_share("bf16", 2, hd, 700, 128, 300, 82, scale)
    for name in ("v_hist",):
        t[name].mul_(scale)
    t["k_hist"].sub_(3.0)
    out = ispa.block_sparse_attn(*t.values(), idx, block=64, q_block=128)
    assert ispa.get_device_status() == ispa.ISPA_OK
    assert torch.isfinite(out["o_full"]).all() and torch.isfinite(out["lse_hist"]).all()
    assert torch.equal(out["o_full"], out["o_loc"])


# ------------------------------------------------------------------------------------------ the flag
def test_cuda_cores_flag_asks_for_fp32_arithmetic(cuda_ok):
    """With cuda_cores the same values give the same bits at any alignment: aligned rows take the multiply-add
    form too."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    for hd, n_q in ((64, 3), (128, 20), (128, 40)):
        qk = [(tensor((n_q, 2, hd), 7, torch.bfloat16, 2.0, p, p), tensor((150, 2, hd), 8, torch.bfloat16, 1.0, p, p)) for p in (0, 1)]
        ll = lse_of(*qk[0])
        a, b = (ispa.attn_mass(q, k, ll, None, torch.zeros((2, 150), device="cuda"), cuda_cores=True) for q, k in qk)
        assert torch.equal(a, b)
    for hd, n_q, q_block in ((64, 2, 1), (128, 3, 1), (128, 5, 128)):
        a, b = (ispa.block_sparse_attn(*sparse_case("bf16", 2, hd, n_q, q_block, 5, 70, 300, 64, 3, 83, p, p)[0].values(),
                                       torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda").repeat(2, -(-n_q // q_block), 1),
                                       block=64, q_block=q_block, cuda_cores=True) for p in (0, 1))
        assert all(torch.equal(a[w], b[w]) for w in a)


# ------------------------------------------------------------------------------------------ streams and buffers
def owner_of(address):
    """The stream whose memory holds this address (the allocator's segments, blocks in use or free)."""
    import torch
    return [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= address < s["address"] + s["total_size"]]


@pytest.mark.parametrize("llayer_,blocks", [(False, True), (False, False), (True, False)])
def test_layer_forward_on_a_stream_works_in_its_memory(cuda_ok, monkeypatch, llayer_, blocks):
    """Buffers that layer_forward drops on return, while a side stream still works on them, are that stream's;
    so is the result."""
    import torch
    from kv_cache_compression_tma_b200 import ispa, llayer
    t, idx = sparse_case("bf16", 2, 64, 3, 1, 5, 70, 300, 64, 3, 84)
    W = tensor((128, 1, 128), 85, torch.bfloat16, 1 / 16.0).flatten(1)
    seen = []

    def spy(name):
        call = getattr(ispa, name)

        def wrapped(*a, **kw):
            out = call(*a, **kw)
            seen.extend(x.data_ptr() for x in out.values() if x is not None)
            return out
        monkeypatch.setattr(ispa, name, wrapped)

    spy("dual_stream_attn")
    spy("block_sparse_attn")
    want = llayer.layer_forward(*t.values(), W, llayer=llayer_, blocks=idx if blocks else None, block=64, q_block=1)
    seen.clear()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = llayer.layer_forward(*t.values(), W, llayer=llayer_, blocks=idx if blocks else None, block=64, q_block=1, stream=side)
    side.synchronize()
    assert torch.equal(y, want) and len(seen) == 4
    assert all(owner_of(a) == [side.cuda_stream] for a in seen + [y.data_ptr()])


def test_results_of_the_other_calls_on_a_stream_come_from_its_memory(cuda_ok):
    """The same of the calls whose results layer_forward does not reach."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    d = 256
    a = tensor((d, 1, d), 86, torch.bfloat16).flatten(1)
    G = torch.eye(d, device="cuda") * 4
    R, S = torch.eye(d, device="cuda"), torch.eye(d, device="cuda")
    tc = ispa.TempCache(2, 64, 32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qw, sw = ispa.quantize_e4m3(a, columns=True, stream=side)
    qa, sa = ispa.quantize_e4m3(a, stream=side)
    out = [qw, sw, qa, sa, ispa.project_w8a8(qa, sa, qw, sw, stream=side), ispa.project(a, a, stream=side)]
    out += [x for x in ispa.absorb(G, R, S, a, 0.1, write_wnew=True, stream=side).values()]
    out += [x for x in ispa.absorb_static(G, R, S, a, 0.1, write_wnew=True, stream=side).values()]
    out += tc.match(tensor((4, 2, 64), 87, torch.bfloat16), stream=side)
    side.synchronize()
    assert ispa.get_device_status() == ispa.ISPA_OK
    assert all(owner_of(x.data_ptr()) == [side.cuda_stream] for x in out)


@pytest.mark.parametrize("blocks", [False, True])
def test_layer_work_holds_the_log_sum_exps_of_a_smaller_chunk(cuda_ok, blocks):
    """A LayerWork made for more rows: its views are arrays as the calls write them, and layer_forward
    allocates nothing but its result."""
    import torch
    from kv_cache_compression_tma_b200 import ispa, llayer
    t, idx = sparse_case("bf16", 4, 64, 5, 1, 5, 70, 300, 64, 3, 88)
    W = tensor((256, 1, 256), 89, torch.bfloat16, 1 / 16.0).flatten(1)
    work = llayer.LayerWork(9, 4, 64, torch.bfloat16)
    y = torch.empty((5, 256), dtype=torch.bfloat16, device="cuda")
    call = lambda: llayer.layer_forward(*t.values(), W, llayer=False, work=work, out=y, blocks=idx if blocks else None, block=64, q_block=1)
    call()
    n0 = torch.cuda.memory_stats()["allocation.all.allocated"]
    call()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == n0
    want = ispa.block_sparse_attn(*t.values(), idx, block=64) if blocks else ispa.dual_stream_attn(*t.values())
    view = work.view(5)
    assert all(torch.equal(view[w], want[w]) for w in ("o_loc", "o_full", "lse_loc", "lse_hist"))


def test_block_index_over_a_cache_whose_slots_change(cuda_ok):
    """Insertion replaces entries in place: a BlockIndex that is given the MassCache itself pools what it holds
    now, while the cache fills, when it first evicts and when its length no longer changes."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    H, hd, cap = 2, 64, 200
    mc, bi = ispa.MassCache(H, hd, cap), ispa.BlockIndex(H, hd, cap, block=64)
    for step in range(4):
        new = [tensor((90, H, hd), 90 + 2 * step + i, torch.bfloat16) for i in range(2)]
        mc.insert(*new, torch.rand((H, 90), device="cuda"))
        bi.extend(mc)
        assert mc.n == min(cap, 90 * (step + 1))
        nb = -(-mc.n // 64)
        assert np.array_equal(bi.means[:nb].cpu().numpy(), orc.block_means(host(mc.k[:mc.n]), 64).astype(np.float32))
        assert bi.select(new[0][:1], 2).max().item() < nb


@pytest.mark.parametrize("hd", [64, 128])
def test_sparse_rows_weigh_values_in_fp32(cuda_ok, hd):
    """Three keys of weights 1, x and 1 with values -b1, 1 and -b2, where b1 + b2 are the first 16 bits of x: what
    is left, (x - b1 - b2) / (2 + x), is below 2.6e-6 and lost to weights of 16 bits.  The scores are one product each,
    |y| <= 2.2 in base 2; x is good to 2^-22 (the exponential), 4 2^-24 |y| ln 2 (scale, difference) and 2^-22 (two
    sums in the tensor core), in all 9e-7 of x <= 1, so 3e-7 of the quotient."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    H, n_q = 24, 3
    q, k, v = (torch.zeros((n, H, hd), dtype=torch.bfloat16, device="cuda") for n in (n_q, 3, 3))
    q[:, :, 0] = torch.tensor([1.0, 0.75, 0.5], device="cuda")[:, None]
    k[1, :, 0] = -(0.5 + torch.arange(H, device="cuda") * 0.46875) * (hd / 64) ** 0.5
    x = torch.exp(q.double()[:, :, 0] * k.double()[1, :, 0] / hd ** 0.5)  # [n_q, H]
    b1 = x.to(torch.bfloat16)
    b2 = (x - b1.double()).to(torch.bfloat16)
    v[1] = 1.0
    for i in range(n_q):  # a value column per query
        v[0, :, i], v[2, :, i] = -b1[i], -b2[i]
    want = (x - b1.double() - b2.double()) / (2.0 + x)
    none = torch.zeros((H, n_q, 0), dtype=torch.int32, device="cuda")
    out = ispa.block_sparse_attn(q, k[:0], v[:0], k, v, k[:0], v[:0], none, block=64)
    got = torch.stack([out["o_loc"].view(n_q, H, hd)[i, :, i] for i in range(n_q)]).double()
    assert want.abs().max().item() > 1e-6
    assert (got - want).abs().max().item() <= 3e-7 + 2.0 ** -8 * 2.6e-6
