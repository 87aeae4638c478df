"""The bounded-history operators on the GPU against the fp64 oracle: accumulated attention weight, cache
insertion with eviction, block means, block selection and dual-stream attention over selected blocks.

Tolerances.  Selections, positions and copied rows are exact.  Block means: the fp64 mean rounded once
(2^-24; the 64-bit sums of the two sides differ by far less).  Attention weights: a logit is a sum of
hd <= 128 products of size |q k| / sqrt(hd) (q of deviation 2, so about 14.5 in all) with roundings of
2^-24 of the running sum each: a random walk of sqrt(128) 2^-24 14.5 = 1e-5, plus 2^-24 of |logit| + |L|
<= 60 in the exponent (4e-6) and the exponential's 2^-22; per key that is below 3e-5 relative, and zeros
are exact.  bf16 outputs of the row kernel: one rounding, 2^-8 of each value, so 2^-8 of the norm, plus
2e-5 of arithmetic; tensor cores: the repository's attention tolerances (P is rounded to bf16 too)."""
import numpy as np
import pytest

import ispa_inputs as inp
from oracle import ispa_oracle as orc
from gpu_helpers import ATTN_TOL, host, rel

pytestmark = pytest.mark.gpu

MASS_TOL = 3e-5
ROW_TOL = {"o_loc": 2.0 ** -8 + 2e-5, "o_full": 2.0 ** -8 + 2e-5, "d": 2.0 ** -8 + 2e-5, "lse_loc": 5e-5, "lse_hist": 5e-5}
F32_TOL = {"o_loc": 2e-5, "o_full": 2e-5, "d": 4e-5, "lse_loc": 5e-5, "lse_hist": 5e-5}


def tensor(shape, seed, dtype, sc=1.0, pad=0, lead=0):
    """Seeded [tokens, H, hd] values on the GPU, rounded to dtype, as a view of a wider row (pad elements)
    that starts `lead` elements into its storage."""
    import torch
    x = inp.gaussian(shape, 90, seed, sc).astype(np.float32)
    n, d = shape[0], int(np.prod(shape[1:]))
    flat = torch.zeros(lead + n * (d + pad), dtype=dtype, device="cuda")
    v = flat[lead:].view(n, d + pad)[:, :d].unflatten(1, shape[1:])
    v.copy_(torch.from_numpy(x).to("cuda"))
    return v


def dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def lse_of(q, k, bias=None):
    """fp32 natural-log LSE of the scaled logits, [H, n_q] (torch, from host fp64)."""
    import torch
    qh, kh = host(q), host(k)
    out = np.full((qh.shape[1], qh.shape[0]), -np.inf)
    for h in range(qh.shape[1]):
        s = qh[:, h] @ kh[:, h].T / np.sqrt(qh.shape[2])
        if bias is not None:
            s = s + bias[h]
        with np.errstate(divide="ignore"):
            m = s.max(1)
            out[h] = np.where(np.isneginf(m), -np.inf, np.log(np.exp(s - np.where(np.isneginf(m), 0, m)[:, None]).sum(1)) + m)
    return torch.from_numpy(out.astype(np.float32)).to("cuda").contiguous()


# ------------------------------------------------------------------------------------------ mass
def check_mass(q, k, ll, lh, mass, decay, bias=None, **kw):
    import torch
    from kv_cache_compression_tma_b200 import ispa
    n_k = k.shape[0]
    want = orc.attn_mass(host(q), host(k), host(ll), None if lh is None else host(lh), host(mass)[:, :n_k], decay,
                         None if bias is None else host(bias)[:, :n_k])
    tail = mass[:, n_k:].clone()
    ispa.attn_mass(q, k, ll, lh, mass, kv_bias=bias, decay=decay, **kw)
    assert ispa.get_device_status() == ispa.ISPA_OK
    got = host(mass)[:, :n_k]
    assert np.array_equal(got[want == 0], want[want == 0])
    nz = want != 0
    assert np.max(np.abs(got[nz] - want[nz]) / np.abs(want[nz]), initial=0.0) <= MASS_TOL
    assert torch.equal(mass[:, n_k:], tail)


@pytest.mark.parametrize("dtype,hd,n_q,n_k,H", [
    ("bf16", 128, 1, 1, 1), ("bf16", 128, 1, 1000, 3), ("bf16", 64, 3, 257, 2), ("bf16", 128, 17, 129, 2),
    ("bf16", 64, 9, 130, 3), ("bf16", 128, 32, 100, 2), ("bf16", 128, 33, 100, 2),
    ("bf16", 128, 128, 256, 2), ("bf16", 64, 129, 255, 2), ("bf16", 128, 300, 700, 2), ("bf16", 64, 513, 130, 1),
    ("fp32", 16, 5, 70, 3), ("fp32", 32, 64, 96, 2), ("fp32", 64, 33, 31, 2), ("fp32", 128, 2, 300, 2),
])
@pytest.mark.parametrize("biased", [False, True])
def test_mass(cuda_ok, dtype, hd, n_q, n_k, H, biased):
    import torch
    q, k = tensor((n_q, H, hd), 1, dt(dtype), 2.0), tensor((n_k, H, hd), 2, dt(dtype))
    bias = None
    if biased:
        b = np.log(1 + np.floor(np.abs(inp.gaussian((H, n_k + 3), 91, 1)) * 2.5).clip(0, 4)).astype(np.float32)
        b[inp.gaussian((H, n_k + 3), 91, 2) > 1.0] = -np.inf
        bias = torch.from_numpy(b).cuda()
    lh = lse_of(q, k, None if bias is None else host(bias)[:, :n_k])
    ll = lh + 0.5
    ll[torch.isinf(ll)] = 1.0
    mass = torch.from_numpy(np.abs(inp.gaussian((H, n_k + 5), 91, 3)).astype(np.float32)).cuda()
    check_mass(q, k, ll, lh, mass, 0.75, bias)


@pytest.mark.parametrize("H,n_q,n_k,hd", [(3, 130, 128 * 151 + 5, 64), (1, 8192 + 130, 300, 128), (2, 16640, 140, 64)])
def test_mass_many_tiles_and_query_chunks(cuda_ok, H, n_q, n_k, hd):
    """More key tiles than SMs (ranges of a CTA that cross heads, single tiles among pairs) and more
    queries than one chunk, against a 64-bit product on the GPU."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    q, k = tensor((n_q, H, hd), 7, torch.bfloat16, 2.0), tensor((n_k, H, hd), 8, torch.bfloat16)
    ll, lh = (3.0 + torch.rand((H, n_q), device="cuda") for _ in range(2))
    ll[:, 5] = lh[:, 5] = -float("inf")
    mass = torch.rand((H, n_k), device="cuda")
    want = 0.5 * mass.double()
    live = torch.isfinite(ll[0])
    for h in range(H):
        for i in range(0, n_q, 2048):
            s = q[i:i + 2048, h].double() @ k[:, h].double().T / np.sqrt(hd)
            w = torch.exp(s - torch.logaddexp(ll[h, i:i + 2048].double(), lh[h, i:i + 2048].double())[:, None])
            want[h] += w[live[i:i + 2048]].sum(0)
    ispa.attn_mass(q, k, ll, lh, mass, decay=0.5)
    assert ispa.get_device_status() == ispa.ISPA_OK
    assert ((mass.double() - want).abs() / want).max().item() <= MASS_TOL


@pytest.mark.parametrize("n_q", [2, 20, 200])
def test_mass_rows_without_keys_masked_nan_and_decay_zero(cuda_ok, n_q):
    """Rows with both lse's -inf add nothing; an excluded key's NaN stays out; decay 0 does not read the
    old mass (NaN there); no history branch; strided and (CUDA cores) unaligned operands."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    H, hd, n_k = 2, 128, 140
    q, k = tensor((n_q, H, hd), 3, torch.bfloat16, 2.0, pad=8), tensor((n_k, H, hd), 4, torch.bfloat16, pad=16)
    bias = torch.zeros((H, n_k + 1), device="cuda")[:, 1:]  # 4-byte aligned only
    bias[:, 7] = -float("inf")
    bias[:, 9] = torch.finfo(torch.float32).min  # as good as excluded
    ll = lse_of(q, k, host(bias))
    k[7] = float("nan")
    k[9] = 1000.0
    ll[:, n_q // 2] = -float("inf")
    mass = torch.full((H, n_k), float("nan"), device="cuda")
    check_mass(q, k, ll, None, mass, 0.0, bias)
    assert (mass[:, [7, 9]] == 0).all()
    for lead in (0, 1):
        qq, kk = tensor((n_q, H, 32), 5, torch.bfloat16, 2.0, 1, lead), tensor((n_k, H, 32), 6, torch.bfloat16, 1.0, 1, lead)
        check_mass(qq, kk, lse_of(qq, kk), None, mass.fill_(1.0), 1.0, cuda_cores=True)
    with pytest.raises(ispa.IspaError) as e:
        ispa.attn_mass(qq, kk, ll, None, mass)
    assert e.value.status == ispa.ISPA_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        ispa.attn_mass(q, k, ll[:, :1], None, mass)
    # no queries: the old weights decay, and that is all
    mass.fill_(3.0)
    ispa.attn_mass(q[:0], k, ll[:, :0].contiguous(), None, mass, decay=0.5)
    assert (mass == 1.5).all()


# ------------------------------------------------------------------------------------------ insert
def check_insert(cap, n, n_new, H, hd, dtype, seed, below=0, frm=None, pad=0, lead=0, separate=False, ties=False, mass_new=True):
    import torch
    from kv_cache_compression_tma_b200 import ispa
    k, v = tensor((cap, H, hd), seed, dt(dtype), pad=pad, lead=lead), tensor((cap, H, hd), seed + 1, dt(dtype), pad=pad, lead=lead)
    kn, vn = tensor((n_new, H, hd), seed + 2, dt(dtype), pad=2 * pad, lead=lead), tensor((n_new, H, hd), seed + 3, dt(dtype), pad=2 * pad, lead=lead)
    m = inp.gaussian((H, cap + 2), 92, seed).astype(np.float32)
    mn = inp.gaussian((H, n_new + 1), 92, seed + 1).astype(np.float32)
    if ties:
        m, mn = np.round(m), np.round(mn)
        m[:, ::7], mn[:, ::5] = np.nan, -0.0
    mass, mass_n = torch.from_numpy(m).cuda(), torch.from_numpy(mn).cuda()[:, :n_new]
    pos = torch.from_numpy(np.argsort(inp.gaussian((H, cap + 2), 92, seed + 2), axis=1).astype(np.int32)).cuda()
    pos_new, frm = cap + 2, (2 ** 31 - 1 if frm is None else cap + 2 + n_new - frm)
    if not mass_new:
        mn = np.zeros_like(mn)
        mass_n = None
    src = orc.cache_insert(m[:, :n], pos.cpu().numpy()[:, :n], mn[:, :n_new], pos_new, cap, below, frm)
    before = [t.clone() for t in (k, v, mass, pos)]
    mo, po = (torch.full_like(mass, 9.0), torch.full_like(pos, 9)) if separate else (mass, pos)
    mo0, po0 = mo.clone(), po.clone()
    total = ispa.cache_insert(k, v, mass, pos, n, kn, vn, mass_n, pos_new, keep_below=below, keep_from=frm,
                              mass_out=mo if separate else None, pos_out=po if separate else None)
    assert total == src.shape[1] == min(cap, n + n_new)
    at = torch.from_numpy(src).cuda()
    hh = torch.arange(H, device="cuda")[:, None]
    for got, old, new in ((k, before[0], kn), (v, before[1], vn)):
        want = torch.cat([old[:n], new])[at, hh].transpose(0, 1)
        assert torch.equal(got[:total], want) and torch.equal(got[total:], old[total:])
    zeros = torch.zeros((H, n_new), device="cuda")
    want = torch.cat([before[2][:, :n], mass_n if mass_new else zeros], 1).gather(1, at)
    assert torch.equal(torch.nan_to_num(mo[:, :total], nan=77.0), torch.nan_to_num(want, nan=77.0))
    news = (pos_new + torch.arange(n_new, device="cuda", dtype=torch.int32)).expand(H, n_new)
    assert torch.equal(po[:, :total], torch.cat([before[3][:, :n], news], 1).gather(1, at))
    same = lambda a, b: torch.equal(torch.nan_to_num(a, nan=77.0), torch.nan_to_num(b, nan=77.0))
    assert same(mo[:, total:], mo0[:, total:]) and torch.equal(po[:, total:], po0[:, total:])
    if separate:
        assert same(mass, before[2]) and torch.equal(pos, before[3])


@pytest.mark.parametrize("cap,n,n_new,H,hd,dtype", [
    (1, 1, 1, 1, 16, "fp32"), (1, 0, 1, 2, 64, "bf16"), (7, 5, 1, 2, 64, "bf16"), (20001, 20001, 1, 2, 32, "bf16"), (1, 0, 3, 2, 64, "bf16"), (8, 0, 5, 2, 64, "bf16"), (100, 100, 1, 3, 128, "bf16"),
    (100, 97, 10, 3, 128, "bf16"), (64, 64, 200, 2, 64, "bf16"), (1025, 1025, 700, 2, 32, "bf16"),
    (5000, 5000, 1300, 2, 64, "bf16"), (20000, 19990, 321, 1, 16, "bf16"), (333, 333, 333, 2, 32, "fp32"),
])
@pytest.mark.parametrize("separate", [False, True])
def test_insert(cuda_ok, cap, n, n_new, H, hd, dtype, separate):
    check_insert(cap, n, n_new, H, hd, dtype, 10, separate=separate)


def test_insert_ties_nan_protection_and_layouts(cuda_ok):
    for cap, n, n_new in ((60, 60, 25), (3000, 2990, 900), (50, 50, 1), (3000, 3000, 1)):
        check_insert(cap, n, n_new, 2, 64, "bf16", 20, ties=True)
        check_insert(cap, n, n_new, 2, 64, "bf16", 21, below=cap // 4, frm=n_new // 2, ties=True, separate=True)
        check_insert(cap, n, n_new, 2, 64, "bf16", 22, frm=n_new, pad=8)            # every new token protected
        check_insert(cap, n, n_new, 2, 64, "bf16", 23, below=2 ** 30, pad=3, lead=1)  # everything protected; unaligned rows
        check_insert(cap, n, n_new, 2, 64, "bf16", 24, mass_new=False)


def test_insert_slices_beyond_shared_memory(cuda_ok):
    """More candidates per CTA than their order keys fit in shared memory."""
    check_insert(700000, 700000, 90, 1, 16, "bf16", 30, ties=True)
    check_insert(700000, 699950, 90, 1, 16, "bf16", 31, separate=True)


# ------------------------------------------------------------------------------------------ blocks
@pytest.mark.parametrize("dtype,H,hd,n_k,block,first,pad,lead", [
    ("bf16", 1, 64, 1, 64, 0, 0, 0), ("bf16", 3, 128, 1000, 128, 0, 8, 0), ("bf16", 2, 64, 640, 64, 7, 0, 0),
    ("bf16", 2, 128, 200, 96, 1, 1, 1), ("bf16", 5, 16, 77, 5, 0, 0, 0), ("fp32", 2, 32, 95, 32, 0, 4, 0),
    ("fp32", 3, 16, 50, 7, 3, 1, 1),
])
def test_block_means(cuda_ok, dtype, H, hd, n_k, block, first, pad, lead):
    import torch
    from kv_cache_compression_tma_b200 import ispa
    k = tensor((n_k, H, hd), 40, dt(dtype), pad=pad, lead=lead)
    nb = -(-n_k // block)
    means = torch.full((nb + 2, H, hd), 5.0, device="cuda")
    ispa.block_means(k, means, block, first=first)
    got = means.cpu().numpy()
    want = orc.block_means(host(k), block)[first:].astype(np.float32)
    if dtype == "bf16":
        assert np.array_equal(got[first:nb], want)
    else:
        assert np.max(np.abs(got[first:nb] - want) / np.abs(want)) <= 2.0 ** -23
    assert (got[:first] == 5.0).all() and (got[nb:] == 5.0).all()


@pytest.mark.parametrize("dtype,H,hd,n_q,q_block,nb,n_sel", [
    ("bf16", 1, 64, 1, 1, 1, 1), ("bf16", 3, 128, 1, 1, 1500, 32), ("bf16", 2, 128, 9, 1, 130, 16),
    ("bf16", 2, 64, 300, 128, 40, 7), ("bf16", 2, 128, 1290, 128, 700, 64), ("bf16", 1, 128, 5, 128, 16384, 300),
    ("bf16", 2, 64, 10, 4, 5, 9), ("fp32", 2, 32, 64, 32, 3, 2), ("fp32", 2, 16, 50, 7, 33, 33), ("bf16", 2, 64, 3, 1, 0, 4),
])
def test_block_select(cuda_ok, dtype, H, hd, n_q, q_block, nb, n_sel):
    import torch
    from kv_cache_compression_tma_b200 import ispa
    q = tensor((n_q, H, hd), 50, dt(dtype), 2.0, pad=3, lead=1)
    means = tensor((nb, H, hd), 51, torch.float32, 0.1, pad=1)
    if nb > 8:  # exact ties
        means[nb // 2:nb // 2 + 3] = means[1]
    idx = ispa.block_select(q, means, n_sel, q_block=q_block)
    assert np.array_equal(idx.cpu().numpy(), orc.block_select(host(q), host(means), n_sel, q_block))


def test_block_select_all_equal_and_nan(cuda_ok):
    import torch
    from kv_cache_compression_tma_b200 import ispa
    q = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    means = torch.ones((500, 1, 64), device="cuda")
    assert ispa.block_select(q, means, 9).cpu().tolist() == [[list(range(9))] * 2]
    means[:498] = float("nan")
    assert ispa.block_select(q, means, 4).cpu().tolist() == [[[0, 1, 498, 499]] * 2]


# ------------------------------------------------------------------------------------------ sparse attention
def sparse_case(dtype, H, hd, n_q, q_block, n_sink, n_loc, n_hist, block, n_sel, seed, pad=0, lead=0):
    import torch
    names = ("k_sink", "v_sink", "k_loc", "v_loc", "k_hist", "v_hist")
    sizes = (n_sink, n_sink, n_loc, n_loc, n_hist, n_hist)
    t = {"q": tensor((n_q, H, hd), seed, dt(dtype), 2.0, pad, lead)}
    for i, (w, n) in enumerate(zip(names, sizes)):
        t[w] = tensor((n, H, hd), seed + 1 + i, dt(dtype), 1.0, pad, lead)
    groups, nb = -(-n_q // q_block), -(-n_hist // block)
    r = np.random.default_rng(seed)
    idx = np.full((H, groups, n_sel), -1, np.int32)
    for h in range(H):
        for g in range(groups):
            m = [min(n_sel, nb), 0, r.integers(0, min(n_sel, nb) + 1)][min(2, (h + g) % 4)]
            idx[h, g, :m] = np.sort(r.permutation(nb)[:m])
    return t, torch.from_numpy(idx).cuda()


def check_sparse(t, idx, block, q_block, tol, **kw):
    import torch
    from kv_cache_compression_tma_b200 import ispa
    out = ispa.block_sparse_attn(*t.values(), idx, block=block, q_block=q_block, **kw)
    assert ispa.get_device_status() == ispa.ISPA_OK
    ref = orc.block_sparse(*(host(x) for x in t.values()), idx.cpu().numpy(), block, q_block)
    n_q = t["q"].shape[0]
    ol, of = (ref[w].reshape(n_q, -1) for w in ("O_loc", "O_full"))
    assert rel(host(out["o_loc"]), ol) <= tol["o_loc"]
    assert rel(host(out["o_full"]), of) <= tol["o_full"]
    assert rel(host(out["d"]), of - ol) <= tol["d"]
    assert np.max(np.abs(host(out["lse_loc"]) - ref["lse_loc"])) <= tol["lse_loc"]
    none = np.isneginf(ref["lse_hist"])
    got = host(out["lse_hist"])
    assert np.array_equal(np.isneginf(got), none)
    assert np.max(np.abs(got[~none] - ref["lse_hist"][~none]), initial=0.0) <= tol["lse_hist"]
    H = none.shape[0]
    rows = torch.from_numpy(none.T).cuda()
    o = [out[w].view(n_q, H, -1) for w in ("o_loc", "o_full", "d")]
    assert torch.equal(o[0][rows], o[1][rows]) and (o[2][rows] == 0).all()
    return out


@pytest.mark.parametrize("H,hd,n_q,n_sink,n_loc,n_hist,block,n_sel", [
    (1, 64, 1, 0, 1, 1, 64, 1), (3, 128, 1, 40, 100, 1000, 64, 5), (2, 128, 5, 0, 33, 777, 128, 3),
    (2, 64, 3, 10, 0, 300, 32, 20), (2, 128, 1, 100, 200, 40000, 128, 200), (1, 128, 2, 5, 5, 50, 7, 4),
])
def test_sparse_rows_bf16(cuda_ok, H, hd, n_q, n_sink, n_loc, n_hist, block, n_sel):
    t, idx = sparse_case("bf16", H, hd, n_q, 1, n_sink, n_loc, n_hist, block, n_sel, 60)
    check_sparse(t, idx, block, 1, ROW_TOL)
    t, idx = sparse_case("bf16", H, hd, n_q, 1, n_sink, n_loc, n_hist, block, n_sel, 61, pad=1, lead=1)
    check_sparse(t, idx, block, 1, ROW_TOL)


@pytest.mark.parametrize("H,hd,n_q,q_block,n_sink,n_loc,n_hist,block,n_sel", [
    (2, 32, 64, 32, 16, 32, 95, 32, 2), (2, 16, 9, 4, 0, 20, 100, 16, 9), (1, 128, 7, 1, 3, 3, 64, 64, 1),
    (3, 64, 5, 128, 2, 9, 200, 10, 6),
])
def test_sparse_rows_fp32(cuda_ok, H, hd, n_q, q_block, n_sink, n_loc, n_hist, block, n_sel):
    t, idx = sparse_case("fp32", H, hd, n_q, q_block, n_sink, n_loc, n_hist, block, n_sel, 62, pad=4)
    check_sparse(t, idx, block, q_block, F32_TOL)


@pytest.mark.parametrize("H,hd,n_q,q_block,n_sink,n_loc,n_hist,block,n_sel", [
    (1, 64, 1, 128, 0, 1, 1, 64, 1), (2, 128, 300, 128, 40, 300, 1000, 64, 5), (2, 128, 257, 128, 0, 130, 777, 128, 3),
    (2, 64, 128, 128, 10, 0, 300, 64, 9), (1, 128, 700, 256, 128, 256, 4000, 128, 33), (3, 64, 130, 384, 1, 1, 63, 128, 2),
    (1, 128, 129, 128, 0, 64, 192, 128, 2), (2, 128, 48, 128, 5, 64, 192, 64, 2), (2, 128, 49, 128, 5, 64, 192, 64, 2),
    (2, 128, 74, 128, 5, 64, 192, 64, 2), (2, 128, 75, 128, 5, 64, 192, 64, 2), (1, 64, 149, 128, 0, 128, 100, 64, 1),
    (2, 128, 128, 128, 0, 129, 129, 128, 2), (1, 128, 400, 128, 100, 400, 5000, 128, 40),
])
@pytest.mark.parametrize("pad", [0, 8])
def test_sparse_tensor_cores(cuda_ok, H, hd, n_q, q_block, n_sink, n_loc, n_hist, block, n_sel, pad):
    t, idx = sparse_case("bf16", H, hd, n_q, q_block, n_sink, n_loc, n_hist, block, n_sel, 64, pad=pad)
    check_sparse(t, idx, block, q_block, ATTN_TOL)


def test_sparse_tensor_cores_odd_lists_and_dense_limit(cuda_ok):
    """Any order, entries that name no block, a ragged block in the middle of the list, NaN in the blocks
    that no list names; and every block listed = the dense kernel's result within its tolerance."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    for block in (64, 128):
        t, _ = sparse_case("bf16", 1, 128, 200, 128, 4, 8, 5 * block - 20, block, 1, 65)
        every = torch.arange(5, dtype=torch.int32, device="cuda").repeat(1, 2, 1)
        a = check_sparse(t, every, block, 128, ATTN_TOL)
        d = ispa.dual_stream_attn(*t.values())
        assert rel(host(a["o_full"]), host(d["o_full"])) <= ATTN_TOL["o_full"]
        for name in ("k_hist", "v_hist"):
            t[name][block:2 * block] = float("nan")
        idx = torch.tensor([[[4, -7, 0, 5, 2 ** 31 - 1, 2, 3], [2, 4, 0, -1, 99, -2 ** 31, 2]]], dtype=torch.int32, device="cuda")
        check_sparse(t, idx, block, 128, ATTN_TOL)
        none = check_sparse(t, idx[:, :, :0].contiguous(), block, 128, ATTN_TOL)
        assert torch.equal(none["o_full"], none["o_loc"])
        with pytest.raises(ispa.IspaError) as e:
            ispa.block_sparse_attn(*t.values(), idx[:, :, :1].contiguous(), block=96, q_block=128)
        assert e.value.status == ispa.ISPA_ERR_UNSUPPORTED


def test_sparse_longest_list(cuda_ok):
    """4096 entries of blocks of 128: three blocks, the last one ragged, 1365 times each.  O_hist is that of the
    three alone and lse_hist larger by log 1365.  Beside the usual tolerances: l is the sum of 1707 tiles'
    sums per group, each rounded by at most 2^-24 of it; O takes 8 products per tile of 3413, each
    truncated by at most 2^-23 of it."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    t, _ = sparse_case("bf16", 1, 128, 160, 128, 4, 30, 300, 128, 1, 70)
    idx = torch.tensor(([0, 1, 2] * 1366)[:4095] + [-1], dtype=torch.int32, device="cuda").repeat(1, 2, 1)
    out = ispa.block_sparse_attn(*t.values(), idx, block=128, q_block=128)
    assert ispa.get_device_status() == ispa.ISPA_OK
    ref = orc.block_sparse(*(host(x) for x in t.values()), idx[:, :, :3].cpu().numpy(), 128, 128)
    share = lambda lh: (1.0 / (1.0 + np.exp(ref["lse_loc"] - lh))).T[:, :, None]
    o_hist = ref["O_loc"] + (ref["O_full"] - ref["O_loc"]) / share(ref["lse_hist"])
    lse_hist = ref["lse_hist"] + np.log(1365.0)
    o_full = ref["O_loc"] + share(lse_hist) * (o_hist - ref["O_loc"])
    extra_l, extra_o = 1707 * 2.0 ** -24, 3413 * 8 * 2.0 ** -23
    assert np.max(np.abs(host(out["lse_hist"]) - lse_hist)) <= ATTN_TOL["lse_hist"] + extra_l
    assert rel(host(out["o_loc"]), ref["O_loc"].reshape(160, -1)) <= ATTN_TOL["o_loc"]
    for w, want in (("o_full", o_full), ("d", o_full - ref["O_loc"])):
        big = np.linalg.norm(o_hist) / np.linalg.norm(want)
        assert rel(host(out[w]), want.reshape(160, -1)) <= ATTN_TOL[w] + (extra_l + extra_o) * big, w


def test_sparse_odd_lists(cuda_ok):
    """Lists in any order, with entries that name no block, a block listed twice, n_sel == 0, and NaN in
    every key and value that no list names."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    t, _ = sparse_case("bf16", 1, 128, 2, 1, 4, 8, 300, 64, 1, 63)
    for name in ("k_hist", "v_hist"):
        t[name][64:128] = float("nan")
        t[name][192:256] = float("nan")
    idx = torch.tensor([[[4, -7, 0, 5, 2 ** 31 - 1, 2], [2, 4, 0, -1, 99, -2 ** 31]]], dtype=torch.int32, device="cuda")
    out = check_sparse(t, idx, 64, 1, ROW_TOL)
    twice = torch.tensor([[[0, 0], [2, 2]]], dtype=torch.int32, device="cuda")
    two = check_sparse(t, twice, 64, 1, ROW_TOL)
    once = check_sparse(t, twice[:, :, :1].contiguous(), 64, 1, ROW_TOL)
    assert torch.allclose(two["lse_hist"], once["lse_hist"] + np.log(2.0), atol=1e-5)
    none = check_sparse(t, idx[:, :, :0].contiguous(), 64, 1, ROW_TOL)
    assert torch.equal(none["o_full"], none["o_loc"]) and torch.equal(none["o_loc"], out["o_loc"])
    with pytest.raises(ValueError):
        ispa.block_sparse_attn(*t.values(), idx[:, :1].contiguous(), block=64)
    with pytest.raises(ispa.IspaError) as e:
        ispa.block_sparse_attn(*t.values(), idx[:, :1].contiguous(), block=64, q_block=2)
    assert e.value.status == ispa.ISPA_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype,n_q,q_block,n_hist,n_sel", [("bf16", 3, 1, 0, 2), ("bf16", 200, 128, 0, 2), ("fp32", 3, 2, 0, 2),
                                                            ("bf16", 0, 1, 10, 2), ("bf16", 0, 128, 10, 2)])
def test_sparse_empty_history_and_no_queries(cuda_ok, dtype, n_q, q_block, n_hist, n_sel):
    """An empty history with a list that names blocks anyway, and a call without queries."""
    import torch
    t, idx = sparse_case(dtype, 2, 64, n_q, q_block, 5, 70, n_hist, 64, n_sel, 66)
    idx.fill_(0)
    out = check_sparse(t, idx, 64, q_block, F32_TOL if dtype == "fp32" else ATTN_TOL) if n_q else None
    if out is not None:
        assert torch.isneginf(out["lse_hist"]).all()
    else:
        from kv_cache_compression_tma_b200 import ispa
        assert ispa.block_sparse_attn(*t.values(), idx, block=64, q_block=q_block)["o_loc"].shape == (0, 128)


@pytest.mark.parametrize("dtype,n_q,q_block,block", [("bf16", 2, 1, 64), ("fp32", 2, 1, 64), ("bf16", 130, 128, 64), ("bf16", 130, 128, 128),
                                                     ("bf16", 150, 128, 64), ("bf16", 200, 128, 128)])
def test_sparse_keys_that_score_minus_infinity(cuda_ok, dtype, n_q, q_block, block):
    """Keys whose products overflow to -inf (the first ones of a branch, too) weigh nothing; a history of
    nothing else gives lse_hist = -inf and O_full = O_loc."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    t, _ = sparse_case(dtype, 1, 64, n_q, q_block, 140, 20, 3 * block, block, 1, 68)
    t["q"].copy_(t["q"].abs() + 1)
    t["k_sink"][:130] = -3e38
    t["k_hist"][:2 * block] = -3e38
    groups = -(-n_q // q_block)
    idx = torch.tensor([[[0, 1, 2]] * (groups - 1) + [[0, 1, -1]]], dtype=torch.int32, device="cuda")
    out = ispa.block_sparse_attn(*t.values(), idx, block=block, q_block=q_block)
    clean = dict(t, k_sink=t["k_sink"][130:], v_sink=t["v_sink"][130:])
    last = torch.tensor([[[2]] * (groups - 1) + [[-1]]], dtype=torch.int32, device="cuda")
    want = ispa.block_sparse_attn(*clean.values(), last, block=block, q_block=q_block)
    tol = F32_TOL if dtype == "fp32" else ATTN_TOL
    for w in ("o_loc", "o_full", "d"):
        assert rel(host(out[w]), host(want[w])) <= tol[w], w
    for w in ("lse_loc", "lse_hist"):
        a, b = host(out[w]), host(want[w])
        assert np.array_equal(np.isneginf(a), np.isneginf(b)) and np.allclose(a[np.isfinite(b)], b[np.isfinite(b)], atol=tol[w])


@pytest.mark.parametrize("n_q,q_block", [(1, 1), (150, 128)])
def test_sparse_outputs_stay_inside_their_rows(cuda_ok, n_q, q_block):
    """Outputs that are views of wider, longer buffers: nothing outside them is written."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    t, idx = sparse_case("bf16", 2, 128, n_q, q_block, 5, 70, 300, 64, 3, 67)
    wide = {w: torch.full((n_q + 9, 256 + 16), 7.0, dtype=torch.bfloat16, device="cuda") for w in ("o_loc", "o_full", "d_out")}
    views = {w: x[4:4 + n_q, :256] for w, x in wide.items()}
    check_sparse(t, idx, 64, q_block, ATTN_TOL, **views)
    for x in wide.values():
        assert (x[:4] == 7).all() and (x[4 + n_q:] == 7).all() and (x[:, 256:] == 7).all()
    with pytest.raises(ValueError):
        ispa.block_sparse_attn(*t.values(), idx, block=64, q_block=q_block, o_loc=views["o_loc"][:, :255])
    for w in views:  # columns apart, a lone row's too
        with pytest.raises(ValueError):
            apart = torch.zeros((n_q, 512), dtype=torch.bfloat16, device="cuda")[:, ::2]
            ispa.block_sparse_attn(*t.values(), idx, block=64, q_block=q_block, **{w: apart})


# ------------------------------------------------------------------------------------------ far offsets
def test_offsets_past_32_bits(cuda_ok):
    """Token strides of 2^30 elements: the last of five tokens starts past 2^32 elements, 8 GB in."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    n, H, hd, ld = 5, 1, 64, 2 ** 30
    if torch.cuda.mem_get_info()[0] < 25e9:
        pytest.skip("needs 25 GB of free device memory")
    far = [torch.empty((n - 1) * ld + H * hd, dtype=torch.bfloat16, device="cuda").as_strided((n, H, hd), (ld, hd, 1)) for _ in range(2)]
    near = [tensor((n, H, hd), 68 + i, torch.bfloat16) for i in range(2)]
    for f, x in zip(far, near):
        f.copy_(x)
    for n_q in (3, 40):
        q = tensor((n_q, H, hd), 69, torch.bfloat16, 2.0)
        ll = lse_of(q, near[0])
        got, want = (ispa.attn_mass(q, k, ll, None, torch.zeros((H, n), device="cuda")) for k in (far[0], near[0]))
        assert torch.equal(got, want)
    idx = torch.tensor([[[0, 2]]], dtype=torch.int32, device="cuda")
    for dtype_q, q_block in ((3, 3), (130, 256)):
        q = tensor((dtype_q, H, hd), 69, torch.bfloat16, 2.0)
        a, b = (ispa.block_sparse_attn(q, *kv, *kv, *kv, idx, block=64 if q_block > 128 else 2, q_block=q_block,
                                       cuda_cores=q_block == 3) for kv in (far, near))
        assert all(torch.equal(a[w], b[w]) for w in a)
    means = [torch.zeros((3, H, hd), device="cuda") for _ in range(2)]
    ispa.block_means(far[0], means[0], 2)
    ispa.block_means(near[0], means[1], 2)
    assert torch.equal(*means)
    new = [tensor((2, H, hd), 70 + i, torch.bfloat16) for i in range(2)]
    state = [(torch.arange(n, device="cuda", dtype=torch.float32).flip(0)[None].contiguous(), torch.arange(n, dtype=torch.int32, device="cuda")[None].contiguous()) for _ in range(2)]
    for kv, (m, p) in zip((far, near), state):
        ispa.cache_insert(*kv, m, p, n, *new, torch.full((1, 2), 9.0, device="cuda"), n)
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1]) and torch.equal(state[0][0], state[1][0])
    assert torch.equal(near[0][4], new[0][1]) and torch.equal(near[0][3], new[0][0])


# ------------------------------------------------------------------------------------------ together
def test_streaming_loop_with_eviction_and_block_selection(cuda_ok):
    """Chunks stream through a MassCache of fixed size: attend, accumulate, insert; then a BlockIndex over
    the cache selects blocks for sparse attention.  Every step against the oracle on the same state."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    H, hd, cap, F = 2, 64, 200, 90
    mc = ispa.MassCache(H, hd, cap)
    sink = tensor((20, H, hd), 70, torch.bfloat16), tensor((20, H, hd), 71, torch.bfloat16)
    for step in range(4):
        s = 72 + 10 * step
        q, kc, vc = (tensor((F, H, hd), s + i, torch.bfloat16, sc) for i, sc in ((0, 2.0), (1, 1.0), (2, 1.0)))
        kh, vh = mc.segment()
        o = ispa.dual_stream_attn(q, *sink, kc, vc, kh, vh)
        before = host(mc.mass)[:, :mc.n]
        mc.accumulate(q, o["lse_loc"], o["lse_hist"], decay=0.9)
        want = orc.attn_mass(host(q), host(kh), host(o["lse_loc"]), host(o["lse_hist"]), before, 0.9)
        assert np.allclose(host(mc.mass)[:, :mc.n], want, rtol=MASS_TOL, atol=0)
        m_new = torch.zeros((H, F), device="cuda")
        ispa.attn_mass(q, kc, o["lse_loc"], o["lse_hist"], m_new, decay=0.0)
        n, mass, pos, old = mc.n, mc.mass.cpu().numpy(), mc.pos.cpu().numpy(), mc.k.clone()
        mc.insert(kc, vc, m_new, first=4, recent=10)
        src = orc.cache_insert(mass[:, :n], pos[:, :n], m_new.cpu().numpy(), step * F, cap, 4, step * F + F - 10)
        at = torch.from_numpy(src).cuda()
        want = torch.cat([old[:n], kc])[at, torch.arange(H, device="cuda")[:, None]].transpose(0, 1)
        assert mc.n == min(cap, (step + 1) * F) and torch.equal(mc.k[:mc.n], want)
        assert set(range(4)) <= set(mc.pos[0, :mc.n].cpu().tolist())
    kh, vh = mc.segment()
    bi = ispa.BlockIndex(H, hd, cap, block=64)
    bi.extend(kh[:100])
    bi.extend(kh)
    assert np.array_equal(bi.means.cpu().numpy(), orc.block_means(host(kh), 64).astype(np.float32))
    idx = bi.select(q[:1], 2)
    assert np.array_equal(idx.cpu().numpy(), orc.block_select(host(q[:1]), host(bi.means), 2, 1))
    t = dict(q=q[:1], ks=sink[0], vs=sink[1], kl=kc, vl=vc, kh=kh, vh=vh)
    check_sparse(t, idx, 64, 1, ROW_TOL)


@pytest.mark.parametrize("n_q,q_block", [(1, 1), (260, 128)])
def test_layer_forward_over_selected_blocks(cuda_ok, n_q, q_block):
    """llayer.layer_forward of an F-Layer with blocks: attention over the picks, then the projection; an
    L-Layer ignores them."""
    import torch
    from kv_cache_compression_tma_b200 import ispa, llayer
    H, hd = 2, 128
    t, _ = sparse_case("bf16", H, hd, n_q, q_block, 30, 140, 900, 64, 4, 74)
    bi = ispa.BlockIndex(H, hd, 1000, block=64)
    bi.extend(t["k_hist"])
    idx = bi.select(t["q"], 4, q_block=q_block)
    W = tensor((H * hd, 1, H * hd), 75, torch.bfloat16, 1 / 16.0).flatten(1)
    work = llayer.LayerWork(n_q + 40, H, hd, torch.bfloat16)
    y = llayer.layer_forward(*t.values(), W, llayer=False, work=work, blocks=idx, block=64, q_block=q_block)
    ref = orc.block_sparse(*(host(x) for x in t.values()), idx.cpu().numpy(), 64, q_block)
    # the attention output's rounding (2^-8) and error (1e-2 in norm at most) pass through W, Y rounds once more
    assert rel(host(y), ref["O_full"].reshape(n_q, -1) @ host(W)) <= 1.5e-2
    local = llayer.layer_forward(*t.values(), W, llayer=True, work=work, blocks=idx, block=64, q_block=q_block)
    assert rel(host(local), ref["O_loc"].reshape(n_q, -1) @ host(W)) <= 1.5e-2


def test_two_streams_at_once(cuda_ok):
    """The same calls on two streams, interleaved, on separate buffers: no state is shared."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    H, hd, n, n_q = 4, 128, 3000, 300
    sets = []
    for s in range(2):
        q, k, v = (tensor((m, H, hd), 95 + 3 * s + i, torch.bfloat16, sc) for i, (m, sc) in enumerate(((n_q, 2.0), (n, 1.0), (n, 1.0))))
        sets.append(dict(q=q, k=k, v=v, ll=torch.full((H, n_q), 8.0 + s, device="cuda"), means=torch.zeros((24, H, hd), device="cuda")))

    def step(x):
        ispa.block_means(x["k"], x["means"], 128)
        idx = ispa.block_select(x["q"], x["means"], 5, q_block=128)
        o = ispa.block_sparse_attn(x["q"], x["k"], x["v"], x["k"], x["v"], x["k"], x["v"], idx, block=128, q_block=128)
        m = ispa.attn_mass(x["q"], x["k"], x["ll"], None, torch.zeros((H, n), device="cuda"))
        k, v, pos = x["k"].clone(), x["v"].clone(), torch.arange(n, dtype=torch.int32, device="cuda").repeat(H, 1)
        ispa.cache_insert(k, v, m, pos, n, x["q"], x["q"], None, n, keep_from=n + 100)
        return [idx, m, k, pos, *o.values()]

    want = [step(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = step(sets[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))
    assert ispa.get_device_status() == ispa.ISPA_OK


def test_host_checks_of_the_binding(cuda_ok):
    """Host tensors, wrong shapes and types, heads that are not dense: refused before a launch."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    k, f = tensor((8, 2, 64), 1, torch.bfloat16), torch.zeros((2, 8), device="cuda")
    i = torch.zeros((2, 8), dtype=torch.int32, device="cuda")
    n0 = ispa.launch_count()
    bad = [lambda: ispa.attn_mass(k, k.cpu(), f, None, f), lambda: ispa.attn_mass(k, k, f, None, f[:, :7]),
           lambda: ispa.attn_mass(k, k.transpose(1, 2).contiguous().transpose(1, 2), f, None, f),
           lambda: ispa.attn_mass(k, k, f.double(), None, f), lambda: ispa.attn_mass(k, k[:, :1], f, None, f),
           lambda: ispa.cache_insert(k, k[:7], f, i, 8, k, k, None, 8), lambda: ispa.cache_insert(k, k, f, i[:, :7], 8, k, k, None, 8),
           lambda: ispa.cache_insert(k, k, f, i, 8, k.float(), k, None, 8), lambda: ispa.cache_insert(k, k, f[:, :4], i[:, :4], 4, k, k, None, 8),
           lambda: ispa.block_means(k, torch.zeros((1, 2, 64), device="cuda"), 4), lambda: ispa.block_select(k, k.float(), 2, out=i[:, :1]),
           lambda: ispa.block_sparse_attn(k, k, k[:7], k, k, k, k, i[:, :8, None].contiguous(), block=4),
           lambda: ispa.block_sparse_attn(k, k, k, k, k, k, k, i[:, :8, None].contiguous().long(), block=4),
           lambda: ispa.block_means(k, torch.zeros((8, 2, 64), device="cuda"), 0), lambda: ispa.block_select(k, k.float(), 2, q_block=0),
           lambda: ispa.block_sparse_attn(k, k, k, k, k, k, k, i[:, :8, None].contiguous(), block=4, q_block=0),
           lambda: ispa.BlockIndex(2, 64, 64, block=0), lambda: ispa.MassCache(2, 64, 8).insert(k, k, first=4, recent=5)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    bi = ispa.BlockIndex(2, 64, 64, block=4)
    bi.extend(k)
    with pytest.raises(ValueError):
        bi.extend(k[:5])
    bi.reset()
    bi.extend(k[:5])
    assert bi.select(k, 3).shape == (2, 8, 3) and ispa.launch_count() == n0 + 3


def test_a_lone_head_has_no_row_stride(cuda_ok):
    """With one head the arrays of a call may differ in width."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    k, kn = tensor((6, 1, 64), 1, torch.bfloat16), tensor((3, 1, 64), 2, torch.bfloat16)
    lse, mass = torch.full((1, 3), 4.0, device="cuda"), torch.zeros((1, 9), device="cuda")
    out = ispa.attn_mass(kn, k, lse, None, mass, mass_out=torch.zeros((1, 7), device="cuda"))
    assert torch.equal(out[:, :6], ispa.attn_mass(kn, k, lse, None, mass)[:, :6])
    pos = torch.arange(7, dtype=torch.int32, device="cuda")[None]
    for m in (mass, mass[:, :6].clone()):  # the state back in place, rows of 9, 6 and 7
        cache, want = k.clone(), k.clone()
        m[0, :6] = torch.tensor([3.0, 0.0, 5.0, 1.0, 4.0, 2.0], device="cuda")
        p = pos.clone()
        assert ispa.cache_insert(cache, cache.clone(), m, p, 6, kn[:2], kn[:2], torch.full((1, 2), 9.0, device="cuda"), 6) == 6
        want[1], want[3] = kn[0], kn[1]
        assert torch.equal(cache, want) and p[0].tolist() == [0, 6, 2, 7, 4, 5, 6]


def test_results_of_a_call_on_a_stream_come_from_its_memory(cuda_ok):
    """A call given a stream allocates from that stream's memory: nothing that another stream still uses is
    written, and what the call drops is not handed out before its kernels are done."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    t, idx = sparse_case("bf16", 2, 128, 3, 1, 5, 70, 300, 64, 3, 69)
    means = ispa.block_means(t["k_hist"], torch.zeros((5, 2, 128), device="cuda"), 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = ispa.block_sparse_attn(*t.values(), idx, block=64, stream=side)
    out["idx"] = ispa.block_select(t["q"], means, 3, stream=side)
    side.synchronize()
    owner = {b["address"]: s["stream"] for s in torch.cuda.memory_snapshot() for b in s["blocks"]}
    assert all(owner[x.data_ptr()] == side.cuda_stream for x in out.values())


def test_captured_and_on_another_stream(cuda_ok):
    """All five calls captured once and replayed on new values in the same buffers, and run eagerly on a
    side stream: the same bits as eager calls on the current stream."""
    import torch
    from kv_cache_compression_tma_b200 import ispa
    H, hd, cap, n_new = 2, 128, 600, 50
    q, k, v = tensor((8, H, hd), 80, torch.bfloat16, 2.0), tensor((cap, H, hd), 81, torch.bfloat16), tensor((cap, H, hd), 82, torch.bfloat16)
    kn, vn = tensor((n_new, H, hd), 83, torch.bfloat16), tensor((n_new, H, hd), 84, torch.bfloat16)
    mass, pos = torch.rand((H, cap), device="cuda"), torch.arange(cap, dtype=torch.int32, device="cuda").repeat(H, 1)
    out = {w: torch.zeros((8, H * hd), dtype=torch.bfloat16, device="cuda") for w in ("o_loc", "o_full", "d_out")}
    out.update({w: torch.zeros((H, 8), device="cuda") for w in ("lse_loc", "lse_hist")})
    means, idx = torch.zeros((10, H, hd), device="cuda"), torch.zeros((H, 8, 3), dtype=torch.int32, device="cuda")
    buffers = [k, v, mass, pos, means, idx, *out.values()]

    def step():
        ispa.block_means(k, means, 64)
        ispa.block_select(q, means, 3, out=idx)
        ispa.block_sparse_attn(q, kn, vn, kn, vn, k, v, idx, block=64, **out)
        ispa.attn_mass(q, k, out["lse_loc"], out["lse_hist"], mass, decay=0.5)
        ispa.cache_insert(k, v, mass, pos, cap, kn, vn, None, cap, keep_from=cap + 20)

    start = [b.clone() for b in buffers]
    reset = lambda: [b.copy_(s) for b, s in zip(buffers, start)]
    step()
    torch.cuda.synchronize()
    want = [b.clone() for b in buffers]
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(buffers, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(buffers, want))
    assert ispa.get_device_status() == ispa.ISPA_OK
