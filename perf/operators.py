"""Measured cases of the bounded-history operators: the attention weight each cached key collects, the
insertion of new tokens into a cache of fixed size by that weight, the selection of history blocks by
a cheap score, and dual-stream attention over the selected blocks.

`run` computes an operator either in its plain form (elementary torch operations, 32-bit arithmetic,
64-bit for the means and scores that decide a selection) or, where `own` is true, through the
package's calls.  Sizes are those of the repository's workloads: latent frames of 1560 tokens, chunks
of 4680 queries, histories of 9 to 120 frames, 12 or 40 heads of 128, and the fp32 layer of 2 heads of 32.
"""
import math

import numpy as np
import torch

own = False  # set by the caller: False = plain form, True = the package's operators

FRAME = 1560
CHUNK = 4680


def listed():
    return [
        # one generated token against a 9-frame history of a 40-head layer: latency and one read of K
        {"name": "mass token 40h", "op": "mass", "dtype": "bf16", "H": 40, "hd": 128, "n_q": 1, "n_k": 14040,
         "biased": False, "decay": 0.99},
        # a warmup-sized chunk over a merged (biased) history of the 12-head layer
        {"name": "mass chunk 12h", "op": "mass", "dtype": "bf16", "H": 12, "hd": 128, "n_q": CHUNK, "n_k": 14040,
         "biased": True, "decay": 1.0},
        # the same chunk on the 40-head layer: the largest product of the set
        {"name": "mass chunk 40h", "op": "mass", "dtype": "bf16", "H": 40, "hd": 128, "n_q": CHUNK, "n_k": 14040,
         "biased": False, "decay": 0.9},
        # the fp32 layer: smallest call, odd key count
        {"name": "mass fp32 2h", "op": "mass", "dtype": "fp32", "H": 2, "hd": 32, "n_q": 64, "n_k": 95,
         "biased": False, "decay": 0.0},
        # one generated token enters a full 14040-entry cache: one entry per head leaves
        {"name": "insert token 40h", "op": "insert", "dtype": "bf16", "H": 40, "hd": 128, "capacity": 14040,
         "n": 14040, "n_new": 1, "recent": 1},
        # a chunk enters a full 120-frame cache, the newest frame protected
        {"name": "insert chunk 12h long", "op": "insert", "dtype": "bf16", "H": 12, "hd": 128, "capacity": 187200,
         "n": 187200, "n_new": CHUNK, "recent": FRAME},
        # one token selects among the blocks of a 120-frame history (its own block's mean refreshed)
        {"name": "select token 40h", "op": "select", "dtype": "bf16", "H": 40, "hd": 128, "n_q": 1, "q_block": 1,
         "n_k": 187200, "n_new": 1, "block": 128, "n_sel": 32},
        # a chunk selects per 128 query rows after three new frames joined a 120-frame history
        {"name": "select chunk 12h", "op": "select", "dtype": "bf16", "H": 12, "hd": 128, "n_q": CHUNK, "q_block": 128,
         "n_k": 187200, "n_new": CHUNK, "block": 128, "n_sel": 64},
        # one token attends over sink, its frame and 64 selected 64-key blocks of a 120-frame history
        {"name": "sparse token 40h", "op": "sparse", "dtype": "bf16", "H": 40, "hd": 128, "n_q": 1, "q_block": 1,
         "n_sink": FRAME, "n_loc": FRAME, "n_hist": 187200, "block": 64, "n_sel": 64},
        # a chunk attends over 64 selected blocks of 128 keys of a 120-frame history
        {"name": "sparse chunk 12h long", "op": "sparse", "dtype": "bf16", "H": 12, "hd": 128, "n_q": CHUNK,
         "q_block": 128, "n_sink": FRAME, "n_loc": CHUNK, "n_hist": 187200, "block": 128, "n_sel": 64},
        # the same on the 40-head layer with a quarter of its 9-frame history
        {"name": "sparse chunk 40h", "op": "sparse", "dtype": "bf16", "H": 40, "hd": 128, "n_q": CHUNK, "q_block": 128,
         "n_sink": FRAME, "n_loc": CHUNK, "n_hist": 14040, "block": 64, "n_sel": 56},
        # the fp32 layer: 64 rows, 96 history keys in blocks of 32, more picks than some rows have
        {"name": "sparse fp32 2h", "op": "sparse", "dtype": "fp32", "H": 2, "hd": 32, "n_q": 64, "q_block": 32,
         "n_sink": 16, "n_loc": 32, "n_hist": 95, "block": 32, "n_sel": 2},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["mass", "insert", "select", "sparse"])
    f32 = rng.random() < 0.2
    c = {"op": op, "dtype": "fp32" if f32 else "bf16", "H": rng.choice([1, 2, 3, 5, 12, 40]),
         "hd": rng.choice([16, 32, 64, 128]) if f32 and op in ("mass", "sparse") else rng.choice([64, 128])}
    if op == "mass":
        c.update(n_q=log(1, 128 if f32 else CHUNK), n_k=log(1, 2000 if f32 else 14040),
                 biased=rng.random() < 0.4, decay=rng.choice([0.0, 0.5, 0.97, 1.0]))
    elif op == "insert":
        cap = log(2, 40000 if c["H"] == 40 else 187200)
        n_new = log(1, CHUNK)
        c.update(capacity=cap, n=cap if rng.random() < 0.7 else rng.randint(0, cap), n_new=n_new,
                 recent=rng.randint(0, min(n_new, FRAME)))
    elif op == "select":
        qb = rng.choice([1, 128])
        n_k = log(1, 187200)
        c.update(n_q=log(1, 16) if qb == 1 else log(1, CHUNK), q_block=qb, n_k=n_k, n_new=rng.randint(1, min(n_k, CHUNK)),
                 block=rng.choice([64, 128]), n_sel=log(1, 128))
    elif f32:
        c.update(n_q=log(1, 300), q_block=rng.choice([1, 32]), n_sink=rng.randint(0, 40), n_loc=rng.randint(1, 200),
                 n_hist=log(1, 2000), block=rng.choice([16, 32]), n_sel=log(1, 24))
    else:
        qb = rng.choice([1, 128])
        c.update(n_q=log(1, 16) if qb == 1 else log(1, CHUNK), q_block=qb, n_sink=rng.randint(0, FRAME),
                 n_loc=log(1, CHUNK), n_hist=log(1, 187200 if c["H"] < 40 else 14040), block=rng.choice([64, 128]),
                 n_sel=log(1, 64 if c["H"] < 40 else 28))
    return c


# ---------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _cache(n, H, hd, dt, g):
    """n cached keys or values: frames of tokens that repeat, with noise, the frame before (rho 0.9)."""
    base = torch.randn((min(FRAME, max(n, 1)), H, hd), generator=g, device="cuda")
    out = torch.empty((n, H, hd), dtype=dt, device="cuda")
    for f in range(0, n, FRAME):
        m = min(FRAME, n - f)
        noise = torch.randn((m, H, hd), generator=g, device="cuda")
        out[f:f + m] = (math.sqrt(0.9) * base[:m] + math.sqrt(0.1) * noise).to(dt)
    return out


def _query(n, H, hd, dt, g):
    """Queries whose scaled logits against unit-variance keys have a standard deviation of about 2."""
    return (2.0 * torch.randn((n, H, hd), generator=g, device="cuda")).to(dt)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    H, hd, dt = case["H"], case["hd"], _dtype(case)
    st = dict(case)
    if case["op"] == "mass":
        n_q, n_k = case["n_q"], case["n_k"]
        q, k = _query(n_q, H, hd, dt, g), _cache(n_k, H, hd, dt, g)
        bias = None
        if case["biased"]:  # log group sizes of a merged cache, some slots empty
            bias = torch.log(torch.randint(1, 6, (H, n_k), generator=g, device="cuda").float())
            bias[torch.rand((H, n_k), generator=g, device="cuda") < 0.05] = -math.inf
        lse_hist = torch.empty((H, n_q), dtype=torch.float32, device="cuda")
        for h in range(H):
            s = (q[:, h] @ k[:, h].T).float() / math.sqrt(hd)
            lse_hist[h] = torch.logsumexp(s if bias is None else s + bias[h], dim=1)
        # the local branch: a chunk and a sink, about half of the history's keys
        lse_loc = 2.0 + math.log(n_k * 0.5 + 1) + 0.3 * torch.randn((H, n_q), generator=g, device="cuda")
        mass = torch.rand((H, n_k), generator=g, device="cuda") * 2 * n_q / n_k
        st.update(q=q, k=k, bias=bias, lse_loc=lse_loc, lse_hist=lse_hist, mass=mass, mass_out=torch.empty_like(mass))
    elif case["op"] == "insert":
        cap, n, n_new = case["capacity"], case["n"], case["n_new"]
        weight = lambda m: torch.where(torch.rand((H, m), generator=g, device="cuda") < 0.02, 0.0,
                                       torch.exp(1.5 * torch.randn((H, m), generator=g, device="cuda")))
        first = 4 * cap  # positions seen so far: the held entries are a quarter of them
        pos = torch.argsort(torch.rand((H, first), generator=g, device="cuda"), dim=1)[:, :cap].to(torch.int32)
        st.update(k=_cache(cap, H, hd, dt, g), v=_cache(cap, H, hd, dt, g), mass=weight(cap), pos=pos.contiguous(),
                  k_new=_cache(n_new, H, hd, dt, g), v_new=_cache(n_new, H, hd, dt, g), mass_new=weight(n_new),
                  pos_new=first, keep_below=16, keep_from=first + n_new - case["recent"],
                  mass_out=torch.zeros((H, cap), dtype=torch.float32, device="cuda"),
                  pos_out=torch.zeros((H, cap), dtype=torch.int32, device="cuda"))
    elif case["op"] == "select":
        n_k, block = case["n_k"], case["block"]
        k = _cache(n_k, H, hd, dt, g)
        n_blocks = -(-n_k // block)
        first = (n_k - case["n_new"]) // block  # the first block that the new tokens touch
        means = torch.empty((n_blocks, H, hd), dtype=torch.float32, device="cuda")
        for b in range(0, first, 64):  # the blocks pooled by earlier steps
            e = min(first, b + 64)
            means[b:e] = k[b * block:e * block].view(e - b, block, H, hd).double().mean(1).float()
        means[first:] = 0
        st.update(q=_query(case["n_q"], H, hd, dt, g), k=k, means=means, first=first,
                  idx=torch.empty((H, -(-case["n_q"] // case["q_block"]), case["n_sel"]), dtype=torch.int32,
                                  device="cuda"))
    else:
        n_q = case["n_q"]
        n_blocks, groups = -(-case["n_hist"] // case["block"]), -(-n_q // case["q_block"])
        S = case["n_sel"]
        pick = torch.argsort(torch.rand((H, groups, n_blocks), generator=g, device="cuda"), dim=2)[:, :, :S]
        idx = torch.full((H, groups, S), n_blocks, dtype=torch.int64, device="cuda")
        idx[:, :, :pick.shape[2]] = pick
        # some groups pick fewer blocks, a few none at all
        fewer = torch.randint(0, S + 1, (H, groups, 1), generator=g, device="cuda")
        fewer[torch.rand((H, groups, 1), generator=g, device="cuda") < 0.9] = S
        idx[torch.arange(S, device="cuda").expand(H, groups, S) >= fewer] = n_blocks
        idx = idx.sort(dim=2).values
        idx[idx == n_blocks] = -1
        st.update(q=_query(n_q, H, hd, dt, g), idx=idx.to(torch.int32).contiguous())
        for name in ("sink", "loc", "hist"):
            st["k_" + name] = _cache(case["n_" + name], H, hd, dt, g)
            st["v_" + name] = _cache(case["n_" + name], H, hd, dt, g)
        st["out"] = {w: torch.empty((n_q, H * hd), dtype=dt, device="cuda") for w in ("o_loc", "o_full", "d_out")}
        st["out"].update({w: torch.empty((H, n_q), dtype=torch.float32, device="cuda") for w in ("lse_loc", "lse_hist")})
    return st


# ---------------------------------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"mass": _plain_mass, "insert": _plain_insert, "select": _plain_select, "sparse": _plain_sparse}[state["op"]](state)


def _run_own(s):
    import kv_cache_compression_tma_b200 as ispa
    if s["op"] == "mass":
        return ispa.attn_mass(s["q"], s["k"], s["lse_loc"], s["lse_hist"], s["mass"], kv_bias=s["bias"],
                              decay=s["decay"], mass_out=s["mass_out"])
    if s["op"] == "insert":
        n = ispa.cache_insert(s["k"], s["v"], s["mass"], s["pos"], s["n"], s["k_new"], s["v_new"], s["mass_new"],
                              s["pos_new"], keep_below=s["keep_below"], keep_from=s["keep_from"],
                              mass_out=s["mass_out"], pos_out=s["pos_out"])
        return s["k"][:n], s["v"][:n], s["mass_out"][:, :n], s["pos_out"][:, :n]
    if s["op"] == "select":
        ispa.block_means(s["k"], s["means"], s["block"], first=s["first"])
        return s["means"], ispa.block_select(s["q"], s["means"], s["n_sel"], q_block=s["q_block"], out=s["idx"])
    o = ispa.block_sparse_attn(s["q"], s["k_sink"], s["v_sink"], s["k_loc"], s["v_loc"], s["k_hist"], s["v_hist"],
                               s["idx"], block=s["block"], q_block=s["q_block"], **s["out"])
    return o["o_loc"], o["o_full"], o["d"], o["lse_loc"], o["lse_hist"]


def _plain_mass(s):
    q, k = s["q"].float().transpose(0, 1), s["k"].float().transpose(0, 1)
    w = torch.matmul(q / math.sqrt(s["hd"]), k.transpose(1, 2))
    w -= torch.logaddexp(s["lse_loc"], s["lse_hist"])[:, :, None]
    if s["bias"] is not None:
        w += s["bias"][:, None, :]
    return s["decay"] * s["mass"] + w.exp_().sum(1)


def _plain_insert(s):
    cap, n, n_new = s["capacity"], s["n"], s["n_new"]
    H, dev = s["H"], s["k"].device
    pos_new = s["pos_new"] + torch.arange(n_new, dtype=torch.int32, device=dev).expand(H, n_new)
    mass = torch.cat([s["mass"][:, :n], s["mass_new"]], 1)
    pos = torch.cat([s["pos"][:, :n], pos_new], 1)
    key = torch.where(mass.isnan(), -math.inf, mass)
    key = torch.where((pos < s["keep_below"]) | (pos >= s["keep_from"]), math.inf, key)
    order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :cap]
    kept = torch.zeros_like(key, dtype=torch.bool).scatter_(1, order, True)
    moved = kept[:, n:]  # surviving new tokens, and the slots they take: the evicted ones, then unused ones
    free = torch.ones((H, cap), dtype=torch.bool, device=dev)
    free[:, :n] = ~kept[:, :n]
    free &= free.cumsum(1) <= moved.sum(1, keepdim=True)
    fh, fs = free.nonzero(as_tuple=True)
    th, t = moved.nonzero(as_tuple=True)
    s["k"][fs, fh] = s["k_new"][t, th]
    s["v"][fs, fh] = s["v_new"][t, th]
    total = min(cap, n + n_new)
    mass_out, pos_out = s["mass"].clone(), s["pos"].clone()
    mass_out[fh, fs] = s["mass_new"][th, t]
    pos_out[fh, fs] = pos_new[th, t]
    return s["k"][:total], s["v"][:total], mass_out[:, :total], pos_out[:, :total]


def _group_mean(x, size):
    """Mean over groups of `size` rows (the last one shorter) in 64 bits."""
    n, groups = x.shape[0], -(-x.shape[0] // size)
    x = torch.nn.functional.pad(x.double(), (0, 0, 0, 0, 0, groups * size - n)).view(groups, size, *x.shape[1:])
    rows = torch.full((groups, 1, 1), size, dtype=torch.float64, device=x.device)
    rows[-1] = n - (groups - 1) * size
    return x.sum(1) / rows


def _plain_select(s):
    s["means"][s["first"]:] = _group_mean(s["k"][s["first"] * s["block"]:], s["block"]).float()
    # 64 bits: a pick must not hang on the order of a sum
    score = torch.matmul(_group_mean(s["q"], s["q_block"]).transpose(0, 1), s["means"].double().permute(1, 2, 0))
    order = torch.argsort(score, dim=2, descending=True, stable=True)[:, :, :s["n_sel"]].sort(dim=2).values
    idx = torch.full_like(s["idx"], -1)
    idx[:, :, :order.shape[2]] = order.to(torch.int32)
    return s["means"], idx


def _plain_sparse(s):
    H, hd, n_q, qb, block = s["H"], s["hd"], s["n_q"], s["q_block"], s["block"]
    idx = s["idx"].long()
    G, S = idx.shape[1], idx.shape[2]
    q = s["q"].float() / math.sqrt(hd)
    qh = q.transpose(0, 1)
    k = torch.cat([s["k_sink"], s["k_loc"]]).float().transpose(0, 1)
    v = torch.cat([s["v_sink"], s["v_loc"]]).float().transpose(0, 1)
    a = torch.matmul(qh, k.transpose(1, 2))
    m = a.amax(2, keepdim=True)
    a = (a - m).exp_()
    l_loc = a.sum(2)
    o_loc = torch.matmul(a, v) / l_loc[:, :, None]
    lse_loc = m[:, :, 0] + l_loc.log()
    del a
    key = idx[..., None] * block + torch.arange(block, device=idx.device)
    live = ((idx[..., None] >= 0) & (key < s["n_hist"])).view(H, G, 1, S * block)
    key = key.clamp(0, s["n_hist"] - 1).view(H, G, S * block)
    head = torch.arange(H, device=idx.device)[:, None, None]
    qg = torch.nn.functional.pad(qh, (0, 0, 0, G * qb - n_q)).view(H, G, qb, hd)
    a = torch.matmul(qg, s["k_hist"][key, head].float().transpose(2, 3))
    a = a.masked_fill_(~live, -math.inf)
    m = a.amax(3, keepdim=True)
    a = (a - m.clamp_min(-1e30)).exp_()
    l_hist = a.sum(3)
    o_hist = torch.matmul(a, s["v_hist"][key, head].float()) / l_hist.clamp_min(1e-30)[..., None]
    lse_hist = (m[..., 0] + l_hist.log()).view(H, G * qb)[:, :n_q]
    o_hist = o_hist.view(H, G * qb, hd)[:, :n_q]
    w = 1.0 / (1.0 + torch.exp(lse_loc - lse_hist))  # the history's share; 0 where it has no key
    o_full = o_loc + w[:, :, None] * (o_hist - o_loc)
    dt = s["q"].dtype
    flat = lambda x: x.transpose(0, 1).reshape(n_q, H * hd).to(dt)
    return flat(o_loc), flat(o_full), flat(o_full - o_loc), lse_loc, lse_hist


# ---------------------------------------------------------------------------------------- work
def work(case):
    H, hd = case["H"], case["hd"]
    es = 2 if case["dtype"] == "bf16" else 4
    row = H * hd * es
    if case["op"] == "mass":
        n_q, n_k = case["n_q"], case["n_k"]
        return {"bytes": (n_q + n_k) * row + 8 * H * n_q + (12 if case["biased"] else 8) * H * n_k,
                "flops": 2.0 * H * n_q * n_k * hd}
    if case["op"] == "insert":
        cap, n, n_new = case["capacity"], case["n"], case["n_new"]
        total = n + n_new
        # of the unprotected new tokens the expected share survives; each survivor's K and V row is read and written
        stay = case["recent"] + (n_new - case["recent"]) * min(1.0, cap / total)
        return {"bytes": H * (8 * total + 8 * min(cap, total)) + stay * row * 4, "flops": 0.0}
    if case["op"] == "select":
        blocks, groups = -(-case["n_k"] // case["block"]), -(-case["n_q"] // case["q_block"])
        fresh = case["n_k"] - (case["n_k"] - case["n_new"]) // case["block"] * case["block"]
        return {"bytes": fresh * row + blocks * H * hd * 4 + case["n_q"] * row + 4.0 * H * groups * case["n_sel"],
                "flops": 2.0 * H * hd * groups * blocks}
    groups = -(-case["n_q"] // case["q_block"])
    loc, sel = case["n_sink"] + case["n_loc"], min(case["n_sel"] * case["block"], case["n_hist"])
    hist = min(case["n_hist"], groups * sel)  # each history key read once at most
    return {"bytes": 2 * (loc + hist) * row + 4 * case["n_q"] * row + 8 * H * case["n_q"],
            "flops": 4.0 * H * hd * case["n_q"] * (loc + sel)}


# ---------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"mass": _exact_mass, "insert": _exact_insert, "select": _exact_select, "sparse": _exact_sparse}[case["op"]](s)


def _exact_mass(s):
    out = s["decay"] * s["mass"].double()
    for h in range(s["H"]):
        z = torch.exp(s["lse_loc"][h].double()) + torch.exp(s["lse_hist"][h].double())
        e = torch.exp((s["k"][:, h].double() @ s["q"][:, h].double().T) / math.sqrt(s["hd"]))
        w = e @ (1.0 / z)
        out[h] += w if s["bias"] is None else w * torch.exp(s["bias"][h].double())
    return out


def _exact_insert(s):
    cap, n, n_new, H = s["capacity"], s["n"], s["n_new"], s["H"]
    total = min(cap, n + n_new)
    mass, pos = s["mass"].double().cpu().numpy(), s["pos"].cpu().numpy()
    mass_new = s["mass_new"].double().cpu().numpy()
    pos_new = s["pos_new"] + np.arange(n_new)
    src = np.tile(np.arange(total), (H, 1))  # which candidate ends in each slot
    for h in range(H):
        m = np.concatenate([mass[h, :n], mass_new[h]])
        p = np.concatenate([pos[h, :n], pos_new])
        m[np.isnan(m)] = -np.inf
        m[(p < s["keep_below"]) | (p >= s["keep_from"])] = np.inf
        leave = np.lexsort((-np.arange(n + n_new), m))[:n + n_new - total]
        gone = set(leave.tolist())
        holes = sorted(i for i in gone if i < n) + list(range(n, total))
        enter = [i for i in range(n, n + n_new) if i not in gone]
        src[h, holes] = enter
    at = torch.from_numpy(src).to(s["k"].device)
    head = torch.arange(H, device=at.device)[:, None]
    pick = lambda a, b: torch.cat([a[:n], b])[at, head].transpose(0, 1).double()
    mass_all = torch.cat([s["mass"][:, :n], s["mass_new"]], 1).double()
    pos_all = torch.cat([s["pos"][:, :n].long(), torch.from_numpy(pos_new).to(at.device).expand(H, n_new)], 1)
    return (pick(s["k"], s["k_new"]), pick(s["v"], s["v_new"]), mass_all.gather(1, at),
            pos_all.gather(1, at).to(torch.int32))


def _exact_select(s):
    block, n_k = s["block"], s["n_k"]
    means = s["means"].double()
    for b in range(s["first"], means.shape[0]):
        means[b] = s["k"][b * block:min(n_k, (b + 1) * block)].double().mean(0)
    return means, None  # the picks are whole numbers


def _exact_sparse(s):
    H, hd, n_q, qb, block, n_hist = s["H"], s["hd"], s["n_q"], s["q_block"], s["block"], s["n_hist"]
    o = [torch.zeros((n_q, H, hd), dtype=torch.float64, device="cuda") for _ in range(3)]
    lse = [torch.zeros((H, n_q), dtype=torch.float64, device="cuda") for _ in range(2)]
    picks = s["idx"].cpu().numpy()
    for h in range(H):
        k = torch.cat([s["k_sink"][:, h], s["k_loc"][:, h]]).double()
        v = torch.cat([s["v_sink"][:, h], s["v_loc"][:, h]]).double()
        for g in range(picks.shape[1]):
            r0, r1 = g * qb, min(n_q, (g + 1) * qb)
            rows = [np.arange(b * block, min(n_hist, (b + 1) * block)) for b in picks[h, g] if b >= 0]
            rows = torch.from_numpy(np.concatenate(rows + [np.zeros(0, np.int64)])).to("cuda")
            q = s["q"][r0:r1, h].double() / math.sqrt(hd)
            kh, vh = s["k_hist"][rows, h].double(), s["v_hist"][rows, h].double()
            a, b = torch.exp(q @ k.T), torch.exp(q @ kh.T)
            za, zb = a.sum(1), b.sum(1)
            loc = (a @ v) / za[:, None]
            full = (a @ v + b @ vh) / (za + zb)[:, None]
            o[0][r0:r1, h], o[1][r0:r1, h], o[2][r0:r1, h] = loc, full, full - loc
            lse[0][h, r0:r1], lse[1][h, r0:r1] = za.log(), zb.log()
    return tuple(x.reshape(n_q, H * hd) for x in o) + tuple(lse)
