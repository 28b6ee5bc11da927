"""Token mixers beside the gated delta rule: measured cases and their plain forms.

Three operators:
* linear attention with a decay for each head ("lin"): a decode step, the chunked forward, and a training pass (forward
  and gradients);
* appending keys and values to a paged cache, with the position rotation on the way ("append");
* attention of one new token for each sequence over that cache ("attn").

With ``own`` false, ``run`` computes each in elementary torch operations in 32 bits, rounded once at the end; with
``own`` true it calls the library.  ``exact`` computes the same from the definitions in 64 bits, token by token.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_LIN_MOST = 65536 * 32 * 128          # elements of v in the largest chunked case
_KV_MOST = 256 * 8192 * 8 * 128       # elements of the longest key cache


# ----------------------------------------------------------------------------------------------------------------
# cases

def _lin(name, mode, B, T, Hk, H, dk, dv, dtype="bf16", n_seqs=0, gate="token", h0=True, fused=True):
    # mode: "step" (B sequences, one token each), "fwd", or "train" (forward and gradients)
    # gate: "token" (a decay for each token and head) or "head" (one for each head); fused: q, k, v side by side
    return {"name": name, "op": "lin", "mode": mode, "B": B, "T": T, "Hk": Hk, "H": H, "dk": dk, "dv": dv,
            "dtype": dtype, "n_seqs": n_seqs, "gate": gate, "h0": h0, "fused": fused}


def _append(name, N, T, Hq, Hk, d, page, context, rot, dtype="bf16", interleaved=False, with_q=True):
    # T: new tokens in all (N for a decode step, one each); context: the most tokens of a sequence after the call
    return {"name": name, "op": "append", "N": N, "T": T, "Hq": Hq, "Hk": Hk, "d": d, "page": page,
            "context": context, "rot": rot, "dtype": dtype, "interleaved": interleaved, "with_q": with_q}


def _attn(name, N, Hq, Hk, d, page, context, dtype="bf16", ragged=True):
    return {"name": name, "op": "attn", "N": N, "Hq": Hq, "Hk": Hk, "d": d, "page": page, "context": context,
            "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # one sequence being decoded, 16 heads: the smallest call, where latency counts
        _lin("lin_step_n1_h16_d128", "step", 1, 1, 16, 16, 128, 128),
        # 256 sequences being decoded, 32 heads: the shape of the delta rule's decode workload
        _lin("lin_step_n256_h32_d128", "step", 256, 1, 32, 32, 128, 128),
        # a prompt of an odd length on one sequence, two value heads a key head
        _lin("lin_fwd_prompt_b1_t1000_h16", "fwd", 1, 1000, 8, 16, 128, 128),
        # prefill at the shape of the delta rule's headline workload
        _lin("lin_fwd_b4_t4096_h16_d128", "fwd", 4, 4096, 16, 16, 128, 128),
        # a packed batch of eight documents, 32 heads: the largest
        _lin("lin_fwd_packed_65536tok_h32", "fwd", 1, 65536, 32, 32, 128, 128, n_seqs=8),
        # a training step at the headline shape, a constant decay for each head
        _lin("lin_train_b4_t4096_h16_d128", "train", 4, 4096, 16, 16, 128, 128, gate="head", h0=False),
        # a packed training batch, decays of every token, grouped value heads
        _lin("lin_train_packed_32768tok_h16", "train", 1, 32768, 8, 16, 128, 128, n_seqs=5),
        # odd head sizes in fp32
        _lin("lin_train_b2_t777_h3_d40_f32", "train", 2, 777, 3, 3, 40, 72, dtype="f32", fused=False),
        # a decode step: 256 sequences, one token each
        _append("append_decode_n256", 256, 256, 32, 8, 128, 64, 4096, 128),
        # ragged prompts of 32 sequences written behind what they have already
        _append("append_prompts_16384tok", 32, 16384, 32, 8, 128, 64, 4096, 64),
        # one sequence with a long context: little to spread over the card but its length
        _attn("attn_n1_ctx32768_h32_8", 1, 32, 8, 128, 64, 32768, ragged=False),
        # 256 sequences of ragged lengths
        _attn("attn_n256_ctx8192_h32_8", 256, 32, 8, 128, 64, 8192),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["lin", "lin", "lin", "append", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "lin":
        mode = rng.choice(["step", "fwd", "fwd", "train"])
        if dtype == "bf16":
            dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (96, 96),
                                 (8 * rng.randint(1, 16), 8 * rng.randint(1, 16))])
            most = _LIN_MOST // 4
        else:
            dk, dv = rng.choice([(64, 64), (128, 128), (rng.randint(1, 128), rng.randint(1, 128))])
            most = _LIN_MOST // 64
        Hk = _log_int(rng, 1, 32)
        H = min(64, Hk * rng.choice([1, 1, 2, 4]))
        Hk = H if H % Hk else Hk
        gate, h0, fused = rng.choice(["token", "token", "head"]), rng.random() < 0.6, rng.random() < 0.5
        if mode == "step":
            return _lin("drawn", mode, _log_int(rng, 1, max(1, min(512, 2 ** 28 // (H * dk * dv)))), 1, Hk, H, dk, dv,
                        dtype, 0, gate, True, fused)
        most //= H * max(dk, dv)
        if rng.random() < 0.5:
            return _lin("drawn", mode, 1, _log_int(rng, 1, max(2, min(65536, most))), Hk, H, dk, dv, dtype,
                        _log_int(rng, 1, 24), gate, h0, fused)
        B = _log_int(rng, 1, 16)
        return _lin("drawn", mode, B, _log_int(rng, 1, max(2, min(16384, most // B))), Hk, H, dk, dv, dtype, 0, gate,
                    h0, fused)
    d = rng.choice([64, 128, 128, 256, 80, 8 * rng.randint(1, 32)])
    Hk = _log_int(rng, 1, 16)
    Hq = Hk * rng.choice([1, 2, 4, 5, 8, 16])
    page = rng.choice([16, 32, 64, 64, 128, 24])
    N = _log_int(rng, 1, 256)
    context = _log_int(rng, 1, max(2, min(65536, _KV_MOST // 4 // (N * Hk * d))))
    if op == "attn":
        return _attn("drawn", N, Hq, Hk, d, page, context, dtype, rng.random() < 0.7)
    T = N if rng.random() < 0.5 else max(1, min(N * context // 2, _log_int(rng, 1, 65536), 2 ** 26 // (Hq * d)))
    return _append("drawn", N, T, Hq, Hk, d, page, context, rng.choice([0, d // 2 * 2, d // 4 * 2]), dtype,
                   rng.random() < 0.4, rng.random() < 0.6)


# ----------------------------------------------------------------------------------------------------------------
# inputs

def _cuts(seed, n, total, most):
    """Offsets of n sequences of at most `most` tokens that fill `total`: cut at random places, so some may be empty."""
    rng = np.random.default_rng([seed, 77])
    lens = np.diff(np.concatenate([[0], np.sort(rng.integers(0, total + 1, size=n - 1)), [total]]))
    spare = int(np.maximum(lens - most, 0).sum())
    lens = np.minimum(lens, most)
    for i in range(n):
        more = min(spare, most - int(lens[i]))
        lens[i] += more
        spare -= more
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) % (1 << 62))
    host = int(seed) % (1 << 31)

    def normal(*shape, dtype=torch.float32, std=1.0):
        x = torch.randn(shape, generator=gen, device=dev, dtype=dtype)
        return x.mul_(std) if std != 1.0 else x

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=gen, device=dev) * (hi - lo) + lo

    c, dt = case, _DT[case["dtype"]]
    s = {"case": dict(case)}
    if c["op"] == "lin":
        B, T, Hk, H, dk, dv = (c[k] for k in ("B", "T", "Hk", "H", "dk", "dv"))
        lead, N = ((B,), B) if c["mode"] == "step" else ((B, T), B)
        s["cu"] = None
        if c["n_seqs"] > 0:
            N = c["n_seqs"]
            s["cu"] = torch.from_numpy(_cuts(host, N, T, T)).to(dev)
        if c["fused"]:       # q, k and v side by side in the convolution's output
            p = normal(*lead, (2 * Hk) * dk + H * dv, dtype=dt)
            s["q"] = p[..., :Hk * dk].unflatten(-1, (Hk, dk))
            s["k"] = p[..., Hk * dk:2 * Hk * dk].unflatten(-1, (Hk, dk))
            s["v"] = p[..., 2 * Hk * dk:].unflatten(-1, (H, dv))
        else:
            s["q"], s["k"], s["v"] = normal(*lead, Hk, dk, dtype=dt), normal(*lead, Hk, dk, dtype=dt), \
                normal(*lead, H, dv, dtype=dt)
        if c["gate"] == "head":      # retentions from a few tokens to a thousand
            s["g"] = -torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(0.5)))
        else:
            A = torch.exp(uniform(H, lo=math.log(1e-2), hi=math.log(8.0)))
            s["g"] = -A * torch.nn.functional.softplus(normal(*lead, H) + normal(H, std=0.1) - 1)
        s["h0"] = normal(N, H, dk, dv) if c["h0"] or c["mode"] == "step" else None
        s["state_out"] = torch.empty(N, H, dk, dv, device=dev) if c["mode"] == "step" else None
        if c["mode"] == "train":
            s["do"] = normal(*lead, H, dv, dtype=dt)
            s["dhT"] = normal(N, H, dk, dv, std=0.1)
        return s
    N, Hq, Hk, d, page, context = (c[k] for k in ("N", "Hq", "Hk", "d", "page", "context"))
    rng = np.random.default_rng([host, 78])
    if c["op"] == "append":
        T = c["T"]
        new = np.ones(N, dtype=np.int64) if T == N else np.diff(_cuts(host, N, T, context)).astype(np.int64)
        lens = np.array([rng.integers(n, context + 1) for n in new])     # after the call
        s["cu"] = None if T == N else torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(dev)
        p = normal(T, (Hq + 2 * Hk) * d, dtype=dt)                       # one projection's output
        s["q"] = p[:, :Hq * d].unflatten(-1, (Hq, d)) if c["with_q"] else None
        s["k"] = p[:, Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
        s["v"] = p[:, (Hq + Hk) * d:].unflatten(-1, (Hk, d))
        s["cos"] = s["sin"] = None
        if c["rot"] > 0:
            ang = torch.arange(context, device=dev, dtype=torch.float64)[:, None] * \
                10000.0 ** (-torch.arange(c["rot"] // 2, device=dev, dtype=torch.float64) * 2 / c["rot"])
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    else:
        lens = rng.integers(0, context + 1, size=N) if c["ragged"] else np.full(N, context)
        lens[int(rng.integers(N))] = context
        s["q"] = normal(N, Hq, d, dtype=dt)
    per = -(-context // page)
    n_pages = N * per                       # every sequence's pages lie anywhere in the pool
    s["table"] = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32).view(N, per)
    s["lengths"] = torch.from_numpy(lens.astype(np.int32)).to(dev)
    s["kc"] = normal(n_pages, page, Hk, d, dtype=dt)
    s["vc"] = normal(n_pages, page, Hk, d, dtype=dt)
    return s


# ----------------------------------------------------------------------------------------------------------------
# one pass

def run(state):
    s, c = state, state["case"]
    return (_own if own else _plain)[c["op"]](s, c)


def _own_lin(s, c):
    import gated_delta_rule_gdn_gb300 as gdn
    if c["mode"] == "step":
        o = gdn.lin_recurrent_step(s["q"], s["k"], s["v"], s["g"], s["h0"], state_out=s["state_out"])
        return {"o": o, "state": s["state_out"]}
    o, hT = gdn.lin_chunk_fwd(s["q"], s["k"], s["v"], s["g"], initial_state=s["h0"], output_final_state=True,
                              cu_seqlens=s["cu"])
    if c["mode"] == "fwd":
        return {"o": o, "state": hT}
    dq, dk, dv, dg, dh0 = gdn.lin_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], initial_state=s["h0"],
                                            d_final_state=s["dhT"], cu_seqlens=s["cu"])
    return {"o": o, "state": hT, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "dh0": dh0}


def _own_append(s, c):
    import gated_delta_rule_gdn_gb300 as gdn
    q = gdn.paged_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lengths"], q=s["q"], cu_seqlens=s["cu"],
                         cos=s["cos"], sin=s["sin"], interleaved=c["interleaved"])
    return {"k_cache": s["kc"], "v_cache": s["vc"], "q": q}


def _own_attn(s, c):
    import gated_delta_rule_gdn_gb300 as gdn
    return {"o": gdn.paged_attn_step(s["q"], s["kc"], s["vc"], s["table"], s["lengths"])}


_own = {"lin": _own_lin, "append": _own_append, "attn": _own_attn}


def _scan(coef, v):
    """v_m + coef_m v_{m-1} + coef_m coef_{m-1} v_{m-2} + ... along dimension 0, by doubling the reach."""
    reach = 1
    while reach < v.shape[0]:
        v[reach:] += coef[reach:] * v[:-reach].clone()
        coef[reach:] = coef[reach:] * coef[:-reach].clone()
        reach *= 2
    return v


def _plain_lin(s, c):
    Hk, H, dk, dv, C = c["Hk"], c["H"], c["dk"], c["dv"], 64
    dt, scale = s["v"].dtype, c["dk"] ** -0.5
    dev, rep = s["v"].device, c["H"] // c["Hk"]
    if c["mode"] == "step":
        q, k = (s[n].float().repeat_interleave(rep, 1) for n in ("q", "k"))
        h = s["g"].exp()[..., None, None] * s["h0"] + k[..., None] * s["v"].float()[..., None, :]
        s["state_out"].copy_(h)
        return {"o": (scale * (q[..., None] * h).sum(-2)).to(dt), "state": s["state_out"]}
    B, T = c["B"], c["T"]
    n = B * T
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(B + 1, device=dev) * T
    N = len(cu) - 1
    # chunks of C tokens that start with their sequence; the last of a sequence may be partly empty
    length = cu[1:] - cu[:-1]
    first = torch.cumsum((length + C - 1) // C, 0) - (length + C - 1) // C           # the first chunk of a sequence
    M = n // C + N
    m = torch.arange(M, device=dev)
    seq = (torch.searchsorted(first, m, right=True) - 1).clamp(0, N - 1)
    off = (m - first[seq])[:, None] * C + torch.arange(C, device=dev)
    live = off < length[seq][:, None]                                                # [M, C]
    tok = (cu[seq][:, None] + off).clamp(max=n - 1)

    def chunks(x):               # [n, heads, d] -> [M, heads, C, d] in 32 bits, zeros where there is no token
        return (x.float()[tok] * live[..., None, None]).transpose(1, 2)

    def tokens(y, like):         # back to the tokens
        out = torch.empty((n,) + (y.shape[1], y.shape[3]), device=dev)
        out[tok[live]] = y.transpose(1, 2)[live]
        return out.reshape(like.shape).to(like.dtype) if like is not None else out

    q, k, v = (chunks(s[x].reshape(n, *s[x].shape[2:])) for x in ("q", "k", "v"))
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    g = s["g"].expand(n, H) if s["g"].dim() == 1 else s["g"].reshape(n, H)
    G = torch.cumsum((g.double()[tok] * live[..., None]).transpose(1, 2), -1)        # [M, H, C]
    end = G[..., -1:]
    low = torch.tril(torch.ones(C, C, device=dev, dtype=torch.bool))
    decay = torch.where(low, torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0)), 0.0).float()
    into, out_of, whole = G.exp().float()[..., None], (end - G).exp().float()[..., None], end.exp().float()[..., None]
    qk = (q @ k.transpose(-1, -2)) * scale
    # the state entering each chunk
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(N, H, dk, dv, device=dev)
    is_first = (m == first[seq])[:, None, None, None]
    add = (k * out_of).transpose(-1, -2) @ v                                         # [M, H, dk, dv]
    enter = torch.cat([torch.zeros_like(add[:1]), add[:-1]])
    keep = torch.cat([torch.zeros_like(whole[:1]), whole[:-1]])
    enter = torch.where(is_first, h0[seq], enter)
    enter = _scan(torch.where(is_first, torch.zeros_like(keep), keep), enter)
    leave = whole * enter + add
    last = (first + (length + C - 1) // C - 1).clamp(min=0)
    hT = torch.where((length > 0)[:, None, None, None], leave[last], h0)
    o = tokens((qk * decay) @ v + scale * into * (q @ enter), s["v"])
    if c["mode"] == "fwd":
        return {"o": o, "state": hT}
    # gradients: the gradient of the state leaving each chunk, from the last chunk of a sequence to its first
    do = chunks(s["do"].reshape(n, H, dv))
    dv_out = s["dhT"]
    is_last = ((m == last[seq]) & (length[seq] > 0))[:, None, None, None]
    back = scale * (q * into).transpose(-1, -2) @ do
    gain = torch.cat([back[1:], torch.zeros_like(back[:1])])
    keep = torch.cat([whole[1:], torch.zeros_like(whole[:1])])
    gain = torch.where(is_last, dv_out[seq], gain)
    gain = _scan(torch.where(is_last, torch.zeros_like(keep), keep).flip(0), gain.flip(0)).flip(0)
    dh0 = whole * gain + back
    dh0 = torch.where((length > 0)[:, None, None, None], dh0[first.clamp(max=M - 1)], dv_out)
    dp = (do @ v.transpose(-1, -2)) * decay * scale
    dq_in = scale * into * (do @ enter.transpose(-1, -2))
    dk_out = out_of * (v @ gain.transpose(-1, -2))
    dq, dk_ = dp @ k + dq_in, dp.transpose(-1, -2) @ q + dk_out
    dv_ = (qk * decay).transpose(-1, -2) @ do + out_of * (k @ gain)
    # dg_t: all pairs of a token before t with one at or behind it, in the chunk and through the states
    pairs = dp * (qk / scale)
    cross = torch.cumsum(pairs.flip(-2), -2).flip(-2)
    cross = torch.cumsum(cross, -1) - cross
    dg = torch.diagonal(cross, dim1=-2, dim2=-1)
    dg = dg + torch.cumsum((q * dq_in).sum(-1).flip(-1), -1).flip(-1)
    b = (k * dk_out).sum(-1)
    dg = dg + torch.cumsum(b, -1) - b + (whole * gain * enter).sum((-1, -2))[..., None]
    dg = tokens(dg[..., None], None)[..., 0]
    dg = dg.double().sum(0).float() if s["g"].dim() == 1 else dg.reshape(s["g"].shape)

    def shared(x, like):         # value heads of one key head
        return tokens(x.reshape(M, Hk, rep, C, dk).sum(2), like)

    return {"o": o, "state": hT, "dq": shared(dq, s["q"]), "dk": shared(dk_, s["k"]), "dv": tokens(dv_, s["v"]),
            "dg": dg, "dh0": dh0 if s["h0"] is not None else None}


def _turn(x, cos, sin, R, interleaved):
    """Rotate the first R channels by the angles of `cos`, `sin` ([tokens, 1, R/2])."""
    if R == 0:
        return x
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., R:]], -1)


def _places(s, c):
    """(position in its sequence, page, place in the page) of every new token."""
    dev = s["k"].device
    t = torch.arange(c["T"], device=dev)
    if s["cu"] is None:
        seq, pos = t, s["lengths"].long() - 1
    else:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        pos = s["lengths"].long()[seq] - (cu[seq + 1] - t)
    return pos, s["table"].long()[seq, pos // c["page"]], pos % c["page"]


def _plain_append(s, c):
    pos, page, place = _places(s, c)
    dt, R = s["k"].dtype, c["rot"]
    cos, sin = (s["cos"][pos][:, None], s["sin"][pos][:, None]) if R > 0 else (None, None)
    s["kc"][page, place] = _turn(s["k"].float(), cos, sin, R, c["interleaved"]).to(dt)
    s["vc"][page, place] = s["v"]
    q = None if s["q"] is None else _turn(s["q"].float(), cos, sin, R, c["interleaved"]).to(dt)
    return {"k_cache": s["kc"], "v_cache": s["vc"], "q": q}


def _plain_attn(s, c):
    N, Hq, Hk, d = c["N"], c["Hq"], c["Hk"], c["d"]
    L = s["table"].shape[1] * c["page"]
    k = s["kc"][s["table"].long()].view(N, L, Hk, d).transpose(1, 2).float()          # [N, Hk, L, d]
    p = s["q"].float().view(N, Hk, Hq // Hk, d) @ k.transpose(-1, -2) * d ** -0.5
    del k
    live = (torch.arange(L, device=p.device) < s["lengths"][:, None])[:, None, None]
    p = p.masked_fill(~live, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = torch.exp(p - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    v = s["vc"][s["table"].long()].view(N, L, Hk, d).transpose(1, 2).float()
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return {"o": o.reshape(N, Hq, d).to(s["q"].dtype)}


_plain = {"lin": _plain_lin, "append": _plain_append, "attn": _plain_attn}


# ----------------------------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "lin":
        n, N = c["B"] * c["T"], c["n_seqs"] or c["B"]
        qk, v = n * c["Hk"] * c["dk"] * es, n * c["H"] * c["dv"] * es
        g = n * c["H"] * 4 if c["gate"] == "token" else c["H"] * 4
        state = N * c["H"] * c["dk"] * c["dv"] * 4
        pair = n * c["H"] * c["dk"] * c["dv"]
        if c["mode"] != "train":
            return {"bytes": 2 * qk + 2 * v + g + state * (2 if c["h0"] or c["mode"] == "step" else 1),
                    "flops": 4 * pair}
        # inputs and d_o once; o, the gradients and the final state once
        return {"bytes": 4 * qk + 4 * v + 2 * g + state * (4 if c["h0"] else 2), "flops": 14 * pair}
    if c["op"] == "append":
        heads = 2 * c["Hk"] + (c["Hq"] if c["with_q"] else 0)
        return {"bytes": c["T"] * (2 * heads * c["d"] * es + c["rot"] * 4) + c["N"] * 8,
                "flops": 3 * c["T"] * (heads - c["Hk"]) * c["rot"]}
    # ragged lengths are uniform over 0..context
    tokens = c["N"] * c["context"] * (0.5 if c["ragged"] and c["N"] > 1 else 1.0)
    return {"bytes": int(tokens * 2 * c["Hk"] * c["d"] * es + 2 * c["N"] * c["Hq"] * c["d"] * es),
            "flops": int(4 * tokens * c["Hq"] * c["d"])}


# ----------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s, c = prepare(case, seed), case
    return {"lin": _exact_lin, "append": _exact_append, "attn": _exact_attn}[c["op"]](s, c)


def _exact_lin(s, c):
    H, rep, scale = c["H"], c["H"] // c["Hk"], c["dk"] ** -0.5
    q, k = (s[x].double().repeat_interleave(rep, -2) for x in ("q", "k"))
    v = s["v"].double()
    if c["mode"] == "step":
        h = torch.exp(s["g"].double())[..., None, None] * s["h0"].double() + torch.einsum("nhk,nhv->nhkv", k, v)
        return {"o": scale * torch.einsum("nhk,nhkv->nhv", q, h), "state": h}
    B, T = c["B"], c["T"]
    a = torch.exp(s["g"].double())
    a = a.expand(B, T, H) if a.dim() == 1 else a
    N = c["n_seqs"] or B
    zero = torch.zeros(N, H, c["dk"], c["dv"], dtype=torch.float64, device=v.device)
    h0 = zero if s["h0"] is None else s["h0"].double()
    hT, starts, ends = h0.clone(), {}, {}          # token -> the sequences that start, or end, with it (a batch: all)
    if s["cu"] is None:
        starts[0], ends[T - 1] = slice(None), slice(None)
    else:
        cu = s["cu"].tolist()
        for i in range(N):
            if cu[i + 1] > cu[i]:
                starts[cu[i]], ends[cu[i + 1] - 1] = slice(i, i + 1), slice(i, i + 1)

    def forth(S, t):
        if t in starts:
            S = h0[starts[t]]
        return torch.addcmul(a[:, t, :, None, None] * S, k[:, t, :, :, None], v[:, t, :, None, :])

    S, marks = h0[:B], {}
    o = torch.empty_like(v)
    for t in range(T):
        if t % 64 == 0:
            marks[t] = S
        S = forth(S, t)
        o[:, t] = scale * (q[:, t, :, None, :] @ S)[..., 0, :]
        if t in ends:
            hT[ends[t]] = S
    if c["mode"] == "fwd":
        return {"o": o, "state": hT}
    do, dhT = s["do"].double(), s["dhT"].double()
    dq, dk, dv, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(v[..., 0])
    dh0, D = dhT.clone(), None
    for t0 in range((T - 1) // 64 * 64, -1, -64):
        S, states = marks[t0], []
        for t in range(t0, min(T, t0 + 64)):
            states.append(h0[starts[t]] if t in starts else S)
            S = forth(S, t)
        after = states[1:] + [S]                   # (the state behind a token; not what replaces it at a start)
        for t in range(min(T, t0 + 64) - 1, t0 - 1, -1):
            before = states[t - t0]
            now = after[t - t0] if t + 1 not in starts else forth(before, t)
            if t in ends:
                D = dhT[ends[t]]
            D = torch.addcmul(D, scale * q[:, t, :, :, None], do[:, t, :, None, :])
            dq[:, t] = scale * (now @ do[:, t, :, :, None])[..., 0]
            dk[:, t] = (D @ v[:, t, :, :, None])[..., 0]
            dv[:, t] = (k[:, t, :, None, :] @ D)[..., 0, :]
            D = a[:, t, :, None, None] * D
            dg[:, t] = (D * before).sum((-1, -2))
            if t in starts:
                dh0[starts[t]] = D
    dq, dk = (x.reshape(B, T, c["Hk"], rep, c["dk"]).sum(3) for x in (dq, dk))
    return {"o": o, "state": hT, "dq": dq, "dk": dk, "dv": dv, "dg": dg.sum((0, 1)) if s["g"].dim() == 1 else dg,
            "dh0": None if s["h0"] is None else dh0}


def _exact_append(s, c):
    T, R, page = c["T"], c["rot"], c["page"]
    new = [1] * c["N"] if s["cu"] is None else (s["cu"][1:] - s["cu"][:-1]).tolist()
    pos = torch.tensor([p for n, length in zip(new, s["lengths"].tolist()) for p in range(length - n, length)],
                       device=s["k"].device)
    seq = torch.tensor([i for i, n in enumerate(new) for _ in range(n)], device=s["k"].device)
    at = s["table"].long()[seq, pos // page] * page + pos % page
    kc, vc = s["kc"].double(), s["vc"].double()

    def turned(x):
        x = x.double()
        if R == 0:
            return x
        w = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
        if c["interleaved"]:
            z = torch.view_as_complex(x[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) * w
            z = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * w
            z = torch.cat([z.real, z.imag], -1)
        return torch.cat([z, x[..., R:]], -1)

    assert len(pos) == T
    kc.view(-1, *kc.shape[2:])[at] = turned(s["k"])
    vc.view(-1, *vc.shape[2:])[at] = s["v"].double()
    return {"k_cache": kc, "v_cache": vc, "q": None if s["q"] is None else turned(s["q"])}


def _exact_attn(s, c):
    Hk, rep, d = c["Hk"], c["Hq"] // c["Hk"], c["d"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for i, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        pages = s["table"][i, :-(-n // c["page"])].long()
        k, v = (s[x][pages].flatten(0, 1)[:n].double() for x in ("kc", "vc"))
        p = torch.einsum("krd,lkd->krl", s["q"][i].double().view(Hk, rep, d), k) * d ** -0.5
        o[i] = torch.einsum("krl,lkd->krd", torch.softmax(p, -1), v).reshape(-1, d)
    return {"o": o}
