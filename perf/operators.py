"""The sequence-mixer operators around the gated delta rule: measured cases and their plain forms.

Three operators:
* the gated linear recurrence ("glr"): a decode step, a scan forward, and a training pass (forward and gradients);
* the norm of every query and key head, with the position rotation ("qk"): forward, and a training pass;
* the short causal convolution over the projected tokens ("conv"): a decode step, a forward and a training pass.

With ``own`` false, ``run`` computes each in elementary torch operations in 32 bits, rounded once at the end; with
``own`` true it calls the library.  ``exact`` computes the same from the definitions in 64 bits, token by token.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_LARGEST = 65536 * 4096          # elements of one [tokens, channels] array of the largest case


# ----------------------------------------------------------------------------------------------------------------
# cases

def _glr(name, mode, B, T, D, dtype="bf16", g_dtype="bf16", n_seqs=0, act=True, gate=True, normalize=True, h0=True,
         fused=True):
    # mode: "step" (B sequences, one token each), "fwd", or "train" (forward and gradients)
    return {"name": name, "op": "glr", "mode": mode, "B": B, "T": T, "D": D, "dtype": dtype, "g_dtype": g_dtype,
            "n_seqs": n_seqs, "act": act, "gate": gate, "normalize": normalize, "h0": h0, "fused": fused}


def _qk(name, mode, B, T, Hq, Hk, d, rot, norm, dtype="bf16", weight=True, interleaved=False, positions=True,
        fused=True):
    return {"name": name, "op": "qk", "mode": mode, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "d": d, "rot": rot,
            "norm": norm, "dtype": dtype, "weight": weight, "interleaved": interleaved, "positions": positions,
            "fused": fused}


def _conv(name, mode, B, T, D, W=4, dtype="bf16", n_seqs=0, bias=True, silu=True, h0=True, fused=True):
    return {"name": name, "op": "conv", "mode": mode, "B": B, "T": T, "D": D, "W": W, "dtype": dtype,
            "n_seqs": n_seqs, "bias": bias, "silu": silu, "h0": h0, "fused": fused}


def listed():
    return [
        # one sequence being decoded: the smallest call, where latency counts
        _glr("glr_step_n1_d2048", "step", 1, 1, 2048),
        # a prompt of an odd length on one sequence
        _glr("glr_fwd_prompt_b1_t1000_d2048", "fwd", 1, 1000, 2048),
        # one long document on few channels of an odd width, decays given, all in fp32
        _glr("glr_fwd_long_b1_t65536_d250_f32", "fwd", 1, 65536, 250, dtype="f32", g_dtype="f32", act=False,
             gate=False, normalize=False, fused=False),
        # a training step of the layer at the width of the delta rule's prefill shape
        _glr("glr_train_b4_t4096_d2048", "train", 4, 4096, 2048, h0=False),
        # a packed training batch of eight documents at twice the width: the largest
        _glr("glr_train_packed_65536tok_d4096", "train", 1, 65536, 4096, n_seqs=8),
        # 256 sequences being decoded, 32 query and key heads: norms with weights, rotation at each one's own position
        _qk("qk_rms_decode_n256_h32", "fwd", 256, 1, 32, 32, 128, 128, "rms"),
        # the delta rule's prefill: unit-norm queries and keys, read out of the convolution's fused output
        _qk("qk_l2_fwd_b4_t4096_h16", "fwd", 4, 4096, 16, 16, 128, 0, "l2", weight=False, positions=False),
        # training with grouped heads, half of each head rotated
        _qk("qk_rms_train_b2_t8192_hq32_hk8_rot64", "train", 2, 8192, 32, 8, 128, 64, "rms"),
        # an odd head size in fp32 with interleaved rotation
        _qk("qk_rms_train_b1_t1000_hq6_hk2_d100_f32", "train", 1, 1000, 6, 2, 100, 48, "rms", dtype="f32",
            interleaved=True, positions=False, fused=False),
        # 256 sequences being decoded through the fused q, k, v convolution
        _conv("conv_step_n256_d6144", "step", 256, 1, 6144),
        # prefill of the fused q, k, v convolution, read out of a wider projection
        _conv("conv_fwd_b4_t4096_d6144", "fwd", 4, 4096, 6144),
        # a packed training batch of eight documents
        _conv("conv_train_packed_65536tok_d4096", "train", 1, 65536, 4096, n_seqs=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glr", "glr", "qk", "conv"])
    most = _LARGEST // 4
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "qk":
        d = rng.choice([64, 96, 100, 128, 128, 192, 256, rng.randint(8, 256)])
        Hk = _log_int(rng, 1, 32)
        Hq = Hk * rng.choice([1, 1, 2, 4])
        mode = rng.choice(["fwd", "fwd", "train"])
        B = _log_int(rng, 1, 256)
        T = _log_int(rng, 1, max(2, min(16384, most // (B * (Hq + Hk) * d))))
        rot = rng.choice([0, d // 2 * 2, d // 4 * 2])
        return _qk(None, mode, B, T, Hq, Hk, d, rot, rng.choice(["rms", "l2"]), dtype, rng.random() < 0.7,
                   rng.random() < 0.4, rng.random() < 0.5, rng.random() < 0.5) | {"name": "drawn"}
    mode = rng.choice(["step", "fwd", "train"])
    D = rng.choice([_log_int(rng, 1, 8192), 64 * _log_int(rng, 1, 128)])
    fused = rng.random() < 0.5
    if mode == "step":
        B, T, n_seqs = _log_int(rng, 1, 1024), 1, 0
    elif rng.random() < 0.5:
        T = _log_int(rng, 1, max(2, min(65536, most // D)))
        B, n_seqs = 1, _log_int(rng, 1, 64)
    else:
        B = _log_int(rng, 1, 32)
        T = _log_int(rng, 1, max(2, min(65536, most // (D * B))))
        n_seqs = 0
    if op == "glr":
        return _glr("drawn", mode, B, T, D, dtype, dtype if fused else rng.choice(["f32", dtype]), n_seqs,
                    rng.random() < 0.6, rng.random() < 0.6, rng.random() < 0.6, rng.random() < 0.6, fused)
    return _conv("drawn", mode, B, T, D, rng.choice([2, 3, 4, 4]), dtype, n_seqs, rng.random() < 0.6,
                 rng.random() < 0.8, rng.random() < 0.6, fused)


# ----------------------------------------------------------------------------------------------------------------
# inputs

def _lengths(seed, n, total):
    """n document lengths that fill `total` tokens: cuts at random places, so some may be empty."""
    rng = np.random.default_rng([seed, 77])
    cuts = np.sort(rng.integers(0, total + 1, size=n - 1))
    return np.concatenate([[0], cuts, [total]]).astype(np.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) % (1 << 62))

    def normal(*shape, dtype=torch.float32, std=1.0):
        x = torch.randn(shape, generator=gen, device=dev, dtype=dtype)
        return x.mul_(std) if std != 1.0 else x

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=gen, device=dev) * (hi - lo) + lo

    c, dt = case, _DT[case["dtype"]]
    s = {"case": dict(case)}
    B, T = c["B"], c["T"]
    lead = (B,) if c["mode"] == "step" else (B, T)
    N = B
    s["cu"] = None
    if c.get("n_seqs", 0) > 0:
        N = c["n_seqs"]
        s["cu"] = torch.from_numpy(_lengths(int(seed) % (1 << 31), N, T)).to(dev)
    if c["op"] == "glr":
        D, gt = c["D"], _DT[c["g_dtype"]]
        if c["fused"]:       # one projection gives the token, its decay logit and its input-gate logit
            p = normal(*lead, 3 * D, dtype=dt)
            s["x"], g, i = p[..., :D], p[..., D:2 * D], p[..., 2 * D:]
        else:
            s["x"], g, i = normal(*lead, D, dtype=dt), normal(*lead, D, dtype=gt), normal(*lead, D, dtype=dt)
        s["i"] = i if c["gate"] else None
        s["A_log"] = s["dt_bias"] = None
        if c["act"]:         # decays from quick forgetting to a memory of thousands of tokens
            s["A_log"] = uniform(D, lo=math.log(1e-3), hi=math.log(2.0))
            s["dt_bias"] = normal(D, std=0.1)
            s["g"] = g
        elif c["fused"]:     # log retention, in place in the projection
            s["g"] = g.copy_(-(g.float().exp() * 0.05))
        else:
            s["g"] = -(g.float().exp() * 0.05).to(gt)
        s["h0"] = normal(N, D) if c["h0"] or c["mode"] == "step" else None
        s["state_out"] = torch.empty(N, D, device=dev) if c["mode"] == "step" else None
        if c["mode"] == "train":
            s["do"] = normal(*lead, D, dtype=dt)
            s["dhT"] = normal(N, D)
    elif c["op"] == "qk":
        Hq, Hk, d, R = c["Hq"], c["Hk"], c["d"], c["rot"]
        if c["fused"]:       # q and k side by side with v in one projection's output
            p = normal(B, T, (Hq + 2 * Hk) * d, dtype=dt)
            s["q"] = p[..., :Hq * d].unflatten(-1, (Hq, d))
            s["k"] = p[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
        else:
            s["q"], s["k"] = normal(B, T, Hq, d, dtype=dt), normal(B, T, Hk, d, dtype=dt)
        s["wq"] = 1 + normal(d, std=0.1) if c["weight"] else None
        s["wk"] = 1 + normal(d, std=0.1) if c["weight"] else None
        s["cos"] = s["sin"] = s["pos"] = None
        if R > 0:            # the rotation table of the longest context, laid out once; positions anywhere in it
            P = 32768
            ang = torch.arange(P, device=dev, dtype=torch.float64)[:, None] * \
                10000.0 ** (-torch.arange(R // 2, device=dev, dtype=torch.float64) * 2 / R)
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
            if c["positions"]:
                start = torch.randint(0, P - T, (B, 1), generator=gen, device=dev)
                s["pos"] = (start + torch.arange(T, device=dev)).to(torch.int32)
        if c["mode"] == "train":
            s["dq"], s["dk"] = normal(B, T, Hq, d, dtype=dt), normal(B, T, Hk, d, dtype=dt)
    else:
        D, W = c["D"], c["W"]
        s["x"] = normal(*lead, D + D // 2 if c["fused"] else D, dtype=dt)[..., :D]
        s["w"] = uniform(D, W, lo=-W ** -0.5, hi=W ** -0.5)
        s["b"] = uniform(D, lo=-W ** -0.5, hi=W ** -0.5) if c["bias"] else None
        s["h0"] = normal(N, W - 1, D, dtype=dt) if c["h0"] or c["mode"] == "step" else None
        s["state_out"] = torch.empty(N, W - 1, D, device=dev, dtype=dt) if c["mode"] == "step" else None
        if c["mode"] == "train":
            s["dy"] = normal(*lead, D, dtype=dt)
            s["dhT"] = normal(N, W - 1, D, dtype=dt)
    return s


# ----------------------------------------------------------------------------------------------------------------
# one pass

def run(state):
    s, c = state, state["case"]
    return (_own if own else _plain)[c["op"]](s, c)


def _own_glr(s, c):
    import gated_delta_rule_gdn_gb300 as gdn
    kw = dict(in_gate=s["i"], A_log=s["A_log"], dt_bias=s["dt_bias"], normalize=c["normalize"])
    if c["mode"] == "step":
        o = gdn.glr_step(s["x"], s["g"], s["h0"], state_out=s["state_out"], **kw)
        return {"o": o, "state": s["state_out"]}
    kw.update(initial_state=s["h0"], cu_seqlens=s["cu"])
    if c["mode"] == "fwd":
        o, hT = gdn.glr_scan_fwd(s["x"], s["g"], output_final_state=True, **kw)
        return {"o": o, "state": hT}
    o, hT, ck = gdn.glr_scan_fwd(s["x"], s["g"], output_final_state=True, output_checkpoints=True, **kw)
    dx, dg, di, dh0, dA, ddt = gdn.glr_scan_bwd(s["x"], s["g"], s["do"], d_final_state=s["dhT"], checkpoints=ck, **kw)
    return {"o": o, "state": hT, "dx": dx, "dg": dg, "di": di, "dh0": dh0, "dA_log": dA, "ddt_bias": ddt}


def _own_qk(s, c):
    import gated_delta_rule_gdn_gb300 as gdn
    kw = dict(q_weight=s["wq"], k_weight=s["wk"], norm=c["norm"], eps=1e-6, cos=s["cos"], sin=s["sin"],
              positions=s["pos"], interleaved=c["interleaved"])
    q, k = gdn.gdn_qk_norm_fwd(s["q"], s["k"], **kw)
    if c["mode"] == "fwd":
        return {"q": q, "k": k}
    dq, dk, dwq, dwk = gdn.gdn_qk_norm_bwd(s["q"], s["k"], s["dq"], s["dk"], **kw)
    return {"q": q, "k": k, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _own_conv(s, c):
    import gated_delta_rule_gdn_gb300 as gdn
    kw = dict(bias=s["b"], activation="silu" if c["silu"] else None)
    if c["mode"] == "step":
        y = gdn.gdn_short_conv_step(s["x"], s["h0"], s["w"], state_out=s["state_out"], **kw)
        return {"y": y, "state": s["state_out"]}
    kw.update(initial_state=s["h0"], cu_seqlens=s["cu"])
    y, hT = gdn.gdn_short_conv_fwd(s["x"], s["w"], output_final_state=True, **kw)
    if c["mode"] == "fwd":
        return {"y": y, "state": hT}
    dx, dw, db, dh0 = gdn.gdn_short_conv_bwd(s["x"], s["w"], s["dy"], d_final_state=s["dhT"], **kw)
    return {"y": y, "state": hT, "dx": dx, "dw": dw, "db": db, "dh0": dh0}


_own = {"glr": _own_glr, "qk": _own_qk, "conv": _own_conv}


# Plain forms.  Sequences: [B, T, D] batches, or one row of packed documents with offsets `cu`.

def _ends(s, B, T, dev):
    """Per batch row: (first token, last token, whether it has any) of every sequence, and its row."""
    if s["cu"] is None:
        n = torch.arange(B, device=dev)
        z = torch.zeros_like(n)
        return n, z, z + max(T - 1, 0), (z + T > 0)
    cu = s["cu"].long()
    z = torch.zeros_like(cu[1:])
    return z, cu[:-1].clamp(max=T - 1), (cu[1:] - 1).clamp(min=0), cu[1:] > cu[:-1]


def _scan(coef, v):
    """v_t + coef_t v_{t-1} + coef_t coef_{t-1} v_{t-2} + ... along dimension 1, by doubling the reach (log2 T
    elementwise passes: the recurrence has no closed elementary form that does not overflow)."""
    reach = 1
    while reach < v.shape[1]:
        v[:, reach:] += coef[:, reach:] * v[:, :-reach]
        coef[:, reach:] = coef[:, reach:] * coef[:, :-reach]
        reach *= 2
    return v


def _gates(s, c):
    """(log a, a, s, sigma(i), x, z) in fp32 of every token."""
    z, x = s["g"].float(), s["x"].float()
    if c["act"]:
        z = z + s["dt_bias"]
        la = -s["A_log"].exp() * (z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())))
    else:
        la = z
    n = torch.sqrt(-torch.expm1(2 * la)) if c["normalize"] else None
    gi = 1 / (1 + torch.exp(-s["i"].float())) if c["gate"] else None
    return la, la.exp(), n, gi, x, z


def _plain_glr(s, c):
    la, a, n, gi, x, z = _gates(s, c)
    u = x.clone()
    if gi is not None:
        u = u * gi
    if n is not None:
        u = u * n
    dt = s["x"].dtype
    if c["mode"] == "step":
        h = a * s["h0"] + u
        s["state_out"].copy_(h)
        return {"o": h.to(dt), "state": s["state_out"]}
    B, T, D = x.shape
    row, first, last, some = _ends(s, B, T, x.device)
    some = some[:, None]
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(len(row), D, device=x.device)
    inject = torch.where(some, a[row, first] * h0, torch.zeros_like(h0))
    u.index_put_((row, first), inject, accumulate=True)
    is_first = torch.zeros(B, T, device=x.device).index_put_((row, first), some[:, 0].float(), accumulate=True) > 0
    coef = torch.where(is_first[..., None], torch.zeros_like(a), a)
    h = _scan(coef, u)
    hT = torch.where(some, h[row, last], h0)
    if c["mode"] == "fwd":
        return {"o": h.to(dt), "state": hT}
    # gradients: D_t = do_t + a_{t+1} D_{t+1}, from the last token of each sequence to its first
    dh = s["do"].float().clone()
    dh.index_put_((row, last), torch.where(some, s["dhT"], torch.zeros_like(s["dhT"])), accumulate=True)
    nxt = torch.where(is_first[..., None], torch.zeros_like(a), a)[:, 1:]
    nxt = torch.cat([nxt, torch.zeros_like(a[:, :1])], 1)
    dh = _scan(nxt.flip(1), dh.flip(1)).flip(1)
    dh0 = torch.where(some, a[row, first] * dh[row, first], s["dhT"])
    prev = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    prev = torch.where(is_first[..., None], torch.zeros_like(prev), prev)
    prev.index_put_((row, first), torch.where(some, h0, torch.zeros_like(h0)), accumulate=True)
    dla = a * dh * prev
    gx = x if gi is None else gi * x
    if n is not None:
        dla = dla - dh * gx * a * a / n
    du = dh if n is None else dh * n
    di = None if gi is None else (du * x * gi * (1 - gi)).to(s["i"].dtype)
    dx = (du if gi is None else du * gi).to(dt)
    dA = ddt = None
    dg = dla
    if c["act"]:
        dA = (dla * la).sum((0, 1))
        dg = -dla * s["A_log"].exp() / (1 + torch.exp(-z))
        ddt = dg.sum((0, 1))
    return {"o": h.to(dt), "state": hT, "dx": dx, "dg": dg.to(s["g"].dtype), "di": di,
            "dh0": dh0 if s["h0"] is not None else None, "dA_log": dA, "ddt_bias": ddt}


def _turn(x, cos, sin, R, interleaved, back=False):
    """Rotate the first R channels by the angles of `cos`, `sin` ([B, T, 1, R/2]); `back` turns the other way."""
    if R == 0:
        return x
    if back:
        sin = -sin
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., R:]], -1)


def _plain_qk(s, c):
    B, T, d, R = c["B"], c["T"], c["d"], c["rot"]
    cos = sin = None
    if R > 0:
        pos = s["pos"].long() if s["pos"] is not None else torch.arange(T, device=s["q"].device).expand(B, T)
        cos, sin = s["cos"][pos][:, :, None], s["sin"][pos][:, :, None]
    f = 1.0 / d if c["norm"] == "rms" else 1.0

    def one(x, w, dz):
        xf = x.float()
        r = torch.rsqrt((xf * xf).sum(-1, keepdim=True) * f + 1e-6)
        xh = xf * r
        y = _turn(xh if w is None else xh * w, cos, sin, R, c["interleaved"]).to(x.dtype)
        if dz is None:
            return y, None, None
        dy = _turn(dz.float(), cos, sin, R, c["interleaved"], back=True)
        dw = None if w is None else (dy * xh).sum((0, 1, 2))
        e = dy if w is None else dy * w
        return y, (r * (e - f * xh * (e * xh).sum(-1, keepdim=True))).to(x.dtype), dw

    train = c["mode"] == "train"
    q, dq, dwq = one(s["q"], s["wq"], s["dq"] if train else None)
    k, dk, dwk = one(s["k"], s["wk"], s["dk"] if train else None)
    return {"q": q, "k": k, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk} if train else {"q": q, "k": k}


def _plain_conv(s, c):
    dt, W, D = s["x"].dtype, c["W"], c["D"]
    w, b = s["w"], s["b"] if s["b"] is not None else 0.0

    def act(p):
        return p / (1 + torch.exp(-p)) if c["silu"] else p

    if c["mode"] == "step":
        win = torch.cat([s["h0"], s["x"][:, None]], 1)
        p = (win.float() * w.t()).sum(1) + b
        s["state_out"].copy_(win[:, 1:])
        return {"y": act(p).to(dt), "state": s["state_out"]}
    B, T = c["B"], c["T"]
    x = s["x"]
    dev = x.device
    row, first, last, some = _ends(s, B, T, dev)
    N = len(row)
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(N, W - 1, D, device=dev, dtype=dt)
    # the sequence and the place in it of every token; a token's window reaches into the sequence's initial state
    t = torch.arange(T, device=dev)
    if s["cu"] is None:
        seq = torch.arange(B, device=dev)[:, None].expand(B, T)
        at = t.expand(B, T)
        length = torch.full((N,), T, device=dev)
    else:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=N - 1)[None]
        at = (t - cu[seq[0]])[None]
        length = cu[1:] - cu[:-1]
    # each sequence's W - 1 initial inputs go in front of its tokens: one row of tokens with gaps
    pad = torch.zeros(B * T + N * (W - 1), D, device=dev, dtype=dt)
    place = (seq + 1) * (W - 1) + (t[None] if s["cu"] is not None else (seq * T + at))
    start = place.new_zeros(N)
    start = torch.cumsum(length + W - 1, 0) - (length + W - 1)
    lead = start[:, None] + torch.arange(W - 1, device=dev)
    pad[place.reshape(-1)] = x.reshape(B * T, D)
    pad[lead] = h0
    win = pad.float().unfold(0, W, 1)                                # [rows - W + 1, D, W]
    p = (win * w).sum(-1) + b
    here = place.reshape(-1) - (W - 1)
    y = act(p[here]).reshape(B, T, D).to(dt)
    tail = (start + length)[:, None] + torch.arange(W - 1, device=dev)
    hT = pad[tail]
    if c["mode"] == "fwd":
        return {"y": y, "state": hT}
    pt = p[here]
    ds = s["dy"].reshape(B * T, D).float()
    if c["silu"]:
        sg = 1 / (1 + torch.exp(-pt))
        ds = ds * (sg * (1 + pt * (1 - sg)))
    db = ds.sum(0) if s["b"] is not None else None
    full = torch.zeros(len(pad) + W - 1, D, device=dev)              # ds at the row of its token, zero elsewhere
    full[place.reshape(-1)] = ds
    dpad = (full.unfold(0, W, 1) * w.flip(1)).sum(-1)
    dw = (ds[..., None] * win[here]).sum(0)
    dpad.index_put_((tail,), s["dhT"].float(), accumulate=True)
    return {"y": y, "state": hT, "dx": dpad[place.reshape(-1)].reshape(B, T, D).to(dt), "dw": dw, "db": db,
            "dh0": dpad[lead].to(dt) if s["h0"] is not None else None}


_plain = {"glr": _plain_glr, "qk": _plain_qk, "conv": _plain_conv}


# ----------------------------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    n = c["B"] * c["T"]
    N = c["n_seqs"] if c.get("n_seqs", 0) > 0 else c["B"]
    if c["op"] == "glr":
        e = n * c["D"]
        gs = 2 if c["g_dtype"] == "bf16" else 4
        ins = e * (es + gs + (es if c["gate"] else 0))
        state = N * c["D"] * 4 * (2 if c["h0"] or c["mode"] == "step" else 1)
        per = 4 + 14 * c["act"] + 6 * c["gate"] + 6 * c["normalize"]
        if c["mode"] != "train":
            return {"bytes": ins + e * es + state, "flops": e * per}
        return {"bytes": 2 * ins + 2 * e * es + 2 * state, "flops": 3 * e * per}
    if c["op"] == "qk":
        e = n * (c["Hq"] + c["Hk"]) * c["d"]
        table = n * c["rot"] * 4 if c["positions"] else c["T"] * c["rot"] * 4
        if c["mode"] != "train":
            return {"bytes": 2 * e * es + table, "flops": e * 6}
        return {"bytes": 4 * e * es + table, "flops": e * 20}
    e, W = n * c["D"], c["W"]
    state = N * (W - 1) * c["D"] * es * (2 if c["h0"] or c["mode"] == "step" else 1)
    wts = c["D"] * (W + c["bias"]) * 4
    if c["mode"] != "train":
        return {"bytes": 2 * e * es + state + wts, "flops": e * (2 * W + 5)}
    return {"bytes": 4 * e * es + 2 * state + 2 * wts, "flops": e * (6 * W + 15)}


# ----------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, token by token

def _spans(s, c):
    """(sequence, batch row, first token, one past the last) of every sequence, on the host."""
    if s["cu"] is None:
        return [(n, n, 0, c["T"]) for n in range(c["B"])]
    cu = s["cu"].tolist()
    return [(n, 0, cu[n], cu[n + 1]) for n in range(len(cu) - 1)]


def exact(case, seed):
    s, c = prepare(case, seed), case
    return {"glr": _exact_glr, "qk": _exact_qk, "conv": _exact_conv}[c["op"]](s, c)


def _leaf(t):
    return None if t is None else t.double().requires_grad_(True)


def _exact_glr(s, c):
    x, g, i, A, dtb = (_leaf(s[k]) for k in ("x", "g", "i", "A_log", "dt_bias"))
    train = c["mode"] == "train"
    with torch.set_grad_enabled(train):
        la = -A.exp() * torch.nn.functional.softplus(g + dtb, threshold=1e9) if c["act"] else g
        a = la.exp()
        u = x
        if c["gate"]:
            u = u * torch.sigmoid(i)
        if c["normalize"]:
            u = u * (-torch.expm1(2 * la)).sqrt()
    an, un = a.detach(), u.detach()
    if c["mode"] == "step":
        h = an * s["h0"].double() + un
        return {"o": h, "state": h}
    N = len(_spans(s, c))
    D = c["D"]
    h0 = s["h0"].double() if s["h0"] is not None else torch.zeros(N, D, device=an.device, dtype=torch.float64)
    h, prev, hT = torch.empty_like(un), torch.empty_like(un), h0.clone()
    if s["cu"] is None:
        cur = h0
        for t in range(c["T"]):
            prev[:, t] = cur
            cur = torch.addcmul(un[:, t], an[:, t], cur)
            h[:, t] = cur
        hT = cur
    else:
        for n, b, lo, hi in _spans(s, c):
            cur = h0[n]
            for t in range(lo, hi):
                prev[b, t] = cur
                cur = torch.addcmul(un[b, t], an[b, t], cur)
                h[b, t] = cur
            hT[n] = cur
    if not train:
        return {"o": h, "state": hT}
    do, dhT = s["do"].double(), s["dhT"].double()
    dh, dh0 = torch.empty_like(do), dhT.clone()
    if s["cu"] is None:
        carry = dhT
        for t in range(c["T"] - 1, -1, -1):
            dh[:, t] = do[:, t] + carry
            carry = an[:, t] * dh[:, t]
        dh0 = carry
    else:
        for n, b, lo, hi in _spans(s, c):
            carry = dhT[n]
            for t in range(hi - 1, lo - 1, -1):
                dh[b, t] = do[b, t] + carry
                carry = an[b, t] * dh[b, t]
            dh0[n] = carry
    at = [(k, t) for k, t in (("dx", x), ("dg", g), ("di", i if c["gate"] else None),
                              ("dA_log", A), ("ddt_bias", dtb)) if t is not None]
    grads = torch.autograd.grad((a, u), [t for _, t in at], (dh * prev, dh))
    out = {"o": h, "state": hT, "dx": None, "dg": None, "di": None, "dh0": dh0 if s["h0"] is not None else None,
           "dA_log": None, "ddt_bias": None}
    out.update({k: v for (k, _), v in zip(at, grads)})
    return out


def _exact_qk(s, c):
    d, R = c["d"], c["rot"]
    B, T = c["B"], c["T"]
    train = c["mode"] == "train"
    leaves, outs = [], []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x, w = _leaf(x), _leaf(w)
        leaves += [x, w]
        n2 = (x * x).mean(-1, keepdim=True) if c["norm"] == "rms" else (x * x).sum(-1, keepdim=True)
        y = x / (n2 + 1e-6).sqrt()
        if w is not None:
            y = y * w
        if R > 0:
            pos = s["pos"].long() if s["pos"] is not None else torch.arange(T, device=x.device).expand(B, T)
            turn = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, :, None]
            if c["interleaved"]:
                z = torch.view_as_complex(y[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) * turn
                z = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(y[..., :R // 2], y[..., R // 2:R]) * turn
                z = torch.cat([z.real, z.imag], -1)
            y = torch.cat([z, y[..., R:]], -1)
        outs.append(y)
    if not train:
        return {"q": outs[0].detach(), "k": outs[1].detach()}
    want = [t for t in leaves if t is not None]
    got = iter(torch.autograd.grad(outs, want, (s["dq"].double(), s["dk"].double())))
    dq, dwq, dk, dwk = (None if t is None else next(got) for t in leaves)
    return {"q": outs[0].detach(), "k": outs[1].detach(), "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _exact_conv(s, c):
    W, D = c["W"], c["D"]
    w, b = _leaf(s["w"]), _leaf(s["b"])
    silu = torch.nn.functional.silu if c["silu"] else (lambda p: p)
    if c["mode"] == "step":
        x, h0 = s["x"].double(), s["h0"].double()
        win = torch.cat([h0, x[:, None]], 1)
        p = torch.einsum("nwd,dw->nd", win, w.detach()) + (0 if b is None else b.detach())
        return {"y": silu(p), "state": win[:, 1:]}
    train = c["mode"] == "train"
    spans = _spans(s, c)
    x = s["x"].double()
    h0 = s["h0"].double() if s["h0"] is not None else torch.zeros(len(spans), W - 1, D, device=x.device,
                                                                  dtype=torch.float64)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    hT, dh0 = torch.empty_like(h0), torch.empty_like(h0)
    dw, db = torch.zeros_like(w), torch.zeros(D, device=x.device, dtype=torch.float64)
    for n, r, lo, hi in spans:                 # one sequence at a time, gradients by autograd
        full = torch.cat([h0[n], x[r, lo:hi]], 0).requires_grad_(train)
        with torch.set_grad_enabled(train):
            p = sum(w[:, j] * full[j:j + hi - lo] for j in range(W))
            out = silu(p if b is None else p + b)
            tail = full[hi - lo:]
        y[r, lo:hi], hT[n] = out.detach(), tail.detach()
        if train:
            want = [full, w] + ([b] if b is not None else [])
            got = torch.autograd.grad((out, tail), want, (s["dy"][r, lo:hi].double(), s["dhT"][n].double()))
            dh0[n], dx[r, lo:hi] = got[0][:W - 1], got[0][W - 1:]
            dw += got[1]
            if b is not None:
                db += got[2]
    if not train:
        return {"y": y, "state": hT}
    return {"y": y, "state": hT, "dx": dx, "dw": dw, "db": db if b is not None else None,
            "dh0": dh0 if s["h0"] is not None else None}
