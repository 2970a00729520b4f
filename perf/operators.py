"""Cases of the layer's stand-alone operators: what each computes, in plain torch and through the library.

The operators, on device tensors (T tokens, k picks per token, E experts, row width d):

  sort         rows of the tokens grouped by expert: offsets, the sorted order and the rows themselves
  unsort       the experts' rows back in token order, each weighted by its gate and summed
  unsort_grad  the gradient of unsort: of the rows and of the gates
  norm         RMSNorm or LayerNorm of rows, with the statistics that the backward pass takes
  norm_grad    the gradient of norm: of the rows, of the gain and of the bias
  matvec       few rows times 4-bit weights with a scale per group of inputs, row ranges per expert
  gated        the same with two weight tensors and the gated GELU: gelu(x W) * (x Wv)

Each case is a dict of sizes.  `run` takes what `prepare` made and computes one operator once: in
elementary torch operations, or (own) by the calls of mixture_experts_softmax_b200.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one decode step of eight sequences at the model's width: a few rows, latency counts
        dict(name="sort_decode", op="sort", dtype="bf16", T=8, k=2, E=8, d=6144, drop=0.0),
        # a full context of 8192 tokens
        dict(name="sort_prefill", op="sort", dtype="bf16", T=8192, k=2, E=8, d=6144, drop=0.0),
        # many narrow experts, a ragged batch with dropped routes, rows that are not 16-byte multiples
        dict(name="sort_many_experts", op="sort", dtype="f16", T=4099, k=8, E=160, d=1030, drop=0.1),
        # the way back of a full context: the experts' products in fp32, tokens in bf16
        dict(name="unsort_prefill", op="unsort", dtype="bf16", rows="f32", T=8192, k=2, E=8, d=6144, drop=0.0),
        # a training step on a full context
        dict(name="unsort_grad_prefill", op="unsort_grad", dtype="bf16", rows="bf16", T=8192, k=2, E=8, d=6144,
             drop=0.0),
        # fp32 training with many experts, a padded batch, an odd row width
        dict(name="unsort_grad_ragged", op="unsort_grad", dtype="f32", rows="f32", T=1021, k=6, E=64, d=2051,
             drop=0.25),
        # the residual block's norm of a decode batch
        dict(name="norm_decode", op="norm", kind="rms", dtype="bf16", T=32, d=6144),
        # layer norm over a long fp32 batch of a narrower model
        dict(name="norm_layer_f32", op="norm", kind="layer", dtype="f32", T=16383, d=2560),
        # the residual block's norm in a training step on a full context
        dict(name="norm_grad_prefill", op="norm_grad", kind="rms", dtype="bf16", T=8192, d=6144),
        # layer norm's gradient, fp16, an odd row width
        dict(name="norm_grad_layer_odd", op="norm_grad", kind="layer", dtype="f16", T=5003, d=1537),
        # the down-projection of a single token: its two experts of eight, finer groups, fp32 sums out
        dict(name="down_one_token", op="matvec", dtype="f16", out="f32", R=2, E=8, K=32768, N=6144, group=64),
        # the gated up-projection of a decode step: eight tokens' sixteen routes over all experts
        dict(name="up_decode", op="gated", dtype="bf16", out="bf16", R=16, E=8, K=6144, N=32768, group=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above, at no more than the work of the largest listed case of its operator."""
    op = rng.choice(["sort", "unsort", "unsort_grad", "norm", "norm_grad", "matvec", "gated"])
    limit = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    while True:
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if op in ("sort", "unsort", "unsort_grad"):
            E = _log(rng, 2, 256)
            c = dict(op=op, dtype=dtype, T=_log(rng, 1, 16384), k=rng.randint(1, min(8, E)), E=E, d=_log(rng, 64, 8192),
                     drop=rng.choice([0.0, 0.0, 0.1, 0.5]))
            if op != "sort":
                c["rows"] = rng.choice([dtype, "f32"])
            if rng.random() < 0.6:
                c["d"] = (c["d"] + 7) // 8 * 8
        elif op in ("norm", "norm_grad"):
            c = dict(op=op, kind=rng.choice(["rms", "layer"]), dtype=dtype, T=_log(rng, 1, 16384), d=_log(rng, 64, 16384))
            if rng.random() < 0.6:
                c["d"] = (c["d"] + 7) // 8 * 8
        else:
            E = rng.choice([1, 1, 8, rng.randint(2, 64)])
            x = rng.choice(["bf16", "f16"])
            c = dict(op=op, dtype=x, out=rng.choice([x, "f32"]), R=rng.randint(1, max(16, min(64, 4 * E))), E=E,
                     K=_log(rng, 256, 32768), N=_log(rng, 256, 32768), group=rng.choice([32, 64, 128]))
            if rng.random() < 0.7:
                c["K"], c["N"] = (c["K"] + 127) // 128 * 128, (c["N"] + 31) // 32 * 32
            # the weights that no row touches have to be made too
            if c["E"] * c["K"] * c["N"] > 8 * 6144 * 32768:
                continue
        if work(c)["bytes"] <= limit:
            return c


def _routes(case):
    """Routes that are kept: a set number of them is dropped."""
    n = case["T"] * case["k"]
    return n - int(n * case["drop"])


def work(case):
    op = case["op"]
    es = SIZE[case["dtype"]]
    if op in ("sort", "unsort", "unsort_grad"):
        T, k, d, n = case["T"], case["k"], case["d"], _routes(case)
        if op == "sort":
            # tokens and choices in; rows, offsets, order and slots out
            return dict(bytes=T * d * es + T * k * 4 + n * d * es + (case["E"] + 1) * 4 + 2 * T * k * 4, flops=0)
        rs = SIZE[case["rows"]]
        if op == "unsort":
            return dict(bytes=n * d * rs + 2 * T * k * 4 + T * d * es, flops=2 * n * d)
        return dict(bytes=T * d * es + 2 * n * d * rs + 3 * T * k * 4, flops=3 * n * d)
    if op == "norm":
        T, d = case["T"], case["d"]
        return dict(bytes=2 * T * d * es + 2 * d * es + T * 8, flops=5 * T * d)
    if op == "norm_grad":
        T, d = case["T"], case["d"]
        return dict(bytes=3 * T * d * es + d * es + T * 8 + 2 * d * 4, flops=11 * T * d)
    E, K, N, R = case["E"], case["K"], case["N"], case["R"]
    ws = 2 if op == "gated" else 1
    weights = min(E, R) * (K * N // 2 + -(-K // case["group"]) * N * 2)   # of the experts that rows go to
    return dict(bytes=ws * weights + R * K * es + R * N * SIZE[case["out"]] + (E + 1) * 4, flops=2 * ws * R * K * N)


# ---- inputs ---------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    # drawn in the type itself: large inputs are made many times
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _choices(case, g):
    """Experts of each token, by skewed random scores as a router's; dropped routes are -1."""
    T, k, E = case["T"], case["k"], case["E"]
    score = torch.randn((T, E), generator=g, device="cuda") + torch.randn((E,), generator=g, device="cuda")
    top = score.softmax(-1).topk(k, dim=-1)
    idx = top.indices.to(torch.int32)
    n = T * k - _routes(case)
    if n:
        lost = torch.randperm(T * k, generator=g, device="cuda")[:n]
        idx.view(-1)[lost] = -1
    return idx, top.values.contiguous()


def _rows_per_expert(case, seed):
    """Offsets of the experts' row ranges: every expert has a row where there are enough of them."""
    E, R = case["E"], case["R"]
    g = torch.Generator()
    g.manual_seed(seed)
    count = torch.zeros(E, dtype=torch.int64)
    order = torch.randperm(E, generator=g)
    count[order[:min(E, R)]] = 1
    if R > E:
        count += torch.bincount(torch.randint(0, E, (R - E,), generator=g), minlength=E)
    return torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DT[case["dtype"]]
    st = dict(case=case)
    if op in ("sort", "unsort", "unsort_grad"):
        T, k, E, d = case["T"], case["k"], case["E"], case["d"]
        idx, gate = _choices(case, g)
        if op == "sort":
            st.update(x=_normal(g, (T, d), dt), idx=idx)
            if own:
                st.update(offsets=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                          perm=torch.empty(T * k, dtype=torch.int32, device="cuda"),
                          slot=torch.empty((T, k), dtype=torch.int32, device="cuda"),
                          rows=torch.zeros((T * k, d), dtype=dt, device="cuda"))
        else:
            rt = DT[case["rows"]]
            st.update(rows=_normal(g, (T * k, d), rt), slot=_sort_order(idx, E)[2].to(torch.int32), gate=gate)
            if op == "unsort_grad":
                st["dout"] = _normal(g, (T, d), dt)
            if own and op == "unsort":
                st["out"] = torch.empty((T, d), dtype=dt, device="cuda")
            elif own:
                st.update(drows=torch.zeros((T * k, d), dtype=rt, device="cuda"), dgate=torch.empty_like(gate))
    elif op in ("norm", "norm_grad"):
        T, d = case["T"], case["d"]
        # a residual stream: rows of different sizes, features with a mean of their own
        x = _normal(g, (T, d), torch.float32) * (0.25 + 4 * torch.rand((T, 1), generator=g, device="cuda"))
        st["x"] = (x + _normal(g, (d,), torch.float32)).to(dt)
        del x
        st["gain"] = (1 + 0.2 * _normal(g, (d,), torch.float32)).to(dt)
        st["bias"] = (0.1 * _normal(g, (d,), torch.float32)).to(dt) if case["kind"] == "layer" else None
        st["eps"] = 1e-5
        if op == "norm":
            if own:
                st.update(y=torch.empty_like(st["x"]), stats=torch.empty((T, 2), device="cuda"))
        else:
            st["dy"] = _normal(g, (T, d), dt)
            st["stats"] = _stats(st["x"], case["kind"], st["eps"])
            if own:
                import mixture_experts_softmax_b200 as moe
                st.update(dx=torch.empty_like(st["x"]), dgain=torch.empty(d, device="cuda"),
                          dbias=torch.empty(d, device="cuda") if case["kind"] == "layer" else None,
                          ws=torch.empty(moe.moe_norm_workspace(T, d), dtype=torch.uint8, device="cuda"))
    else:
        E, K, N, R, G = case["E"], case["K"], case["N"], case["R"], case["group"]
        st["x"] = _normal(g, (R, K), dt)
        st["offsets"] = _rows_per_expert(case, seed).cuda()
        names = ("w", "wv") if op == "gated" else ("w",)
        for name in names:
            q = torch.randint(-8, 8, (E, K, N), generator=g, device="cuda", dtype=torch.int8)
            s = (torch.randn((E, -(-K // G), N), generator=g, device="cuda") / (8 * math.sqrt(K))).to(torch.bfloat16)
            if own:
                import mixture_experts_softmax_b200 as moe
                # laid out once, as a program does when it loads its weights
                p = torch.empty(moe.moe_w4_packed_bytes(E, K, N, G), dtype=torch.uint8, device="cuda")
                moe.check(moe.moe_w4_pack(E, K, N, G, q, s, p), "moe_w4_pack")
                st[name] = p
            else:
                st[name] = (q, s)
        if own:
            st["y"] = torch.empty((R, N), dtype=DT[case["out"]], device="cuda")
    return st


# ---- one pass -------------------------------------------------------------------------------


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import mixture_experts_softmax_b200 as moe
    c = st["case"]
    code = {"bf16": moe.MOE_BF16, "f16": moe.MOE_F16, "f32": moe.MOE_F32}
    op, dt = c["op"], code[c["dtype"]]
    if op == "sort":
        moe.check(moe.moe_sort_rows(dt, c["T"], c["k"], c["E"], c["d"], st["x"], st["idx"], st["offsets"], st["perm"],
                                    st["slot"], st["rows"]), "moe_sort_rows")
        return st["offsets"], st["perm"], st["slot"], st["rows"]
    if op == "unsort":
        moe.check(moe.moe_unsort_rows(code[c["rows"]], dt, c["T"], c["k"], c["d"], st["rows"], st["slot"], st["gate"],
                                      st["out"]), "moe_unsort_rows")
        return st["out"]
    if op == "unsort_grad":
        moe.check(moe.moe_unsort_rows_backward(code[c["rows"]], dt, c["T"], c["k"], c["d"], st["dout"], st["rows"],
                                               st["slot"], st["gate"], st["drows"], st["dgate"]),
                  "moe_unsort_rows_backward")
        return st["drows"], st["dgate"]
    if op in ("norm", "norm_grad"):
        kind = moe.MOE_NORM_RMS if c["kind"] == "rms" else moe.MOE_NORM_LAYER
        if op == "norm":
            moe.check(moe.moe_norm_forward(kind, dt, c["T"], c["d"], st["x"], st["gain"], st["bias"], st["eps"],
                                           st["y"], st["stats"]), "moe_norm_forward")
            return st["y"], st["stats"]
        moe.check(moe.moe_norm_backward(kind, dt, c["T"], c["d"], st["x"], st["gain"], st["stats"], st["dy"], st["dx"],
                                        st["dgain"], st["dbias"], st["ws"]), "moe_norm_backward")
        return [t for t in (st["dx"], st["dgain"], st["dbias"]) if t is not None]
    moe.check(moe.moe_w4_matvec(dt, code[c["out"]], c["E"], c["K"], c["N"], c["group"], c["R"], st["x"], st["offsets"],
                                st["w"], st.get("wv"), st["y"]), "moe_w4_matvec")
    return st["y"]


def _sort_order(idx, E):
    """offsets [E+1], perm [T*k] (-1 behind the last row), slot [T, k] (-1: dropped) of a stable sort by expert."""
    flat = idx.reshape(-1).long()
    keep = (flat >= 0) & (flat < E)
    key = torch.where(keep, flat, E)
    order = key.argsort(stable=True)
    count = (key[:, None] == torch.arange(E, device=key.device)[None, :]).sum(0)
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    place = torch.arange(flat.numel(), device=key.device)
    perm = torch.where(place < offsets[E], order, -1)
    slot = torch.empty_like(place)
    slot[order] = torch.where(place < offsets[E], place, -1)
    return offsets, perm, slot.view(idx.shape)


def _stats(x, kind, eps):
    """mean (0 for RMSNorm) and 1 / sqrt(variance + eps) of each row, fp32 [T, 2]."""
    x = x.float()
    mean = x.mean(1) if kind == "layer" else torch.zeros_like(x[:, 0])
    var = ((x - mean[:, None]) ** 2).mean(1)
    return torch.stack([mean, 1 / (var + eps).sqrt()], 1)


def _gelu(a):
    return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))


def _run_plain(st):
    c = st["case"]
    op, dt = c["op"], DT[c["dtype"]]
    if op == "sort":
        offsets, perm, slot = _sort_order(st["idx"], c["E"])
        rows = torch.where((perm >= 0)[:, None], st["x"][perm.clamp(min=0) // c["k"]], 0)
        return offsets.int(), perm.int(), slot.int(), rows.to(dt)
    if op in ("unsort", "unsort_grad"):
        T, k, d = c["T"], c["k"], c["d"]
        slot = st["slot"].long().view(-1)
        keep = slot >= 0
        gate = torch.where(keep, st["gate"].view(-1), 0)
        if op == "unsort":
            picked = torch.where(keep[:, None], st["rows"][slot.clamp(min=0)].float(), 0)
            return (picked * gate[:, None]).view(T, k, d).sum(1).to(dt)
        dout = st["dout"].float()
        dgate = torch.zeros_like(st["gate"])
        drows = torch.zeros(T * k + 1, d, dtype=DT[c["rows"]], device=slot.device)   # the last row takes dropped routes
        to = torch.where(keep, slot, T * k).view(T, k)
        for j in range(k):
            picked = torch.where(keep.view(T, k)[:, j, None], st["rows"][slot.view(T, k)[:, j].clamp(min=0)].float(), 0)
            dgate[:, j] = (dout * picked).sum(1)
            drows[to[:, j]] = (dout * gate.view(T, k)[:, j, None]).to(drows.dtype)
        return drows[:-1], dgate
    if op == "norm":
        stats = _stats(st["x"], c["kind"], st["eps"])
        y = (st["x"].float() - stats[:, :1]) * stats[:, 1:] * st["gain"].float()
        if st["bias"] is not None:
            y = y + st["bias"].float()
        return y.to(dt), stats
    if op == "norm_grad":
        x, dy, stats = st["x"].float(), st["dy"].float(), st["stats"]
        xhat = (x - stats[:, :1]) * stats[:, 1:]
        dgain = (dy * xhat).sum(0)
        dhat = dy * st["gain"].float()
        dx = dhat - xhat * (dhat * xhat).mean(1, keepdim=True)
        if st["bias"] is None:
            return [(dx * stats[:, 1:]).to(dt), dgain]
        dx = dx - dhat.mean(1, keepdim=True)
        return [(dx * stats[:, 1:]).to(dt), dgain, dy.sum(0)]
    y = torch.zeros((c["R"], c["N"]), dtype=torch.float32, device="cuda")
    x, offsets = st["x"].float(), st["offsets"]
    row = torch.arange(c["R"], device="cuda")
    for e in range(c["E"]):
        # a masked product over all rows: the row counts stay on the device
        mine = (row >= offsets[e]) & (row < offsets[e + 1])
        a = x @ _weights(st["w"], e, c, torch.float32)
        if op == "gated":
            a = _gelu(a) * (x @ _weights(st["wv"], e, c, torch.float32))
        y = torch.where(mine[:, None], a, y)
    return y.to(DT[c["out"]])


def _weights(w, e, c, dtype):
    """Expert e's weights, [K, N]: 4-bit values times the scale of their group of inputs."""
    q, s = w
    K, N, G = c["K"], c["N"], c["group"]
    if K % G == 0:
        return (q[e].view(K // G, G, N).to(dtype) * s[e].to(dtype)[:, None, :]).view(K, N)
    return q[e].to(dtype) * s[e].to(dtype).repeat_interleave(G, 0)[:K]


# ---- the definition in 64 bits --------------------------------------------------------------


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, f8 = case["op"], torch.float64
    if op == "sort":
        T, k, E, d = case["T"], case["k"], case["E"], case["d"]
        flat = st["idx"].flatten().cpu()
        perm = torch.full((T * k,), -1, dtype=torch.int32)
        slot = torch.full((T * k,), -1, dtype=torch.int32)
        rows = torch.zeros((T * k, d), dtype=f8, device="cuda")
        offsets = torch.zeros(E + 1, dtype=torch.int32)
        at = 0
        for e in range(E):
            routes = torch.nonzero(flat == e)[:, 0]
            n = routes.numel()
            perm[at:at + n] = routes.int()
            slot[routes] = torch.arange(at, at + n, dtype=torch.int32)
            rows[at:at + n] = st["x"][(routes // k).cuda()].to(f8)
            at += n
            offsets[e + 1] = at
        return offsets, perm, slot.view(T, k), rows
    if op == "unsort":
        T, k, d = case["T"], case["k"], case["d"]
        out = torch.zeros((T, d), dtype=f8, device="cuda")
        for j in range(k):
            t = torch.nonzero(st["slot"][:, j] >= 0)[:, 0]
            out[t] += st["gate"][t, j, None].to(f8) * st["rows"][st["slot"][t, j].long()].to(f8)
        return out
    if op == "unsort_grad":
        T, k, d = case["T"], case["k"], case["d"]
        drows = torch.zeros((T * k, d), dtype=f8, device="cuda")
        dgate = torch.zeros((T, k), dtype=f8, device="cuda")
        for j in range(k):
            t = torch.nonzero(st["slot"][:, j] >= 0)[:, 0]
            r = st["slot"][t, j].long()
            g = st["dout"][t].to(f8)
            dgate[t, j] = torch.einsum("td,td->t", g, st["rows"][r].to(f8))
            drows[r] = g * st["gate"][t, j, None].to(f8)
        return drows, dgate
    if op in ("norm", "norm_grad"):
        x, gain = st["x"].to(f8), st["gain"].to(f8)
        layer = case["kind"] == "layer"
        if op == "norm":
            mean = x.sum(1) / x.shape[1] if layer else torch.zeros_like(x[:, 0])
            x -= mean[:, None]
            rstd = (x.square().sum(1) / x.shape[1] + st["eps"]).rsqrt()
            y = x * rstd[:, None] * gain
            return (y + st["bias"].to(f8) if layer else y), torch.stack([mean, rstd], 1)
        # the gradient at the statistics that the call is given
        mean, rstd = st["stats"].to(f8).unbind(1)
        dy = st["dy"].to(f8)
        h = (x - mean[:, None]) * rstd[:, None]
        d = dy * gain
        n = x.shape[1]
        dx = d - h * (torch.einsum("td,td->t", d, h) / n)[:, None]
        if layer:
            dx -= (d.sum(1) / n)[:, None]
        out = [dx * rstd[:, None], torch.einsum("td,td->d", dy, h)]
        return out + [dy.sum(0)] if layer else out
    K, N, G = case["K"], case["N"], case["group"]
    y = torch.zeros((case["R"], N), dtype=f8, device="cuda")
    offsets = st["offsets"].tolist()
    scale_of = torch.arange(K, device="cuda") // G
    for e in range(case["E"]):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        x = st["x"][a:b].to(f8)
        for n in range(0, N, 4096):
            prod = [x @ (q[e, :, n:n + 4096].to(f8) * s[e, :, n:n + 4096].to(f8)[scale_of])
                    for q, s in (st[name] for name in ("w", "wv") if name in st)]
            if op == "gated":
                u = prod[0]
                gelu = u / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u * u * u)))
                y[a:b, n:n + 4096] = gelu * prod[1]
            else:
                y[a:b, n:n + 4096] = prod[0]
    return y
