"""The operators of the 16-bit expert path, as they are measured: grouped products, SwiGLU and low-rank adapters.

A case is one call: a product of ragged groups of rows with each group's own matrix (``product``), the gradient of
its rows (``rows_grad``) or of its matrices (``weights_grad``), the SwiGLU between an expert's two products
(``swiglu``) and its gradient (``swiglu_grad``), or a shared projection with the low-rank adapters of many requests
(``adapters``).  ``run`` computes it in its plain form (elementary torch operations in fp32, rounded once) or, with
``own``, through the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    """The layer's own shape is d = 2048, f = 768, 512 experts, top-10 (tiny: d = 256, f = 128, 16 experts, top-2)."""
    return [
        # one decoded token: its ten experts' gate and up matrices, each read for one row
        {"name": "product, 1 token", "op": "product", "experts": 512, "rows": 10, "n": 1536, "k": 2048,
         "spread": "flat", "dtype": "bf16", "behind": 0},
        # a verify or small serving batch of 64 tokens: most groups hold a few rows
        {"name": "product, 64 tokens", "op": "product", "experts": 512, "rows": 640, "n": 1536, "k": 2048,
         "spread": "zipf", "dtype": "bf16", "behind": 0},
        # a whole prefill chunk of 8192 tokens at top-10, uneven groups
        {"name": "product, prefill chunk", "op": "product", "experts": 512, "rows": 81920, "n": 1536, "k": 2048,
         "spread": "zipf", "dtype": "bf16", "behind": 0},
        # fine-tuning a 64-expert layer: the down product's input gradient, with unused rows behind the groups
        {"name": "rows_grad, 64 experts", "op": "rows_grad", "experts": 64, "rows": 40003, "n": 2048, "k": 768,
         "spread": "zipf", "dtype": "bf16", "behind": 61},
        # the same layer's gate/up weight gradient, 16 bits
        {"name": "weights_grad, 64 experts", "op": "weights_grad", "experts": 64, "rows": 40003, "n": 1536, "k": 2048,
         "spread": "zipf", "dtype": "bf16", "out": "bf16", "accumulate": False, "behind": 61},
        # gradient accumulation in fp32 over odd sizes and empty groups
        {"name": "weights_grad, odd sizes", "op": "weights_grad", "experts": 16, "rows": 3001, "n": 200, "k": 328,
         "spread": "holes", "dtype": "fp16", "out": "fp32", "accumulate": True, "behind": 0},
        # SwiGLU of a 64-token batch, weighted by the routing weights
        {"name": "swiglu, 64 tokens", "op": "swiglu", "rows": 640, "f": 768, "weighted": True, "dtype": "bf16",
         "behind": 0},
        # its gradient for a training chunk, with the activations recomputed for the down weights' gradient
        {"name": "swiglu_grad, 81920 rows", "op": "swiglu_grad", "rows": 81920, "f": 768, "weighted": True,
         "dtype": "bf16", "behind": 0},
        # one decoded token with its request's adapter
        {"name": "adapters, 1 token", "op": "adapters", "tokens": 1, "n": 2048, "k": 2048, "rank": 16, "loaded": 32,
         "layout": "requests", "projection": True, "accumulate": False, "dtype": "bf16", "out": "bf16"},
        # a decode batch in which every token is another request
        {"name": "adapters, 48 requests", "op": "adapters", "tokens": 48, "n": 2048, "k": 2048, "rank": 16,
         "loaded": 64, "layout": "mixed", "projection": True, "accumulate": False, "dtype": "bf16", "out": "bf16"},
        # a prefill chunk of a few requests
        {"name": "adapters, prefill chunk", "op": "adapters", "tokens": 8192, "n": 2048, "k": 2048, "rank": 32,
         "loaded": 16, "layout": "requests", "projection": True, "accumulate": False, "dtype": "bf16", "out": "bf16"},
        # adapters added to a layer's fp32 output, no projection of their own
        {"name": "adapters, beside a layer", "op": "adapters", "tokens": 1500, "n": 2048, "k": 2048, "rank": 64,
         "loaded": 24, "layout": "requests", "projection": False, "accumulate": True, "dtype": "fp16", "out": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, lo, hi):
    return 8 * _log(rng, lo // 8, hi // 8)


def draw(rng):
    op = rng.choice(["product", "product", "rows_grad", "weights_grad", "swiglu", "swiglu_grad", "adapters", "adapters"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    behind = rng.choice([0, 0, rng.randint(1, 300)])
    if op in ("product", "rows_grad", "weights_grad"):
        c = {"op": op, "experts": _log(rng, 1, 512), "rows": _log(rng, 1, 81920), "n": _eights(rng, 64, 2048),
             "k": _eights(rng, 64, 2048), "spread": rng.choice(["flat", "zipf", "zipf", "holes"]), "dtype": dtype,
             "behind": behind}
        if op == "weights_grad":
            c["experts"] = min(c["experts"], 64)
            c["rows"] = min(c["rows"], 40003)
            c["out"] = rng.choice([dtype, "fp32"])
            c["accumulate"] = c["out"] == "fp32" and rng.random() < 0.5
        return c
    if op in ("swiglu", "swiglu_grad"):
        return {"op": op, "rows": _log(rng, 1, 81920), "f": _eights(rng, 64, 2048), "weighted": rng.random() < 0.5,
                "dtype": dtype, "behind": behind}
    projection = rng.random() < 0.6
    return {"op": op, "tokens": _log(rng, 1, 8192), "n": _eights(rng, 256, 4096), "k": _eights(rng, 256, 4096),
            "rank": rng.choice([8, 16, 16, 24, 32, 64]), "loaded": _log(rng, 1, 64),
            "layout": rng.choice(["requests", "requests", "mixed"]), "projection": projection,
            "accumulate": not projection and rng.random() < 0.7, "dtype": dtype,
            "out": rng.choice([dtype, dtype, "fp32"])}


# ------------------------------------------------------------------------------------------------ inputs
def _sizes(case, g):
    """Rows of each group: one each or even (flat), a router's uneven load (zipf), mostly empty groups (holes)."""
    E, rows = case["experts"], case["rows"]
    if case["spread"] == "flat":
        # the rows go to distinct groups in turn, from a random one on
        order = torch.randperm(E, generator=g, device="cuda")
        ids = order[torch.arange(rows, device="cuda") % E]
    else:
        # a router's choice: each token takes its top k of noise plus a popularity prior (Zipf 1.1), no expert twice
        k = max(1, min(10, E // 4))
        prior = -1.1 * torch.arange(1, E + 1, device="cuda", dtype=torch.float32).log()
        if case["spread"] == "holes":
            prior[1::2] = -1e4
        noise = torch.rand((rows + k - 1) // k, E, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
        ids = (prior - (-noise.log()).log()).topk(k, dim=1).indices.flatten()[:rows]
        ids = torch.randperm(E, generator=g, device="cuda")[ids]
    return torch.bincount(ids, minlength=E)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        return t.normal_(0.0, scale, generator=g)

    s = {"case": case}
    op = case["op"]
    if op in ("product", "rows_grad", "weights_grad"):
        E, N, K, M = case["experts"], case["n"], case["k"], case["rows"] + case["behind"]
        sizes = _sizes(case, g)
        s["offsets"] = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).to(torch.int32)
        ends = s["offsets"].tolist()  # the plain form walks the groups on the host
        s["groups"] = [(e, ends[e], ends[e + 1]) for e in range(E) if ends[e + 1] > ends[e]]
        if op != "weights_grad":
            s["w"] = normal(E, N, K, scale=0.02)
            s["x"] = normal(M, K if op == "product" else N)
            s["out"] = torch.zeros(M, N if op == "product" else K, dtype=dt, device="cuda")
        else:
            s["dy"], s["x"] = normal(M, N), normal(M, K)
            s["out"] = torch.zeros(E, N, K, dtype=DTYPES[case["out"]], device="cuda")
            if case["accumulate"]:
                s["before"] = normal(E, N, K, dtype=torch.float32)
    elif op in ("swiglu", "swiglu_grad"):
        M, f = case["rows"] + case["behind"], case["f"]
        s["gu"] = normal(M, 2 * f)
        s["rw"] = torch.rand(M, generator=g, device="cuda") if case["weighted"] else None
        s["n_rows"] = torch.tensor([case["rows"]], dtype=torch.int32, device="cuda")
        s["h"] = torch.zeros(M, f, dtype=dt, device="cuda")
        if op == "swiglu_grad":
            s["dh"] = normal(M, f)
            s["dgu"] = torch.zeros(M, 2 * f, dtype=dt, device="cuda")
            s["drw"] = torch.zeros(M, device="cuda") if case["weighted"] else None
    else:
        T, N, K, r, L = case["tokens"], case["n"], case["k"], case["rank"], case["loaded"]
        s["x"] = normal(T, K)
        s["w"] = normal(N, K, scale=0.02) if case["projection"] else None
        s["a"] = normal(L, r, K, scale=1.0 / math.sqrt(K))
        s["b"] = normal(L, N, r, scale=0.1)
        s["scale"] = 0.5 + torch.rand(L, generator=g, device="cuda")
        if case["layout"] == "requests":  # a few requests of many tokens each, one after the other
            cuts = torch.randint(0, T + 1, (min(T, 7),), generator=g, device="cuda").sort().values
            part = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
            one = torch.randint(-1 if L > 1 else 0, L, (8,), generator=g, device="cuda")
            ids = one[part]
        else:  # every token its own request, some without an adapter
            ids = torch.randint(-1, L, (T,), generator=g, device="cuda")
        s["ids"] = ids.to(torch.int32)
        if case["accumulate"]:
            s["before"] = normal(T, N, dtype=DTYPES[case["out"]])
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _plain_product(s, transpose):
    out = s["out"]
    for e, lo, hi in s["groups"]:
        w = s["w"][e].float()
        out[lo:hi] = s["x"][lo:hi].float() @ (w if transpose else w.T)
    return out


def _plain_weights_grad(s):
    out = s["out"]
    out.copy_(s["before"]) if "before" in s else out.zero_()
    for e, lo, hi in s["groups"]:
        dw = s["dy"][lo:hi].float().T @ s["x"][lo:hi].float()
        out[e] = out[e] + dw if "before" in s else dw
    return out


def _plain_swiglu(s):
    rows, f = s["case"]["rows"], s["case"]["f"]
    gate, up = s["gu"][:rows, :f].float(), s["gu"][:rows, f:].float()
    h = gate / (1 + torch.exp(-gate)) * up
    s["h"][:rows] = h * s["rw"][:rows, None] if s["rw"] is not None else h
    return s["h"]


def _plain_swiglu_grad(s):
    rows, f = s["case"]["rows"], s["case"]["f"]
    gate, up, dh = s["gu"][:rows, :f].float(), s["gu"][:rows, f:].float(), s["dh"][:rows].float()
    sig = 1 / (1 + torch.exp(-gate))
    act = gate * sig
    h, dhw = act * up, dh
    if s["rw"] is not None:
        rw = s["rw"][:rows, None]
        s["drw"][:rows] = (h * dh).sum(1)
        h, dhw = h * rw, dh * rw
    s["h"][:rows] = h
    s["dgu"][:rows, :f] = dhw * up * sig * (1 + gate * (1 - sig))
    s["dgu"][:rows, f:] = dhw * act
    return (s["dgu"], s["h"]) + ((s["drw"],) if s["rw"] is not None else ())


def _plain_adapters(s):
    case, x, ids = s["case"], s["x"].float(), s["ids"].long()
    T, N, r, L = case["tokens"], case["n"], case["rank"], case["loaded"]
    used = (ids >= 0).float()
    at = ids.clamp(min=0)
    weight = (used * s["scale"][at])[:, None]
    if T <= L:  # each token's own adapter
        v = torch.bmm(s["a"][at].float(), x[:, :, None])
        y = torch.bmm(s["b"][at].float(), v)[:, :, 0] * weight
    else:  # all adapters at once, the token's own kept
        v = (x @ s["a"].float().reshape(L * r, -1).T).reshape(T, L, r)
        own_v = v.gather(1, at[:, None, None].expand(T, 1, r)) * weight[:, :, None]
        v = torch.zeros_like(v).scatter_(1, at[:, None, None].expand(T, 1, r), own_v)
        y = v.reshape(T, L * r) @ s["b"].float().transpose(1, 2).reshape(L * r, N)
    if s["w"] is not None:
        y = y + x @ s["w"].float().T
    if "before" in s:
        y = y + s["before"].float()
    return y.to(DTYPES[case["out"]])


def _plain(s):
    op = s["case"]["op"]
    if op in ("product", "rows_grad"):
        return _plain_product(s, op == "rows_grad")
    if op == "weights_grad":
        return _plain_weights_grad(s)
    return {"swiglu": _plain_swiglu, "swiglu_grad": _plain_swiglu_grad, "adapters": _plain_adapters}[op](s)


# ------------------------------------------------------------------------------------------------ the library's calls
def _own(s):
    import bit_expert_ffn_gemv_b200 as moe
    case, op = s["case"], s["case"]["op"]
    if op in ("product", "rows_grad"):
        return moe.grouped_matmul(s["x"], s["w"], s["offsets"], out=s["out"], transpose=op == "rows_grad")
    if op == "weights_grad":
        if "before" in s:
            s["out"].copy_(s["before"])
        return moe.grouped_matmul_wgrad(s["dy"], s["x"], s["offsets"], out=s["out"], accumulate="before" in s)
    if op == "swiglu":
        return moe.swiglu(s["gu"], s["rw"], out=s["h"], n_rows=s["n_rows"])
    if op == "swiglu_grad":
        dgu, h, drw = moe.swiglu_backward(s["gu"], s["dh"], s["rw"], dgu=s["dgu"], h=s["h"], drw=s["drw"],
                                          n_rows=s["n_rows"])
        return (dgu, h) + ((drw,) if drw is not None else ())
    flags = (moe.MOE_OUT_FP32 if case["out"] == "fp32" else 0) | (moe.MOE_ACCUMULATE if "before" in s else 0)
    out = s["before"].clone() if "before" in s else None
    return moe.adapter_project(s["x"], s["a"], s["b"], s["ids"], w=s["w"], scale=s["scale"], out=out, flags=flags)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    op, size = case["op"], {"bf16": 2, "fp16": 2, "fp32": 4}
    if op in ("product", "rows_grad", "weights_grad"):
        E, N, K, M = case["experts"], case["n"], case["k"], case["rows"]
        if op == "weights_grad":
            moved = 2 * M * (N + K) + E * N * K * size[case["out"]] * (2 if case["accumulate"] else 1)
        else:
            # groups that hold a row, as expected of the spread
            if case["spread"] == "flat":
                active = min(E, M)
            else:
                p = [i ** -1.1 for i in range(1, E + 1)]
                if case["spread"] == "holes":
                    p[1::2] = [0.0] * (E // 2)
                active = sum(1 - (1 - v / sum(p)) ** M for v in p)
            moved = 2 * M * (N + K) + 2 * active * N * K + 4 * (E + 1)
        return {"bytes": moved, "flops": 2 * M * N * K}
    if op in ("swiglu", "swiglu_grad"):
        M, f = case["rows"], case["f"]
        extra = 4 * M * case["weighted"]
        return {"bytes": 2 * M * f * (3 if op == "swiglu" else 6) + extra * (1 if op == "swiglu" else 2),
                "flops": M * f * (6 if op == "swiglu" else 14)}
    T, N, K, r, L = case["tokens"], case["n"], case["k"], case["rank"], case["loaded"]
    # at most seven cuts make eight requests; their adapters are drawn with "none" among them
    drawn = min(T, 8) if case["layout"] == "requests" else T
    used = L * (1 - (1 - 1 / (L + 1)) ** drawn)
    moved = 2 * T * K + T * N * size[case["out"]] * (2 if case["accumulate"] else 1) + 2 * used * r * (K + N) + 4 * T
    flops = 2 * T * r * (K + N)
    if case["projection"]:
        moved += 2 * N * K
        flops += 2 * T * N * K
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op in ("product", "rows_grad"):
        y = torch.zeros(s["out"].shape, dtype=d, device="cuda")
        for e, lo, hi in s["groups"]:
            spec = "rk,nk->rn" if op == "product" else "rn,nk->rk"
            y[lo:hi] = torch.einsum(spec, s["x"][lo:hi].to(d), s["w"][e].to(d))
        return y
    if op == "weights_grad":
        dw = s["before"].to(d) if "before" in s else torch.zeros(s["out"].shape, dtype=d, device="cuda")
        for e, lo, hi in s["groups"]:
            dw[e] += torch.einsum("rn,rk->nk", s["dy"][lo:hi].to(d), s["x"][lo:hi].to(d))
        return dw
    if op in ("swiglu", "swiglu_grad"):
        rows, f = case["rows"], case["f"]
        gu = s["gu"][:rows].to(d)
        w = s["rw"][:rows].to(d)[:, None] if s["rw"] is not None else torch.ones(rows, 1, dtype=d, device="cuda")
        gate, up = gu.split(f, dim=1)
        sig = torch.sigmoid(gate)

        def whole(v):
            out = torch.zeros((s["gu"].shape[0],) + tuple(v.shape[1:]), dtype=d, device="cuda")
            out[:rows] = v
            return out

        h = whole(w * gate * sig * up)
        if op == "swiglu":
            return h
        dh = s["dh"][:rows].to(d)
        slope = sig + gate * sig * (1 - sig)
        dgu = whole(torch.cat([w * dh * up * slope, w * dh * gate * sig], dim=1))
        if s["rw"] is None:
            return dgu, h
        return dgu, h, whole((dh * gate * sig * up).sum(1))
    x, ids = s["x"].to(d), s["ids"].long()
    y = torch.zeros(case["tokens"], case["n"], dtype=d, device="cuda")
    if s["w"] is not None:
        y += torch.einsum("tk,nk->tn", x, s["w"].to(d))
    for a in range(case["loaded"]):
        mine = (ids == a).nonzero()[:, 0]
        v = torch.einsum("tk,rk->tr", x[mine], s["a"][a].to(d))
        y[mine] += float(s["scale"][a]) * torch.einsum("tr,nr->tn", v, s["b"][a].to(d))
    if "before" in s:
        y += s["before"].to(d)
    return y
