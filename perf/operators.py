"""Measured cases of the operators around dense experts: rows sorted by expert and back, and the
matrix products with a fused epilogue (plain and grouped by expert).

Every case has an `op`:
  dispatch           idx [T][K] -> pos, order, offsets (the pairs in expert order) and the pairs'
                     rows rows[pos[t][k]] = x[t]
  dispatch_backward  dx[t] = sum_k drows[pos[t][k]]
  combine            y[t] = residual[t] + sum_k gate[t][k] * z[pos[t][k]]
  combine_backward   dz[pos[t][k]] = gate[t][k] * dy[t], dgate[t][k] = <dy[t], z[pos[t][k]]>
  linear             y = act(x W^T + b) [* (x U^T + c)] [+ residual]
  grouped            the same product of each expert's rows with that expert's weights
A pair whose expert id lies outside [0, experts) is not routed: it has no position (pos = -1) and
adds nothing.

`own` chooses between the plain forms (elementary torch operations in 32 bits) and the calls a
user makes of the package.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "fp64": 8}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _rows(name, op, tokens, top_k, experts, hidden, dtype, pad=0, routed=0, out="", gates="fp64", residual=False):
    return {"name": name, "op": op, "tokens": tokens, "top_k": top_k, "experts": experts, "hidden": hidden,
            "dtype": dtype, "pad": pad, "routed": routed or experts, "out": out or dtype, "gates": gates,
            "residual": residual}


def _linear(name, rows, k, n, dtype, act="none", gated=False, bias=False, residual=False, out=""):
    return {"name": name, "op": "linear", "rows": rows, "k": k, "n": n, "dtype": dtype, "act": act, "gated": gated,
            "bias": bias, "residual": residual, "out": out or dtype}


def _grouped(name, tokens, top_k, experts, k, n, dtype, act="none", gated=False, bias=False, residual=False, out="",
             pad=0, routed=0):
    return {"name": name, "op": "grouped", "tokens": tokens, "top_k": top_k, "experts": experts, "k": k, "n": n,
            "dtype": dtype, "act": act, "gated": gated, "bias": bias, "residual": residual, "out": out or dtype,
            "pad": pad, "routed": routed or experts}


def listed():
    return [
        # one token of a 128-expert layer of hidden 2048 at batch-1 decode: pure latency
        _rows("dispatch_token_bf16", "dispatch", 1, 8, 128, 2048, "bf16"),
        # a long prefill of the same layer, its batch padded at the end
        _rows("dispatch_prefill_bf16", "dispatch", 16384, 8, 128, 2048, "bf16", pad=500),
        # the gradient of a 64-expert, top-6 layer's rows over a ragged batch
        _rows("dispatch_backward_fp16", "dispatch_backward", 4099, 6, 64, 2048, "fp16"),
        # batch-64 decode with the router's fp64 gates, added to the residual stream
        _rows("combine_decode_bf16", "combine", 64, 8, 128, 2048, "bf16", residual=True),
        # fp32 expert outputs of a GPU that holds half of the routed experts
        _rows("combine_prefill_fp32", "combine", 8191, 6, 32, 2048, "fp32", routed=64, out="bf16", gates="fp32",
              residual=True),
        # gradients of the expert outputs and of the gates over a padded training batch
        _rows("combine_backward_bf16", "combine_backward", 4096, 8, 128, 2048, "bf16", pad=37),
        # one token through a square projection added to the residual stream
        _linear("linear_token_bf16", 1, 2048, 2048, "bf16", bias=True, residual=True),
        # always-on experts (two of 1408) of a batch-64 decode step: gate/up with SwiGLU
        _linear("linear_decode_swiglu_bf16", 64, 2048, 2816, "bf16", act="silu", gated=True),
        # the up projection of a wide feed-forward block over a ragged prefill
        _linear("linear_prefill_gelu_fp16", 4099, 2048, 8192, "fp16", act="gelu", bias=True, residual=True),
        # batch-64 decode through 128 experts' gate/up with SwiGLU: every expert's weights are read
        _grouped("grouped_decode_swiglu_bf16", 64, 8, 128, 2048, 768, "bf16", act="silu", gated=True),
        # a 2048-token prefill through the same experts
        _grouped("grouped_prefill_swiglu_bf16", 2048, 8, 128, 2048, 768, "bf16", act="silu", gated=True),
        # the down projection of a prefill, with a bias and fp32 outputs
        _grouped("grouped_prefill_down_fp16", 2040, 8, 128, 768, 2048, "fp16", bias=True, out="fp32", pad=9),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("dispatch", "dispatch_backward", "combine", "combine_backward", "linear", "grouped"))
    dtype = rng.choice(("bf16", "fp16", "fp32") if op not in ("linear", "grouped") else ("bf16", "fp16"))
    if op == "linear":
        rows = _log(rng, 1, 8192)
        k = 8 * _log(rng, 8, 1024)
        n = _log(rng, 16, 8192)
        gated = rng.random() < 0.4
        while 2 * rows * n * k * (2 if gated else 1) > 1.3e11:
            rows = max(1, rows // 2)
        return _linear("", rows, k, n, dtype, act=rng.choice(ACTS), gated=gated, bias=rng.random() < 0.5,
                       residual=rng.random() < 0.5, out=rng.choice((dtype, "fp32")))
    top_k = rng.randint(1, 8)
    routed = max(top_k, _log(rng, 4, 256))
    experts = routed if rng.random() < 0.7 else max(1, routed // 2)
    if op == "grouped":
        tokens = _log(rng, 1, 4096)
        k = 8 * _log(rng, 8, 512)
        n = _log(rng, 16, 4096)
        gated = rng.random() < 0.5
        while experts * k * n * (2 if gated else 1) > 2.0e8:
            n = max(16, n // 2)
        while 2 * tokens * top_k * k * n * (2 if gated else 1) > 1.0e11:
            tokens = max(1, tokens // 2)
        return _grouped("", tokens, top_k, experts, k, n, dtype, act=rng.choice(ACTS), gated=gated,
                        bias=rng.random() < 0.5, residual=rng.random() < 0.3, out=rng.choice((dtype, "fp32")),
                        pad=rng.choice((0, tokens // 7)), routed=routed)
    tokens = _log(rng, 1, 16384)
    hidden = _log(rng, 64, 4096)
    if rng.random() < 0.75:
        hidden = (hidden + 7) // 8 * 8
    while tokens * top_k * hidden * BYTES[dtype] > (3.5e8 if op == "combine_backward" else 5.0e8):
        tokens //= 2
    return _rows("", op, tokens, top_k, experts, hidden, dtype, pad=rng.choice((0, tokens // 9)), routed=routed,
                 out=rng.choice((dtype, "fp32")) if op == "combine" else "", gates=rng.choice(("fp32", "fp64")),
                 residual=op == "combine" and rng.random() < 0.5)


def _routing(case, gen):
    """Expert ids int32 [T][K] (distinct per token, some experts busier than others) and gates."""
    T, K, E = case["tokens"], case["top_k"], case["routed"]
    logits = torch.randn((T, E), generator=gen, device="cuda") + torch.randn((E,), generator=gen, device="cuda")
    top = torch.topk(logits, K, dim=1)
    idx = top.indices.to(torch.int32)
    if case["pad"]:
        idx[T - case["pad"]:] = -1      # a padded token routes nowhere
    gates = torch.softmax(top.values.double(), dim=1)
    return idx.contiguous(), gates.to(torch.float32 if case.get("gates") == "fp32" else torch.float64).contiguous()


def _sort_plain(idx, experts):
    key = torch.where((idx >= 0) & (idx < experts), idx, experts).reshape(-1)
    sorted_key, order = torch.sort(key, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=idx.device)
    pos = torch.where(key < experts, pos, -1).reshape(idx.shape)
    edges = torch.arange(experts + 1, device=idx.device, dtype=sorted_key.dtype)
    offsets = torch.searchsorted(sorted_key, edges)
    return pos.to(torch.int32), order.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=case["dtype"], scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(DTYPES[dtype])

    s = {"case": case}
    op = case["op"]
    if op in ("linear", "grouped"):
        k, n, lead = case["k"], case["n"], ()
        if op == "grouped":
            idx, _ = _routing(case, gen)
            _, _, s["offsets"] = _sort_plain(idx, case["experts"])
            s["edges"] = s["offsets"].tolist()    # for the plain form's loop over the experts
            rows, lead = idx.numel(), (case["experts"],)
        else:
            rows = case["rows"]
        s["x"] = normal(rows, k)
        s["w"] = normal(*lead, n, k, scale=0.02)
        s["w_mul"] = normal(*lead, n, k, scale=0.02) if case["gated"] else None
        s["bias"] = normal(*lead, n, scale=0.1) if case["bias"] else None
        s["bias_mul"] = normal(*lead, n, scale=0.1) if case["bias"] and case["gated"] else None
        s["residual"] = normal(rows, n, dtype=case["out"]) if case["residual"] else None
        s["out"] = torch.zeros((rows, n), dtype=DTYPES[case["out"]], device="cuda")
    else:
        T, K, H = case["tokens"], case["top_k"], case["hidden"]
        s["idx"], s["gates"] = _routing(case, gen)
        if op == "dispatch":
            s["x"] = normal(T, H)
            s["rows"] = torch.zeros((T * K, H), dtype=DTYPES[case["dtype"]], device="cuda")
        else:
            s["pos"], _, _ = _sort_plain(s["idx"], case["experts"])
            if op == "dispatch_backward":
                s["drows"] = normal(T * K, H)
            else:
                s["z"] = normal(T * K, H)
        if op == "combine":
            s["residual"] = normal(T, H, dtype=case["out"]) if case["residual"] else None
        if op == "combine_backward":
            s["dy"] = normal(T, H)
            s["dz"] = torch.zeros((T * K, H), dtype=DTYPES[case["dtype"]], device="cuda")
    if own:
        from dynamic_any_precision_b200 import dpa
        if op == "dispatch":
            s["ws"] = dpa.new_sort_workspace(case["tokens"] * case["top_k"], case["experts"], device="cuda")
        elif op in ("linear", "grouped"):
            s["ws"] = dpa.new_linear_workspace(device="cuda")
    return s


def _act(v, act):
    if act == "relu":
        return torch.clamp_min(v, 0.0)
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))    # no cancellation for negative v
    if act == "gelu_tanh":
        # 0.5 v (1 + tanh(p)) = v / (1 + exp(-2p)), without cancellation for negative v
        return v / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _product_plain(x, w, bias, act, w_mul, bias_mul, residual, out_dtype):
    x = x.float()
    v = x @ w.float().T
    if bias is not None:
        v = v + bias.float()
    v = _act(v, act)
    if w_mul is not None:
        u = x @ w_mul.float().T
        v = v * (u + bias_mul.float() if bias_mul is not None else u)
    if residual is not None:
        v = v + residual.float()
    return v.to(out_dtype)


def _gathered(rows, pos):
    """rows[pos] in 32 bits, [T][K][H], zero where pos is -1."""
    got = rows[pos.clamp_min(0).long()].float()
    return torch.where((pos >= 0)[:, :, None], got, 0.0)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "dispatch":
        pos, order, offsets = _sort_plain(s["idx"], case["experts"])
        live = torch.arange(order.numel(), device=order.device) < offsets[-1]
        rows = s["x"][(order // case["top_k"]).long()]
        return {"pos": pos, "order": order, "offsets": offsets, "rows": torch.where(live[:, None], rows, 0.0)}
    if op == "dispatch_backward":
        return _gathered(s["drows"], s["pos"]).sum(dim=1).to(s["drows"].dtype)
    if op == "combine":
        y = (_gathered(s["z"], s["pos"]) * s["gates"].float()[:, :, None]).sum(dim=1)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(DTYPES[case["out"]])
    if op == "combine_backward":
        pos, dy = s["pos"], s["dy"].float()
        dgates = (_gathered(s["z"], pos) * dy[:, None, :]).sum(dim=2)
        weighted = (s["gates"].float()[:, :, None] * dy[:, None, :]).to(s["dz"].dtype)
        P = pos.numel()
        dz = torch.zeros((P + 1, dy.shape[1]), dtype=s["dz"].dtype, device=dy.device)
        dz[torch.where(pos >= 0, pos, P).long().reshape(-1)] = weighted.reshape(P, -1)
        return {"dz": dz[:P], "dgates": dgates}
    part = (case["act"],)
    if op == "linear":
        return _product_plain(s["x"], s["w"], s["bias"], *part, s["w_mul"], s["bias_mul"], s["residual"],
                              DTYPES[case["out"]])
    y = torch.zeros_like(s["out"])
    for e in range(case["experts"]):
        a, b = s["edges"][e], s["edges"][e + 1]
        if a < b:
            pick = [None if s[name] is None else s[name][e] for name in ("bias", "w_mul", "bias_mul")]
            res = None if s["residual"] is None else s["residual"][a:b]
            y[a:b] = _product_plain(s["x"][a:b], s["w"][e], pick[0], *part, pick[1], pick[2], res, y.dtype)
    return y


def _run_own(s):
    from dynamic_any_precision_b200 import dpa

    case = s["case"]
    op = case["op"]
    if op == "dispatch":
        pos, order, offsets = dpa.sort_pairs(s["idx"], case["experts"], s["ws"])
        return {"pos": pos, "order": order, "offsets": offsets, "rows": dpa.permute_rows(s["x"], pos, out=s["rows"])}
    if op == "dispatch_backward":
        return dpa.permute_rows_backward(s["drows"], s["pos"])
    if op == "combine":
        return dpa.unpermute_rows(s["z"], s["pos"], s["gates"], residual=s["residual"], out_dtype=DTYPES[case["out"]])
    if op == "combine_backward":
        dz, dgates = dpa.unpermute_rows_backward(s["dy"], s["z"], s["pos"], s["gates"], dz=s["dz"])
        return {"dz": dz, "dgates": dgates}
    rest = dict(bias=s["bias"], act=case["act"], w_mul=s["w_mul"], bias_mul=s["bias_mul"], residual=s["residual"],
                out=s["out"])
    if op == "linear":
        return dpa.linear(s["x"], s["w"], s["ws"], **rest)
    return dpa.grouped_linear(s["x"], s["offsets"], s["w"], s["ws"], **rest)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op in ("linear", "grouped"):
        mats = 2 if case["gated"] else 1
        k, n = case["k"], case["n"]
        if op == "linear":
            rows, used = case["rows"], 1
        else:
            rows = (case["tokens"] - case["pad"]) * case["top_k"] * case["experts"] // case["routed"]
            used = min(case["experts"], rows)
        es, eo = BYTES[case["dtype"]], BYTES[case["out"]]
        size = used * mats * n * (k + (1 if case["bias"] else 0)) * es + rows * k * es + rows * n * eo
        if case["residual"]:
            size += rows * n * eo
        return {"bytes": size, "flops": 2 * rows * n * k * mats}
    T, K, H = case["tokens"], case["top_k"], case["hidden"]
    tokens = T - case["pad"]
    live = tokens * K * case["experts"] // case["routed"]
    es = BYTES[case["dtype"]]
    if op == "dispatch":
        return {"bytes": 12 * T * K + 4 * case["experts"] + tokens * H * es + live * H * es, "flops": 0}
    if op == "dispatch_backward":
        return {"bytes": 4 * T * K + live * H * es + T * H * es, "flops": live * H}
    gates = T * K * (4 + BYTES[case["gates"]])
    if op == "combine":
        eo = BYTES[case["out"]]
        return {"bytes": gates + live * H * es + T * H * eo * (2 if case["residual"] else 1), "flops": 2 * live * H}
    return {"bytes": gates + 4 * T * K + 2 * live * H * es + T * H * es, "flops": 3 * live * H}


def _act64(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "silu":
        return v * torch.sigmoid(v)
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "grouped"):
        rows = s["x"].shape[0]
        spans = [(0, rows, None)]
        if op == "grouped":
            spans = [(s["edges"][e], s["edges"][e + 1], e) for e in range(case["experts"])]
        y = torch.zeros((rows, case["n"]), dtype=torch.float64, device="cuda")
        for a, b, e in spans:
            if a == b:
                continue

            def of(name):
                t = s[name]
                return None if t is None else (t if e is None else t[e]).double()

            x = s["x"][a:b].double()
            bias = of("bias")
            v = torch.einsum("mk,nk->mn", x, of("w"))
            v = _act64(v if bias is None else v + bias, case["act"])
            if case["gated"]:
                u = torch.einsum("mk,nk->mn", x, of("w_mul"))
                v = v * (u if bias is None else u + of("bias_mul"))
            y[a:b] = v if s["residual"] is None else v + s["residual"][a:b].double()
        return y
    T, K, H, E = case["tokens"], case["top_k"], case["hidden"], case["experts"]
    ids = s["idx"].cpu().numpy().reshape(-1)
    runs = [np.flatnonzero(ids == e) for e in range(E)]
    order = np.concatenate(runs + [np.flatnonzero((ids < 0) | (ids >= E))])
    live = sum(len(r) for r in runs)
    token = torch.from_numpy(order[:live] // K).cuda()
    slot = torch.from_numpy(order[:live] % K).cuda()
    if op == "dispatch":
        pos = np.full(T * K, -1, np.int32)
        pos[order[:live]] = np.arange(live)
        rows = torch.zeros((T * K, H), dtype=torch.float64, device="cuda")
        rows[:live] = s["x"].double()[token]
        offsets = np.concatenate([[0], np.cumsum([len(r) for r in runs])])
        return {"pos": torch.from_numpy(pos.reshape(T, K)).cuda(),
                "order": torch.from_numpy(order.astype(np.int32)).cuda(),
                "offsets": torch.from_numpy(offsets.astype(np.int32)).cuda(), "rows": rows}
    gates = s["gates"].double()
    if op in ("dispatch_backward", "combine"):
        src = s["drows"] if op == "dispatch_backward" else s["z"]
        y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        for k in range(K):      # each token has at most one position per slot
            at = (slot == k).nonzero()[:, 0]
            rows = src[at].double()
            if op == "combine":
                rows = rows * gates[token[at], k][:, None]
            y[token[at]] += rows
        if op == "combine" and s["residual"] is not None:
            y += s["residual"].double()
        return y
    dz = torch.zeros((T * K, H), dtype=torch.float64, device="cuda")
    dgates = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    for k in range(K):
        at = (slot == k).nonzero()[:, 0]
        dy = s["dy"].double()[token[at]]
        dz[at] = dy * gates[token[at], k][:, None]
        dgates[token[at], k] = (s["z"][at].double() * dy).sum(dim=1)
    return {"dz": dz, "dgates": dgates}
