"""Workloads of the expert-grouped linear layer and of the block norm, with a
plain torch form of each operator.

Operators
  route    router: top-k softmax over expert logits, and the permutation that
           sorts the (token, expert) pairs by expert
  gemm     W4A4 products grouped by expert, on quantized activations
  linear   the same from bf16 rows: gather (or SwiGLU), quantize, multiply
  norm     block norm: expert combine, norm of the branch, gate, residual
           update, norm of the stream, NVFP4 or dense output

With ``own`` false, run() computes the plain form (FP32 torch operations);
with ``own`` true it calls this repository's library.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of 8 requests through a 64-expert router: latency
        dict(name="route decode", op="route", M=8, E=64, k=8, dtype="f32", renorm=True, masked=0.0),
        # a batch of prompts, bf16 logits (ties happen), some experts masked out for some tokens
        dict(name="route prompt", op="route", M=16384, E=128, k=8, dtype="bf16", renorm=False, masked=0.05),
        # decode: 64 rows over 64 experts, about one row each; the weights are streamed once
        dict(name="gemm decode", op="gemm", T=64, spare=0, E=64, N=2048, K=5120, out="bf16", skew=0.5),
        # odd everything, FP32 out, a buffer with 24 unused rows behind the last group
        dict(name="gemm ragged", op="gemm", T=1000, spare=24, E=24, N=1000, K=1056, out="f32", skew=1.0),
        # prompts: 512 rows an expert on average, tensor-core bound
        dict(name="gemm prompt", op="gemm", T=32768, spare=0, E=64, N=2048, K=5120, out="bf16", skew=0.5),
        # decode of 8 tokens with 8 experts each, from the hidden state
        dict(name="linear decode", op="linear", M=8, k=8, E=64, N=2048, K=5120, act="none", x="bf16", out="bf16"),
        # prompts through the up projections: every token is gathered 8 times
        dict(name="linear prompt", op="linear", M=2048, k=8, E=64, N=2048, K=5120, act="none", x="bf16", out="bf16"),
        # down projection: SwiGLU of the up projections' output, quantized, multiplied
        dict(name="linear swiglu", op="linear", M=2003, k=8, E=64, N=5120, K=1024, act="swiglu", x="bf16", out="bf16"),
        # end of an expert block at decode: combine 8 expert rows, residual, next norm, NVFP4
        dict(name="norm decode", op="norm", M=8, K=5120, k=8, heads=0, post=False, gate="none", residual=True,
             pre=True, quant=True, dense=False, dtype="bf16"),
        # block norm over a prompt: residual update and the next block's norm
        dict(name="norm prompt", op="norm", M=16384, K=5120, k=0, heads=0, post=False, gate="none", residual=True,
             pre=True, quant=False, dense=True, dtype="bf16"),
        # gated output norm over heads of 128 of a recurrent layer, for a W4A4 GEMM and for small bf16 projections
        dict(name="norm heads", op="norm", M=4096, K=4096, k=0, heads=128, post=True, gate="silu", residual=False,
             pre=False, quant=True, dense=True, dtype="bf16"),
        # norms on both sides of an MLP block, gated residual, FP32 stream, odd row count
        dict(name="norm sandwich", op="norm", M=1003, K=17408, k=0, heads=0, post=True, gate="sigmoid", residual=True,
             pre=True, quant=False, dense=True, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "gemm", "linear", "norm"])
    if op == "route":
        E = _log_int(rng, 8, 512)
        k, dtype = rng.randint(1, min(E, 16)), rng.choice(["f32", "bf16"])
        M = _log_int(rng, 1, 16384 * 8 * 128 // (max(E, 128) * max(k, 8) * (2 if dtype == "f32" else 1)))
        return dict(op=op, M=M, E=E, k=k, dtype=dtype,
                    renorm=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.1, 0.9]))
    if op in ("gemm", "linear"):
        E = _log_int(rng, 1, 128)
        K = 32 * _log_int(rng, 2, 160)
        N = min(_log_int(rng, 64, 5120), 64 * 2048 * 5120 // (E * K))
        if rng.random() < 0.7:
            N = max(8, N // 8 * 8)
        if op == "gemm":
            out = rng.choice(["bf16", "bf16", "f32"])
            T = _log_int(rng, 1, min(32768, 32768 * 2048 // N * 5120 // K, 32768 * 2048 // (N * (2 if out == "f32" else 1))))
            return dict(op=op, T=T, spare=rng.choice([0, 0, 1, 200]), E=E, N=N, K=K, out=out,
                        skew=rng.choice([0.0, 0.5, 1.5]))
        k = rng.randint(1, min(E, 10))
        M = _log_int(rng, 1, max(1, min(8192, 8192 * 2048 * 5120 // (N * K)) // k))
        act = rng.choice(["none", "none", "swiglu"])
        # SwiGLU in FP32 may round differently next to a code's border, so its result is a bf16 one
        return dict(op=op, M=M, k=k, E=E, N=N, K=K, act=act, x=rng.choice(["bf16", "bf16", "f32"]),
                    out="bf16" if act == "swiglu" else rng.choice(["bf16", "f32"]))
    heads = rng.choice([0, 0, 64, 128, 256])
    K = 32 * _log_int(rng, 8, 544) if not heads else heads * _log_int(rng, 2, 17408 // heads)
    M = _log_int(rng, 1, min(16384, 16384 * 5120 // K // 3))
    k = rng.choice([0, 0, 0, 2, 8])
    post = heads > 0 or rng.random() < 0.3
    residual, quant = rng.random() < 0.7, rng.random() < 0.5
    return dict(op=op, M=M if not k else max(1, M // k), K=K, k=k, heads=heads, post=post,
                gate=rng.choice(["none", "silu", "sigmoid"]), residual=residual, pre=residual or rng.random() < 0.5,
                quant=quant, dense=not quant or not residual or rng.random() < 0.3,
                dtype=rng.choice(["bf16", "bf16", "f32"]))


# ------------------------------------------------------------------ inputs

def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _activation(g, rows, K, dtype):
    """Unit normal with a few outlier channels, as hidden states have them."""
    x = _randn(g, rows, K)
    ch = torch.randperm(K, generator=g, device=DEV)[: max(1, K // 1000)]
    x[:, ch] *= 60.0
    return x.to(dtype)


def _round_e2m1(a):
    """Magnitudes to the E2M1 grid, as the index of the grid value: nearest, ties to even."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))


def _quantize(x, gs):
    """NVFP4 blocks of FP32 rows; gs: FP32, broadcast over blocks. (signed 4-bit codes, E4M3 scales)"""
    b = x.view(x.shape[0], -1, 16)
    t = b.abs().amax(2) / 6.0 * gs
    s = t.clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
    sf = s.float()
    r = torch.where(sf > 0, gs / sf, torch.zeros_like(sf))
    y = b * r.unsqueeze(2)
    code = _round_e2m1(y.abs()) | (torch.signbit(b).to(torch.uint8) << 3)
    return code.view(x.shape), s


def _pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()


def _tc_index(pos, nblk):
    """Byte offsets in the tensor-core scale order of nblk scales in each of the scale rows pos."""
    kc = -(-nblk // 4)
    j = torch.arange(nblk, device=DEV)
    p = pos.view(-1, 1)
    return ((p >> 7) * kc + (j >> 2)) * 512 + (p & 31) * 16 + ((p >> 5) & 3) * 4 + (j & 3)


def _tc_bytes(blocks, nblk):
    return blocks * (-(-nblk // 4)) * 512


def _grouped_blocks(T, E):
    """128-row scale blocks that T rows in E groups need at most."""
    return (T + 127 * min(E, T)) // 128


def _scale_rows(offsets, rows):
    """(group, row in it, scale row) of each of the first `rows` rows: a group starts a new 128-row scale block."""
    t = torch.arange(rows, device=DEV)
    off = offsets.long()
    e = torch.searchsorted(off[1:].contiguous(), t, right=True)
    p = t - off[e]
    blocks = (off[1:] - off[:-1] + 127) // 128
    first = torch.cumsum(blocks, 0) - blocks
    return e, p, first[e] * 128 + p


def _weights(g, E, N, K):
    """Quantized weights of E experts: codes, scales (each expert's in the tensor-core order), global scales."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(E, _tc_bytes(-(-N // 128), K // 16), dtype=torch.uint8, device=DEV)
    gs = torch.empty(E, device=DEV)
    at = _tc_index(torch.arange(N, device=DEV), K // 16).view(-1)
    for e in range(E):
        w = _randn(g, N, K) * (0.02 * (0.5 + (e % 7) / 4))
        gs[e] = E4M3_MAX * 6.0 / w.abs().max()
        c, s = _quantize(w, gs[e])
        codes[e] = _pack(c)
        scales[e][at] = s.view(torch.uint8).view(-1)
    return codes, scales, gs


def _offsets_of(counts):
    off = torch.zeros(counts.numel() + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.cumsum(counts, 0)
    return off


def _assign(g, M, k, E):
    """The tokens of each expert when M tokens take k of E experts each: (row_index, offsets)."""
    pref = torch.rand(M, E, generator=g, device=DEV).log().neg().log().neg() + 0.5 * _randn(g, 1, E)
    ids = pref.topk(k, 1).indices.view(-1)
    order = torch.argsort(ids, stable=True)
    return (order // k).to(torch.int32), _offsets_of(torch.bincount(ids, minlength=E))


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "route":
        M, E, k = c["M"], c["E"], c["k"]
        x = 2.0 * _randn(g, M, E) + 0.5 * _randn(g, 1, E)
        if c["masked"]:
            x[torch.rand(M, E, generator=g, device=DEV) < c["masked"]] = float("-inf")
        s["logits"] = x.to(_dt(c["dtype"]))
        s["expert_ids"] = torch.empty(M, k, dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(M, k, device=DEV)
        s["slots"] = torch.empty(M, k, dtype=torch.int32, device=DEV)
        s["row_index"] = torch.empty(M * k, dtype=torch.int32, device=DEV)
        s["group_offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        s["workspace"] = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
        return s
    if c["op"] in ("gemm", "linear"):
        E, N, K = c["E"], c["N"], c["K"]
        s["w_codes"], s["w_scales"], s["w_gs"] = _weights(g, E, N, K)
        if c["op"] == "gemm":
            rows, T = c["T"], c["T"] + c["spare"]
            p = torch.softmax(c["skew"] * _randn(g, E), 0)
            at = torch.multinomial(p, rows, replacement=True, generator=g)
            s["offsets"] = _offsets_of(torch.bincount(at, minlength=E))
            x = _activation(g, T, K, torch.float32)
            s["a_gs"] = (E4M3_MAX * 6.0 / x.abs().max()) * (1.0 + 0.25 * torch.rand(E, generator=g, device=DEV))
            e, _, pos = _scale_rows(s["offsets"], rows)
            codes, scales = _quantize(x[:rows], s["a_gs"][e].view(-1, 1))
            s["a_codes"] = torch.zeros(T, K // 2, dtype=torch.uint8, device=DEV)
            s["a_codes"][:rows] = _pack(codes)
            s["a_scales"] = torch.zeros(_tc_bytes(_grouped_blocks(T, E), K // 16), dtype=torch.uint8, device=DEV)
            s["a_scales"][_tc_index(pos, K // 16)] = scales.view(torch.uint8)
        else:
            rows = T = c["M"] * c["k"]
            index, s["offsets"] = _assign(g, c["M"], c["k"], E)
            if c["act"] == "swiglu":
                s["x"], s["row_index"] = _randn(g, T, 2 * K).to(_dt(c["x"])), None
                amax = 12.0
            else:
                s["x"], s["row_index"] = _activation(g, c["M"], K, _dt(c["x"])), index
                amax = s["x"].float().abs().max()
            s["a_gs"] = (E4M3_MAX * 6.0 / amax) * (1.0 + 0.25 * torch.rand(E, generator=g, device=DEV))
            s["a_codes"] = torch.empty(T, K // 2, dtype=torch.uint8, device=DEV)
            s["a_scales"] = torch.empty(_tc_bytes(_grouped_blocks(T, E), K // 16), dtype=torch.uint8, device=DEV)
        s["rows"] = rows
        s["longest"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["out"] = torch.zeros(T, N, dtype=_dt(c["out"]), device=DEV)
        return s
    M, K, dt = c["M"], c["K"], _dt(c["dtype"])
    if c["k"]:
        E = max(8, c["k"])
        ids = torch.rand(M, E, generator=g, device=DEV).topk(c["k"], 1).indices.view(-1)
        slots = torch.empty(M * c["k"], dtype=torch.int32, device=DEV)
        slots[torch.argsort(ids, stable=True)] = torch.arange(M * c["k"], dtype=torch.int32, device=DEV)
        s["slots"] = slots.view(M, c["k"])
        s["slot_weights"] = torch.softmax(_randn(g, M, c["k"]), 1)
    s["y"] = _activation(g, M * max(1, c["k"]), K, dt)
    s["post_weight"] = 1.0 + 0.2 * _randn(g, c["heads"] or K) if c["post"] else None
    s["gate"] = None if c["gate"] == "none" else (2.0 * _randn(g, M, K)).to(dt)
    s["residual"] = _activation(g, M, K, dt) if c["residual"] else None
    s["pre_weight"] = 1.0 + 0.2 * _randn(g, K) if c["pre"] else None
    s["residual_out"] = torch.empty(M, K, dtype=dt, device=DEV) if c["residual"] else None
    s["out"] = torch.empty(M, K, dtype=dt, device=DEV) if c["dense"] else None
    s["scale"] = 0.7 if c["residual"] else 1.0
    s["eps"] = 1e-6
    if c["quant"]:
        s["gs"] = E4M3_MAX * 6.0 / 80.0
        s["codes"] = torch.empty(M, K // 2, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(_tc_bytes(-(-M // 128), K // 16), dtype=torch.uint8, device=DEV)
        # E2M1 values of the two codes of a byte (exact in E4M3), to return codes as values
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
        b = torch.arange(256, device=DEV)
        both = torch.stack([grid[b & 15], grid[b >> 4]], 1).to(torch.float8_e4m3fn)
        s["grid"], s["pairs"] = grid, both.view(torch.int16).view(256)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"route": _own_route, "gemm": _own_gemm, "linear": _own_linear, "norm": _own_norm}[op](s)
    return {"route": _plain_route, "gemm": _plain_gemm, "linear": _plain_linear, "norm": _plain_norm}[op](s)


def _own_route(s):
    import nvfp4_w4a4_quantized_10_b200 as nv
    c = s["case"]
    nv.nvfp4_route(s["logits"], nv.ROUTE_SOFTMAX_TOPK if c["renorm"] else nv.ROUTE_SOFTMAX_ALL, s["expert_ids"],
                   s["weights"], s["slots"], s["row_index"], s["group_offsets"], s["workspace"])
    return {k: s[k] for k in ("expert_ids", "weights", "slots", "row_index", "group_offsets")}


def _plain_route(s):
    c = s["case"]
    M, E, k = c["M"], c["E"], c["k"]
    x = torch.nan_to_num(s["logits"].float(), nan=float("-inf"), posinf=torch.finfo(torch.float32).max,
                         neginf=float("-inf"))
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    taken = top > float("-inf")
    first = torch.where(taken[:, :1], top[:, :1], torch.zeros_like(top[:, :1]))
    e = torch.exp(top - first)
    total = e.sum(1, keepdim=True) if c["renorm"] else torch.exp(x - first).sum(1, keepdim=True)
    weights = torch.where(taken, e / total, torch.zeros_like(e))
    key = torch.where(taken, ids, torch.full_like(ids, E)).view(-1)
    order = torch.argsort(key, stable=True)
    at = torch.arange(M * k, device=DEV)
    slots = torch.empty_like(at)
    slots[order] = at
    counts = (key.view(-1, 1) == torch.arange(E, device=DEV)).sum(0)
    offsets = torch.cat([torch.zeros_like(counts[:1]), torch.cumsum(counts, 0)])
    return {"expert_ids": torch.where(taken, ids, torch.full_like(ids, -1)).to(torch.int32), "weights": weights,
            "slots": torch.where(taken, slots.view(M, k), torch.full_like(ids, -1)).to(torch.int32),
            "row_index": torch.where(at < offsets[-1], order // k, torch.full_like(at, -1)).to(torch.int32),
            "group_offsets": offsets.to(torch.int32)}


def _own_gemm(s):
    import nvfp4_w4a4_quantized_10_b200 as nv
    nv.nvfp4_grouped_gemm(s["a_codes"], s["a_scales"], s["a_gs"], s["w_codes"], s["w_scales"], s["w_gs"],
                          s["offsets"], s["out"])
    return s["out"]


def _values(codes):
    """E2M1 values of packed codes, FP32."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    return torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).flatten(-2)


def _grouped_product(s, a, e, p):
    """out rows of dequantized activations a (row t: row p[t] of group e[t]), through one batched product."""
    c = s["case"]
    E, N, K = c["E"], c["N"], c["K"]
    nblk = K // 16
    at = _tc_index(torch.arange(N, device=DEV), nblk)
    ws = s["w_scales"][:, at].view(torch.float8_e4m3fn).float()
    w = (_values(s["w_codes"]).view(E, N, nblk, 16) * ws.unsqueeze(-1)).view(E, N, K)
    pad = torch.zeros(E, s["longest"], K, device=DEV)
    pad[e, p] = a
    alpha = 1.0 / (s["a_gs"].double() * s["w_gs"].double())
    o = torch.bmm(pad, w.transpose(1, 2))[e, p] * alpha.float()[e].view(-1, 1)
    out = torch.zeros(s["out"].shape, device=DEV)
    out[: s["rows"]] = o
    return out.to(s["out"].dtype)


def _plain_gemm(s):
    K = s["case"]["K"]
    e, p, pos = _scale_rows(s["offsets"], s["rows"])
    sc = s["a_scales"][_tc_index(pos, K // 16)].view(torch.float8_e4m3fn).float()
    a = _values(s["a_codes"][: s["rows"]]).view(s["rows"], K // 16, 16) * sc.unsqueeze(-1)
    return _grouped_product(s, a.view(s["rows"], K), e, p)


def _own_linear(s):
    import nvfp4_w4a4_quantized_10_b200 as nv
    nv.nvfp4_grouped_quantize(s["x"], s["offsets"], s["a_gs"], s["a_codes"], s["a_scales"], row_index=s["row_index"],
                              act=nv.ACT_SWIGLU if s["case"]["act"] == "swiglu" else nv.ACT_NONE)
    nv.nvfp4_grouped_gemm(s["a_codes"], s["a_scales"], s["a_gs"], s["w_codes"], s["w_scales"], s["w_gs"],
                          s["offsets"], s["out"])
    return s["out"]


def _plain_linear(s):
    c = s["case"]
    K = c["K"]
    e, p, _ = _scale_rows(s["offsets"], s["rows"])
    x = s["x"].float()
    if c["act"] == "swiglu":
        x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
    else:
        x = x[s["row_index"].long()]
    gs = s["a_gs"][e].view(-1, 1)
    code, sc = _quantize(x, gs)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    a = grid[code.int()].view(s["rows"], K // 16, 16) * sc.float().unsqueeze(-1)
    return _grouped_product(s, a.view(s["rows"], K), e, p)


def _own_norm(s):
    import nvfp4_w4a4_quantized_10_b200 as nv
    c = s["case"]
    gate = {"none": nv.GATE_NONE, "silu": nv.GATE_SILU, "sigmoid": nv.GATE_SIGMOID}[c["gate"]]
    nv.nvfp4_block_norm(s["y"], slots=s.get("slots"), slot_weights=s.get("slot_weights"),
                        post_weight=s["post_weight"], gate=s["gate"], gate_kind=gate, residual=s["residual"],
                        residual_scale=s["scale"], residual_out=s["residual_out"], pre_weight=s["pre_weight"],
                        eps=s["eps"], out=s["out"], codes=s.get("codes"), block_scales=s.get("scales"),
                        global_scale=s.get("gs", 1.0))
    out = {"residual": s["residual_out"], "out": s["out"]}
    if c["quant"]:
        # two codes of a byte as the two E2M1 values they stand for, scales as E4M3 numbers
        v = torch.index_select(s["pairs"], 0, s["codes"].view(-1).int())
        out["values"] = v.view(torch.float8_e4m3fn).view(c["M"], c["K"])
        out["scales"] = s["scales"].view(torch.float8_e4m3fn)
    return out


def _plain_norm(s):
    c = s["case"]
    M, K = c["M"], c["K"]
    b = s["y"].float()
    if c["k"]:
        b = (b[s["slots"].long()] * s["slot_weights"].unsqueeze(-1)).sum(1)
    if c["post"]:
        h = b.view(M, -1, c["heads"] or K)
        b = (h * torch.rsqrt(h.square().mean(2, keepdim=True) + s["eps"]) * s["post_weight"]).view(M, K)
    if s["gate"] is not None:
        z = s["gate"].float()
        b = b * torch.sigmoid(z) if c["gate"] == "sigmoid" else b * (z * torch.sigmoid(z))
    v = b * s["scale"]
    if c["residual"]:
        v = v + s["residual"].float()
    out = {"residual": v.to(s["residual"].dtype) if c["residual"] else None}
    h = v * torch.rsqrt(v.square().mean(1, keepdim=True) + s["eps"]) * s["pre_weight"] if c["pre"] else v
    out["out"] = h.to(s["y"].dtype) if c["dense"] else None
    if not c["quant"]:
        return out
    code, sc = _quantize(h, torch.full((1, 1), s["gs"], device=DEV))
    tc = torch.zeros(s["scales"].numel(), dtype=torch.uint8, device=DEV)
    tc[_tc_index(torch.arange(M, device=DEV), K // 16)] = sc.view(torch.uint8)
    out["values"] = s["grid"][code.int()].to(torch.float8_e4m3fn)
    out["scales"] = tc.view(torch.float8_e4m3fn)
    return out


# ------------------------------------------------------------------ bytes and operations

def work(case):
    c = case
    if c["op"] == "route":
        M, E, k = c["M"], c["E"], c["k"]
        return {"bytes": M * E * (4 if c["dtype"] == "f32" else 2) + M * k * 16 + (E + 1) * 4, "flops": 4 * M * E}
    if c["op"] in ("gemm", "linear"):
        E, N, K = c["E"], c["N"], c["K"]
        T = c["T"] if c["op"] == "gemm" else c["M"] * c["k"]
        active = E * (1.0 - (1.0 - 1.0 / E) ** T)          # experts with a row, on average
        out = T * N * (4 if c["out"] == "f32" else 2)
        if c["op"] == "gemm":
            a = T * K * 9 / 16
        else:
            a = (2 * T if c["act"] == "swiglu" else c["M"]) * K * (4 if c["x"] == "f32" else 2)
        return {"bytes": a + out + active * N * K * 9 / 16, "flops": 2.0 * T * N * K}
    M, K = c["M"], c["K"]
    z = 2 if c["dtype"] == "bf16" else 4
    n = max(1, c["k"]) + (c["gate"] != "none") + 2 * c["residual"]
    return {"bytes": M * K * (n * z + 9 / 16 * c["quant"] + z * c["dense"]), "flops": M * K * (12.0 + 2 * c["k"])}


# ------------------------------------------------------------------ 64-bit

def _decode(code):
    """E2M1 from its bits: sign, two exponent bits (bias 1), one mantissa bit."""
    code = code.long()
    ex, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(ex == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2((ex - 1).double()))
    return torch.where(code >= 8, -mag, mag)


def _decode_e4m3(byte):
    byte = byte.long()
    ex, m = (byte >> 3) & 15, (byte & 7).double()
    return torch.where(ex == 0, m / 8.0 * 2.0 ** -6, (1.0 + m / 8.0) * torch.exp2((ex - 7).double()))


def _unscramble(buf, first, rows, nblk):
    """Scales of rows first*128 ... of a tensor-core ordered buffer, by undoing the order chunk by chunk."""
    kc, nb = -(-nblk // 4), -(-rows // 128)
    v = buf.view(-1, kc, 32, 4, 4)[first:first + nb]                      # block, chunk, row % 32, row / 32, scale
    return v.permute(0, 3, 2, 1, 4).reshape(nb * 128, kc * 4)[:rows, :nblk]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        return _exact_route(c, s)
    if c["op"] == "norm":
        return _exact_norm(c, s)
    E, N, K = c["E"], c["N"], c["K"]
    off = s["offsets"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    block = 0
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        wc = s["w_codes"][e]
        w = torch.stack([_decode(wc & 15), _decode(wc >> 4)], 2).view(N, K // 16, 16)
        w = (w * _decode_e4m3(_unscramble(s["w_scales"][e], 0, N, K // 16)).unsqueeze(2)).view(N, K)
        if c["op"] == "gemm":
            ac = s["a_codes"][lo:hi]
            a = torch.stack([_decode(ac & 15), _decode(ac >> 4)], 2).view(hi - lo, K // 16, 16)
            a = a * _decode_e4m3(_unscramble(s["a_scales"], block, hi - lo, K // 16)).unsqueeze(2)
            block += -(-(hi - lo) // 128)
        else:
            if c["act"] == "swiglu":
                x = s["x"][lo:hi].double()
                x = (x[:, :K] / (1.0 + torch.exp(-x[:, :K])) * x[:, K:]).float()
            else:
                x = s["x"].index_select(0, s["row_index"][lo:hi].long()).float()
            # the format itself is defined by FP32 steps
            b = x.view(hi - lo, K // 16, 16)
            g = s["a_gs"][e]
            sc = torch.clamp(b.abs().max(2).values.div(6.0).mul(g), max=E4M3_MAX).to(torch.float8_e4m3fn).float()
            y = (b * torch.where(sc > 0, g / sc, 0.0 * sc).unsqueeze(2)).double()
            grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
            mag = y.abs().clamp(max=6.0)
            up = torch.searchsorted(grid, mag.contiguous()).clamp(max=7)
            dn = (up - 1).clamp(min=0)
            du, dd = grid[up] - mag, mag - grid[dn]
            pick = torch.where((du < dd) | ((du == dd) & (up % 2 == 0)), up, dn)
            a = grid[pick] * torch.sign(y) * sc.double().unsqueeze(2)
        alpha = 1.0 / (s["a_gs"][e].double() * s["w_gs"][e].double())
        out[lo:hi] = a.view(hi - lo, K) @ w.T * alpha
    return out


def _exact_route(c, s):
    M, E, k = c["M"], c["E"], c["k"]
    x = s["logits"].double()
    col = torch.arange(E, device=DEV).expand(M, E)
    left, ids, vals = x.clone(), [], []
    for _ in range(k):
        v = left.max(1, keepdim=True).values
        i = torch.where(left == v, col, torch.full_like(col, E)).min(1, keepdim=True).values
        ids.append(torch.where(v > float("-inf"), i, torch.full_like(i, -1)))
        vals.append(v)
        left = left.scatter(1, i, float("-inf"))
    ids, vals = torch.cat(ids, 1), torch.cat(vals, 1)
    lse = torch.logsumexp(vals if c["renorm"] else x, 1, keepdim=True)
    weights = torch.where(ids >= 0, torch.exp(vals - lse), torch.zeros_like(vals))
    hot = torch.zeros(M, E + 1, dtype=torch.int64, device=DEV)
    hot.scatter_(1, torch.where(ids >= 0, ids, torch.full_like(ids, E)), 1)
    hot = hot[:, :E]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), hot.sum(0).cumsum(0)])
    place = offsets[:-1] + hot.cumsum(0) - hot
    slots = torch.where(ids >= 0, place.gather(1, ids.clamp(min=0)), torch.full_like(ids, -1))
    row = torch.full((M * k + 1,), -1, dtype=torch.int64, device=DEV)
    token = torch.arange(M, device=DEV).view(-1, 1).expand(M, k)
    row[torch.where(slots >= 0, slots, torch.full_like(slots, M * k))] = token
    return {"expert_ids": ids, "weights": weights, "slots": slots, "row_index": row[:-1], "group_offsets": offsets}


def _exact_norm(c, s):
    M, K = c["M"], c["K"]
    y = s["y"].double()
    if c["k"]:
        # row m: the weighted rows that its slots name, as one product for each column block
        b = torch.zeros(M, K, dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            b += s["slot_weights"][:, j:j + 1].double() * y.index_select(0, s["slots"][:, j].long())
    else:
        b = y
    if c["post"]:
        w = c["heads"] or K
        ss = torch.linalg.vector_norm(b.reshape(-1, w), dim=1, keepdim=True)
        b = (b.reshape(-1, w) / torch.sqrt(ss * ss / w + s["eps"]) * s["post_weight"].double()).reshape(M, K)
    if s["gate"] is not None:
        z = s["gate"].double()
        f = 1.0 / (1.0 + torch.exp(-z))
        b = b * (f if c["gate"] == "sigmoid" else z * f)
    v = s["scale"] * b + (s["residual"].double() if c["residual"] else 0.0)
    out = {"residual": v if c["residual"] else None}
    if c["pre"]:
        ss = torch.linalg.vector_norm(v, dim=1, keepdim=True)
        v = v / torch.sqrt(ss * ss / K + s["eps"]) * s["pre_weight"].double()
    out["out"] = v if c["dense"] else None
    if c["quant"]:                             # next to a rounding border a code has no 64-bit value of its own
        out["values"] = out["scales"] = None
    return out
