"""Cases and plain forms of the operators around the MoE layer.

* RMSNorm with the residual's addition in front of the layer, with a bf16
  output or an E4M3 output with one scale per 128 columns;
* the whole MoE layer for a few tokens in one launch (bf16 and MXFP4 expert
  weights);
* the block-scaled FP8 matrix product (E4M3 operands, one fp32 scale per row
  and 128 of K on the left, per 128 x 128 block on the right), dense or
  grouped by expert.

With ``own`` false, ``run`` computes an operator from elementary torch
operations in 32 bits; with ``own`` true it calls the library.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn
# E2M1 values by code: sign, two exponent bits (bias 1, field 0 subnormal), one mantissa bit
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
AMAX_MIN = 2.0 ** -100  # floor of a quantisation block's largest magnitude
E4M3_MAX = 448.0


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token in front of the layer: latency only
        dict(name="norm_1", op="norm", T=1, D=2880, ldx=2880, res="bf16", out="bf16"),
        # a decode batch whose x is a slice of a wider projection's rows, fp32 residual stream, 8-bit output
        dict(name="norm_257_strided", op="norm", T=257, D=4112, ldx=6208, res="f32", out="e4m3"),
        # the 20B-shaped prefill batch, bf16 residual stream, the output as the layer reads it
        dict(name="norm_8192", op="norm", T=8192, D=2880, ldx=2880, res="bf16", out="bf16"),
        # the 120B-shaped prefill batch, the output as an FP8 product reads it
        dict(name="norm_16384_e4m3", op="norm", T=16384, D=2880, ldx=2880, res="bf16", out="e4m3"),
        # decode of one sequence, 20B shape
        dict(name="few_bf16_1", op="few", T=1, D=2880, E=32, k=4, I=2880, w="bf16", act="swiglu"),
        # decode of sixteen sequences, 20B shape: most experts get a row or more
        dict(name="few_bf16_16", op="few", T=16, D=2880, E=32, k=4, I=2880, w="bf16", act="swiglu"),
        # decode of one sequence with MXFP4 weights and the GPT-OSS activation
        dict(name="few_mxfp4_1", op="few", T=1, D=2880, E=32, k=4, I=2880, w="mxfp4", act="gptoss"),
        # seven sequences on the 120B shape (128 experts) with MXFP4 weights
        dict(name="few_mxfp4_7", op="few", T=7, D=2880, E=128, k=4, I=2880, w="mxfp4", act="gptoss"),
        # a dense projection of a decode batch: the weights are what is read
        dict(name="fp8_dense_17", op="fp8", R=17, E=0, N=5760, K=2880, out="bf16", bias=True),
        # the same projection of a prefill batch
        dict(name="fp8_dense_8192", op="fp8", R=8192, E=0, N=5760, K=2880, out="bf16", bias=False),
        # the experts' second product of a decode batch (64 tokens, top-4), fp32 rows for the combine
        dict(name="fp8_grouped_256", op="fp8", R=256, E=32, N=2880, K=2880, out="f32", bias=True),
        # the experts' first product of the 20B-shaped prefill batch (8192 tokens, top-4), uneven segments
        dict(name="fp8_grouped_32768", op="fp8", R=32768, E=32, N=5760, K=2880, out="bf16", bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "few", "fp8"))
    if op == "norm":
        T, D = _log(rng, 1, 16384), 16 * rng.randint(4, 320)
        return dict(op=op, T=T, D=D, ldx=D + 16 * rng.choice((0, 0, rng.randint(1, 64))),
                    res=rng.choice(("none", "bf16", "f32")), out=rng.choice(("bf16", "e4m3")))
    if op == "few":
        E = rng.choice((8, 16, 32, 64, 128))
        D, I = 64 * rng.randint(8, 64), 64 * rng.randint(8, 64)
        T = max(1, min(_log(rng, 1, 16), 65536 // max(D, I)))
        w = rng.choice(("bf16", "mxfp4"))
        if E * D * I > 32 * 2880 * 2880 and w == "bf16":  # no more weight bytes than the largest listed case holds
            E = 8
        return dict(op=op, T=T, D=D, E=E, k=rng.randint(1, 6), I=I, w=w, act=rng.choice(("swiglu", "gptoss")))
    E = rng.choice((0, 0, 1, 8, 32))
    N, K = 16 * rng.randint(16, 360), 16 * rng.randint(16, 180)
    return dict(op=op, R=_log(rng, 1, 8192 if E == 0 else 32768), E=E, N=N, K=K, out=rng.choice(("bf16", "f32")),
                bias=rng.choice((True, False)))


# ---------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _experts(g, E, rows, cols):
    return (_randn(g, E, rows, cols) * 0.02).to(BF16)


def _mxfp4(g, E, rows, cols):
    codes = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(119, 128, (E, rows, cols // 32), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales


def _blocks(n):
    return -(-n // 128)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        wide = _randn(g, T, case["ldx"]).to(BF16)
        s = dict(case=case, x=wide[:, :D], gamma=(1.0 + 0.2 * _randn(g, D)).to(BF16), eps=1e-5, residual=None)
        if case["res"] != "none":
            # a residual stream is larger than one block's output and has a few large channels
            r = 4.0 * _randn(g, T, D) * (1.0 + 15.0 * (torch.rand(D, generator=g, device="cuda") > 0.99))
            s["residual"] = r.to(BF16 if case["res"] == "bf16" else torch.float32)
        return s
    if case["op"] == "few":
        T, D, E, I = case["T"], case["D"], case["E"], case["I"]
        s = dict(case=case, x=_randn(g, T, D).to(BF16), Wr=(_randn(g, E, D) * D ** -0.5).to(BF16),
                 br=(_randn(g, E) * 0.02).to(BF16), b1=(_randn(g, E, 2 * I) * 0.02).to(BF16),
                 b2=(_randn(g, E, D) * 0.02).to(BF16), s1=None, s2=None)
        if case["w"] == "bf16":
            s["W1"], s["W2"] = _experts(g, E, 2 * I, D), _experts(g, E, D, I)
        else:
            s["W1"], s["s1"] = _mxfp4(g, E, 2 * I, D)
            s["W2"], s["s2"] = _mxfp4(g, E, D, I)
        return s
    R, N, K, E = case["R"], case["N"], case["K"], max(1, case["E"])
    # activations as a norm leaves them, quantised per row and 128 columns; weights quantised per 128 x 128 block
    KB, NB = _blocks(K), _blocks(N)
    a = torch.nn.functional.pad(_randn(g, R, K), (0, KB * 128 - K)).view(R, KB, 128)
    a_scale = a.abs().amax(-1) / E4M3_MAX
    aq = (a / a_scale[..., None]).view(R, KB * 128)[:, :K].to(E4M3).contiguous()
    w = torch.empty((E, N, K), dtype=E4M3, device="cuda")
    w_scale = torch.empty((E, NB, KB), dtype=torch.float32, device="cuda")
    for e in range(E):
        v = torch.nn.functional.pad(_randn(g, N, K) * 0.02, (0, KB * 128 - K, 0, NB * 128 - N)).view(NB, 128, KB, 128)
        w_scale[e] = v.abs().amax((1, 3)) / E4M3_MAX
        w[e] = (v / w_scale[e][:, None, :, None]).view(NB * 128, KB * 128)[:N, :K].to(E4M3)
    s = dict(case=case, a=aq, a_scale=a_scale, w=w, w_scale=w_scale, offsets=None, max_rows=R,
             bias=(_randn(g, E, N) * 0.02).to(BF16) if case["bias"] else None)
    if case["E"]:
        # uneven segments: a uniform routing's counts with every eighth expert left empty
        p = torch.rand(E, generator=g, device="cuda") + 0.5
        if E >= 8:
            p[::8] = 0.0
        e_of = torch.multinomial(p, R, replacement=True, generator=g)
        counts = torch.bincount(e_of, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["max_rows"] = int(counts.max())
    return s


# ------------------------------------------------------------- the plain forms
def _norm_plain(s):
    v, out = s["x"].float(), {}
    if s["residual"] is not None:
        out["res"] = (v + s["residual"].float()).to(s["residual"].dtype)
        v = out["res"].float()
    y = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + s["eps"]) * s["gamma"].float()
    if s["case"]["out"] == "bf16":
        out["y"] = y.to(BF16)
        return out
    T, D = y.shape
    nb = _blocks(D)
    yb = torch.nn.functional.pad(y, (0, nb * 128 - D)).view(T, nb, 128)
    out["scale"] = yb.abs().amax(-1).clamp_min(AMAX_MIN) / E4M3_MAX
    out["q"] = (yb / out["scale"][..., None]).view(T, nb * 128)[:, :D].to(E4M3)
    return out


def _dequant(w, scales):
    """bf16 weights, or MXFP4 codes and scales, as fp32."""
    if scales is None:
        return w.float()
    table = torch.tensor(E2M1, device=w.device)
    codes = torch.stack((w & 15, w >> 4), -1).flatten(-2).int()
    v = torch.index_select(table, 0, codes.flatten()).view(*codes.shape[:-1], -1, 32)
    return (v * torch.exp2(scales.float() - 127.0)[..., None]).flatten(-2)


ALPHA, LIMIT = 1.702, 7.0  # of the GPT-OSS activation


def _glu(u, act):
    g, u = u.chunk(2, -1)
    if act == "gptoss":
        g, u = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
        return g * torch.sigmoid(ALPHA * g) * (u + 1)
    return g * torch.sigmoid(g) * u


def _few_plain(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["x"].float()
    logits = x @ s["Wr"].float().t() + s["br"].float()
    top, idx = (v[:, :k] for v in torch.sort(logits, dim=1, descending=True, stable=True))
    gate = torch.softmax(top, 1)
    pick = (lambda w: None if w is None else w[idx.flatten()]) if T * k < E else (lambda w: w)
    W1, W2 = _dequant(pick(s["W1"]), pick(s["s1"])), _dequant(pick(s["W2"]), pick(s["s2"]))
    b1, b2 = pick(s["b1"]).float()[:, None], pick(s["b2"]).float()[:, None]
    rows = x.repeat_interleave(k, 0)[:, None] if T * k < E else x[None]  # a row per assignment, or every token on every expert
    h = _glu(torch.matmul(rows, W1.transpose(1, 2)) + b1, c["act"]).to(BF16).float()  # the layer's h is bf16
    o = torch.matmul(h, W2.transpose(1, 2)) + b2
    if T * k < E:
        y = (o.view(T, k, -1) * gate[..., None]).sum(1)
    else:
        y = (o * torch.zeros_like(logits).scatter(1, idx, gate).t()[..., None]).sum(0)
    return {"y": y.to(BF16)}


def _fp8_plain(s):
    R, N, K = s["case"]["R"], s["case"]["N"], s["case"]["K"]
    a = s["a"].float() * s["a_scale"].repeat_interleave(128, 1)[:, :K]
    w = s["w"].float() * s["w_scale"].repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    if s["offsets"] is None:
        out = a @ w[0].t()
        e = torch.zeros(R, dtype=torch.int64, device=a.device)
    else:
        off = s["offsets"].long()
        r = torch.arange(R, device=a.device)
        e = torch.searchsorted(off[1:], r, right=True)
        padded = (off[:-1, None] + torch.arange(s["max_rows"], device=a.device)).clamp_max(R - 1)
        out = torch.matmul(a[padded], w.transpose(1, 2))[e, r - off[e]]
    if s["bias"] is not None:
        out = out + s["bias"].float()[e]
    return {"out": out.to(BF16 if s["case"]["out"] == "bf16" else torch.float32)}


# --------------------------------------------------------- the library's calls
def _own(s):
    import mixture_experts_ffn_layer_b200 as moe

    c = s["case"]
    if c["op"] == "norm":
        if c["out"] == "bf16":
            y, res = moe.rmsnorm(s["x"], s["gamma"], s["eps"], residual=s["residual"])
            out = {"y": y}
        else:
            q, scale, res = moe.rmsnorm_fp8(s["x"], s["gamma"], s["eps"], residual=s["residual"])
            out = {"q": q, "scale": scale}
        if res is not None:
            out["res"] = res
        return out
    if c["op"] == "few":
        if "ws" not in s:  # a decoding program keeps the sizes and the workspace
            s["dims"] = moe.dims(c["T"], c["D"], c["E"], c["k"], c["I"], moe.MOE_W_BF16 if c["w"] == "bf16" else moe.MOE_W_MXFP4,
                                 moe.MOE_ACT_GPTOSS if c["act"] == "gptoss" else moe.MOE_ACT_SWIGLU, ALPHA, LIMIT)
            s["ws"] = moe.alloc_workspace(s["dims"])
        y = torch.empty((c["T"], c["D"]), dtype=BF16, device="cuda")
        moe.moe_forward_few(s["dims"], s["x"], s["Wr"], s["br"], s["W1"], s["b1"], s["W2"], s["b2"], y, s["ws"],
                            W1_scales=s["s1"], W2_scales=s["s2"])
        return {"y": y}
    out_dtype = BF16 if c["out"] == "bf16" else torch.float32
    if "ws" not in s:
        s["ws"] = moe.alloc_fp8_workspace(moe.fp8_dims(c["R"], max(1, c["E"]), c["N"], c["K"], out_dtype))
    return {"out": moe.fp8_matmul(s["a"], s["a_scale"], s["w"], s["w_scale"], s["ws"], offsets=s["offsets"], bias=s["bias"],
                                  out_dtype=out_dtype)}


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm_plain, "few": _few_plain, "fp8": _fp8_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the floors
def work(case):
    if case["op"] == "norm":
        T, D, res = case["T"], case["D"], {"none": 0, "bf16": 4, "f32": 8}[case["res"]]
        out = 2 * D if case["out"] == "bf16" else D + 4 * _blocks(D)
        return {"bytes": T * (D * (2 + res) + out) + 2 * D, "flops": 4 * T * D}
    if case["op"] == "few":
        T, D, E, k, I = (case[n] for n in ("T", "D", "E", "k", "I"))
        # experts that at least one of T independent choices of k among E takes, on average
        active = E * (1.0 - (1.0 - k / E) ** T)
        per = 2.0 if case["w"] == "bf16" else 17.0 / 32.0
        return {"bytes": active * (3 * D * I * per + 2 * (2 * I + D)) + 2 * E * D + 4 * T * D,
                "flops": 6 * T * k * D * I + 2 * T * E * D}
    R, N, K, E = case["R"], case["N"], case["K"], max(1, case["E"])
    active = E if case["E"] < 8 else E - -(-E // 8)
    active = min(active, R)
    return {"bytes": R * (K + 4 * _blocks(K)) + active * (N * K + 4 * _blocks(N) * _blocks(K) + 2 * N * case["bias"])
            + R * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * R * N * K}


# ---------------------------------------------------- the definitions in 64 bits
def _exact_expert(w, scales, e):
    if scales is None:
        return w[e].double()
    table = torch.tensor(E2M1, dtype=torch.float64, device=w.device)
    lo, hi = table[(w[e] % 16).long()], table[torch.div(w[e], 16, rounding_mode="floor").long()]
    v = torch.empty((w.shape[1], 2 * w.shape[2]), dtype=torch.float64, device=w.device)
    v[:, 0::2], v[:, 1::2] = lo, hi
    return v * torch.pow(2.0, scales[e].double() - 127.0).repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        v, out = s["x"].double(), {}
        if s["residual"] is not None:
            out["res"] = (v + s["residual"].double()).to(s["residual"].dtype).double()
            v = out["res"]
        y = v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / case["D"] + s["eps"]) * s["gamma"].double()
        if case["out"] == "bf16":
            out["y"] = y
            return out
        out["q"], out["scale"] = torch.empty_like(y), y.new_empty((case["T"], _blocks(case["D"])))
        for b in range(_blocks(case["D"])):
            part = y[:, 128 * b:128 * b + 128]
            out["scale"][:, b] = torch.clamp(part.abs().max(1).values, min=AMAX_MIN) / E4M3_MAX
            out["q"][:, 128 * b:128 * b + 128] = part / out["scale"][:, b:b + 1]
        return out
    if case["op"] == "few":
        x, y = s["x"].double(), torch.zeros((case["T"], case["D"]), dtype=torch.float64, device="cuda")
        logits = torch.nn.functional.linear(x, s["Wr"].double(), s["br"].double()).cpu()
        for t in range(case["T"]):
            order = sorted(range(case["E"]), key=lambda e: (-float(logits[t, e]), e))[:case["k"]]
            ex = [math.exp(float(logits[t, e]) - float(logits[t, order[0]])) for e in order]
            for e, v in zip(order, ex):
                u = _exact_expert(s["W1"], s["s1"], e) @ x[t] + s["b1"][e].double()
                gate, up = u[:case["I"]], u[case["I"]:]
                if case["act"] == "gptoss":
                    gate, up = torch.clamp(gate, max=LIMIT), torch.clamp(up, -LIMIT, LIMIT) + 1.0
                h = gate / (1.0 + torch.exp(-(ALPHA if case["act"] == "gptoss" else 1.0) * gate)) * up
                o = _exact_expert(s["W2"], s["s2"], e) @ h.to(BF16).double() + s["b2"][e].double()
                y[t] += v / sum(ex) * o
        return {"y": y}
    K, N = case["K"], case["N"]
    out = torch.zeros((case["R"], N), dtype=torch.float64, device="cuda")
    ends = [0, case["R"]] if s["offsets"] is None else s["offsets"].tolist()
    for e in range(len(ends) - 1):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        for b in range(_blocks(K)):
            part = s["a"][lo:hi, 128 * b:128 * b + 128].double() @ s["w"][e][:, 128 * b:128 * b + 128].double().t()
            out[lo:hi] += part * s["a_scale"][lo:hi, b:b + 1].double() * s["w_scale"][e][:, b].double().repeat_interleave(128)[:N]
        if s["bias"] is not None:
            out[lo:hi] += s["bias"][e].double()
    return {"out": out}
