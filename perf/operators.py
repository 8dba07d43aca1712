"""The decoding-step operators, as cases that can be measured.

Three operators that sit beside the W4A4 linear of this library in one layer of a served model:

  norm          osc_add_rmsnorm_quantize_fp8: the residual's addition, the RMS norm and the MXFP8
                quantization of the normed rows (with, on request, the normed rows in bf16)
  gemv          osc_gemv: a prepared 4-bit weight times a few bf16 token rows, the table's channels
                taken from the bf16 weight columns W_L
  gemv_grouped  osc_gemv_grouped: the same for routed rows, each against its own expert's weight

`run` computes them in their plain form (elementary torch operations in 32 bits, rounded once),
or, where `own` is true, by the library's entry points. `exact` gives the definition in 64 bits.
"""
import math
import random

import torch

own = False
_osc = None


# ---- the cases --------------------------------------------------------------------------------

def listed():
    return [
        # one token of a decoding step, between two layers of a model with hidden size 4096
        dict(name="norm_m1", op="norm", M=1, K=4096, res=True, normed=False),
        # a decoding batch before an expert layer: the router reads the normed rows in bf16
        dict(name="norm_m16_k2048_y", op="norm", M=16, K=2048, res=True, normed=True),
        # the prefill of 2048 tokens before the attention projection
        dict(name="norm_m2048", op="norm", M=2048, K=4096, res=True, normed=False),
        # a ragged batch of prompts, no residual (the first norm of a model), a wider model
        dict(name="norm_m4001_k6144_nores", op="norm", M=4001, K=6144, res=False, normed=False),
        # the largest prefill
        dict(name="norm_m16384", op="norm", M=16384, K=4096, res=True, normed=False),
        # the attention projection of one token
        dict(name="gemv_qkv_m1", op="gemv", M=1, K=4096, N=6144, G=32, table=0.7),
        # the gate and up projection of one token, the group size that high clustering chooses
        dict(name="gemv_ffn_m1_g64", op="gemv", M=1, K=4096, N=24576, G=64, table=0.7),
        # the down projection of a few tokens: a long K, small groups, no table
        dict(name="gemv_w2_m5_g16", op="gemv", M=5, K=12288, N=4096, G=16, table=0.0),
        # the gate and up projection of a decoding batch
        dict(name="gemv_ffn_m16", op="gemv", M=16, K=4096, N=24576, G=32, table=0.7),
        # one token through its 8 of 128 experts: gate and up
        dict(name="grouped_up_t1", op="gemv_grouped", T=1, top=8, fan=8, E=128, K=2048, N=1536, G=32, table=0.7),
        # a decoding batch through the experts' down projection: a row of its own for each choice
        dict(name="grouped_down_t16", op="gemv_grouped", T=16, top=8, fan=1, E=128, K=768, N=2048, G=32, table=0.7),
        # a larger decoding batch, where most experts have several rows
        dict(name="grouped_up_t33", op="gemv_grouped", T=33, top=8, fan=8, E=128, K=2048, N=1536, G=32, table=0.7),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gemv", "gemv_grouped"])
    if op == "norm":
        M, K = _spread(rng, 1, 16384), 256 * rng.randint(1, 48)
        return dict(op=op, M=max(1, min(M, 16384 * 4096 // K // 2)), K=K, res=rng.random() < 0.7, normed=rng.random() < 0.4)
    G, table = rng.choice([16, 32, 64]), rng.choice([0.0, 0.3, 0.7, 0.95])
    if op == "gemv":
        K, N = 256 * _spread(rng, 1, 48), 16 * _spread(rng, 2, 1536)
        return dict(op=op, M=_spread(rng, 1, 20), K=K, N=min(N, 4096 * 24576 // K // 16 * 16), G=G, table=table)
    top, E = rng.choice([1, 2, 4, 8]), rng.choice([8, 32, 64, 128])
    return dict(op=op, T=_spread(rng, 1, 33), top=top, fan=rng.choice([1, top]), E=E, K=256 * _spread(rng, 1, 8),
                N=16 * _spread(rng, 4, 128), G=G, table=table)


# ---- inputs -----------------------------------------------------------------------------------

def _slots(G):
    """Width of one scale slot of the weight layout."""
    return 16 if G == 16 else 32


def _entries(K, G, share):
    return int(share * (K // G))


def _kl(K, G, share):
    return (_entries(K, G, share) + 15) // 16 * 16


def _swizzle(slots):
    """Scale bytes (E, rows, slots) in the tensor-core scale layout: one flat run for each of E."""
    E, rows, n = slots.shape
    pad = (rows + 127) // 128 * 128
    full = torch.zeros((E, pad, n), dtype=torch.uint8, device=slots.device)
    full[:, :rows] = slots
    return full.view(E, pad // 128, 4, 32, n // 4, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(E, -1)


def _weight(gen, E, N, K, G, sd=0.02):
    """Normal weights of E experts in MXFP4 (codes and scales in the library's layouts), quantized here."""
    dev = gen.device
    QW = torch.empty((E, N, K // 2), dtype=torch.uint8, device=dev)
    slot = torch.empty((E, N, K // _slots(G)), dtype=torch.uint8, device=dev)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
    for e in range(E):
        W = torch.randn((N, K // G, G), generator=gen, device=dev) * sd
        ex = torch.floor(torch.log2(W.abs().amax(2).clamp_min(1e-30))) - 2
        code = torch.bucketize(W.abs() * torch.exp2(-ex)[..., None], edges).to(torch.uint8)
        code = (code | ((W < 0).to(torch.uint8) << 3)).view(N, K // 2, 2)
        QW[e] = code[..., 0] | (code[..., 1] << 4)
        slot[e] = (ex + 127).to(torch.uint8).repeat_interleave(G // _slots(G), 1)
    return QW, _swizzle(slot)


def _tables(gen, E, K, G, share):
    """E tables of K/G entries (one protected channel in a share of the groups, -1 elsewhere)."""
    n, dev = K // G, gen.device
    order = torch.rand((E, n), generator=gen, device=dev).argsort(1)
    ch = torch.randint(0, G, (E, n), generator=gen, device=dev)
    return torch.where(order < _entries(K, G, share), ch, torch.full_like(ch, -1)).to(torch.int8)


def _tokens(gen, M, K, G, L):
    """Normal rows whose outliers, of 20 to 80, sit at the channels of the table L (K/G entries)."""
    dev = gen.device
    X = torch.randn((M, K), generator=gen, device=dev)
    at = torch.arange(K // G, device=dev) * G + L.long().clamp_min(0)
    big = torch.empty((M, K // G), device=dev).uniform_(20, 80, generator=gen)
    X[:, at] = torch.where(L >= 0, big * torch.sign(X[:, at]), X[:, at])
    return X.to(torch.bfloat16)


def _experts(gen, T, top, E):
    """Each token's `top` different experts, some experts more popular than others (weights 1/rank^1.1)."""
    dev = gen.device
    rank = torch.randperm(E, generator=gen, device=dev) + 1
    u = torch.rand((T, E), generator=gen, device=dev).clamp_min(1e-9)
    key = -1.1 * torch.log(rank.float()) - torch.log(-torch.log(u))
    return key.topk(top, 1).indices.to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        scale = 1 + 9 * torch.rand((M, 1), generator=gen, device=dev)
        s["X"] = (torch.randn((M, K), generator=gen, device=dev) * scale).to(torch.bfloat16)
        s["res_rows"] = (torch.randn((M, K), generator=gen, device=dev) * 4).to(torch.bfloat16) if case["res"] else None
        s["gamma"] = (1 + 0.3 * torch.randn(K, generator=gen, device=dev)).to(torch.bfloat16)
        s["eps"] = 1e-6
        s["H"] = torch.empty((M, K), dtype=torch.bfloat16, device=dev) if case["res"] else None
        s["Y"] = torch.empty((M, K), dtype=torch.bfloat16, device=dev) if case["normed"] else None
        s["QX8"] = torch.empty((M, K), dtype=torch.uint8, device=dev)
        s["SX"] = torch.empty((M + 127) // 128 * 128 * K // 32, dtype=torch.uint8, device=dev)
        # the values that the 8-bit codes and scales stand for
        s["values"], s["scales"] = s["QX8"].view(torch.float8_e4m3fn), s["SX"].view(torch.float8_e8m0fnu)
        return s
    K, N, G, E = case["K"], case["N"], case["G"], case.get("E", 1)
    s["K_L"] = _kl(K, G, case["table"])
    s["QW"], s["SW"] = _weight(gen, E, N, K, G)
    s["L"] = _tables(gen, E, K, G, case["table"]) if s["K_L"] else None
    entries = torch.full((K // G,), -1, device=dev) if s["L"] is None else s["L"][0]
    s["WL"] = None
    if s["K_L"]:
        s["WL"] = (torch.randn((E, N, s["K_L"]), generator=gen, device=dev) * 0.02).to(torch.bfloat16)
        s["WL"][:, :, _entries(K, G, case["table"]):] = 0
    if case["op"] == "gemv":
        s["X"] = _tokens(gen, case["M"], K, G, entries)
        s["Y"] = torch.empty((case["M"], N), dtype=torch.bfloat16, device=dev)
        return s
    s["rows"] = case["T"] * case["top"]
    s["X"] = _tokens(gen, s["rows"] // case["fan"], K, G, entries)
    s["expert"] = _experts(gen, case["T"], case["top"], E).reshape(-1)
    s["Y"] = torch.empty((s["rows"], N), dtype=torch.bfloat16, device=dev)
    return s


# ---- the plain forms --------------------------------------------------------------------------

def _plain_norm(s):
    M, K = s["M"], s["K"]
    h = s["X"].float()
    if s["res_rows"] is not None:
        h = h + s["res_rows"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"]) * s["gamma"].float()
    block = y.view(M, K // 32, 32)
    amax = block.abs().amax(2)
    ex = torch.where(amax > 0, torch.frexp(amax).exponent - 9, -127).clamp(-127, 127)
    q = torch.ldexp(block, -ex[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(M, K)
    out = [q, _swizzle((ex + 127).to(torch.uint8)[None]).view(-1).view(torch.float8_e8m0fnu)]
    if s["res_rows"] is not None:
        out.append(h.to(torch.bfloat16))
    if s["normed"]:
        out.append(y.to(torch.bfloat16))
    return out


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _dequantize(QW, SW, N, K, G):
    """The weights in 32 bits, (E, N, K), from codes (E, N, K/2) and swizzled scales (E, bytes)."""
    E, V = QW.shape[0], _slots(G)
    value = torch.tensor(_E2M1 + [-v for v in _E2M1], device=QW.device)
    codes = torch.stack((QW & 15, QW >> 4), 3).view(E, N, K)
    slot = SW.view(E, -1, K // V // 4, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, -1, K // V)[:, :N]
    scale = torch.exp2(slot.float() - 127)
    return (value[codes.int()].view(E, N, K // V, V) * scale[..., None]).view(E, N, K)


def _split(X, L, K, G, K_L):
    """X (rows, K) in 32 bits without its row's table channels, and those channels' values (rows, K_L).
    L: (rows, K/G)."""
    X = X.float()
    at = torch.arange(K // G, device=X.device) * G + L.long().clamp_min(0)
    out = torch.gather(X, 1, at) * (L >= 0)
    B = torch.zeros((X.shape[0], K_L + 1), device=X.device)
    column = torch.where(L >= 0, torch.cumsum(L >= 0, 1) - 1, K_L)
    B.scatter_(1, column, out)
    return X.scatter_add(1, at, -out), B[:, :K_L]


def _plain_gemv(s):
    W = _dequantize(s["QW"], s["SW"], s["N"], s["K"], s["G"])[0]
    if not s["K_L"]:
        return (s["X"].float() @ W.t()).to(torch.bfloat16)
    X, B = _split(s["X"], s["L"].expand(s["M"], -1), s["K"], s["G"], s["K_L"])
    return (X @ W.t() + B @ s["WL"][0].float().t()).to(torch.bfloat16)


def _plain_grouped(s):
    e = s["expert"].long()
    X = s["X"].repeat_interleave(s["fan"], 0)
    W = _dequantize(s["QW"][e], s["SW"][e], s["N"], s["K"], s["G"])
    if not s["K_L"]:
        return torch.bmm(W, X.float()[..., None])[..., 0].to(torch.bfloat16)
    X, B = _split(X, s["L"][e], s["K"], s["G"], s["K_L"])
    Y = torch.bmm(W, X[..., None]) + torch.bmm(s["WL"][e].float(), B[..., None])
    return Y[..., 0].to(torch.bfloat16)


# ---- one pass ---------------------------------------------------------------------------------

def _call(s):
    """The same by the library, as a serving program calls it: outputs in buffers that it keeps."""
    global _osc
    if _osc is None:
        from w4a4_outlier_separated_b200 import osc as _osc
    if s["op"] == "norm":
        _osc.osc_add_rmsnorm_quantize_fp8(s["X"], s["res_rows"], s["gamma"], s["eps"], s["H"], s["Y"], s["QX8"], s["SX"])
        return [t for t in (s["values"], s["scales"], s["H"], s["Y"]) if t is not None]
    if s["op"] == "gemv":
        _osc.osc_gemv(s["X"], s["G"], s["L"], s["K_L"], s["QW"], s["SW"], s["WL"], s["N"], s["Y"])
        return s["Y"]
    _osc.osc_gemv_grouped(s["X"], s["fan"], s["expert"], s["E"], s["G"], s["L"], s["K_L"], s["QW"], s["SW"], s["WL"],
                          s["N"], s["Y"])
    return s["Y"]


def run(state):
    if own:
        return _call(state)
    return {"norm": _plain_norm, "gemv": _plain_gemv, "gemv_grouped": _plain_grouped}[state["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------------------

def _distinct(T, top, E):
    """How many different experts T tokens choose, on average (a fixed sample of the choice in `prepare`)."""
    rng, total = random.Random(0), 0
    weight = [(r + 1) ** -1.1 for r in range(E)]
    for _ in range(16):
        seen = set()
        for _ in range(T):
            keys = sorted(range(E), key=lambda r: rng.expovariate(1.0) / weight[r])
            seen.update(keys[:top])
        total += len(seen)
    return total / 16


def work(case):
    K = case["K"]
    if case["op"] == "norm":
        M = case["M"]
        scales = (M + 127) // 128 * 128 * K // 32
        per = 2 + 1 + (4 if case["res"] else 0) + (2 if case["normed"] else 0)
        return {"bytes": M * K * per + scales + 2 * K, "flops": 8.0 * M * K}
    N, G = case["N"], case["G"]
    K_L = _kl(K, G, case["table"])
    weight = N * K / 2 + N * K / _slots(G) + 2 * N * K_L + (K // G if K_L else 0)
    if case["op"] == "gemv":
        M = case["M"]
        return {"bytes": weight + 2 * M * (K + N), "flops": 2.0 * M * N * (K + K_L)}
    rows = case["T"] * case["top"]
    return {"bytes": weight * _distinct(case["T"], case["top"], case["E"]) + 2 * rows * (K / case["fan"] + N) + 4 * rows,
            "flops": 2.0 * rows * N * (K + K_L)}


# ---- the definition in 64 bits ----------------------------------------------------------------

def _scale_bytes(flat, rows, slots):
    """(rows, slots) scale bytes out of the tensor-core layout, by its address formula."""
    r = torch.arange(rows, device=flat.device)[:, None]
    c = torch.arange(slots, device=flat.device)[None]
    byte = ((r // 128) * (slots // 4) + c // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + c % 4
    return flat.reshape(-1)[byte]


def _weight64(QW, SW, N, K, G):
    """One expert's weights: sign * (1.m * 2^(e-1), or m / 2 where e = 0) * 2^(scale - 127)."""
    code = torch.empty((N, K), dtype=torch.int64, device=QW.device)
    code[:, 0::2], code[:, 1::2] = (QW % 16).long(), (QW // 16).long()
    m, e, negative = code % 2, code // 2 % 4, code >= 8
    value = torch.where(e == 0, m.double() / 2, (1 + m.double() / 2) * torch.pow(2.0, (e - 1).double()))
    V = _slots(G)
    two = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=QW.device), _scale_bytes(SW, N, K // V).double() - 127)
    return torch.where(negative, -value, value) * two.repeat_interleave(V, 1)


def _product64(x, QW, SW, WL, L, N, K, G):
    """Rows x (in 64 bits) against one weight, channel by channel of the table from W_L."""
    W = _weight64(QW, SW, N, K, G)
    if L is not None:
        place = 0
        for group, channel in enumerate(L.tolist()):
            if channel >= 0:
                W[:, group * G + channel] = WL[:, place].double()
                place += 1
    return x @ W.t()


def exact(case, seed):
    s = prepare(case, seed)
    K, table = case["K"], None
    if case["op"] == "norm":
        M = case["M"]
        h = s["X"].double() + (s["res_rows"].double() if case["res"] else 0)
        y = s["gamma"].double() * h / torch.sqrt((h * h).sum(1) / K + s["eps"])[:, None]
        amax = y.reshape(M, K // 32, 32).abs().max(2).values
        e = torch.floor(torch.log2(amax)) - 8
        # the elements before their rounding to 8 bits; the scales, whose exponent steps where a
        # largest value crosses a power of two, have no value that a rounding leaves near
        q = (y.reshape(M, K // 32, 32) / torch.pow(2.0, e)[..., None]).clamp(-448, 448).reshape(M, K)
        return [q, None] + ([h] if case["res"] else []) + ([y] if case["normed"] else [])
    N, G = case["N"], case["G"]
    if case["op"] == "gemv":
        table = None if s["L"] is None else s["L"][0]
        return _product64(s["X"].double(), s["QW"][0], s["SW"][0], None if table is None else s["WL"][0], table, N, K, G)
    Y = torch.zeros((s["rows"], N), dtype=torch.float64, device=s["X"].device)
    choice = s["expert"].tolist()
    for e in sorted(set(choice)):
        rows = [r for r, x in enumerate(choice) if x == e]
        table = None if s["L"] is None else s["L"][e]
        x = s["X"][[r // case["fan"] for r in rows]].double()
        Y[rows] = _product64(x, s["QW"][e], s["SW"][e], None if table is None else s["WL"][e], table, N, K, G)
    return Y
