"""Cases of the 8-bit integer and ragged-by-expert products, their plain forms and their
values in 64 bits.

  quantize      X[M,K] -> int8 codes and one scale per row: s = amax|x| / 127 (1 for an
                all-zero row), q = round-half-even(x / s)
  int8          C = act(sa[m] sb[n] sum_k Aq[m,k] Bq[n,k] + bias[n])
  ragged        rows offsets[e] .. offsets[e+1]-1 of A times expert e's matrix:
                C[t] = act(A[t] B[e] + bias[e]); rows of no expert keep what they held
  wgrad         dB[e] = A[rows of e]^T D[rows of e], dbias[e] = sum of D's rows of e
  int8_ragged   the int8 product with expert e's codes and scales for the rows of e

`own` selects the library's calls; otherwise the same values come from elementary torch
operations in 32 bits, rounded once.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # One decode step's activations of 16 sequences: the launch is all there is.
        dict(name="quantize decode", op="quantize", M=16, K=4096, dtype="bf16"),
        # A long prompt's FFN activations before the down projection: pure memory traffic.
        dict(name="quantize prefill", op="quantize", M=8192, K=16384, dtype="bf16"),
        # One token through the FFN's up projection: streams the 64 MB of weight codes.
        dict(name="int8 decode", op="int8", M=1, K=4096, N=16384, out="bf16", act="none", bias=False),
        # A short odd batch with odd feature counts (padded row pitches), FP16 out.
        dict(name="int8 odd", op="int8", M=333, K=4100, N=4107, out="f16", act="silu", bias=True),
        # Prefill of 8192 tokens through the up projection with its bias and GeLU.
        dict(name="int8 prefill", op="int8", M=8192, K=4096, N=16384, out="bf16", act="gelu_tanh", bias=True),
        # 64 routed rows of a decode batch over 32 small experts, five of them idle.
        dict(name="ragged decode", op="ragged", T=64, E=32, active=27, tail=0, skew=0.5, K=2048, N=4096, dtype="bf16",
             out="bf16", act="none", bias=False, transposed=False),
        # Training step of eight wide experts, forward, activation fused.
        dict(name="ragged forward", op="ragged", T=16384, E=8, active=8, tail=0, skew=0.5, K=4096, N=16384, dtype="bf16",
             out="bf16", act="silu", bias=False, transposed=False),
        # Gradient of the inputs of 64 fine-grained experts (weights read transposed), FP16,
        # an odd token count, idle experts and a padded batch.
        dict(name="ragged dX", op="ragged", T=8191, E=64, active=61, tail=57, skew=1.0, K=1024, N=2048, dtype="f16",
             out="f16", act="none", bias=False, transposed=True),
        # Weight gradient of eight wide experts, BF16 out.
        dict(name="wgrad wide", op="wgrad", T=16384, E=8, active=8, tail=0, skew=0.5, K=4096, N=4096, dtype="bf16",
             out="bf16", dbias=False),
        # Weight and bias gradients of 64 fine-grained experts, odd token count, FP32 out.
        dict(name="wgrad fine", op="wgrad", T=12345, E=64, active=59, tail=33, skew=1.0, K=2048, N=1000, dtype="bf16",
             out="f32", dbias=True),
        # Decode batch over quantised experts.
        dict(name="int8 experts decode", op="int8_ragged", T=48, E=32, active=24, tail=0, skew=0.5, K=4096, N=2048,
             out="bf16", act="none", bias=False),
        # Prefill over quantised experts with bias and activation.
        dict(name="int8 experts prefill", op="int8_ragged", T=16384, E=32, active=31, tail=5, skew=1.0, K=4096, N=4096,
             out="f16", act="silu", bias=True),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]; odd ones as often as even ones."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "int8", "ragged", "wgrad", "int8_ragged"])
    if op == "quantize":
        K = _log(rng, 64, 16384)
        return dict(op=op, M=_log(rng, 1, 8192), K=K, dtype=rng.choice(["bf16", "f16", "f32"]))
    out = rng.choice(["bf16", "f16", "f32"])
    act = rng.choice(["none", "none", "silu", "gelu_tanh"])
    bias = rng.random() < 0.5
    if op == "int8":
        return dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 256, 8192), N=_log(rng, 256, 16384), out=out, act=act,
                    bias=bias)
    T, E = _log(rng, 8, 16384), _log(rng, 2, 64)
    tail = rng.choice([0, 0, rng.randint(0, T // 4)])
    active = max(1, min(T - tail, E - rng.randint(0, E // 4)))
    K = _log(rng, 256, 4096)
    N = min(_log(rng, 256, 4096), (1 << 28) // (E * K))  # the matrices of all experts: half of the widest case's
    c = dict(op=op, T=T, E=E, active=active, tail=tail, skew=rng.choice([0.0, 0.5, 1.0]), K=K, N=N, out=out)
    if op == "wgrad":
        c.update(dtype=rng.choice(["bf16", "f16"]), dbias=rng.random() < 0.5)
    else:
        c.update(act=act, bias=bias)
        if op == "ragged":
            c.update(dtype=rng.choice(["bf16", "f16"]), transposed=rng.random() < 0.5)
    return c


# ---------------------------------------------------------------- inputs


def _pitched(t, align=16):
    """The same values with rows that start on `align`-byte boundaries, as a serving
    program's padded buffers have them."""
    n = t.shape[-1]
    unit = align // t.element_size()
    pad = -(-n // unit) * unit
    if pad == n:
        return t
    buf = torch.zeros(t.shape[:-1] + (pad,), dtype=t.dtype, device=t.device)
    buf[..., :n] = t
    return buf[..., :n]


def _normal(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _codes(g, shape):
    """int8 codes as a row quantiser leaves them: normal, a few at the limits."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda").mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
    return out


def _offsets(case, seed):
    """Row offsets of the experts: `active` of them get at least one row each, the rest of
    the rows by weights exp(skew z); the last `tail` rows belong to none."""
    r = np.random.default_rng(seed + 77)
    used = case["T"] - case["tail"]
    w = np.exp(case["skew"] * r.standard_normal(case["active"]))
    counts = np.zeros(case["E"], np.int64)
    which = np.sort(r.permutation(case["E"])[:case["active"]])
    counts[which] = 1 + r.multinomial(used - case["active"], w / w.sum())
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "quantize":
        # Activations: a few channels are much larger than the rest.
        x = _normal(g, (case["M"], case["K"]), torch.float32)
        x *= torch.exp(_normal(g, (case["K"],), torch.float32))
        s["x"] = _pitched(x.to(DT[case["dtype"]]))
        return s
    K, N = case["K"], case["N"]
    if op in ("ragged", "wgrad", "int8_ragged"):
        T, E = case["T"], case["E"]
        o = _offsets(case, seed)
        s["offsets"] = torch.from_numpy(o).cuda()
        s["cap"] = int((o[1:] - o[:-1]).max())
    if op == "int8":
        s["a"], s["sa"] = _pitched(_codes(g, (case["M"], K))), torch.rand(case["M"], generator=g, device="cuda") * 0.02 + 0.01
        s["b"], s["sb"] = _pitched(_codes(g, (N, K))), (torch.rand(N, generator=g, device="cuda") + 0.5) * (0.03 / K ** 0.5)
    elif op == "int8_ragged":
        s["a"], s["sa"] = _pitched(_codes(g, (T, K))), torch.rand(T, generator=g, device="cuda") * 0.02 + 0.01
        s["b"] = _pitched(_codes(g, (E, N, K)))
        s["sb"] = (torch.rand((E, N), generator=g, device="cuda") + 0.5) * (0.03 / K ** 0.5)
    elif op == "ragged":
        dt = DT[case["dtype"]]
        s["a"] = _pitched(_normal(g, (T, K), dt))
        if case["transposed"]:  # the forward's weights [E, N, K], read as their transposes
            s["b"] = _pitched(_normal(g, (E, N, K), dt, K ** -0.5)).transpose(1, 2)
        else:
            s["b"] = _pitched(_normal(g, (E, K, N), dt, K ** -0.5))
    else:
        dt = DT[case["dtype"]]
        s["a"] = _pitched(_normal(g, (T, K), dt))
        s["d"] = _pitched(_normal(g, (T, N), dt, T ** -0.5))
        s["out"] = _pitched(torch.empty((E, K, N), dtype=DT[case["out"]], device="cuda"))
        s["dbias"] = torch.empty((E, N), dtype=torch.float32, device="cuda") if case["dbias"] else None
        return s
    rows = case["M"] if op == "int8" else T
    s["bias"] = None
    if case["bias"]:
        s["bias"] = _normal(g, (N,) if op == "int8" else (E, N), torch.bfloat16, 0.5)
    s["out"] = _pitched(torch.full((rows, N), 0.25, dtype=DT[case["out"]], device="cuda"))
    return s


# ---------------------------------------------------------------- one pass


def _act(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu_tanh":
        return x / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _rows(s, T):
    """Row numbers of every expert, padded to the longest one's count, and which of them are real."""
    o = s["offsets"].long()
    rows = o[:-1, None] + torch.arange(s["cap"], device=o.device)
    return rows.clamp(max=T - 1), rows < o[1:, None]


def _by_expert(x, rows, real):
    return torch.where(real[..., None], x.float()[rows], 0.0)


def _to_rows(s, y, keep):
    """The rows of the padded products y[E, cap, N] back in token order; rows of no expert from `keep`."""
    o = s["offsets"].long()
    t = torch.arange(keep.shape[0], device=o.device)
    e = torch.searchsorted(o[1:], t, right=True).clamp(max=o.numel() - 2)
    mine = (t >= o[0]) & (t < o[-1])
    at = (t - o[e]).clamp(0, y.shape[1] - 1)
    return torch.where(mine[:, None], y[e, at].to(keep.dtype), keep)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        x = s["x"].float()
        amax = x.abs().amax(dim=1)
        scale = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 127.0))
        return (x / scale[:, None]).round().to(torch.int8), scale
    if op == "int8":
        y = (s["a"].float() @ s["b"].float().t()) * (s["sa"][:, None] * s["sb"][None, :])
        if c["bias"]:
            y = y + s["bias"].float()
        return _act(y, c["act"]).to(DT[c["out"]])
    rows, real = _rows(s, c["T"])
    x = _by_expert(s["a"], rows, real)
    if op == "wgrad":
        d = _by_expert(s["d"], rows, real)
        dw = torch.bmm(x.transpose(1, 2), d).to(DT[c["out"]])
        return (dw, d.sum(dim=1)) if c["dbias"] else dw
    if op == "int8_ragged":
        y = torch.bmm(x, s["b"].float().transpose(1, 2)) * (s["sa"][rows][..., None] * s["sb"][:, None, :])
    else:
        y = torch.bmm(x, s["b"].float())
    if c["bias"]:
        y = y + s["bias"].float()[:, None, :]
    return _to_rows(s, _act(y, c["act"]), s["out"])


def run(s):
    if not own:
        return _plain(s)
    import sm_gemm_b200 as sg
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        return sg.quantize_int8_rowwise(s["x"])
    if op == "int8":
        return sg.gemm_int8_scaled(s["a"], s["sa"], s["b"], s["sb"], bias=s["bias"], act=c["act"], out=s["out"])
    if op == "ragged":
        return sg.gemm_bf16_ragged(s["a"], s["b"], s["offsets"], bias=s["bias"], act=c["act"], out=s["out"])
    if op == "int8_ragged":
        return sg.gemm_int8_ragged(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], bias=s["bias"], act=c["act"],
                                   out=s["out"])
    dw = sg.gemm_bf16_ragged_wgrad(s["a"], s["d"], s["offsets"], out=s["out"], dbias=s["dbias"])
    return (dw, s["dbias"]) if c["dbias"] else dw


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op, K = case["op"], case["K"]
    if op == "quantize":
        M = case["M"]
        return {"bytes": M * K * (SIZE[case["dtype"]] + 1) + 4 * M, "flops": 3 * M * K}
    N, so = case["N"], SIZE[case["out"]]
    if op == "int8":
        M = case["M"]
        return {"bytes": (M + N) * (K + 4) + M * N * so + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    used, E, active = case["T"] - case["tail"], case["E"], case["active"]
    flops = 2 * used * N * K
    if op == "wgrad":
        return {"bytes": used * (K + N) * 2 + E * K * N * so + (4 * E * N if case["dbias"] else 0) + 4 * (E + 1),
                "flops": flops + (used * N if case["dbias"] else 0)}
    si = 1 if op == "int8_ragged" else 2
    extra = 4 * used + 4 * active * N if op == "int8_ragged" else 0
    return {"bytes": used * K * si + active * K * N * si + used * N * so + extra + (2 * active * N if case["bias"] else 0)
            + 4 * (E + 1), "flops": flops}


# ---------------------------------------------------------------- the same in 64 bits, expert by expert


def _act64(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        top = s["x"].double().abs().max(dim=1).values
        return None, torch.where(top > 0, top / 127.0, torch.ones_like(top))
    if op == "int8":
        y = s["a"].double() @ s["b"].double().T
        y = y * s["sa"].double()[:, None] * s["sb"].double()[None, :]
        return _act64(y if s["bias"] is None else y + s["bias"].double(), case["act"])
    o = s["offsets"].tolist()
    if op == "wgrad":
        dw = torch.zeros((case["E"], case["K"], case["N"]), dtype=torch.float64, device="cuda")
        db = torch.zeros((case["E"], case["N"]), dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            x, d = s["a"][o[e]:o[e + 1]].double(), s["d"][o[e]:o[e + 1]].double()
            dw[e] = x.T @ d
            db[e] = d.sum(0)
        return (dw, db) if case["dbias"] else dw
    y = s["out"].double().clone()
    for e in range(case["E"]):
        r = slice(o[e], o[e + 1])
        if op == "int8_ragged":
            z = (s["a"][r].double() @ s["b"][e].double().T) * s["sa"][r].double()[:, None] * s["sb"][e].double()
        else:
            z = s["a"][r].double() @ s["b"][e].double()
        y[r] = _act64(z if s["bias"] is None else z + s["bias"][e].double(), case["act"])
    return y
