"""The layer's expert products, as calls that can be timed and compared.

Three operators around the sparse MoE layer:

* ``grouped``: matrix products grouped by expert.  Row r of x in
  [offsets[e], offsets[e+1]) belongs to expert e, and y_r = W_e x_r with W of
  shape [E, M, K].  Its backward pass is dx_r = W_e^T dy_r and
  dW_e = sum over e's rows of dy_r x_r^T.
* ``quantize``: weights to 4 bits with one bf16 scale per group of K, and back.
* ``linear`` and ``layer``: products of bf16 tokens with such weights, for one matrix
  (y = x W^T) and for the whole expert layer (routed SwiGLU experts, the weighted
  combine and the shared expert).

4-bit weights: a matrix [M, K] is held as q, uint8 [M, K/2] (column 2j in the low and
2j+1 in the high four bits of byte j), and scales, bf16 [K/group, M]; its value at
(m, k) is (q(m, k) - 8) * scales[k // group, m].

``run`` computes an operator in elementary torch operations, or, where ``own`` is
true, through the library's calls.  ``exact`` computes it in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # The smallest training step of an expert matrix: the fp32 configuration the
        # parity tests use (64 tokens x 4 experts, D 256, two stacked 128-row halves).
        dict(name="grouped_train_fp32_small", op="grouped", way="train", dtype="fp32", rows=256,
             spare=0, E=16, M=256, K=256, skew=0.0),
        # Gate and up rows of a decode batch of 32 tokens x 8 experts, GLM-4.5-Air's
        # sizes: one to a few rows per expert, bound by reading the experts.
        dict(name="grouped_decode_air", op="grouped", way="forward", dtype="bf16", rows=256,
             spare=0, E=128, M=2816, K=4096, skew=0.0),
        # Down projection of a prompt of 8192 tokens x 8 experts, GLM-4.5's sizes.
        dict(name="grouped_prefill_down", op="grouped", way="forward", dtype="bf16", rows=65536,
             spare=0, E=160, M=5120, K=1536, skew=0.6),
        # Backward of gate and up for one of eight expert-parallel ranks, GLM-5's sizes:
        # 32 of 256 experts, skewed loads.
        dict(name="grouped_backward_glm5", op="grouped", way="backward", dtype="bf16", rows=16384,
             spare=0, E=32, M=4096, K=6144, skew=0.8),
        # A short odd batch in a longer buffer: empty experts, ragged segments, rows
        # behind the last one (a padded batch), the down projection of GLM-4.5-Air.
        dict(name="grouped_train_ragged", op="grouped", way="train", dtype="bf16", rows=3001,
             spare=71, E=128, M=4096, K=1408, skew=1.1),
        # One expert-parallel rank's gate and up matrices put into 4 bits and read back,
        # as a server does when it loads a bf16 checkpoint.
        dict(name="quantize_glm5_rank", op="quantize", E=32, M=4096, K=6144, group=128),
        # One small matrix with short groups (a shared expert's down projection).
        dict(name="quantize_small", op="quantize", E=1, M=4096, K=1408, group=32),
        # The shared expert's gate and up rows for a single token: latency counts.
        dict(name="linear_one_token", op="linear", N=1, M=2816, K=4096, group=128),
        # A dense projection for an odd batch (a few sequences with drafted tokens).
        dict(name="linear_odd_batch", op="linear", N=77, M=12288, K=5120, group=64),
        # Whole expert layers with 4-bit weights: a single token, and decode batches.
        dict(name="layer_air_one_token", op="layer", N=1, D=4096, E=128, k=8, d=1408, d_sh=1408,
             group=128, alpha=1.0, idle=0),
        dict(name="layer_air_decode", op="layer", N=32, D=4096, E=128, k=8, d=1408, d_sh=1408,
             group=128, alpha=1.0, idle=0),
        # 64 slots of a server's batch, three of them idle (their ids are the sentinel E).
        dict(name="layer_glm5_decode", op="layer", N=64, D=6144, E=256, k=8, d=2048, d_sh=2048,
             group=64, alpha=2.5, idle=3),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped", "quantize", "linear", "linear", "layer",
                     "layer"])
    if op == "grouped":
        way = rng.choice(["forward", "backward", "train"])
        if rng.random() < 0.2:  # fp32: the small sizes that precision is checked at
            return dict(op=op, way=way, dtype="fp32", rows=_log_int(rng, 1, 4000),
                        spare=rng.choice([0, 0, 5]), E=_log_int(rng, 1, 64),
                        M=_log_int(rng, 8, 1024, 4), K=_log_int(rng, 8, 1024, 4),
                        skew=rng.choice([0.0, 1.0]))
        E, M, K = _log_int(rng, 1, 256), _log_int(rng, 64, 6144, 8), _log_int(rng, 64, 6144, 8)
        most = 1.2e9 if way == "forward" else 7.0e8  # weights in all
        while E * M * K > most:
            E = (E + 1) // 2
        rows = _log_int(rng, 1, 65536)
        turns = {"forward": 1, "backward": 2, "train": 3}[way]
        rows = max(1, min(rows, int(1.6e12 / (2.0 * M * K * turns))))
        return dict(op=op, way=way, dtype="bf16", rows=rows, spare=rng.choice([0, 0, 1, 200]),
                    E=E, M=M, K=K, skew=rng.choice([0.0, 0.6, 1.1]))
    group = rng.choice([32, 64, 128])
    if op == "quantize":
        M, K = _log_int(rng, 8, 6144, 8), group * _log_int(rng, 1, 6144 // group)
        E = max(1, min(_log_int(rng, 1, 64), int(8.0e8 / (M * K))))
        return dict(op=op, E=E, M=M, K=K, group=group)
    if op == "linear":
        return dict(op=op, N=_log_int(rng, 1, 256), M=_log_int(rng, 64, 12288, 8),
                    K=group * _log_int(rng, 1, 6144 // group), group=group)
    E = _log_int(rng, 2, 256)
    N = _log_int(rng, 1, 128)
    return dict(op=op, N=N, D=128 * _log_int(rng, 2, 48), E=E, k=rng.randint(1, min(8, E)),
                d=128 * _log_int(rng, 1, 16), d_sh=128 * _log_int(rng, 1, 16), group=group,
                alpha=rng.choice([1.0, 2.5]), idle=rng.choice([0, 0, N // 8]))


# ----------------------------------------------------------------------------- inputs
def _sizes(case, seed):
    """Rows of each expert: a multinomial over popularities (rank + 1)^-skew."""
    r = np.random.default_rng(seed + 11)
    p = (r.permutation(case["E"]) + 1.0) ** -case["skew"]
    return r.multinomial(case["rows"], p / p.sum()).tolist()


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _tokens(n, dim, g, dtype):
    """Rows as the layer gets them: normalised to a root mean square of one."""
    z = torch.randn((n, dim), generator=g, device=DEV, dtype=torch.float32)
    return (z * torch.rsqrt(z.pow(2).mean(-1, keepdim=True) + 1e-6)).to(dtype)


def _weights(E, M, K, g, dtype):
    w = torch.empty((E, M, K), device=DEV, dtype=dtype)
    for e in range(E):
        w[e] = _normal((M, K), g, 0.02, dtype)
    return w


def _held(E, M, K, group, g):
    """4-bit weights of shape [E, M, K], from normal ones."""
    q = torch.empty((E, M, K // 2), device=DEV, dtype=torch.uint8)
    s = torch.empty((E, K // group, M), device=DEV, dtype=torch.bfloat16)
    for e in range(E):
        q[e], s[e] = _put(_normal((M, K), g, 0.02, torch.bfloat16), group)
    return q, s


def prepare(case, seed):
    g = _generator(seed)
    st = dict(case)
    if case["op"] == "grouped":
        dt = _TYPES[case["dtype"]]
        sizes = _sizes(case, seed)
        total = case["rows"] + case["spare"]
        st["sizes"] = sizes
        st["offsets"] = torch.tensor([0] + np.cumsum(sizes).tolist(), dtype=torch.int32, device=DEV)
        st["W"] = _weights(case["E"], case["M"], case["K"], g, dt)
        st["x"] = _tokens(total, case["K"], g, dt)
        if case["way"] != "forward":
            st["dy"] = _normal((total, case["M"]), g, 0.1, dt)
    elif case["op"] == "quantize":
        st["W"] = _weights(case["E"], case["M"], case["K"], g, torch.bfloat16)
    elif case["op"] == "linear":
        q, s = _held(1, case["M"], case["K"], case["group"], g)
        st["q"], st["s"] = q[0], s[0]
        st["x"] = _tokens(case["N"], case["K"], g, torch.bfloat16)
    else:
        N, D, E, k = case["N"], case["D"], case["E"], case["k"]
        st["gate_up"] = _held(E, 2 * case["d"], D, case["group"], g)
        st["down"] = _held(E, D, case["d"], case["group"], g)
        st["sh_gate_up"] = tuple(t[0] for t in _held(1, 2 * case["d_sh"], D, case["group"], g))
        st["sh_down"] = tuple(t[0] for t in _held(1, D, case["d_sh"], case["group"], g))
        st["x"] = _tokens(N, D, g, torch.bfloat16)
        score = torch.rand((N, E), generator=g, device=DEV)
        top = score.topk(k, dim=1)
        st["ids"] = top.indices.to(torch.int32)
        st["w"] = (case["alpha"] * top.values / top.values.sum(1, keepdim=True)).contiguous()
        st["ids"][N - case["idle"]:] = E
        # the plain form's own plan: which (token, slot) pairs each chosen expert has
        ids = st["ids"].cpu()
        st["pairs"] = []
        for e in sorted(set(ids.flatten().tolist()) - {E}):
            tok, slot = torch.nonzero(ids == e, as_tuple=True)
            st["pairs"].append((e, tok.to(DEV), slot.to(DEV)))
    return st


# ----------------------------------------------------------------------------- plain forms
def _put(w, group):
    """One bf16 matrix [M, K] in 4 bits: (q, scales)."""
    M, K = w.shape
    v = w.float().view(M, K // group, group)
    s = (v.abs().amax(-1) / 7.0).to(torch.bfloat16)
    sf = s.float()[:, :, None]
    n = torch.where(sf > 0, torch.round(v / sf), torch.zeros_like(v)).clamp(-8, 7) + 8
    n = n.to(torch.uint8).view(M, K)
    return n[:, 0::2] | (n[:, 1::2] << 4), s.t().contiguous()


def _get(q, s):
    """The fp32 values of one matrix in 4 bits."""
    M, half = q.shape
    n = torch.stack((q & 15, q >> 4), dim=2).view(M, 2 * half).float() - 8.0
    return (n.view(M, s.shape[0], -1) * s.t().float()[:, :, None]).view(M, 2 * half)


def _grouped_plain(st):
    x, W, sizes, way = st["x"], st["W"], st["sizes"], st["way"]
    out = []
    if way != "backward":
        y = torch.zeros((x.shape[0], st["M"]), device=DEV, dtype=x.dtype)
        a = 0
        for e, n in enumerate(sizes):
            if n:
                y[a:a + n] = (x[a:a + n].float() @ W[e].float().t()).to(x.dtype)
            a += n
        out.append(y)
    if way != "forward":
        dx, dW = torch.zeros_like(x), torch.zeros_like(W)
        a = 0
        for e, n in enumerate(sizes):
            if n:
                d = st["dy"][a:a + n].float()
                dx[a:a + n] = (d @ W[e].float()).to(x.dtype)
                dW[e] = (d.t() @ x[a:a + n].float()).to(x.dtype)
            a += n
        out += [dx, dW]
    return out


def _expert(x, gate_up, down):
    """One SwiGLU expert in fp32."""
    g, u = (x @ gate_up.t()).chunk(2, dim=1)
    return (g / (1.0 + torch.exp(-g)) * u) @ down.t()


def _layer_plain(st):
    x = st["x"].float()
    y = _expert(x, _get(*st["sh_gate_up"]), _get(*st["sh_down"]))
    (gq, gs), (dq, ds) = st["gate_up"], st["down"]
    for e, tok, slot in st["pairs"]:
        o = _expert(x[tok], _get(gq[e], gs[e]), _get(dq[e], ds[e]))
        y.index_add_(0, tok, o * st["w"][tok, slot][:, None])
    return y.to(torch.bfloat16)


# ----------------------------------------------------------------------------- run
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(st):
    if st["op"] == "grouped":
        return _grouped_plain(st)
    if st["op"] == "quantize":
        back = torch.empty_like(st["W"])
        for e in range(st["E"]):
            back[e] = _get(*_put(st["W"][e], st["group"])).to(torch.bfloat16)
        return back
    if st["op"] == "linear":
        return (st["x"].float() @ _get(st["q"], st["s"]).t()).to(torch.bfloat16)
    return _layer_plain(st)


def _run_own(st):
    import sparse_moe_layer_02_b200 as moe

    if st["op"] == "grouped":
        out = []
        if st["way"] != "backward":
            out.append(moe.moe_grouped_linear(st["x"], st["W"], st["offsets"]))
        if st["way"] != "forward":
            out.append(moe.moe_grouped_linear_dgrad(st["dy"], st["W"], st["offsets"]))
            out.append(moe.moe_grouped_linear_wgrad(st["dy"], st["x"], st["offsets"]))
        return out
    if st["op"] == "quantize":
        return moe.moe_dequantize(*moe.moe_quantize(st["W"], st["group"]))
    if st["op"] == "linear":
        return moe.moe_linear_quant(st["x"], st["q"], st["s"])
    return moe.moe_forward_quant(st["x"], st["gate_up"], st["down"], st["sh_gate_up"],
                                 st["sh_down"], st["ids"], st["w"])


# ----------------------------------------------------------------------------- work
def _hit(E, draws):
    """Experts with at least one of `draws` even draws."""
    return E * (1.0 - (1.0 - 1.0 / E) ** draws)


def work(case):
    if case["op"] == "grouped":
        es = 2 if case["dtype"] == "bf16" else 4
        rows, E, M, K = case["rows"], case["E"], case["M"], case["K"]
        hit = sum(1 for n in _sizes(case, 0) if n)
        x, y, w = rows * K * es, rows * M * es, M * K * es
        table = (E + 1) * 4
        parts = {"forward": (1, x + hit * w + y), "backward": (2, y + hit * w + x + x + E * w),
                 "train": (3, x + hit * w + y + y + x + E * w)}
        turns, nbytes = parts[case["way"]]
        return {"bytes": nbytes + table, "flops": 2.0 * turns * rows * M * K}
    if case["op"] == "quantize":
        n = case["E"] * case["M"] * case["K"]
        return {"bytes": 2.0 * n + 2.0 * n, "flops": 3.0 * n}
    if case["op"] == "linear":
        N, M, K = case["N"], case["M"], case["K"]
        return {"bytes": M * K / 2 + 2.0 * M * K / case["group"] + 2.0 * N * (M + K),
                "flops": 2.0 * N * M * K}
    N, D, k = case["N"] - case["idle"], case["D"], case["k"]
    hit = case["E"] * (1.0 - (1.0 - k / case["E"]) ** N)
    per = 0.5 + 2.0 / case["group"]
    return {"bytes": per * 3 * D * (hit * case["d"] + case["d_sh"]) + 4.0 * case["N"] * D
            + 8.0 * case["N"] * k,
            "flops": 6.0 * D * (N * k * case["d"] + case["N"] * case["d_sh"])}


# ----------------------------------------------------------------------------- exact
def _values64(q, s):
    """The values of 4-bit weights in 64 bits, nibble by nibble."""
    M, half = q.shape
    v = torch.empty((M, 2 * half), device=DEV, dtype=torch.float64)
    v[:, 0::2] = torch.remainder(q, 16).double() - 8.0
    v[:, 1::2] = torch.div(q, 16, rounding_mode="floor").double() - 8.0
    return v * s.double().t().repeat_interleave(2 * half // s.shape[0], dim=1)


def _swiglu64(x, gu, dn):
    h = x @ gu.t()
    d = h.shape[1] // 2
    return ((h[:, :d] * torch.sigmoid(h[:, :d])) * h[:, d:]) @ dn.t()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "grouped":
        off = st["offsets"].tolist()
        x, W = st["x"], st["W"]
        need = 8 * (x.numel() * 2 + x.shape[0] * case["M"] * 2 + W.numel())
        if need > 60e9:
            return None
        spans = [(e, slice(off[e], off[e + 1])) for e in range(case["E"]) if off[e] < off[e + 1]]
        out = []
        if case["way"] != "backward":
            y = torch.zeros((x.shape[0], case["M"]), device=DEV, dtype=torch.float64)
            for e, r in spans:
                torch.mm(x[r].double(), W[e].double().t(), out=y[r])
            out.append(y)
        if case["way"] != "forward":
            dx = torch.zeros(x.shape, device=DEV, dtype=torch.float64)
            dW = torch.zeros(W.shape, device=DEV, dtype=torch.float64)
            for e, r in spans:
                d = st["dy"][r].double()
                torch.mm(d, W[e].double(), out=dx[r])
                torch.mm(d.t(), x[r].double(), out=dW[e])
            out += [dx, dW]
        return out
    if case["op"] == "quantize":
        back = torch.empty(st["W"].shape, device=DEV, dtype=torch.float64)
        G = case["group"]
        for e in range(case["E"]):
            w = st["W"][e].double().reshape(-1, G)
            step = (w.abs().max(dim=1, keepdim=True).values / 7.0).to(torch.bfloat16).double()
            level = torch.where(step > 0, torch.round(w / step), torch.zeros_like(w))
            back[e] = (level.clamp(-8, 7) * step).view(case["M"], case["K"])
        return back
    if case["op"] == "linear":
        return st["x"].double() @ _values64(st["q"], st["s"]).t()
    x = st["x"].double()
    y = _swiglu64(x, _values64(*st["sh_gate_up"]), _values64(*st["sh_down"]))
    ids, w = st["ids"].long(), st["w"].double()
    for e in sorted(set(ids.flatten().tolist()) - {case["E"]}):
        share = (w * (ids == e)).sum(1)
        rows = (ids == e).any(1).nonzero().flatten()
        o = _swiglu64(x[rows], _values64(st["gate_up"][0][e], st["gate_up"][1][e]),
                      _values64(st["down"][0][e], st["down"][1][e]))
        y[rows] += share[rows, None] * o
    return y
