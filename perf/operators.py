"""Cases for the operators of the 4-bit KV cache: quantising new rows as they are
written and reading them back, full-attention decode, the Atop-N step and its
threshold refresh over such a cache.

The cache: row t of head h of sequence b holds d values as d/2 bytes of e2m1
codes (value 2i in the low half of byte i) and d/16 e4m3 scales, one for 16
values; an optional fp32 scale g per head. A value is e2m1 * e4m3 * g.
"""
import math

import torch

own = False

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]

# (h_q, h_k, h_v, d): Llama-3.2-1B and Qwen2.5-1.5B attention, each with its own
# GQA heads and with SAGA's (fewer key than value heads), and the small shapes of the tests
HEADS = {"llama_gqa": (32, 8, 8, 64), "llama_saga": (32, 2, 8, 64), "qwen_gqa": (12, 2, 2, 128),
         "qwen_saga": (12, 1, 4, 128), "small": (16, 2, 4, 64), "tiny": (4, 1, 2, 64),
         "mha": (8, 8, 8, 64), "one_key_head": (16, 1, 1, 128)}


def case(name, op, heads, B, L, dtype="bf16", ragged=False, gscale=False, N=0, T=0):
    return {"name": name, "op": op, "heads": heads, "B": B, "L": L, "dtype": dtype,
            "ragged": ragged, "gscale": gscale, "N": N, "T": T}


def listed():
    return [
        # one decoded token of one sequence joins the cache: latency only
        case("append_token", "append", "qwen_saga", 1, 5001, T=1),
        # ragged chunks of a small fp32 model, a sequence without new tokens among them
        case("append_ragged_f32", "append", "tiny", 3, 1024, dtype="f32", ragged=True, T=37),
        # the prompts of a batch are written and read back for their own attention
        case("append_prompt", "append", "llama_saga", 8, 1000, ragged=True, gscale=True, T=8192),
        # a window of one sequence is read back in fp32
        case("read_window_f32", "read", "small", 2, 1777, dtype="f32", ragged=True, gscale=True, T=333),
        # a whole batch of caches is read back, for a path that wants bf16 rows
        case("read_cache", "read", "llama_saga", 8, 32768, T=32768),
        # the smallest fp32 decode batch, with an empty sequence
        case("dense_tiny_f32", "dense", "tiny", 3, 1024, dtype="f32", ragged=True),
        # ragged serving batch, SAGA heads, long value rows
        case("dense_saga_ragged", "dense", "qwen_saga", 16, 65536, ragged=True, gscale=True),
        # one layer of the 128K batch-8 stack with its GQA heads
        case("dense_gqa_128k", "dense", "llama_gqa", 8, 131072),
        # one layer at batch 1 and 128K, Atop-N
        case("step_b1_128k", "step", "qwen_saga", 1, 131072, N=2048),
        # one layer of the 128K batch-8 stack, Atop-N
        case("step_b8_128k", "step", "llama_saga", 8, 131072, gscale=True, N=2048),
        # the smallest refresh
        case("refresh_tiny_f32", "refresh", "tiny", 1, 1024, dtype="f32", N=64),
        # a ragged batch that refreshes
        case("refresh_ragged", "refresh", "llama_saga", 16, 131072, ragged=True, N=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "dense", "dense", "step", "refresh"])
    heads = rng.choice(sorted(HEADS))
    h_q, h_k, h_v, d = HEADS[heads]
    B = _log(rng, 1, 16)
    row = (h_k + h_v) * d
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    c = {"op": op, "heads": heads, "B": B, "dtype": dtype, "ragged": rng.random() < 0.5,
         "gscale": rng.random() < 0.5, "N": 0, "T": 0}
    if op in ("append", "read"):
        most = 4e4 if op == "append" and dtype == "f32" else 4e7
        c["T"] = _log(rng, 1, max(2, min(16384, most / (row * B))))
        c["L"] = _log(rng, 1, 4096) + (c["T"] if op == "read" else 0)
        # fp32 rows without a head scale: x / t then lies on a rounding border in 32 bits where it does in 64
        c["gscale"] = c["gscale"] and (op == "read" or dtype == "bf16")
    else:
        c["L"] = _log(rng, 1, min(131072, 1e9 / (row * B)))
        if op != "dense":
            c["N"] = _log(rng, 1, max(2, c["L"] // 8))
    return c


# ---- the cache's arithmetic in plain torch, fp32 -------------------------------
def quantise(x, g):
    """fp32 [..., d] -> codes uint8 [..., d/2], scales uint8 [..., d/16]; g fp32, broadcast over [..., d/16]."""
    xb = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    s = (xb.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    t = (s.float() * g).unsqueeze(-1)
    y = torch.where(t > 0, xb.abs() / t, torch.zeros((), device=x.device))
    c = torch.zeros_like(y, dtype=torch.uint8)
    for at, closed in ((.25, 0), (.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5., 0)):
        c += (y >= at) if closed else (y > at)
    c += torch.signbit(xb) * 8
    c = c.reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return c[..., 0] + c[..., 1] * 16, s.view(torch.uint8)


def values(codes, scales, g):
    """The fp32 values of codes [..., d/2] and scales [..., d/16]; g broadcast over [..., d/16]."""
    tab = torch.tensor(E2M1 + [-v for v in E2M1], device=codes.device)
    v = torch.stack((tab[(codes & 15).int()], tab[(codes >> 4).int()]), -1)
    v = v.reshape(*codes.shape[:-1], scales.shape[-1], 16)
    v = v * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1) * g.unsqueeze(-1)
    return v.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _scale(g, heads, device):
    """g [heads] (or none) as [heads][1][1], for caches [B][heads][cap][d/16]."""
    return (torch.ones(heads, device=device) if g is None else g).view(heads, 1, 1)


def _plant(gen, x):
    """1% of the rows point one way, with three times the length: the scores' upper tail."""
    u = torch.randn(x.shape[-1], device=x.device, generator=gen)
    pick = torch.rand(x.shape[:-1], device=x.device, generator=gen) < 0.01
    return torch.where(pick.unsqueeze(-1), 3 * u / u.norm() + 0.5 * x, x)


def prepare(case, seed):
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    B, L, T, op = case["B"], case["L"], case["T"], case["op"]
    gen = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    cap = (L + (T if op == "append" else 0) + 3) // 4 * 4
    lens = torch.full((B,), L, device="cuda", dtype=torch.int32)
    if case["ragged"]:
        lens = (torch.rand(B, device="cuda", generator=gen) * L).to(torch.int32) + 1
        lens[0] = L
        if B > 2 and op != "read":
            lens[B - 1] = 0
    s = {"case": case, "cap": cap, "l": lens, "dt": dt, "gk": None, "gv": None}
    if case["gscale"]:
        s["gk"] = torch.rand(h_k, device="cuda", generator=gen) * 0.1 + 0.01
        s["gv"] = torch.rand(h_v, device="cuda", generator=gen) * 0.1 + 0.01
    gk, gv = _scale(s["gk"], h_k, "cuda"), _scale(s["gv"], h_v, "cuda")
    if op == "append":
        s["kc"], s["ks"], s["vc"], s["vs"] = (torch.zeros(B, h, cap, d // w, dtype=torch.uint8, device="cuda")
                                              for h, w in ((h_k, 2), (h_k, 16), (h_v, 2), (h_v, 16)))
        s["k_new"], s["v_new"] = _plant(gen, rand(B, T, h_k, d)).to(dt), rand(B, T, h_v, d).to(dt)
        s["n_new"] = None
        if case["ragged"]:
            s["n_new"] = (torch.rand(B, device="cuda", generator=gen) * (T + 1)).to(torch.int32)
            s["n_new"][0] = T
            if B > 1:
                s["n_new"][1] = 0
        s["l0"] = lens.clone()
    else:
        s["kc"], s["ks"] = quantise(_plant(gen, rand(B, h_k, cap, d)), gk)
        s["vc"], s["vs"] = quantise(rand(B, h_v, cap, d), gv)
    if op == "read":
        s["start"] = (lens - T).clamp(min=0) if case["ragged"] else None
    if op in ("append", "read"):
        s["K"] = torch.zeros(B, h_k, T, d, dtype=dt, device="cuda")
        s["V"] = torch.zeros(B, h_v, T, d, dtype=dt, device="cuda")
    else:
        s["q"] = rand(B, h_q, d).to(dt)
        s["out"] = torch.zeros(B, h_q, d, device="cuda")
        s["tau"] = torch.zeros(B, h_q, device="cuda")
    if op == "step":
        # a stored threshold that keeps about N: it lies between two scores, in the widest gap near
        # the N-th, so that no rounding of a score decides what is kept
        A = _scores(s)
        lo, hi = max(0, min(case["N"], L - 1) - 64), min(L, case["N"] + 64)
        top = A.topk(hi, -1).values[..., lo:]
        gap = torch.nan_to_num(top[..., :-1] - top[..., 1:], nan=-1.0, posinf=-1.0)
        if gap.shape[-1]:
            at = gap.argmax(-1, keepdim=True)
            mid = (top.gather(-1, at) + top.gather(-1, at + 1)) / 2
            s["tau"] = torch.where(gap.gather(-1, at) > 0, mid, torch.full_like(mid, -math.inf)).squeeze(-1).contiguous()
        else:
            s["tau"].fill_(-math.inf)
        s["count"] = torch.zeros(B, h_q, dtype=torch.int32, device="cuda")
    if own:
        import sparse_decode_attention_step_b200 as saga
        s["shp"] = saga.shape(B, h_q, h_k, h_v, d, saga.SAGA_F32 if dt == torch.float32 else saga.SAGA_BF16, cap,
                              cap if op in ("append", "read") else L)
        s["cache"] = saga.Q4Cache(s["shp"], s["kc"], s["ks"], s["vc"], s["vs"], s["gk"], s["gv"])
        s["ws"] = saga.Q4Workspace(s["shp"])
    return s


# ---- one pass ------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_decode_attention_step_b200 as saga
    c, shp, cache, ws = s["case"], s["shp"], s["cache"], s["ws"]
    if c["op"] == "append":
        s["l"].copy_(s["l0"])
        saga.q4_append_kv(shp, cache, s["k_new"], s["v_new"], c["T"], s["l"], ws, n_new=s["n_new"])
        saga.q4_read_kv(shp, cache, c["T"], s["l"], s["K"], s["V"], ws, start=s["l0"])
        return {"K": s["K"], "V": s["V"], "l": s["l"]}
    if c["op"] == "read":
        saga.q4_read_kv(shp, cache, c["T"], s["l"], s["K"], s["V"], ws, start=s["start"])
        return {"K": s["K"], "V": s["V"]}
    if c["op"] == "dense":
        saga.q4_dense_decode(shp, cache, s["q"], s["l"], s["out"], ws)
        return {"out": s["out"]}
    if c["op"] == "step":
        saga.q4_decode_step(shp, cache, s["q"], s["l"], s["tau"], s["out"], ws, sel_count=s["count"])
        return {"out": s["out"], "count": s["count"]}
    saga.q4_refresh_threshold(shp, cache, s["q"], s["l"], c["N"], s["tau"], ws)
    return {"tau": s["tau"]}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "append":
        s["l"].copy_(s["l0"])
        _append(s)
        return dict(_window(s, s["l0"]), l=s["l"])
    if c["op"] == "read":
        return _window(s, s["start"])
    A = _scores(s)
    if c["op"] == "dense":
        return {"out": _attend(s, A, A > -math.inf)}
    if c["op"] == "step":
        keep = (A >= s["tau"].unsqueeze(-1)) & (A > -math.inf)
        return {"out": _attend(s, A, keep), "count": keep.sum(-1, dtype=torch.int32)}
    n = min(c["N"], A.shape[-1])
    tau = A.topk(n, -1).values[..., -1]
    return {"tau": torch.where((s["l"] > c["N"]).unsqueeze(-1), tau, torch.full_like(tau, -math.inf))}


def _append(s):
    h_q, h_k, h_v, d = HEADS[s["case"]["heads"]]
    T, B = s["case"]["T"], s["case"]["B"]
    n = torch.full_like(s["l"], T) if s["n_new"] is None else s["n_new"]
    at = s["l"].long().unsqueeze(1) + torch.arange(T, device="cuda")
    b = torch.arange(B, device="cuda").unsqueeze(1)
    new = (torch.arange(T, device="cuda") < n.unsqueeze(1)).view(B, T, 1, 1)
    for x, g, h, codes, scales in ((s["k_new"], s["gk"], h_k, s["kc"], s["ks"]), (s["v_new"], s["gv"], h_v, s["vc"], s["vs"])):
        qc, qs = quantise(x.float(), _scale(g, h, "cuda").squeeze(-1))
        codes[b, :, at] = torch.where(new, qc, codes[b, :, at])
        scales[b, :, at] = torch.where(new, qs, scales[b, :, at])
    s["l"] += n


def _window(s, start):
    h_q, h_k, h_v, d = HEADS[s["case"]["heads"]]
    T, B = s["case"]["T"], s["case"]["B"]
    at = torch.arange(T, device="cuda").expand(B, T) if start is None else start.long().unsqueeze(1) + torch.arange(T, device="cuda")
    b, t = torch.arange(B, device="cuda").unsqueeze(1), at.clamp(max=s["cap"] - 1)
    live = (at < s["l"].unsqueeze(1)).view(B, T, 1, 1)
    both = []
    for g, h, codes, scales in ((s["gk"], h_k, s["kc"], s["ks"]), (s["gv"], h_v, s["vc"], s["vs"])):
        v = values(codes[b, :, t], scales[b, :, t], _scale(g, h, "cuda").squeeze(-1))
        both.append(torch.where(live, v, torch.zeros((), device="cuda")).transpose(1, 2).to(s["dt"]).contiguous())
    return {"K": both[0], "V": both[1]}


def _scores(s):
    """fp32 [B][h_q][L], -inf behind each sequence's end."""
    h_q, h_k, h_v, d = HEADS[s["case"]["heads"]]
    B, L = s["case"]["B"], s["case"]["L"]
    K = values(s["kc"][:, :, :L], s["ks"][:, :, :L], _scale(s["gk"], h_k, "cuda"))
    A = (s["q"].float().view(B, h_k, h_q // h_k, d) @ K.transpose(2, 3)).view(B, h_q, L) / math.sqrt(d)
    return A.masked_fill(torch.arange(L, device="cuda") >= s["l"].view(B, 1, 1), -math.inf)


def _attend(s, A, keep):
    h_q, h_k, h_v, d = HEADS[s["case"]["heads"]]
    B, L = s["case"]["B"], s["case"]["L"]
    V = values(s["vc"][:, :, :L], s["vs"][:, :, :L], _scale(s["gv"], h_v, "cuda"))
    A = A.masked_fill(~keep, -math.inf)
    p = torch.exp(A - A.amax(-1, keepdim=True).clamp(min=-3e38))
    o = (p.view(B, h_v, h_q // h_v, L) @ V).view(B, h_q, d)
    return o / p.sum(-1, keepdim=True).clamp(min=1e-30)


# ---- what a pass cannot do without ---------------------------------------------
def work(case):
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    B, L, op = case["B"], case["L"], case["op"]
    esz = 4 if case["dtype"] == "f32" else 2
    row = d * 9 / 16                                   # codes and scales of one row
    # ragged lengths: uniform over the range on average, the first sequence at full length
    mean = (L + (B - 1) * L / 2) / B if case["ragged"] else L
    if op == "append":
        n = B * case["T"] * (0.5 if case["ragged"] and B > 1 else 1.0) * (h_k + h_v)
        return {"bytes": n * (2 * d * esz + 2 * row), "flops": n * d * 8}
    if op == "read":
        n = B * min(case["T"], mean) * (h_k + h_v)
        return {"bytes": n * (d * esz + row), "flops": n * d * 2}
    ends = B * h_q * d * (esz + 4)
    if op == "dense":
        return {"bytes": B * mean * (h_k + h_v) * row + ends, "flops": 4.0 * B * mean * h_q * d}
    if op == "step":
        kept = B * h_v * min(mean, case["N"] * h_q / h_v)   # each kept row at most once per query head
        return {"bytes": B * mean * h_k * row + kept * row + ends,
                "flops": 2.0 * B * mean * h_q * d + 2.0 * B * h_q * min(mean, case["N"]) * d}
    return {"bytes": B * mean * h_k * row + B * h_q * (d * esz + 4), "flops": 2.0 * B * mean * h_q * d}


# ---- the definitions in 64 bits --------------------------------------------------
def _e2m1(code):
    """(-1)^s * m/2 for an exponent of 0, else (-1)^s * 2^(e-1) * (1 + m/2)."""
    m, e, sign = (code & 1).double(), ((code >> 1) & 3).double(), 1 - 2 * (code >> 3).double()
    return sign * torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2)


def _e4m3(byte):
    m, e = (byte & 7).double(), ((byte >> 3) & 15).double()
    return torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), torch.exp2(torch.full_like(e, -9.0)) * m)


def _held(codes, scales, g):
    """float64 values of one sequence's cache [heads][n][d]."""
    v = torch.stack((_e2m1(codes & 15), _e2m1(codes >> 4)), -1).flatten(-2)
    v = v * _e4m3(scales).repeat_interleave(16, -1)
    return v if g is None else v * g.double().view(-1, 1, 1)


def _stored(x, g):
    """float64 rows [n][heads][d] as the cache stores them, from the quantiser's definition."""
    g = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if g is None else g.double()
    b = x.double().unflatten(-1, (-1, 16))
    r = (b.abs().amax(-1) / (6 * g.view(1, -1, 1))).clamp(max=448)
    step = torch.exp2(torch.floor(torch.log2(r.clamp(min=2.0 ** -30))).clamp(min=-6) - 3)
    t = (torch.round(r / step) * step * g.view(1, -1, 1)).unsqueeze(-1)
    y = (b / t.clamp(min=1e-300)).abs().clamp(max=6)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
    return (torch.sign(b) * torch.round(y / step) * step * t).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    B, T, op = case["B"], case["T"], case["op"]
    lens = s["l"].tolist()
    if op in ("append", "read"):
        K = torch.zeros(B, h_k, T, d, dtype=torch.float64, device="cuda")
        V = torch.zeros(B, h_v, T, d, dtype=torch.float64, device="cuda")
        for b in range(B):
            if op == "append":
                n = T if s["n_new"] is None else int(s["n_new"][b])
                K[b, :, :n] = _stored(s["k_new"][b, :n], s["gk"]).transpose(0, 1)
                V[b, :, :n] = _stored(s["v_new"][b, :n], s["gv"]).transpose(0, 1)
                lens[b] += n
            else:
                a = 0 if s["start"] is None else int(s["start"][b])
                e = max(a, min(a + T, lens[b]))
                K[b, :, :e - a] = _held(s["kc"][b, :, a:e], s["ks"][b, :, a:e], s["gk"])
                V[b, :, :e - a] = _held(s["vc"][b, :, a:e], s["vs"][b, :, a:e], s["gv"])
        both = {"K": K, "V": V}
        return dict(both, l=torch.tensor(lens, dtype=torch.int32)) if op == "append" else both
    out = torch.zeros(B, h_q, d, dtype=torch.float64, device="cuda")
    tau = torch.full((B, h_q), -math.inf, dtype=torch.float64, device="cuda")
    count = torch.zeros(B, h_q, dtype=torch.int32, device="cuda")
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        K = _held(s["kc"][b, :, :n], s["ks"][b, :, :n], s["gk"])
        A = torch.matmul(s["q"][b].double().view(h_k, h_q // h_k, d), K.mT).reshape(h_q, n) / d ** 0.5
        if op == "refresh":
            if n > case["N"]:
                tau[b] = A.sort(-1, descending=True).values[:, case["N"] - 1]
            continue
        if op == "step":
            A = torch.where(A >= s["tau"][b].double().unsqueeze(-1), A, -math.inf)
            count[b] = (A > -math.inf).sum(-1)
        V = _held(s["vc"][b, :, :n], s["vs"][b, :, :n], s["gv"])
        P = torch.nan_to_num(torch.softmax(A, -1), nan=0.0)
        out[b] = torch.matmul(P.view(h_v, h_q // h_v, n), V).reshape(h_q, d)
    if op == "refresh":
        return {"tau": tau}
    return {"out": out, "count": count} if op == "step" else {"out": out}
