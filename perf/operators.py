"""The step's input operators, as cases to measure: hidden states to e4m3 codes
with a scale per 128 (quant), projections on those codes (linear), and the row,
page and slot arrays of a batch built from request lengths (plan).

`own` False runs plain torch; True runs the library's calls.
"""
import math

import torch

own = False

HIDDEN = 7168            # model width of the hidden states
LATENT = 2048            # a query latent
HEADS_IDX, HEADS_ATT = 32, 64
E4M3_MAX = 448.0
AMAX_FLOOR = E4M3_MAX * 2.0 ** -120
WINDOW = 128
PAGE = 64
THETA = 10000.0
EPS = 1e-6


def listed():
    return [
        # the hidden states of a batch-8 decode step, normalised and quantised before the projections
        {"name": "quant_norm_decode", "op": "quant", "T": 8, "K": HIDDEN, "norm": True, "block_rows": 1},
        # the hidden states of a 4,096-token prefill chunk
        {"name": "quant_prefill", "op": "quant", "T": 4096, "K": HIDDEN, "norm": False, "block_rows": 1},
        # the weights of the attention query projection, quantised when they are loaded
        {"name": "quant_weights", "op": "quant", "T": HEADS_ATT * 512, "K": LATENT, "norm": False, "block_rows": 128},
        # decode, batch 8: the main-KV input C (hidden 7168 -> 512)
        {"name": "kv_decode", "op": "linear", "T": 8, "K": HIDDEN, "N": 512, "out": "bf16", "head": 0},
        # decode, batch 8: the indexer queries, 32 heads x 128, as codes and scales with RoPE
        {"name": "index_q_decode", "op": "linear", "T": 8, "K": LATENT, "N": HEADS_IDX * 128, "out": "fp8", "head": 128},
        # decode, batch 8: the attention queries, 64 heads x 512 with RoPE
        {"name": "attn_q_decode", "op": "linear", "T": 8, "K": LATENT, "N": HEADS_ATT * 512, "out": "bf16", "head": 512},
        # an odd batch between decode and prefill, odd widths, fp32 out
        {"name": "odd_fp32", "op": "linear", "T": 333, "K": 1360, "N": 1001, "out": "fp32", "head": 0},
        # the three projections for a 4,096-token prefill chunk
        {"name": "kv_prefill", "op": "linear", "T": 4096, "K": HIDDEN, "N": 512, "out": "bf16", "head": 0},
        {"name": "index_q_prefill", "op": "linear", "T": 4096, "K": LATENT, "N": HEADS_IDX * 128, "out": "fp8", "head": 128},
        {"name": "attn_q_prefill", "op": "linear", "T": 4096, "K": LATENT, "N": HEADS_ATT * 512, "out": "bf16", "head": 512},
        # a decode step of 8 sequences of up to 1M tokens: one new token each
        {"name": "plan_decode", "op": "plan", "B": 8, "max_ctx": 1 << 20, "max_new": 1, "ratio_m": 1, "max_rows": 8},
        # a mixed step: prompts' chunks and single tokens of 256 sequences, entries of two tokens
        {"name": "plan_mixed", "op": "plan", "B": 256, "max_ctx": 1 << 17, "max_new": 128, "ratio_m": 2, "max_rows": 16384},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "plan"])
    if op == "quant":
        rows = rng.choice([1, 1, 128])
        return {"op": op, "T": _log(rng, 1, 8192), "K": 16 * _log(rng, 1, 512), "norm": rows == 1 and rng.random() < 0.5,
                "block_rows": rows}
    if op == "linear":
        T, K = _log(rng, 1, 4096), 16 * _log(rng, 4, 512)
        out = rng.choice(["fp32", "bf16", "fp8"])
        top = min(32768, int(4096 * 2048 * 32768 / (T * K)))
        N = _log(rng, 1, top) if out != "fp8" else 128 * _log(rng, 1, max(1, top // 128))
        head = 0
        if N >= 128 and rng.random() < 0.5:
            head = rng.choice([128, 256, 512])
            N = max(head, N // head * head)
        return {"op": op, "T": T, "K": K, "N": N, "out": out, "head": head}
    B = _log(rng, 1, 1024)
    new = rng.choice([1, 1, 2, 17, 300])
    return {"op": op, "B": B, "max_ctx": _log(rng, 1, 1 << 17), "max_new": new, "ratio_m": rng.choice([1, 2]),
            "max_rows": max(1, min(B * new, 16384))}


def _blocks(n):
    return (n + 127) // 128


def _pad_blocks(y):
    """[T,K] -> [T, blocks, 128], zeros behind the last column."""
    T, K = y.shape
    nb = _blocks(K)
    out = y.new_zeros(T, nb * 128)
    out[:, :K] = y
    return out.view(T, nb, 128)


def _e4m3(y):
    """Nearest e4m3 value (ties to even), saturating."""
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _quant_rows(y):
    """Codes [T,K] and scales [T,blocks] of fp32 rows."""
    T, K = y.shape
    g = _pad_blocks(y)
    amax = g.abs().amax(dim=-1)
    top = amax.clamp(min=AMAX_FLOOR)
    codes = _e4m3(g * (E4M3_MAX / top)[..., None])
    scale = torch.where(amax > 0, top / E4M3_MAX, torch.ones_like(amax))
    return codes.view(torch.uint8).reshape(T, -1)[:, :K].contiguous().view(torch.float8_e4m3fn), scale


def _quant_tiles(y):
    """Codes [N,K] and scales [blocks,blocks] of 128 x 128 tiles."""
    N, K = y.shape
    rb = _blocks(N)
    full = y.new_zeros(rb * 128, _blocks(K) * 128)
    full[:N, :K] = y
    g = full.view(rb, 128, -1, 128)
    amax = g.abs().amax(dim=(1, 3))
    top = amax.clamp(min=AMAX_FLOOR)
    codes = _e4m3(g * (E4M3_MAX / top)[:, None, :, None])
    scale = torch.where(amax > 0, top / E4M3_MAX, torch.ones_like(amax))
    codes = codes.view(torch.uint8).reshape(rb * 128, -1)[:N, :K].contiguous()
    return codes.view(torch.float8_e4m3fn), scale


def _hidden(T, K, g, dev):
    """Hidden states: N(0,1) with a few channels an order of magnitude larger."""
    x = torch.randn(T, K, generator=g, device=dev)
    loud = torch.rand(K, generator=g, device=dev) < 0.01
    return torch.where(loud, 12.0 * x, x).to(torch.bfloat16)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "quant":
        T, K = case["T"], case["K"]
        rows = case["block_rows"]
        s["x"] = _hidden(T, K, g, dev) if rows == 1 else (
            torch.randn(T, K, generator=g, device=dev) / math.sqrt(K)).to(torch.bfloat16)
        s["gamma"] = 1.0 + 0.1 * torch.randn(K, generator=g, device=dev) if case["norm"] else None
        s["codes"] = torch.empty(T, K, dtype=torch.uint8, device=dev)
        s["scale"] = torch.empty(T if rows == 1 else _blocks(T), _blocks(K), device=dev)
        return s
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        s["x"], s["x_scale"] = _quant_rows(_hidden(T, K, g, dev).float())
        s["w"], s["w_scale"] = _quant_tiles(torch.randn(N, K, generator=g, device=dev) / math.sqrt(K))
        s["pos"] = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32) if case["head"] else None
        kind = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}[case["out"]]
        s["out"] = torch.empty(T, N, dtype=kind, device=dev)
        s["out_scale"] = torch.empty(T, N // 128, device=dev) if case["out"] == "fp8" else None
        torch.cuda.synchronize()  # run() passes w_ready: the weights were written well before the first call
        return s
    B, m, cap = case["B"], case["ratio_m"], case["max_rows"]
    ctx = torch.randint(0, case["max_ctx"] + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    new = torch.randint(1, case["max_new"] + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    if case["max_new"] > 1:  # single tokens and paused sequences between the chunks
        kind = torch.randint(0, 4, (B,), generator=g, device=dev)
        new = torch.where(kind == 0, torch.ones_like(new), torch.where(kind == 1, torch.zeros_like(new), new))
    before = torch.cumsum(new, 0, dtype=torch.int32) - new
    new = torch.minimum(new, (cap - before).clamp(min=0))
    stride = (case["max_ctx"] + case["max_new"]) // m // PAGE + 1
    old = (ctx // m + PAGE - 1) // PAGE
    owned = B * stride
    perm = torch.randperm(owned + B * (case["max_new"] // PAGE + 2), generator=g, device=dev, dtype=torch.int32)
    col = torch.arange(stride, device=dev)[None, :]
    s["ctx"], s["new"] = ctx, new
    s["page_table"] = torch.where(col < old[:, None], perm[:owned].view(B, stride), -1).to(torch.int32).contiguous()
    s["free"] = perm[owned:].contiguous()
    s["head"] = torch.full((1,), 3 % max(1, B), dtype=torch.int32, device=dev)
    ring = WINDOW + case["max_new"] - 1
    s["ring"] = ring
    s["ring_id"] = torch.randperm(B, generator=g, device=dev, dtype=torch.int32)

    def buf(*shape):
        return torch.full(shape, -7, dtype=torch.int32, device=dev)

    s["o"] = {"row_start": buf(B + 1), "row_seq": buf(cap), "row_pos": buf(cap), "n_visible": buf(B),
              "entry_start": buf(B + 1), "entry_slot": buf(cap), "entry_pos": buf(cap), "entry_row": buf(cap),
              "swa_new": buf(cap), "swa_slot": buf(cap, WINDOW), "free_head_out": buf(1)}
    return s


def _rope_plain(y, pos, head):
    """Turns the last 64 columns of every head, in interleaved pairs, by pos * theta^(-2p/64)."""
    T, N = y.shape
    rate = THETA ** (-torch.arange(32, dtype=torch.float64, device=y.device) / 32)
    ang = torch.remainder(pos.double()[:, None] * rate, 2 * math.pi)
    sn, cs = torch.sin(ang).float()[:, None, :], torch.cos(ang).float()[:, None, :]
    z = y.reshape(T, N // head, head).clone()
    a, b = z[..., head - 64::2].clone(), z[..., head - 63::2].clone()
    z[..., head - 64::2] = a * cs - b * sn
    z[..., head - 63::2] = a * sn + b * cs
    return z.reshape(T, N)


def _plain_quant(s):
    y = s["x"].float()
    if s["gamma"] is not None:
        y = y / torch.sqrt((y * y).mean(dim=-1, keepdim=True) + EPS) * s["gamma"]
    codes, scale = _quant_rows(y) if s["case"]["block_rows"] == 1 else _quant_tiles(y)
    return {"codes": codes, "scale": scale}


def _plain_linear(s):
    c = s["case"]
    K, N = c["K"], c["N"]
    xs = s["x_scale"].repeat_interleave(128, dim=1)[:, :K]
    ws = s["w_scale"].repeat_interleave(128, dim=0)[:N].repeat_interleave(128, dim=1)[:, :K]
    y = (s["x"].float() * xs) @ (s["w"].float() * ws).t()
    if c["head"]:
        y = _rope_plain(y, s["pos"], c["head"])
    if c["out"] == "fp8":
        codes, scale = _quant_rows(y)
        return {"out": codes, "scale": scale}
    return {"out": y if c["out"] == "fp32" else y.to(torch.bfloat16)}


def _plain_plan(s):
    c, o = s["case"], s["o"]
    B, m, cap, ring = c["B"], c["ratio_m"], c["max_rows"], s["ring"]
    dev = s["ctx"].device
    ctx, new = s["ctx"].long(), s["new"].long()
    zero = torch.zeros(1, dtype=torch.long, device=dev)
    row_start = torch.cat([zero, torch.cumsum(new, 0)])
    e0, e1 = ctx // m, (ctx + new) // m
    entry_start = torch.cat([zero, torch.cumsum(e1 - e0, 0)])
    p0, p1 = (e0 + PAGE - 1) // PAGE, (e1 + PAGE - 1) // PAGE
    page_start = torch.cat([zero, torch.cumsum(p1 - p0, 0)])
    head = s["head"].long()
    col = torch.arange(s["page_table"].shape[1], device=dev)[None, :]
    fresh = (col >= p0[:, None]) & (col < p1[:, None])
    take = (head + page_start[:-1])[:, None] + col - p0[:, None]
    table = torch.where(fresh, s["free"].long()[take.clamp(0, s["free"].numel() - 1)], s["page_table"].long())
    t = torch.arange(cap, device=dev)
    live = t < row_start[-1]
    seq = torch.searchsorted(row_start[1:], t, right=True).clamp(max=B - 1)
    pos = ctx[seq] + t - row_start[seq]
    base = s["ring_id"].long()[seq] * ring
    win = pos[:, None] - (WINDOW - 1) + torch.arange(WINDOW, device=dev)[None, :]
    slots = torch.where(win >= 0, base[:, None] + win % ring, -1)
    has = t < entry_start[-1]
    es = torch.searchsorted(entry_start[1:], t, right=True).clamp(max=B - 1)
    e = e0[es] + t - entry_start[es]
    e_slot = table[es, (e // PAGE).clamp(0, table.shape[1] - 1)] * PAGE + e % PAGE
    e_row = row_start[es] + (e + 1) * m - 1 - ctx[es]

    def keep(mask, value, old):
        return torch.where(mask, value, old.long()).to(torch.int32)

    return {"page_table": table.to(torch.int32), "row_start": row_start.to(torch.int32),
            "row_seq": keep(live, seq, o["row_seq"]), "row_pos": keep(live, pos, o["row_pos"]),
            "n_visible": e1.to(torch.int32), "entry_start": entry_start.to(torch.int32),
            "entry_slot": keep(has, e_slot, o["entry_slot"]), "entry_pos": keep(has, e * m, o["entry_pos"]),
            "entry_row": keep(has, e_row, o["entry_row"]), "swa_new": keep(live, base + pos % ring, o["swa_new"]),
            "swa_slot": keep(live[:, None], slots, o["swa_slot"]), "free_head_out": (head + page_start[-1:]).to(torch.int32)}


def run(state):
    case = state["case"]
    if not own:
        return {"quant": _plain_quant, "linear": _plain_linear, "plan": _plain_plan}[case["op"]](state)
    from serving_lightning_indexer_gb300 import csa2
    if case["op"] == "quant":
        csa2.quant_fp8(state["x"], state["codes"], state["scale"], gamma=state["gamma"], eps=EPS,
                       block_rows=case["block_rows"])
        return {"codes": state["codes"].view(torch.float8_e4m3fn), "scale": state["scale"]}
    if case["op"] == "linear":
        csa2.fp8_linear(state["x"].view(torch.uint8), state["x_scale"], state["w"].view(torch.uint8), state["w_scale"],
                        state["out"], out_scale=state["out_scale"], row_pos=state["pos"], rope_head=case["head"],
                        rope_theta=THETA, w_ready=True)
        if case["out"] == "fp8":
            return {"out": state["out"].view(torch.float8_e4m3fn), "scale": state["out_scale"]}
        return {"out": state["out"]}
    o = state["o"]
    csa2.batch_plan(state["ctx"], state["new"], case["ratio_m"], page_table=state["page_table"], free_pages=state["free"],
                    free_head=state["head"], swa_ring=state["ring"], ring_id=state["ring_id"], **o)
    return {"page_table": state["page_table"], **o}


def work(case):
    if case["op"] == "quant":
        T, K = case["T"], case["K"]
        scales = (T if case["block_rows"] == 1 else _blocks(T)) * _blocks(K)
        return {"bytes": 3 * T * K + 4 * scales + (4 * K if case["norm"] else 0), "flops": (6 if case["norm"] else 2) * T * K}
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        size = {"fp32": 4, "bf16": 2, "fp8": 1}[case["out"]]
        scales = T * _blocks(K) + _blocks(N) * _blocks(K) + (T * N // 128 if case["out"] == "fp8" else 0)
        return {"bytes": T * K + N * K + size * T * N + 4 * scales, "flops": 2 * T * N * K}
    B, new, m = case["B"], case["max_new"], case["ratio_m"]
    rows = min(case["max_rows"], B if new == 1 else B * (1 + new) // 4)
    return {"bytes": 4 * B * 7 + rows * (12 + 4 * WINDOW) + rows // m * 12, "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] == "quant":
        v = s["x"].double()
        if s["gamma"] is not None:
            v = v * torch.rsqrt(v.square().sum(-1, keepdim=True) / v.shape[1] + EPS) * s["gamma"].double()
        return dict(zip(("codes", "scale"), _exact_codes(v, case["block_rows"])))
    rows = torch.arange(case["N"], device=s["w"].device) // 128
    cols = torch.arange(case["K"], device=s["w"].device) // 128
    a = s["x"].double() * s["x_scale"].double()[:, cols]
    b = s["w"].double() * s["w_scale"].double()[rows][:, cols]
    v = torch.einsum("tk,nk->tn", a, b)
    if case["head"]:
        D = case["head"]
        power = torch.arange(0, -64, -2, dtype=torch.float64, device=v.device) / 64
        turn = torch.outer(s["pos"].double(), torch.exp(power * math.log(THETA)))
        pairs = torch.view_as_complex(v.view(len(v), -1, D)[:, :, D - 64:].reshape(len(v), -1, 32, 2).contiguous())
        pairs = pairs * torch.polar(torch.ones_like(turn), turn)[:, None, :]
        v.view(len(v), -1, D)[:, :, D - 64:] = torch.view_as_real(pairs).reshape(len(v), -1, 64)
    if case["out"] == "fp8":
        return dict(zip(("out", "scale"), _exact_codes(v, 1)))
    return {"out": v}


def _exact_codes(v, rows):
    """Code values and scales of 64-bit numbers, block by block of `rows` x 128."""
    T, K = v.shape
    r = torch.arange(T, device=v.device) // rows
    nb = _blocks(K)
    wide = torch.nn.functional.pad(v.abs(), (0, nb * 128 - K)).view(T, nb, 128).amax(-1)
    top = torch.zeros(int(r[-1]) + 1, nb, dtype=torch.float64, device=v.device)
    top = top.scatter_reduce(0, r[:, None].expand(T, nb), wide, "amax")
    use = top.clamp(min=AMAX_FLOOR)
    c = torch.arange(K, device=v.device) // 128
    codes = (v * E4M3_MAX / use[r][:, c]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double()
    return codes, torch.where(top > 0, use / E4M3_MAX, torch.ones_like(top))
