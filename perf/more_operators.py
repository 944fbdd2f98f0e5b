"""Operators around the step's layers, as cases to measure: the residual's addition
with RMSNorm and e4m3 codes (norm), projections on those codes with low-rank adapters
of many requests (lora), and log probabilities, entropy and top alternatives of
rows of logits (logprobs).

`own` False runs plain torch; True runs the library's calls.
"""
import math

import torch

own = False

HIDDEN = 7168            # model width of the hidden states
LATENT = 2048            # a query latent
HEADS_IDX, HEADS_ATT = 32, 64
VOCAB = 1 << 17
E4M3_MAX = 448.0
AMAX_FLOOR = E4M3_MAX * 2.0 ** -120
THETA = 10000.0
EPS = 1e-6


def listed():
    return [
        # the hidden states of a batch-8 decode step between two layers
        {"name": "residual_decode", "op": "norm", "T": 8, "K": HIDDEN, "res": "bf16", "y": False},
        # the same for a 4,096-token prefill chunk
        {"name": "residual_prefill", "op": "norm", "T": 4096, "K": HIDDEN, "res": "bf16", "y": False},
        # a residual stream kept in fp32, an odd number of rows, a short last block; the rows in bf16 as well
        {"name": "residual_odd_fp32", "op": "norm", "T": 1003, "K": 2064, "res": "fp32", "y": True},
        # decode, batch 8, an adapter for each request: the main-KV input C
        {"name": "lora_kv_decode", "op": "lora", "T": 8, "K": HIDDEN, "N": 512, "rank": 16, "adapters": 8, "run": 1,
         "out": "bf16", "head": 0},
        # decode, batch 8, four adapters: the indexer queries as codes and scales with RoPE
        {"name": "lora_index_q_decode", "op": "lora", "T": 8, "K": LATENT, "N": HEADS_IDX * 128, "rank": 64, "adapters": 4,
         "run": 1, "out": "fp8", "head": 128},
        # a decode batch of 64 requests with 16 adapters: the attention queries
        {"name": "lora_attn_q_batch", "op": "lora", "T": 64, "K": LATENT, "N": HEADS_ATT * 512, "rank": 32, "adapters": 16,
         "run": 1, "out": "bf16", "head": 512},
        # prompts of an odd batch, odd widths, fp32 out
        {"name": "lora_odd_fp32", "op": "lora", "T": 333, "K": 1360, "N": 1001, "rank": 24, "adapters": 5, "run": 40,
         "out": "fp32", "head": 0},
        # a 4,096-token prefill chunk of several prompts, four adapters: the attention queries
        {"name": "lora_attn_q_prefill", "op": "lora", "T": 4096, "K": LATENT, "N": HEADS_ATT * 512, "rank": 64, "adapters": 4,
         "run": 600, "out": "bf16", "head": 512},
        # one token's log probability alone
        {"name": "logprobs_one", "op": "logprobs", "T": 1, "V": 32000, "in": "bf16", "top": 0, "mask": False},
        # a batch-8 decode step's answer with 20 alternatives
        {"name": "logprobs_decode", "op": "logprobs", "T": 8, "V": VOCAB, "in": "fp32", "top": 20, "mask": False},
        # constrained answers: masked logits, one row with nothing left, an odd vocabulary
        {"name": "logprobs_masked", "op": "logprobs", "T": 333, "V": 50001, "in": "fp32", "top": 5, "mask": True},
        # the tokens of a prompt under the model
        {"name": "logprobs_prompt", "op": "logprobs", "T": 2048, "V": VOCAB, "in": "bf16", "top": 1, "mask": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "lora", "lora", "logprobs"])
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 6000), "K": 16 * _log(rng, 1, 448), "res": rng.choice(["bf16", "fp32"]),
                "y": rng.random() < 0.5}
    if op == "lora":
        T, K = _log(rng, 1, 4096), 16 * _log(rng, 4, 448)
        out = rng.choice(["fp32", "bf16", "fp8"])
        top = min(32768, int(2048 * 2048 * 32768 / (T * K)))
        N = _log(rng, 8, max(8, top)) if out != "fp8" else 128 * _log(rng, 1, max(1, top // 128))
        head = 0
        if N >= 128 and rng.random() < 0.5:
            head = rng.choice([128, 256, 512])
            N = max(head, N // head * head)
        return {"op": op, "T": T, "K": K, "N": N, "rank": 8 * _log(rng, 1, 16), "adapters": _log(rng, 1, 24),
                "run": 1 if T <= 64 else _log(rng, 16, T), "out": out, "head": head}
    T = _log(rng, 1, 2048)
    V = _log(rng, 1, min(1 << 18, VOCAB * 2048 // T))
    return {"op": op, "T": T, "V": V, "in": rng.choice(["fp32", "bf16"]) if T * V <= 1 << 27 else "bf16",
            "top": rng.choice([0, 1, 5, 20, 32]), "mask": rng.random() < 0.3}


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
    return torch.where(loud, 12.0 * x, x)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": case}
    T = case["T"]
    if case["op"] == "norm":
        K = case["K"]
        kind = torch.bfloat16 if case["res"] == "bf16" else torch.float32
        s["x"] = (0.5 * torch.randn(T, K, generator=g, device=dev)).to(torch.bfloat16)   # a layer's output
        s["residual"] = _hidden(T, K, g, dev).to(kind)
        s["gamma"] = 1.0 + 0.1 * torch.randn(K, generator=g, device=dev)
        s["residual_out"] = torch.empty(T, K, dtype=kind, device=dev)
        s["codes"] = torch.empty(T, K, dtype=torch.uint8, device=dev)
        s["scale"] = torch.empty(T, _blocks(K), device=dev)
        s["y"] = torch.empty(T, K, dtype=torch.bfloat16, device=dev) if case["y"] else None
        return s
    if case["op"] == "lora":
        K, N, R, n = case["K"], case["N"], case["rank"], case["adapters"]
        s["x"], s["x_scale"] = _quant_rows(_hidden(T, K, g, dev))
        s["w"], s["w_scale"] = _quant_tiles(torch.randn(N, K, generator=g, device=dev) / math.sqrt(K))
        s["a"] = (torch.randn(n, R, K, generator=g, device=dev) / math.sqrt(K)).to(torch.bfloat16)
        s["b"] = (0.3 * torch.randn(n, N, R, generator=g, device=dev) / math.sqrt(R)).to(torch.bfloat16)
        s["adapter_scale"] = 0.5 + torch.rand(n, generator=g, device=dev)
        # requests of `run` rows each; one in nine has no adapter
        runs = (T + case["run"] - 1) // case["run"]
        ids = torch.randint(0, n, (runs,), generator=g, device=dev, dtype=torch.int32)
        none = torch.randint(0, 9, (runs,), generator=g, device=dev) == 0
        ids = torch.where(none, torch.full_like(ids, -1), ids)
        s["row_adapter"] = ids.repeat_interleave(case["run"])[:T].contiguous()
        s["pos"] = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32) if case["head"] else None
        kind = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}[case["out"]]
        s["out"] = torch.empty(T, N, dtype=kind, device=dev)
        s["out_scale"] = torch.empty(T, N // 128, device=dev) if case["out"] == "fp8" else None
        torch.cuda.synchronize()  # run() passes w_ready: the weights were written well before the first call
        return s
    V, n = case["V"], case["top"]
    x = 2.0 * torch.randn(T, V, generator=g, device=dev)
    # a few likely tokens a row
    x.scatter_add_(1, torch.randint(0, V, (T, 8), generator=g, device=dev), 14.0 * torch.rand(T, 8, generator=g, device=dev))
    if case["mask"]:
        x = torch.where(torch.rand(T, V, generator=g, device=dev) < 0.9, torch.full_like(x, -math.inf), x)
        if T > 2:
            x[T // 2] = -math.inf                      # a row with nothing left
            x[T // 3, : V // 2] = torch.finfo(torch.bfloat16).min
    x = x.to(torch.float32 if case["in"] == "fp32" else torch.bfloat16)
    token = torch.empty(T, dtype=torch.int32, device=dev)
    for t0 in range(0, T, 256):  # drawn from the rows' own probabilities
        part = x[t0:t0 + 256].float()
        part = part - torch.log(-torch.log(torch.rand(part.shape, generator=g, device=dev).clamp(1e-20, 1 - 1e-7)))
        token[t0:t0 + 256] = part.argmax(dim=1).to(torch.int32)
    s["logits"] = x
    s["token"] = torch.where(torch.randint(0, 50, (T,), generator=g, device=dev) == 0, torch.full_like(token, -1), token)

    def buf():
        return torch.empty(T, device=dev)

    s["o"] = {"logprob": buf(), "entropy": buf(), "lse": buf(),
              "top_id": torch.empty(T, n, dtype=torch.int32, device=dev) if n else None,
              "top_logprob": torch.empty(T, n, device=dev) if n else None}
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


def _plain_norm(s):
    r = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    v = r.float()
    y = v / torch.sqrt((v * v).mean(dim=-1, keepdim=True) + EPS) * s["gamma"]
    codes, scale = _quant_rows(y)
    out = {"residual": r, "codes": codes, "scale": scale}
    if s["y"] is not None:
        out["y"] = y.to(torch.bfloat16)
    return out


def _plain_lora(s):
    c = s["case"]
    T, K, N, R, n = c["T"], c["K"], c["N"], c["rank"], c["adapters"]
    x = s["x"].float() * s["x_scale"].repeat_interleave(128, dim=1)[:, :K]
    w = s["w"].float() * s["w_scale"].repeat_interleave(128, dim=0)[:N].repeat_interleave(128, dim=1)[:, :K]
    # all adapters' inner products; a row keeps its own adapter's, times the adapter's factor
    v = (x @ s["a"].float().view(n * R, K).t()).view(T, n, R)
    mine = s["row_adapter"][:, None] == torch.arange(n, device=x.device, dtype=torch.int32)[None, :]
    v = torch.where(mine[:, :, None], v * s["adapter_scale"][None, :, None], torch.zeros_like(v))
    y = x @ w.t() + v.view(T, n * R) @ s["b"].float().permute(0, 2, 1).reshape(n * R, N)
    if c["head"]:
        y = _rope_plain(y, s["pos"], c["head"])
    if c["out"] == "fp8":
        codes, scale = _quant_rows(y)
        return {"out": codes, "scale": scale}
    return {"out": y if c["out"] == "fp32" else y.to(torch.bfloat16)}


def _plain_logprobs(s):
    n = s["case"]["top"]
    x = s["logits"].float()
    x = torch.where(torch.isfinite(x), x + 0.0, torch.full_like(x, -math.inf))
    top, at = x.max(dim=1, keepdim=True)
    empty = top[:, 0] == -math.inf
    d = x - torch.where(empty[:, None], torch.zeros_like(top), top)
    # the largest term, 1, is left out of the sum and comes back in log1p: next to a
    # likely token the others' sum is what its log probability is
    e = torch.exp(d).scatter(1, at, 0.0)
    rest = e.sum(dim=1)
    log_total = torch.where(empty, torch.zeros_like(rest), torch.log1p(rest))
    lse = top[:, 0] + log_total
    entropy = log_total - torch.where(e == 0, torch.zeros_like(e), d * e).sum(dim=1) / (1 + rest)
    tok = s["token"].long()
    log_p = d.gather(1, tok.clamp(min=0)[:, None])[:, 0] - log_total
    out = {"logprob": torch.where(tok >= 0, log_p, torch.zeros_like(log_p)), "entropy": entropy, "lse": lse}
    if n:
        # unique keys: the value's order, then the lower token
        bits = x.view(torch.int32)
        order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
        key = (order << 32) + (0xFFFFFFFF - torch.arange(x.shape[1], device=x.device))
        best = torch.topk(key, min(n, x.shape[1]), dim=1).values
        ids = 0xFFFFFFFF - (best & 0xFFFFFFFF)
        gone = x.gather(1, ids) == -math.inf
        log_p = torch.where(gone, torch.full_like(d[:, :1], -math.inf), d.gather(1, ids) - log_total[:, None])
        more = n - best.shape[1]
        out["top_id"] = torch.nn.functional.pad(torch.where(gone, -1, ids).to(torch.int32), (0, more), value=-1)
        out["top_logprob"] = torch.nn.functional.pad(log_p, (0, more), value=-math.inf)
    return out


def run(state):
    case = state["case"]
    if not own:
        return {"norm": _plain_norm, "lora": _plain_lora, "logprobs": _plain_logprobs}[case["op"]](state)
    from serving_lightning_indexer_gb300 import csa2
    if case["op"] == "norm":
        csa2.add_norm_fp8(state["x"], state["residual"], state["residual_out"], state["gamma"], codes=state["codes"],
                          scale=state["scale"], y=state["y"], eps=EPS)
        out = {"residual": state["residual_out"], "codes": state["codes"].view(torch.float8_e4m3fn), "scale": state["scale"]}
        if state["y"] is not None:
            out["y"] = state["y"]
        return out
    if case["op"] == "lora":
        csa2.lora_linear(state["x"].view(torch.uint8), state["x_scale"], state["w"].view(torch.uint8), state["w_scale"],
                         state["a"], state["b"], state["row_adapter"], state["out"], adapter_scale=state["adapter_scale"],
                         out_scale=state["out_scale"], row_pos=state["pos"], rope_head=case["head"], rope_theta=THETA,
                         w_ready=True)
        if case["out"] == "fp8":
            return {"out": state["out"].view(torch.float8_e4m3fn), "scale": state["out_scale"]}
        return {"out": state["out"]}
    csa2.logprobs(state["logits"], token=state["token"], **state["o"])
    return {k: v for k, v in state["o"].items() if v is not None}


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        K = case["K"]
        size = 2 if case["res"] == "bf16" else 4
        return {"bytes": T * K * (2 + 2 * size + 1 + (2 if case["y"] else 0)) + 4 * T * _blocks(K) + 4 * K, "flops": 7 * T * K}
    if case["op"] == "lora":
        K, N, R = case["K"], case["N"], case["rank"]
        size = {"fp32": 4, "bf16": 2, "fp8": 1}[case["out"]]
        scales = T * _blocks(K) + _blocks(N) * _blocks(K) + (T * N // 128 if case["out"] == "fp8" else 0)
        runs = (T + case["run"] - 1) // case["run"]
        used = case["adapters"] * (1 - (1 - 8 / 9 / case["adapters"]) ** runs)  # adapters that some row has
        return {"bytes": T * K + N * K + size * T * N + 4 * scales + 2 * used * R * (K + N) + 4 * T,
                "flops": 2 * T * N * K + 2 * T * R * (K + N)}
    V = case["V"]
    return {"bytes": T * (V * (4 if case["in"] == "fp32" else 2) + 16 + 8 * case["top"]), "flops": 5 * T * V}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        r = s["x"].double() + s["residual"].double()
        kept = r.to(s["residual"].dtype)
        v = kept.double()
        v = v * torch.rsqrt(v.square().sum(-1, keepdim=True) / v.shape[1] + EPS) * s["gamma"].double()
        codes, scale = _exact_codes(v)
        out = {"residual": kept.double() if case["res"] == "bf16" else r, "codes": codes, "scale": scale}
        if case["y"]:
            out["y"] = v
        return out
    if case["op"] == "lora":
        dev = s["w"].device
        rows, cols = torch.arange(case["N"], device=dev) // 128, torch.arange(case["K"], device=dev) // 128
        x = s["x"].double() * s["x_scale"].double()[:, cols]
        w = s["w"].double() * s["w_scale"].double()[rows][:, cols]
        v = torch.einsum("tk,nk->tn", x, w)
        for i in range(case["adapters"]):
            at = (s["row_adapter"] == i).nonzero()[:, 0]
            if len(at):
                inner = torch.einsum("tk,rk->tr", x[at], s["a"][i].double()) * s["adapter_scale"][i].double()
                v[at] += torch.einsum("tr,nr->tn", inner, s["b"][i].double())
        if case["head"]:
            D = case["head"]
            power = torch.arange(0, -64, -2, dtype=torch.float64, device=dev) / 64
            turn = torch.outer(s["pos"].double(), torch.exp(power * math.log(THETA)))
            pairs = torch.view_as_complex(v.view(len(v), -1, D)[:, :, D - 64:].reshape(len(v), -1, 32, 2).contiguous())
            pairs = pairs * torch.polar(torch.ones_like(turn), turn)[:, None, :]
            v.view(len(v), -1, D)[:, :, D - 64:] = torch.view_as_real(pairs).reshape(len(v), -1, 64)
        return dict(zip(("out", "scale"), _exact_codes(v))) if case["out"] == "fp8" else {"out": v}
    found = {k: [] for k in ("logprob", "entropy", "lse", "top_logprob")}
    n = case["top"]
    for t0 in range(0, case["T"], 512):
        x = s["logits"][t0:t0 + 512].double()
        x = torch.where(x.isfinite(), x, -math.inf)
        lse = torch.logsumexp(x, 1)
        log_p = x - torch.where(lse == -math.inf, 0.0, lse)[:, None]
        tok = s["token"][t0:t0 + 512].long()
        found["lse"].append(lse)
        found["entropy"].append(-torch.where(log_p == -math.inf, 0.0, log_p * log_p.exp()).sum(1))
        found["logprob"].append(torch.where(tok < 0, 0.0, log_p.gather(1, tok.clamp(min=0)[:, None])[:, 0]))
        if n:
            best = log_p.sort(dim=1, descending=True).values[:, :n]
            found["top_logprob"].append(torch.nn.functional.pad(best, (0, n - best.shape[1]), value=-math.inf))
    return {k: torch.cat(v) if v else None for k, v in found.items()}


def _exact_codes(v):
    """Code values and scales of 64-bit numbers, block by block of 128 columns."""
    T, K = v.shape
    nb = _blocks(K)
    top = torch.nn.functional.pad(v.abs(), (0, nb * 128 - K)).view(T, nb, 128).amax(-1)
    use = top.clamp(min=AMAX_FLOOR)
    c = torch.arange(K, device=v.device) // 128
    codes = (v * E4M3_MAX / use[:, c]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double()
    return codes, torch.where(top > 0, use / E4M3_MAX, torch.ones_like(top))
