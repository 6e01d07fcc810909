"""The serving-step and training operators of the gated delta rule, as measured cases.

Three operators, each in a plain form (elementary torch operations in 32 bits)
and, with `own` true, as the calls a user makes of this package:

  decode    gdn_decode: the recurrent form.  Every sequence's f32 state, reached
            through a pointer table, takes its 0, 1 or a few new rows in place.
  tables    gdn_state_tables: from the request lengths and state slots of one
            engine step, the packed row offsets, the state pointer table, the
            maps row -> sequence and row -> slot, and the 64-row chunk map.
  backward  gdn_chunk_backward: the gradients of q, k, v, g, beta and the
            initial state of packed sequences, from the gradients of the
            outputs and of the final states.

Per sequence and value head, with the state held as H = S^T [d_k, d_v]:
    H <- exp(g_t) H;  H <- H + beta_t k_t (v_t - H^T k_t)^T;  o_t = scale H^T q_t.
Inputs follow the package's workloads: q and k of unit length, v ~ N(0, 1),
g = logsigmoid(N(2, 1)), beta = sigmoid(N(0, 1)), states ~ N(0, 0.02).
"""
import math
import random

import torch

own = False

CHUNK = 64
DEV = "cuda"


def listed():
    return [
        # One token of one request of a small model: nothing but latency.
        {"name": "decode one d64", "op": "decode", "batch": 1, "rows": 1, "ragged": False, "pad": 0,
         "hk": 2, "hv": 2, "d": 64, "scale": 1.0},
        # The decode step of the verify workload's batch, one token a request.
        {"name": "decode 64x48", "op": "decode", "batch": 64, "rows": 1, "ragged": False, "pad": 0,
         "hk": 16, "hv": 48, "d": 128, "scale": 1.0},
        # A mixed step: 0 to 6 rows a request, two padding entries in the table.
        {"name": "decode ragged", "op": "decode", "batch": 37, "rows": 6, "ragged": True, "pad": 2,
         "hk": 16, "hv": 32, "d": 128, "scale": 0.0883883},
        # A full serving batch.
        {"name": "decode 256x48", "op": "decode", "batch": 256, "rows": 1, "ragged": False, "pad": 0,
         "hk": 16, "hv": 48, "d": 128, "scale": 1.0},
        # The tables of a decode step: one row a request.
        {"name": "tables decode", "op": "tables", "n": 64, "most": 1, "pad": 0, "spare": 0},
        # A mixed step: decodes, prompt chunks, empty and padding entries, row buffers longer than the step.
        {"name": "tables mixed", "op": "tables", "n": 300, "most": 512, "pad": 9, "spare": 1000},
        # Thousands of requests of up to 512 rows.
        {"name": "tables large", "op": "tables", "n": 4096, "most": 512, "pad": 100, "spare": 0},
        # The tiny prefill workload's shape, trained.
        {"name": "backward tiny d64", "op": "backward", "lens": "256", "hk": 2, "hv": 2, "d": 64, "h0": False, "scale": 1.0},
        # Short, empty and ragged sequences around the chunk's borders.
        {"name": "backward ragged", "op": "backward", "lens": "1,63,64,0,65,777,130", "hk": 2, "hv": 6, "d": 128, "h0": True, "scale": 0.0883883},
        # The single-sequence workload.
        {"name": "backward 4096x32", "op": "backward", "lens": "4096", "hk": 16, "hv": 32, "d": 128, "h0": True, "scale": 1.0},
        # The headline prefill workload's shape.
        {"name": "backward 4576x48", "op": "backward", "lens": "4576", "hk": 16, "hv": 48, "d": 128, "h0": False, "scale": 1.0},
        # The varlen workload's batch.
        {"name": "backward varlen", "op": "backward", "lens": "3670,1053,3636,3547,4688,709,2874,4497", "hk": 16, "hv": 48, "d": 128, "h0": True, "scale": 1.0},
    ]


HEADS = [(1, 1, 64), (2, 2, 64), (2, 8, 64), (4, 4, 128), (2, 6, 128), (4, 12, 128), (8, 16, 128), (16, 32, 128), (16, 48, 128)]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "tables", "backward", "backward"])
    if op == "tables":
        return {"op": op, "n": _log(rng, 8, 4096), "most": _log(rng, 1, 512), "pad": rng.randint(0, 2), "spare": rng.choice([0, rng.randint(1, 2000)])}
    hk, hv, d = rng.choice(HEADS)
    scale = rng.choice([1.0, round(d ** -0.5, 7)])
    if op == "decode":
        ragged = rng.random() < 0.5
        batch = _log(rng, 2 if ragged else 1, 256)
        return {"op": op, "batch": batch, "rows": rng.randint(2, 6) if ragged else 1, "ragged": ragged,
                "pad": rng.randint(0, 1) if ragged else 0, "hk": hk, "hv": hv, "d": d, "scale": scale}
    total, count = _log(rng, 1, 24000), rng.choice([1, 1, 2, 3, 5, 8])
    cuts = sorted(rng.randint(0, total) for _ in range(count - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    # The plain form pads every sequence to the longest: keep the padded size within the largest case's.
    while max(lens) * len(lens) > 38000:
        lens.remove(min(lens))
    return {"op": op, "lens": ",".join(map(str, lens)), "hk": hk, "hv": hv, "d": d, "h0": rng.random() < 0.5, "scale": scale}


# -- inputs -------------------------------------------------------------------


def _unit(x):
    return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(torch.bfloat16)


def _rows(gen, rows, hk, hv, d):
    def n(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    return {"q": _unit(n(rows, hk, d)), "k": _unit(n(rows, hk, d)), "v": n(rows, hv, d).to(torch.bfloat16),
            "g": torch.nn.functional.logsigmoid(n(rows, hv) + 2.0), "beta": torch.sigmoid(n(rows, hv))}


def _offsets(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _request_lens(case):
    """The new rows of each request, the same for every seed: mostly single tokens, some long, some none."""
    if case["most"] == 1:
        return [1] * case["n"]
    rng = random.Random(case["n"])
    return [rng.choice([0, 1, 1, 1, rng.randint(1, case["most"])]) for _ in range(case["n"])]


def _decode_lens(case):
    """The new rows of each sequence, the same for every seed: 0 to `rows` of them, or one each."""
    rng = random.Random(case["batch"])
    return [rng.randint(0, case["rows"]) for _ in range(case["batch"] - 1)] + [1] if case["ragged"] else [1] * case["batch"]


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed % (1 << 62))
    s = {"case": case, "op": case["op"]}
    if case["op"] == "tables":
        n = case["n"]
        lens = _request_lens(case)
        slots = list(range(n + n // 4 + 1))
        rng.shuffle(slots)
        slots = slots[:n]
        for b in rng.sample(range(n), min(n, case["pad"])):
            slots[b] = -1
        rows, chunks = sum(lens), sum(-(-x // CHUNK) for x in lens)
        # The pool of states whose slots the tables point at: 4 heads of [64, 64] f32 a slot.
        s |= {"lens": _int32(lens), "slots": _int32(slots), "pool": torch.empty(n + n // 4 + 1, 4, 64, 64, device=DEV)}
        # The step's buffers, kept from step to step; rows behind the last request stay as they are.
        s["tables"] = {"cu_seqlens": torch.empty(n + 1, dtype=torch.int32, device=DEV), "h_table": torch.empty(n, dtype=torch.int64, device=DEV),
                       "row_seq": torch.full((rows + case["spare"],), -7, dtype=torch.int32, device=DEV),
                       "row_slot": torch.full((rows + case["spare"],), -7, dtype=torch.int32, device=DEV),
                       "cu_chunks": torch.empty(n + 1, dtype=torch.int32, device=DEV),
                       "chunk_seq": torch.full((chunks + case["spare"],), -7, dtype=torch.int32, device=DEV)}
        s |= {"rows": rows, "chunks": chunks}
        return s
    hk, hv, d = case["hk"], case["hv"], case["d"]
    if case["op"] == "decode":
        batch = case["batch"]
        lens = _decode_lens(case)
        count = batch + batch // 8 + 1
        slots = list(range(count))
        rng.shuffle(slots)
        slots = slots[:batch]
        for b in rng.sample(range(batch), case["pad"]):
            slots[b] = -1
        pool = torch.randn(count, hv, d, d, generator=gen, device=DEV) * 0.02
        live = [b for b in range(batch) if slots[b] >= 0]
        s |= _rows(gen, sum(lens), hk, hv, d)
        s |= {"pool": pool, "lens": lens, "slots": torch.tensor(slots, device=DEV), "live": torch.tensor(live, device=DEV),
              "h_table": torch.tensor([pool[x].data_ptr() if x >= 0 else 0 for x in slots], dtype=torch.int64, device=DEV),
              "cu_seqlens": _int32(_offsets(lens)) if case["ragged"] else None, "most": max(lens)}
        return s
    lens = [int(x) for x in case["lens"].split(",")]
    n, total = len(lens), sum(lens)
    s |= _rows(gen, total, hk, hv, d)
    s |= {"cu_seqlens": _int32(_offsets(lens)), "n": n, "most": max(lens),
          "do": torch.randn(total, hv, d, generator=gen, device=DEV).to(torch.bfloat16),
          "h0": torch.randn(n, hv, d, d, generator=gen, device=DEV) * 0.02 if case["h0"] else None,
          "dhT": torch.randn(n, hv, d, d, generator=gen, device=DEV) * 0.02 if case["h0"] else None}
    return s


# -- one pass -----------------------------------------------------------------


def run(s):
    if own:
        import linear_attention_ssm_gdn_b200 as gdn

        scale = s["case"].get("scale")
        if s["op"] == "decode":
            o = gdn.gdn_decode(s["h_table"], s["q"], s["k"], s["v"], s["g"], s["beta"], cu_seqlens=s["cu_seqlens"], scale=scale)
            return {"o": o, "pool": s["pool"]}
        if s["op"] == "tables":
            t = gdn.gdn_state_tables(s["lens"], s["slots"], s["pool"], out=s["tables"])
            return _from_pool(t, s["pool"])
        dq, dk, dv, dg, dbeta, dh0 = gdn.gdn_chunk_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu_seqlens"], s["do"],
                                                            h0=s["h0"], dhT=s["dhT"], scale=scale)
        return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta, "dh0": dh0}
    return {"decode": _decode, "tables": _tables, "backward": _backward}[s["op"]](s)


def _from_pool(t, pool):
    """The tables with the pointers counted from the pool's start (its address differs from process to process), -1 for none."""
    return {**t, "h_table": t["h_table"].clamp_min(pool.data_ptr() - 1) - pool.data_ptr()}


def _decode(s):
    """The recurrence on gathered states, one row of every sequence at a time."""
    case, pool = s["case"], s["pool"]
    batch, vpg, d = case["batch"], case["hv"] // case["hk"], case["d"]
    q = s["q"].float().repeat_interleave(vpg, 1)
    k = s["k"].float().repeat_interleave(vpg, 1)
    v, g, beta = s["v"].float(), s["g"], s["beta"]
    rows = v.shape[0]
    if s["cu_seqlens"] is None:
        start = torch.arange(batch, device=DEV)
        count = torch.ones_like(start)
    else:
        start, count = s["cu_seqlens"][:-1].long(), s["cu_seqlens"].diff().long()
    count = torch.where(s["slots"] >= 0, count, 0)
    h = pool[s["slots"].clamp_min(0)]
    o = torch.zeros(rows + 1, case["hv"], d, dtype=torch.bfloat16, device=DEV)
    for t in range(s["most"]):
        on = t < count
        at = torch.where(on, start + t, 0)
        gt, bt = torch.where(on[:, None], g[at], 0.0), torch.where(on[:, None], beta[at], 0.0)
        h = h * gt.exp()[..., None, None]
        u = v[at] - torch.matmul(k[at].unsqueeze(-2), h).squeeze(-2)
        h = h + k[at].unsqueeze(-1) * (bt[..., None] * u).unsqueeze(-2)
        ot = case["scale"] * torch.matmul(q[at].unsqueeze(-2), h).squeeze(-2)
        o[torch.where(on, at, rows)] = ot.to(torch.bfloat16)
    pool[s["slots"][s["live"]]] = h[s["live"]]
    return {"o": o[:rows], "pool": pool}


def _tables(s):
    t, lens, slots, pool = s["tables"], s["lens"], s["slots"], s["pool"]
    n = lens.shape[0]
    seq = torch.arange(n, dtype=torch.int32, device=DEV)
    chunks = (lens + (CHUNK - 1)) // CHUNK
    t["cu_seqlens"][0] = 0
    t["cu_seqlens"][1:] = torch.cumsum(lens, 0)
    t["cu_chunks"][0] = 0
    t["cu_chunks"][1:] = torch.cumsum(chunks, 0)
    row_seq = torch.repeat_interleave(seq, lens, output_size=s["rows"])
    t["row_seq"][: s["rows"]] = row_seq
    t["row_slot"][: s["rows"]] = slots[row_seq]
    t["chunk_seq"][: s["chunks"]] = torch.repeat_interleave(seq, chunks, output_size=s["chunks"])
    t["h_table"][:] = torch.where(slots >= 0, pool.data_ptr() + slots.long() * (pool.stride(0) * 4), 0)
    return _from_pool(t, pool)


def _backward(s):
    """The chunk form, forward and backward: per 64-row chunk with entry state H, cumulative gates G, decays
    D_rs = e^(G_r - G_s) for s <= r and A = strictly lower diag(beta) (K K^T * D):
        X = beta (V - e^G K H),  N = (I + A)^-1 X,  O = scale (e^G Q H + (Q K^T * D) N),
        H' = e^(G_C) H + (e^(G_C - G) K)^T N,
    every sequence padded to whole chunks of the longest one (beta = g = 0 changes no state)."""
    case = s["case"]
    hk, hv, d, scale = case["hk"], case["hv"], case["d"], case["scale"]
    vpg, n, nc = hv // hk, s["n"], -(-s["most"] // CHUNK)
    cu = s["cu_seqlens"].long()
    total = s["q"].shape[0]
    place = torch.arange(nc * CHUNK, device=DEV)
    on = place < cu.diff()[:, None]
    at = torch.where(on, cu[:-1, None] + place, 0)

    def chunked(x, heads=1):  # [T, h, ...] -> [n, h * heads, nc, C, ...] in 32 bits, zeros in the padding
        y = torch.where(on.view(n, -1, *[1] * (x.dim() - 1)), x[at].float(), 0.0)
        y = y.view(n, nc, CHUNK, *x.shape[1:]).movedim(3, 1)
        return y.repeat_interleave(heads, 1) if heads > 1 else y

    Q, K = chunked(s["q"], vpg), chunked(s["k"], vpg)
    V, dO, beta = chunked(s["v"]), chunked(s["do"]), chunked(s["beta"])[..., None]
    G = chunked(s["g"]).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    strict = low.tril(-1)
    D = torch.where(low, G[..., :, None] - G[..., None, :], -math.inf).exp()
    eG, eC, eT = G.exp()[..., None], G[..., -1].exp()[..., None, None], (G[..., -1:] - G).exp()[..., None]
    KK = torch.where(strict, D * (K @ K.mT), 0.0)
    A = beta * KK
    eye = torch.eye(CHUNK, device=DEV)
    T = torch.linalg.solve_triangular(eye + A, eye.expand_as(A), upper=False, unitriangular=True)
    M = D * (Q @ K.mT)
    Kd, gK, gQ = eT * K, eG * K, scale * eG * Q

    h = s["h0"] if s["h0"] is not None else torch.zeros(n, hv, d, d, device=DEV)
    H, N, X = [], [], []
    for c in range(nc):
        H.append(h)
        X.append(V[:, :, c] - gK[:, :, c] @ h)
        N.append(T[:, :, c] @ (beta[:, :, c] * X[-1]))
        h = eC[:, :, c] * h + Kd[:, :, c].mT @ N[-1]
    H, N, X = torch.stack(H, 2), torch.stack(N, 2), torch.stack(X, 2)

    dN0, gQdO, bgK = scale * (M.mT @ dO), gQ.mT @ dO, beta * gK
    dh = s["dhT"] if s["dhT"] is not None else torch.zeros(n, hv, d, d, device=DEV)
    dH, dX = [None] * nc, [None] * nc
    for c in range(nc - 1, -1, -1):
        dH[c] = dh
        dX[c] = T[:, :, c].mT @ (dN0[:, :, c] + Kd[:, :, c] @ dh)
        dh = eC[:, :, c] * dh + gQdO[:, :, c] - bgK[:, :, c].mT @ dX[c]
    dH, dX = torch.stack(dH, 2), torch.stack(dX, 2)

    dM = scale * torch.where(low, dO @ N.mT, 0.0)
    dA = torch.where(strict, -(dX @ N.mT), 0.0)
    E, F, L = dO @ H.mT, dX @ H.mT, N @ dH.mT
    P, R = dM * D, dA * beta * D
    dQ = scale * eG * E + P @ K
    dK = P.mT @ Q + torch.where(strict, R, 0.0) @ K + R.mT @ K - beta * eG * F + eT * L
    dV = beta * dX
    dbeta = (dX * X).sum(-1) + (dA * KK).sum(-1)
    back = eT[..., 0] * (K * L).sum(-1)
    PM, RA = dM * M, dA * A
    dG = scale * eG[..., 0] * (E * Q).sum(-1) - (beta * eG)[..., 0] * (F * K).sum(-1) - back + PM.sum(-1) - PM.sum(-2) + RA.sum(-1) - RA.sum(-2)
    dG[..., -1] += back.sum(-1) + eC[..., 0, 0] * (H * dH).sum((-2, -1))
    dg = dG.flip(-1).cumsum(-1).flip(-1)

    def packed(x):  # [n, h, nc, C, ...] -> [T, h, ...]
        y = x.movedim(1, 3).reshape(n, nc * CHUNK, x.shape[1], *x.shape[4:])
        out = torch.empty(total + 1, *y.shape[2:], device=DEV)
        out[torch.where(on, at, total)] = y
        return out[:total]

    def shared(x):  # sums the gradients of the value heads that share a key head
        return x.view(n, hk, vpg, *x.shape[2:]).sum(2)

    return {"dq": packed(shared(dQ)).to(torch.bfloat16), "dk": packed(shared(dK)).to(torch.bfloat16), "dv": packed(dV).to(torch.bfloat16),
            "dg": packed(dg), "dbeta": packed(dbeta), "dh0": dh if s["h0"] is not None else None}


# -- what a pass cannot do without ----------------------------------------------


def work(case):
    if case["op"] == "tables":
        lens = _request_lens(case)
        rows, chunks = sum(lens), sum(-(-x // CHUNK) for x in lens)
        return {"bytes": 8 * case["n"] + 16 * case["n"] + 8 + 8 * rows + 4 * chunks, "flops": 0}
    hk, hv, d = case["hk"], case["hv"], case["d"]
    if case["op"] == "decode":
        rows = sum(_decode_lens(case))
        row = 4 * hk * d + 4 * hv * d + 8 * hv
        live = case["batch"] - case["pad"]
        return {"bytes": rows * row + 8 * live * hv * d * d, "flops": rows * hv * 8 * d * d}
    lens = [int(x) for x in case["lens"].split(",")]
    total, n = sum(lens), len(lens)
    states = (3 if case["h0"] else 0) * 4 * n * hv * d * d
    # reads q, k, v, do, g, beta; writes dq, dk, dv, dg, dbeta
    byte = total * (8 * hk * d + 6 * hv * d + 16 * hv) + states
    # per row and head: H^T k, H += k u^T, do H^T, q do^T, dH^T k, k du^T, du H, dH u (2 d^2 each), and the chunk's
    # C x C products over d (k k, q k, do n, dx n; M dO; P k, P^T q, R k + R^T k; T x and T^T y), half of each masked
    return {"bytes": byte, "flops": total * hv * (16 * d * d + 10 * CHUNK * d)}


# -- 64 bits ----------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None
    vpg, scale = case["hv"] // case["hk"], case["scale"]
    q, k = (s[x].double()[:, torch.arange(case["hv"], device=DEV) // vpg] for x in ("q", "k"))
    v, a, beta = s["v"].double(), s["g"].double().exp(), s["beta"].double()
    if case["op"] == "decode":
        # S <- a S (I - beta k k^T) + beta v k^T,  o = scale S q, sequence by sequence, with S = H^T.
        cu = _offsets(s["lens"])
        pool, o = s["pool"].double(), torch.zeros(v.shape, dtype=torch.float64, device=DEV)
        for b, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            S = pool[slot].mT
            for t in range(cu[b], cu[b + 1]):
                Sk = torch.einsum("hvk,hk->hv", S, k[t])
                S = a[t][:, None, None] * (S - torch.einsum("h,hv,hk->hvk", beta[t], Sk, k[t])) + torch.einsum("h,hv,hk->hvk", beta[t], v[t], k[t])
                o[t] = scale * torch.einsum("hvk,hk->hv", S, q[t])
            pool[slot] = S.mT
        return {"o": o, "pool": pool}
    # Token by token: forward with the states kept at every 64th row, then each run of 64 rows again and backward.
    lens = [int(x) for x in case["lens"].split(",")]
    cu, hv, d = _offsets(lens), case["hv"], case["d"]
    n, total, most = len(lens), cu[-1], max(lens)
    do = s["do"].double()
    h = s["h0"].double() if case["h0"] else torch.zeros(n, hv, d, d, dtype=torch.float64, device=DEV)
    lens_t, cu_t = torch.tensor(lens, device=DEV), torch.tensor(cu[:-1], device=DEV)

    def step(t, h):  # H, the decayed H, and u of row t; sequences that ended keep their H
        on = t < lens_t
        at = torch.where(on, cu_t + t, 0)
        at_, b_ = torch.where(on[:, None], a[at], 1.0), torch.where(on[:, None], beta[at], 0.0)
        hd = at_[..., None, None] * h
        u = v[at] - (k[at].unsqueeze(-2) @ hd).squeeze(-2)
        return on, at, at_, b_, hd, u, hd + k[at].unsqueeze(-1) * (b_[..., None] * u).unsqueeze(-2)

    kept = []
    for t in range(most):
        if t % 64 == 0:
            kept.append(h)
        h = step(t, h)[-1]
    dh = s["dhT"].double() if case["h0"] else torch.zeros_like(h)
    out = {x: torch.zeros(total + 1, hv, *([d] if x in ("dq", "dk", "dv") else []), dtype=torch.float64, device=DEV) for x in ("dq", "dk", "dv", "dg", "dbeta")}
    for c in range(len(kept) - 1, -1, -1):
        h, run_ = kept.pop(), []
        for t in range(64 * c, min(most, 64 * c + 64)):
            prior = h
            on, at, at_, b_, hd, u, h = step(t, h)
            run_.append((on, at, at_, b_, prior, u, h))
        for on, at, at_, b_, prior, u, after in reversed(run_):
            put = torch.where(on, at, total)
            m = on[:, None, None]
            dot = torch.where(m, do[at], 0.0)
            dq = scale * (after @ dot.unsqueeze(-1)).squeeze(-1)
            dh = dh + scale * q[at].unsqueeze(-1) * dot.unsqueeze(-2)
            w = (k[at].unsqueeze(-2) @ dh).squeeze(-2)  # k^T dH
            du = b_[..., None] * w
            hd = at_[..., None, None] * prior
            dk = b_[..., None] * (dh @ u.unsqueeze(-1)).squeeze(-1) - (hd @ du.unsqueeze(-1)).squeeze(-1)
            dhd = dh - k[at].unsqueeze(-1) * du.unsqueeze(-2)
            for name, x in (("dq", dq), ("dk", dk), ("dv", du), ("dbeta", (w * u).sum(-1)), ("dg", (dhd * hd).sum((-2, -1)))):
                out[name][put] = x
            dh = at_[..., None, None] * dhd
    out = {x: y[:total] for x, y in out.items()}
    for x in ("dq", "dk"):
        out[x] = out[x].view(total, case["hk"], vpg, d).sum(2)
    return {**out, "dh0": dh if case["h0"] else None}
