"""The operators of the 8-bit KV cache and of drafted-token trees: what is measured of them.

  append    bf16 keys and values written to the 8-bit cache (e4m3 codes, one power-of-two scale
            per token and KV head), the summaries of the blocks that this completes, and the
            written rows read back
  read      rows of the 8-bit cache as bf16, for a prefill over them
  decode    one query per sequence over the 8-bit cache (DashAttention's two stages)
  tree      a tree of drafted tokens per sequence over a bf16 cache
  tree_q8   the same over the 8-bit cache

Every case is synthetic with the structure of the repository's workloads: each 64-key block has
a topic, keys are 2 topic + N(0, I), queries 2 topic + N(0, I); a head selects about the blocks
of its topic.
"""
import math

import torch

own = False

BLOCK = 64
E_MIN, E_MAX = -118, 120           # scale exponents of the 8-bit cache
COARSE = 0.05                      # coarse scale of every case: a head selects its topic's blocks


# ---------------------------------------------------------------- cases

def listed():
    def c(name, op, B, Hq, Hkv, T, d, **more):
        return {"name": name, "op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "d": d, "alpha": 1.5,
                "topics": 16, "N": 1, "n": 1, "full": False, **more}
    return [
        # a chunk of a long prompt on four sequences of different lengths
        c("append_prompt", "append", 4, 32, 8, 16384, 128, n=4096),
        # the step of every decoded token: one row per sequence
        c("append_token", "append", 8, 32, 8, 16384, 128, n=1),
        # the accepted path of a drafted tree: rows picked by index, small heads
        c("append_path", "append", 3, 6, 2, 1024, 64, n=5, N=13),
        # a whole cached document for a prefill over it
        c("read_96k", "read", 1, 32, 8, 98304, 128, n=98304),
        # a ragged batch of recent windows at odd offsets
        c("read_window", "read", 5, 12, 3, 4096, 64, n=1001),
        # the repository's 96K decode workload, on the 8-bit cache
        c("decode_96k", "decode", 8, 32, 8, 98304, 128, full=True),
        # one user's step at 16K: latency counts
        c("decode_16k", "decode", 1, 16, 2, 16384, 128, full=True),
        # ragged batch, 12 query heads per KV head, d = 64, alpha = 2
        c("decode_wide", "decode", 5, 24, 2, 5056, 64, alpha=2.0, topics=8),
        # a 16-node tree over the 96K cache of eight sequences
        c("tree_96k", "tree", 8, 32, 8, 98304, 128, N=16, full=True),
        # one user's 64-node tree at 16K, the path crossing a block's end
        c("tree_16k", "tree", 1, 16, 2, 16384 + 40, 128, N=64, full=True),
        # a ragged batch of 24-node trees on the 8-bit cache
        c("tree_q8_32k", "tree_q8", 4, 32, 8, 32768, 128, N=24),
        # short contexts, five drafted tokens: latency counts
        c("tree_q8_short", "tree_q8", 2, 6, 2, 896, 64, N=5, topics=4),
    ]


def draw(rng):
    def logu(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    op = rng.choice(["append", "read", "decode", "decode", "tree", "tree", "tree_q8"])
    d = rng.choice([64, 128])
    while True:
        B, Hkv, G = logu(1, 12), rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        T = logu(40, 98304)
        if op != "tree":
            T = max(BLOCK, T // BLOCK * BLOCK)           # the 8-bit cache holds whole blocks
        N = rng.randint(1, 64) if op in ("tree", "tree_q8") else 1
        n = 1
        if op == "append":
            N = rng.choice([1, 1, 1, 7, 31, 64])         # above 1: the rows of an accepted path
            n = rng.choice([1, rng.randint(1, N)]) if N > 1 else min(T, logu(1, 8192))
        if op == "read":
            n = logu(1, T)
        rows = B * Hkv * G * N * T
        if rows <= 8 * 32 * 16 * 98304 and B * Hkv * T <= 64 * 98304 and (op != "append" or B * Hkv * T <= 1 << 20):
            break
    return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "T": T, "d": d, "alpha": rng.choice([1.5, 1.5, 2.0]),
            "topics": rng.choice([4, 8, 16, 32]), "N": N, "n": n, "full": rng.random() < 0.3}


def _lens(case):
    """Tokens each sequence holds before the call: full, or spread up to T."""
    B, T = case["B"], case["T"]
    room = case["n"] if case["op"] == "append" else 0
    if case["full"]:
        return [T - room] * B
    lens = [min(T, max(0 if case["op"].startswith("tree") else 1, T * (b + 1) // B - 29 * (B - 1 - b))) for b in range(B)]
    return [max(0, min(T - room, x)) for x in lens]


# ---------------------------------------------------------------- 8-bit values

def _quantise(x):
    """Codes (e4m3) and biased scale exponents of rows x [..., d]; a row with a NaN or an
    infinity gets the scale byte 255, which stands for NaN."""
    x = x.float()
    bad = ~torch.isfinite(x).all(-1)
    amax = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    m, k = torch.frexp(amax)
    e = torch.where(m <= 0.875, k - 9, k - 8).clamp(min=E_MIN)
    e = torch.where(amax > 0, e, torch.full_like(e, E_MIN))
    y = x * torch.exp2(-e.float()).unsqueeze(-1)
    y = torch.where(torch.isfinite(x), y, torch.zeros_like(y))
    top = torch.where(e == E_MAX, torch.full_like(amax, 240.0), torch.full_like(amax, 448.0)).unsqueeze(-1)
    y = torch.minimum(torch.maximum(y, -top), top)       # 256 2^120 would be no bf16 number
    return y.to(torch.float8_e4m3fn), torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def _values(code, scale):
    """fp32 values that codes [..., d] with scale exponents [...] stand for."""
    f = torch.where(scale == 255, torch.full_like(scale, math.nan, dtype=torch.float32), torch.exp2(scale.float() - 127.0))
    return code.float() * f.unsqueeze(-1)


# ---------------------------------------------------------------- inputs

def _tree(N, g):
    """Parents of a drafted tree in topological order: a chain that branches."""
    u = torch.rand(N, generator=g)
    back = 1 + (u * u * 4).long()                        # mostly the node before, sometimes an earlier one
    return (torch.arange(N) - back).clamp(min=-1).int()


def prepare(case, seed):
    dev = "cuda"
    B, Hq, Hkv, T, d, N, n = (case[k] for k in ("B", "Hq", "Hkv", "T", "d", "N", "n"))
    op, G, nt, nb = case["op"], Hq // Hkv, case["topics"], T // BLOCK
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    gc = torch.Generator()
    gc.manual_seed(seed)
    rn = lambda *s: torch.randn(*s, device=dev, generator=g)  # noqa: E731
    topics = 2.0 * rn(nt, d)
    s = {"case": case, "kv_len": torch.tensor(_lens(case), dtype=torch.int32, device=dev), "ws": None}
    # caches, one sequence at a time (the largest hold gigabytes)
    eight = op != "tree"
    kind = torch.float8_e4m3fn if eight else torch.bfloat16
    for name in ("k_cache", "v_cache"):
        s[name] = torch.empty(B, Hkv, T, d, dtype=kind, device=dev)
        if eight:
            s[name[0] + "_scale"] = torch.empty(B, Hkv, T, dtype=torch.uint8, device=dev)
    s["ksum"] = torch.zeros(B, Hkv, max(nb, 1), d, device=dev)
    for b in range(B):
        topic = torch.randint(0, nt, (nb + 1,), device=dev, generator=g).repeat_interleave(BLOCK)[:T]
        for name in ("k_cache", "v_cache"):
            x = rn(Hkv, T, d)
            if name == "k_cache":
                x += topics[topic]
            if eight:
                code, scale = _quantise(x)
                s[name][b], s[name[0] + "_scale"][b] = code, scale
                x = _values(code, scale) if name == "k_cache" else None
            else:
                x = s[name][b].copy_(x).float()
            if name == "k_cache" and nb:
                s["ksum"][b] = x[:, :nb * BLOCK].view(Hkv, nb, BLOCK, d).mean(2)
            del x
    if op in ("decode", "tree", "tree_q8"):
        head = torch.randint(0, nt, (B, Hq, 1), device=dev, generator=g).expand(B, Hq, N)
        other = torch.randint(0, nt, (B, Hq, N), device=dev, generator=g)
        # the drafted tokens continue one text: a head keeps its topic but for one node in eight
        pick = torch.where(torch.rand(B, Hq, N, device=dev, generator=g) < 0.125, other, head) if N > 1 else head
        q = (topics[pick] + rn(B, Hq, N, d)).bfloat16()
        s["q"] = q if op != "decode" else q[:, :, 0].contiguous()
    if op == "decode":
        s["kv_len"].clamp_(min=1)
    if op in ("tree", "tree_q8"):
        dt = torch.randint(0, nt, (B, 1, N), device=dev, generator=g)
        s["k_draft"] = (topics[dt] + rn(B, Hkv, N, d)).bfloat16()
        s["v_draft"] = rn(B, Hkv, N, d).bfloat16()
        s["parent"] = torch.stack([_tree(N, gc) for _ in range(B)]).to(dev)
    if op == "append":
        rows = max(n, N)
        # per-token sizes differ, and a few channels of the keys are large
        size = torch.exp(0.5 * rn(B, Hkv, rows, 1))
        chan = torch.where(torch.rand(Hkv, 1, d, device=dev, generator=g) < 0.03, 12.0, 1.0)
        s["k_new"] = (rn(B, Hkv, rows, d) * size * chan).bfloat16()
        s["v_new"] = (rn(B, Hkv, rows, d) * size).bfloat16()
        s["n_new"] = s["src"] = None
        if N > 1:
            s["src"] = torch.stack([torch.randperm(N, generator=gc)[:n].sort().values for _ in range(B)]).int().to(dev)
            s["n_new"] = torch.randint(0, n + 1, (B,), generator=gc).int().to(dev)
        s["after"] = s["kv_len"] + (s["n_new"] if N > 1 else n)
    if op == "read":
        s["start"] = (s["kv_len"] - n).clamp(min=0).int()
    return s


# ---------------------------------------------------------------- plain forms

def _entmax(x, alpha):
    """Weights of alpha-entmax over the last axis of x = (alpha - 1) scores (fp64; -inf: absent),
    alpha 1.5 or 2, from the sorted row's closed form; rows with nothing get zeros."""
    z, _ = torch.sort(x, dim=-1, descending=True)
    here = torch.isfinite(z)
    top = z[..., :1]
    y = torch.where(here, z - top, torch.zeros_like(z))
    k = torch.arange(1, x.shape[-1] + 1, device=x.device, dtype=x.dtype)
    s1 = torch.cumsum(y, -1)
    if alpha == 2.0:
        tau = (s1 - 1.0) / k
    else:
        mean = s1 / k
        tau = mean - ((1.0 - (torch.cumsum(y * y, -1) - k * mean * mean)) / k).clamp(min=0.0).sqrt()
    count = (here & (tau < y)).sum(-1, keepdim=True)
    tau = torch.gather(tau, -1, (count - 1).clamp(min=0))
    w = torch.where(torch.isfinite(x), (x - top - tau).clamp(min=0.0), torch.zeros_like(x))
    w = torch.where(count > 0, w, torch.zeros_like(w))
    return w if alpha == 2.0 else w * w


def _softmax_v(logit, v):
    """softmax over the last axis (rows with no key give zeros) times v."""
    top = logit.amax(-1, keepdim=True)
    e = torch.exp(logit - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    return torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_decode(s, k, v):
    c = s["case"]
    B, Hq, Hkv, T, d = (c[x] for x in ("B", "Hq", "Hkv", "T", "d"))
    G, nb = Hq // Hkv, T // BLOCK
    q = s["q"].float().view(B, Hkv, G, d)
    bt = ((s["kv_len"] - 1) // BLOCK).view(B, 1, 1, 1)
    j = torch.arange(nb, device=q.device)
    x = torch.matmul(q, s["ksum"][:, :, :nb].transpose(2, 3)).double() * ((c["alpha"] - 1.0) * COARSE / math.sqrt(d))
    p = _entmax(x.masked_fill(j >= bt, -math.inf), c["alpha"])
    logp = torch.log(p).float()
    logp = torch.where(j == bt, torch.zeros_like(logp), logp)
    logit = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d) + logp.repeat_interleave(BLOCK, -1)
    t = torch.arange(T, device=q.device)
    logit = logit.masked_fill(t >= s["kv_len"].view(B, 1, 1, 1), -math.inf)
    return _softmax_v(logit, v).view(B, Hq, d).bfloat16()


def _reach(parent):
    """[B, N, N]: whether the row's node is the column's node or descends from it; and depths."""
    N = parent.shape[1]
    at = torch.arange(N, device=parent.device)
    r = ((parent.unsqueeze(-1) == at) | (at.unsqueeze(-1) == at)).float()
    r = (torch.matmul(r, r) > 0).float()
    r = (torch.matmul(r, r) > 0).float()
    r = (torch.matmul(r, r) > 0).float()
    r = (torch.matmul(r, r) > 0).float()
    r = (torch.matmul(r, r) > 0).float()
    r = torch.matmul(r, r) > 0
    return r, r.sum(-1) - 1


def _plain_tree(s, k, v):
    c = s["case"]
    B, Hq, Hkv, T, d, N = (c[x] for x in ("B", "Hq", "Hkv", "T", "d", "N"))
    G, nb = Hq // Hkv, T // BLOCK
    dev = k.device
    q = s["q"].float().view(B, Hkv, G, N, d)
    L = s["kv_len"].view(B, 1, 1, 1, 1)
    F, r = L // BLOCK, L % BLOCK                          # full blocks, tokens of the open one
    reach, depth = _reach(s["parent"])                    # [B, N, N], [B, N]
    anc = reach.view(B, 1, 1, N, N)
    crossed = r + depth.view(B, 1, 1, N, 1) >= BLOCK      # the open block is complete and past for this node
    in_open = r + depth.view(B, 1, 1, 1, N) < BLOCK       # drafted token that lies in the open block
    lg = torch.matmul(q, k.unsqueeze(2).transpose(3, 4))  # [B, Hkv, G, N, T]
    ld = torch.matmul(q, s["k_draft"].float().unsqueeze(2).transpose(3, 4))
    t = torch.arange(T, device=dev)
    tail = (t >= F * BLOCK) & (t < L)
    # score of the open block where a node's path completes it: the mean over its 64 keys
    j = torch.arange(nb + 1, device=dev)
    cx = (c["alpha"] - 1.0) * COARSE / math.sqrt(d)
    total = lg.masked_fill(~tail, 0.0).sum(-1, keepdim=True) + ld.masked_fill(~(anc & in_open), 0.0).sum(-1, keepdim=True)
    x = torch.full((B, Hkv, G, N, nb + 1), -math.inf, dtype=torch.float64, device=dev)
    x[..., :nb] = torch.matmul(q, s["ksum"][:, :, :nb].unsqueeze(2).transpose(3, 4)).double() * cx
    x = x.masked_fill(j >= F, -math.inf)
    x = torch.where((j == F) & crossed, total.double() * (cx / BLOCK), x)
    p = _entmax(x, c["alpha"])
    logp = torch.log(p).float()
    open_logp = torch.where(crossed, torch.gather(logp, -1, F.expand(B, Hkv, G, N, 1).long()), torch.zeros_like(logp[..., :1]))
    logp = torch.where(j == F, open_logp, logp)
    lg = lg / math.sqrt(d) + logp.repeat_interleave(BLOCK, -1)[..., :T]
    lg = lg.masked_fill(t >= L, -math.inf)
    ld = ld / math.sqrt(d) + torch.where(crossed & in_open, open_logp, torch.zeros_like(open_logp))
    ld = ld.masked_fill(~anc, -math.inf)
    logit = torch.cat((lg, ld), -1)
    del lg, ld
    both = torch.cat((v, s["v_draft"].float()), 2).unsqueeze(2)
    return _softmax_v(logit, both).view(B, Hq, N, d).bfloat16()


def _plain_append(s):
    c = s["case"]
    B, Hkv, T, d, n = (c[x] for x in ("B", "Hkv", "T", "d", "n"))
    dev = s["k_new"].device
    i = torch.arange(n, device=dev)
    L = s["kv_len"].long().view(B, 1)
    new = s["n_new"].long().view(B, 1) if s["n_new"] is not None else torch.full((B, 1), n, device=dev)
    live = i < new
    src = s["src"].long() if s["src"] is not None else i.expand(B, n)
    b_at, i_at = live.nonzero(as_tuple=True)
    pos, row = (L + i)[b_at, i_at], src[b_at, i_at]
    back = []
    for x, cache, scale in ((s["k_new"], s["k_cache"], s["k_scale"]), (s["v_new"], s["v_cache"], s["v_scale"])):
        code, e = _quantise(x[b_at, :, row])              # [rows, Hkv, d]
        cache.view(torch.uint8)[b_at, :, pos] = code.view(torch.uint8)
        scale[b_at, :, pos] = e
        out = torch.zeros(B, Hkv, n, d, dtype=torch.bfloat16, device=dev)
        out[b_at, :, i_at] = _values(code, e).bfloat16()
        back.append(out)
    # summaries of the blocks that are now complete
    j = L // BLOCK + torch.arange((n + BLOCK - 1) // BLOCK + 1, device=dev)
    b_at, j_at = ((j + 1) * BLOCK <= L + new).nonzero(as_tuple=True)
    j_at = j[b_at, j_at]
    t = j_at.unsqueeze(-1) * BLOCK + torch.arange(BLOCK, device=dev)
    b_row = b_at.unsqueeze(-1)
    k = _values(s["k_cache"].view(torch.uint8)[b_row, :, t].view(s["k_cache"].dtype), s["k_scale"][b_row, :, t])
    s["ksum"][b_at, :, j_at] = k.mean(1)
    return back[0], back[1], s["ksum"]


def _plain_read(s):
    c = s["case"]
    B, T, n = c["B"], c["T"], c["n"]
    t = s["start"].long().view(B, 1) + torch.arange(n, device=s["start"].device)
    ok = (t < s["kv_len"].view(B, 1)).view(B, 1, n, 1)
    b_at, t = torch.arange(B, device=t.device).unsqueeze(-1), t.clamp(max=T - 1)
    out = []
    for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        x = _values(cache.view(torch.uint8)[b_at, :, t].view(cache.dtype), scale[b_at, :, t]).transpose(1, 2)
        out.append(torch.where(ok, x, torch.zeros_like(x)).bfloat16())
    return out


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from sparse_hierarchical_attention_pool_b200 import dash_attn as da
        kw = {"alpha": c["alpha"], "coarse_scale": COARSE}
        if op == "append":
            cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
            da.dash_cache_append(s["k_new"], s["v_new"], s["kv_len"], *cache, ksum=s["ksum"], n=c["n"], n_new=s["n_new"], src=s["src"])
            k, v = da.dash_cache_read(*cache, c["n"], start=s["kv_len"], kv_len=s["after"])
            return k, v, s["ksum"]
        if op == "read":
            return da.dash_cache_read(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], c["n"], start=s["start"], kv_len=s["kv_len"])
        if op == "decode":
            out, s["ws"] = da.dash_decode_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["ksum"], s["kv_len"], workspace=s["ws"], **kw)
            return out
        draft = (s["q"], s["k_draft"], s["v_draft"], s["parent"], s["k_cache"], s["v_cache"])
        if op == "tree":
            out, s["ws"] = da.dash_decode_tree(*draft, s["ksum"], s["kv_len"], workspace=s["ws"], **kw)
        else:
            out, s["ws"] = da.dash_decode_tree_q8(*draft, s["k_scale"], s["v_scale"], s["ksum"], s["kv_len"], workspace=s["ws"], **kw)
        return out
    if op == "append":
        return _plain_append(s)
    if op == "read":
        return _plain_read(s)
    if op == "tree":
        return _plain_tree(s, s["k_cache"].float(), s["v_cache"].float())
    k, v = _values(s["k_cache"], s["k_scale"]), _values(s["v_cache"], s["v_scale"])
    return _plain_decode(s, k, v) if op == "decode" else _plain_tree(s, k, v)


# ---------------------------------------------------------------- work

def work(case):
    """Each input row that the result depends on read once, each output written once.  The
    blocks of a KV group are those that its queries' topics select."""
    op, B, Hq, Hkv, T, d, N, n = (case[k] for k in ("op", "B", "Hq", "Hkv", "T", "d", "N", "n"))
    G = Hq // Hkv
    row = 2 * (d + 1) if op != "tree" else 4 * d          # K and V of one token in the cache
    if op == "append":
        done = sum((x + n) // BLOCK - x // BLOCK for x in _lens(case))
        open_rows = sum(x % BLOCK for x in _lens(case) if (x + n) // BLOCK > x // BLOCK)
        # rows in, codes and scales out, the open block's earlier keys, summaries, rows read back
        return {"bytes": B * Hkv * n * (4 * d + row + 4 * d) + Hkv * (open_rows * (d + 1) + done * 4 * d),
                "flops": B * Hkv * n * 6 * d}
    if op == "read":
        live = sum(min(n, x) for x in _lens(case))
        return {"bytes": Hkv * live * row + B * Hkv * n * 4 * d, "flops": Hkv * live * 2 * d}
    draws = G * (1.0 + 0.125 * (N - 1))                   # topics that a KV group's queries draw
    one = 1.0 / case["topics"]
    share = 1.0 - (1.0 - one) ** draws
    nbytes, flops = B * Hq * N * d * 4 + (B * Hkv * N * d * 4 if op != "decode" else 0), 0.0
    for x in _lens(case):
        past = max(x - 1, 0) // BLOCK if op == "decode" else x // BLOCK
        tail = max(x, 1) - past * BLOCK if op == "decode" else x % BLOCK
        nbytes += Hkv * (past * 4 * d + (share * past * BLOCK + tail) * row)
        flops += Hq * N * (2.0 * d * past + 4.0 * d * (one * past * BLOCK + tail + (N if op != "decode" else 0) / 2.0))
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------- 64 bits

def _exact_values(x):
    """fp64 values that the 8-bit cache holds for rows x: rounding on the e4m3 grid by hand."""
    x = x.double()
    mag = torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0).abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(mag.clamp(min=2.0 ** -140) / 448.0))
    e = torch.where(mag > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(mag <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(min=E_MIN)
    y = (x * torch.exp2(-e)).clamp(-448.0, 448.0)
    y = torch.where(e == E_MAX, y.clamp(-240.0, 240.0), y)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.where(torch.isfinite(x).all(-1, keepdim=True), torch.round(y / step) * step * torch.exp2(e), math.nan)


def _exact_threshold(x, alpha):
    lo = x.amax(-1, keepdim=True) - 1.0
    hi = lo + 1.0
    for _ in range(70):
        mid = 0.5 * (lo + hi)
        big = ((x - mid).clamp(min=0.0) ** (1.0 / (alpha - 1.0))).sum(-1, keepdim=True) >= 1.0
        lo, hi = torch.where(big, mid, lo), torch.where(big, hi, mid)
    return 0.5 * (lo + hi)


def _exact_row(q, keys, vals, marks, x, alpha):
    """One query row set q [R, d] over keys [M, d]: marks [R, M] holds each key's block index,
    -1 for prior 1 and -2 for a key that is not attended; x [R, nb] block values."""
    logit = q @ keys.T / math.sqrt(q.shape[-1])
    if x.shape[-1]:
        tau = _exact_threshold(x, alpha)
        logp = torch.log((x - tau).clamp(min=0.0)) / (alpha - 1.0)
        prior = torch.gather(logp, -1, marks.clamp(min=0))
        logit = torch.where(marks >= 0, logit + prior, logit)
    logit = torch.where(marks == -2, torch.full_like(logit, -math.inf), logit)
    return torch.softmax(logit, -1) @ vals


def exact(case, seed):
    op, B, Hq, Hkv, T, d, N, n = (case[k] for k in ("op", "B", "Hq", "Hkv", "T", "d", "N", "n"))
    s = prepare(case, seed)
    dev, G = s["kv_len"].device, Hq // Hkv
    lens = s["kv_len"].tolist()
    eight = op != "tree"

    def held(name, b, g, lo, hi):
        x = s[name + "_cache"][b, g, lo:hi].double()
        return x * torch.exp2(s[name + "_scale"][b, g, lo:hi].double() - 127.0).unsqueeze(-1) if eight else x

    if op in ("append", "read"):
        out = [torch.zeros(B, Hkv, n, d, dtype=torch.float64, device=dev) for _ in "kv"]
        if op == "read":
            for b in range(B):
                lo = int(s["start"][b])
                hi = min(lo + n, lens[b])
                for g in range(Hkv):
                    for o, name in zip(out, "kv"):
                        o[b, g, :hi - lo] = held(name, b, g, lo, hi)
            return out
        ksum = s["ksum"].double()
        for b in range(B):
            m = int(s["n_new"][b]) if s["n_new"] is not None else n
            rows = s["src"][b, :m].long() if s["src"] is not None else torch.arange(m, device=dev)
            for o, name in zip(out, "kv"):
                o[b, :, :m] = _exact_values(s[name + "_new"][b][:, rows])
            L = lens[b]
            for j in range(L // BLOCK, (L + m) // BLOCK):
                before = torch.stack([held("k", b, g, j * BLOCK, max(L, j * BLOCK)) for g in range(Hkv)])
                after = out[0][b, :, max(0, j * BLOCK - L):(j + 1) * BLOCK - L]
                ksum[b, :, j] = torch.cat((before, after), 1).mean(1)
        return [*out, ksum]
    nodes = N if op != "decode" else 1
    out = torch.zeros(B, Hq, nodes, d, dtype=torch.float64, device=dev)
    q = s["q"].double().view(B, Hkv, G, nodes, d)
    cx = (case["alpha"] - 1.0) * COARSE / math.sqrt(d)
    for b in range(B):
        L = lens[b]
        t = torch.arange(L, device=dev)
        full = (L - 1) // BLOCK if op == "decode" else L // BLOCK
        if op != "decode":
            parent = s["parent"][b].tolist()
            paths = []
            for i in range(N):
                paths.append((paths[parent[i]] if parent[i] >= 0 else []) + [i])
            depth = [len(p) - 1 for p in paths]
            anc = torch.zeros(N, N, dtype=torch.bool)
            for i, p in enumerate(paths):
                anc[i, p] = True
            anc, depth = anc.to(dev), torch.tensor(depth, device=dev)
        for g in range(Hkv):
            keys, vals = held("k", b, g, 0, L), held("v", b, g, 0, L)
            qq = q[b, g].reshape(G * nodes, d)
            x = qq @ s["ksum"][b, g, :full].double().T * cx
            block = t // BLOCK
            marks = torch.where(block >= full, torch.full_like(block, -1), block).expand(G * nodes, L)
            if op != "decode":
                kd, vd = s["k_draft"][b, g].double(), s["v_draft"][b, g].double()
                r = L - full * BLOCK
                crossed = (r + depth >= BLOCK).repeat(G)               # per row (head-major)
                low = (r + depth < BLOCK)
                mine = anc.repeat(G, 1)
                keys, vals = torch.cat((keys, kd)), torch.cat((vals, vd))
                dmark = torch.where(mine, torch.full((G * N, N), -1, device=dev), torch.full((G * N, N), -2, device=dev))
                marks = torch.cat((marks, dmark), 1)
                is_open = torch.cat((block >= full, low))
                swap = crossed.unsqueeze(-1) & is_open & (marks == -1)
                lg = qq @ keys.T
                mean = torch.where(swap, lg, torch.zeros_like(lg)).sum(-1, keepdim=True) / BLOCK * cx
                x = torch.cat((x, torch.where(crossed.unsqueeze(-1), mean, torch.full_like(mean, -math.inf))), 1)
                marks = torch.where(swap, torch.full_like(marks, full), marks)
                x = torch.where(torch.isfinite(x).any(-1, keepdim=True), x, torch.zeros_like(x))
            out[b, g * G:(g + 1) * G] = _exact_row(qq, keys, vals, marks, x, case["alpha"]).view(G, nodes, d)
    return out if op != "decode" else out[:, :, 0]
