"""The serving operators around a verify step, as cases to be timed.

Three kinds of case, by their "op":
  rules    spec_logit_rules: penalties, biases and grammar masks on target or draft rows
  history  spec_history_clear / spec_history_add: the token state that the penalties read
  kv       spec_kv_map / spec_kv_release: the paged cache's tables and slots for the lengths of a step

With `own` false a pass is computed in plain torch operations; with `own`
true it is the library's calls on the same tensors. Sizes are those of the
repository's five workloads and tests (vocabulary 151,936 and 50,257, blocks
of 16, 8 to 64 requests, a budget of half the slots), and generic cache sizes.
"""
import math

import numpy as np
import torch

own = False

V_LARGE, V_ODD = 151936, 50257
NEG = float("-inf")


# ------------------------------------------------------------------- cases

def listed():
    rules = dict(op="rules", K=1, packed=False, dtype="bf16", bias=0, mask="none", inplace=True)
    kv = dict(op="kv")
    return [
        # one request decoding one token, penalties only: the smallest call, all latency
        dict(rules, name="rules-decode-B1", rows="target", B=1, L=0, V=V_LARGE, hist=400),
        # plain decoding at high concurrency: long histories, biases, one row a request
        dict(rules, name="rules-decode-B256", rows="target", B=256, L=0, V=V_LARGE, hist=4000, bias=64),
        # the target rows of the stress workload after allocation: packed, ragged lengths, a third under a grammar
        dict(rules, name="rules-target-B64-packed", rows="target", B=64, L=16, V=V_LARGE, hist=4000, bias=64,
             packed=True, mask="some"),
        # the draft rows of the mixture workload: four branches a request, penalties and biases
        dict(rules, name="rules-draft-B32-K4", rows="draft", B=32, L=16, K=4, V=V_LARGE, hist=2000, bias=32),
        # structured output: every target row of every request under a grammar, nothing else
        dict(rules, name="rules-grammar-B32", rows="target", B=32, L=16, V=V_LARGE, hist=0, mask="all"),
        # raw logits kept for log-probabilities: written to a second tensor
        dict(rules, name="rules-copy-B32", rows="target", B=32, L=16, V=V_LARGE, hist=2000, mask="some", inplace=False),
        # fp32 rows of an odd vocabulary (no 16-byte rows), everything at once
        dict(rules, name="rules-f32-odd-B8", rows="target", B=8, L=5, V=V_ODD, hist=1000, bias=300, mask="some",
             inplace=False, dtype="f32"),
        # the tokens of one verify step enter the state
        dict(op="history", name="history-commit-B64", what="commit", B=64, L=16, V=V_LARGE),
        # a wave of new requests: seats cleared, prompts of up to 8192 tokens entered
        dict(op="history", name="history-admit-B32", what="admit", B=32, L=8192, V=V_LARGE),
        # one step of the stress workload: half the slots, pages of 16, rejected positions' pages returned
        dict(kv, name="kv-step-B64", what="cycle", B=64, L=16, page=16, ctx=4096),
        # a large serving batch with contexts up to 32k
        dict(kv, name="kv-step-B1024", what="cycle", B=1024, L=16, page=16, ctx=32768),
        # a prefill wave: whole prompts, all pages new
        dict(kv, name="kv-prefill-B32", what="prefill", B=32, L=8192, page=64, ctx=0),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rules", "rules", "rules", "history", "kv"])
    if op == "rules":
        rows = rng.choice(["target", "target", "draft"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        B, L = _log_int(rng, 1, 256), rng.randint(0, 16)
        V = rng.choice([_log_int(rng, 64, V_LARGE), 8 * _log_int(rng, 64, V_LARGE // 8), V_LARGE, V_ODD])
        K = 1
        if rows == "draft":
            L, K = max(L, 1), rng.choice([1, 2, 4])
        while B > 1 and B * K * (L + 1) * V * (4 if dtype == "f32" else 2) > 400e6:
            B = (B + 1) // 2
        mask = rng.choice(["none", "some", "all"])
        hist = rng.choice([0, _log_int(rng, 8, 16000), _log_int(rng, 8, 4000)])
        if mask == "none":
            hist = max(hist, 100)
        return dict(op=op, rows=rows, B=B, L=L, K=K, V=V, dtype=dtype, hist=hist, mask=mask,
                    bias=rng.choice([0, _log_int(rng, 1, 300)]) if hist else 0,
                    packed=rows == "target" and L > 0 and rng.random() < 0.5, inplace=rng.random() < 0.6)
    if op == "history":
        what = rng.choice(["commit", "admit"])
        L = rng.randint(1, 32) if what == "commit" else _log_int(rng, 16, 8192)
        return dict(op=op, what=what, B=_log_int(rng, 1, 64), L=L, V=rng.choice([_log_int(rng, 64, V_LARGE), V_LARGE]))
    what = rng.choice(["cycle", "cycle", "prefill"])
    if what == "prefill":
        return dict(op=op, what=what, B=_log_int(rng, 1, 32), L=_log_int(rng, 1, 8192),
                    page=rng.choice([16, 32, 64, 48]), ctx=0)
    B, ctx = _log_int(rng, 1, 1024), _log_int(rng, 16, 32768)
    return dict(op=op, what=what, B=B, L=rng.randint(0, 16), ctx=ctx,
                page=rng.choice([16, 32, 64, 48] if B * ctx > 1 << 20 else [1, 16, 32, 64, 48]))


# ------------------------------------------------------------------ inputs

class _Rng:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed * 2654435761 % (1 << 62) + 17)

    def rand(self, *shape):
        return torch.rand(shape, generator=self.g, device="cuda")

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda")

    def ints(self, lo, hi, *shape):  # lo <= x < hi
        return torch.randint(lo, hi, shape, generator=self.g, device="cuda")

    def perm(self, n):
        return torch.randperm(n, generator=self.g, device="cuda")

    def tokens(self, V, *shape):
        """Token ids with the frequencies of a vocabulary ordered by rank: log-uniform (Zipf) over the ids."""
        return (torch.pow(float(V), self.rand(*shape).double()).long() - 1).clamp_(0, V - 1)


def _pack_bits(bits):
    """[..., V] truth values -> [..., ceil(V / 32)] int32 words, bit v % 32 of word v // 32."""
    V = bits.shape[-1]
    W = (V + 31) // 32
    pad = torch.zeros(bits.shape[:-1] + (W * 32,), dtype=torch.bool, device=bits.device)
    pad[..., :V] = bits
    at = torch.arange(32, device=bits.device)
    return (pad.view(bits.shape[:-1] + (W, 32)).long() << at).sum(-1).int()


def _unpack_bits(words, V):
    at = torch.arange(32, device=words.device, dtype=torch.int32)
    return ((words[..., None] >> at) & 1).bool().flatten(-2)[..., :V]


def _lengths(r, B, L, budget):
    """Verify lengths of an allocation: the budget's best prefix products over survival scores; int32 [B]."""
    if L == 0:
        return torch.zeros(B, dtype=torch.int32, device="cuda")
    P = torch.cumprod(0.4 + 0.6 * r.rand(B, L).double(), dim=1).flatten()
    take = min(budget, B * (L + 1)) - B
    best = torch.argsort(P, descending=True, stable=True)[:take]
    return torch.bincount(best // L, minlength=B).int()


def _history_tables(r, S, V, n):
    """Counts and seen bits of seats with about n tokens each, three quarters of them prompt."""
    counts = torch.zeros(S, V, dtype=torch.int32, device="cuda")
    seen = torch.zeros(S, V, dtype=torch.bool, device="cuda")
    if n:
        live = r.rand(S, n) < 0.5 + 0.5 * r.rand(S, 1)
        prompt = torch.arange(n, device="cuda")[None, :] < (3 * n) // 4
        tok = r.tokens(V, S, n)
        seat = torch.arange(S, device="cuda")[:, None].expand(S, n)
        seen[seat[live], tok[live]] = True
        out = live & ~prompt
        counts.index_put_((seat[out], tok[out]), torch.ones((), dtype=torch.int32, device="cuda"), accumulate=True)
    return counts, _pack_bits(seen)


def _prepare_rules(c, r):
    B, L, K, V = c["B"], c["L"], c["K"], c["V"]
    R = L + 1 if c["rows"] == "target" else L
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    s = dict(c=c, R=R, len=None, row_off=None, tokens=r.tokens(V, B, L).int(), mask=None, mask_rows=None)
    n_rows = B * K * R
    if c["packed"]:
        n_rows = max(B, B * (L + 1) // 2)
        s["len"] = _lengths(r, B, L, n_rows)
        s["row_off"] = (torch.cumsum(s["len"] + 1, 0) - (s["len"] + 1)).int()
    x = torch.empty(n_rows, V, dtype=dt, device="cuda")
    for i in range(0, n_rows, 128):
        x[i:i + 128] = r.randn(min(128, n_rows - i), V) * 2.5
    s["x"] = x if c["packed"] else x.view(B, R, V) if c["rows"] == "target" else x.view(B, K, R, V)
    s["out"] = s["x"] if c["inplace"] else torch.zeros_like(s["x"])
    if c["hist"]:
        S = B + 3
        s["seats"] = r.perm(S)[:B].int()
        s["counts"], s["seen"] = _history_tables(r, S, V, c["hist"])
        s["repetition"], s["frequency"], s["presence"] = 1.0 + 0.3 * r.rand(S), 0.5 * r.rand(S), 0.5 * r.rand(S)
        s["bias_tokens"] = s["bias_values"] = None
        if c["bias"]:
            bt = r.ints(0, V, S, c["bias"])
            bt[r.rand(S, c["bias"]) < 0.1] = -1
            s["bias_tokens"], s["bias_values"] = bt.int(), r.randn(S, c["bias"]) * 3
    if c["mask"] != "none":
        # two of three masked rows allow a hundred tokens or so, the others nearly all
        use = torch.ones(B, dtype=torch.bool) if c["mask"] == "all" else torch.arange(B) % 3 == 0
        M = int(use.sum())
        words = torch.empty(M, R, (V + 31) // 32, dtype=torch.int32, device="cuda")
        for m in range(M):
            broad = r.rand(R, 1) < 1 / 3
            words[m] = _pack_bits(torch.where(broad, r.rand(R, V) > 0.02, r.rand(R, V) < min(0.5, 100.0 / V)))
        s["mask"] = words
        at = torch.full((B,), -1, dtype=torch.int32)
        at[use] = torch.arange(M, dtype=torch.int32)
        s["mask_rows"] = at.cuda()
    if own:
        import speculative_decoding_block_spec_b200 as specv
        s["history"] = None
        if c["hist"]:
            s["history"] = specv.History(s["counts"], s["seen"], s["repetition"], s["frequency"], s["presence"],
                                         s["bias_tokens"], s["bias_values"])
        s["ws"] = specv.Workspace(specv.rules_workspace_size(B))
    return s


def _prepare_history(c, r):
    B, L, V = c["B"], c["L"], c["V"]
    S = B + 3
    s = dict(c=c, V=V, seats=r.perm(S)[:B].int(), off=None)
    s["counts"], s["seen"] = _history_tables(r, S, V, 2000)
    if c["what"] == "commit":  # the out_tokens of a verify call: accepted prefix, terminal token, then -1
        n = r.ints(1, L + 2, B, 1)
        at = torch.arange(L + 1, device="cuda")[None, :]
        s["tokens"] = torch.where(at < n, r.tokens(V, B, L + 1), -1).int()
    else:
        n = r.ints(max(1, L // 16), L + 1, B)
        n[-1] = L
        s["off"] = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(n, 0)]).int()
        s["tokens"] = r.tokens(V, B * L).int()  # a buffer of fixed size: what is behind the last prompt is not read
    if own:
        import speculative_decoding_block_spec_b200 as specv
        s["history"] = specv.History(s["counts"], s["seen"])
        s["ws"] = specv.Workspace(specv.rules_workspace_size(B))
    return s


def _prepare_kv(c, r):
    B, L, ps = c["B"], c["L"], c["page"]
    S = B + 5
    if c["what"] == "prefill":
        N = B * max(L, 1)
        ctx = torch.zeros(B, dtype=torch.long, device="cuda")
        n = r.ints(max(1, L // 2), L + 1, B)
    else:
        N = max(B, B * (L + 1) // 2)
        ctx = r.ints(1, c["ctx"] + 1, B)
        n = _lengths(r, B, L, N).long() + 1
    most = (c["ctx"] + L + 1 + ps - 1) // ps + 1
    P = S * most
    seats = r.perm(S)[:B]
    free = r.perm(P).int()
    s = dict(c=c, N=N, P=P, most=most, seats=seats.int(), ctx=ctx.int())
    s["off"] = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(n, 0)]).int()
    s["keep"] = (ctx if c["what"] == "prefill" else ctx + torch.minimum(n, r.ints(1, L + 2, B))).int()
    # each request holds the pages of its context; the others are free
    owned = torch.zeros(S, dtype=torch.long, device="cuda")
    owned[seats] = (ctx + ps - 1) // ps
    end = torch.cumsum(owned, 0)
    at = torch.arange(most, device="cuda")[None, :]
    table = torch.full((S, most), -1, dtype=torch.int32, device="cuda")
    rank = (end - owned)[:, None] + at
    table = torch.where(at < owned[:, None], free[P - 1 - rank.clamp_(max=P - 1)], table)
    s["owned"], s["page_table"], s["free"] = owned.int(), table, free
    s["free_count"] = (P - end[-1:]).int()
    s["slots"] = torch.empty(N, dtype=torch.int64, device="cuda")
    s["positions"] = torch.empty(N, dtype=torch.int32, device="cuda")
    s["seq_len"] = torch.empty(B, dtype=torch.int32, device="cuda")
    s["block_table"] = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    if own:
        import speculative_decoding_block_spec_b200 as specv
        s["pages"] = specv.KvPages(s["page_table"], s["owned"], s["free"], s["free_count"], ps)
        s["ws"] = specv.Workspace(specv.kv_workspace_size(B))
    return s


def prepare(case, seed):
    r = _Rng(int(seed))
    return {"rules": _prepare_rules, "history": _prepare_history, "kv": _prepare_kv}[case["op"]](case, r)


# ------------------------------------------------------------------ passes

def _row_index(s):
    """(request, position, valid) of every row of the logits, flat."""
    c, R = s["c"], s["R"]
    B, K = c["B"], c["K"]
    if c["packed"]:
        at = torch.arange(s["x"].shape[0], device="cuda", dtype=torch.int32)
        b = torch.searchsorted(s["row_off"], at, right=True) - 1
        i = at - s["row_off"][b]
        return b, i.long(), i <= s["len"][b]
    b = torch.arange(B, device="cuda")[:, None, None].expand(B, K, R).flatten()
    i = torch.arange(R, device="cuda")[None, None, :].expand(B, K, R).flatten()
    return b, i, torch.ones_like(b, dtype=torch.bool)


def _plain_rules(s):
    c = s["c"]
    V = c["V"]
    b, i, valid = _row_index(s)
    x = s["x"].reshape(-1, V).float()
    z = x
    if c["hist"]:
        seat = s["seats"].long()[b]
        k = torch.arange(c["L"], device="cuda")[None, :]
        inside = (k < i[:, None]).int()
        prefix = torch.zeros(x.shape, dtype=torch.int32, device="cuda")
        prefix.scatter_add_(1, s["tokens"].long()[b], inside)
        count = s["counts"][seat] + prefix
        seen = _unpack_bits(s["seen"][s["seats"].long()], V)[b] | (prefix > 0)
        rep = s["repetition"][seat][:, None]
        z = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
        z = z - s["frequency"][seat][:, None] * count - s["presence"][seat][:, None] * (count > 0)
        if c["bias"]:
            bt = s["bias_tokens"][s["seats"].long()].long()
            bv = torch.where(bt >= 0, s["bias_values"][s["seats"].long()], 0.0)
            dense = torch.zeros(c["B"], V, device="cuda").scatter_add_(1, bt.clamp(min=0), bv)
            z = z + dense[b]
    if c["mask"] != "none":
        m = s["mask_rows"].long()[b]
        allowed = _unpack_bits(s["mask"], V)[m.clamp(min=0), i.clamp(max=s["R"] - 1)] | (m < 0)[:, None]
        z = z.masked_fill(~allowed, NEG)
    out = s["out"].view(-1, V)
    out.copy_(torch.where(valid[:, None], z.to(out.dtype), out))
    return s["out"]


def _own_rules(s):
    import speculative_decoding_block_spec_b200 as specv
    return specv.spec_logit_rules(s["x"], s["history"], seats=s.get("seats"), draft_tokens=s["tokens"],
                                  verify_len=s["len"], target_row_off=s["row_off"], mask=s["mask"],
                                  mask_rows=s["mask_rows"], out=s["out"], workspace=s["ws"])


def _plain_history(s):
    counts, seen, V = s["counts"], s["seen"], s["V"]
    seats, tok = s["seats"].long(), s["tokens"].long()
    if s["c"]["what"] == "commit":
        seat = seats[:, None].expand(tok.shape)
        use = tok >= 0
        counts.index_put_((seat, tok.clamp(min=0)), use.int(), accumulate=True)
    else:
        counts[seats] = 0
        seen[seats] = 0
        at = torch.arange(tok.shape[0], device="cuda", dtype=torch.int32)
        use = at < s["off"][-1]
        seat = seats[(torch.searchsorted(s["off"], at, right=True) - 1).clamp(max=seats.shape[0] - 1)]
    bits = torch.zeros(counts.shape[0], V, dtype=torch.int32, device="cuda")
    bits.index_put_((seat, tok.clamp(min=0)), use.int(), accumulate=True)
    seen |= _pack_bits(bits > 0)
    return {"counts": counts, "seen": seen}


def _own_history(s):
    import speculative_decoding_block_spec_b200 as specv
    h = s["history"]
    if s["c"]["what"] == "commit":
        specv.spec_history_add(h, s["tokens"], seats=s["seats"], output=True, workspace=s["ws"])
    else:
        specv.spec_history_clear(h, s["seats"], workspace=s["ws"])
        specv.spec_history_add(h, s["tokens"], offsets=s["off"], seats=s["seats"], output=False, workspace=s["ws"])
    return {"counts": s["counts"], "seen": s["seen"]}


def _plain_kv_map(s):
    ps, N, P, most = s["c"]["page"], s["N"], s["P"], s["most"]
    seats, ctx, off = s["seats"].long(), s["ctx"].long(), s["off"].long()
    total = ctx + off[1:] - off[:-1]
    pages = (total + ps - 1) // ps
    owned = s["owned"].long()[seats]
    fits = pages <= most
    need = torch.where(fits, (pages - owned).clamp(min=0), 0)
    end = torch.cumsum(need, 0)
    fc = s["free_count"].long()
    ok = fits & ((need == 0) | (end <= fc))
    at = torch.arange(most, device="cuda")[None, :]
    rank = (end - need)[:, None] + at - owned[:, None]
    new = (at >= owned[:, None]) & (at < pages[:, None]) & ok[:, None]
    table = torch.where(new, s["free"][(fc - 1 - rank).clamp(0, P - 1)], s["page_table"][seats])
    s["page_table"][seats] = table
    s["owned"][seats] = torch.where(ok, torch.maximum(owned, pages), owned).int()
    s["block_table"].copy_(torch.where((at < pages[:, None]) & ok[:, None], table, s["block_table"]))
    s["seq_len"].copy_(torch.where(ok, total, -1).int())
    s["free_count"] -= torch.where(ok, need, 0).sum().int()
    t = torch.arange(N, device="cuda")
    b = (torch.searchsorted(off, t, right=True) - 1).clamp(max=off.shape[0] - 2)
    pos = ctx[b] + t - off[b]
    live = (t < off[-1]) & ok[b]
    page = table[b, (pos // ps).clamp(max=most - 1)].long()
    s["slots"].copy_(torch.where(live, page * ps + pos % ps, -1))
    s["positions"].copy_(torch.where(live, pos, 0).int())


def _plain_kv_release(s):
    ps, P, most = s["c"]["page"], s["P"], s["most"]
    seats = s["seats"].long()
    owned = s["owned"].long()[seats]
    kept = torch.minimum(owned, (s["keep"].long() + ps - 1) // ps)
    n = owned - kept
    end = torch.cumsum(n, 0)
    at = torch.arange(most, device="cuda")[None, :]
    gone = (at >= kept[:, None]) & (at < owned[:, None])
    table = s["page_table"][seats]
    to = torch.where(gone, s["free_count"].long() + (end - n)[:, None] + at - kept[:, None], P)
    stack = torch.cat([s["free"], s["free"][:1]])
    stack[to.flatten()] = table.flatten()
    s["free"].copy_(stack[:P])
    s["page_table"][seats] = torch.where(gone, -1, table)
    s["owned"][seats] = kept.int()
    s["free_count"] += n.sum().int()


def _plain_kv(s):
    _plain_kv_map(s)
    _plain_kv_release(s)


def _own_kv(s):
    import speculative_decoding_block_spec_b200 as specv
    specv.spec_kv_map(s["pages"], s["ctx"], s["off"], s["N"], seats=s["seats"], block_table=s["block_table"],
                      out=(s["slots"], s["positions"], s["seq_len"]), workspace=s["ws"])
    specv.spec_kv_release(s["pages"], s["seats"], keep_len=s["keep"], workspace=s["ws"])


def run(state):
    op = state["c"]["op"]
    if op == "rules":
        return _own_rules(state) if own else _plain_rules(state)
    if op == "history":
        return _own_history(state) if own else _plain_history(state)
    if own:
        _own_kv(state)
    else:
        _plain_kv(state)
    return {k: state[k] for k in ("slots", "positions", "seq_len", "block_table", "page_table", "owned", "free",
                                  "free_count")}


# -------------------------------------------------------------------- work

def _distinct(V, n):
    """Expected number of distinct tokens among n log-uniform ones."""
    if n <= 0:
        return 0.0
    p = np.log1p(1.0 / np.arange(1, V + 1)) / math.log(V)
    return float(np.sum(-np.expm1(n * np.log1p(-np.minimum(p, 1 - 1e-12)))))


def work(case):
    c = case
    if c["op"] == "rules":
        B, L, K, V = c["B"], c["L"], c["K"], c["V"]
        es = 2 if c["dtype"] == "bf16" else 4
        R = L + 1 if c["rows"] == "target" else L
        rows = max(B, B * (L + 1) // 2) if c["packed"] else B * K * R
        d = _distinct(V, 0.75 * c["hist"])
        edits = rows * (d + 0.9 * c["bias"] + R / 2) if c["hist"] else 0
        words = B * V / 8 if c["hist"] else 0
        masked = {"none": 0, "some": 1 / 3, "all": 1}[c["mask"]] * rows
        n = words + B * d * 4 + B * c["bias"] * 8 + masked * V / 8 + B * L * 4
        if c["inplace"]:
            n += edits * 2 * es + masked * (2 / 3 + 0.02 / 3) * V * es
        else:
            n += 2 * rows * V * es
        return {"bytes": n, "flops": 5 * edits + masked * V}
    if c["op"] == "history":
        if c["what"] == "commit":
            n = c["B"] * (c["L"] + 2) / 2
            return {"bytes": n * (4 + 2 * 4 + 2 * 4), "flops": 0}
        n = c["B"] * c["L"] * 0.53
        d = _distinct(c["V"], c["L"] * 0.53)
        return {"bytes": n * 4 + 2 * c["B"] * (c["V"] / 8 + d * 4), "flops": 0}
    B, L, ps = c["B"], c["L"], c["page"]
    N = B * max(L, 1) if c["what"] == "prefill" else max(B, B * (L + 1) // 2)
    tokens = N * (0.75 if c["what"] == "prefill" else 1)
    pages = B * ((c["ctx"] / 2 + tokens / B) / ps + 1)
    new = tokens / ps
    return {"bytes": N * (8 + 4) + pages * 8 + new * 16 + B * 4 * 8, "flops": 0}


# ------------------------------------------------------- 64-bit definition

def exact(case, seed):
    """What a pass over `rules` returns, in 64 bits, token by token from the rule; whole numbers have no such value."""
    if case["op"] != "rules":
        return None
    if work(case)["flops"] / 5 > 6e6 and case["mask"] == "none" or case["B"] * case["L"] * case["hist"] > 8e6:
        return None
    s = prepare(case, seed)
    c, R, V = case, s["R"], case["V"]
    y = s["x"].reshape(-1, V).double()
    touched = torch.zeros(y.shape[0], dtype=torch.bool)
    lens = s["len"].tolist() if c["packed"] else None
    first = s["row_off"].tolist() if c["packed"] else None
    seats = s["seats"].tolist() if c["hist"] else None
    drafts = s["tokens"].tolist()
    masks = s["mask_rows"].tolist() if c["mask"] != "none" else None
    lane = torch.arange(V, device="cuda")
    for b in range(c["B"]):
        if c["packed"]:
            rows = [(first[b] + i, i) for i in range(lens[b] + 1)]
        else:
            rows = [((b * c["K"] + z) * R + i, i) for z in range(c["K"]) for i in range(R)]
        if c["hist"]:
            q = seats[b]
            seen0 = torch.nonzero((s["seen"][q, lane // 32] >> (lane % 32)) & 1).flatten().tolist()
            n0 = s["counts"][q].tolist()
            r, f, p = (float(s[k][q]) for k in ("repetition", "frequency", "presence"))
            add = {}
            if c["bias"]:
                for t, a in zip(s["bias_tokens"][q].tolist(), s["bias_values"][q].tolist()):
                    if t >= 0:
                        add[t] = add.get(t, 0.0) + a
        base = {}
        for row, i in rows:
            touched[row] = True
            if c["hist"]:
                if i not in base:
                    more = {}
                    for t in drafts[b][:i]:
                        more[t] = more.get(t, 0) + 1
                    known = set(seen0) | set(more)
                    ids = sorted(known | set(add))
                    n = [n0[t] + more.get(t, 0) for t in ids]
                    base[i] = [torch.tensor(v, dtype=torch.float64, device="cuda") for v in (
                        [r if t in known else 1.0 for t in ids],
                        [f * m + (p if m > 0 else 0.0) for m in n], [add.get(t, 0.0) for t in ids])]
                    base[i].append(torch.tensor(ids, dtype=torch.long, device="cuda"))
                rr, minus, plus, ids = base[i]
                v = y[row, ids]
                y[row, ids] = torch.where(v > 0, v / rr, v * rr) - minus + plus
            if masks is not None and masks[b] >= 0:
                ok = (s["mask"][masks[b], i][lane // 32] >> (lane % 32)) & 1
                y[row, ok == 0] = NEG
    start = s["out"].reshape(-1, V).double()
    return torch.where(touched.cuda()[:, None], y, start).view(s["out"].shape)
