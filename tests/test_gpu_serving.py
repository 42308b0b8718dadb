"""Serving operators on the GPU against the plain 64-bit definitions
(oracle/serving.py).

Tolerance of an edited logit. The kernel computes
z = x fl(1 / r) - (f c + p) + bias in fp32. Each of its at most 5 + n_b
operations (n_b bias entries of one token, 7 at most here) rounds a value no
larger than S = |x / r or x r| + |f| c + |p| + sum |bias|, by 2^-24 of it; the
parameters are the same fp32 numbers on both sides. So |z_gpu - z| <= E =
12 * 2^-24 * S, and the final rounding adds half a step of the type, 2^-8
(bf16) or 0 (fp32: z is already fp32) of |z| + E. Elements that no rule names
must keep their bits. Whole numbers (counts, bits, slots, tables) are equal.
"""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_block_spec_b200 as specv
from oracle import serving as plain
from speculative_decoding_block_spec_b200 import synth
from speculative_decoding_block_spec_b200.synth import f32_to_bf16_bits

from parity_util import check_verify, logits_to_torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]
I32 = torch.int32


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def words(a):
    return dev(np.ascontiguousarray(a).view(np.int32))


def host(t):
    """bf16 as bit patterns, else as is."""
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16).cpu().numpy().view(np.uint16)
    return t.cpu().numpy()


def to_type(x, dtype):
    return f32_to_bf16_bits(x) if dtype == "bf16" else x.astype(np.float32)


class Case:
    """Random rows, histories, penalties, biases and masks of one call."""

    def __init__(self, seed, B, K, L, V, *, rows, dtype="bf16", packed=False, hist=50, bias=0, mask=None, seats=True,
                 vlen=True, params=True):
        g = np.random.default_rng(seed)
        self.B, self.K, self.L, self.V, self.rows, self.dtype = B, K, L, V, rows, dtype
        self.vlen = g.integers(0, L + 1, B).astype(np.int32) if vlen else None
        self.row_off, n = None, B * K * rows
        if packed:
            ln = (self.vlen if vlen else np.full(B, L)) + 1
            self.row_off = (np.cumsum(ln) - ln + 1).astype(np.int32)  # a row before the first: must stay as it was
            n = int(ln.sum()) + 3
        self.x = to_type(g.standard_normal((n, V)).astype(np.float32) * 3, dtype)
        self.tokens = g.integers(0, min(V, 40), (B, L)).astype(np.int32)  # few ids: repeats, also of seen tokens
        self.kw, self.seats = {}, None
        if hist is not None:
            S = B + 3
            if seats:
                self.seats = g.permutation(S)[:B].astype(np.int32)
                if B > 2:
                    self.seats[1], self.seats[2] = -1, self.seats[0]  # no seat; one seat read by two requests
            counts = np.zeros((S, V), np.int32)
            seen = np.zeros((S, V), bool)
            for s in range(S):
                ids = g.integers(0, V, hist) if s % 2 else g.integers(0, min(V, 3 * hist + 1), hist)
                seen[s, ids] = True
                np.add.at(counts[s], ids[: hist // 2], 1)
            counts[0, ids[:1]], seen[0, ids[:1]] = 70000, True
            self.kw.update(counts=counts, seen=plain.pack_bits(seen))
            if params:
                self.kw.update(repetition=g.uniform(0.7, 1.5, S).astype(np.float32),
                               frequency=g.uniform(-0.5, 1, S).astype(np.float32),
                               presence=g.uniform(-0.5, 1, S).astype(np.float32))
            if bias:
                bt = g.integers(0, V, (S, bias)).astype(np.int32)
                bt[:, bias // 2] = bt[:, 0]              # one token twice
                bt[g.random((S, bias)) < 0.1] = -1
                self.kw.update(bias_tokens=bt, bias_values=(g.standard_normal((S, bias)) * 4).astype(np.float32))
        self.mask = self.mask_rows = None
        if mask:
            M = B if mask == "own" else max(1, B // 2)
            ok = g.random((M, rows + 1, V)) < g.choice([0.01, 0.5, 0.99], (M, rows + 1, 1))
            ok[0, 0] = False                             # a row that allows nothing
            ok[-1, -1] = True
            self.mask = plain.pack_bits(ok)
            if V % 32:                                   # bits past V mean nothing
                self.mask[..., -1] |= np.uint32(0xffffffff << (V % 32) & 0xffffffff)
            if mask != "own":
                self.mask_rows = g.integers(-1, M, B).astype(np.int32)

    def oracle(self):
        return plain.logit_rules(self.x, self.B, self.K, self.rows, self.L, row_off=self.row_off, tokens=self.tokens,
                                 verify_len=self.vlen, seats=self.seats, mask=self.mask, mask_rows=self.mask_rows,
                                 **self.kw)

    def history(self):
        k = self.kw
        if not k:
            return None
        return specv.History(dev(k["counts"]), words(k["seen"]), dev(k.get("repetition")), dev(k.get("frequency")),
                             dev(k.get("presence")), dev(k.get("bias_tokens")), dev(k.get("bias_values")))

    def view(self, t):
        return t if self.row_off is not None else t.view(self.B, self.K, self.rows, self.V)

    def call(self, x, out=None, **kw):
        args = dict(seats=dev(self.seats), draft_tokens=dev(self.tokens), verify_len=dev(self.vlen),
                    target_row_off=dev(self.row_off), mask=None if self.mask is None else words(self.mask),
                    mask_rows=dev(self.mask_rows), out=out)
        args.update(kw)
        return specv.spec_logit_rules(x, self.history(), **args)


def check_rows(got, x, ref, dtype, before=None):
    """got, x: host rows; before: what the rows that are not processed hold."""
    before = x if before is None else before
    done = ref["done"]
    np.testing.assert_array_equal(got[~done], before[~done])
    keep = done[:, None] & ~ref["touched"]
    np.testing.assert_array_equal(got[keep], x[keep])
    z, y = ref["z"], plain.widen(got)
    edit = done[:, None] & ref["touched"]
    e = 12 * 2.0 ** -24 * ref["size"]
    h = 2.0 ** -8 if dtype == "bf16" else 0.0
    fine = edit & np.isfinite(z)
    with np.errstate(invalid="ignore"):
        bound = h * (np.abs(z) + e) + e
    bad = np.abs(y[fine] - z[fine]) > bound[fine]
    assert not bad.any(), (z[fine][bad][:5], y[fine][bad][:5])
    np.testing.assert_array_equal(y[edit & ~np.isfinite(z)], z[edit & ~np.isfinite(z)])


SHAPES = [
    dict(B=1, K=1, L=0, V=64, rows=1),
    dict(B=3, K=1, L=0, V=1, rows=1, hist=1),
    dict(B=5, K=1, L=0, V=1025, rows=1, bias=3),
    dict(B=3, K=1, L=4, V=257, rows=5, bias=7, mask="own"),
    dict(B=3, K=1, L=4, V=1000, rows=5, bias=1, mask="some"),
    dict(B=3, K=1, L=4, V=1001, rows=5, packed=True, bias=5, mask="some", hist=900),
    dict(B=4, K=3, L=5, V=4096, rows=5, bias=40, mask="some", hist=4000),
    dict(B=4, K=2, L=5, V=4095, rows=6, bias=40, mask="some"),          # branches of target rows
    dict(B=2, K=8, L=3, V=2048, rows=3, mask="own", hist=None),
    dict(B=2, K=1, L=32, V=300, rows=33, bias=20, hist=200),
    dict(B=2, K=1, L=32, V=8192, rows=33, packed=True, mask="own", hist=8000),
    dict(B=2, K=1, L=2, V=50257, rows=3, bias=300, mask="own", hist=3000),
    dict(B=3, K=1, L=2, V=65536, rows=3, bias=1024, hist=30, seats=False, vlen=False),
    dict(B=2, K=1, L=1, V=151936, rows=2, bias=64, mask="some", hist=5000),
    dict(B=6, K=1, L=2, V=640, rows=3, bias=6, params=False),           # NULL penalties: biases alone
    dict(B=2, K=1, L=3, V=200000, rows=4, bias=200, mask="own", hist=6000),     # more than one tile of the vocabulary
    dict(B=1, K=2, L=2, V=1 << 20, rows=2, bias=30, hist=3000, vlen=False),                 # the largest vocabulary
    dict(B=40, K=1, L=8, V=1500, rows=9, bias=5, mask="some"),
    dict(B=30, K=4, L=4, V=16384, rows=4, hist=300, mask="some"),       # many long rows: copied and edited in one kernel
    dict(B=64, K=1, L=7, V=16391, rows=8, packed=True, bias=9, mask="own"),
    dict(B=1, K=1, L=1, V=20000, rows=2, bias=5, hist=60000, vlen=False),                   # nearly every token seen: several rounds
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", range(len(SHAPES)))
def test_rules_match_the_definition(n, dtype):
    c = Case(100 + n, dtype=dtype, **SHAPES[n])
    ref = c.oracle()
    assert ref["flags"] == 0 and ref["done"].any()
    ws = specv.Workspace(specv.rules_workspace_size(c.B))
    x = c.view(logits_to_torch(c.x))
    y = c.view(logits_to_torch(to_type(np.full(c.x.shape, 7.0, np.float32), dtype)))
    before = host(y).reshape(c.x.shape).copy()
    assert c.call(x, out=y, workspace=ws) is y
    check_rows(host(y).reshape(c.x.shape), c.x, ref, dtype, before)
    np.testing.assert_array_equal(host(x).reshape(c.x.shape), c.x)      # out of place: the input stays
    assert c.call(x, workspace=ws) is x
    check_rows(host(x).reshape(c.x.shape), c.x, ref, dtype)
    np.testing.assert_array_equal(host(x)[..., :], host(torch.where(torch.from_numpy(ref["done"]).cuda().view(
        x.shape[:-1] + (1,)), y, x))) if c.row_off is None else None    # both forms give the same bits
    assert ws.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 3])
def test_rules_on_rows_at_odd_addresses(dtype, shift):
    """V keeps 16-byte rows, the buffers' addresses do not."""
    c = Case(7, 3, 1, 4, 1024, rows=5, dtype=dtype, bias=9, mask="own")
    ref = c.oracle()
    n = c.x.size
    for out_shift in (None, shift, 0, 2):
        big = logits_to_torch(np.concatenate([c.x.ravel()[:shift], c.x.ravel(), c.x.ravel()[:4]]))
        x = big[shift:shift + n].view(c.B, 1, c.rows, c.V)
        if out_shift is None:
            c.call(x)
            check_rows(host(x).reshape(c.x.shape), c.x, ref, dtype)
        else:
            buf = torch.full((n + 8,), 5.0, dtype=x.dtype, device="cuda")
            y = buf[out_shift:out_shift + n].view(x.shape)
            before = host(y).reshape(c.x.shape).copy()
            c.call(x, out=y)
            check_rows(host(y).reshape(c.x.shape), c.x, ref, dtype, before)
            assert torch.all(buf[:out_shift] == 5.0) and torch.all(buf[out_shift + n:] == 5.0)
        assert torch.equal(big[:shift].float().cpu(), torch.from_numpy(
            plain.widen(c.x.ravel()[:shift])).float())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [4096, 5000, 4097])
def test_masks_keep_the_bits_of_what_they_allow(V, dtype):
    """Rows under masks that allow a few, some, half and nearly all tokens, NaN payloads among the allowed: every
    allowed element keeps its bits, in place and in the copy."""
    g = np.random.default_rng(V)
    B, R = 5, 3
    x = to_type(g.standard_normal((B * R, V)).astype(np.float32), dtype)
    if dtype == "bf16":
        x[:, ::5] = 0x7f81 + (np.arange(x[:, ::5].shape[1]) % 100).astype(np.uint16)
    else:
        x.view(np.uint32)[:, ::5] = 0x7f800001 + np.arange(x[:, ::5].shape[1], dtype=np.uint32)
    ok = g.random((B, R, V)) < np.array([0.0005, 0.02, 0.5, 0.97, 0.9995])[:, None, None]
    ok[0, 1], ok[4, 1] = False, True
    ok[0, 2] = False
    ok[0, 2, [0, 1, 33, 1023, 1024, 2047, V - 1]] = True
    want = np.where(ok.reshape(B * R, V), x, to_type(np.full(1, -np.inf, np.float32), dtype))
    words_ = words(plain.pack_bits(ok))
    t = logits_to_torch(x).view(B, R, V)
    y = torch.zeros_like(t)
    specv.spec_logit_rules(t, mask=words_, out=y)
    specv.spec_logit_rules(t, mask=words_)
    for got in (y, t):
        got = host(got).reshape(B * R, V)
        np.testing.assert_array_equal(got.view(np.uint32 if dtype == "f32" else np.uint16),
                                      want.view(np.uint32 if dtype == "f32" else np.uint16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rules_on_infinities_and_nan(dtype):
    c = Case(11, 2, 1, 2, 300, rows=3, dtype=dtype, hist=150, bias=4, mask="own", vlen=False, seats=False)
    x = plain.widen(c.x).astype(np.float32)
    x[:, ::7], x[:, 1::7], x[:, 2::7] = -np.inf, np.nan, np.inf
    x[:, 3::7] = np.finfo(np.float32).min if dtype == "f32" else -3.3895314e38
    c.x = to_type(x, dtype)
    c.kw["repetition"][:] = 1.25                      # the lowest value times r: -inf in fp32
    ref = c.oracle()
    with np.errstate(over="ignore"):
        z32 = ref["z"].astype(np.float32).astype(np.float64)
    y = logits_to_torch(c.x).view(2, 1, 3, 300)
    c.call(y)
    got = plain.widen(host(y).reshape(c.x.shape))
    edit = ref["touched"] & ref["done"][:, None]
    np.testing.assert_array_equal(np.isnan(got[edit]), np.isnan(z32[edit]))
    allowed = plain.bits_of(c.mask, 300)[:, :3].reshape(-1, 300)
    assert np.all(got[~allowed] == -np.inf)           # NaN and +inf under the mask too
    # near the type's limit a rounding decides between the largest value and infinity: compared away from it
    far = edit & (np.abs(z32) < 1e38)
    e = 12 * 2.0 ** -24 * ref["size"]
    h = 2.0 ** -8 if dtype == "bf16" else 0.0
    with np.errstate(invalid="ignore"):
        assert np.all(np.abs(got[far] - z32[far]) <= (h * (np.abs(z32) + e) + 2 * e)[far])
    inf = edit & np.isinf(z32) & (np.isinf(x) | (np.abs(ref["z"]) > 3.5e38))
    np.testing.assert_array_equal(got[inf], z32[inf])


def test_rules_leave_out_what_they_cannot_do():
    base = dict(B=5, K=1, L=3, V=700, rows=4, dtype="f32", bias=5, mask="some")

    def run(change, want, packed=False):
        c = Case(21, packed=packed, **base)
        c.seats, c.mask_rows = np.arange(5, dtype=np.int32), np.array([0, 1, -1, 1, 0], np.int32)
        change(c)
        ref = c.oracle()
        assert ref["flags"] == want
        for inplace in (True, False):
            ws = specv.Workspace(256)
            x = c.view(logits_to_torch(c.x))
            y = x if inplace else torch.full_like(x, 3.0)
            before = host(y).reshape(c.x.shape).copy()
            c.call(x, out=y, workspace=ws)
            check_rows(host(y).reshape(c.x.shape), c.x, ref, "f32", before)
            assert ws.status() == want

    def put(name, at, value):
        return lambda c: c.kw[name].__setitem__(at, value)

    run(lambda c: c.vlen.__setitem__(2, 4), specv.DEV_VERIFY_LEN)
    run(lambda c: c.vlen.__setitem__(2, -1), specv.DEV_VERIFY_LEN)
    run(lambda c: c.seats.__setitem__(1, 8), specv.DEV_INDEX)
    run(lambda c: c.mask_rows.__setitem__(3, 2), specv.DEV_INDEX)
    for v in (0.0, -1.0, np.nan, np.inf, 1e-38, 1e38):
        run(put("repetition", 3, v), specv.DEV_PARAM)
    run(put("frequency", 0, np.nan), specv.DEV_PARAM)
    run(put("presence", 4, -np.inf), specv.DEV_PARAM)
    run(lambda c: (c.vlen.fill(3), c.tokens.__setitem__((1, 0), 700), c.tokens.__setitem__((2, 1), -5)), specv.DEV_TOKEN_RANGE)
    run(lambda c: c.kw["bias_tokens"].__setitem__((2, 1), 700), specv.DEV_TOKEN_RANGE)
    run(lambda c: c.row_off.__setitem__(0, -1), specv.DEV_INDEX, packed=True)
    run(lambda c: c.row_off.__setitem__(4, c.x.shape[0] - c.vlen[4]), specv.DEV_INDEX, packed=True)


def test_rules_ignore_tokens_behind_the_verify_length():
    """Drafted tokens at and past verify_len are not tested; what stands there is nobody's error."""
    c = Case(17, 4, 1, 6, 900, rows=7, dtype="f32")
    ref = c.oracle()
    for b in range(4):
        c.tokens[b, c.vlen[b]:] = [-1, 10 ** 6, 5, 2 ** 31 - 1, -7, 3][c.vlen[b]:]
    ws = specv.Workspace(256)
    x = logits_to_torch(c.x).view(4, 1, 7, 900)
    c.call(x, workspace=ws)
    check_rows(host(x).reshape(c.x.shape), c.x, ref, "f32")
    assert ws.status() == 0


def test_biases_of_one_token_add_up_in_list_order():
    """A thousand entries of few tokens, also drafted ones: sums in list order, the same in every run."""
    V, L, n = 5000, 4, 1000
    g = np.random.default_rng(3)
    bt = g.integers(0, 7, (1, n)).astype(np.int32) * 600
    bv = (g.standard_normal((1, n)) * 10.0 ** g.integers(-3, 4, (1, n))).astype(np.float32)
    sums = np.zeros(V, np.float32)
    for t, v in zip(bt[0], bv[0]):
        sums[t] += v                                  # fp32, in list order
    h = specv.History(torch.zeros((1, V), dtype=I32, device="cuda"), torch.zeros((1, (V + 31) // 32), dtype=I32, device="cuda"),
                      presence=torch.zeros(1, device="cuda"), repetition=torch.full((1,), 2.0, device="cuda"),
                      bias_tokens=dev(bt), bias_values=dev(bv))
    tok = dev(np.array([[600, 1200, 601, 600]], np.int32))
    first = None
    for _ in range(5):
        x = torch.zeros((1, L + 1, V), device="cuda")
        specv.spec_logit_rules(x, h, draft_tokens=tok)
        np.testing.assert_array_equal(x[0].cpu().numpy(), np.broadcast_to(sums, (L + 1, V)))
        assert first is None or torch.equal(first, x)
        first = x


def test_rules_repetition_alone_and_rows_without_a_seat():
    """NULL frequency and presence: the counts are not needed; a request without a seat is copied as it is."""
    c = Case(61, 3, 1, 2, 3000, rows=3, dtype="f32", mask="own")
    del c.kw["frequency"], c.kw["presence"]
    c.seats[0] = -1
    x = logits_to_torch(c.x).view(3, 1, 3, 3000)
    y = torch.full_like(x, 2.0)
    before = host(y).reshape(c.x.shape).copy()
    c.call(x, out=y)
    check_rows(host(y).reshape(c.x.shape), c.x, c.oracle(), "f32", before)


def test_empty_blocks_and_batches_of_padding():
    """The draft rows of an empty block, a step without tokens, a batch of padding: nothing happens, nothing is flagged."""
    h, ws = specv.History.empty(2, 100, 3), specv.Workspace(256)
    h.repetition.fill_(2.0)
    none, pad = torch.empty((3, 0), dtype=I32, device="cuda"), torch.full((3,), -1, dtype=I32, device="cuda")
    draft = torch.empty((3, 2, 0, 100), device="cuda")
    assert specv.spec_logit_rules(draft, h, seats=pad, draft_tokens=none, workspace=ws) is draft
    x = torch.randn((3, 1, 100), device="cuda")
    before = x.clone()
    specv.spec_logit_rules(x, h, seats=pad, draft_tokens=none, workspace=ws)
    specv.spec_history_add(h, torch.zeros((3, 4), dtype=I32, device="cuda"), seats=pad, workspace=ws)
    specv.spec_history_clear(h, pad, workspace=ws)
    assert torch.equal(x, before) and int(h.counts.sum()) == 0 and ws.status() == 0
    kv = Kv(2, 4, 6, 4, 3, 0)
    kv.map([5, 0, 9], [0, 0, 0, 0], [-1, -1, -1])
    kv.release([-1, -1, -1], [1, 2, 3])


def test_rules_neutral_call_writes_nothing():
    c = Case(5, 2, 1, 2, 500, rows=3, dtype="bf16")
    c.kw["repetition"][:], c.kw["frequency"][:], c.kw["presence"][:] = 1, 0, 0
    x = logits_to_torch(c.x).view(2, 1, 3, 500)
    c.call(x)
    np.testing.assert_array_equal(host(x).reshape(c.x.shape), c.x)
    y = torch.zeros_like(x)
    specv.spec_logit_rules(x, out=y, draft_tokens=dev(c.tokens))         # no rules at all: a copy
    assert torch.equal(x, y)


def test_a_row_that_allows_nothing_is_reported_by_verification():
    B, L, V = 2, 3, 512
    x = synth.custom(B=B, L=L, V=V, T=1.0, dtype="f32", seed=3, cid=700)
    target, draft = logits_to_torch(x.target), logits_to_torch(x.draft)
    ok = np.ones((1, L + 1, V), bool)
    ok[0, 0] = False
    specv.spec_logit_rules(target, draft_tokens=dev(x.tokens), mask=words(plain.pack_bits(ok)),
                           mask_rows=dev(np.array([-1, 0], np.int32)))
    ws = specv.Workspace(specv.verify_workspace_size(B, L, 1, V))
    acc, _ = specv.spec_verify_block(target, draft, dev(x.tokens), dev(x.u), dev(x.g), 1.0, workspace=ws)
    assert acc[0] >= 0 and acc[1] == -1 and ws.status() == specv.DEV_NONFINITE


def test_rules_past_32_bit_offsets():
    """State tables and logits of more than 2^31 elements."""
    V, S = 151936, 15000
    counts = torch.zeros((S, V), dtype=I32, device="cuda")
    seen = torch.zeros((S, V // 32), dtype=I32, device="cuda")
    counts[S - 1, V - 1], seen[S - 1, V // 32 - 1] = 3, -2 ** 31
    h = specv.History(counts, seen, frequency=torch.full((S,), 0.5, device="cuda"))
    B, L = 880, 16
    x = torch.ones((B, L + 1, V), dtype=torch.bfloat16, device="cuda")   # 2.27e9 elements
    tok = torch.zeros((B, L), dtype=I32, device="cuda")
    seats = torch.full((B,), -1, dtype=I32, device="cuda")
    seats[B - 1] = S - 1
    specv.spec_logit_rules(x, h, seats=seats, draft_tokens=tok)
    assert x[B - 1, 5, V - 1] == -0.5 and x[B - 1, 5, 0] == 1 - 2.5 and x[B - 1, 16, 0] == -7
    x[B - 1, :, V - 1], x[B - 1, :, 0] = 1, 1
    assert bool(torch.all(x == 1))
    specv.spec_history_add(h, torch.tensor([[V - 1]], dtype=I32, device="cuda"), seats=seats[B - 1:])
    assert counts[S - 1, V - 1] == 4
    specv.spec_history_clear(h, seats[B - 1:])
    assert counts[S - 1, V - 1] == 0 and int(seen.count_nonzero()) == 0


# ------------------------------------------------------------------ history

@pytest.mark.parametrize("V", [1, 33, 1000, 50257])
@pytest.mark.parametrize("output", [True, False])
def test_history_matches_the_definition(V, output):
    g = np.random.default_rng(V)
    S, B = 6, 9
    seats = np.array([0, 3, 3, -1, 5, 9, 1, 3, 0], np.int32)             # twice, none, outside
    counts = np.zeros((S, V), np.int32)
    seen = np.zeros((S, (V + 31) // 32), np.uint32)
    h, ws = specv.History(dev(counts), words(seen)), specv.Workspace(256)
    # padded rows
    toks = g.integers(-1, min(V + 1, 2 ** 31 - 1), (B, 17)).astype(np.int32)
    counts, seen, f1 = plain.history_add(counts, seen, seats, toks, output)
    specv.spec_history_add(h, dev(toks), seats=dev(seats), output=output, workspace=ws)
    # ragged, with empty requests and tokens before the first and behind the last
    n = np.array([0, 700, 1, 3, 0, 40, 2500, 0, 5])
    off = (np.concatenate([[0], np.cumsum(n)]) + 4).astype(np.int32)
    flat = g.integers(0, V, off[-1] + 11).astype(np.int32)
    flat[5:300] = 0                                                      # one token many times
    counts, seen, f2 = plain.history_add(counts, seen, seats, [flat[off[b]:off[b + 1]] for b in range(B)], output)
    specv.spec_history_add(h, dev(flat), offsets=dev(off), seats=dev(seats), output=output, workspace=ws)
    np.testing.assert_array_equal(h.counts.cpu().numpy(), counts)
    np.testing.assert_array_equal(h.seen.cpu().numpy().view(np.uint32), seen)
    assert ws.status() == f1 | f2
    # empty calls
    specv.spec_history_add(h, dev(toks[:, :0]), seats=dev(seats))
    specv.spec_history_add(h, dev(flat[:0]), offsets=dev(np.zeros(B + 1, np.int32)), seats=dev(seats))
    # clear two seats (one twice), keep the others
    specv.spec_history_clear(h, dev(np.array([3, -1, 3, 7, 0], np.int32)), workspace=ws)
    counts[[0, 3]], seen[[0, 3]] = 0, 0
    np.testing.assert_array_equal(h.counts.cpu().numpy(), counts)
    np.testing.assert_array_equal(h.seen.cpu().numpy().view(np.uint32), seen)


@pytest.mark.parametrize("output", [True, False])
def test_history_of_long_prompts(output):
    """Blocks of tokens inside one request, across two, before the first and behind the last; low and high ids."""
    g = np.random.default_rng(9)
    V, S, B = 60000, 4, 5
    seats = np.array([2, 9, 0, -1, 2], np.int32)
    n = np.array([3000, 2500, 1024, 5000, 6000])
    off = (np.concatenate([[0], np.cumsum(n)]) + 1500).astype(np.int32)
    flat = (V ** g.random(off[-1] + 3000) - 1).astype(np.int32)
    flat[1600], flat[off[2] + 7] = V, V + 5
    h, ws = specv.History.empty(S, V), specv.Workspace(256)
    counts, seen, f = plain.history_add(np.zeros((S, V), np.int32), np.zeros((S, V // 32), np.uint32), seats,
                                        [flat[off[b]:off[b + 1]] for b in range(B)], output)
    specv.spec_history_add(h, dev(flat), offsets=dev(off), seats=dev(seats), output=output, workspace=ws)
    np.testing.assert_array_equal(h.counts.cpu().numpy(), counts)
    np.testing.assert_array_equal(h.seen.cpu().numpy().view(np.uint32), seen)
    assert ws.status() == f == specv.DEV_INDEX | specv.DEV_TOKEN_RANGE


@pytest.mark.parametrize("off", [[0, 5, 4, 8], [-1, 2, 4, 8], [0, 2, 4, 9], [3, 2, 2, 2]])
def test_history_refuses_bad_offsets(off):
    h, ws = specv.History.empty(3, 100), specv.Workspace(256)
    specv.spec_history_add(h, torch.ones(8, dtype=I32, device="cuda"), offsets=dev(np.array(off, np.int32)), workspace=ws)
    assert ws.status() == specv.DEV_LENGTHS and int(h.counts.sum()) == 0 and int(h.seen.sum()) == 0


# ---------------------------------------------------------------------- kv

class Kv:
    """The library's tables beside the definition's lists."""

    def __init__(self, seats, max_pages, n_pages, ps, B, N, ids=None, block_table=True, positions=True):
        free = np.random.default_rng(1).permutation(n_pages) if ids is None else np.asarray(ids)
        self.plain = plain.Pages(seats, max_pages, free, ps)
        self.pages = specv.KvPages.empty(seats, max_pages, n_pages, ps)
        self.pages.free_pages.copy_(dev(free.astype(np.int32)))
        self.ws, self.N = specv.Workspace(specv.kv_workspace_size(B)), N
        self.bt = torch.full((B, max_pages), -9, dtype=I32, device="cuda") if block_table else None
        self.bt_want = np.full((B, max_pages), -9, np.int32)
        self.out = (torch.empty(N, dtype=torch.int64, device="cuda"),
                    torch.empty(N, dtype=I32, device="cuda") if positions else None,
                    torch.empty(B, dtype=I32, device="cuda"))

    def map(self, ctx, off, seats):
        r = self.plain.map(ctx, off, self.N, seats)
        specv.spec_kv_map(self.pages, dev(np.array(ctx, np.int32)), dev(np.array(off, np.int32)), self.N,
                          seats=None if seats is None else dev(np.array(seats, np.int32)), block_table=self.bt,
                          out=self.out, workspace=self.ws)
        np.testing.assert_array_equal(self.out[0].cpu().numpy(), r["slots"])
        if self.out[1] is not None:
            np.testing.assert_array_equal(self.out[1].cpu().numpy(), r["positions"])
        np.testing.assert_array_equal(self.out[2].cpu().numpy(), r["seq_len"])
        for b, t in enumerate(r["tables"]):
            self.bt_want[b, :len(t)] = t
        if self.bt is not None:
            np.testing.assert_array_equal(self.bt.cpu().numpy(), self.bt_want)
        self.same(r["flags"])
        return r

    def release(self, seats, keep=None):
        f = self.plain.release(seats, keep)
        specv.spec_kv_release(self.pages, dev(np.array(seats, np.int32)),
                              keep_len=None if keep is None else dev(np.array(keep, np.int32)), workspace=self.ws)
        self.same(f)

    def same(self, flags):
        p = self.pages
        n = int(p.free_count)
        assert p.free_pages[:n].tolist() == self.plain.stack
        table, owned = p.page_table.cpu().numpy(), p.owned.tolist()
        for s, held in enumerate(self.plain.held):
            assert owned[s] == len(held) and table[s, :len(held)].tolist() == held
            assert np.all(table[s, len(held):] == -1)
        assert self.ws.status() == flags
        self.ws.init()


@pytest.mark.parametrize("ps,seats,max_pages,n_pages", [(16, 12, 40, 200), (1, 6, 300, 900), (48, 12, 9, 60), (7, 40, 1500, 4000)])
def test_kv_steps_match_the_definition(ps, seats, max_pages, n_pages):
    """Admission, decoding with rejected positions, finished requests, padding, shortage of pages."""
    g = np.random.default_rng(ps)
    B = min(seats, 8)
    N = 600
    kv = Kv(seats, max_pages, n_pages, ps, B, N, block_table=ps != 1, positions=ps != 48)
    ctx = np.zeros(seats, np.int64)
    seen = set()
    for step in range(25):
        batch = g.permutation(seats)[:B].astype(np.int32)
        batch[g.random(B) < 0.15] = -1
        new = np.where(g.random(B) < 0.3, g.integers(0, 130, B), g.integers(0, 18, B))
        off = np.concatenate([[0], np.cumsum(new)])
        if off[-1] > N:
            new[:] = 3
            off = np.concatenate([[0], np.cumsum(new)])
        off = off + (step % 3 if off[-1] + 2 <= N else 0)
        c = np.where(batch >= 0, ctx[batch], 0)
        r = kv.map(c, off, batch)
        seen.add(r["flags"])
        got = np.array(r["seq_len"])
        keep = np.where(got > 0, np.minimum(got, c + g.integers(0, 6, B)), c)
        kv.release(batch, keep)
        for b in range(B):
            if batch[b] >= 0:
                ctx[batch[b]] = keep[b]
        done = batch[(g.random(B) < 0.2) & (batch >= 0)]
        if len(done):
            kv.release(done)
            ctx[done] = 0
    assert 0 in seen


def test_kv_runs_out_of_pages():
    kv = Kv(4, 8, 10, 4, 4, 64)
    kv.map([0, 0, 0, 0], [0, 16, 32, 48, 49], None)       # 4 + 4 pages, then 4 of 2 left, then none for the last
    assert kv.out[2].tolist() == [16, 16, -1, -1]
    kv.release([1], [5])
    kv.map([16, 5, 0, 0], [0, 0, 3, 19, 20], None)
    kv.map([16, 5, 0, 0], [0, 17, 20, 20, 20], None)      # 33 tokens: 9 pages, more than a row holds
    assert kv.out[2].tolist() == [-1, 8, 0, 0]
    kv.release([0, 1, 2, 3])
    assert int(kv.pages.free_count) == 10


def test_kv_refusals():
    kv = Kv(4, 8, 20, 4, 4, 16)
    kv.map([0, 0, 0, 0], [0, 4, 8, 12, 16], [0, 1, 1, 3])             # a seat named twice
    kv.map([4, 0, 0, -1], [0, 1, 2, 3, 4], [0, 4, 2, 3])              # outside the table; an impossible length
    kv.map([0, 0, 0, 2 ** 31 - 1], [0, 1, 2, 3, 4], [0, 1, 2, 3])     # the sum passes 32 bits
    for off in ([0, 4, 3, 8, 9], [0, 1, 2, 3, 17], [-1, 0, 1, 2, 3]):
        kv.map([0, 0, 0, 0], off, [0, 1, 2, 3])
        assert kv.out[2].tolist() == [-1] * 4
    kv.release([0, 0, 2, -1])                                         # twice: left out
    kv.release([0, 4, 2, 1], [-1, 0, 1, 1])
    kv.pages.free_count.fill_(20)                                     # a stack that has no room for what comes back
    kv.plain.stack = kv.pages.free_pages.tolist()
    kv.release([0, 1, 2, 3])
    kv.pages.free_count.fill_(21)
    specv.spec_kv_map(kv.pages, torch.zeros(4, dtype=I32, device="cuda"), torch.arange(5, dtype=I32, device="cuda"), 16,
                      out=kv.out, workspace=kv.ws)
    assert kv.ws.status() == specv.DEV_LENGTHS and kv.out[2].tolist() == [-1] * 4 and set(kv.out[0].tolist()) == {-1}


def test_kv_many_requests_and_long_caches():
    """B at its limit with no tokens for many; page numbers whose slots pass 32 bits; 100,000 tokens in one request."""
    B = specv_max_b = 4096
    kv = Kv(65536, 3, 9000, 64, B, 8192, ids=2 ** 31 - 1 - np.arange(9000))
    g = np.random.default_rng(0)
    seats = g.permutation(65536)[:specv_max_b]
    off = np.concatenate([[0], np.cumsum(g.integers(0, 3, B))])
    off = np.minimum(off, 8192)
    r = kv.map(g.integers(0, 60, B), off, seats)
    assert max(r["slots"]) > 2 ** 36
    kv.release(seats)
    kv = Kv(2, 8000, 9000, 16, 2, 120000)
    kv.map([0, 5], [0, 100000, 100017], None)
    kv.release([0, 1], [99999, 21])


# ----------------------------------------------------------- a run of them

def _step_tables(B, L, V, K, S, page, budget, g):
    """Device buffers of one serving step, at fixed addresses."""
    x = synth.custom(B=B, L=L, V=V, K=K, T=1.1, dtype="bf16", n_peaks=6, peak=6.0, draft_sigma=0.6, budget=budget,
                     seed=31, cid=710)
    d = dict(target=logits_to_torch(x.target), draft=logits_to_torch(x.draft), tokens=dev(x.tokens), u=dev(x.u),
             g=dev(x.g), mix_w=dev(x.mix_w), scores=dev(x.scores))
    return x, d


@pytest.mark.parametrize("graph", [False, True])
def test_a_serving_step(graph):
    """Allocation, paging, rules on target and draft, verification, history and release, over several steps with
    changing data; captured once and replayed, or launched call by call."""
    B, L, V, K, S, page = 6, 8, 4096, 2, 9, 16
    budget = B * (L + 1) // 2
    g = np.random.default_rng(5)
    x, d = _step_tables(B, L, V, K, S, page, budget, g)
    seats_h = np.array([4, 0, 7, 2, 8, 5], np.int32)
    h = specv.History.empty(S, V, 4)
    h.repetition.copy_(dev(g.uniform(1, 1.4, S).astype(np.float32)))
    h.frequency.copy_(dev(g.uniform(0, 0.6, S).astype(np.float32)))
    h.presence.copy_(dev(g.uniform(0, 0.6, S).astype(np.float32)))
    h.bias_tokens.copy_(dev(g.integers(0, V, (S, 4)).astype(np.int32)))
    h.bias_values.copy_(dev(g.standard_normal((S, 4)).astype(np.float32)))
    pages = specv.KvPages.empty(S, 40, 300, page)
    model = plain.Pages(S, 40, np.arange(299, -1, -1), page)
    ctx_h = g.integers(20, 60, B).astype(np.int32)
    prompts = [g.integers(0, V, n).astype(np.int32) for n in ctx_h]
    off0 = np.concatenate([[0], np.cumsum(ctx_h)]).astype(np.int32)
    seats = dev(seats_h)
    specv.spec_history_add(h, dev(np.concatenate(prompts)), offsets=dev(off0), seats=seats, output=False)
    specv.spec_kv_map(pages, torch.zeros(B, dtype=I32, device="cuda"), dev(off0), int(off0[-1]), seats=seats)
    model.map([0] * B, off0, int(off0[-1]), seats_h)
    ok = g.random((2, L + 1, V)) < 0.7
    ok_d, mask_rows = words(plain.pack_bits(ok)), dev(np.array([-1, 1, -1, 0, -1, -1], np.int32))
    ctx = dev(ctx_h)
    packed = torch.empty((budget, V), dtype=torch.bfloat16, device="cuda")
    draft = torch.empty_like(d["draft"])
    e = lambda *s, dt=I32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    dvl = (e(B), e(B + 1), e(budget))
    kv_out, bt = (e(budget, dt=torch.int64), e(budget), e(B)), torch.full((B, 40), -1, dtype=I32, device="cuda")
    ver = (e(B), e(B, L + 1))
    keep = e(B)
    ws = dict(dvl=specv.Workspace(specv.dvl_workspace_size(B)), ver=specv.Workspace(specv.verify_workspace_size(B, L, K, V)),
              rules=specv.Workspace(specv.rules_workspace_size(B)), kv=specv.Workspace(specv.kv_workspace_size(B)))

    def step():
        vl, off, _ = specv.dvl_allocate_pack(d["scores"], budget, dense_target=d["target"], packed_target=packed,
                                             workspace=ws["dvl"], out=dvl)
        specv.spec_kv_map(pages, ctx, off, budget, seats=seats, block_table=bt, out=kv_out, workspace=ws["kv"])
        rules = dict(seats=seats, draft_tokens=d["tokens"], verify_len=vl, mask=ok_d, mask_rows=mask_rows,
                     workspace=ws["rules"])
        specv.spec_logit_rules(packed, h, target_row_off=off, **rules)
        specv.spec_logit_rules(d["draft"], h, out=draft, **rules)
        acc, out = specv.spec_verify_mixture(packed, draft, d["mix_w"], d["tokens"], d["u"], d["g"], 1.1, verify_len=vl,
                                             target_row_off=off[:B], workspace=ws["ver"], out=ver)
        specv.spec_history_add(h, out, seats=seats, workspace=ws["rules"])
        torch.add(ctx, acc, out=keep)
        keep.add_(1)
        specv.spec_kv_release(pages, seats, keep_len=keep, workspace=ws["kv"])
        ctx.copy_(keep)

    counts, seen = h.counts.cpu().numpy().copy(), h.seen.cpu().numpy().view(np.uint32).copy()
    params = dict(repetition=h.repetition.cpu().numpy(), frequency=h.frequency.cpu().numpy(),
                  presence=h.presence.cpu().numpy(), bias_tokens=h.bias_tokens.cpu().numpy(),
                  bias_values=h.bias_values.cpu().numpy())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    captured, flags = None, 0
    with torch.cuda.stream(s):
        if graph:
            captured = torch.cuda.CUDAGraph()
            s.synchronize()
            with torch.cuda.graph(captured, stream=s):
                step()
        for trial in range(4):
            scores = -np.sort(-g.beta(5, 2, (B, L)), axis=1).astype(np.float32)
            u, toks = g.random((B, L), dtype=np.float32), x.tokens.copy()
            if trial % 2:
                toks[:, 1] = toks[:, 0]                       # a drafted token twice in a block
            d["scores"].copy_(dev(scores))
            d["u"].copy_(dev(u))
            d["tokens"].copy_(dev(toks))
            captured.replay() if graph else step()
            s.synchronize()
            ra = oracle.dvl_allocate(scores, budget)
            vl, off = ra["verify_len"], ra["offsets"]
            np.testing.assert_array_equal(dvl[1].cpu().numpy(), off)
            # paging
            r = model.map(ctx_h, off, budget, seats_h)
            np.testing.assert_array_equal(kv_out[0].cpu().numpy(), r["slots"])
            np.testing.assert_array_equal(kv_out[1].cpu().numpy(), r["positions"])
            for b in range(B):
                assert bt[b, :len(r["tables"][b])].tolist() == r["tables"][b]
            # rules
            common = dict(tokens=toks, verify_len=vl, seats=seats_h, counts=counts, seen=seen,
                          mask=plain.pack_bits(ok), mask_rows=mask_rows.cpu().numpy(), **params)
            dense = oracle.pack(x.target, vl, off, budget)
            rt = plain.logit_rules(dense, B, 1, L + 1, L, row_off=off[:B], **common)
            check_rows(host(packed), dense, rt, "bf16")
            flat = x.draft.reshape(-1, V)
            rd = plain.logit_rules(flat, B, K, L, L, **common)
            got = host(draft).reshape(-1, V)
            check_rows(got, flat, rd, "bf16", got)
            # verification of the edited rows, then the state
            ref = oracle.verify(host(packed), host(draft), toks, u, x.g, 1.1, mix_w=x.mix_w, verify_len=vl,
                                target_row_off=off[:B], diag=True)
            flags |= ref["flags"]
            acc, out = ver[0].cpu().numpy(), ver[1].cpu().numpy()
            check_verify(acc, out, ref, verify_len=vl)
            counts, seen, _ = plain.history_add(counts, seen, seats_h, out, True)
            np.testing.assert_array_equal(h.counts.cpu().numpy(), counts)
            np.testing.assert_array_equal(h.seen.cpu().numpy().view(np.uint32), seen)
            ctx_h = ctx_h + acc + 1
            model.release(seats_h, ctx_h)
            assert pages.free_pages[:int(pages.free_count)].tolist() == model.stack
            np.testing.assert_array_equal(ctx.cpu().numpy(), ctx_h)
    # a drafted token that the mask forbids has probability 0 on both sides: verification reports it, as the oracle does
    assert {k: w.status() for k, w in ws.items()} == dict(dvl=0, ver=flags, rules=0, kv=0)
    del captured


def test_calls_on_two_streams_share_a_rules_workspace():
    """Two calls at once on their own rows, one history, one workspace: it holds the status word alone."""
    a, b = Case(41, 4, 1, 3, 20000, rows=4, bias=8), Case(42, 4, 1, 3, 20000, rows=4, bias=8)
    ws = specv.Workspace(256)
    xs = [logits_to_torch(c.x).view(4, 1, 4, 20000) for c in (a, b)]
    args = [dict(seats=dev(c.seats), draft_tokens=dev(c.tokens), verify_len=dev(c.vlen)) for c in (a, b)]
    hs = [c.history() for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, x, h, k in zip(streams, xs, hs, args):
        with torch.cuda.stream(s):
            specv.spec_logit_rules(x, h, workspace=ws, **k)
    torch.cuda.synchronize()
    for c, x in zip((a, b), xs):
        check_rows(host(x).reshape(c.x.shape), c.x, c.oracle(), "bf16")
    assert ws.status() == 0


def test_two_host_threads_call_at_once():
    """Calls from two host threads on streams of their own, with different needs of shared memory."""
    import threading
    cases = [Case(51, 3, 1, 2, 9000, rows=3, bias=1000), Case(52, 3, 1, 2, 9000, rows=3, bias=2)]
    xs, errors = [], []
    for c in cases:
        xs.append([logits_to_torch(c.x).view(3, 1, 3, 9000) for _ in range(30)])
    hs = [c.history() for c in cases]
    ks = [dict(seats=dev(c.seats), draft_tokens=dev(c.tokens), verify_len=dev(c.vlen), workspace=specv.Workspace(256))
          for c in cases]
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for x in xs[i]:
                    specv.spec_logit_rules(x, hs[i], **ks[i])
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for c, x in zip(cases, xs):
        ref = c.oracle()
        check_rows(host(x[0]).reshape(c.x.shape), c.x, ref, "bf16")
        assert all(torch.equal(x[0].view(torch.int16), y.view(torch.int16)) for y in x[1:])


# ------------------------------------------------------------------ padding

@pytest.mark.parametrize("pad", [-1, -2, -7, -2 ** 31])
def test_any_negative_seat_is_padding(pad):
    """Every call takes every negative seat as no seat: nothing is read, written or flagged for it."""
    kv = Kv(4, 8, 30, 4, 4, 24)
    kv.map([5, 3, 9, 2], [0, 3, 7, 9, 12], [2, pad, pad, 0])
    assert kv.out[2].tolist() == [8, 0, 0, 5]
    kv.map([8, 2 ** 31 - 1, -4, 5], [1, 2, 6, 6, 8], [2, pad, pad, 0])    # whatever stands beside it
    assert kv.out[2].tolist() == [9, 0, 0, 7]
    kv.map([0, 0, 0, 0], [0, 4, 8, 12, 16], [pad] * 4)
    assert kv.out[2].tolist() == [0] * 4
    kv.release([pad, 2, pad, 0], [-1, 3, 0, 1])
    kv.release([pad] * 4)
    c = Case(71, 4, 2, 3, 1000, rows=4, dtype="f32", bias=4, mask="some")
    c.seats[1] = c.seats[3] = c.mask_rows[0] = pad
    ref, ws = c.oracle(), specv.Workspace(256)
    x = c.view(logits_to_torch(c.x))
    h = c.history()
    c.call(x, workspace=ws)
    check_rows(host(x).reshape(c.x.shape), c.x, ref, "f32")
    before = h.counts.clone(), h.seen.clone()
    seats = dev(np.full(3, pad, np.int32))
    specv.spec_history_add(h, torch.ones((3, 5), dtype=I32, device="cuda"), seats=seats, workspace=ws)
    specv.spec_history_add(h, torch.ones(3000, dtype=I32, device="cuda"), seats=seats, workspace=ws,
                           offsets=dev(np.array([0, 2500, 2600, 3000], np.int32)))
    specv.spec_history_clear(h, seats, workspace=ws)
    assert torch.equal(h.counts, before[0]) and torch.equal(h.seen, before[1]) and ws.status() == ref["flags"] == 0


# ------------------------------------------------- which rows a step edits

@pytest.mark.parametrize("K", [1, 3])
def test_a_forbidden_draft_is_rejected_with_an_allowed_token(K):
    """A block drafter drew its tokens from the unedited rows: the target rows alone are edited. A drafted token that
    the grammar forbids has p = 0 and is rejected, and the terminal token is one that the grammar allows."""
    B, L, V = 4, 3, 512
    x = synth.custom(B=B, L=L, V=V, K=K, T=1.0, dtype="f32", seed=5, cid=720)
    ok = np.random.default_rng(2).random((B, L + 1, V)) < 0.5
    for b in range(B):
        ok[b, np.arange(L), x.tokens[b]] = True
    ok[1, 1, x.tokens[1, 1]] = ok[2, 0, x.tokens[2, 0]] = False
    u = np.full((B, L), 1e-4, np.float32)                                # every p / q is above it or 0
    target, draft = logits_to_torch(x.target), logits_to_torch(x.draft)
    specv.spec_logit_rules(target, draft_tokens=dev(x.tokens), mask=words(plain.pack_bits(ok)))
    ws = specv.Workspace(specv.verify_workspace_size(B, L, K, V))
    args = (dev(x.tokens), dev(u), dev(x.g), 1.0)
    acc, out = (specv.spec_verify_block(target, draft, *args, workspace=ws) if K == 1 else
                specv.spec_verify_mixture(target, draft, dev(x.mix_w), *args, workspace=ws))
    acc, out = acc.cpu().numpy(), out.cpu().numpy()
    assert acc.tolist() == [3, 1, 0, 3] and ws.status() == 0
    for b in range(B):
        assert ok[b, np.arange(acc[b] + 1), out[b, :acc[b] + 1]].all()
    ref = oracle.verify(host(target), x.draft, x.tokens, u, x.g, 1.0, mix_w=x.mix_w, diag=True)
    check_verify(acc, out, ref)


@pytest.mark.parametrize("graph", [False, True])
def test_the_documented_step(graph):
    """Allocation, paging, the target's rows, rules on them, verification against the draft rows as they were drawn
    from, history and release, over several steps; a batch with padding, drafted tokens that a grammar forbids, and
    requests that get no pages and sit a step out. Launched call by call, or captured once and replayed."""
    B, L, V, K, S, page, n_pages = 6, 8, 4096, 2, 9, 16, 16
    budget, T = B * (L + 1) // 2, 1.1
    g = np.random.default_rng(6)
    x, d = _step_tables(B, L, V, K, S, page, budget, g)
    seats_h = np.array([4, 0, -3, 2, 8, 5], np.int32)
    params = dict(repetition=g.uniform(1, 1.4, S), frequency=g.uniform(0, 0.6, S), presence=g.uniform(0, 0.6, S),
                  bias_values=g.standard_normal((S, 4)))
    params = {k: v.astype(np.float32) for k, v in params.items()}
    params["bias_tokens"] = g.integers(0, V, (S, 4)).astype(np.int32)
    h = specv.History.empty(S, V, 4)
    for k, v in params.items():
        getattr(h, k).copy_(dev(v))
    pages, model = specv.KvPages.empty(S, 40, n_pages, page), plain.Pages(S, 40, np.arange(n_pages - 1, -1, -1), page)
    ctx_h = np.array([40, 37, 0, 60, 20, 43], np.int32)
    off0 = np.concatenate([[0], np.cumsum(ctx_h)]).astype(np.int32)
    prompts, seats = g.integers(0, V, off0[-1]).astype(np.int32), dev(seats_h)
    specv.spec_history_add(h, dev(prompts), offsets=dev(off0), seats=seats, output=False)
    specv.spec_kv_map(pages, torch.zeros(B, dtype=I32, device="cuda"), dev(off0), int(off0[-1]), seats=seats)
    assert model.map([0] * B, off0, int(off0[-1]), seats_h)["flags"] == 0
    counts, seen, _ = plain.history_add(np.zeros((S, V), np.int32), np.zeros((S, V // 32), np.uint32), seats_h,
                                        [prompts[off0[b]:off0[b + 1]] for b in range(B)], False)
    ok, mrows = g.random((2, L + 1, V)) < 0.7, np.array([-1, 1, -1, 0, -1, 1], np.int32)
    mask, mask_rows, ctx = words(plain.pack_bits(ok)), dev(mrows), dev(ctx_h)
    e = lambda *s, dt=I32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    packed = torch.empty((budget, V), dtype=torch.bfloat16, device="cuda")
    dvl, ver, keep = (e(B), e(B + 1), e(budget)), (e(B), e(B, L + 1)), e(B)
    kv_out, bt = (e(budget, dt=torch.int64), e(budget), e(B)), torch.full((B, 40), -1, dtype=I32, device="cuda")
    ws = dict(dvl=specv.Workspace(specv.dvl_workspace_size(B)), ver=specv.Workspace(specv.verify_workspace_size(B, L, K, V)),
              rules=specv.Workspace(specv.rules_workspace_size(B)), kv=specv.Workspace(specv.kv_workspace_size(B)))

    def step():
        vl, off, slot_map = specv.dvl_allocate_pack(d["scores"], budget, workspace=ws["dvl"], out=dvl)
        _, _, seq_len = specv.spec_kv_map(pages, ctx, off, budget, seats=seats, block_table=bt, out=kv_out,
                                          workspace=ws["kv"])
        vl.masked_fill_(seq_len < 0, -1)
        # the target's forward pass over the allocated slots
        torch.index_select(d["target"].view(-1, V), 0, slot_map.clamp(min=0), out=packed)
        specv.spec_logit_rules(packed, h, seats=seats, draft_tokens=d["tokens"], verify_len=vl, target_row_off=off,
                               mask=mask, mask_rows=mask_rows, workspace=ws["rules"])
        acc, out = specv.spec_verify_mixture(packed, d["draft"], d["mix_w"], d["tokens"], d["u"], d["g"], T,
                                             verify_len=vl, target_row_off=off[:B], workspace=ws["ver"], out=ver)
        specv.spec_history_add(h, out, seats=seats, workspace=ws["rules"])
        torch.add(ctx, acc, out=keep)
        keep.add_(1)
        specv.spec_kv_release(pages, seats, keep_len=keep, workspace=ws["kv"])
        ctx.copy_(keep)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    captured, flags, refused, forbidden = None, dict(dvl=0, ver=0, rules=0, kv=0), 0, 0
    with torch.cuda.stream(s):
        if graph:
            captured = torch.cuda.CUDAGraph()
            s.synchronize()
            with torch.cuda.graph(captured, stream=s):
                step()
        for trial in range(6):
            scores = -np.sort(-g.beta(5, 2, (B, L)), axis=1).astype(np.float32)
            u, toks = g.random((B, L), dtype=np.float32), x.tokens.copy()
            if trial % 2:
                toks[:, 1] = toks[:, 0]
            for k, v in dict(scores=scores, u=u, tokens=toks).items():
                d[k].copy_(dev(v))
            captured.replay() if graph else step()
            s.synchronize()
            ra = oracle.dvl_allocate(scores, budget)
            off, r = ra["offsets"], model.map(ctx_h, ra["offsets"], budget, seats_h)
            np.testing.assert_array_equal(kv_out[0].cpu().numpy(), r["slots"])
            np.testing.assert_array_equal(kv_out[2].cpu().numpy(), r["seq_len"])
            vl = np.where(np.array(r["seq_len"]) < 0, -1, ra["verify_len"]).astype(np.int32)
            dense = host(d["target"]).reshape(-1, V)[np.maximum(ra["slot_map"], 0)]
            rt = plain.logit_rules(dense, B, 1, L + 1, L, row_off=off[:B], tokens=toks, verify_len=vl, seats=seats_h,
                                   counts=counts, seen=seen, mask=plain.pack_bits(ok), mask_rows=mrows, **params)
            check_rows(host(packed), dense, rt, "bf16")
            ref = oracle.verify(host(packed), x.draft, toks, u, x.g, T, mix_w=x.mix_w, verify_len=vl,
                                target_row_off=off[:B], diag=True)
            acc, out = ver[0].cpu().numpy(), ver[1].cpu().numpy()
            check_verify(acc, out, ref, verify_len=vl)
            for b in range(B):
                if vl[b] < 0:
                    assert acc[b] == -1 and (out[b] == -1).all()         # refused: it sits the step out
                    refused += 1
                elif mrows[b] >= 0:
                    at = np.arange(acc[b] + 1)
                    assert ok[mrows[b], at, out[b, at]].all()
                    forbidden += int(not ok[mrows[b], np.arange(vl[b]), toks[b, :vl[b]]].all())
            counts, seen, _ = plain.history_add(counts, seen, seats_h, out, True)
            np.testing.assert_array_equal(h.counts.cpu().numpy(), counts)
            np.testing.assert_array_equal(h.seen.cpu().numpy().view(np.uint32), seen)
            ctx_h = ctx_h + acc + 1
            f = model.release(seats_h, ctx_h)
            assert pages.free_pages[:int(pages.free_count)].tolist() == model.stack
            np.testing.assert_array_equal(ctx.cpu().numpy(), ctx_h)
            for k, v in dict(ver=ref["flags"], rules=rt["flags"], kv=r["flags"] | f).items():
                flags[k] |= v
    assert refused and forbidden
    assert flags == dict(dvl=0, ver=specv.DEV_VERIFY_LEN, rules=specv.DEV_VERIFY_LEN, kv=specv.DEV_PAGES)
    assert {k: w.status() for k, w in ws.items()} == flags
    del captured


# ---------------------------------------------- elements that stay as they are

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,V", [(3, 5000), (150, 16384)])
def test_elements_that_no_rule_changes_keep_their_bits(B, V, dtype):
    """With r = 1 a token that only the prompt holds is not changed, although the penalties are on: NaN payloads and
    signed zeros stay, in place, in the copy, and where rows are copied and edited in one kernel."""
    L = 2
    c = Case(81, B, 1, L, V, rows=L + 1, dtype=dtype, hist=400, bias=6, vlen=False)
    c.kw["repetition"][:] = 1
    nan = np.arange(c.x[:, ::3].shape[1])
    if dtype == "bf16":
        c.x[:, ::3], c.x[:, 1::3] = 0x7f81 + (nan % 100).astype(np.uint16), 0x8000
    else:
        c.x.view(np.uint32)[:, ::3], c.x[:, 1::3] = 0x7f800001 + nan.astype(np.uint32), -0.0
    changed = np.zeros(c.x.shape, bool)
    prompt_only = 0
    for b in range(B):
        s = c.seats[b]
        for i in range(L + 1):
            if s < 0:
                continue
            row = changed[b * (L + 1) + i]
            row[c.kw["counts"][s] > 0] = True
            row[c.tokens[b, :i]] = True
            row[c.kw["bias_tokens"][s][c.kw["bias_tokens"][s] >= 0]] = True
            prompt_only += int((plain.bits_of(c.kw["seen"][s], V) & ~row)[::3].sum())
    assert prompt_only > 50 * B
    raw = np.uint16 if dtype == "bf16" else np.uint32
    x = c.view(logits_to_torch(c.x))
    y = torch.zeros_like(x)
    c.call(x, out=y)
    c.call(x)
    for got in (y, x):
        got = host(got).reshape(c.x.shape).view(raw)
        np.testing.assert_array_equal(got[~changed], c.x.view(raw)[~changed])
    assert torch.equal(x.view(torch.int16 if dtype == "bf16" else I32), y.view(torch.int16 if dtype == "bf16" else I32))


# ------------------------------------------------------- workspaces, launches

def test_kv_calls_on_a_workspace_that_other_calls_used():
    """The kv calls keep their ticket where no call has scratch: what a softmax or a history call left in the
    workspace does not matter."""
    B = 200
    ws = specv.Workspace(max(specv.kv_workspace_size(B), specv.softmax_workspace_size(64)))
    kv = Kv(B, 40, 9000, 16, B, 6000)                                    # several blocks each
    kv.ws = ws
    x = torch.randn((64, 4096), device="cuda")
    g = np.random.default_rng(4)
    seats = g.permutation(B)
    h = specv.History.empty(4, 100)

    def others():
        specv.softmax_T(x, 1.0, workspace=ws)
        specv.spec_history_add(h, torch.ones((4, 3), dtype=I32, device="cuda"), workspace=ws)
        assert int(ws.buf[256:260].view(I32)) != 0

    for _ in range(3):
        others()
        kv.map(g.integers(0, 500, B), np.concatenate([[0], np.cumsum(g.integers(0, 30, B))]), seats)
        others()
        kv.release(seats, g.integers(0, 300, B))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("top_p", [None, 0.9])
def test_empty_blocks_right_behind_their_allocation(top_p, graph):
    """L = 0: no statistics run between the allocation and the decision, which must not read the lengths and offsets
    before they are written. The buffers hold another valid allocation before."""
    B, V = 500, 256
    target = torch.zeros((B, V), device="cuda")
    want = torch.randint(0, V, (B,), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    target[torch.arange(B), want] = 20.0
    n = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    vl, off = n(B, dt=I32), n(B + 1, dt=I32)
    acc, out = n(B, dt=I32), n(B, 1, dt=I32)
    size = specv.verify_workspace_size if top_p is None else specv.verify_top_p_workspace_size
    ws, wd = specv.Workspace(size(B, 0, 1, V)), specv.Workspace(specv.dvl_workspace_size(B))
    draft, tokens, u, gumbel, scores = n(B, 0, V), n(B, 0, dt=I32), n(B, 0), torch.zeros((B, 1, V), device="cuda"), n(B, 0)
    stale = torch.arange(B, -1, -1, dtype=I32, device="cuda") % B

    def step():
        specv.dvl_allocate_pack(scores, B, workspace=wd, out=(vl, off, None))
        args = (target, draft, tokens, u, gumbel, 1.0) + (() if top_p is None else (top_p,))
        call = specv.spec_verify_block if top_p is None else specv.spec_verify_block_top_p
        call(*args, verify_len=vl, target_row_off=off[:B], workspace=ws, out=(acc, out))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    captured = None
    with torch.cuda.stream(s):
        if graph:
            captured = torch.cuda.CUDAGraph()
            s.synchronize()
            with torch.cuda.graph(captured, stream=s):
                step()
        for _ in range(20):
            vl.zero_()
            off.copy_(stale)
            out.fill_(-5)
            s.synchronize()
            captured.replay() if graph else step()
            s.synchronize()
            assert int((out.view(-1) != want).sum()) == 0 and int(acc.count_nonzero()) == 0
    assert ws.status() == 0 and wd.status() == 0
    del captured


# ----------------------------------- refusals inside steps and in every kernel

@pytest.mark.parametrize("ps,seats,max_pages,n_pages", [(16, 12, 40, 30), (3, 10, 20, 60)])
def test_kv_steps_with_refusals(ps, seats, max_pages, n_pages):
    """Steps in which some requests find no page left, or need more than a row holds, between others that grow, shrink
    and finish."""
    g = np.random.default_rng(ps)
    B, N = 8, 500
    kv = Kv(seats, max_pages, n_pages, ps, B, N)
    ctx = np.zeros(seats, np.int64)
    flags, mixed = [], 0
    for step in range(30):
        batch = g.permutation(seats)[:B].astype(np.int32)
        batch[g.random(B) < 0.1] = -1 - step
        new = np.where(g.random(B) < 0.3, g.integers(0, 62, B), g.integers(0, 18, B))
        c = np.where(batch >= 0, ctx[np.maximum(batch, 0)], 0)
        r = kv.map(c, np.concatenate([[0], np.cumsum(new)]), batch)
        flags.append(r["flags"])
        got = np.array(r["seq_len"])
        mixed += bool((got < 0).any() and ((got > c) & (batch >= 0)).any())
        keep = np.where(got > 0, np.minimum(got, c + g.integers(0, 30, B)), c)
        kv.release(batch, keep)
        ctx[batch[batch >= 0]] = keep[batch >= 0]
        done = batch[(g.random(B) < 0.1) & (batch >= 0)]
        if len(done):
            kv.release(done)
            ctx[done] = 0
    assert set(flags) == {0, specv.DEV_PAGES} and mixed > 3


def test_refusals_where_rows_are_copied_and_edited_in_one_kernel():
    """Out of place, 450 rows of 16,391 tokens: a request of each impossible kind keeps its rows."""
    base = dict(B=150, K=1, L=2, V=16391, rows=3, dtype="bf16", bias=5, mask="some", hist=20)
    S = 153

    def run(change, want, packed=False):
        c = Case(23, packed=packed, **base)
        c.seats, c.mask_rows = np.arange(150, dtype=np.int32), np.arange(150, dtype=np.int32) % 75
        change(c)
        ref, ws = c.oracle(), specv.Workspace(256)
        assert ref["flags"] == want
        x = c.view(logits_to_torch(c.x))
        y = torch.full_like(x, 3.0)
        before = host(y).reshape(c.x.shape).copy()
        c.call(x, out=y, workspace=ws)
        check_rows(host(y).reshape(c.x.shape), c.x, ref, "bf16", before)
        assert ws.status() == want

    run(lambda c: (c.vlen.__setitem__(20, 3), c.vlen.__setitem__(149, -1)), specv.DEV_VERIFY_LEN)
    run(lambda c: (c.seats.__setitem__(1, S), c.seats.__setitem__(2, -9)), specv.DEV_INDEX)
    run(lambda c: (c.mask_rows.__setitem__(77, 75), c.mask_rows.__setitem__(3, -4)), specv.DEV_INDEX)
    run(lambda c: (c.kw["repetition"].__setitem__(8, np.nan), c.kw["presence"].__setitem__(9, np.inf)), specv.DEV_PARAM)
    run(lambda c: (c.row_off.__setitem__(0, -1), c.row_off.__setitem__(4, c.x.shape[0] - c.vlen[4])), specv.DEV_INDEX,
        packed=True)
    run(lambda c: (c.vlen.fill(2), c.tokens.__setitem__((1, 0), 16391), c.kw["bias_tokens"].__setitem__((2, 1), 16391)),
        specv.DEV_TOKEN_RANGE)


def test_two_tiles_where_rows_are_copied_and_edited_in_one_kernel():
    """450 rows of 163,910 tokens, 70 of them in a second tile of the edit kernel, with seen, drafted and biased tokens in
    both: the copy has the bits of the form in place, and that follows the definition."""
    B, L, V = 150, 2, 163910
    c = Case(24, B, 1, L, V, rows=L + 1, hist=300, bias=8)
    g = np.random.default_rng(1)
    c.tokens = np.where(g.random((B, L)) < 0.5, V - 1 - g.integers(0, 70, (B, L)), c.tokens).astype(np.int32)
    bt = c.kw["bias_tokens"]
    bt[:, 1:4] = V - 1 - g.integers(0, 70, bt[:, 1:4].shape)
    bits = plain.bits_of(c.kw["seen"][:, -3:], 70)
    high = g.random(bits.shape) < 0.3
    c.kw["seen"][:, -3:] = plain.pack_bits(bits | high)
    x = c.view(logits_to_torch(c.x))
    y = torch.full_like(x, 2.0)
    ws = specv.Workspace(256)
    c.call(x, out=y, workspace=ws)
    c.call(x, workspace=ws)
    done = torch.arange(L + 1, device="cuda")[None, None, :, None] <= dev(c.vlen)[:, None, None, None]
    assert torch.equal(y.view(torch.int16), torch.where(done, x, torch.full_like(x, 2.0)).view(torch.int16))
    got = host(x).reshape(c.x.shape)
    for b in (0, 1, 2, 77, 149):
        rows = slice(b * (L + 1), (b + 1) * (L + 1))
        ref = plain.logit_rules(c.x[rows], 1, 1, L + 1, L, tokens=c.tokens[b:b + 1], verify_len=c.vlen[b:b + 1],
                                seats=c.seats[b:b + 1], **c.kw)
        check_rows(got[rows], c.x[rows], ref, "bf16")
    assert ws.status() == 0


def test_flags_of_calls_on_two_streams_are_collected():
    """Two calls at once read one history through seats of their own, share a workspace and raise different flags."""
    V = 20000
    a, b = (Case(43 + k, 6, 1, 3, V, rows=4, dtype="f32", bias=8) for k in range(2))
    b.kw = {k: v.copy() for k, v in a.kw.items()}
    a.seats, b.seats = np.array([0, 1, 2, 3, 0, -1], np.int32), np.array([4, 5, 6, 7, 8, 4], np.int32)
    b.kw["frequency"][6] = a.kw["frequency"][6] = np.nan
    a.vlen[2], a.vlen[3] = -1, 4
    refs, ws = [c.oracle() for c in (a, b)], specv.Workspace(256)
    assert [r["flags"] for r in refs] == [specv.DEV_VERIFY_LEN, specv.DEV_PARAM]
    h, start = a.history(), [logits_to_torch(c.x).view(6, 1, 4, V) for c in (a, b)]
    args = [dict(seats=dev(c.seats), draft_tokens=dev(c.tokens), verify_len=dev(c.vlen)) for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(40):
        xs = [x.clone() for x in start]
        ws.init()
        torch.cuda.synchronize()
        for s, x, k in zip(streams, xs, args):
            with torch.cuda.stream(s):
                specv.spec_logit_rules(x, h, workspace=ws, **k)
        torch.cuda.synchronize()
        assert ws.status() == specv.DEV_VERIFY_LEN | specv.DEV_PARAM
        for c, x, r in zip((a, b), xs, refs):
            check_rows(host(x).reshape(c.x.shape), c.x, r, "f32")
