"""Serving operators, host side (CPU only): refusals of the C ABI where no GPU
is visible, the binding's shape checks, and hand-worked cases of the plain
definitions that the GPU tests compare with."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_block_spec_b200 as specv
from oracle import serving as plain
from speculative_decoding_block_spec_b200 import synth

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E, I32 = torch.empty, torch.int32

REJECT = r'''
import ctypes, sys
sys.path.insert(0, %r)
import speculative_decoding_block_spec_b200 as specv
from speculative_decoding_block_spec_b200.serving import _CHistory, _CPages
lib = specv.lib()
P = 1 << 20                       # an aligned placeholder, never dereferenced
ARG, UNSUP, WS = -1, -2, -4

def hist(**kw):
    c = _CHistory(counts=P, seen=P, repetition=P, frequency=P, presence=P, n_bias=0, seats=8, V=64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c

names = ["x", "out", "dtype", "off", "n_rows", "B", "K", "rows", "L", "V", "tok", "vlen", "h", "seats", "mask", "nm",
         "ml", "mr", "ws", "wsb", "st"]
def rules(h=None, **kw):
    a = dict(zip(names, [P, P, 1, None, 2 * 5, 2, 1, 5, 4, 64, P, None, ctypes.byref(h if h is not None else hist()), None, None, 0, 0,
                         None, P, 256, None]))
    a.update(kw)
    return lib.spec_logit_rules(*[a[n] for n in names])

assert rules(x=None) == ARG and rules(out=None) == ARG and rules(dtype=2) == ARG and rules(V=0) == ARG
assert rules(B=0) == ARG and rules(K=0) == ARG and rules(L=-1) == ARG and rules(rows=3) == ARG and rules(rows=6) == ARG
assert rules(n_rows=9) == ARG                                  # dense rows are B * K * rows
assert rules(B=5000, n_rows=25000) == UNSUP and rules(K=9, n_rows=90) == UNSUP
assert rules(L=33, rows=34, n_rows=68) == UNSUP and rules(V=(1 << 20) + 1) == UNSUP
assert rules(off=P, K=2, n_rows=20) == ARG                     # packed rows have one branch
assert rules(off=P, rows=4, n_rows=8) == ARG                   # and are target rows
assert rules(tok=None) == ARG                                  # a history needs the drafted tokens
assert rules(h=hist(V=32)) == ARG and rules(h=hist(seats=1)) == ARG    # request 1 has no seat 1
assert rules(h=hist(counts=None)) == ARG and rules(h=hist(seen=None)) == ARG and rules(h=hist(n_bias=-1)) == ARG
assert rules(h=hist(n_bias=4)) == ARG and rules(h=hist(n_bias=1025, bias_tokens=P, bias_values=P)) == UNSUP
assert rules(h=hist(seats=65537)) == UNSUP
assert rules(mask=P, nm=1, ml=5) == ARG                        # mask b for request b
assert rules(mask=P, nm=2, ml=4) == ARG and rules(mask=P, nm=0, ml=5, mr=P) == ARG
assert rules(x=P + 1) == ARG and rules(seats=P + 2) == ARG and rules(mask=P + 1, nm=2, ml=5) == ARG
assert rules(out=P + 64) == ARG                                # overlaps, not in place
assert rules(ws=None) == WS and rules(wsb=255) == WS and rules(ws=P + 8) == WS
assert lib.spec_rules_workspace_size(0) == 0 == lib.spec_rules_workspace_size(4097) and lib.spec_rules_workspace_size(8) == 256
assert lib.spec_kv_workspace_size(0) == 0 == lib.spec_kv_workspace_size(4097) and lib.spec_kv_workspace_size(8) == 512

H = ctypes.byref(hist())
add = lambda h=H, seats=P, B=2, tok=P, n=8, off=None, output=1, ws=P, wsb=256: lib.spec_history_add(h, seats, B, tok, n, off, output, ws, wsb, None)
assert add(h=None) == ARG and add(B=0) == ARG and add(B=4097) == UNSUP and add(tok=None) == ARG and add(n=-1) == ARG
assert add(n=7) == ARG and add(n=1 << 31) == ARG and add(output=2) == ARG and add(off=P + 1) == ARG and add(ws=None) == WS
assert add(B=9, seats=None, n=9) == ARG
assert lib.spec_history_clear(None, P, 2, P, 256, None) == ARG and lib.spec_history_clear(H, P, 0, P, 256, None) == ARG
assert lib.spec_history_clear(H, P, 2, P, 128, None) == WS

def pages(**kw):
    c = _CPages(page_table=P, owned=P, free_pages=P, free_count=P, seats=8, max_pages=4, n_pages=16, page_size=16)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)
def kv(p=None, seats=P, B=2, ctx=P, off=P, n=8, slots=P, pos=P, seq=P, bt=P, ws=P, wsb=512):
    return lib.spec_kv_map(p or pages(), seats, B, ctx, off, n, slots, pos, seq, bt, ws, wsb, None)
assert lib.spec_kv_map(None, P, 2, P, P, 8, P, P, P, P, P, 512, None) == ARG
assert kv(ctx=None) == ARG and kv(off=None) == ARG and kv(seq=None) == ARG and kv(slots=None) == ARG and kv(n=-1) == ARG
assert kv(B=0) == ARG and kv(B=4097) == UNSUP and kv(slots=P + 4) == ARG and kv(seats=None, B=9) == ARG
for bad in (dict(page_table=None), dict(owned=None), dict(free_pages=None), dict(free_count=None), dict(max_pages=0),
            dict(n_pages=0), dict(page_size=0), dict(seats=0)):
    assert kv(p=pages(**bad)) == ARG, bad
assert kv(p=pages(seats=65537)) == UNSUP and kv(p=pages(max_pages=1 << 30)) == UNSUP
assert kv(ws=None) == WS and kv(wsb=256) == WS
assert lib.spec_kv_release(None, P, 2, P, P, 512, None) == ARG and lib.spec_kv_release(pages(), P, 0, P, P, 512, None) == ARG
assert lib.spec_kv_release(pages(), P, 2, P + 2, P, 512, None) == ARG and lib.spec_kv_release(pages(), P, 2, P, P, 256, None) == WS
print("ok")
'''


def test_c_abi_refuses_before_any_launch():
    r = subprocess.run([sys.executable, "-c", REJECT % ROOT], env=dict(os.environ, CUDA_VISIBLE_DEVICES=""),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), (r.stdout[-2000:], r.stderr[-4000:])


def _hist(seats=4, V=64, n=3):
    return specv.History.empty(seats, V, n, device="cpu")


def test_binding_checks_state_tables():
    h = _hist()
    assert h.counts.shape == (4, 64) and h.seen.shape == (4, 2) and h.bias_tokens.shape == (4, 3)
    z = torch.zeros
    with pytest.raises(ValueError, match="seen"):
        specv.History(z(4, 64, dtype=I32), z(4, 3, dtype=I32))
    with pytest.raises(TypeError, match="counts"):
        specv.History(z(4, 64), z(4, 2, dtype=I32))
    with pytest.raises(ValueError, match="bias"):
        specv.History(z(4, 64, dtype=I32), z(4, 2, dtype=I32), bias_tokens=z(4, 2, dtype=I32))
    with pytest.raises(ValueError, match="presence"):
        specv.History(z(4, 64, dtype=I32), z(4, 2, dtype=I32), presence=z(3))
    p = specv.KvPages.empty(3, 5, 7, 16, device="cpu")
    assert p.free_pages.tolist() == [6, 5, 4, 3, 2, 1, 0] and int(p.free_count) == 7
    with pytest.raises(ValueError, match="owned"):
        specv.KvPages(z(3, 5, dtype=I32), z(2, dtype=I32), z(7, dtype=I32), z(1, dtype=I32), 16)
    with pytest.raises(ValueError, match="page_size"):
        specv.KvPages(z(3, 5, dtype=I32), z(3, dtype=I32), z(7, dtype=I32), z(1, dtype=I32), 0)


@pytest.mark.parametrize("kw,msg", [
    (dict(logits=E(3, 64)), "expected"),                                          # decoding rows are [B, 1, V]
    (dict(logits=E(3, 6, 64)), "logits"),                                         # neither L nor L + 1 rows
    (dict(logits=E(2, 5, 64)), "logits"),                                         # another B
    (dict(logits=E(3, 5, 64), draft_tokens=None), "draft_tokens"),
    (dict(logits=E(3, 5, 32)), "history"),
    (dict(logits=E(3, 5, 64), seats=E(2, dtype=I32)), "seats"),
    (dict(logits=E(3, 5, 64), verify_len=E(4, dtype=I32)), "verify_len"),
    (dict(logits=E(3, 5, 64), mask=E(3, 4, 2, dtype=I32)), "mask"),               # fewer mask rows than rows
    (dict(logits=E(3, 5, 64), mask=E(3, 5, 3, dtype=I32)), "mask"),
    (dict(logits=E(3, 5, 64), mask=E(2, 5, 2, dtype=I32)), "mask_rows"),
    (dict(logits=E(3, 5, 64), mask_rows=E(3, dtype=I32)), "mask_rows"),
    (dict(logits=E(3, 5, 64), out=E(3, 4, 64)), "out"),
    (dict(logits=E(9, 64), target_row_off=E(2, dtype=I32)), "target_row_off"),
    (dict(logits=E(3, 5, 64), target_row_off=E(3, dtype=I32)), "packed"),
    (dict(logits=E(5, 3, 64).transpose(0, 1)), "contiguous"),
])
def test_binding_checks_rules(kw, msg):
    args = dict(draft_tokens=E(3, 4, dtype=I32), history=_hist())
    args.update(kw)
    with pytest.raises(ValueError, match=msg):
        specv.spec_logit_rules(args.pop("logits"), args.pop("history"), **args)


def test_binding_checks_the_other_calls():
    h, p = _hist(), specv.KvPages.empty(3, 5, 7, 16, device="cpu")
    with pytest.raises(ValueError, match="tokens"):
        specv.spec_history_add(h, E(3, dtype=I32))
    with pytest.raises(ValueError, match="seats"):
        specv.spec_history_add(h, E(5, 2, dtype=I32))
    with pytest.raises(TypeError, match="seats"):
        specv.spec_history_clear(h, E(3))
    with pytest.raises(ValueError, match="offsets"):
        specv.spec_kv_map(p, E(3, dtype=I32), E(3, dtype=I32), 8)
    with pytest.raises(ValueError, match="block_table"):
        specv.spec_kv_map(p, E(3, dtype=I32), E(4, dtype=I32), 8, block_table=E(3, 4, dtype=I32))
    with pytest.raises(ValueError, match="kv_slots"):
        specv.spec_kv_map(p, E(3, dtype=I32), E(4, dtype=I32), 8,
                          out=(E(7, dtype=torch.int64), E(8, dtype=I32), E(3, dtype=I32)))
    with pytest.raises(ValueError, match="seats"):
        specv.spec_kv_map(p, E(4, dtype=I32), E(5, dtype=I32), 8)
    with pytest.raises(ValueError, match="keep_len"):
        specv.spec_kv_release(p, E(2, dtype=I32), keep_len=E(3, dtype=I32))
    # no CPU path: well-formed host tensors are refused
    with pytest.raises((TypeError, RuntimeError, AssertionError)):
        specv.spec_history_clear(h, torch.zeros(2, dtype=I32), workspace=None)


# ------------------------------------------------------- the plain definitions

def test_plain_rules_by_hand():
    # V = 4, one request, L = 2, tokens (1, 1): row 0 sees the history alone, row 1 one more 1, row 2 two
    x = np.array([[2.0, -2.0, 4.0, 1.0]] * 3, np.float32)
    counts = np.array([[0, 1, 0, 0]], np.int32)
    seen = plain.pack_bits(np.array([[True, True, False, False]]))
    r = plain.logit_rules(x, 1, 1, 3, 2, tokens=np.array([[1, 1]], np.int32), counts=counts, seen=seen,
                          repetition=[2.0], frequency=[0.5], presence=[0.25], bias_tokens=np.array([[3, -1, 3]]),
                          bias_values=np.array([[1.0, 9.0, 2.0]]),
                          mask=plain.pack_bits(np.array([[[True, True, False, True]] * 2 + [[False] * 4]])))
    assert r["z"][0].tolist() == [1.0, -4.0 - 0.5 - 0.25, -np.inf, 4.0]
    assert r["z"][1].tolist() == [1.0, -4.0 - 1.0 - 0.25, -np.inf, 4.0]
    assert r["z"][2].tolist() == [-np.inf] * 4 and r["flags"] == 0


def test_plain_pages_by_hand():
    p = plain.Pages(seats=3, max_pages=3, free=[5, 6, 7, 8, 9], page_size=2)
    r = p.map([0, 3, 0], [0, 3, 4, 4], 6, seats=[2, 0, -1])
    # request 0: 3 tokens, 2 pages (9, 8); request 1: 4 tokens in the cache after the step, 2 pages (7, 6)
    assert r["slots"] == [18, 19, 16, 13, -1, -1] and r["positions"] == [0, 1, 2, 3, 0, 0]
    assert r["seq_len"] == [3, 4, 0] and p.stack == [5] and p.held == [[7, 6], [], [9, 8]]
    assert p.map([3], [0, 4], 4, seats=[2])["flags"] == plain.FLAG_PAGES      # 4 pages: more than a row holds
    assert p.map([4, 0], [0, 1, 4], 4, seats=[0, 1])["seq_len"] == [5, -1]    # the last page, then none
    assert p.release([2, 0], [2, 0]) == 0 and p.stack == [8, 7, 6, 5] and p.held == [[], [], [9]]
    assert p.release([1, 1]) == plain.FLAG_INDEX


def test_plain_history_by_hand():
    c, s, fl = plain.history_add(np.zeros((2, 40), np.int32), np.zeros((2, 2), np.uint32), [1, 1], [[3, 3, -1], [39, 40]],
                                 True)
    assert c[1, 3] == 2 and c[1, 39] == 1 and c.sum() == 3 and s.tolist() == [[0, 0], [8, 128]]
    assert fl == plain.FLAG_TOKEN_RANGE


@pytest.mark.parametrize("pad", [-1, -2, -2 ** 31])
def test_plain_pages_take_every_negative_seat_as_padding(pad):
    p = plain.Pages(seats=2, max_pages=3, free=[5, 6, 7], page_size=2)
    r = p.map([1, 2 ** 31 - 1, 0], [0, 1, 3, 4], 4, seats=[1, pad, pad])
    assert r["seq_len"] == [2, 0, 0] and r["slots"] == [15, -1, -1, -1] and r["flags"] == 0 and p.stack == [5, 6]
    assert p.release([pad, 1, pad], [-3, 0, 1]) == 0 and p.stack == [5, 6, 7]


# ------------------------------------- which rows a verify step has to edit

def _edited(x, tokens, ok, **kw):
    B, L = tokens.shape
    r = plain.logit_rules(x.reshape(-1, x.shape[-1]), B, 1, x.shape[1], L, tokens=tokens, mask=plain.pack_bits(ok), **kw)
    return r["z"].astype(np.float32).reshape(x.shape)


def test_a_forbidden_draft_is_rejected_when_the_target_alone_is_edited():
    """The second of three drafted tokens is forbidden. With the target rows edited it is rejected and an allowed token
    ends the block; with the draft rows edited after the draw both probabilities are 0, and there is no decision."""
    x = synth.custom(B=1, L=3, V=64, T=1.0, dtype="f32", seed=9, cid=721)
    ok = np.ones((1, 4, 64), bool)
    ok[0, 1, x.tokens[0, 1]] = False
    u = np.zeros((1, 3), np.float32)
    target, draft = _edited(x.target, x.tokens, ok), _edited(x.draft, x.tokens, ok)
    r = oracle.verify(target, x.draft, x.tokens, u, x.g, 1.0)
    assert r["accept_len"].tolist() == [1] and r["flags"] == 0 and r["out_tokens"][0, 0] == x.tokens[0, 0]
    assert r["out_tokens"][0, 1] >= 0 and ok[0, 1, r["out_tokens"][0, 1]]
    r = oracle.verify(target, draft, x.tokens, u, x.g, 1.0)
    assert r["accept_len"].tolist() == [-1] and r["flags"] == specv.DEV_NONFINITE


def test_edited_target_rows_against_the_proposal_as_drawn_are_lossless():
    """Blocks of two tokens drawn from fixed rows q; penalties and a mask on the target rows. The first token follows the
    edited row 0, the second, where the first was accepted as a, the edited row 1 of prefix a: each frequency within 5
    standard deviations (at most 63 of them: one outside has a chance of 4e-5). With the draft rows edited after the draw the
    same statistic is far outside, so it would see the error."""
    g = np.random.default_rng(11)
    V, N = 8, 60000
    t, q = g.standard_normal((3, V)).astype(np.float32), g.standard_normal((2, V)).astype(np.float32)
    ok = np.ones((3, V), bool)
    ok[0, 2] = ok[1, 5] = False
    kw = dict(counts=np.array([[2, 0, 0, 1, 0, 0, 0, 0]], np.int32), repetition=[1.6], frequency=[0.4], presence=[0.8],
              seen=plain.pack_bits(np.array([[True, True, False, True] + [False] * 4])))
    pairs = np.array([(a, b) for a in range(V) for b in range(V)], np.int32)
    one = dict(kw, seats=np.zeros(len(pairs), np.int32), mask_rows=np.zeros(len(pairs), np.int32))
    et = _edited(np.broadcast_to(t, (V * V, 3, V)), pairs, ok[None], **one)
    eq = _edited(np.broadcast_to(q, (V * V, 2, V)), pairs, ok[None], **one)

    def softmax(z):
        w = np.exp(z.astype(np.float64) - z.max(-1, keepdims=True))
        return w / w.sum(-1, keepdims=True)

    draw = [g.choice(V, N, p=softmax(q[i])) for i in range(2)]
    tokens, at = np.stack(draw, 1).astype(np.int32), draw[0] * V + draw[1]
    u = g.random((N, 2), dtype=np.float32)
    gumbel = -np.log(-np.log(g.random((N, 3, V)))).astype(np.float32)

    def worst(draft):
        r = oracle.verify(et[at], draft, tokens, u, gumbel, 1.0)
        first, second = r["out_tokens"][:, 0], r["out_tokens"][:, 1]
        p0, z = softmax(et[0, 0]), []
        groups = [(first[first >= 0], p0)]
        for a in range(V):
            groups.append((second[(r["accept_len"] >= 1) & (first == a)], softmax(et[a * V, 1])))
        for got, p in groups:
            n = len(got)
            if n >= 2000:
                freq = np.bincount(got, minlength=V) / n
                assert (freq[p == 0] == 0).all()
                z += list(np.abs(freq - p)[p > 0] / np.sqrt(p * (1 - p) / n)[p > 0])
        return max(z), len(z)

    z, n = worst(np.broadcast_to(q, (N, 2, V)).copy())
    assert z < 5 and n <= 63, (z, n)
    assert worst(eq[at])[0] > 20
