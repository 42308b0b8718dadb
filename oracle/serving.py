"""Plain 64-bit definitions of the serving operators (numpy, host).

TEST INFRASTRUCTURE ONLY, like the rest of this package: one loop per
definition, no step shared with the CUDA path. bf16 logits are uint16 bit
patterns, as in oracle.verify.
"""
import numpy as np

FLAG_TOKEN_RANGE, FLAG_VERIFY_LEN, FLAG_INDEX, FLAG_PARAM, FLAG_PAGES, FLAG_LENGTHS = 1, 4, 16, 32, 64, 128


def widen(x):
    """Logits as float64 (bf16 bits or float32)."""
    x = np.ascontiguousarray(x)
    with np.errstate(invalid="ignore"):  # signalling NaN patterns
        if x.dtype == np.uint16:
            return (x.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        return x.astype(np.float64)


def bits_of(words, V):
    """[..., W] uint32 words -> [..., V] bool."""
    w = np.ascontiguousarray(words).view(np.uint32)
    return ((w[..., :, None] >> np.arange(32, dtype=np.uint32)) & 1).astype(bool).reshape(w.shape[:-1] + (-1,))[..., :V]


def pack_bits(bits):
    V = bits.shape[-1]
    pad = np.zeros(bits.shape[:-1] + ((V + 31) // 32 * 32,), bool)
    pad[..., :V] = bits
    w = pad.reshape(bits.shape[:-1] + (-1, 32)).astype(np.uint32) << np.arange(32, dtype=np.uint32)
    return w.sum(-1, dtype=np.uint64).astype(np.uint32)


def logit_rules(x, B, K, rows, L, *, row_off=None, tokens=None, verify_len=None, seats=None, counts=None, seen=None,
                repetition=None, frequency=None, presence=None, bias_tokens=None, bias_values=None, mask=None,
                mask_rows=None):
    """x [n_rows, V]: returns dict(z float64 [n_rows, V] (rows not processed keep x), size float64 (the magnitudes
    that were added up, for error bounds), touched bool [n_rows, V] (elements a rule names), done bool [n_rows], flags)."""
    x = widen(x)
    n_rows, V = x.shape
    z, size = x.copy(), np.abs(x)
    touched, done, flags = np.zeros(x.shape, bool), np.zeros(n_rows, bool), 0
    for b in range(B):
        ell = L if verify_len is None else int(verify_len[b])
        if not 0 <= ell <= L:
            flags |= FLAG_VERIFY_LEN
            continue
        n = ell + rows - L
        seat = -1
        if counts is not None:
            seat = b if seats is None else int(seats[b])
            if seat >= counts.shape[0]:
                flags |= FLAG_INDEX
                continue
        r = f = p = None
        if seat >= 0:
            r = 1.0 if repetition is None else float(repetition[seat])
            f = 0.0 if frequency is None else float(frequency[seat])
            p = 0.0 if presence is None else float(presence[seat])
            if not (2.0 ** -100 <= r <= 2.0 ** 100 and np.isfinite(f) and np.isfinite(p)):
                flags |= FLAG_PARAM
                continue
        if row_off is not None and not (0 <= row_off[b] and row_off[b] + n <= n_rows):
            flags |= FLAG_INDEX
            continue
        m = -1
        if mask is not None:
            m = b if mask_rows is None else int(mask_rows[b])
            if m >= mask.shape[0]:
                flags |= FLAG_INDEX
                continue
        for q in range(K):
            for i in range(n):
                row = int(row_off[b]) + i if row_off is not None else (b * K + q) * rows + i
                done[row] = True
                if seat >= 0:
                    c = counts[seat].astype(np.int64)
                    known = bits_of(seen[seat], V).copy()
                    for k in range(i):
                        t = int(tokens[b, k])
                        if 0 <= t < V:
                            c[t] += 1
                            known[t] = True
                        elif r != 1.0 or f != 0.0 or p != 0.0:
                            flags |= FLAG_TOKEN_RANGE
                    with np.errstate(invalid="ignore", over="ignore"):
                        v = np.where(known, np.where(x[row] > 0, x[row] / r, x[row] * r), x[row])
                        size[row] = np.abs(v) + abs(f) * c + abs(p) * (c > 0)
                        v = v - f * c - p * (c > 0)
                    touched[row] |= known
                    if bias_tokens is not None:
                        for t, a in zip(bias_tokens[seat], bias_values[seat]):
                            if 0 <= t < V:
                                v[t] += float(a)
                                size[row, t] += abs(float(a))
                                touched[row, t] = True
                            elif t >= V:
                                flags |= FLAG_TOKEN_RANGE
                    z[row] = v
                if m >= 0:
                    off = ~bits_of(mask[m, i], V)
                    z[row, off] = -np.inf
                    touched[row] |= off
    return dict(z=z, size=size, touched=touched, done=done, flags=flags)


def history_add(counts, seen, seats, groups, output):
    """groups: one token list per request. Returns (counts, seen, flags)."""
    counts, V = counts.copy(), counts.shape[1]
    bits, flags = bits_of(seen, V).copy(), 0
    for b, toks in enumerate(groups):
        s = b if seats is None else int(seats[b])
        for t in toks:
            t = int(t)
            if t < 0 or s < 0:
                continue
            if s >= counts.shape[0]:
                flags |= FLAG_INDEX
            elif t >= V:
                flags |= FLAG_TOKEN_RANGE
            else:
                bits[s, t] = True
                if output:
                    counts[s, t] += 1
    return counts, pack_bits(bits), flags


class Pages:
    """The page bookkeeping of spec_kv_map / spec_kv_release with Python lists."""

    def __init__(self, seats, max_pages, free, page_size):
        self.held = [[] for _ in range(seats)]
        self.stack = [int(p) for p in free]  # the last entry is the top
        self.n_pages, self.max_pages, self.ps = len(self.stack), max_pages, page_size

    def _twice(self, seats):
        s = [int(x) for x in seats if x >= 0]
        return {x for x in s if s.count(x) > 1}

    def map(self, ctx, off, N, seats=None):
        """Returns dict(slots, positions, seq_len, tables, flags)."""
        B = len(ctx)
        seats = list(range(B)) if seats is None else [int(x) for x in seats]
        slots, pos = [-1] * N, [0] * N
        seq, tables, flags = [], [], 0
        if any(o < 0 or o > N for o in off) or any(off[b] > off[b + 1] for b in range(B)):
            return dict(slots=slots, positions=pos, seq_len=[-1] * B, tables=[[] for _ in range(B)],
                        flags=FLAG_LENGTHS)
        twice = self._twice([s for s in seats if s < len(self.held)])
        room, asked = len(self.stack), 0
        taken = 0
        for b in range(B):
            s, total = seats[b], int(ctx[b]) + int(off[b + 1]) - int(off[b])
            if s < 0:
                seq.append(0)
                tables.append([])
                continue
            ok = True
            if s >= len(self.held) or s in twice:
                flags, ok = flags | FLAG_INDEX, False
            elif ctx[b] < 0 or total > 0x7fffffff:
                flags, ok = flags | FLAG_LENGTHS, False
            else:
                want = -(-total // self.ps)
                need = max(0, want - len(self.held[s]))
                if want > self.max_pages:
                    flags, ok = flags | FLAG_PAGES, False
                else:
                    asked += need
                    if need and asked > room:
                        flags, ok = flags | FLAG_PAGES, False
            if not ok:
                seq.append(-1)
                tables.append([])
                continue
            for _ in range(need):
                self.held[s].append(self.stack[room - 1 - taken])
                taken += 1
            seq.append(total)
            tables.append(self.held[s][:want])
            for t in range(int(off[b]), int(off[b + 1])):
                at = int(ctx[b]) + t - int(off[b])
                slots[t] = self.held[s][at // self.ps] * self.ps + at % self.ps
                pos[t] = at
        del self.stack[room - taken:]
        return dict(slots=slots, positions=pos, seq_len=seq, tables=tables, flags=flags)

    def release(self, seats, keep=None):
        twice, flags, back, keeps = self._twice([s for s in seats if s < len(self.held)]), 0, [], []
        for b, s in enumerate(seats):
            s = int(s)
            if s < 0:
                continue
            k = 0 if keep is None else int(keep[b])
            if s >= len(self.held) or s in twice:
                flags |= FLAG_INDEX
            elif k < 0:
                flags |= FLAG_LENGTHS
            else:
                n = min(len(self.held[s]), -(-k // self.ps))
                back += self.held[s][n:]
                keeps.append((s, n))
        if len(self.stack) + len(back) > self.n_pages:
            return FLAG_LENGTHS
        for s, n in keeps:
            del self.held[s][n:]
        self.stack += back
        return flags
