"""64-bit plain forms of the operators of include/gdn_block.h, for the tests: written from the definitions, on the CPU."""
import math

import torch

F64 = torch.float64


def lens_to_cu(qs, device="cpu"):
    cu = [0]
    for q in qs:
        cu.append(cu[-1] + q)
    return torch.tensor(cu, dtype=torch.int32, device=device)


def attention(q, k_cache, v_cache, table, kv_lens, qs, scale, window=0):
    """o, lse and the weighted magnitude sum_j p_j |v_j| of every query, all fp64 (loops over queries and heads)."""
    q, kc, vc = q.cpu().to(F64), k_cache.cpu().to(F64), v_cache.cpu().to(F64)
    table, kv_lens = table.cpu(), kv_lens.cpu()
    T, Hq, D = q.shape
    P, Hkv = kc.shape[1], kc.shape[2]
    o, mag = torch.zeros(T, Hq, D, dtype=F64), torch.zeros(T, Hq, D, dtype=F64)
    lse = torch.full((T, Hq), -math.inf, dtype=F64)
    at = 0
    for n, ql in enumerate(qs):
        kv = int(kv_lens[n])
        slots = torch.arange(kv)
        pages = table[n, slots // P].long()
        k, v = kc[pages, slots % P], vc[pages, slots % P]
        for i in range(ql):
            pos = kv - ql + i
            lo = max(0, pos - window + 1) if window else 0
            if pos < 0:
                continue
            for h in range(Hq):
                kk, vv = k[lo:pos + 1, h // (Hq // Hkv)], v[lo:pos + 1, h // (Hq // Hkv)]
                z = scale * (kk @ q[at + i, h])
                lse[at + i, h] = torch.logsumexp(z, 0)
                p = torch.exp(z - lse[at + i, h])
                o[at + i, h] = p @ vv
                mag[at + i, h] = p @ vv.abs()
        at += ql
    return o, lse, mag


def rotate(x, table, positions, interleaved=False, inverse=False):
    """x [T, H, D] fp64, table [rows, rot / 2, 2]; a position outside the table leaves its token as it is."""
    x, table, positions = x.cpu().to(F64), table.cpu().to(F64), positions.cpu()
    rot, y = 2 * table.shape[1], x.clone()
    for t in range(x.shape[0]):
        p = int(positions[t])
        if not 0 <= p < table.shape[0]:
            continue
        c, s = table[p, :, 0], table[p, :, 1] * (-1 if inverse else 1)
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            y[t, :, a] = x[t, :, a] * c[i] - x[t, :, b] * s[i]
            y[t, :, b] = x[t, :, b] * c[i] + x[t, :, a] * s[i]
    return y


def norm(x, weight, residual=None, eps=1e-6, offset=0.0):
    h = x.cpu().to(F64) + (0 if residual is None else residual.cpu().to(F64))
    rstd = (h.square().mean(-1) + eps).rsqrt()
    return h, rstd, h * rstd[..., None] * (weight.cpu().to(F64) + offset)


def norm_grads(dy, h, weight, rstd, dh=None, offset=0.0):
    dy, h, w, r = dy.cpu().to(F64), h.cpu().to(F64), weight.cpu().to(F64) + offset, rstd.cpu().to(F64)[:, None]
    g = dy * w
    dx = r * g - h * r ** 3 * (g * h).mean(-1, keepdim=True)
    if dh is not None:
        dx = dx + dh.cpu().to(F64)
    return dx, (dy * h * r).sum(0)


class Pages:
    """The bookkeeping of a paged cache in Python lists, by the rules of gdn_block.h."""

    def __init__(self, seqs, width, pages, page):
        self.table, self.lens = [[-1] * width for _ in range(seqs)], [0] * seqs
        self.ref, self.width, self.page = [0] * pages, width, page

    def _free(self):
        return [i for i, r in enumerate(self.ref) if r <= 0]

    def _held(self, n):
        return -(-n // self.page)

    def extend(self, seqs, add):
        free, ok, asked = self._free(), [], 0
        for s, d in zip(seqs, add):
            good = 0 <= s < len(self.lens) and d >= 0 and self.lens[s] + d <= self.width * self.page
            if good and self.lens[s] % self.page and d:
                good = self.ref[self.table[s][self._held(self.lens[s]) - 1]] == 1
            need = self._held(self.lens[s] + d) - self._held(self.lens[s]) if good else 0
            asked += need
            if need and asked > len(free):
                good = False
            if good:
                first = self._held(self.lens[s])
                for j in range(need):
                    page = free[asked - need + j]
                    self.table[s][first + j] = page
                    self.ref[page] = 1
                self.lens[s] += d
            ok.append(int(good))
        return ok

    def fork(self, parents, children):
        """Returns (new pages, copied page pairs, copied state pairs)."""
        free, new, copies, states, rank = self._free(), [], [], [], 0
        n = len(self.lens)
        empty = [x == 0 for x in self.lens]
        lens = list(self.lens)
        for p, c in zip(parents, children):
            if not (0 <= p < n and 0 <= c < n and p != c and empty[c]):
                new.append(-2)
                continue
            full, part = lens[p] // self.page, lens[p] % self.page != 0
            if part:
                if rank >= len(free):
                    rank += 1
                    new.append(-2)
                    continue
                new.append(free[rank])
                rank += 1
            else:
                new.append(-1)
            self.table[c] = self.table[p][:full] + [-1] * (self.width - full)
            for pg in self.table[p][:full]:
                self.ref[pg] += 1
            if part:
                self.table[c][full] = new[-1]
                self.ref[new[-1]] = 1
                copies.append((self.table[p][full], new[-1]))
            states.append((p, c))
            self.lens[c] = lens[p]
        return new, copies, states

    def free(self, seqs):
        for s in seqs:
            if 0 <= s < len(self.lens):
                for pg in self.table[s]:
                    if pg >= 0:
                        self.ref[pg] -= 1
                self.table[s] = [-1] * self.width
                self.lens[s] = 0

    def compact(self):
        live = sum(r > 0 for r in self.ref)
        holes = [i for i in range(live) if self.ref[i] <= 0]
        highs = [i for i in range(live, len(self.ref)) if self.ref[i] > 0]
        to = dict(zip(highs, holes))
        for s, d in to.items():
            self.ref[d], self.ref[s] = self.ref[s], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return list(to.items())
