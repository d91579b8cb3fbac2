"""Shared-prefix decode by its definition, in 64 bits, and the bound its outputs have to keep."""
import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


class Case:
    """Seeded inputs of one call.  Keys [0, prefix) lie in the pages of prefix_table, each row's
    own keys in pages of its own; everything else in the pool -- spare pages, the slots past a
    row's end, the slots of a row's first own page that belong to the prefix -- is NaN, and the
    entries of the block table below the prefix name no page at all."""

    def __init__(self, B, H_q, H_kv, d, top_k, prefix, suffix, page_size, dtype="fp16", seed=0,
                 idx=None, lens=None, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        dt = {"fp16": torch.float16, "bf16": torch.bfloat16}[dtype]
        self.B, self.H_q, self.H_kv, self.d, self.G = B, H_q, H_kv, d, H_q // H_kv
        self.prefix, self.page_size, self.dtype = prefix, page_size, dt
        self.scale = d ** -0.5
        self.q = (torch.randn((B, H_q, d), generator=g) * spread).to(dt)
        first, shared = prefix // page_size, -(-prefix // page_size)
        pages = -(-(prefix + suffix) // page_size)
        pages = max(pages, first + 1)
        if lens is None:
            lens = prefix + torch.randint(0, suffix + 1, (B,), generator=g)
            lens[-1] = prefix + suffix
        self.lens = torch.as_tensor(lens).to(torch.int32)
        n = shared + B * (pages - first) + 3
        self.k_pages = torch.full((n, H_kv, page_size, d), float("nan"), dtype=dt)
        self.v_pages = self.k_pages.clone()
        perm = torch.randperm(n, generator=g).to(torch.int32)
        self.prefix_table = perm[:shared].clone()
        self.table = torch.full((B, pages), -7, dtype=torch.int32)
        self.table[:, first:] = perm[shared:shared + B * (pages - first)].reshape(B, -1)
        for pool in (self.k_pages, self.v_pages):
            for i in range(shared):
                m = min(page_size, prefix - i * page_size)
                pool[int(self.prefix_table[i]), :, :m] = torch.randn((H_kv, m, d), generator=g).to(dt)
            for b in range(B):
                for i in range(first, pages):
                    lo = max(prefix - i * page_size, 0)
                    hi = min(page_size, int(self.lens[b]) - i * page_size)
                    if hi > lo:
                        pool[int(self.table[b, i]), :, lo:hi] = torch.randn(
                            (H_kv, hi - lo, d), generator=g).to(dt)
        if idx is None:
            idx = torch.rand((B, H_kv), generator=g).argsort(dim=1)[:, :top_k]
        self.idx = torch.as_tensor(idx).to(torch.int32).contiguous()

    def keys(self, pool, b, h):
        """float64 [lens[b], d]: the row's keys (or values) of one KV head, walked one by one."""
        ps, rows = self.page_size, []
        for n in range(int(self.lens[b])):
            page = self.prefix_table[n // ps] if n < self.prefix else self.table[b, n // ps]
            rows.append(pool[int(page), h, n % ps])
        return torch.stack(rows).double()

    def reference(self, scale=None, rows=None):
        """(want, bound) float64 [B, H_q, d]; NaN where nothing is written.

        The bound: one rounding of the output (u |o|) and one of every weight P before the
        second product (u A, A = the weighted mean of |v|, u half a step); fp16 weights below
        2^-14 round by up to 2^-25 of the largest; a score is a d-term fp32 sum, off by at most
        (d + 2) 2^-23 of the sum of its terms' sizes S, which changes a weight and the sum of
        weights by as much; exp2 is 2^-21 off; and the sums over n keys are fp32, n 2^-23."""
        scale = self.scale if scale is None else scale
        u = HALF_STEP[self.dtype]
        want = torch.full((self.B, self.H_q, self.d), float("nan"), dtype=torch.float64)
        bound = torch.zeros_like(want)
        for b in range(self.B) if rows is None else rows:
            for h in set(self.idx[b].tolist()):
                if not 0 <= h < self.H_kv:
                    continue
                k, v = self.keys(self.k_pages, b, h), self.keys(self.v_pages, b, h)
                q = self.q[b, h * self.G:(h + 1) * self.G].double()
                w = torch.softmax(q @ k.T * scale, dim=1)
                o, A = w @ v, w @ v.abs()
                S = abs(scale) * (q.abs() @ k.abs().T).max()
                n = k.shape[0]
                tiny = n * 2.0 ** -25 * w.max(dim=1, keepdim=True).values * v.abs().max() \
                    if self.dtype == torch.float16 else 0.0
                want[b, h * self.G:(h + 1) * self.G] = o
                bound[b, h * self.G:(h + 1) * self.G] = \
                    u * (o.abs() + A) + tiny + A * (2 * (self.d + 2) * 2.0 ** -23 * S + 2.0 ** -20
                                                    + n * 2.0 ** -23)
        return want, bound

    def check(self, out, want, bound, fill):
        got = out.detach().cpu()
        written = ~torch.isnan(want)
        assert (got[~written] == fill).all(), "a row that is not selected was written"
        assert torch.isfinite(got[written]).all()
        excess = ((got.double() - want).abs() - bound)[written]
        assert excess.numel() == 0 or excess.max() <= 0, \
            f"off by {float(excess.max())} over the bound"

    def on(self, device="cuda"):
        return [t.to(device) for t in (self.q, self.k_pages, self.v_pages, self.idx, self.lens,
                                       self.table)] + [self.prefix_table.to(device)]
