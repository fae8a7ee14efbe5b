"""One sparse-attention decode layer on the library's operators, with random weights.

A step takes the P draft tokens of every request (P = 1: plain decode) through

  idx_add_rmsnorm_fp8   residual addition and norm of the hidden state, e4m3 with row scales
  a bf16 projection     (a plain library product) to queries, keys, values, index queries/keys
  idx_store_kv          the new keys and values into the paged cache, the index keys into
                        the index pool
  idx_add_rmsnorm_fp8   the index queries, head by head, into the e4m3 form the scorer takes
  idx_score_topk        the 128-token blocks each index head chooses
  idx_attn_blocks       attention over those blocks (or idx_attn_paged over everything)

With rotary=True the queries and keys are normed head by head and turned by their position on
the way (time, height and width where positions has three rows), which with the stores and the
index queries' form is

  idx_norm_rope_store   one pass over the projection for the attention, one for the index

and with kv_dtype "nvfp4" the cache is held in four bits (idx_store_kv_nvfp4,
idx_attn_blocks_nvfp4, idx_attn_paged_nvfp4).

    python examples/sparse_decode_layer.py [--requests 4] [--context 3000] [--steps 3]
                                           [--kv-dtype nvfp4] [--rotary]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_packed_gb300 as idx  # noqa: E402

PAGE, DIM = 64, 128


def rotation_table(positions, rotary_dim=DIM, base=1e6, device="cuda"):
    """fp32 [positions, rotary_dim]: the cosines of a position's angles, then their sines."""
    turn = base ** (-torch.arange(0, rotary_dim, 2, device=device, dtype=torch.float64) / rotary_dim)
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * turn
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class SparseDecodeLayer:
    def __init__(self, hidden=1024, q_heads=16, kv_heads=1, index_heads=4, topk=16, init_blocks=1,
                 local_blocks=4, max_requests=4, max_tokens=8192, drafts=1, kv_dtype="bf16", seed=0,
                 device="cuda", rotary=False):
        g = torch.Generator(device=device).manual_seed(seed)
        self.hidden, self.q_heads, self.kv_heads, self.index_heads = hidden, q_heads, kv_heads, index_heads
        self.topk, self.init_blocks, self.local_blocks = topk, init_blocks, local_blocks
        self.drafts, self.kv_dtype, self.device = drafts, kv_dtype, device
        self.heads = (q_heads, kv_heads, kv_heads, index_heads, 1)
        self.norm_weight = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.index_norm, self.q_norm, self.k_norm = torch.ones((3, DIM), dtype=torch.bfloat16, device=device)
        # the angles of the positions, and the axis that each pair goes by with three of them
        self.table = rotation_table(max_tokens, device=device) if rotary else None
        self.pair_axis = bytes(i % 3 for i in range(DIM // 2))
        self.outer = (1.0, 1.0)     # of an NVFP4 cache's keys and values: both are near 1 here
        self.w = (torch.randn((sum(self.heads) * DIM, hidden), generator=g, device=device)
                  * hidden ** -0.5).to(torch.bfloat16)
        # pages of all requests, in a random order behind a page table
        self.max_pages = -(-max_tokens // PAGE)
        pages = max_requests * self.max_pages
        self.page_table = torch.randperm(pages, generator=g, device=device).to(torch.int32).reshape(
            max_requests, self.max_pages)
        self.k, self.v = (self._plane(pages * kv_heads, kv_dtype) for _ in range(2))
        self.index_keys = self._plane(pages, "fp8_e4m3")
        self.score_ws = idx.alloc_workspace(max_requests, drafts, index_heads, self.max_pages, device)
        self.attn_ws = max((idx.alloc_attn_workspace(drafts, q_heads, kv_heads, n, device)
                            for n in (0, index_heads)), key=lambda t: t.numel())

    def _plane(self, head_pages, dtype):
        """payload and scale of one plane; a page's tokens are written before they are read."""
        rows = head_pages * PAGE
        if dtype == "bf16":
            return torch.empty((rows, DIM), dtype=torch.bfloat16, device=self.device), None
        if dtype == "nvfp4":
            return (torch.empty((rows, DIM // 2), dtype=torch.uint8, device=self.device),
                    torch.empty((rows, DIM // 16), dtype=torch.uint8, device=self.device))
        return (torch.empty((rows, DIM), dtype=torch.uint8, device=self.device),
                torch.empty((rows, 1), dtype=torch.float32, device=self.device))

    def slots(self, request, positions):
        """Cache slots (page * 64 + offset) of these positions of these requests."""
        return self.page_table[request, positions // PAGE].long() * PAGE + positions % PAGE

    def _norm(self, x, residual, weight):
        """Codes and row scales of the norm of x (+ residual), and the new residual."""
        out = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        scale = torch.empty((x.shape[0], 1), device=x.device)
        new = None if residual is None else torch.empty_like(residual)
        idx.idx_add_rmsnorm_fp8(x, residual, weight, 1e-6, 0, out, scale, new)
        return out, scale, new

    def _norm_rope_store(self, parts, slots, positions):
        """Queries, and index queries with their scales, normed and turned; the keys and values
        into the caches."""
        q, k, v, iq, ik = parts
        by = self.pair_axis if positions.dim() == 2 else None
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        idx.idx_norm_rope_store(q, k, v, self.q_norm, self.k_norm, 1e-6, self.table, positions, by, False,
                                slots, out, None, *self.k, *self.v, self.kv_dtype, self.kv_heads,
                                *(self.outer if self.kv_dtype == "nvfp4" else ()))
        codes = torch.empty(iq.shape, dtype=torch.float8_e4m3fn, device=q.device)
        scale = torch.empty(iq.shape[:2], device=q.device)
        idx.idx_norm_rope_store(iq, ik, None, self.index_norm, self.index_norm, 1e-6, self.table, positions, by,
                                False, slots, codes, scale, *self.index_keys, None, None, "fp8_e4m3", 1)
        return out, k, v, (codes, scale), ik

    def write(self, x, residual, slots, positions=None):
        """The tokens' projections; their keys and values go into the caches.  positions, with a
        rotation: int32 [tokens], or [3, tokens]."""
        codes, scale, new = self._norm(x, residual, self.norm_weight)
        # e4m3 codes are exact in bf16: the row scale comes after the product
        proj = ((codes.to(torch.bfloat16) @ self.w.T) * scale).to(torch.bfloat16)
        parts = proj.reshape(x.shape[0], sum(self.heads), DIM).split(self.heads, dim=1)
        if self.table is not None:
            return self._norm_rope_store(parts, slots, positions), new
        if self.kv_dtype == "nvfp4":
            idx.idx_store_kv_nvfp4(parts[1], parts[2], slots, *self.k, *self.v, self.kv_heads, *self.outer)
        else:
            idx.idx_store_kv(parts[1], parts[2], slots, *self.k, *self.v, self.kv_dtype, self.kv_heads)
        idx.idx_store_kv(parts[4], None, slots, *self.index_keys, None, None, "fp8_e4m3", 1)
        return parts, new

    def step(self, x, residual, request, lens, sparse=True, positions=None):
        """x, residual [R * P, hidden]; request: int32 [R], page-table row of each; lens: int32
        [R], tokens of each request with these P; positions: those of write, or None: the tokens'
        places in their requests.  Returns out [R, P, q_heads, 128], its lse,
        the new residual and the block ids (None when not sparse)."""
        R, P = request.numel(), self.drafts
        pos = lens[:, None] - P + torch.arange(P, device=self.device, dtype=torch.int32)
        row_lens = pos + 1
        slots = self.slots(request[:, None].long(), pos.long()).reshape(-1)
        parts, new = self.write(x, residual, slots, pos.reshape(-1) if positions is None else positions)
        q = parts[0].reshape(R, P, self.q_heads, DIM).contiguous()
        out, lse = torch.empty_like(q), torch.empty((R, P, self.q_heads), device=self.device)
        scale = DIM ** -0.5
        nvfp4 = self.kv_dtype == "nvfp4"
        if not sparse:
            if nvfp4:
                idx.idx_attn_paged_nvfp4(q, *self.k, *self.v, self.page_table, request, row_lens, self.kv_heads,
                                         scale, out, lse, self.attn_ws, *self.outer)
            else:
                idx.idx_attn_paged(q, *self.k, *self.v, self.kv_dtype, self.page_table, request, row_lens,
                                   self.kv_heads, scale, out, lse, self.attn_ws)
            return out, lse, new, None
        G = self.index_heads
        if self.table is None:
            iq, iq_scale, _ = self._norm(parts[3].reshape(-1, DIM), None, self.index_norm)
        else:
            iq, iq_scale = parts[3]
        ids = torch.empty((R, P * G, self.topk), dtype=torch.int32, device=self.device)
        scores = torch.empty((R, P * G, self.topk), device=self.device)
        idx.idx_score_topk(iq.reshape(R, P, G, DIM), iq_scale.reshape(R, P * G), *self.index_keys,
                           "fp8_e4m3", self.page_table, request, row_lens, P, G, self.init_blocks,
                           self.local_blocks, self.topk, ids, scores, self.score_ws)
        if nvfp4:
            idx.idx_attn_blocks_nvfp4(q, *self.k, *self.v, self.page_table, request, row_lens, ids, G,
                                      self.kv_heads, scale, out, lse, self.attn_ws, *self.outer)
        else:
            idx.idx_attn_blocks(q, *self.k, *self.v, self.kv_dtype, self.page_table, request, row_lens, ids,
                                G, self.kv_heads, scale, out, lse, self.attn_ws)
        return out, lse, new, ids


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--context", type=int, default=3000)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--steps", type=int, default=3)
    ap.add_argument("--kv-dtype", default="bf16", choices=["bf16", "fp8_e4m3", "nvfp4"])
    ap.add_argument("--rotary", action="store_true")
    a = ap.parse_args()
    R, P = a.requests, a.drafts
    layer = SparseDecodeLayer(max_requests=R, max_tokens=a.context + a.steps * P + PAGE, drafts=P,
                              kv_dtype=a.kv_dtype, rotary=a.rotary)
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda n: torch.randn((n, layer.hidden), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    request = torch.arange(R, dtype=torch.int32, device="cuda")
    pos = torch.arange(a.context, device="cuda")
    for r in range(R):      # the prompt
        layer.write(rand(a.context), rand(a.context), layer.slots(torch.full_like(pos, r), pos), pos.int())
    lens = torch.full((R,), a.context, dtype=torch.int32, device="cuda")
    for s in range(a.steps):
        lens = lens + P
        x, res = rand(R * P), rand(R * P)
        out, lse, _, ids = layer.step(x, res, request, lens)
        full, full_lse, _, _ = layer.step(x, res, request, lens, sparse=False)
        kept = torch.exp(lse - full_lse).mean().item()
        print(f"step {s}: {layer.topk} of {-(-int(lens[0]) // 128)} blocks a list hold "
              f"{100 * kept:.1f}% of the attention weight; "
              f"|sparse - full| {(out.float() - full.float()).abs().mean().item():.4f}")


if __name__ == "__main__":
    main()
