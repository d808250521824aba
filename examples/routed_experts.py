"""A routed-experts block on libmxq, from the residual stream to the residual stream.

    python examples/routed_experts.py [--tokens 4096] [--train]

Forward, as a serving program runs it with experts held in MXFP4:

  1. add_rmsnorm          h = x + residual, y = norm(h)
  2. y @ router^T         the router's logits (a plain matrix product)
  3. route_topk           expert ids and weights
  4. mxq_dispatch_pack_mx the pairs sorted by expert, each row MXFP8 in the send buffer
  5. mxq_mxfp4_grouped_mm_packed   first expert product, on the payload as received
  6. silu, quantize_mxfp4, mxfp4_grouped_mm   second expert product, on 4-bit rows
  7. the rows back to their tokens, times the router's weights

--train also runs the gradients that reach the router and the norm while the experts stay
frozen: route_topk_bwd and add_rmsnorm_bwd.
"""
import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from float8_quantization_moe_amd import mxq  # noqa: E402

EPS = 1e-5


@dataclass
class Block:
    """Weights of one block: the norm's and the router's in bf16, the experts' MXFP4 codes and scales."""
    norm: torch.Tensor       # (K)
    router: torch.Tensor     # (E, K)
    bias: torch.Tensor       # (E) fp32, balances the load; for the selection only
    up: tuple                # codes (E, F, K/2), scales (E, F, K/32)
    down: tuple              # codes (E, K, F/2), scales (E, K, F/32)
    topk: int

    @staticmethod
    def random(K, F, E, topk, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def experts(n, k):
            q, s = [], []
            for _ in range(E):                       # one expert at a time: the bf16 weights are not kept
                w = (0.02 * torch.randn((n, k), generator=g, device="cuda")).to(torch.bfloat16)
                c = mxq.quantize_mxfp4(w, mxq.MXQ_SCALE_RCEIL)
                q.append(c[0])
                s.append(c[1])
            return torch.stack(q), torch.stack(s)

        return Block(norm=torch.ones(K, dtype=torch.bfloat16, device="cuda"),
                     router=(0.02 * torch.randn((E, K), generator=g, device="cuda")).to(torch.bfloat16),
                     bias=torch.zeros(E, device="cuda"), up=experts(F, K), down=experts(K, F), topk=topk)


def forward(b: Block, x: torch.Tensor, residual: torch.Tensor):
    """x, residual (M, K) bf16 -> (h, out, saved): the next residual stream, the block's output, and what
    backward needs."""
    M, K = x.shape
    E, topk, pairs = b.router.shape[0], b.topk, M * b.topk
    h, y = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(M, dtype=torch.float32, device=x.device)
    mxq.mxq_add_rmsnorm(x, residual, b.norm, EPS, h=h, y=y, rstd=rstd)
    logits = y @ b.router.t()
    ids, weights = mxq.route_topk(logits, topk, bias=b.bias, score="sigmoid", renormalize=True)

    packed = torch.empty((pairs, K + K // 32), dtype=torch.uint8, device=x.device)
    ends = torch.empty(E, dtype=torch.int32, device=x.device)
    src = torch.empty(pairs, dtype=torch.int32, device=x.device)
    work = torch.empty(mxq.mxq_dispatch_pack_workspace_bytes(M, K, topk, E), dtype=torch.uint8, device=x.device)
    mxq.mxq_dispatch_pack_mx(y, ids, E, packed, ends, src, work)

    F = b.up[0].shape[1]
    up = torch.empty((pairs, F), dtype=torch.bfloat16, device=x.device)
    mxq.mxq_mxfp4_grouped_mm_packed(packed, b.up[0], b.up[1], ends, up)
    q, s = mxq.quantize_mxfp4(torch.nn.functional.silu(up))
    rows = mxq.mxfp4_grouped_mm(q, s, b.down[0], b.down[1], ends, x_format=mxq.MXQ_FMT_E2M1)

    # each pair's row; pairs that were dropped (id -1) have none and weight 0
    place = torch.full((pairs + 1,), pairs, dtype=torch.int64, device=x.device)
    place[torch.where(src >= 0, src, pairs).long()] = torch.arange(pairs, device=x.device)
    rows = torch.cat((rows, torch.zeros_like(rows[:1])))
    per_pair = rows[place[:pairs]].view(M, topk, K)
    out = (weights.unsqueeze(-1) * per_pair.float()).sum(1).to(x.dtype)
    return h, out, (h, rstd, y, logits, ids, per_pair)


def backward(b: Block, saved, dh: torch.Tensor, dout: torch.Tensor):
    """Gradients of the input (of x and of residual alike), the norm's weight and the router, with the experts
    frozen and their rows' dependence on y left out (the router's path only)."""
    h, rstd, y, logits, ids, per_pair = saved
    dweights = (dout.float().unsqueeze(1) * per_pair.float()).sum(-1)
    dlogits = mxq.route_topk_bwd(logits, ids, dweights, score="sigmoid", renormalize=True)
    drouter = dlogits.t() @ y
    dy = dlogits @ b.router
    dx, dnorm = mxq.add_rmsnorm_bwd(h, b.norm, rstd, dy, dh)
    return dx, dnorm, drouter


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--ffn", type=int, default=8192)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--topk", type=int, default=2)
    ap.add_argument("--train", action="store_true")
    a = ap.parse_args()
    b = Block.random(a.hidden, a.ffn, a.experts, a.topk)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    residual = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for step in range(4):
        start.record()
        h, out, saved = forward(b, x, residual)
        if a.train:
            dx, dnorm, drouter = backward(b, saved, torch.ones_like(h), out)
        stop.record()
        torch.cuda.synchronize()
        print(f"step {step}: {start.elapsed_time(stop):.3f} ms, |out| {out.float().norm().item():.4f}"
              + (f", |dx| {dx.float().norm().item():.4f}, |drouter| {drouter.float().norm().item():.4f}" if a.train else ""),
              flush=True)


if __name__ == "__main__":
    main()
