"""Trains the experts of a small expanded-layout MoE layer on one GPU.

A student layer learns to reproduce a teacher's outputs on a set of tokens: per
step the set goes forward and backward in two micro-batches (the second adds
to the weights' gradients), the gradients' norm is clipped by a device-side factor,
and one AdamW launch updates the float32 parameters and the bfloat16 copies
that the products read.

    python examples/train_experts.py --steps 60 --state-bits 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import expanded_layout_expert_gb300 as mx  # noqa: E402


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512, help="tokens per micro-batch")
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--intermediate", type=int, default=256)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--top-k", type=int, default=2)
    ap.add_argument("--lr", type=float, default=2e-3)
    ap.add_argument("--clip", type=float, default=1.0)
    ap.add_argument("--state-bits", type=int, default=32, choices=(32, 8))
    a = ap.parse_args(argv)
    T, H, I, E, K = a.tokens, a.hidden, a.intermediate, a.experts, a.top_k
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, std):
        return torch.randn(*shape, generator=g, device="cuda") * std

    shapes = ((E, 2 * I, H), H ** -0.5), ((E, H, I), I ** -0.5)
    teacher = mx.TrainableExperts(*(normal(*s, std=d).bfloat16() for s, d in shapes), K=K, max_tokens=T)
    master = [normal(*s, std=d) for s, d in shapes]
    student = mx.TrainableExperts(*(p.bfloat16() for p in master), K=K, max_tokens=T)
    opt = mx.AdamW(master, copies=student.parameters, lr=a.lr, betas=(0.9, 0.95), weight_decay=0.0,
                   state_bits=a.state_bits)
    router = normal(H, E, std=H ** -0.5)
    batches = []
    for _ in range(2):
        x = normal(T, H, std=1.0).bfloat16()
        ids, w = mx.route_topk(x.float() @ router, K)
        batches.append((x, ids, w, teacher.forward(x, ids, w).float()))
    losses = []
    for step in range(a.steps):
        loss = torch.zeros((), device="cuda")
        for micro, (x, ids, w, target) in enumerate(batches):
            diff = student.forward(x, ids, w).float() - target
            loss += diff.square().mean() / 2
            student.backward((diff / H).bfloat16(), accumulate=micro > 0)
        norm = torch.stack([d.norm() for d in student.gradients]).norm()
        opt.step(student.gradients, grad_scale=(a.clip / (norm + 1e-6)).clamp(max=1.0).reshape(1))
        losses.append(loss)
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step:4d}  loss {loss.item():.5f}")
    torch.cuda.synchronize()
    if student.status.item():
        raise RuntimeError(f"device status {student.status.item()}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    main()
