"""Train the adapters of several users over one frozen layer, then serve a batch that mixes them.

    python examples/train_and_serve.py [steps]

Training, per user: an RMS norm (lora_norm_fwd), the adapted projection (lora_linear_fwd), the
gradients of both (lora_linear_bwd, lora_norm_bwd); then one lora_adamw_step over every user's A and
B (bf16 with fp32 masters, 8-bit moments) and the norm's weight, which the users share.  Serving: the trained
adapters in an AdapterBank, one row per request, each with its user's slot (lora_linear_fwd_multi).
The targets are a teacher's outputs: the same layer with another adapter per user and another norm.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import weight_patches_gb300 as wpg  # noqa: E402

USERS, TOKENS, INNER, OUT, RANK = 4, 512, 1536, 1536, 16
EPS = 1e-6


def block8(n, device):
    """Zeroed 8-bit moments of n elements: (m, v)."""
    scales = lambda: torch.zeros((n + 255) // 256, device=device)  # noqa: E731
    return (wpg.Block8(torch.zeros(n, dtype=torch.int8, device=device), scales()),
            wpg.Block8(torch.zeros(n, dtype=torch.uint8, device=device), scales()))


def main(steps: int = 60, quiet: bool = False):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(0)
    rand = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device=dev) * std)  # noqa: E731
    bf = lambda t: t.to(torch.bfloat16)  # noqa: E731

    W = bf(rand(OUT, INNER, std=INNER ** -0.5))
    x = [bf(rand(TOKENS, INNER)) for _ in range(USERS)]
    # the teacher: its own norm weight and an adapter per user
    teacher_norm = 1 + rand(INNER, std=0.1)
    target = []
    for u in range(USERS):
        y, _ = wpg.lora_norm_fwd(x[u], teacher_norm, None, EPS, wpg.WP_NORM_RMS)
        teach = wpg.Adapter(bf(rand(RANK, INNER, std=INNER ** -0.5)), bf(rand(OUT, RANK, std=0.5)), RANK)
        target.append(wpg.lora_linear_fwd(y, W, None, [teach], out_dtype=torch.float32))

    # what is trained: A (random) and B (zero) per user, and the shared norm weight
    norm = torch.ones(INNER, device=dev)
    A = [bf(rand(RANK, INNER, std=INNER ** -0.5)) for _ in range(USERS)]
    B = [torch.zeros(OUT, RANK, dtype=torch.bfloat16, device=dev) for _ in range(USERS)]
    params = [norm] + A + B
    masters = [None] + [p.float() for p in A + B]
    moments = [block8(p.numel(), dev) for p in params]
    plan = wpg.lora_adamw_plan(params, [m for m, _ in moments], [v for _, v in moments], masters=masters)
    adapters = [wpg.Adapter(a, b, RANK) for a, b in zip(A, B)]

    losses = []
    for step in range(1, steps + 1):
        dnorm, dA, dB = torch.zeros_like(norm), [], []
        loss = torch.zeros((), device=dev)
        for u in range(USERS):
            y, stats = wpg.lora_norm_fwd(x[u], norm, None, EPS, wpg.WP_NORM_RMS)
            out = wpg.lora_linear_fwd(y, W, None, [adapters[u]], out_dtype=torch.float32)
            diff = out - target[u]
            loss += diff.square().mean() / USERS
            dy, ga, gb = wpg.lora_linear_bwd(y, W, bf(diff * (2 / TOKENS)), [adapters[u]])
            _, dw, _ = wpg.lora_norm_bwd(dy, x[u], norm, stats, wpg.WP_NORM_RMS, need_db=False)
            dnorm += dw
            dA += ga
            dB += gb
        # the gradients' norm, clipped on the device: the step reads the factor there
        grads = [dnorm] + dA + dB
        clip = (30.0 / torch.stack([g.norm() for g in grads]).norm()).clamp(max=1.0).reshape(1)
        wpg.lora_adamw_step(plan, grads, lr=4e-3, weight_decay=0.0, step=step, grad_scale_tensor=clip)
        losses.append(loss)
    losses = torch.stack(losses).tolist()
    if not quiet:
        print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps of {USERS} x {TOKENS} tokens")

    # serving: one decode row per request, any order of users, some without an adapter
    bank = wpg.AdapterBank(torch.stack(A), torch.stack(B), torch.ones(USERS, device=dev))
    slot = torch.randint(-1, USERS, (24,), generator=gen, device=dev, dtype=torch.int32)
    rows = bf(rand(len(slot), INNER))
    y, _ = wpg.lora_norm_fwd(rows, norm, None, EPS, wpg.WP_NORM_RMS)
    served = wpg.lora_linear_fwd_multi(y, W, None, bank, slot)
    worst = 0.0
    for u in range(-1, USERS):
        mine = slot == u
        if mine.any():
            own = wpg.lora_linear_fwd(y[mine], W, None, [adapters[u]] if u >= 0 else [])
            worst = max(worst, float((served[mine].float() - own.float()).abs().max() / own.float().abs().max()))
    torch.cuda.synchronize()
    assert wpg.lora_device_status() == 0
    if not quiet:
        print(f"serving: {len(slot)} rows of {USERS} users and none, within {worst:.1e} of each user's own call")
    return losses, worst


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
