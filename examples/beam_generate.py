"""Beam search over a hybrid model of random weights: layers of the modal Hyena
operator and of linear attention in turn, a prompt a group, on one MI355X.

    python3 examples/beam_generate.py [--layers 4] [--width 512] [--groups 4] [--beams 4] [--prompt 300] [--steps 32]
"""

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def random_model(torch, layers, width, vocab, heads=8, modes=16, seed=0, device="cuda"):
    from distilled_modal_ssm_amd.hybrid import HybridLM
    from workloads.generate import ModalParams
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    weight = lambda n, k: (rn(n, k) / k ** 0.5).to(device, torch.bfloat16)  # noqa: E731
    out = []
    for i in range(layers):
        if i % 2 == 0:
            r, th = 0.5 + 0.49 * torch.rand(heads, modes, generator=g), 3.14159 * torch.rand(heads, modes, generator=g)
            poles = torch.stack([r * th.cos(), r * th.sin()], -1)
            op = ("hyena", ModalParams(poles.numpy(), (rn(heads, modes, 2) / (2 * modes) ** 0.5).numpy(),
                                       rn(heads).numpy()))
        else:  # heads that forget over 3 to 300 tokens
            op = ("attention", -torch.exp(-torch.linspace(1.1, 5.7, heads)).to(device))
        out.append((*op, weight(3 * width, width), weight(width, width)))
    return HybridLM(out, weight(vocab, width) * width ** 0.5, 3 * weight(vocab, width), device=device)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("layers", 4), ("width", 512), ("groups", 4), ("beams", 4), ("prompt", 300), ("steps", 32),
                        ("vocab", 8192)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    import torch
    model = random_model(torch, a.layers, a.width, a.vocab)
    prompts = torch.randint(0, a.vocab, (a.groups, a.prompt), generator=torch.Generator().manual_seed(1)).cuda()
    model.generate(prompts, a.beams, 2)  # first use of the library and of torch's memory
    torch.cuda.synchronize()
    t = time.perf_counter()
    tokens, scores = model.generate(prompts, a.beams, a.steps, end_token=0)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.groups} prompts x {a.beams} beams, {a.prompt} + {a.steps} tokens, {a.layers} layers of {a.width}: {t * 1e3:.1f} ms")
    print("best of the first prompt:", tokens[0, 0].tolist(), f"log probability {float(scores[0, 0]):.3f}")


if __name__ == "__main__":
    main()
