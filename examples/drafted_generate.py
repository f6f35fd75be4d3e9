"""Generation with drafts over hybrid models of random weights: gated recurrences with now and then a
layer of linear attention, projections in 8 bits, on one MI355X; a model of one layer drafts.

    python3 examples/drafted_generate.py [--layers 6] [--width 512] [--batch 8] [--drafts 4] [--prompt 300] [--steps 64]
"""

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def random_model(torch, kinds, width, vocab, heads=8, modes=16, seed=0, like=None, device="cuda"):
    """kinds: the layers' ("hyena", "attention", "gated").  like: another model whose embedding and head, cut to
    this width, make the two models agree now and then."""
    from distilled_modal_ssm_amd.hybrid import HybridLM
    from workloads.generate import ModalParams
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    weight = lambda n, k: (rn(n, k) / k ** 0.5).to(device, torch.bfloat16)  # noqa: E731
    out = []
    for kind in kinds:
        if kind == "hyena":
            r, th = 0.5 + 0.49 * torch.rand(heads, modes, generator=g), 3.14159 * torch.rand(heads, modes, generator=g)
            poles = torch.stack([r * th.cos(), r * th.sin()], -1)
            p = ModalParams(poles.numpy(), (rn(heads, modes, 2) / (2 * modes) ** 0.5).numpy(), rn(heads).numpy())
        elif kind == "attention":  # heads that forget over 3 to 300 tokens
            p = -torch.exp(-torch.linspace(1.1, 5.7, heads)).to(device)
        else:
            p = "norm"
        out.append((kind, p, weight(3 * width, width), weight(width, width)))
    if like is not None:
        cut = lambda w: w[:, :width].contiguous()  # noqa: E731
        return HybridLM(out, cut(like.embedding), cut(like.head), device=device)
    return HybridLM(out, weight(vocab, width) * width ** 0.5, 3 * weight(vocab, width), device=device)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("layers", 6), ("width", 512), ("batch", 8), ("drafts", 4), ("prompt", 300), ("steps", 64),
                        ("vocab", 8192)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    import torch
    kinds = ["attention" if i % 3 == 2 else "gated" for i in range(a.layers)]
    model = random_model(torch, kinds, a.width, a.vocab)
    draft = random_model(torch, ["gated"], 64, a.vocab, seed=1, like=model).quantized()
    model = model.quantized()
    prompts = torch.randint(0, a.vocab, (a.batch, a.prompt), generator=torch.Generator().manual_seed(1)).cuda()
    model.generate_drafted(prompts, draft, 2, drafts=a.drafts)  # first use of the library and of torch's memory
    torch.cuda.synchronize()
    t = time.perf_counter()
    tokens, rate = model.generate_drafted(prompts, draft, a.steps, drafts=a.drafts, temperature=4.0)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.batch} prompts, {a.prompt} + {a.steps} tokens, {a.layers} layers of {a.width}: {t * 1e3:.1f} ms, "
          f"{rate:.2f} of the drafts kept")
    print("first prompt:", tokens[0].tolist())


if __name__ == "__main__":
    main()
