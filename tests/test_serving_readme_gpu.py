"""The serving example of the README, as it stands there, against the definitions in 64 bits."""
import os
import re

import pytest
import torch

import exact_io_aware_52_b200 as fa
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
B, H, H_KV, D, PAGE = 3, 8, 2, 128, 64
SCALE = D ** -0.5


def dev():
    return torch.device("cuda:0")


def blocks():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    text = open(path).read()
    return re.findall(r"```python\n(.*?)```", text[text.index("## Serving"):], re.S)


class Run:
    """The variables of the example, and the keys, values and queries of every token so far."""

    def __init__(self, room):
        g = self.g = torch.Generator().manual_seed(80)
        codes = torch.zeros(B * room + 2, H_KV, PAGE, D, dtype=torch.uint8, device=dev())
        table = torch.randperm(B * room + 2, generator=g)[:B * room].view(B, room).to(torch.int32).to(dev())
        scales = torch.zeros(B * room + 2, H_KV, device=dev())
        self.env = dict(k=codes, v=codes.clone(), k_scale=scales, v_scale=scales.clone(), table=table, scale=SCALE)
        self.q = [torch.zeros(H, 0, D, dtype=F64)] * B
        self.w = ref.angles(D, scaling="parts", factor=8.0, original_length=4096.0)

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device=dev())

    def tokens(self, lengths):
        """New tokens for each sequence, of which lengths[b] count; their queries are kept as turned in 64 bits."""
        N = max(lengths)
        x = torch.randn(B, N, H + 2 * H_KV, D, generator=self.g).to(BF16)
        for b, n in enumerate(lengths):
            have = self.q[b].shape[1]
            turned = ref.rope(x[b:b + 1, :n, :H].transpose(1, 2), torch.arange(have, have + n)[None], self.w)[0]
            self.q[b] = torch.cat([self.q[b], turned], 1)
        q, k, v = (t.transpose(1, 2).to(dev()) for t in (x[:, :, :H], x[:, :, H:H + H_KV], x[:, :, H + H_KV:]))
        return q, k, v

    def check(self, o, b, n):
        """o: the last n tokens of sequence b.  The turned queries are rounded to bf16 (2^-8 of each), so scores err by
        2^-8 sum |q k| scale; the attention over contiguous keys rounds its weights to bf16 (2^-8), and a bf16 output is off
        by 2^-8.  The fp32 steps (below 2^-10 in all) are in the second 2^-8 of the weights' term."""
        e = self.env
        have = self.q[b].shape[1]
        kk = ref.dense(e["k"].view(ref.E4M3).float().cpu(), e["k_scale"].cpu(), e["table"].cpu(), b, have, PAGE)
        vv = ref.dense(e["v"].view(ref.E4M3).float().cpu(), e["v_scale"].cpu(), e["table"].cpu(), b, have, PAGE)
        want, _, oabs, mag = ref.attend(self.q[b][None, :, have - n:], [kk], [vv], [have], True, SCALE)
        bound = (2 * 2.0 ** -8 * mag[..., None] + 2.0 ** -7) * (oabs + want.abs()) + 2.0 ** -8 * want.abs()
        assert ((o.cpu().to(F64) - want[0]).abs() <= bound[0]).all()


def test_the_example():
    assert len(blocks()) == 3, "new prompts, prompts over what is held, single tokens"
    first, more, token = blocks()
    run = Run(room=8)
    env = run.env
    lengths = [100, 1, 257]
    env["q"], env["new_k"], env["new_v"] = run.tokens(lengths)
    env["lengths"] = run.ints(lengths)
    exec(first, env)
    for b, n in enumerate(lengths):
        run.check(env["o"][b, :, :n], b, n)
    held = lengths
    lengths = [33, 130, 64]
    env["q"], env["new_k"], env["new_v"] = run.tokens(lengths)
    env["lengths"], env["held"] = run.ints(lengths), run.ints(held)
    exec(more, env)
    for b, n in enumerate(lengths):
        run.check(env["outputs"][b][0], b, n)
    held = [a + b for a, b in zip(held, lengths)]
    for _ in range(3):
        env["q1"], env["k1"], env["v1"] = run.tokens([1] * B)
        env["held"] = run.ints(held)
        exec(token, env)
        for b in range(B):
            run.check(env["o"][b], b, 1)
        held = [n + 1 for n in held]


def test_prompts_over_what_is_held_by_single_tokens():
    """The same chunk attended by the call for a few tokens, sequences of the same number of new tokens."""
    run = Run(room=8)
    env = run.env
    rotary = fa.Rotary(D, scaling="parts", factor=8.0, original_length=4096)
    cache = fa.PagedCache(env["k"], env["v"], env["k_scale"], env["v_scale"], env["table"])
    held = [0, 0, 0]
    for lengths in ([90, 90, 90], [7, 7, 7], [20, 20, 20]):
        q, k, v = run.tokens(lengths)
        start = run.ints(held)
        fa.cache_append(cache, k, v, start, rotary=rotary)
        q = fa.rope(rotary, q, pos=start.view(-1, 1) + torch.arange(q.shape[2], dtype=torch.int32, device=dev()))
        held = [n + m for n, m in zip(held, lengths)]
        o, _ = fa.cache_attention(cache, q, run.ints(held), True, SCALE)
        for b, n in enumerate(lengths):
            run.check(o[b], b, n)
